// Linear attention with a decay for each head, for gfx950:
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale * q_t^T S_t.
#include "mixers.h"
#include "mixer_types.h"

namespace w4a16 {

namespace {

// ---- one token per request ---------------------------------------------------------------------
// The state is read once, updated in registers, used and written once: 8 bytes of HBM traffic per
// element and nothing else of that order. A work-group owns CV columns of one head's state; a
// thread holds DK / RG rows of four columns, all loaded before the first is used. The products
// with q are summed over the row groups by lane swaps inside a wave and through LDS across waves.
//
// Few heads and requests leave CUs idle, so below 128 of them a work-group owns 32 columns; from there on
// a whole state, with streaming loads and stores (a model's other layers push it out of every cache
// before the next token). Graphs of 48 layers of 32 heads of 128 x 128, us per layer, split / whole /
// whole streaming: 1 request 3.1 / 3.8 / 4.1, 2 requests 3.6 / 4.1 / 4.3, 4 requests 5.9 / 6.3 / 4.8,
// 16 requests 16.8 / 15.9 / 12.4, 256 requests 215 / 211 / 183 (5.9 TB/s).
constexpr int kStepThreads = 256;

template <class Type, int DK, int DV, int CV, bool STREAM>
__global__ __launch_bounds__(kStepThreads) void linear_step_kernel(LinearArgs a)
{
    typedef typename Type::T T;
    constexpr int LPR = CV / 4, RG = kStepThreads / LPR, ROWS = DK / RG, PARTS = DV / CV;
    static_assert(ROWS >= 1 && RG * ROWS == DK, "rows divide over the row groups");
    __shared__ float qs[DK], ks[DK];
    __shared__ f32x4 part[kStepThreads / 64][LPR];
    const int tid = threadIdx.x, col = tid % LPR, rg = tid / LPR;
    const int h = blockIdx.x / PARTS, c0 = (blockIdx.x % PARTS) * CV + col * 4;
    const int64_t b = blockIdx.y;
    const int64_t slot = a.cu ? a.cu[b] : b;
    T *o = (T *)a.out + b * a.ldo + h * a.hso + c0;
    if (slot < 0 || slot >= a.num_states) {   // no state: a zero row (whole work-group)
        if (rg == 0)
            for (int e = 0; e < 4; ++e)
                o[e] = Type::from(0.0f);
        return;
    }
    const int64_t base = (slot * a.H + h) * (int64_t)(DK * DV) + (int64_t)rg * DV + c0;
    f32x4 s[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        s[r] = STREAM ? __builtin_nontemporal_load((const f32x4 *)(a.state_in + base + r * RG * DV))
                      : *(const f32x4 *)(a.state_in + base + r * RG * DV);
    const int hk = h / (a.H / a.Hk);
    if (tid < DK) {
        qs[tid] = a.scale * Type::f(((const T *)a.q)[b * a.ldq + hk * a.hsq + tid]);
        ks[tid] = Type::f(((const T *)a.k)[b * a.ldk + hk * a.hsk + tid]);
    }
    const T *vp = (const T *)a.v + b * a.ldv + h * a.hsv + c0;
    f32x4 v, acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = Type::f(vp[e]);
    const float decay = expf(a.g[b * a.ldg + h * a.hsg]);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float k = ks[rg + r * RG], q = qs[rg + r * RG];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[r][e] = fmaf(k, v[e], decay * s[r][e]);
            acc[e] = fmaf(q, s[r][e], acc[e]);
        }
        if (STREAM)
            __builtin_nontemporal_store(s[r], (f32x4 *)(a.state_out + base + r * RG * DV));
        else
            *(f32x4 *)(a.state_out + base + r * RG * DV) = s[r];
    }
#pragma unroll
    for (int d = LPR; d < 64; d <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc[e] += __shfl_xor(acc[e], d);
    if ((tid & 63) < LPR)
        part[tid >> 6][col] = acc;
    __syncthreads();
    if (rg == 0) {
        f32x4 sum = part[0][col];
#pragma unroll
        for (int w = 1; w < kStepThreads / 64; ++w)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum[e] += part[w][col][e];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = Type::from(sum[e]);
    }
}

template <class Type, int DK, int DV>
void step_of(const LinearArgs &a, hipStream_t stream)
{
    if ((int64_t)a.B * a.H < 128)
        linear_step_kernel<Type, DK, DV, 32, false><<<dim3(a.H * (DV / 32), a.B), dim3(kStepThreads), 0, stream>>>(a);
    else
        linear_step_kernel<Type, DK, DV, DV, true><<<dim3(a.H, a.B), dim3(kStepThreads), 0, stream>>>(a);
}

template <class Type>
void step_typed(const LinearArgs &a, hipStream_t stream)
{
    if (a.Dk == 64)
        a.Dv == 64 ? step_of<Type, 64, 64>(a, stream) : step_of<Type, 64, 128>(a, stream);
    else
        a.Dv == 64 ? step_of<Type, 128, 64>(a, stream) : step_of<Type, 128, 128>(a, stream);
}

// ---- packed sequences ----------------------------------------------------------------------------
// Sequences are cut into segments of L tokens and those into chunks of 64. With b_i the running sum of
// the log decays inside a chunk (its own token included) and S the state before it, per head:
//   o_i = scale * (e^{b_i} q_i^T S + sum_{j<=i} e^{b_i - b_j} (q_i . k_j) v_j)
//   S  <- e^{b_63} S + sum_j k_j (e^{b_63 - b_j} v_j)^T
// All products are MFMA 16x16x32. Of the state a wave owns a quarter of the Dv columns, in registers in
// float32; of the outputs a tile of 16 tokens, so scores are formed once. k, the state rounded for q S and
// the rows of v in operand order are shared through LDS, two barriers per chunk; the next chunk's rows
// are on their way during the products.
//
// Operands never cross lanes. A contraction's order is free as long as both operands agree:
//   scores are formed transposed (k q^T): a lane then holds token i = lane % 16 of a tile of queries and
//   the keys 4g..4g+3 (g = lane / 16) of a tile of 16; two such tiles are the first operand of the
//   product with v for the keys {4g..4g+3, 16 + 4g..16 + 4g+3} of 32, and v rows are taken in that order;
//   the state's tile j has rows dk = EK m + j (EK = Dk / 16, m = 4g + r in a lane), as a lane's EK
//   consecutive values of k rows give them; two tiles are the second operand of the product q S, whose
//   first operand, q at dk = EK (4g + r) + {j, j + 1}, are words that the lane has loaded for the scores.
//
// Roundings, all to the type for a matrix product (float32 products would take eight times the matrix
// units' time): scores with their decay; S in q S, where the outputs' own rounding is as large; and
// e^{b_63 - b_j} v_j, kept as a sum of three bfloat16 or two float16 values (24 and 22 bits) where the
// result reaches a returned state or another segment, else of two bfloat16 or one float16. With that
// outputs of 32768 bfloat16 tokens are off by 2.35e-3 of their norm (2.57e-3 with one bfloat16 value,
// 1.66e-3 by their own rounding alone; S in float16 as well would make it 2.0e-3 for another 20 us of 400),
// states by 5e-7. Decays are summed in float64 over a chunk; the scores' take the sums in float32, off by
// 2^-24 of their size. A log decay below -193 counts as that: with growth by up to e^88, float32's
// largest, behind it that is e^-105, zero in float32, and so a state that is cleared by -inf costs its neighbours
// few digits.
//
// The scale comes last: with e^{b_i} it could leave float32's range where the output does not.
//
// Scores have more range than float16. Those of a query are bounded by its norm, the chunk's largest norm of a
// key (from sums of squares, which also show what is not finite) and the largest e^{b_i - b_j} where decays are
// positive; the power of two that brings this bound to 2^15 goes with e^{b_i} and is taken back from the
// query's sum. Scores below 2^-29 of the bound lose digits. (Costs 0.3 us of 43 for nine sequences of up to 300
// tokens.)
//
// So has e^{b_63 - b_j} v_j (decays of a whole segment may stand there), and its second term, 2^-11 of the first,
// is soon among the subnormals. Column by column the state is therefore held as 2^up times itself, with the
// power that brings the chunk's largest |v| times the largest e^{b_63 - b_j} to 2^15: 22 bits down to 2^-17 of
// that, 11 down to 2^-29. The factor goes with the decay of the state; a sum over chunks keeps its smallest
// one. (Terms that only get 2^11 times their remainders, against k times 2^-11, put that among the subnormals for
// k below 0.1.) With it nine sequences of up to 300 tokens take 44.4 us instead of 43.3.
//
// One segment per sequence needs one launch. Longer ones take three: what each segment adds to a state
// (k and v read once), the states before every segment and after the last (a running sum over segments),
// then the outputs of all segments side by side.
//
// What bounds it (128 x 128, 32 heads of 32768 bfloat16 tokens, 402 us in all): the outputs move 1.07 GB in
// 240 to 255 us (4.2 to 4.5 TB/s, where a copy of 4 GiB reaches 4.7); the segments' sums read 0.54 GB in 171 us, with
// the vector units busy for 44 and the matrix units for 32 % of it (the three terms). A short sequence
// is bound by the chain of its chunks, 4.4 us each (float16 4.8): two barriers, and between them the products of a
// wave, which are alone on their SIMD; before them stand 8.6 us of launch and states read and written.
constexpr int kChunk = 64;
constexpr int kSegmentThreads = 256;
constexpr float kNone = -193.0f;
constexpr int kMostUp = 100;
constexpr int kWaveSeqs = 64;   // up to here every wave finds its segment by itself

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma(Bf16, u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(Fp16, u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack2(Bf16, float a, float b)
{
    const bf16x2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t pack2(Fp16, float a, float b)
{
    const f16x2 r = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float low(Bf16, uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float high(Bf16, uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
__device__ __forceinline__ float low(Fp16, uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[0]; }
__device__ __forceinline__ float high(Fp16, uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[1]; }

// Rounds a pair and keeps what that leaves in its place, for the next term. The remainder goes by the bits
// that the product gets: left to itself, the compiler rounds v * d once for one use and twice (float32
// first) for the other.
template <class Type>
__device__ __forceinline__ uint32_t take(Type t, float &a, float &b)
{
    uint32_t both = pack2(t, a, b);
    asm volatile("" : "+v"(both));
    a -= low(t, both);
    b -= high(t, both);
    return both;
}
// As many values of the type as hold a float32's digits, or nearly.
template <class Type>
struct Terms {
    static constexpr int count = __is_same(Type, Bf16) ? 3 : 2;
};

// The larger magnitudes (without signs) of two pairs of float16 values; NaN is above infinity.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t larger_pair(uint32_t x, uint32_t y)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, x),
                                                                  __builtin_bit_cast(u16x2, y)));
}
// The same over the four lanes that share lane % 16; and a sum.
__device__ __forceinline__ uint32_t larger_pair4(uint32_t x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = larger_pair(r[0], r[1]);
    const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return larger_pair(s[0], s[1]);
}
__device__ __forceinline__ float sum4(float v)
{
    uint32_t x = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    v = __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
    x = __builtin_bit_cast(uint32_t, v);
    const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return __builtin_bit_cast(float, (uint32_t)s[0]) + __builtin_bit_cast(float, (uint32_t)s[1]);
}
// acc plus the squares of a pair. (Should subnormal values count as zeros there, root_exponent covers it.)
__device__ __forceinline__ float add_squares(uint32_t w, float acc)
{
    const f16x2 x = __builtin_bit_cast(f16x2, w);
    return __builtin_amdgcn_fdot2(x, x, acc, false);
}
// e with sqrt(sum) <= 2^e, where up to 2^7 float16 subnormals may be missing in the sum.
__device__ __forceinline__ int32_t root_exponent(float sum)
{
    return (__builtin_amdgcn_frexp_expf(fmaxf(sum, 0x1p-21f)) + 1) >> 1;
}
__device__ __forceinline__ float power(int32_t e) { return __builtin_ldexpf(1.0f, e); }

// Rows of a chunk as a buffer: `n` of them, `ld` elements apart and `width` long. What lies past the last
// row's end reads as zeros and isn't written, so that a chunk's loads need no branches: where one comes
// between a load and its use, the compiler waits for every load in flight.
typedef __amdgpu_buffer_rsrc_t Rows;
__device__ __forceinline__ Rows rows_of(const void *p, int32_t n, int32_t ld, int width, int bytes)
{
    const uint32_t count = min(max(n, 0), kChunk);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0,
                                             count ? ((count - 1) * (uint32_t)ld + width) * bytes : 0, 0x00027000);
}
template <int N>
struct Words;
template <>
struct Words<1> {
    typedef uint32_t T __attribute__((ext_vector_type(1)));
    static __device__ __forceinline__ T load(Rows r, uint32_t at)
    {
        return T{__builtin_amdgcn_raw_buffer_load_b32(r, at, 0, 0)};
    }
};
template <>
struct Words<2> {
    typedef u32x2 T;
    static __device__ __forceinline__ T load(Rows r, uint32_t at)
    {
        return __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0);
    }
};
// A value that is not known to stay the same: sums with it are made where they are used, instead of held in
// registers for the whole loop.
__device__ __forceinline__ uint32_t fresh(uint32_t x)
{
    asm volatile("" : "+v"(x));
    return x;
}
__device__ __forceinline__ int32_t fresh_scalar(int32_t x)
{
    asm volatile("" : "+s"(x));
    return x;
}
__device__ __forceinline__ u32x4 load4(Rows r, uint32_t at)
{
    return __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
}

template <int N>
struct Count {
    static constexpr int value = N;
};

// Keeps a branch that is hardly ever taken a branch, rather than selects on the way past it.
__device__ __forceinline__ void rare() { asm volatile("; rare"); }

// acc plus both bfloat16 values times zero: NaN from the first one on that is not finite.
__device__ __forceinline__ float times_zero(uint32_t w, float acc)
{
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), bf16x2{(__bf16)0.0f, (__bf16)0.0f}, acc, false);
}

// The sign's place is set for a value that is not finite (its exponent field, plus one unit of it).
__device__ __forceinline__ uint32_t odd_bits(Bf16, uint32_t w) { return (w & 0x7FFF7FFFu) + 0x00800080u; }
__device__ __forceinline__ uint32_t odd_bits(Fp16, uint32_t w) { return (w & 0x7FFF7FFFu) + 0x04000400u; }
// The pair with zeros in the place of such values.
template <class Type>
__device__ __forceinline__ uint32_t only_finite(Type t, uint32_t w)
{
    const uint32_t o = odd_bits(t, w);
    return w & ((o & 0x8000u ? 0u : 0xFFFFu) | (o & 0x80000000u ? 0u : 0xFFFF0000u));
}

// The largest magnitude of two values and one found before. (fmaxf would first quiet each value.)
__device__ __forceinline__ float larger(float most, float x, float y)
{
    asm("v_max3_f32 %0, %0, |%1|, |%2|" : "+v"(most) : "v"(x), "v"(y));
    return most;
}
// The largest of all lanes, of values without a sign: as integers, rotated inside rows of 16, then rows swapped.
template <int ROTATE>
__device__ __forceinline__ uint32_t rotated_max(uint32_t x)
{
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + ROTATE, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_max(float v)
{
    uint32_t x = rotated_max<8>(__builtin_bit_cast(uint32_t, v));
    x = rotated_max<1>(rotated_max<2>(rotated_max<4>(x)));
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = max(r[0], r[1]);
    const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return __builtin_bit_cast(float, max(s[0], s[1]));
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, true);
    return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Running sum over the 64 lanes: shifts by 1, 2, 4, 8 inside rows of 16, then the rows' ends.
__device__ __forceinline__ double running_sum(double x)
{
    x = dpp_add<0x111, 0xF>(x);
    x = dpp_add<0x112, 0xF>(x);
    x = dpp_add<0x114, 0xF>(x);
    x = dpp_add<0x118, 0xF>(x);
    x = dpp_add<0x142, 0xA>(x);
    return dpp_add<0x143, 0xC>(x);
}

struct Cuts {           // how a call's sequences are cut
    int32_t L;          // tokens per segment, a multiple of kChunk
    int32_t inner;      // segments of sequences that have several, at most
    int32_t slots;      // states in the workspace: one more than segments for each such sequence
    int32_t *maps;      // more than kWaveSeqs sequences: [3][num_seqs + 1] starts; segments, and inner ones, before each
    float *states;      // [slots][H][Dk][Dv]
    float *decays;      // [slots][H]: a segment's whole decay
};

struct Segment {
    int32_t seq, index, last;   // sequence, number inside it, whether it is the sequence's last one
    int32_t t0, t1;             // tokens
    int32_t slot;               // state slot of the segment, where the sequence has several
    bool single;                // it is the only one of its sequence
};

// Slots before sequence b: its inner segments before, and one for each sequence that has them.
__device__ __forceinline__ int32_t slot_before(int32_t several, int32_t segments, int32_t b)
{
    return several + b - (segments - several);
}

// One sequence per lane, kWaveSeqs of them at most: its tokens, its segments, those of the sequences
// before it, and how many of these have one segment only and need no slots.
struct LaneCut {
    int32_t start, end, n, before, ones;
};

__device__ __forceinline__ LaneCut lane_cut(const LinearArgs &a, const Cuts &c)
{
    const int lane = threadIdx.x & 63;
    const int at = min(lane, a.B);
    LaneCut s;
    s.start = min(max(a.cu[at], 0), a.T);
    s.end = min(max(a.cu[min(at + 1, a.B)], 0), a.T);
    for (int d = 1; d < 64; d <<= 1) {   // running maximum of the starts
        const int32_t o = __shfl_up(s.start, d);
        if (lane >= d)
            s.start = max(s.start, o);
    }
    s.end = max(s.start, s.end);
    s.n = lane < a.B ? max(1, (int32_t)(((int64_t)(s.end - s.start) + c.L - 1) / c.L)) : 0;
    const uint64_t single = __ballot(s.n == 1);
    s.ones = __builtin_popcountll(single & ((1ull << lane) - 1));
    s.before = s.n;
    if (__ballot(s.n > 1)) {
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(s.before, d);
            if (lane >= d)
                s.before += o;
        }
        s.before -= s.n;
    } else {   // one each
        s.before = lane;
    }
    return s;
}

// Segment number `unit` of all (inner: of those of sequences that have several). A sequence without
// tokens has one segment. False past the end.
__device__ bool find_segment(const LinearArgs &a, const Cuts &c, int unit, bool inner, Segment *s)
{
    int32_t start, end, slot0;
    if (!a.cu) {
        s->seq = 0;
        start = 0;
        end = a.T;
        s->index = unit;
        slot0 = 0;
        const int32_t n = max(1, (int32_t)(((int64_t)a.T + c.L - 1) / c.L));
        if (unit >= n || (inner && n == 1))
            return false;
    } else if (a.B <= kWaveSeqs) {
        const int lane = threadIdx.x & 63;
        const LaneCut cut = lane_cut(a, c);
        const int32_t key = inner ? cut.before - cut.ones : cut.before;
        const uint64_t hit = __ballot(lane < a.B && key <= unit);
        const int seq = 63 - __builtin_clzll(hit);   // lane 0's key is 0
        s->seq = seq;
        start = __builtin_amdgcn_readlane(cut.start, seq);
        end = __builtin_amdgcn_readlane(cut.end, seq);
        s->index = unit - __builtin_amdgcn_readlane(key, seq);
        slot0 = __builtin_amdgcn_readlane(slot_before(cut.before - cut.ones, cut.before, lane), seq);
        const int32_t segments = __builtin_amdgcn_readlane(cut.n, seq);
        if (s->index >= segments || (inner && segments == 1))
            return false;
    } else {
        const int32_t *starts = c.maps, *segments = starts + a.B + 1, *several = segments + a.B + 1;
        const int32_t *key = inner ? several : segments;
        if (unit >= key[a.B])
            return false;
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (key[mid] <= unit)
                lo = mid;
            else
                hi = mid;
        }
        s->seq = lo;
        start = starts[lo];
        end = max(start, min(max(a.cu[lo + 1], 0), a.T));
        s->index = unit - key[lo];
        slot0 = slot_before(several[lo], segments[lo], lo);
    }
    s->slot = slot0 + s->index;
    s->t0 = (int32_t)min((int64_t)start + (int64_t)s->index * c.L, (int64_t)end);
    s->last = end - s->t0 <= c.L;
    s->t1 = s->last ? end : s->t0 + c.L;
    s->single = s->last && s->index == 0;
    return true;
}

// The running sums that find_segment searches, for many sequences: one work-group.
constexpr int kMapThreads = 1024;
__global__ __launch_bounds__(kMapThreads) void linear_maps_kernel(LinearArgs a, Cuts c)
{
    __shared__ int32_t wave_x[kMapThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int32_t *starts = c.maps, *segments = starts + a.B + 1, *several = segments + a.B + 1;
    __shared__ int32_t wave_one[kMapThreads / 64];
    int32_t top = 0, sum = 0, ones = 0;   // before this round of kMapThreads sequences
    for (int b0 = 0; b0 < a.B; b0 += kMapThreads) {
        const int b = b0 + tid;
        int32_t x = b < a.B ? min(max(a.cu[b], 0), a.T) : 0;
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(x, d);
            if (lane >= d)
                x = max(x, o);
        }
        __syncthreads();
        if (lane == 63)
            wave_x[wave] = x;
        __syncthreads();
        x = max(x, top);
        for (int w = 0; w < kMapThreads / 64; ++w) {
            if (w < wave)
                x = max(x, wave_x[w]);
            top = max(top, wave_x[w]);
        }
        int32_t n = 0;
        if (b < a.B) {
            const int32_t y = max(x, min(max(a.cu[b + 1], 0), a.T));
            n = max(1, (int32_t)(((int64_t)(y - x) + c.L - 1) / c.L));
        }
        int32_t s = n;
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(s, d);
            if (lane >= d)
                s += o;
        }
        const uint64_t single = __ballot(n == 1);
        int32_t one = ones + __builtin_popcountll(single & ((1ull << lane) - 1));
        __syncthreads();
        if (lane == 63) {
            wave_x[wave] = s;
            wave_one[wave] = __builtin_popcountll(single);
        }
        __syncthreads();
        s += sum - n;
        for (int w = 0; w < kMapThreads / 64; ++w) {
            if (w < wave) {
                s += wave_x[w];
                one += wave_one[w];
            }
            sum += wave_x[w];
            ones += wave_one[w];
        }
        if (b < a.B) {
            starts[b] = x;
            segments[b] = s;
            several[b] = s - one;
        }
    }
    if (tid == 0) {
        segments[a.B] = sum;
        several[a.B] = sum - ones;
    }
}

template <class Type, int DK, int DV, bool OUT>
struct ChunkLds {
    static constexpr bool fp16 = __is_same(Type, Fp16);
    uint16_t k[kChunk][DK + 8];
    u32x4 v[2][DV / 16][64];                          // second operands: half of the chunk, column
    u32x4 s[OUT ? DK / 32 : 1][OUT ? DV / 16 : 1][64];   // and the state's: pair of tiles, column
    float b[kChunk], eb[kChunk], ed[kChunk];          // per token: b (log2), e^b (bfloat16), e^(b_63 - b)
    // float16: by how much a wave's part of s is smaller; sums of squares of k; largest magnitudes of v (half
    // of the chunk, column in pairs); a wave's queries' factors, before and after the products with v
    float grow[kSegmentThreads / 64], squares[kSegmentThreads / 64];
    uint32_t most_v[fp16 ? 2 : 1][16][DV / 32];
    float row[fp16 && OUT ? kSegmentThreads / 64 : 1][16], last[fp16 && OUT ? kSegmentThreads / 64 : 1][16];
    // What is not finite, in even and odd chunks: whether, first token of k, dims of k, first tokens of v
    uint32_t odd[2], bad_token[2], bad_dims[2][DK / 32], bad_column[2][DV];
};

// One segment of one head. OUT: its outputs, and the final state where it is the sequence's only one;
// otherwise (inner segments) what it adds to the state, and its whole decay. REST: the state is kept
// to the digits of what is returned, or starts others. (With a final state from the last one of
// several as well, those few work-groups alone took 340 us where the others took 230.)
template <class Type, int DK, int DV, bool OUT, bool REST>
__device__ __forceinline__ void run_segment(const LinearArgs &a, const Cuts &cuts, const Segment &seg,
                                            ChunkLds<Type, DK, DV, OUT> &lds)
{
    constexpr bool fp16 = __is_same(Type, Fp16);
    // a wave owns CW of the EV columns of a lane
    constexpr int threads = kSegmentThreads, NW = threads / 64, EK = DK / 16, WK = EK / 2, EV = DV / 16, CW = EV / NW;
    constexpr int pieces = DK / 8, loads = kChunk * pieces / threads, step = threads / pieces;
    constexpr int contractions = DK / 32;
    // below 2^24
    const int32_t ldq = (int32_t)a.ldq, ldk = (int32_t)a.ldk, ldv = (int32_t)a.ldv, ldo = (int32_t)a.ldo;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4, h = blockIdx.x;
    const int hk = h / (a.H / a.Hk);
    const uint16_t *qp = (const uint16_t *)a.q + hk * a.hsq, *kp = (const uint16_t *)a.k + hk * a.hsk;
    const uint16_t *vp = (const uint16_t *)a.v + h * a.hsv;
    uint16_t *op = (uint16_t *)a.out + h * a.hso;
    const float *gp = a.g + h * a.hsg;
    const int64_t state_at = (int64_t)(4 * g * EK) * DV + EV * col + CW * wave;   // of s[0][.][0]
    const int64_t state_size = (int64_t)DK * DV;
    // This wave's tile of 16 queries: later ones have more keys, so work-groups that may share a CU take
    // them in opposite orders.
    const int it = (blockIdx.x ^ blockIdx.y) & 1 ? 3 - wave : wave;
    // This wave's share of the v operands: 2 CW columns of one half of the chunk.
    const int v_half = 2 * CW * wave / EV, v_first = 2 * CW * wave % EV;
    // A lane's part of an address, in bytes; token strides are below 2^24, so it fits 32 bits.
    const uint32_t row0 = tid / pieces, dim0 = (tid % pieces) * 8;
    const uint32_t q_lane = 2 * (col * (uint32_t)ldq + DK / 4 * g), k_lane = 2 * (row0 * (uint32_t)ldk + dim0);
    const uint32_t v_lane = 2 * (4 * g * (uint32_t)ldv + EV * col + v_first);
    const uint32_t o_lane = 2 * (4 * g * (uint32_t)ldo + EV * col);

    // s[j][c][r]: row EK (4g + r) + j, column EV col + CW wave + c
    f32x4 s[EK][CW];
    const float *from = nullptr;
    if (OUT && !seg.single)
        from = cuts.states + ((int64_t)seg.slot * a.H + h) * state_size + state_at;
    else if (OUT && a.state_in)
        from = a.state_in + ((int64_t)seg.seq * a.H + h) * state_size + state_at;
#pragma unroll
    for (int j = 0; j < EK; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float x[CW] = {};
            if (from)
                __builtin_memcpy(x, __builtin_assume_aligned(from + (int64_t)(EK * r + j) * DV, 4 * CW), 4 * CW);
#pragma unroll
            for (int c = 0; c < CW; ++c)
                s[j][c][r] = x[c];
        }

    // float16: s is held as 2^up times itself, column by column
    int32_t up[CW];
#pragma unroll
    for (int c = 0; c < CW; ++c)
        up[c] = OUT ? 0 : kMostUp;

    u32x4 q[contractions];   // dims (Dk / 4) g .. + Dk / 4 of token 16 it + col
    u32x4 kn[loads];
    typename Words<CW>::T vn[8];
    float gn = 0.0f;
    auto fetch_q = [&](int32_t t) {   // a chunk's rows; zeros past the segment's end
        const int32_t ldq = fresh_scalar((int32_t)a.ldq);
        const Rows rows = rows_of(qp + (int64_t)t * ldq, seg.t1 - t, ldq, DK, 2);
        const uint32_t at = fresh(q_lane) + 32 * it * (uint32_t)ldq;
#pragma unroll
        for (int c = 0; c < contractions; ++c)
            q[c] = load4(rows, at + 16 * c);
    };
    // The chunk's k, v and decays in `parts` pieces, which are issued between other work: all at once
    // they would hold up every wave at the same place.
    auto fetch = [&](int32_t t, auto parts_type, int part) {
        constexpr int parts = decltype(parts_type)::value;
        const int32_t n = t < seg.t0 ? 0 : seg.t1 - t;
        const int32_t ldk = fresh_scalar((int32_t)a.ldk), ldv = fresh_scalar((int32_t)a.ldv);
        const int32_t ldg = fresh_scalar((int32_t)a.ldg);
        const uint32_t k_at = fresh(k_lane), v_at = fresh(v_lane);
        const Rows kr = rows_of(kp + (int64_t)t * ldk, n, ldk, DK, 2);
        const Rows vr = rows_of(vp + (int64_t)t * ldv, n, ldv, DV, 2);
#pragma unroll
        for (int i = 0; i < loads; ++i)
            if (i * parts / loads == part)
                kn[i] = load4(kr, k_at + 2 * i * step * (uint32_t)ldk);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e * parts / 8 == part)
                vn[e] = Words<CW>::load(vr, v_at + 2 * (32 * v_half + 16 * (e / 4) + (e & 3)) * (uint32_t)ldv);
        if (part == parts - 1)
            gn = __builtin_bit_cast(float, Words<1>::load(rows_of(gp + (int64_t)t * ldg, n, ldg, 1, 4),
                                                          4 * fresh(lane) * (uint32_t)ldg)[0]);
    };

    if (tid < 2) {
        lds.odd[tid] = 0;
        lds.bad_token[tid] = kChunk;
    }
    if (tid < DK / 16)
        lds.bad_dims[tid & 1][tid >> 1] = 0;
    for (int i = tid; i < 2 * DV; i += threads)
        lds.bad_column[i & 1][i >> 1] = kChunk;
    bool odd = false;

    // What a segment adds is summed from its last chunk to its first: a chunk then weighs as much as the
    // decays behind it say, and the sum needs no factor per chunk (a tenth of the work outside the products).
    double whole = 0.0;   // sum of log2 decays of the segment's chunks so far
    constexpr int32_t way = OUT ? kChunk : -kChunk;
    const int32_t chunks = (seg.t1 - seg.t0 + kChunk - 1) / kChunk;
    int32_t t = OUT ? seg.t0 : seg.t0 + (chunks - 1) * kChunk;
    if (chunks > 0) {
        fetch(t, Count<1>(), 0);
        if (OUT)
            fetch_q(t);
    }
    for (int32_t chunks_left = chunks; chunks_left > 0; --chunks_left, t += way) {
        const int32_t n = seg.t1 - t;
        const float gc = lane >= n ? 0.0f : gn < kNone ? kNone : gn;
        const double b = running_sum((double)gc * 1.44269504088896340736);
        const uint64_t bu = __builtin_bit_cast(uint64_t, b);
        const double end = __builtin_bit_cast(
            double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(bu >> 32), 63) << 32 |
                        (uint32_t)__builtin_amdgcn_readlane((int)bu, 63));
        const float whole_chunk = __builtin_amdgcn_exp2f((float)end);
        const double behind = OUT ? end : whole + end;
        whole += end;
        // float16: the largest e^(b_63 - b), as a power of two, and a token's largest e^(b_i - b_j). Without
        // growth they are that of the last token, and 1.
        int32_t most_ed = 0;
        float gain = 0.0f;
        if constexpr (fp16) {
            double least = end;
            if (__ballot(gc > 0.0f)) {
                rare();
                float x = (float)b;
                for (int d = 1; d < 64; d <<= 1) {
                    const float o = __shfl_up(x, d);
                    if (lane >= d)
                        x = fminf(x, o);
                }
                gain = __shfl((float)b - x, 16 * it + col);
                least = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
            }
            const float x = fminf(fmaxf((float)(behind - least), -1e6f), 1e6f);
            most_ed = __builtin_amdgcn_readfirstlane((int32_t)__builtin_ceilf(x));
        }
        const int parity = chunks_left & 1;
        __syncthreads();   // the previous chunk has been read

        // Values of k and v that are not finite (rare) become zeros and mark what they reach: the
        // outputs of their own and later tokens, their columns or rows of the state. With the matrix
        // products they would also reach earlier tokens, by way of a zero weight.
        if (odd) {   // the last chunk's marks have been read
            rare();
            if (tid < DK / 32)
                lds.bad_dims[parity ^ 1][tid] = 0;
            if (tid == 0) {
                lds.odd[parity ^ 1] = 0;
                lds.bad_token[parity ^ 1] = kChunk;
            }
            for (int i = tid; i < DV; i += threads)
                lds.bad_column[parity ^ 1][i] = kChunk;
        }
        float squares = 0.0f;
        uint32_t most_v[CW] = {};
        auto sizes = [&]() {
            squares = 0.0f;
#pragma unroll
            for (int i = 0; i < loads; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    squares = add_squares(kn[i][e], squares);
#pragma unroll
            for (int x = 0; x < CW; ++x) {
                most_v[x] = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    most_v[x] = larger_pair(most_v[x], vn[e][x] & 0x7FFF7FFFu);
            }
        };
        bool finite;
        if constexpr (fp16) {
            sizes();
            finite = squares < INFINITY;
#pragma unroll
            for (int x = 0; x < CW; ++x)
                finite = finite && !(odd_bits(Type(), most_v[x]) & 0x80008000u);
        } else {
            float seen = 0.0f;   // 0, or NaN where something is not finite
#pragma unroll
            for (int i = 0; i < loads; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    seen = times_zero(kn[i][e], seen);
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int x = 0; x < CW; ++x)
                    seen = times_zero(vn[e][x], seen);
            finite = seen == seen;
        }
        if (__ballot(!finite)) {
            rare();
            lds.odd[parity] = 1;
#pragma unroll
            for (int i = 0; i < loads; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t o = odd_bits(Type(), kn[i][e]) & 0x80008000u;
                    if (o) {
                        kn[i][e] = only_finite(Type(), kn[i][e]);
                        if ((int)row0 + i * step >= n)   // rows that lie closer than their length: not the sequence's
                            continue;
                        const uint32_t d = dim0 + 2 * e;   // even: both dims in one word
                        atomicMin(&lds.bad_token[parity], row0 + i * step);
                        atomicOr(&lds.bad_dims[parity][d / 32], ((o >> 15 & 1) | (o >> 30)) << (d % 32));
                    }
                }
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int x = 0; x < CW; ++x) {
                    const uint32_t o = odd_bits(Type(), vn[e][x]), d = EV * col + v_first + 2 * x;
                    vn[e][x] = only_finite(Type(), vn[e][x]);
                    const uint32_t row = 32 * v_half + 16 * (e / 4) + 4 * g + (e & 3);
                    if ((int)row >= n)
                        continue;
                    if (o & 0x8000u)
                        atomicMin(&lds.bad_column[parity][d], row);
                    if (o & 0x80000000u)
                        atomicMin(&lds.bad_column[parity][d + 1], row);
                }
            if constexpr (fp16)
                sizes();
        }
        if constexpr (fp16) {
            squares = wave_max(squares);
            if (lane == 0)
                lds.squares[wave] = squares;
#pragma unroll
            for (int x = 0; x < CW; ++x) {
                const uint32_t most = larger_pair4(most_v[x]);
                if (g == 0)
                    lds.most_v[v_half][col][v_first / 2 + x] = most;
            }
        }
#pragma unroll
        for (int i = 0; i < loads; ++i)
            *(u32x4 *)&lds.k[row0 + i * step][dim0] = kn[i];
#pragma unroll
        for (int x = 0; x < CW; ++x) {   // rows paired up: columns v_first + 2x and + 2x + 1
            u32x4 v0, v1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v0[e] = __builtin_amdgcn_perm(vn[2 * e + 1][x], vn[2 * e][x], 0x05040100u);
                v1[e] = __builtin_amdgcn_perm(vn[2 * e + 1][x], vn[2 * e][x], 0x07060302u);
            }
            lds.v[v_half][v_first + 2 * x][lane] = v0;
            lds.v[v_half][v_first + 2 * x + 1][lane] = v1;
        }
        int32_t s_exponent = 0;   // float16: all of s is below 2^this
        if (OUT) {
            float shrink[CW];
#pragma unroll
            for (int c = 0; c < CW; ++c)
                shrink[c] = 1.0f;   // bfloat16 needs none
            if constexpr (fp16) {
                float most = 0.0f;
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    float x = 0.0f;
#pragma unroll
                    for (int j = 0; j < EK; ++j) {
                        x = larger(x, s[j][c][0], s[j][c][1]);
                        x = larger(x, s[j][c][2], s[j][c][3]);
                    }
                    most = larger(most, __builtin_ldexpf(x, -up[c]), 0.0f);
                }
                most = wave_max(most);
                if (!(most < INFINITY)) {   // the finite ones' scale
                    rare();
                    most = 0.0f;
#pragma unroll
                    for (int j = 0; j < EK; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int c = 0; c < CW; ++c) {
                                const float x = fabsf(__builtin_ldexpf(s[j][c][r], -up[c]));
                                most = x < INFINITY && x > most ? x : most;
                            }
                    most = wave_max(most);
                }
                s_exponent = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(most));
                const int32_t to = min(15 - s_exponent, 100);
#pragma unroll
                for (int c = 0; c < CW; ++c)
                    shrink[c] = power(min(to - up[c], 127));
                if (lane == 0)
                    lds.grow[wave] = power(-to);
            }
#pragma unroll
            for (int p = 0; p < WK; ++p)
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    u32x4 x;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        x[r] = pack2(Type(), s[2 * p][c][r] * shrink[c], s[2 * p + 1][c][r] * shrink[c]);
                    lds.s[p][CW * wave + c][lane] = x;
                }
        }
        if (wave == 0) {
            if (OUT) {
                lds.b[lane] = (float)b;
                if constexpr (!fp16)
                    lds.eb[lane] = __builtin_amdgcn_exp2f((float)b);
            }
            lds.ed[lane] = lane < n ? __builtin_amdgcn_exp2f((float)(behind - b - most_ed)) : 0.0f;
        }
        __syncthreads();
        odd = __builtin_amdgcn_readfirstlane(lds.odd[parity]) != 0;
        __builtin_amdgcn_sched_barrier(0);

        if (OUT) {   // on both ways: queries still on their way on one of them would be waited for behind it
#pragma unroll
            for (int c = 0; c < contractions; ++c)
                asm volatile("" : "+v"(q[c]));
        }
        if (OUT && it * 16 < n) {
            f32x4 o[EV];
#pragma unroll
            for (int j = 0; j < EV; ++j)
                o[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int p = 0; p < WK; ++p) {
                fetch(t + kChunk, Count<WK>(), p);
                __builtin_amdgcn_sched_barrier(0);
                u32x4 x;   // words of dims EK r + 2p of the lane's
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    x[r] = q[(WK * r + p) / 4][(WK * r + p) % 4];
#pragma unroll
                for (int j = 0; j < EV; ++j)
                    o[j] = mfma(Type(), x, lds.s[p][j][lane], o[j]);
            }
            float bi = lds.b[16 * it + col];
            f32x4 row;   // factors of tokens 16 it + 4g ..
            if constexpr (fp16) {   // no score of token 16 it + col is above 2^-e, from the norms of q and k
                float norm = 0.0f;
#pragma unroll
                for (int c = 0; c < contractions; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        norm = add_squares(q[c][e], norm);
                const f32x4 k2 = *(const f32x4 *)lds.squares;   // a row's squares are those of `pieces` lanes
                const float k_norm = fmaxf(fmaxf(k2[0], k2[1]), fmaxf(k2[2], k2[3])) * pieces;
                const int32_t e = max(-(root_exponent(sum4(norm)) + root_exponent(k_norm) +
                                        (int32_t)__builtin_ceilf(fminf(gain, 1e6f))), -120);
                bi += (float)(15 + e);
                if (g == 0) {
                    lds.row[wave][col] = __builtin_amdgcn_exp2f(bi);
                    lds.last[wave][col] = __builtin_ldexpf(a.scale, -15 - e);
                }
                __builtin_amdgcn_wave_barrier();
                row = *(const f32x4 *)&lds.row[wave][4 * g];
            } else {
                row = *(const f32x4 *)&lds.eb[16 * it + 4 * g];
            }
#pragma unroll
            for (int j = 0; j < EV; ++j) {
                const float grow = fp16 ? lds.grow[j / CW] : 1.0f;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    o[j][r] *= row[r] * grow;
            }
            for (int half = 0; 2 * half <= it; ++half) {
                u32x4 w = {0, 0, 0, 0};   // scores of token 16 it + col with 8 keys of the half
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int jt = 2 * half + k;
                    if (jt > it)
                        break;
                    f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int c = 0; c < contractions; ++c)
                        x = mfma(Type(), *(const u32x4 *)&lds.k[16 * jt + col][DK / 4 * g + 8 * c], q[c], x);
                    const f32x4 bj = *(const f32x4 *)&lds.b[16 * jt + 4 * g];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        x[r] *= __builtin_amdgcn_exp2f(bi - bj[r]);
                        x[r] = jt < it || 4 * g + r <= col ? x[r] : 0.0f;
                    }
                    w[2 * k] = pack2(Type(), x[0], x[1]);
                    w[2 * k + 1] = pack2(Type(), x[2], x[3]);
                }
#pragma unroll
                for (int j = 0; j < EV; ++j)
                    o[j] = mfma(Type(), w, lds.v[half][j][lane], o[j]);
            }
            f32x4 last = {a.scale, a.scale, a.scale, a.scale};
            if constexpr (fp16)
                last = *(const f32x4 *)&lds.last[wave][4 * g];
#pragma unroll
            for (int j = 0; j < EV; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    o[j][r] *= last[r];
            if (odd) {
                rare();
#pragma unroll
                for (int j = 0; j < EV; ++j) {
                    const uint32_t bad = min(lds.bad_token[parity], lds.bad_column[parity][EV * col + j]);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        o[j][r] = 16 * it + 4 * g + r >= bad ? NAN : o[j][r];
                }
            }
            const int32_t ldo = fresh_scalar((int32_t)a.ldo);
            const Rows rows = rows_of(op + (int64_t)t * ldo, n, ldo, DV, 2);
            const uint32_t o_at = fresh(o_lane);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                uint32_t x[EV / 2];
#pragma unroll
                for (int j = 0; j < EV; j += 2)
                    x[j / 2] = pack2(Type(), o[j][r], o[j + 1][r]);
                const uint32_t at = 16 * it + 4 * g + r < n ? o_at + 2 * (16 * it + r) * (uint32_t)ldo : ~0u;
                if constexpr (EV == 8)
                    __builtin_amdgcn_raw_buffer_store_b128(u32x4{x[0], x[1], x[2], x[3]}, rows, at, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b64(u32x2{x[0], x[1]}, rows, at, 0, 0);
            }
        }

        if (OUT && n <= kChunk && !REST)
            break;   // nobody reads the state after this segment
        if (OUT)
            fetch_q(t + kChunk);
        __builtin_amdgcn_sched_barrier(0);
        // s after the chunk's decay. float16: and with the power of two that brings this chunk's largest
        // e^(b_63 - b) |v| of the column just below 2^15 (a sum over chunks: the largest so far), unless s itself
        // would pass 2^120 with it; v meets what of that e^(b_63 - b) does not.
        float fade[CW], v_up[CW];
        bool same = true;
#pragma unroll
        for (int c = 0; c < CW; ++c)
            fade[c] = whole_chunk;
        if constexpr (fp16) {
            uint32_t most_v[(CW + 1) / 2];
#pragma unroll
            for (int x = 0; x < (CW + 1) / 2; ++x)
                most_v[x] = larger_pair(lds.most_v[0][col][CW * wave / 2 + x], lds.most_v[1][col][CW * wave / 2 + x]);
            const int32_t room = 120 - s_exponent - max((int32_t)__builtin_ceilf(fminf((float)end, 1e6f)), 0);
#pragma unroll
            for (int c = 0; c < CW; ++c) {
                const float most = (CW * wave + c) & 1 ? high(Type(), most_v[c / 2]) : low(Type(), most_v[c / 2]);
                const int32_t want = most > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(most) - most_ed : kMostUp;
                const int32_t now = max(OUT ? min(min(want, kMostUp), min(room, up[c] + 100)) : min(want, up[c]), -140);
                fade[c] = OUT ? __builtin_amdgcn_exp2f(fminf((float)end + (float)(now - up[c]), 126.0f))
                              : power(now - up[c]);
                same = same && now == up[c];
                up[c] = now;
                v_up[c] = power(now + most_ed);
            }
        }
        if (OUT || (fp16 && __ballot(!same))) {
#pragma unroll
            for (int j = 0; j < EK; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < CW; ++c)
                        s[j][c][r] *= fade[c];
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            constexpr int terms = REST ? Terms<Type>::count : Terms<Type>::count - 1;
            u32x4 x[terms][CW];   // e^(b_63 - b_j) v_j, rounded, and what the rounding leaves
#pragma unroll
            for (int c = 0; c < CW; ++c)
                x[0][c] = lds.v[half][CW * wave + c][lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x2 d = *(const f32x2 *)&lds.ed[32 * half + 16 * (e / 2) + 4 * g + 2 * (e & 1)];
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    float v0 = low(Type(), x[0][c][e]), v1 = high(Type(), x[0][c][e]);
                    if constexpr (fp16) {
                        v0 *= v_up[c];
                        v1 *= v_up[c];
                    }
                    v0 *= d[0];
                    v1 *= d[1];
#pragma unroll
                    for (int i = 0; i < terms; ++i)
                        x[i][c][e] = take(Type(), v0, v1);
                }
            }
            uint32_t rows[8][WK];   // dims EK col .. of the half's eight keys
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint16_t *p = &lds.k[32 * half + 16 * (e / 4) + 4 * g + (e & 3)][EK * col];
                if constexpr (WK == 4) {
                    const u32x4 u = *(const u32x4 *)p;
                    rows[e][0] = u[0]; rows[e][1] = u[1]; rows[e][2] = u[2]; rows[e][3] = u[3];
                } else {
                    const u32x2 u = *(const u32x2 *)p;
                    rows[e][0] = u[0]; rows[e][1] = u[1];
                }
            }
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                if (!OUT) {
                    fetch(t + way, Count<2 * WK>(), half * WK + w);
                    __builtin_amdgcn_sched_barrier(0);
                }
                u32x4 k0, k1;   // dims EK col + 2w and + 2w + 1
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    k0[e] = __builtin_amdgcn_perm(rows[2 * e + 1][w], rows[2 * e][w], 0x05040100u);
                    k1[e] = __builtin_amdgcn_perm(rows[2 * e + 1][w], rows[2 * e][w], 0x07060302u);
                }
#pragma unroll
                for (int i = 0; i < terms; ++i) {
#pragma unroll
                    for (int c = 0; c < CW; ++c) {
                        s[2 * w][c] = mfma(Type(), k0, x[i][c], s[2 * w][c]);
                        s[2 * w + 1][c] = mfma(Type(), k1, x[i][c], s[2 * w + 1][c]);
                    }
                }
            }
        }
        if (odd) {
            rare();
#pragma unroll
            for (int c = 0; c < CW; ++c) {
                const bool column = lds.bad_column[parity][EV * col + CW * wave + c] < kChunk;
#pragma unroll
                for (int j = 0; j < EK; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int d = EK * (4 * g + r) + j;
                        const bool row = lds.bad_dims[parity][d / 32] >> (d % 32) & 1;
                        s[j][c][r] = row || column ? NAN : s[j][c][r];
                    }
            }
        }
    }

    if (OUT && !REST)
        return;
    float *to = OUT ? a.state_out + ((int64_t)seg.seq * a.H + h) * state_size
                    : cuts.states + ((int64_t)(seg.slot + 1) * a.H + h) * state_size;
#pragma unroll
    for (int j = 0; j < EK; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float x[CW];
#pragma unroll
            for (int c = 0; c < CW; ++c)
                x[c] = fp16 ? __builtin_ldexpf(s[j][c][r], -up[c]) : s[j][c][r];
            __builtin_memcpy(__builtin_assume_aligned(to + state_at + (int64_t)(EK * r + j) * DV, 4 * CW), x, 4 * CW);
        }
    if (!OUT && tid == 0)
        cuts.decays[(int64_t)(seg.slot + 1) * a.H + h] = __builtin_amdgcn_exp2f((float)whole);
}

template <class Type, int DK, int DV, bool OUT>
__global__ __launch_bounds__(kSegmentThreads, 2) void linear_chunk_kernel(LinearArgs a, Cuts cuts)
{
    __shared__ __align__(16) ChunkLds<Type, DK, DV, OUT> lds;
    Segment seg;
    if (!find_segment(a, cuts, blockIdx.y, !OUT, &seg))
        return;
    if (!OUT || seg.single)
        run_segment<Type, DK, DV, OUT, true>(a, cuts, seg, lds);
    else
        run_segment<Type, DK, DV, OUT, false>(a, cuts, seg, lds);
}

// The state before every segment of a sequence that has several, and the last one: a segment's slot
// holds what the segment before it adds, and then that state (the first one's: state_in, which may be
// the same memory as state_out). Four elements per thread, the additions of four segments in flight.
__global__ __launch_bounds__(256) void linear_states_kernel(LinearArgs a, Cuts c)
{
    const int32_t size = a.Dk * a.Dv;
    const int h = blockIdx.x, part = blockIdx.z;
    int32_t slot0, n;
    const int seq = blockIdx.y;
    if (!a.cu) {
        slot0 = 0;
        n = (int32_t)(((int64_t)a.T + c.L - 1) / c.L);
    } else if (a.B <= kWaveSeqs) {
        const LaneCut cut = lane_cut(a, c);
        slot0 = __builtin_amdgcn_readlane(slot_before(cut.before - cut.ones, cut.before, threadIdx.x & 63), seq);
        n = __builtin_amdgcn_readlane(cut.n, seq);
    } else {
        const int32_t *segments = c.maps + a.B + 1, *several = segments + a.B + 1;
        slot0 = slot_before(several[seq], segments[seq], seq);
        n = several[seq + 1] - several[seq];
    }
    if (n <= 1)
        return;
    const int32_t at = (part * 256 + (int)threadIdx.x) * 4;
    const int64_t step = (int64_t)a.H * size;
    float *p = c.states + ((int64_t)slot0 * a.H + h) * size + at;
    const float *d = c.decays + (int64_t)slot0 * a.H + h;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a.state_in)
        s = *(const f32x4 *)(a.state_in + ((int64_t)seq * a.H + h) * size + at);
    *(f32x4 *)p = s;
    constexpr int U = 4;
    for (int k = 1; k <= n; k += U) {
        f32x4 x[U];
        float f[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k + u <= n) {
                x[u] = *(const f32x4 *)(p + (k + u) * step);
                f[u] = d[(int64_t)(k + u) * a.H];
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (k + u <= n) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[e] = fmaf(f[u], s[e], x[u][e]);
                if (k + u < n)
                    *(f32x4 *)(p + (k + u) * step) = s;
            }
    }
    *(f32x4 *)(a.state_out + ((int64_t)seq * a.H + h) * size + at) = s;
}

template <class Type, int DK, int DV>
hipError_t linear_of(const LinearArgs &a, const Cuts &c, hipStream_t stream)
{
    const dim3 block(kSegmentThreads);
    if (a.cu && a.B > kWaveSeqs)
        linear_maps_kernel<<<dim3(1), dim3(kMapThreads), 0, stream>>>(a, c);
    if (c.inner > 0) {
        linear_chunk_kernel<Type, DK, DV, false><<<dim3(a.H, c.inner), block, 0, stream>>>(a, c);
        linear_states_kernel<<<dim3(a.H, a.B, DK * DV / 1024), dim3(256), 0, stream>>>(a, c);
    }
    linear_chunk_kernel<Type, DK, DV, true><<<dim3(a.H, a.T / c.L + a.B), block, 0, stream>>>(a, c);
    return hipGetLastError();
}

template <class Type>
hipError_t linear_typed(const LinearArgs &a, const Cuts &c, hipStream_t stream)
{
    if (a.Dk == 64)
        return a.Dv == 64 ? linear_of<Type, 64, 64>(a, c, stream) : linear_of<Type, 64, 128>(a, c, stream);
    return a.Dv == 64 ? linear_of<Type, 128, 64>(a, c, stream) : linear_of<Type, 128, 128>(a, c, stream);
}

// Tokens per segment, as many as leave one segment per CU (256 of them: the workspace's size may be asked for
// where there is no device) and at least 128; past 512 tokens as many as leave two. A segment's state is
// written and read once (128 KB per head of 128 x 128, against 1.5 KB per token), so longer ones move less and
// shorter ones end sooner. Measured, us for tokens x heads of 128 x 128, bfloat16, with segments of 128 / 256 / 512: 700 x 8 26 / 39 / 65,
// 2048 x 8 33 / 42 / 67, 1024 x 32 41 / 44 / 68, 2048 x 32 67 / 55 / 71, 8192 x 8 83 / 64 / 75; of 512
// and 1024: 8192 x 32 125 and 137; of 1024, 2048 and 4096: 32768 x 32 439, 400 and 472. Up to 256 tokens
// in all, where a cut can only halve them, it costs more than it gives (200 x 16: 25 and 22).
int32_t segment_length(int32_t T, int32_t H)
{
    const int64_t all = (int64_t)T * H;
    int64_t L = all / 256 < 512 ? all / 256 : all / 512 < 512 ? 512 : all / 512;
    L = (L + kChunk - 1) / kChunk * kChunk;
    if (L < (T <= 256 ? 256 : 128))
        L = T <= 256 ? 256 : 128;
    if (L > 4096)
        L = 4096;
    while (T / L > 16384)
        L *= 2;
    return (int32_t)L;
}

int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }

// No call of at most T tokens has more whole segments than this: segments of L tokens, which are 128 to 512
// and, rounded down, T H / 256 at least, are fewer than 258 / H; those of 512 to 4096, T H / 512 at least, at most
// 513 / H; and so on. It never falls as T rises, which T / segment_length(T) does.
int32_t most_whole(int32_t T, int32_t H)
{
    if (T <= 256)
        return H <= 258 ? T / 256 : 0;
    const int32_t a = T / 128 < 258 / H ? T / 128 : 258 / H, b = T / 512 < 513 / H ? T / 512 : 513 / H;
    const int32_t c = T / 4096 < 16384 ? T / 4096 : 16384, ab = a > b ? a : b;
    return ab > c ? ab : c;
}

// A sequence of several segments has x + 1 <= 2x of them, x the whole segments before its last token,
// and all such x sum up to at most T / L. One sequence without bounds has T / L and one, if that.
void count_slots(Cuts &c, int32_t whole, int32_t num_seqs)
{
    c.inner = num_seqs == 1 ? whole + (whole > 0) : 2 * whole;
    c.slots = c.inner + (num_seqs < whole ? num_seqs : whole);
}

// Places in the workspace; returns its size.
int64_t place(Cuts &c, int32_t num_seqs, int32_t H, int32_t Dk, int32_t Dv, float *work)
{
    const int64_t states = (int64_t)c.slots * H * Dk * Dv * 4, decays = round16((int64_t)c.slots * H * 4);
    const int64_t maps = num_seqs > kWaveSeqs ? round16(3 * ((int64_t)num_seqs + 1) * 4) : 0;
    c.states = work;
    c.decays = (float *)((char *)work + states);
    c.maps = (int32_t *)((char *)c.decays + decays);
    return states + decays + maps;
}

}  // namespace

int64_t linear_workspace(int32_t T, int32_t num_seqs, int32_t H, int32_t Dk, int32_t Dv)
{
    Cuts c{};
    count_slots(c, most_whole(T, H), num_seqs);
    return place(c, num_seqs, H, Dk, Dv, nullptr);
}

hipError_t launch_linear(const LinearArgs &a, hipStream_t stream)
{
    Cuts c;
    c.L = segment_length(a.T, a.H);
    count_slots(c, a.T / c.L, a.B);
    place(c, a.B, a.H, a.Dk, a.Dv, a.work);
    return a.type ? linear_typed<Fp16>(a, c, stream) : linear_typed<Bf16>(a, c, stream);
}

hipError_t launch_linear_step(const LinearArgs &a, hipStream_t stream)
{
    a.type ? step_typed<Fp16>(a, stream) : step_typed<Bf16>(a, stream);
    return hipGetLastError();
}

}  // namespace w4a16
