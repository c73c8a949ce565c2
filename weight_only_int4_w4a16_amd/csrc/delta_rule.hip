// The gated delta rule, for gfx950:
//   S_t = e^{g_t} S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - e^{g_t} S_{t-1}^T k_t),   o_t = scale * q_t^T S_t.
#include "chunks.h"
#include "mixers.h"
#include "mixer_types.h"

namespace w4a16 {

namespace {

// ---- one token per request ---------------------------------------------------------------------
// The state is read once, updated in registers and written once: 8 bytes of HBM traffic per element and nothing
// else of that order. Both products with the old state, k^T S and q^T S, come from one pass over the registers and
// one sum over the row groups; with d = e^g they give u = beta (v - d S^T k) and o = d S^T q + (q . k) u.
constexpr int kStepThreads = 256;

template <class Type, int DK, int DV, int CV, bool STREAM>
__global__ __launch_bounds__(kStepThreads) void delta_step_kernel(DeltaArgs a)
{
    typedef typename Type::T T;
    constexpr int LPR = CV / 4, RG = kStepThreads / LPR, ROWS = DK / RG, PARTS = DV / CV, NW = kStepThreads / 64;
    static_assert(ROWS >= 1 && RG * ROWS == DK, "rows divide over the row groups");
    __shared__ float qs[DK], ks[DK];
    __shared__ f32x4 part[2][NW][LPR];
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
        qs[tid] = Type::f(((const T *)a.q)[b * a.ldq + hk * a.hsq + tid]);
        ks[tid] = Type::f(((const T *)a.k)[b * a.ldk + hk * a.hsk + tid]);
    }
    const T *vp = (const T *)a.v + b * a.ldv + h * a.hsv + c0;
    f32x4 v, sk = {0.0f, 0.0f, 0.0f, 0.0f}, sq = sk;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = Type::f(vp[e]);
    const float decay = expf(a.g[b * a.ldg + h * a.hsg]), beta = a.beta[b * a.ldb + h * a.hsb];
    __syncthreads();
    float qk = 0.0f;   // every wave sums all of q . k
    for (int i = tid & 63; i < DK; i += 64)
        qk = fmaf(qs[i], ks[i], qk);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        qk += __shfl_xor(qk, d);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float k = ks[rg + r * RG], q = qs[rg + r * RG];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[r][e] *= decay;
            sk[e] = fmaf(k, s[r][e], sk[e]);
            sq[e] = fmaf(q, s[r][e], sq[e]);
        }
    }
#pragma unroll
    for (int d = LPR; d < 64; d <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sk[e] += __shfl_xor(sk[e], d);
            sq[e] += __shfl_xor(sq[e], d);
        }
    if ((tid & 63) < LPR) {
        part[0][tid >> 6][col] = sk;
        part[1][tid >> 6][col] = sq;
    }
    __syncthreads();
    sk = part[0][0][col];
    sq = part[1][0][col];
#pragma unroll
    for (int w = 1; w < NW; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sk[e] += part[0][w][col][e];
            sq[e] += part[1][w][col][e];
        }
    f32x4 u;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        u[e] = beta * (v[e] - sk[e]);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float k = ks[rg + r * RG];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s[r][e] = fmaf(k, u[e], s[r][e]);
        if (STREAM)
            __builtin_nontemporal_store(s[r], (f32x4 *)(a.state_out + base + r * RG * DV));
        else
            *(f32x4 *)(a.state_out + base + r * RG * DV) = s[r];
    }
    if (rg == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = Type::from(a.scale * fmaf(qk, u[e], sq[e]));
    }
}

template <class Type, int DK, int DV>
void step_of(const DeltaArgs &a, hipStream_t stream)
{
    if ((int64_t)a.B * a.H < 128)
        delta_step_kernel<Type, DK, DV, 32, false><<<dim3(a.H * (DV / 32), a.B), dim3(kStepThreads), 0, stream>>>(a);
    else
        delta_step_kernel<Type, DK, DV, DV, true><<<dim3(a.H, a.B), dim3(kStepThreads), 0, stream>>>(a);
}

template <class Type>
void step_typed(const DeltaArgs &a, hipStream_t stream)
{
    if (a.Dk == 64)
        a.Dv == 64 ? step_of<Type, 64, 64>(a, stream) : step_of<Type, 64, 128>(a, stream);
    else
        a.Dv == 64 ? step_of<Type, 128, 64>(a, stream) : step_of<Type, 128, 128>(a, stream);
}

// ---- packed sequences ----------------------------------------------------------------------------
// Sequences are cut into chunks of 64 tokens. With b_i the running sum of the log decays inside a chunk (its own
// token included) and S the state before it, per head:
//   (1 + A) U = diag(beta) (V - diag(e^b) K S),   A_ij = beta_i e^{b_i - b_j} k_i . k_j for j < i
//   o_i = scale * (e^{b_i} q_i^T S + sum_{j<=i} P_ij u_j),   P_ij = e^{b_i - b_j} q_i . k_j
//   S  <- e^{b_63} S + K^T diag(e^{b_63 - b}) U
// What does not need S comes first, for all chunks side by side: T = (1 + A)^-1 diag(beta) and P, 64 x 64 each. Then
// a work-group per sequence, head and 16 columns of V goes from chunk to chunk: X = K S, R = V - diag(e^b) X, U = T R.
constexpr int kDeltaThreads = 256, kWaves = 4;
constexpr int kFrags = 6;   // operands of a lower triangle: rows 16 w.., columns 32 c.. (c <= w / 2)
__device__ __forceinline__ constexpr int frag(int w, int c) { return w < 2 ? w : 2 * w - 2 + c; }

// Four values' next term, as two words.
__device__ __forceinline__ u32x2 take4(f32x4 &v)
{
    float a = v[0], b = v[1], c = v[2], d = v[3];
    const u32x2 w = {take(Bf16(), a, b), take(Bf16(), c, d)};
    v = f32x4{a, b, c, d};
    return w;
}

// What a chunk of a head needs besides its rows, in the workspace.
template <class Type>
struct Prepared {
    static constexpr int p_terms = __is_same(Type, Fp16) ? 2 : 1;
    u32x4 t[3][kFrags][64], p[p_terms][kFrags][64];   // first operands: T in three bfloat16 terms, P
    float eb[kChunk], ed[kChunk];                     // e^b, e^(b_63 - b)
    int32_t bad;                                      // first token with a k, beta or decay that is not finite, or 64
    float whole;                                      // e^b_63
    int32_t pad[30];
};
static_assert(sizeof(Prepared<Bf16>) % 128 == 0 && sizeof(Prepared<Fp16>) % 128 == 0, "whole cache lines");

// Sequence s has its chunks' places from here on: as many as it has chunks, or more, lie before the next one's.
__device__ __forceinline__ int32_t first_place(const DeltaArgs &a, int s)
{
    return a.cu ? min(max(a.cu[s], 0), a.T) / kChunk + s : 0;
}
__device__ __forceinline__ void tokens_of(const DeltaArgs &a, int s, int32_t *t0, int32_t *t1)
{
    *t0 = a.cu ? min(max(a.cu[s], 0), a.T) : 0;
    *t1 = a.cu ? max(min(max(a.cu[s + 1], 0), a.T), *t0) : a.T;
}

// The last sequence whose places start at or before `place`, or -1; 64 of them at a time.
__device__ __forceinline__ int sequence_at(const DeltaArgs &a, int32_t place)
{
    if (!a.cu)
        return 0;
    const int lane = threadIdx.x & 63;
    int lo = 0, n = a.B;
    while (n > 0) {
        const int step = (n + 63) / 64, at = lo + lane * step;
        const uint64_t hit = __ballot(lane * step < n && first_place(a, at) <= place);
        if (!hit)
            return -1;
        const int k = 63 - __builtin_clzll(hit);
        if (step == 1)
            return lo + k;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return -1;
}

__device__ __forceinline__ f32x4 mfma_f32(f32x4 a, f32x4 b, f32x4 c)   // contraction of 16, lane group g has 4g ..
{
#pragma unroll
    for (int s = 0; s < 4; ++s)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
    return c;
}

// T and P of one chunk and head. Wave w has rows 16 w ..; products of K rows are formed both ways round, so that
// each result lies in the lanes where it is an operand. A and T are float32: diagonal blocks of 16 x 16 by
// substitution (no powers of A, which may be large where T is not), the others by float32 matrix products,
//   T_ij = -(sum_{j<m<=i} T_im A_mj) T_jj.
template <class Type, int DK>
__global__ __launch_bounds__(kDeltaThreads) void delta_prepare_kernel(DeltaArgs a, Prepared<Type> *work)
{
    constexpr int C = DK / 32;
    __shared__ f32x4 lds_a[10][64], lds_t[kWaves][64];
    __shared__ double lds_b[kChunk];
    __shared__ __align__(16) float lds_beta[kChunk];
    __shared__ int32_t lds_bad[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4, h = blockIdx.y, hk = h / (a.H / a.Hk);
    const int32_t place = (int32_t)blockIdx.x;
    const int seq = sequence_at(a, place);
    if (seq < 0)
        return;
    int32_t t0, t1;
    tokens_of(a, seq, &t0, &t1);
    t0 += (place - first_place(a, seq)) * kChunk;
    if (t0 >= t1)
        return;
    const int32_t n = min(t1 - t0, kChunk);
    Prepared<Type> &to = work[(int64_t)place * a.H + h];

    const int32_t ldq = (int32_t)a.ldq, ldk = (int32_t)a.ldk;   // below 2^24
    const Rows kr = rows_of((const uint16_t *)a.k + hk * a.hsk + (int64_t)t0 * ldk, n, ldk, DK, 2);
    const Rows qr = rows_of((const uint16_t *)a.q + hk * a.hsq + (int64_t)t0 * ldq, n, ldq, DK, 2);
    u32x4 ki[C], qi[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        ki[c] = load4(kr, 2 * ((16 * w + col) * (uint32_t)ldk + 32 * c + 8 * g));
        qi[c] = load4(qr, 2 * ((16 * w + col) * (uint32_t)ldq + 32 * c + 8 * g));
    }
    float decay = 0.0f, beta = 0.0f;
    if (lane < n) {
        decay = a.g[(int64_t)(t0 + lane) * a.ldg + h * a.hsg];
        beta = a.beta[(int64_t)(t0 + lane) * a.ldb + h * a.hsb];
    }
    const bool odd = !(decay < INFINITY) || !(fabsf(beta) < INFINITY);
    const uint64_t odd_tokens = __ballot(odd);
    decay = odd ? 0.0f : decay < kNone ? kNone : decay;
    beta = odd ? 0.0f : beta;
    const double b = running_sum((double)decay * 1.44269504088896340736);
    uint32_t bits = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            bits |= odd_bits(Type(), ki[c][e]);
    uint64_t odd_rows = __ballot((bits & 0x80008000u) != 0 && 16 * w + col < n);
    odd_rows |= odd_rows >> 32;
    odd_rows |= odd_rows >> 16;
    if (lane == 0)
        lds_bad[w] = odd_rows & 0xFFFF ? 16 * w + __builtin_ctzll(odd_rows) : kChunk;
    if (w == 0) {
        lds_b[lane] = b;
        lds_beta[lane] = beta;
    }
    __syncthreads();
    int32_t bad = odd_tokens ? __builtin_ctzll(odd_tokens) : kChunk;
#pragma unroll
    for (int i = 0; i < kWaves; ++i)
        bad = min(bad, lds_bad[i]);
    const int32_t lim = min(n, bad);   // tokens from here on count for nothing
    if (w == 0) {
        const double end = lds_b[kChunk - 1];
        to.eb[lane] = __builtin_amdgcn_exp2f((float)b);
        to.ed[lane] = __builtin_amdgcn_exp2f((float)(end - b));
        if (lane == 0) {
            to.bad = bad;
            to.whole = __builtin_amdgcn_exp2f((float)end);
        }
    }

    const double b_col = lds_b[16 * w + col];
    f32x4 own = {0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 p[Prepared<Type>::p_terms][2] = {};
#pragma unroll
    for (int j = 0; j < kWaves; ++j) {
        if (j > w)
            continue;
        u32x4 kj[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            kj[c] = j == w ? ki[c] : load4(kr, 2 * ((16 * j + col) * (uint32_t)ldk + 32 * c + 8 * g));
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            x = mfma(Type(), ki[c], kj[c], x);   // tokens i = 16 w + 4 g .. in the lane of token j = 16 j + col
            y = mfma(Type(), kj[c], qi[c], y);   // tokens j = 16 j + 4 g .. in the lane of token i = 16 w + col
        }
        const double bj_col = lds_b[16 * j + col];
        const f32x4 beta_i = *(const f32x4 *)&lds_beta[16 * w + 4 * g];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int32_t i = 16 * w + 4 * g + r, jj = 16 * j + col;
            x[r] = jj < i && i < lim ? x[r] * __builtin_amdgcn_exp2f((float)(lds_b[i] - bj_col)) * beta_i[r] : 0.0f;
            const int32_t i2 = 16 * w + col, j2 = 16 * j + 4 * g + r;
            y[r] = j2 <= i2 && j2 < lim ? y[r] * __builtin_amdgcn_exp2f((float)(b_col - lds_b[j2])) : 0.0f;
        }
        lds_a[w * (w + 1) / 2 + j][lane] = x;
#pragma unroll
        for (int term = 0; term < Prepared<Type>::p_terms; ++term) {
            const u32x2 o = take4(y);
            p[term][j / 2][2 * (j & 1)] = o[0];
            p[term][j / 2][2 * (j & 1) + 1] = o[1];
        }
    }
#pragma unroll
    for (int term = 0; term < Prepared<Type>::p_terms; ++term)
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (c <= w / 2)
                to.p[term][frag(w, c)][lane] = p[term][c];

    // The diagonal block: a lane has column `col`, row after row.
    float t[16];
#pragma unroll
    for (int r = 0; r < 16; ++r)
        t[r] = r == col ? 1.0f : 0.0f;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int m = 0; m < 15; ++m)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            if (4 * r4 + 3 <= m)
                continue;
            const f32x4 x = lds_a[w * (w + 1) / 2 + w][16 * r4 + m];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (4 * r4 + r > m)
                    t[4 * r4 + r] = fmaf(-x[r], t[m], t[4 * r4 + r]);
        }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        own[r] = g == 0 ? t[r] : g == 1 ? t[4 + r] : g == 2 ? t[8 + r] : t[12 + r];
    lds_t[w][lane] = own;   // rows 4 g .. of column `col`
    __syncthreads();
    f32x4 tt[kWaves];       // T_wj transposed: columns 16 j + 4 g .. in the lane of row 16 w + col
#pragma unroll
    for (int r = 0; r < 4; ++r)
        own[r] = lds_t[w][col / 4 * 16 + 4 * g + r][col & 3];
#pragma unroll
    for (int j = kWaves - 1; j >= 0; --j) {
        tt[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (j == w)
            tt[j] = own;
        if (j >= w)
            continue;
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int m = j + 1; m < kWaves; ++m)
            if (m <= w)
                x = mfma_f32(lds_a[m * (m + 1) / 2 + j][lane], tt[m], x);
        x = mfma_f32(lds_t[j][lane], x, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
        for (int r = 0; r < 4; ++r)
            tt[j][r] = -x[r];
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (c > w / 2)
            continue;
        f32x4 x = tt[2 * c], y = tt[2 * c + 1];
        const f32x4 bx = *(const f32x4 *)&lds_beta[32 * c + 4 * g], by = *(const f32x4 *)&lds_beta[32 * c + 16 + 4 * g];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            x[r] *= bx[r];
            y[r] *= by[r];
        }
#pragma unroll
        for (int term = 0; term < 3; ++term) {
            const u32x2 o = take4(x), o2 = take4(y);
            to.t[term][frag(w, c)][lane] = u32x4{o[0], o[1], o2[0], o2[1]};
        }
    }
}

// Words of two 16-bit values as bfloat16: as they are, or float16 as the sum of two.
template <class Type>
struct Split {
    static constexpr int terms = __is_same(Type, Fp16) ? 2 : 1;
    static __device__ __forceinline__ void of(uint32_t w, uint32_t *o)
    {
        if constexpr (terms == 1) {
            o[0] = w;
        } else {
            float x = low(Fp16(), w), y = high(Fp16(), w);
            o[0] = take(Bf16(), x, y);
            o[1] = pack2(Bf16(), x, y);
        }
    }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
// Contraction of 16 (two words) or 32 (four) bfloat16 values.
__device__ __forceinline__ f32x4 mfma_words(u32x2 a, u32x2 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, a), __builtin_bit_cast(s16x4, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_words(u32x4 a, u32x4 b, f32x4 c) { return mfma(Bf16(), a, b, c); }

// N + M terms of two operands' products that are above 2^-24 of the whole, the small ones first.
template <int NA, int NB, int MOST, class V>
__device__ __forceinline__ f32x4 products(const V *x, const V *y, f32x4 c)
{
#pragma unroll
    for (int sum = MOST; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (sum - i >= 0 && sum - i < NB)
                c = mfma_words(x[i], y[sum - i], c);
    return c;
}

template <int N>
struct WordsOf;
template <>
struct WordsOf<2> {
    typedef u32x2 T;
    static __device__ __forceinline__ T load(Rows r, uint32_t at) { return __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, 0); }
};
template <>
struct WordsOf<4> {
    typedef u32x4 T;
    static __device__ __forceinline__ T load(Rows r, uint32_t at) { return load4(r, at); }
};

// A work-group goes over the chunks of one sequence, head and 16 columns. Wave w holds the rows of S with dk in
// [DK / 4 w, DK / 4 (w + 1)), in float32, and multiplies K and Q by them as they are: a lane's values of S are the
// second operand's, for the same dims of a K row. The four waves' sums of X meet in LDS, wave w takes the tokens
// 16 w .. on to R; R and U are shared through LDS in operand order, so that no other values cross lanes.
template <class Type, int DK>
__global__ __launch_bounds__(kDeltaThreads, 2) void delta_chunk_kernel(DeltaArgs a, const Prepared<Type> *work, int slices)
{
    constexpr int EK = DK / 64, NW = 2 * EK, KT = Split<Type>::terms, PT = Prepared<Type>::p_terms;
    typedef typename WordsOf<NW>::T Words;
    __shared__ f32x4 lds_x[kWaves][kWaves][64], lds_q[kWaves][kWaves][64];
    __shared__ __align__(16) u32x2 lds_r[3][2][64][2], lds_u[5][2][64][2];
    __shared__ int32_t lds_bad[2][16], lds_odd[2];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    // All slices of a head on one XCD (work-groups go to the 8 of them in turn).
    const int64_t rest = blockIdx.x / 8, unit = rest / slices * 8 + blockIdx.x % 8;
    if (unit >= (int64_t)a.B * a.H)
        return;
    const int seq = (int)(unit / a.H), h = (int)(unit - (int64_t)seq * a.H), hk = h / (a.H / a.Hk);
    const int c0 = (int)(rest % slices) * 16;
    int32_t t0, t1;
    tokens_of(a, seq, &t0, &t1);
    const Prepared<Type> *from = work + (int64_t)first_place(a, seq) * a.H + h;
    const uint16_t *qp = (const uint16_t *)a.q + hk * a.hsq, *kp = (const uint16_t *)a.k + hk * a.hsk;
    const uint16_t *vp = (const uint16_t *)a.v + h * a.hsv + c0;
    uint16_t *op = (uint16_t *)a.out + h * a.hso + c0;
    const int32_t ldq = (int32_t)a.ldq, ldk = (int32_t)a.ldk, ldv = (int32_t)a.ldv, ldo = (int32_t)a.ldo;

    // s[j][r]: row DK / 4 w + EK (4 g + r) + j
    const int64_t state_at = ((int64_t)unit * DK + DK / 4 * w + EK * 4 * g) * a.Dv + c0 + col;
    f32x4 s[EK];
#pragma unroll
    for (int j = 0; j < EK; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            s[j][r] = a.state_in ? a.state_in[state_at + (int64_t)(EK * r + j) * a.Dv] : 0.0f;
    if (tid < 32)
        lds_bad[tid >> 4][tid & 15] = kChunk;
    if (tid < 2)
        lds_odd[tid] = 0;

    Words kn[kWaves], qn[kWaves];   // rows 16 i + col, this wave's dims from 4 EK g on
    uint32_t kt[16];                // dims EK col .. of tokens 32 c + 16 x + 4 g + e
    u32x4 tn[3][2], pn[PT][2];
    uint32_t vn[4];                 // tokens 16 w + 4 g ..
    f32x4 ebn, edn;
    int32_t badn = kChunk;
    float wholen = 1.0f;
    auto fetch_kq = [&](int32_t t) {
        const Rows kr = rows_of(kp + (int64_t)t * ldk, t1 - t, ldk, DK, 2);
        const Rows qr = rows_of(qp + (int64_t)t * ldq, t1 - t, ldq, DK, 2);
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            kn[i] = WordsOf<NW>::load(kr, 2 * ((16 * i + col) * (uint32_t)ldk + DK / 4 * w + 4 * EK * g));
            qn[i] = WordsOf<NW>::load(qr, 2 * ((16 * i + col) * (uint32_t)ldq + DK / 4 * w + 4 * EK * g));
        }
    };
    auto fetch_kt = [&](int32_t t) {
        const Rows kr = rows_of(kp + (int64_t)t * ldk, t1 - t, ldk, DK, 2);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const uint32_t at = 2 * ((32 * (e / 8) + 16 * (e / 4 % 2) + 4 * g + e % 4) * (uint32_t)ldk + DK / 4 * w + EK * col);
            kt[e] = EK == 2 ? __builtin_amdgcn_raw_buffer_load_b32(kr, at, 0, 0)
                            : __builtin_amdgcn_raw_buffer_load_b16(kr, at, 0, 0);
        }
    };
    auto prepared = [&](int32_t t) {   // zeros past the last chunk; operands that are none lie past its end
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>((const void *)from), 0,
                                                 t < t1 ? sizeof(Prepared<Type>) : 0, 0x00027000);
    };
    auto fetch_t = [&](Rows x) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                tn[i][c] = load4(x, c <= w / 2 ? (uint32_t)((i * kFrags + frag(w, c)) * 64 + lane) * 16 : ~0u);
    };
    auto fetch_p = [&](Rows x) {
#pragma unroll
        for (int i = 0; i < PT; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                pn[i][c] = load4(x, c <= w / 2 ? (uint32_t)(((3 + i) * kFrags + frag(w, c)) * 64 + lane) * 16 : ~0u);
    };
    auto fetch_v = [&](int32_t t, Rows x) {
        const Rows vr = rows_of(vp + (int64_t)t * ldv, t1 - t, ldv, 16, 2);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            vn[r] = __builtin_amdgcn_raw_buffer_load_b16(vr, 2 * ((16 * w + 4 * g + r) * (uint32_t)ldv + col), 0, 0);
        constexpr uint32_t at = (3 + PT) * kFrags * 64 * 16;
        ebn = __builtin_bit_cast(f32x4, load4(x, at + 4 * (16 * w + 4 * g)));
        edn = __builtin_bit_cast(f32x4, load4(x, at + 4 * (kChunk + 16 * w + 4 * g)));
        badn = __builtin_amdgcn_raw_buffer_load_b32(x, at + 8 * kChunk, 0, 0);
        wholen = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(x, at + 8 * kChunk + 4, 0, 0));
    };
    if (t0 < t1) {
        const Rows x = prepared(t0);
        fetch_kq(t0);
        fetch_v(t0, x);
        fetch_t(x);
        fetch_kt(t0);
        fetch_p(x);
    }
    __syncthreads();

    int parity = 0;
    for (int32_t t = t0; t < t1; t += kChunk, parity ^= 1) {
        const int32_t n = min(t1 - t, kChunk);
        from += a.H;
        const Rows next = prepared(t + kChunk);
        // X and Q S: this wave's dims
        {
            Words sb[3];
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                float x = EK == 2 ? s[0][i] : s[0][2 * i], y = EK == 2 ? s[EK - 1][i] : s[0][2 * i + 1];
#pragma unroll
                for (int term = 0; term < 3; ++term)
                    sb[term][i] = take(Bf16(), x, y);
            }
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                Words ka[KT], qa[KT];
#pragma unroll
                for (int j = 0; j < NW; ++j) {
                    uint32_t o[KT];
                    Split<Type>::of(kn[i][j], o);
#pragma unroll
                    for (int term = 0; term < KT; ++term)
                        ka[term][j] = o[term];
                    Split<Type>::of(qn[i][j], o);
#pragma unroll
                    for (int term = 0; term < KT; ++term)
                        qa[term][j] = o[term];
                }
                const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                lds_x[w][i][lane] = products<KT, 3, 2>(ka, sb, zero);
                lds_q[w][i][lane] = products<KT, 2, 1>(qa, sb, zero);
            }
        }
        fetch_kq(t + kChunk);
        __syncthreads();

        // R and e^b Q S of tokens 16 w ..
        const f32x4 eb = ebn, ed = edn;
        const int32_t bad = __builtin_amdgcn_readfirstlane(badn), lim = min(n, bad);
        const float whole = wholen;
        f32x4 x = lds_x[0][w][lane], o = lds_q[0][w][lane];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) {
            const f32x4 y = lds_x[i][w][lane], z = lds_q[i][w][lane];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[r] += y[r];
                o[r] += z[r];
            }
        }
        float v[4], check = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            v[r] = low(Type(), vn[r]);
            check = fmaf(v[r], 0.0f, check);
        }
        if (__ballot(check != check)) {   // values that are not finite: zeros, and a mark for what comes after them
            rare();
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int32_t token = 16 * w + 4 * g + r;
                if (!(fabsf(v[r]) < INFINITY)) {
                    v[r] = 0.0f;
                    if (token < n)
                        atomicMin(&lds_bad[parity][col], token);
                }
            }
            lds_odd[parity] = 1;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            x[r] = 16 * w + 4 * g + r < lim ? fmaf(-eb[r], x[r], v[r]) : 0.0f;
            o[r] *= eb[r];
        }
        fetch_v(t + kChunk, next);
#pragma unroll
        for (int term = 0; term < 3; ++term)
            lds_r[term][w / 2][lane][w & 1] = take4(x);
        __syncthreads();

        // U of tokens 16 w ..
        const bool odd = __builtin_amdgcn_readfirstlane(lds_odd[parity]) != 0;
        f32x4 u = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            u32x4 ta[3], rb[3];
#pragma unroll
            for (int term = 0; term < 3; ++term) {
                ta[term] = tn[term][c];
                rb[term] = *(const u32x4 *)lds_r[term][c][lane];
            }
            u = products<3, 3, 2>(ta, rb, u);
        }
        fetch_t(next);
        {
            f32x4 y = u, z;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                z[r] = u[r] * ed[r];
#pragma unroll
            for (int term = 0; term < 3; ++term) {
                lds_u[term][w / 2][lane][w & 1] = take4(z);
                if (term < 2)
                    lds_u[3 + term][w / 2][lane][w & 1] = take4(y);
            }
        }
        if (w == 0 && lane < 16) {   // the last chunk's marks have been read
            lds_bad[parity ^ 1][lane] = kChunk;
            if (lane == 0)
                lds_odd[parity ^ 1] = 0;
        }
        __syncthreads();

        // S, and the outputs of tokens 16 w ..
#pragma unroll
        for (int j = 0; j < EK; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                s[j][r] *= whole;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            u32x4 ub[3], ka[EK][KT];
#pragma unroll
            for (int term = 0; term < 3; ++term)
                ub[term] = *(const u32x4 *)lds_u[term][c][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < EK; ++j) {
                    uint32_t d[KT];
                    Split<Type>::of(__builtin_amdgcn_perm(kt[8 * c + 2 * i + 1], kt[8 * c + 2 * i],
                                                          j ? 0x07060302u : 0x05040100u), d);
#pragma unroll
                    for (int term = 0; term < KT; ++term)
                        ka[j][term][i] = d[term];
                }
#pragma unroll
            for (int j = 0; j < EK; ++j)
                s[j] = products<KT, 3, 2>(ka[j], ub, s[j]);
        }
        fetch_kt(t + kChunk);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            u32x4 ub[2], pa[PT];
#pragma unroll
            for (int term = 0; term < 2; ++term)
                ub[term] = *(const u32x4 *)lds_u[3 + term][c][lane];
#pragma unroll
            for (int term = 0; term < PT; ++term)
                pa[term] = pn[term][c];
            o = products<PT, 2, 1>(pa, ub, o);
        }
        fetch_p(next);
        int32_t reached = bad;
        if (odd) {
            rare();
            reached = min(reached, lds_bad[parity][col]);
        }
        if (odd || bad < n) {
            rare();
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                o[r] = 16 * w + 4 * g + r >= reached ? NAN : o[r];
#pragma unroll
                for (int j = 0; j < EK; ++j)
                    s[j][r] = reached < n ? NAN : s[j][r];
            }
        }
        const Rows rows = rows_of(op + (int64_t)t * ldo, n, ldo, 16, 2);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int32_t token = 16 * w + 4 * g + r;
            const uint32_t y = pack2(Type(), o[r] * a.scale, 0.0f);
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)y, rows, token < n ? 2 * (token * (uint32_t)ldo + col) : ~0u, 0, 0);
        }
    }
#pragma unroll
    for (int j = 0; j < EK; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            a.state_out[state_at + (int64_t)(EK * r + j) * a.Dv] = s[j][r];
}

int64_t places(int32_t T, int32_t num_seqs) { return num_seqs == 1 ? ((int64_t)T + kChunk - 1) / kChunk : T / kChunk + (int64_t)num_seqs; }

template <class Type, int DK>
hipError_t delta_of(const DeltaArgs &a, hipStream_t stream)
{
    Prepared<Type> *work = (Prepared<Type> *)a.work;
    const dim3 block(kDeltaThreads);
    const int slices = a.Dv / 16;
    const int64_t units = ((int64_t)a.B * a.H + 7) / 8 * 8;
    if (a.T > 0)
        delta_prepare_kernel<Type, DK><<<dim3((unsigned)places(a.T, a.B), a.H), block, 0, stream>>>(a, work);
    delta_chunk_kernel<Type, DK><<<dim3((unsigned)(units * slices)), block, 0, stream>>>(a, work, slices);
    return hipGetLastError();
}

}  // namespace

int64_t delta_workspace(int32_t T, int32_t num_seqs, int32_t H, int32_t type)
{
    return places(T, num_seqs) * H * (int64_t)(type ? sizeof(Prepared<Fp16>) : sizeof(Prepared<Bf16>));
}

hipError_t launch_delta(const DeltaArgs &a, hipStream_t stream)
{
    if (a.Dk == 64)
        return a.type ? delta_of<Fp16, 64>(a, stream) : delta_of<Bf16, 64>(a, stream);
    return a.type ? delta_of<Fp16, 128>(a, stream) : delta_of<Bf16, 128>(a, stream);
}

hipError_t launch_delta_step(const DeltaArgs &a, hipStream_t stream)
{
    a.type ? step_typed<Fp16>(a, stream) : step_typed<Bf16>(a, stream);
    return hipGetLastError();
}

}  // namespace w4a16
