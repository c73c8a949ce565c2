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
//
// As for linear attention's single token, 32 columns to a work-group below 128 of (request, head), a whole state
// and streaming loads and stores from there on: 1 request of 32 heads 4.0 us, 250 requests 173 to 186 us (5.7 to 6.1
// TB/s).
//
// What is not finite counts as NaN, so that it reaches the same places as in packed sequences: an infinite k_i, v, beta or
// decay would leave zeros and infinities in the state.
constexpr int kStepThreads = 256;

__device__ __forceinline__ float finite_or_nan(float x) { return fabsf(x) < INFINITY ? x : NAN; }

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
        ks[tid] = finite_or_nan(Type::f(((const T *)a.k)[b * a.ldk + hk * a.hsk + tid]));
    }
    const T *vp = (const T *)a.v + b * a.ldv + h * a.hsv + c0;
    f32x4 v, sk = {0.0f, 0.0f, 0.0f, 0.0f}, sq = sk;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = finite_or_nan(Type::f(vp[e]));
    const float g = a.g[b * a.ldg + h * a.hsg], decay = g < INFINITY ? expf(g) : NAN;
    const float beta = finite_or_nan(a.beta[b * a.ldb + h * a.hsb]);
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
//
// Roundings. Everything but P reaches the state, so S, R, T and e^(b_63 - b) U enter their products (16x16x32, bfloat16)
// as sums of three bfloat16 values, of which the products above 2^-24 of the whole are taken: 3 where K, which is
// bfloat16, is the other operand, 6 for T R. float32 products would take 16 times a bfloat16 one's time. Float16 K and Q
// are sums of two (5 products); with float16 operands the state's columns would need factors of their own, found
// from chunk to chunk. The outputs take two values of S, U and P. Errors against float64 over 20000 tokens: states
// 1.0e-7 of the norm (in float32 throughout 1.4e-7); outputs are off by their own rounding alone, 1.66e-3 (with one value of
// P 2.2e-3, and 657 us for these instead of 692: 15 for 6 KB more to write per chunk and head, 20 for loading it).
// Decays are summed in float64, and differences of sums taken there.
//
// What bounds it: 20000 tokens of 32 heads of 128 (16 for q and k) take 117 us for T and P (0.48 GB: 4.1 TB/s, where a
// copy of 4 GiB reaches 4.7) and 606 us for the chunks (medians of a trace; 694 us for both by events), a chain of 313
// steps. A copy with the cycle counter read between phases, and one value of P, showed 4060 cycles a step in the
// carrying waves: 1040 on X, 540 on R, 1290 on U, 615 on S and 570 at the three barriers between. By count, their 36
// products would take 580 and the 182 KB that a step moves through LDS 1450 at 128 bytes a cycle; the rest is latency. 8
// heads, which leave most CUs idle, take 513 us where 32 take 692 by the same loop. Steps that counted, whole calls of this
// size, with one value of P: outputs by waves of their own together with K's other view through LDS and pieces of 8 bytes
// for V and the outputs 982 -> 720 us; loads before barriers rather than in a phase's middle 781 -> 692 on the way there; S
// read for the outputs after R and K turned early 661 -> 656; 16 spilled registers in float16 (2 are left) 1513 -> 781.
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
constexpr int kScoreTerms = 2;
struct Prepared {
    u32x4 t[3][kFrags][64], p[kScoreTerms][kFrags][64];   // first operands: T in three bfloat16 terms, P in two
    float eb[kChunk], ed[kChunk];                     // e^b, e^(b_63 - b)
    int32_t bad;                                      // first token with a k, beta or decay that is not finite, or 64
    float whole;                                      // e^b_63
    int32_t pad[30];
};
static_assert(sizeof(Prepared) % 128 == 0, "whole cache lines");

// Sequence s has its chunks' places from here on: as many as it has chunks, or more, lie before the next one's.
__device__ __forceinline__ int32_t first_place(const DeltaArgs &a, int s)
{
    return a.cu ? min(max(a.cu[s], 0), a.T) / kChunk + s : 0;
}
__device__ __forceinline__ void tokens_of(const DeltaArgs &a, int s, int32_t *t0, int32_t *t1)
{
    *t0 = a.cu ? __builtin_amdgcn_readfirstlane(min(max(a.cu[s], 0), a.T)) : 0;
    *t1 = a.cu ? max(__builtin_amdgcn_readfirstlane(min(max(a.cu[s + 1], 0), a.T)), *t0) : a.T;
}

// The tokens [t0, t1) of the chunk at `place`; false where it is none's. Its sequence is the last one whose places
// start there or before: 63 are looked through at a time, so that the last look has both of its ends.
__device__ __forceinline__ bool chunk_at(const DeltaArgs &a, int32_t place, int32_t *t0, int32_t *t1)
{
    if (!a.cu) {
        *t0 = place * kChunk;
        *t1 = a.T;
    } else {
        const int lane = threadIdx.x & 63;
        for (int lo = 0, n = a.B;;) {
            const int step = (n + 62) / 63, seq = lo + lane * step;
            const int32_t start = min(max(a.cu[min(seq, a.B)], 0), a.T);
            const uint64_t hit = __ballot(lane * step < n && start / kChunk + seq <= place);
            if (!hit)
                return false;
            const int k = 63 - __builtin_clzll(hit);
            if (step == 1) {
                const int32_t first = __builtin_amdgcn_readlane(start, k);
                *t1 = __builtin_amdgcn_readlane(start, k + 1);
                const int64_t at = first + (int64_t)(place - first / kChunk - lo - k) * kChunk;
                if (at >= *t1)
                    return false;
                *t0 = (int32_t)at;
                break;
            }
            lo += k * step;
            n = min(step, n - k * step);
        }
    }
    return *t0 < *t1;
}

__device__ __forceinline__ f32x4 mfma_f32(f32x4 a, f32x4 b, f32x4 c)   // contraction of 16, lane group g has 4g ..
{
#pragma unroll
    for (int s = 0; s < 4; ++s)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[s], b[s], c, 0, 0, 0);
    return c;
}

typedef double f64x4 __attribute__((ext_vector_type(4)));

// x or zero, without the branch around x that a selection becomes.
__device__ __forceinline__ float masked(float x, bool keep)
{
    return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & (keep ? ~0u : 0u));
}

// Blocks along x, an axis on which a launch holds fewer than 2^32 threads; more of them go along y (2 us of 656 for 20000
// tokens of 32 heads; with the width read from the grid 11).
constexpr int kWide = 20;

// Work-groups go to the 8 XCDs in turn, and each XCD has its own L2. Of `groups` that read the same rows, each of
// `size` work-groups, all of one go to one XCD: group and number inside it of a work-group.
struct Xcd {
    uint32_t groups, size;
    __device__ __forceinline__ bool place(uint32_t *group, uint32_t *inside) const
    {
        const uint32_t block = blockIdx.y << kWide | blockIdx.x;
        const uint32_t rest = block / 8, eight = rest / size;
        *inside = rest - eight * size;
        *group = eight * 8 + block % 8;
        return *group < groups;
    }
    dim3 grid() const
    {
        const int64_t blocks = ((int64_t)groups + 7) / 8 * 8 * size, wide = 1 << kWide;
        return blocks <= wide ? dim3((unsigned)blocks) : dim3((unsigned)wide, (unsigned)((blocks + wide - 1) / wide));
    }
};

// T and P of one chunk and head. Wave w has rows 16 w ..; products of K rows are formed both ways round, so that
// each result lies in the lanes where it is an operand. A and T are float32: diagonal blocks of 16 x 16 by
// substitution (no powers of A, which may be large where T is not), the others by float32 matrix products,
//   T_ij = -(sum_{j<m<=i} T_im A_mj) T_jj.
// (K of the other waves through LDS, sums of decays by vectors: 140 -> 117 us for 10016 of them; heads that share K on
// one XCD: 107.) Alone, for one chunk, it takes 7.5 us: a chain of loads, 15 steps of substitution and 9 products in turn.
template <class Type, int DK>
__global__ __launch_bounds__(kDeltaThreads) void delta_prepare_kernel(DeltaArgs a, Prepared *work, Xcd xcd)
{
    constexpr int C = DK / 32;
    __shared__ u32x4 lds_k[kWaves - 1][C][64];
    __shared__ f32x4 lds_a[10][64], lds_t[kWaves][64];
    __shared__ __align__(16) double lds_b[kChunk];
    __shared__ __align__(16) float lds_beta[kChunk];
    __shared__ int32_t lds_bad[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    uint32_t group, inside;   // a place and head of K, heads that share it
    if (!xcd.place(&group, &inside))
        return;
    const int32_t place = (int32_t)(group / (uint32_t)a.Hk);
    const int hk = (int)(group - (uint32_t)place * (uint32_t)a.Hk), h = hk * (int)xcd.size + (int)inside;
    int32_t t0, t1;
    if (!chunk_at(a, place, &t0, &t1))
        return;
    const int32_t n = min(t1 - t0, kChunk);
    Prepared &to = work[(int64_t)place * a.H + h];

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
    if (w < kWaves - 1) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            lds_k[w][c][lane] = ki[c];
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

    const double bi_col = lds_b[16 * w + col];
    const f64x4 bi = *(const f64x4 *)&lds_b[16 * w + 4 * g];
    const f32x4 beta_i = *(const f32x4 *)&lds_beta[16 * w + 4 * g];
    f32x4 own = {0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 p[kScoreTerms][2] = {};
#pragma unroll
    for (int j = 0; j < kWaves; ++j) {
        if (j > w)
            continue;
        u32x4 kj[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            kj[c] = j == w ? ki[c] : lds_k[min(j, kWaves - 2)][c][lane];
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            x = mfma(Type(), ki[c], kj[c], x);   // tokens i = 16 w + 4 g .. in the lane of token j = 16 j + col
            y = mfma(Type(), kj[c], qi[c], y);   // tokens j = 16 j + 4 g .. in the lane of token i = 16 w + col
        }
        const double bj_col = lds_b[16 * j + col];
        const f64x4 bj = *(const f64x4 *)&lds_b[16 * j + 4 * g];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float a_ij = x[r] * __builtin_amdgcn_exp2f((float)(bi[r] - bj_col)) * beta_i[r];
            const float p_ij = y[r] * __builtin_amdgcn_exp2f((float)(bi_col - bj[r]));
            const int32_t i = 16 * w + 4 * g + r, j2 = 16 * j + 4 * g + r;
            x[r] = masked(a_ij, (16 * j + col < i) & (i < lim));
            y[r] = masked(p_ij, (j2 <= 16 * w + col) & (j2 < lim));
        }
        lds_a[w * (w + 1) / 2 + j][lane] = x;
#pragma unroll
        for (int term = 0; term < kScoreTerms; ++term) {
            const u32x2 o = take4(y);
            p[term][j / 2][2 * (j & 1)] = o[0];
            p[term][j / 2][2 * (j & 1) + 1] = o[1];
        }
    }
#pragma unroll
    for (int term = 0; term < kScoreTerms; ++term)
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

// The products of NA and NB terms of two operands that matter (of term i and j with i + j <= MOST), small ones
// first, for N results side by side: none waits for the one before it.
template <int NA, int NB, int MOST, int N, class A, class B>
__device__ __forceinline__ void products(const A &a, const B &b, f32x4 *c)
{
#pragma unroll
    for (int sum = MOST; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (sum - i >= 0 && sum - i < NB)
#pragma unroll
                for (int x = 0; x < N; ++x)
                    c[x] = mfma_words(a(x, i), b(x, sum - i), c[x]);
}

// What a work-group's waves share. Operands that go from wave to wave lie as the reader's lanes need them.
template <class Words>
struct DeltaLds {
    f32x4 x[kWaves][kWaves][64];                      // K S: sums over a wave's rows of S, for each tile of tokens
    Words s[2][kWaves][64];                           // S, two terms
    u32x2 r[3][2][64][2], u[3][2][64][2], uo[2][2][64][2];   // R, e^(b_63 - b) U, U
    f32x4 v[kWaves][64];                              // V: tokens 16 w + 4 g .. of a column
    Words k[kWaves][kChunk][5];                       // a wave's part of K, rows 4 words or 2 and a pad of as many
    int32_t bad[2][16], odd[2];                       // values that are not finite: first tokens by column, whether any
};

struct DeltaUnit {
    int32_t t0, t1, hk, h, c0;
    int64_t unit;
};

// Waves 0 to 3 carry the state: wave w holds the rows of S with dk in [DK / 4 w, DK / 4 (w + 1)), in float32, and
// multiplies K by them as they are: a lane's values of S are the second operand's, for the same dims of a K row. The
// four sums of X meet in LDS; wave w takes the tokens 16 w .. on to R and U, which all need.
template <class Type, int DK, class Lds>
__device__ __forceinline__ void carry_state(const DeltaArgs &a, const Prepared *from, const DeltaUnit &d, int w, Lds &lds)
{
    constexpr int EK = DK / 64, NW = 2 * EK, KT = Split<Type>::terms;
    constexpr int SIDE = KT == 1 ? kWaves : 2;   // tiles of X side by side, as many as registers allow
    typedef typename WordsOf<NW>::T Words;
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
    const int32_t t0 = d.t0, t1 = d.t1;
    const uint16_t *k_rows = (const uint16_t *)a.k + d.hk * a.hsk;
    const int32_t ldk = (int32_t)a.ldk;

    // s[j][r]: row DK / 4 w + EK (4 g + r) + j
    const int32_t state_at = (DK / 4 * w + EK * 4 * g) * a.Dv + d.c0 + col, state_size = DK * a.Dv;
    f32x4 s[EK];
    {
        const Rows from = __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(a.state_in + d.unit * state_size), 0,
                                                            a.state_in ? 4 * state_size : 0, 0x00027000);
#pragma unroll
        for (int j = 0; j < EK; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                s[j][r] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                    from, 4 * (state_at + (EK * r + j) * a.Dv), 0, 0));
    }

    Words kn[kWaves];        // rows 16 i + col, this wave's dims from 4 EK g on
    u32x4 tn[3][2];
    f32x4 ebn, edn;
    u32x2 endn = {kChunk, 0};
    auto fetch_k = [&](int32_t t) {
        const Rows kr = rows_of(k_rows + (int64_t)t * ldk, t1 - t, ldk, DK, 2);
#pragma unroll
        for (int i = 0; i < kWaves; ++i)
            kn[i] = WordsOf<NW>::load(kr, 2 * ((16 * i + col) * (uint32_t)ldk + DK / 4 * w + 4 * EK * g));
    };
    auto prepared = [&](int32_t t) {   // zeros past the last chunk; operands that are none lie past its end
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>((const void *)from), 0,
                                                 t < t1 ? sizeof(Prepared) : 0, 0x00027000);
    };
    auto fetch_t = [&](Rows x) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                tn[i][c] = load4(x, c <= w / 2 ? (uint32_t)((i * kFrags + frag(w, c)) * 64 + lane) * 16 : ~0u);
    };
    auto fetch_factors = [&](Rows x) {
        constexpr uint32_t at = (3 + kScoreTerms) * kFrags * 64 * 16;
        ebn = __builtin_bit_cast(f32x4, load4(x, at + 4 * (16 * w + 4 * g)));
        edn = __builtin_bit_cast(f32x4, load4(x, at + 4 * (kChunk + 16 * w + 4 * g)));
        endn = __builtin_amdgcn_raw_buffer_load_b64(x, at + 8 * kChunk, 0, 0);
    };
    if (t0 < t1) {
        const Rows x = prepared(t0);
        fetch_k(t0);
        fetch_factors(x);
        fetch_t(x);
    }
    // The loop would wait for them, and then in every round for all that is in flight.
#pragma unroll
    for (int j = 0; j < EK; ++j)
        asm volatile("" : "+v"(s[j]));

    int parity = 0;
    for (int32_t t = t0; t < t1; t += kChunk, parity ^= 1) {
        const int32_t n = min(t1 - t, kChunk);
        from += a.H;
        const Rows next = prepared(t + kChunk);
        // X: this wave's dims
        {
            Words sb[3];
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                float x = EK == 2 ? s[0][i] : s[0][2 * i], y = EK == 2 ? s[EK - 1][i] : s[0][2 * i + 1];
#pragma unroll
                for (int term = 0; term < 3; ++term)
                    sb[term][i] = take(Bf16(), x, y);
            }
            lds.s[0][w][lane] = sb[0];
            lds.s[1][w][lane] = sb[1];
#pragma unroll
            for (int i = 0; i < kWaves; ++i)   // for a look at it from the other side
                lds.k[w][16 * i + col][g] = kn[i];
#pragma unroll
            for (int i0 = 0; i0 < kWaves; i0 += SIDE) {
                Words ka[SIDE][KT];
                f32x4 x[SIDE];
#pragma unroll
                for (int i = 0; i < SIDE; ++i) {
                    x[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < NW; ++j) {
                        uint32_t o[KT];
                        Split<Type>::of(kn[i0 + i][j], o);
#pragma unroll
                        for (int term = 0; term < KT; ++term)
                            ka[i][term][j] = o[term];
                    }
                }
                products<KT, 3, 2, SIDE>([&](int i, int term) { return ka[i][term]; },
                                         [&](int, int term) { return sb[term]; }, x);
#pragma unroll
                for (int i = 0; i < SIDE; ++i)
                    lds.x[w][i0 + i][lane] = x[i];
                if (SIDE < kWaves)
                    __builtin_amdgcn_sched_barrier(0);
            }
        }
        fetch_k(t + kChunk);
        __syncthreads();

        // R of tokens 16 w ..
        const f32x4 eb = ebn, ed = edn;
        const int32_t bad = __builtin_amdgcn_readfirstlane(endn[0]), lim = min(n, bad);
        const uint32_t whole_bits = endn[1];
        const float whole = __builtin_bit_cast(float, whole_bits);
        f32x4 xs[kWaves];
#pragma unroll
        for (int i = 0; i < kWaves; ++i)
            xs[i] = lds.x[i][w][lane];
        const f32x4 v = lds.v[w][lane];
        __builtin_amdgcn_sched_barrier(0);
        f32x4 x;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            x[r] = fmaf(-eb[r], (xs[0][r] + xs[1][r]) + (xs[2][r] + xs[3][r]), v[r]);
        if (lim < kChunk) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                x[r] = 16 * w + 4 * g + r < lim ? x[r] : 0.0f;
        }
#pragma unroll
        for (int term = 0; term < 3; ++term)
            lds.r[term][w / 2][lane][w & 1] = take4(x);
        fetch_factors(next);
        __syncthreads();

        // U of tokens 16 w ..
        const bool odd = __builtin_amdgcn_readfirstlane(lds.odd[parity]) != 0;
        f32x4 u[2];
        u32x4 rb[2][3];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            u[c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int term = 0; term < 3; ++term)
                rb[c][term] = *(const u32x4 *)lds.r[term][c][lane];
        }
        uint32_t kt[16];   // K with tokens in pairs: dims EK col .. of tokens 32 c + 16 x + 4 g + e
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const uint16_t *p = (const uint16_t *)lds.k[w][32 * (e / 8) + 16 * (e / 4 % 2) + 4 * g + e % 4] + EK * col;
            kt[e] = EK == 2 ? *(const uint32_t *)p : *p;
        }
        __builtin_amdgcn_sched_barrier(0);
        products<3, 3, 2, 2>([&](int c, int term) { return tn[term][c]; },
                             [&](int c, int term) { return rb[c][term]; }, u);
        u32x4 kp[2][EK];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < EK; ++j)
                    kp[c][j][i] = __builtin_amdgcn_perm(kt[8 * c + 2 * i + 1], kt[8 * c + 2 * i], j ? 0x07060302u : 0x05040100u);
        {
            f32x4 y, z;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                y[r] = u[0][r] + u[1][r];
                z[r] = y[r] * ed[r];
            }
#pragma unroll
            for (int term = 0; term < 3; ++term)
                lds.u[term][w / 2][lane][w & 1] = take4(z);
#pragma unroll
            for (int term = 0; term < 2; ++term)
                lds.uo[term][w / 2][lane][w & 1] = take4(y);
        }
        if (w == 0 && lane < 16) {   // the last chunk's marks have been read
            lds.bad[parity ^ 1][lane] = kChunk;
            if (lane == 0)
                lds.odd[parity ^ 1] = 0;
        }
        fetch_t(next);
        __syncthreads();

        // S
        {
            f32x4 sum[2 * EK];   // of each half of the chunk
#pragma unroll
            for (int j = 0; j < EK; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    sum[j][r] = s[j][r] * whole;
                    sum[EK + j][r] = 0.0f;
                }
            constexpr int HALVES = KT == 1 ? 2 : 1;   // side by side
#pragma unroll
            for (int c0 = 0; c0 < 2; c0 += HALVES) {
                u32x4 ub[HALVES][3], ka[HALVES][EK][KT];
#pragma unroll
                for (int c = 0; c < HALVES; ++c) {
#pragma unroll
                    for (int term = 0; term < 3; ++term)
                        ub[c][term] = *(const u32x4 *)lds.u[term][c0 + c][lane];
#pragma unroll
                    for (int j = 0; j < EK; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t o[KT];
                            Split<Type>::of(kp[c0 + c][j][i], o);
#pragma unroll
                            for (int term = 0; term < KT; ++term)
                                ka[c][j][term][i] = o[term];
                        }
                }
                products<KT, 3, 2, HALVES * EK>([&](int x, int term) { return ka[x / EK][x % EK][term]; },
                                                [&](int x, int term) { return ub[x / EK][term]; }, sum + c0 * EK);
                if (HALVES == 1)
                    __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int j = 0; j < EK; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    s[j][r] = sum[j][r] + sum[EK + j][r];
        }
        if (odd || bad < n) {
            rare();
            const int32_t reached = min(bad, lds.bad[parity][col]);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < EK; ++j)
                    s[j][r] = reached < n ? NAN : s[j][r];
        }
    }
#pragma unroll
    for (int j = 0; j < EK; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            a.state_out[d.unit * state_size + state_at + (EK * r + j) * a.Dv] = s[j][r];
}

// Waves 4 to 7 make the outputs, next to the others on their SIMDs: wave 4 + w those of the tokens 16 w .., transposed,
// so that a lane has four columns of one token. They also bring V to the others, as float32.
template <class Type, int DK, class Lds>
__device__ __forceinline__ void make_outputs(const DeltaArgs &a, const Prepared *from, const DeltaUnit &d, int w, Lds &lds)
{
    constexpr int EK = DK / 64, NW = 2 * EK, KT = Split<Type>::terms;
    typedef typename WordsOf<NW>::T Words;
    const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4, token = 16 * w + col;
    const int32_t t0 = d.t0, t1 = d.t1;
    const uint16_t *qp = (const uint16_t *)a.q + d.hk * a.hsq, *vp = (const uint16_t *)a.v + d.h * a.hsv + d.c0;
    uint16_t *op = (uint16_t *)a.out + d.h * a.hso + d.c0;
    const int32_t ldq = (int32_t)a.ldq, ldv = (int32_t)a.ldv, ldo = (int32_t)a.ldo;
    Words qn[kWaves];   // dims of wave i from 4 EK g on
    u32x4 pn[kScoreTerms][2];
    u32x2 vn;           // columns 4 g ..
    float ebn = 0.0f;
    int32_t badn = kChunk;
    constexpr uint32_t at = (3 + kScoreTerms) * kFrags * 64 * 16;
    auto prepared = [&](int32_t t) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>((const void *)from), 0,
                                                 t < t1 ? sizeof(Prepared) : 0, 0x00027000);
    };
    auto fetch_v = [&](int32_t t) {
        vn = WordsOf<2>::load(rows_of(vp + (int64_t)t * ldv, t1 - t, ldv, 16, 2), 2 * (token * (uint32_t)ldv + 4 * g));
    };
    auto fetch_q = [&](int32_t t, Rows x) {
        const Rows qr = rows_of(qp + (int64_t)t * ldq, t1 - t, ldq, DK, 2);
#pragma unroll
        for (int i = 0; i < kWaves; ++i)
            qn[i] = WordsOf<NW>::load(qr, 2 * (token * (uint32_t)ldq + DK / 4 * i + 4 * EK * g));
        ebn = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(x, at + 4 * token, 0, 0));
        badn = __builtin_amdgcn_raw_buffer_load_b32(x, at + 8 * kChunk, 0, 0);
    };
    auto fetch_p = [&](Rows x) {
#pragma unroll
        for (int i = 0; i < kScoreTerms; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                pn[i][c] = load4(x, c <= w / 2 ? (uint32_t)(((3 + i) * kFrags + frag(w, c)) * 64 + lane) * 16 : ~0u);
    };
    if (t0 < t1) {
        const Rows x = prepared(t0);
        fetch_v(t0);
        fetch_q(t0, x);
        fetch_p(x);
    }
    int parity = 0;
    for (int32_t t = t0; t < t1; t += kChunk, parity ^= 1) {
        const int32_t n = min(t1 - t, kChunk);
        from += a.H;
        const Rows next = prepared(t + kChunk);
        float v[4] = {low(Type(), vn[0]), high(Type(), vn[0]), low(Type(), vn[1]), high(Type(), vn[1])}, check = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            check = fmaf(v[r], 0.0f, check);
        if (__ballot(check != check)) {   // values that are not finite: zeros, and a mark for what comes after them
            rare();
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (!(fabsf(v[r]) < INFINITY)) {
                    v[r] = 0.0f;
                    if (token < n)
                        atomicMin(&lds.bad[parity][4 * g + r], token);
                }
            lds.odd[parity] = 1;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
            lds.v[w][16 * (col / 4) + 4 * g + r][col % 4] = v[r];
        fetch_v(t + kChunk);
        Words qa[kWaves][KT];
#pragma unroll
        for (int i = 0; i < kWaves; ++i)
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                uint32_t x[KT];
                Split<Type>::of(qn[i][j], x);
#pragma unroll
                for (int term = 0; term < KT; ++term)
                    qa[i][term][j] = x[term];
            }
        const float eb = ebn;
        const int32_t bad = __builtin_amdgcn_readfirstlane(badn);
        __syncthreads();
        __syncthreads();

        f32x4 o[kWaves];   // Q S, over the rows of each wave
        {
            Words sb[kWaves][2];
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                sb[i][0] = lds.s[0][i][lane];
                sb[i][1] = lds.s[1][i][lane];
            }
            products<2, KT, 1, kWaves>([&](int i, int term) { return sb[i][term]; },
                                       [&](int i, int term) { return qa[i][term]; }, o);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                o[0][r] = eb * ((o[0][r] + o[1][r]) + (o[2][r] + o[3][r]));
                o[1][r] = 0.0f;
            }
        }
        fetch_q(t + kChunk, next);
        __syncthreads();

        const bool odd = __builtin_amdgcn_readfirstlane(lds.odd[parity]) != 0;
        {
            u32x4 ub[2][2];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int term = 0; term < 2; ++term)
                    ub[c][term] = *(const u32x4 *)lds.uo[term][c][lane];
            products<2, kScoreTerms, 1, 2>([&](int c, int term) { return ub[c][term]; },
                                           [&](int c, int term) { return pn[term][c]; }, o);
        }
        fetch_p(next);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            o[0][r] = (o[0][r] + o[1][r]) * a.scale;
        if (odd || bad < n) {
            rare();
#pragma unroll
            for (int r = 0; r < 4; ++r)
                o[0][r] = token >= min(bad, lds.bad[parity][4 * g + r]) ? NAN : o[0][r];
        }
        const u32x2 y = {pack2(Type(), o[0][0], o[0][1]), pack2(Type(), o[0][2], o[0][3])};
        __builtin_amdgcn_raw_buffer_store_b64(y, rows_of(op + (int64_t)t * ldo, n, ldo, 16, 2),
                                              token < n ? 2 * (token * (uint32_t)ldo + 4 * g) : ~0u, 0, 0);
    }
}

// A work-group goes over the chunks of one sequence, head and 16 columns.
constexpr int kChunkThreads = 512;

template <class Type, int DK>
__global__ __launch_bounds__(kChunkThreads, 4) void delta_chunk_kernel(DeltaArgs a, const Prepared *work, Xcd xcd,
                                                                       int heads)
{
    typedef typename WordsOf<DK / 32>::T Words;
    __shared__ __align__(16) DeltaLds<Words> lds;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t group, inside;   // `heads` heads of a sequence, their slices
    if (!xcd.place(&group, &inside))
        return;
    const uint32_t slices = xcd.size / (uint32_t)heads, unit = group * (uint32_t)heads + inside / slices;
    const int seq = (int)(unit / (uint32_t)a.H);
    DeltaUnit d;
    d.unit = unit;
    d.h = (int)(unit - (uint32_t)seq * (uint32_t)a.H);
    d.hk = d.h / (a.H / a.Hk);
    d.c0 = (int)(inside % slices) * 16;
    tokens_of(a, seq, &d.t0, &d.t1);
    const Prepared *from = work + (int64_t)__builtin_amdgcn_readfirstlane(first_place(a, seq)) * a.H + d.h;
    if (tid < 32)
        lds.bad[tid >> 4][tid & 15] = kChunk;
    if (tid < 2)
        lds.odd[tid] = 0;
    __syncthreads();
    if (wave < kWaves) {
        __builtin_amdgcn_s_setprio(3);   // the others have time
        carry_state<Type, DK>(a, from, d, wave, lds);
    } else {
        make_outputs<Type, DK>(a, from, d, wave - kWaves, lds);
    }
}

int64_t places(int32_t T, int32_t num_seqs) { return num_seqs == 1 ? ((int64_t)T + kChunk - 1) / kChunk : T / kChunk + (int64_t)num_seqs; }

template <class Type, int DK>
hipError_t delta_of(const DeltaArgs &a, hipStream_t stream)
{
    Prepared *work = (Prepared *)a.work;
    const uint32_t share = (uint32_t)(a.H / a.Hk), slices = (uint32_t)a.Dv / 16;
    if (a.T > 0) {
        const Xcd xcd{(uint32_t)(places(a.T, a.B) * a.Hk), share};
        delta_prepare_kernel<Type, DK><<<xcd.grid(), dim3(kDeltaThreads), 0, stream>>>(a, work, xcd);
    }
    // Heads that share K and Q together, unless that leaves some of the 8 XCDs with more than 5/4 of the average.
    const uint32_t groups = (uint32_t)a.B * (uint32_t)a.Hk, eights = (groups + 7) / 8;
    const int heads = eights * 32 <= groups * 5 ? (int)share : 1;
    const Xcd xcd{(uint32_t)a.B * (uint32_t)a.H / (uint32_t)heads, slices * (uint32_t)heads};
    delta_chunk_kernel<Type, DK><<<xcd.grid(), dim3(kChunkThreads), 0, stream>>>(a, work, xcd, heads);
    return hipGetLastError();
}

}  // namespace

int64_t delta_workspace(int32_t T, int32_t num_seqs, int32_t H)
{
    if (places(T, num_seqs) * H > 1 << 30)   // 34 TB of them
        return -1;
    return places(T, num_seqs) * H * (int64_t)sizeof(Prepared);
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
