// The gated delta rule, for gfx950:
//   S_t = e^{g_t} S_{t-1} + k_t u_t^T,   u_t = beta_t (v_t - e^{g_t} S_{t-1}^T k_t),   o_t = scale * q_t^T S_t.
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
// One work-group per sequence, head and 32 columns, a token at a time; the state stays in registers.
constexpr int kColumns = 32;

template <class Type, int DK>
__global__ __launch_bounds__(256) void delta_kernel(DeltaArgs a)
{
    typedef typename Type::T T;
    constexpr int RG = 256 / kColumns, ROWS = DK / RG;
    __shared__ float qs[DK], ks[DK], part[2][RG][kColumns];
    const int tid = threadIdx.x, col = tid % kColumns, rg = tid / kColumns;
    const int slices = a.Dv / kColumns, h = blockIdx.x / slices, c = (blockIdx.x % slices) * kColumns + col;
    const int hk = h / (a.H / a.Hk);
    const int64_t b = blockIdx.y;
    int64_t t0 = 0, t1 = a.T;
    if (a.cu) {
        t0 = min(max(a.cu[b], 0), a.T);
        t1 = max((int64_t)min(max(a.cu[b + 1], 0), a.T), t0);
    }
    const int64_t base = (b * a.H + h) * (int64_t)(DK * a.Dv) + (int64_t)rg * a.Dv + c;
    float s[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        s[r] = a.state_in ? a.state_in[base + (int64_t)r * RG * a.Dv] : 0.0f;
    for (int64_t t = t0; t < t1; ++t) {
        __syncthreads();
        if (tid < DK) {
            qs[tid] = Type::f(((const T *)a.q)[t * a.ldq + hk * a.hsq + tid]);
            ks[tid] = Type::f(((const T *)a.k)[t * a.ldk + hk * a.hsk + tid]);
        }
        __syncthreads();
        const float v = Type::f(((const T *)a.v)[t * a.ldv + h * a.hsv + c]), beta = a.beta[t * a.ldb + h * a.hsb];
        const float decay = expf(a.g[t * a.ldg + h * a.hsg]);
        float sk = 0.0f, sq = 0.0f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            s[r] *= decay;
            sk = fmaf(ks[rg + r * RG], s[r], sk);
        }
        part[0][rg][col] = sk;
        __syncthreads();
        sk = 0.0f;
        for (int w = 0; w < RG; ++w)
            sk += part[0][w][col];
        const float u = beta * (v - sk);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            s[r] = fmaf(ks[rg + r * RG], u, s[r]);
            sq = fmaf(qs[rg + r * RG], s[r], sq);
        }
        part[1][rg][col] = sq;
        __syncthreads();
        if (rg == 0) {
            sq = 0.0f;
            for (int w = 0; w < RG; ++w)
                sq += part[1][w][col];
            ((T *)a.out)[t * a.ldo + h * a.hso + c] = Type::from(a.scale * sq);
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        a.state_out[base + (int64_t)r * RG * a.Dv] = s[r];
}

}  // namespace

int64_t delta_workspace(int32_t, int32_t, int32_t, int32_t) { return 16; }

hipError_t launch_delta(const DeltaArgs &a, hipStream_t stream)
{
    const dim3 grid(a.H * (a.Dv / kColumns), a.B), block(256);
    if (a.Dk == 64)
        a.type ? delta_kernel<Fp16, 64><<<grid, block, 0, stream>>>(a) : delta_kernel<Bf16, 64><<<grid, block, 0, stream>>>(a);
    else
        a.type ? delta_kernel<Fp16, 128><<<grid, block, 0, stream>>>(a) : delta_kernel<Bf16, 128><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_delta_step(const DeltaArgs &a, hipStream_t stream)
{
    a.type ? step_typed<Fp16>(a, stream) : step_typed<Bf16>(a, stream);
    return hipGetLastError();
}

}  // namespace w4a16
