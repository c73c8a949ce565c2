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
constexpr int kStepThreads = 256;

template <class Type, int DK, int DV, int CV>
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
        s[r] = *(const f32x4 *)(a.state_in + base + r * RG * DV);
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
    linear_step_kernel<Type, DK, DV, DV><<<dim3(a.H, a.B), dim3(kStepThreads), 0, stream>>>(a);
}

template <class Type>
void step_typed(const LinearArgs &a, hipStream_t stream)
{
    if (a.Dk == 64)
        a.Dv == 64 ? step_of<Type, 64, 64>(a, stream) : step_of<Type, 64, 128>(a, stream);
    else
        a.Dv == 64 ? step_of<Type, 128, 64>(a, stream) : step_of<Type, 128, 128>(a, stream);
}

// ---- packed sequences: the recurrence itself -----------------------------------------------------
// One wave per 64 columns of a head's state and sequence; a lane holds one column.
template <class Type, int DK>
__global__ __launch_bounds__(64) void linear_recurrent_kernel(LinearArgs a)
{
    typedef typename Type::T T;
    __shared__ float qs[DK], ks[DK];
    const int lane = threadIdx.x, parts = a.Dv / 64;
    const int h = blockIdx.x / parts, c = (blockIdx.x % parts) * 64 + lane;
    const int64_t b = blockIdx.y;
    int32_t t0 = 0, t1 = a.T;
    if (a.cu) {
        for (int s = 0; s <= b; ++s)
            t0 = max(t0, min(a.cu[s], a.T));
        t1 = max(t0, min(a.cu[b + 1], a.T));
    }
    const int64_t base = (b * a.H + h) * (int64_t)DK * a.Dv + c;
    float s[DK];
#pragma unroll
    for (int r = 0; r < DK; ++r)
        s[r] = a.state_in ? a.state_in[base + (int64_t)r * a.Dv] : 0.0f;
    const int hk = h / (a.H / a.Hk);
    for (int64_t t = t0; t < t1; ++t) {
        __syncthreads();
        for (int r = lane; r < DK; r += 64) {
            qs[r] = a.scale * Type::f(((const T *)a.q)[t * a.ldq + hk * a.hsq + r]);
            ks[r] = Type::f(((const T *)a.k)[t * a.ldk + hk * a.hsk + r]);
        }
        __syncthreads();
        const float v = Type::f(((const T *)a.v)[t * a.ldv + h * a.hsv + c]);
        const float decay = expf(a.g[t * a.ldg + h * a.hsg]);
        float acc = 0.0f;
#pragma unroll
        for (int r = 0; r < DK; ++r) {
            s[r] = fmaf(ks[r], v, decay * s[r]);
            acc = fmaf(qs[r], s[r], acc);
        }
        ((T *)a.out)[t * a.ldo + h * a.hso + c] = Type::from(acc);
    }
#pragma unroll
    for (int r = 0; r < DK; ++r)
        a.state_out[base + (int64_t)r * a.Dv] = s[r];
}

template <class Type>
void linear_typed(const LinearArgs &a, hipStream_t stream)
{
    const dim3 grid(a.H * (a.Dv / 64), a.B), block(64);
    if (a.Dk == 64)
        linear_recurrent_kernel<Type, 64><<<grid, block, 0, stream>>>(a);
    else
        linear_recurrent_kernel<Type, 128><<<grid, block, 0, stream>>>(a);
}

}  // namespace

int64_t linear_workspace(int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_linear(const LinearArgs &a, int, hipStream_t stream)
{
    a.type ? linear_typed<Fp16>(a, stream) : linear_typed<Bf16>(a, stream);
    return hipGetLastError();
}

hipError_t launch_linear_step(const LinearArgs &a, int, hipStream_t stream)
{
    a.type ? step_typed<Fp16>(a, stream) : step_typed<Bf16>(a, stream);
    return hipGetLastError();
}

}  // namespace w4a16
