// Attention of one new token per request over a paged key-value cache, for gfx950.
#include "mixers.h"
#include "mixer_types.h"

namespace w4a16 {

namespace {

// One wave per request and query head: 64 positions at a time, a lane scores one of them, then
// every lane sums its own values of the output over the 64. The maximum and the sum run along.
template <class Type, bool E4M3>
__global__ __launch_bounds__(64) void attention_kernel(AttentionArgs a)
{
    typedef typename Type::T T;
    __shared__ float qs[256], ps[64];
    __shared__ int64_t rows[64];
    const int lane = threadIdx.x, h = blockIdx.x, kv = h / (a.Hq / a.Hkv);
    const int64_t b = blockIdx.y;
    for (int d = lane; d < a.dim; d += 64)
        qs[d] = a.scale * Type::f(((const T *)a.q)[b * a.ldq + h * a.hsq + d]);
    __syncthreads();
    const int64_t n = min((int64_t)a.lens[b], (int64_t)a.max_pages * a.page_size);
    const int64_t lo = a.window ? max((int64_t)a.lens[b] - a.window, (int64_t)0) : 0;
    const float k_scale = E4M3 && a.k_scale ? a.k_scale[kv] : 1.0f;
    const float v_scale = E4M3 && a.v_scale ? a.v_scale[kv] : 1.0f;
    auto value = [&](const void *p, int64_t i) -> float {
        if (E4M3)
            return __builtin_amdgcn_cvt_f32_fp8(((const uint8_t *)p)[i], 0);
        return Type::f(((const T *)p)[i]);
    };
    float top = -INFINITY, sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t j0 = lo; j0 < n; j0 += 64) {
        const int64_t j = j0 + lane;
        int32_t page = -1;
        if (j < n)
            page = a.table[b * a.row_stride + j / a.page_size];
        const bool seen = page >= 0 && page < a.num_pages;
        float x = -INFINITY;
        __syncthreads();
        rows[lane] = -1;
        if (seen) {
            const int64_t slot = j % a.page_size;
            const int64_t at = page * a.k_page + slot * a.k_slot + kv * a.k_head;
            rows[lane] = page * a.v_page + slot * a.v_slot + kv * a.v_head;
            float dot = 0.0f;
            for (int d = 0; d < a.dim; ++d)
                dot = fmaf(qs[d], value(a.k, at + d), dot);
            x = dot * k_scale;
        }
        float m = x;
        for (int d = 1; d < 64; d <<= 1)
            m = fmaxf(m, __shfl_xor(m, d));
        m = fmaxf(m, top);
        const float p = seen ? expf(x - (m == -INFINITY ? 0.0f : m)) : 0.0f;
        const float fade = top == -INFINITY ? 0.0f : expf(top - m);
        float s = p;
        for (int d = 1; d < 64; d <<= 1)
            s += __shfl_xor(s, d);
        sum = sum * fade + s;
        top = m;
        ps[lane] = p;
        __syncthreads();
        for (int e = 0; e < 4; ++e)
            acc[e] *= fade;
        for (int i = 0; i < 64; ++i)
            if (rows[i] >= 0)
                for (int e = 0; e < 4; ++e)
                    if (lane + 64 * e < a.dim)
                        acc[e] = fmaf(ps[i], value(a.v, rows[i] + lane + 64 * e), acc[e]);
    }
    for (int e = 0; e < 4; ++e)
        if (lane + 64 * e < a.dim)
            ((T *)a.out)[b * a.ldo + h * a.hso + lane + 64 * e] =
                Type::from(sum > 0.0f || sum != sum ? acc[e] * v_scale / sum : 0.0f);
    if (a.lse && lane == 0)
        a.lse[b * a.Hq + h] = top == -INFINITY ? -INFINITY : top + logf(sum);
}

}  // namespace

int64_t attention_workspace(int32_t, int32_t, int32_t) { return 16; }

hipError_t launch_attention(const AttentionArgs &a, int, hipStream_t stream)
{
    const dim3 grid(a.Hq, a.B), block(64);
    if (a.e4m3)
        a.type ? attention_kernel<Fp16, true><<<grid, block, 0, stream>>>(a)
               : attention_kernel<Bf16, true><<<grid, block, 0, stream>>>(a);
    else
        a.type ? attention_kernel<Fp16, false><<<grid, block, 0, stream>>>(a)
               : attention_kernel<Bf16, false><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace w4a16
