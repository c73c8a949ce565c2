// Attention of one new token per request over a paged cache of 8-bit codes with a scale for each block of
// tokens and head, for gfx950.
#include "attention_runs.h"

namespace w4a16 {

namespace {

// One work-group per request and query head; a wave takes every fourth position.
template <class Type>
__global__ __launch_bounds__(256) void quantized_attention_kernel(QuantizedAttentionArgs a)
{
    typedef typename Type::T T;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.y, h = blockIdx.x;
    const int kv = h / (a.Hq / a.Hkv);
    __shared__ float tops[4], totals[4], sums[4][256];
    const Span span = span_of(a, b);
    float q[4], o[4] = {};
    for (int e = 0; e < 4; ++e)
        q[e] = lane + 64 * e < a.dim ? Type::f(((const T *)a.q)[b * a.ldq + h * a.hsq + lane + 64 * e]) : 0.0f;
    auto value = [&](uint8_t code) {
        return a.int8 ? (float)(int8_t)code : __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
    };
    float top = -INFINITY, total = 0.0f;
    for (int64_t j = span.lo + wave; j < span.n; j += 4) {
        const int64_t at = j / a.page_size, slot = j - at * a.page_size;
        const int32_t page = a.table[b * a.row_stride + at];
        if (page < 0 || page >= a.num_pages)
            continue;
        const uint8_t *k = (const uint8_t *)a.k + page * a.k_page + slot * a.k_slot + kv * a.k_head;
        const uint8_t *v = (const uint8_t *)a.v + page * a.v_page + slot * a.v_slot + kv * a.v_head;
        const int64_t block = slot / a.block;
        const float ks = a.k_scale[page * a.k_scale_page + block * a.k_scale_block + kv * a.k_scale_head];
        const float vs = a.v_scale[page * a.v_scale_page + block * a.v_scale_block + kv * a.v_scale_head];
        float x = 0.0f;
        for (int e = 0; e < 4; ++e)
            if (lane + 64 * e < a.dim)
                x = fmaf(q[e], value(k[lane + 64 * e]), x);
        for (int d = 1; d < 64; d <<= 1)
            x += __shfl_xor(x, d);
        x *= ks * a.scale * kLog2e;
        const float m = fmaxf(x, top), ref = m == -INFINITY ? 0.0f : m;
        const float fade = __builtin_amdgcn_exp2f(top - ref), p = __builtin_amdgcn_exp2f(x - ref);
        top = m;
        total = total * fade + p;
        for (int e = 0; e < 4; ++e)
            if (lane + 64 * e < a.dim)
                o[e] = o[e] * fade + p * vs * value(v[lane + 64 * e]);
    }
    for (int e = 0; e < 4; ++e)
        sums[wave][lane + 64 * e] = o[e];
    if (lane == 0) {
        tops[wave] = top;
        totals[wave] = total;
    }
    __syncthreads();
    float m = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])), l = 0.0f, sum = 0.0f;
    const float ref = m == -INFINITY ? 0.0f : m;
    for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(tops[w] - ref);
        l += totals[w] * f;
        sum += sums[w][tid] * f;
    }
    if (tid < a.dim)
        ((T *)a.out)[b * a.ldo + h * a.hso + tid] = Type::from(l == 0.0f ? 0.0f : sum / l);
    if (tid == 0 && a.lse)
        a.lse[(int64_t)b * a.Hq + h] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

}  // namespace

hipError_t launch_quantized_attention(const QuantizedAttentionArgs &a, int, hipStream_t stream)
{
    const dim3 grid(a.Hq, a.B), block(256);
    a.type ? quantized_attention_kernel<Fp16><<<grid, block, 0, stream>>>(a)
           : quantized_attention_kernel<Bf16><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace w4a16
