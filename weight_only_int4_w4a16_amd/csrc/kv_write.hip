// Writes into the paged key-value cache for gfx950: a token's rows go to its slot, as they are or
// divided by the head's scale and rounded to e4m3. Memory-bound: 2 bytes read and 2 or 1 written per
// value. A thread moves the values of one 16-byte store at a time (8, or 16 as e4m3) and stays with its
// piece of the row, eight work-groups per CU going over the tokens: head, dims and scale are worked out
// once, and the slot's page by a multiplication. 16411 tokens of 8 heads of 128 as e4m3: 19.7 us (5.1 TB/s);
// 100000 tokens: e4m3 120 us (5.1), bfloat16 155 us (5.3). With the divisions of a flat index per piece the
// first took 25 to 28 us where this took 22; with 4, 8 and 16 work-groups per CU the last takes 162, 155 and 156 us,
// the others differ less.
//
// The e4m3 code is that of the float32 quotient x / scale. With r = 1 / scale correctly rounded,
// q0 = x r and q = q0 - (q0 scale - x) r (two fused operations) is that quotient exactly wherever
// nothing over- or underflows (Markstein), for one division per thread; scales far from 1 take the
// division itself. (With x - q0 scale, which is +0 for -0, a zero would lose its sign.)
#include "mixers.h"
#include "mixer_types.h"

namespace w4a16 {

namespace {

constexpr int kThreads = 256;

// slot / page_size as a multiplication: m = ceil(2^(31 + l) / page_size), l = ceil(log2(page_size)), is
// below 2^32 and exact for slots below 2^31.
struct PageOf {
    uint32_t m, shift;
    explicit PageOf(uint32_t page_size)
    {
        uint32_t l = 0;
        while (l < 31 && (1u << l) < page_size)
            ++l;
        shift = 31 + l;
        m = (uint32_t)(((1ull << shift) + page_size - 1) / page_size);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t slot) const
    {
        return (uint32_t)(((uint64_t)slot * m) >> shift);
    }
};

// A thread stays with its piece of a token's row and goes over tokens, so that what a piece is (head,
// dims, scale) is worked out once. Rows of more than 256 pieces take several work-groups (z).
template <class Type, bool E4M3>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvWriteArgs a, PageOf page_of, uint32_t width)
{
    typedef typename Type::T T;
    const int s = blockIdx.y;                        // keys, values
    constexpr int V = E4M3 ? 16 : 8;                 // 16 bytes written
    const uint32_t per_head = (uint32_t)a.dim / V, per_token = per_head * (uint32_t)a.heads;
    const uint32_t row = threadIdx.x / width, c = blockIdx.z * kThreads + (threadIdx.x - row * width);
    const uint32_t rows = kThreads / width;
    if (row >= rows || c >= per_token)
        return;
    const uint32_t h = c / per_head, d = (c - h * per_head) * V;
    const int64_t slots = (int64_t)a.num_pages * a.page_size;
    const T *x = (const T *)a.x[s] + h * a.hs[s] + d;
    const int64_t own = h * a.head[s] + d;
    const float scale = E4M3 && a.scale[s] ? a.scale[s][h] : 1.0f, r = 1.0f / scale;
    const bool near = scale > 0x1p-60f && scale < 0x1p60f;
    for (int64_t t = (int64_t)blockIdx.x * rows + row; t < a.T; t += (int64_t)gridDim.x * rows) {
        const int32_t slot = a.slot_map[t];
        if (slot < 0 || slot >= slots)
            continue;
        const T *from = x + t * a.ld[s];
        union { u32x4 u[V / 8]; T v[V]; } in;
#pragma unroll
        for (int i = 0; i < V / 8; ++i)
            in.u[i] = *(const u32x4 *)(from + 8 * i);
        const uint32_t page = page_of((uint32_t)slot);
        const int64_t at = page * a.page[s] + ((uint32_t)slot - page * (uint32_t)a.page_size) * a.slot[s] + own;
        if constexpr (!E4M3) {
            *(u32x4 *)((T *)a.cache[s] + at) = in.u[0];
        } else {
            float f[V];
            if (near) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float v = Type::f(in.v[e]), q0 = v * r, q = fmaf(-fmaf(q0, scale, -v), r, q0);
                    f[e] = clamp448(fabsf(q0) < 1e30f ? q : q0);   // infinities and NaN as they are
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    f[e] = clamp448(Type::f(in.v[e]) / scale);
            }
            u32x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = pack_e4m3(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
            *(u32x4 *)((uint8_t *)a.cache[s] + at) = o;
        }
    }
}

}  // namespace

hipError_t launch_kv_write(const KvWriteArgs &a, int cus, hipStream_t stream)
{
    const int64_t per_token = (int64_t)a.heads * (a.dim / (a.e4m3 ? 16 : 8));
    const uint32_t width = per_token < kThreads ? (uint32_t)per_token : kThreads, rows = kThreads / width;
    const int64_t slices = (per_token + kThreads - 1) / kThreads;   // below 2^16: 65535 heads of 1024
    int64_t blocks = ((int64_t)a.T + rows - 1) / rows;
    const int64_t most = (int64_t)cus * 8 / slices;
    if (blocks > (most < 1 ? 1 : most))
        blocks = most < 1 ? 1 : most;
    const dim3 grid((unsigned)blocks, 2, (unsigned)slices), block(kThreads);
    const PageOf page_of((uint32_t)a.page_size);
    if (a.e4m3)
        a.fp16 ? kv_write_kernel<Fp16, true><<<grid, block, 0, stream>>>(a, page_of, width)
               : kv_write_kernel<Bf16, true><<<grid, block, 0, stream>>>(a, page_of, width);
    else   // 16-bit values as they are
        kv_write_kernel<Bf16, false><<<grid, block, 0, stream>>>(a, page_of, width);
    return hipGetLastError();
}

}  // namespace w4a16
