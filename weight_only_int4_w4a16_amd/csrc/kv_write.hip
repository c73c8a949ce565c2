// Writes into the paged key-value cache for gfx950: a token's rows go to its slot, as they are or
// divided by the head's scale and rounded to e4m3. Memory-bound: 2 bytes read and 2 or 1 written per
// value. A thread moves 16 values (two 16-byte loads), so a wave covers 2 KB of one or more tokens
// and an e4m3 store is 16 bytes wide as well.
#include "mixers.h"
#include "mixer_types.h"

namespace w4a16 {

namespace {

constexpr int kThreads = 256;

template <class Type, bool E4M3>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvWriteArgs a)
{
    typedef typename Type::T T;
    const int s = blockIdx.y;                        // keys, values
    const uint32_t per_head = (uint32_t)a.dim / 16, per_token = per_head * (uint32_t)a.heads;
    const int64_t n = (int64_t)a.T * per_token;
    const int64_t slots = (int64_t)a.num_pages * a.page_size;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = i / per_token;
        const uint32_t c = (uint32_t)(i - t * per_token), h = c / per_head, d = (c - h * per_head) * 16;
        const int32_t slot = a.slot_map[t];
        if (slot < 0 || slot >= slots)
            continue;
        const T *x = (const T *)a.x[s] + t * a.ld[s] + h * a.hs[s] + d;
        const u32x4 lo = *(const u32x4 *)x, hi = *(const u32x4 *)(x + 8);
        const uint32_t p = (uint32_t)slot / (uint32_t)a.page_size;
        const int64_t at = p * a.page[s] + ((uint32_t)slot - p * (uint32_t)a.page_size) * a.slot[s] +
                           h * a.head[s] + d;
        if (!E4M3) {
            T *y = (T *)a.cache[s] + at;
            *(u32x4 *)y = lo;
            *(u32x4 *)(y + 8) = hi;
        } else {
            const float scale = a.scale[s] ? a.scale[s][h] : 1.0f;
            union { u32x4 u[2]; T v[16]; } in{{lo, hi}};
            float f[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
                f[e] = clamp448(Type::f(in.v[e]) / scale);
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
    const int64_t n = (int64_t)a.T * a.heads * (a.dim / 16);
    int64_t blocks = (n + kThreads - 1) / kThreads;
    if (blocks > (int64_t)cus * 16)
        blocks = (int64_t)cus * 16;
    const dim3 grid((unsigned)blocks, 2), block(kThreads);
    if (a.e4m3)
        a.fp16 ? kv_write_kernel<Fp16, true><<<grid, block, 0, stream>>>(a)
               : kv_write_kernel<Bf16, true><<<grid, block, 0, stream>>>(a);
    else
        kv_write_kernel<Bf16, false><<<grid, block, 0, stream>>>(a);   // 16-bit values as they are
    return hipGetLastError();
}

}  // namespace w4a16
