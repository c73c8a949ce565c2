// A key-value cache of 8-bit codes with a scale for each block of tokens and head, for gfx950: rows are
// quantised as they are written, and read back.
//   write: s' = max(amax / Q, 2^-126, s), code = x / s' to the nearest code; where a block's scale grows, what it
//   held becomes code * s / s'.     read: code * s, rounded once.
// Both are bound by memory: 2 bytes read and 1 written per value, or 1 and 2.
//
// Roundings go by the exact quotients and products. Scales come from the values, so quotients on a border
// between two codes are common (one in a thousand, where 8-bit significands divide), and a float32 quotient
// falls on the border from both sides. A float32 result next to the exact one, with the sign of what it is off by (one
// fused operation, exact), is made odd where it is not exact: it then rounds to fewer bits as the exact one.
#include "mixers.h"
#include "mixer_types.h"

namespace w4a16 {

namespace {

constexpr int kRowThreads = 256;
constexpr float kLeast = 0x1p-126f;

// x, one of the two float32 values around a real one (or it), with the sign of what is missing: the odd one.
__device__ __forceinline__ float made_odd(float x, float rest)
{
    const uint32_t u = __builtin_bit_cast(uint32_t, x);
    const uint32_t off = ((__builtin_bit_cast(uint32_t, rest) ^ u) >> 31) ? ~0u : 1u;   // towards zero or away
    return __builtin_bit_cast(float, rest != 0.0f && !(u & 1) ? u + off : u);
}

// x / s for the rounding to a code: r is about 1 / s, both at least 2^-60 and x no larger than 2^9 s. (Two
// steps take the quotient to one of its neighbours.)
__device__ __forceinline__ float quotient(float x, float s, float r)
{
    const float q0 = x * r, q = fmaf(-fmaf(q0, s, -x), r, q0);
    return made_odd(q, -fmaf(q, s, -x));
}

template <bool INT8>
__device__ __forceinline__ float largest()
{
    return INT8 ? 127.0f : 448.0f;
}

// Four quotients to codes.
template <bool INT8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d)
{
    if constexpr (!INT8) {
        return pack_e4m3(clamp448(a), clamp448(b), clamp448(c), clamp448(d));
    } else {
        auto code = [](float x) {
            return (uint32_t)(int32_t)__builtin_rintf(fminf(fmaxf(x, -127.0f), 127.0f)) & 0xFFu;
        };
        return code(a) | code(b) << 8 | code(c) << 16 | code(d) << 24;
    }
}

template <bool INT8, int I>
__device__ __forceinline__ float value_of(uint32_t w)
{
    if constexpr (INT8)
        return (float)(int8_t)(w >> (8 * I));
    else
        return __builtin_amdgcn_cvt_f32_fp8((int)w, I);
}

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t larger_pair(uint32_t x, uint32_t y)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, x),
                                                                  __builtin_bit_cast(u16x2, y)));
}

// A wave quantises the runs that start among `range` tokens, for one head and keys or values. Magnitudes are
// compared as the integers that their bits are, infinities and NaN above all others.
constexpr int kPieces = 8;   // 16-byte pieces of a run's rows that a lane holds at a time

template <class Type, bool INT8>
__global__ __launch_bounds__(kRowThreads) void quantized_write_kernel(QuantizedRowsArgs a, int range)
{
    typedef typename Type::T T;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t block = a.c.block, dim = a.c.dim, per_row = dim / 8;
    const int kinds = 2 * a.c.heads;
    const int64_t slots = (int64_t)a.c.num_pages * a.c.page_size;
    auto slot_of = [&](int64_t t) {
        const int32_t x = t >= 0 && t < a.T ? a.slot_map[t] : -1;
        return x < slots ? x : -1;
    };
    auto follows = [&](int32_t x, int32_t before) { return before >= 0 && x == before + 1 && x % block != 0; };
    for (int64_t unit = (int64_t)blockIdx.x * (kRowThreads / 64) + wave;; unit += (int64_t)gridDim.x * (kRowThreads / 64)) {
    const int64_t t0 = unit / kinds * range;
    const int kind = (int)(unit % kinds), s = kind & 1, h = kind >> 1;
    if (t0 >= a.T)
        return;
    const int32_t own = lane < range ? slot_of(t0 + lane) : -1, before = slot_of(t0 + lane - 1);
    uint64_t starts = __ballot(own >= 0 && !follows(own, before));
    while (starts) {
        const int i = __builtin_ctzll(starts);
        starts &= starts - 1;
        const int64_t t = t0 + i;
        const int32_t slot = __builtin_amdgcn_readlane(own, i);
        const int32_t page = slot / a.c.page_size, in_page = slot - page * a.c.page_size;
        const int32_t b = in_page / block, off = in_page - b * block;
        const uint64_t run = __ballot((uint32_t)slot_of(t + lane) == (uint32_t)slot + lane);
        const int32_t rows = min(~run ? __builtin_ctzll(~run) : 64, block - off);
        const int32_t pieces = rows * per_row;
        const T *x = (const T *)a.x[s] + h * a.hs[s] + t * a.ld[s];
        uint8_t *codes = a.c.codes[s] + page * a.c.page[s] + h * a.c.head[s] + (int64_t)b * block * a.c.slot[s];
        float *scale_at = a.c.scale[s] + page * a.c.scale_page[s] + b * a.c.scale_block[s] + h * a.c.scale_head[s];
        const float old = off ? *scale_at : 0.0f;
        u32x4 in[kPieces];
        auto load = [&](int32_t p0) {
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const int32_t p = p0 + 64 * j + lane, row = p / per_row;
                in[j] = u32x4{0, 0, 0, 0};
                if (p < pieces)
                    in[j] = *(const u32x4 *)(x + row * a.ld[s] + (p - row * per_row) * 8);
            }
        };
        uint32_t most = 0;
        for (int32_t p0 = 0; p0 < pieces; p0 += 64 * kPieces) {
            load(p0);
#pragma unroll
            for (int j = 0; j < kPieces; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    most = larger_pair(most, in[j][e] & 0x7FFF7FFFu);
        }
        most = max(most & 0xFFFFu, most >> 16);
        for (int d = 1; d < 64; d <<= 1)
            most = max(most, (uint32_t)__shfl_xor((int)most, d));
        const float amax = Type::f(__builtin_bit_cast(T, (uint16_t)most));
        float scale = fmaxf(amax / largest<INT8>(), kLeast);
        if (off)
            scale = old <= scale ? scale : old;   // NaN stays
        if (!(amax < INFINITY))
            scale = NAN;
        if (lane == 0)
            *scale_at = scale;
        const bool none = scale != scale;
        const float lift = scale < 0x1p-60f ? 0x1p64f : 1.0f, up = scale * lift, r = 1.0f / up;
        for (int32_t p0 = 0; p0 < pieces; p0 += 64 * kPieces) {
            if (pieces > 64 * kPieces)
                load(p0);
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const int32_t p = p0 + 64 * j + lane, row = p / per_row;
                if (p >= pieces)
                    continue;
                union { u32x4 u; T v[8]; } y;
                y.u = in[j];
                float q[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    q[e] = quotient(Type::f(y.v[e]) * lift, up, r);
                u32x2 o = {codes4<INT8>(q[0], q[1], q[2], q[3]), codes4<INT8>(q[4], q[5], q[6], q[7])};
                if (none)
                    o = u32x2{0, 0};
                *(u32x2 *)(codes + (off + row) * a.c.slot[s] + (p - row * per_row) * 8) = o;
            }
        }
        // What the block held goes over to the new scale, in float64 (rare: a block's scale has grown).
        if (off && scale > old) {
            const double from = old, to = scale;
            auto again = [&](float code) {
                const double x = (double)code * from / to;
                const float q = (float)x;
                return made_odd(q, (float)(x - (double)q));
            };
            for (int32_t p = lane; p < block * per_row; p += 64) {
                const int32_t row = p / per_row;
                if (row >= off && row < off + rows)
                    continue;
                u32x2 *at = (u32x2 *)(codes + row * a.c.slot[s] + (p - row * per_row) * 8);
                u32x2 o = *at;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    o[e] = codes4<INT8>(again(value_of<INT8, 0>(o[e])), again(value_of<INT8, 1>(o[e])),
                                        again(value_of<INT8, 2>(o[e])), again(value_of<INT8, 3>(o[e])));
                *at = o;
            }
        }
    }
    }
}

// A thread takes one piece of 16 codes of a slot's row.
template <class Type, bool INT8>
__global__ __launch_bounds__(kRowThreads) void quantized_read_kernel(QuantizedRowsArgs a)
{
    typedef typename Type::T T;
    const int s = blockIdx.y;
    const uint32_t per_row = (uint32_t)a.c.dim / 16, per_token = per_row * (uint32_t)a.c.heads;
    const int64_t slots = (int64_t)a.c.num_pages * a.c.page_size, all = (int64_t)a.T * per_token;
    for (int64_t i = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kRowThreads) {
        const int64_t t = i / per_token;
        const uint32_t c = (uint32_t)(i - t * per_token), h = c / per_row, d = (c - h * per_row) * 16;
        const int32_t slot = a.slot_map[t];
        T *to = (T *)a.x[s] + t * a.ld[s] + h * a.hs[s] + d;
        union { u32x4 u[2]; T v[16]; } out;
        out.u[0] = out.u[1] = u32x4{0, 0, 0, 0};
        if (slot >= 0 && slot < slots) {
            const int32_t page = slot / a.c.page_size, in_page = slot - page * a.c.page_size;
            const u32x4 w = *(const u32x4 *)(a.c.codes[s] + page * a.c.page[s] + in_page * a.c.slot[s] +
                                             h * a.c.head[s] + d);
            const float scale = a.c.scale[s][page * a.c.scale_page[s] + in_page / a.c.block * a.c.scale_block[s] +
                                             h * a.c.scale_head[s]];
            auto value = [&](float code) {
                const float p = code * scale;
                return Type::from(made_odd(p, fmaf(code, scale, -p)));
            };
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                out.v[4 * e] = value(value_of<INT8, 0>(w[e]));
                out.v[4 * e + 1] = value(value_of<INT8, 1>(w[e]));
                out.v[4 * e + 2] = value(value_of<INT8, 2>(w[e]));
                out.v[4 * e + 3] = value(value_of<INT8, 3>(w[e]));
            }
        }
        *(u32x4 *)to = out.u[0];
        *(u32x4 *)(to + 8) = out.u[1];
    }
}

}  // namespace

hipError_t launch_quantized_write(const QuantizedRowsArgs &a, hipStream_t stream)
{
    const int range = 1;
    const int64_t units = ((int64_t)a.T + range - 1) / range * 2 * a.c.heads;
    const int64_t blocks = (units + kRowThreads / 64 - 1) / (kRowThreads / 64);
    const dim3 grid((unsigned)(blocks < 1 << 20 ? blocks : 1 << 20)), block(kRowThreads);
    if (a.c.int8)
        a.fp16 ? quantized_write_kernel<Fp16, true><<<grid, block, 0, stream>>>(a, range)
               : quantized_write_kernel<Bf16, true><<<grid, block, 0, stream>>>(a, range);
    else
        a.fp16 ? quantized_write_kernel<Fp16, false><<<grid, block, 0, stream>>>(a, range)
               : quantized_write_kernel<Bf16, false><<<grid, block, 0, stream>>>(a, range);
    return hipGetLastError();
}

hipError_t launch_quantized_read(const QuantizedRowsArgs &a, int cus, hipStream_t stream)
{
    const int64_t all = (int64_t)a.T * a.c.heads * (a.c.dim / 16);
    int64_t blocks = (all + kRowThreads - 1) / kRowThreads;
    if (blocks > (int64_t)cus * 16)
        blocks = (int64_t)cus * 16;
    const dim3 grid((unsigned)blocks, 2), block(kRowThreads);
    if (a.c.int8)
        a.fp16 ? quantized_read_kernel<Fp16, true><<<grid, block, 0, stream>>>(a)
               : quantized_read_kernel<Bf16, true><<<grid, block, 0, stream>>>(a);
    else
        a.fp16 ? quantized_read_kernel<Fp16, false><<<grid, block, 0, stream>>>(a)
               : quantized_read_kernel<Bf16, false><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace w4a16
