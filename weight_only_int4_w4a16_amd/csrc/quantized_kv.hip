// A key-value cache of 8-bit codes with a scale for each block of tokens and head, for gfx950: rows are
// quantised as they are written, and read back.
//   write: s' = max(amax / Q, 2^-126, s), code = x / s' to the nearest code; where a block's scale grows, what it
//   held becomes code * s / s'.     read: code * s, rounded once.
// Both are bound by memory: 2 bytes read and 1 written per value, or 1 and 2.
// Measured with 8 heads of 128: 12257 tokens of 40 requests written as e4m3 27 us (2.8 TB/s: a wave's slots, rows,
// maximum and stores come one after the other, and counters show the vector units busy for 48 % of it), 15 tokens 4.6 us;
// 60000 tokens read 84 us (4.4 TB/s, where a copy of 4 GiB reaches 4.7), 500 of 4 heads 3 us.
//
// Roundings go by the exact quotients and products. Scales come from the values, so quotients on a border
// between two codes are common (one in a thousand, where 8-bit significands divide), and a float32 quotient
// falls on the border from both sides. Of the two float32 values around the exact one the odd one is taken: it rounds
// to fewer bits as the exact one does. Which it is shows the sign of what is missing, from one fused operation.
#include "mixers.h"
#include "mixer_types.h"

namespace w4a16 {

namespace {

constexpr int kRowThreads = 256, kRowWaves = kRowThreads / 64;
constexpr int kWide = 22;   // blocks along x, of which a launch holds fewer than 2^32 threads
constexpr float kLeast = 0x1p-126f;

// x >= 0, next to a value that is larger by `rest` (or smaller): the odd one of the float32 values around that one.
__device__ __forceinline__ float made_odd(float x, float rest)
{
    const uint32_t below = __builtin_bit_cast(uint32_t, x) + (uint32_t)(__builtin_bit_cast(int32_t, rest) >> 31);
    return __builtin_bit_cast(float, below | (rest != 0.0f ? 1u : 0u));
}

template <bool INT8>
__device__ __forceinline__ float largest()
{
    return INT8 ? 127.0f : 448.0f;
}

// x / s for the rounding to a code: r is about 1 / s, both at least 2^-62 and |x| no larger than 2^9 s. (Two
// steps take the quotient to one of its neighbours.)
template <bool INT8>
__device__ __forceinline__ float quotient(float x, float s, float r)
{
    const float q0 = fabsf(x) * r, q = fmaf(fmaf(-q0, s, fabsf(x)), r, q0);
    return copysignf(fminf(made_odd(q, fmaf(-q, s, fabsf(x))), largest<INT8>()), x);
}

// Four quotients, no larger than the largest code, to codes.
template <bool INT8>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d)
{
    if constexpr (!INT8) {
        return pack_e4m3(a, b, c, d);
    } else {   // as bytes 1 to 255, and back
        uint32_t w = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_rintf(a) + 128.0f, 0, 0);
        w = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_rintf(b) + 128.0f, 1, w);
        w = __builtin_amdgcn_cvt_pk_u8_f32(__builtin_rintf(c) + 128.0f, 2, w);
        return __builtin_amdgcn_cvt_pk_u8_f32(__builtin_rintf(d) + 128.0f, 3, w) ^ 0x80808080u;
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

// The largest of all lanes: rotated inside rows of 16, then rows swapped.
template <int ROTATE>
__device__ __forceinline__ uint32_t rotated_max(uint32_t x)
{
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + ROTATE, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    x = rotated_max<1>(rotated_max<2>(rotated_max<4>(rotated_max<8>(x))));
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = max(r[0], r[1]);
    const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return max(s[0], s[1]);
}

// A wave quantises the runs that start among `range` tokens, of one head (the heads of a token lie next to each other)
// and keys or values (y). Magnitudes are compared as the integers that their bits are, infinities and NaN above all
// others.
constexpr int kPieces = 8;   // 16-byte pieces of a run's rows that a lane holds at a time

template <class Type, bool INT8>
__global__ __launch_bounds__(kRowThreads) void quantized_write_kernel(QuantizedRowsArgs a, int range)
{
    typedef typename Type::T T;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int s = blockIdx.y;
    const uint32_t unit = (blockIdx.z << kWide | blockIdx.x) * kRowWaves + wave, part = unit / (uint32_t)a.c.heads;
    const int h = (int)(unit - part * (uint32_t)a.c.heads);
    const int64_t t0 = (int64_t)part * range;
    if (t0 >= a.T)
        return;
    const int32_t block = a.c.block, dim = a.c.dim, per_row = dim / 8;   // 8 to 32
    const uint32_t of_row = (65536 + per_row - 1) / per_row;             // p / per_row = p of_row >> 16 below 2048
    const int64_t slots = (int64_t)a.c.num_pages * a.c.page_size;
    auto slot_of = [&](int64_t t) {
        const int32_t x = t >= 0 && t < a.T ? a.slot_map[t] : -1;
        return x < slots ? x : -1;
    };
    auto follows = [&](int32_t x, int32_t before) { return before >= 0 && x == before + 1 && x % block != 0; };
    const int32_t own = slot_of(t0 + lane), behind = slot_of(t0 + 64 + lane), before = slot_of(t0 + lane - 1);
    uint64_t starts = __ballot(lane < range && own >= 0 && !follows(own, before));
    while (starts) {
        const int i = __builtin_ctzll(starts);
        starts &= starts - 1;
        const int64_t t = t0 + i;
        const int32_t slot = __builtin_amdgcn_readlane(own, i);
        const int32_t page = slot / a.c.page_size, in_page = slot - page * a.c.page_size;
        const int32_t b = in_page / block, off = in_page - b * block;
        const int32_t x0 = __shfl(own, lane + i & 63), x1 = __shfl(behind, lane + i & 63);
        const uint64_t run = __ballot((uint32_t)(lane + i < 64 ? x0 : x1) == (uint32_t)slot + lane);
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
                const uint32_t p = p0 + 64 * j + lane, row = p * of_row >> 16;
                in[j] = u32x4{0, 0, 0, 0};
                if (p < (uint32_t)pieces)
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
        most = wave_max(max(most & 0xFFFFu, most >> 16));
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
        auto quantise = [&](int32_t p0, float factor) {
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const uint32_t p = p0 + 64 * j + lane, row = p * of_row >> 16;
                if (p >= (uint32_t)pieces)
                    continue;
                union { u32x4 u; T v[8]; } y;
                y.u = in[j];
                float q[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    q[e] = quotient<INT8>(Type::f(y.v[e]) * factor, up, r);
                u32x2 o = {codes4<INT8>(q[0], q[1], q[2], q[3]), codes4<INT8>(q[4], q[5], q[6], q[7])};
                if (none)
                    o = u32x2{0, 0};
                *(u32x2 *)(codes + (off + row) * a.c.slot[s] + (p - row * per_row) * 8) = o;
            }
        };
        for (int32_t p0 = 0; p0 < pieces; p0 += 64 * kPieces) {
            if (pieces > 64 * kPieces)
                load(p0);
            if (lift == 1.0f)
                quantise(p0, 1.0f);   // no multiplication
            else
                quantise(p0, lift);
        }
        // What the block held goes over to the new scale, in float64 (rare: a block's scale has grown).
        if (off && scale > old) {
            const double from = old, to = scale;
            auto again = [&](float code) {
                const double x = fabs((double)code * from / to);
                const float q = (float)x;
                return copysignf(fminf(made_odd(q, (float)(x - (double)q)), largest<INT8>()), code);
            };
            for (int32_t p = lane; p < block * per_row; p += 64) {
                const int32_t row = p * of_row >> 16;
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

// A thread stays with its piece of 8 values of a token's row and goes over tokens. Rows of more than 256 pieces take
// several work-groups (z).
template <class Type, bool INT8>
__global__ __launch_bounds__(kRowThreads) void quantized_read_kernel(QuantizedRowsArgs a, uint32_t width)
{
    typedef typename Type::T T;
    const int s = blockIdx.y;
    const uint32_t per_head = (uint32_t)a.c.dim / 8, per_token = per_head * (uint32_t)a.c.heads;
    const uint32_t row = threadIdx.x / width, c = blockIdx.z * kRowThreads + (threadIdx.x - row * width);
    const uint32_t rows = kRowThreads / width;
    if (row >= rows || c >= per_token)
        return;
    const uint32_t h = c / per_head, d = (c - h * per_head) * 8;
    const int64_t slots = (int64_t)a.c.num_pages * a.c.page_size;
    const uint8_t *codes = a.c.codes[s] + h * a.c.head[s] + d;
    const float *scales = a.c.scale[s] + h * a.c.scale_head[s];
    T *out = (T *)a.x[s] + h * a.hs[s] + d;
    for (int64_t t = (int64_t)blockIdx.x * rows + row; t < a.T; t += (int64_t)gridDim.x * rows) {
        const int32_t slot = a.slot_map[t];
        union { u32x4 u; T v[8]; } o;
        o.u = u32x4{0, 0, 0, 0};
        if (slot >= 0 && slot < slots) {
            const int32_t page = slot / a.c.page_size, in_page = slot - page * a.c.page_size;
            const u32x2 w = *(const u32x2 *)(codes + page * a.c.page[s] + in_page * a.c.slot[s]);
            const float scale = scales[page * a.c.scale_page[s] + in_page / a.c.block * a.c.scale_block[s]];
            auto value = [&](float code) {
                const float p = fabsf(code * scale);
                return Type::from(copysignf(made_odd(p, fmaf(fabsf(code), scale, -p)), code));
            };
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                o.v[4 * e] = value(value_of<INT8, 0>(w[e]));
                o.v[4 * e + 1] = value(value_of<INT8, 1>(w[e]));
                o.v[4 * e + 2] = value(value_of<INT8, 2>(w[e]));
                o.v[4 * e + 3] = value(value_of<INT8, 3>(w[e]));
            }
        }
        *(u32x4 *)(out + t * a.ld[s]) = o.u;
    }
}

}  // namespace

hipError_t launch_quantized_write(const QuantizedRowsArgs &a, hipStream_t stream)
{
    // As many tokens to a wave as leave 8192 waves in the launch, 8 for each SIMD (their registers let 5 of them reside
    // with int8, 4 with e4m3), 16 at most: prompts of 12257 tokens with 4, 8, 16 and 32 to a wave 40.7, 35.2, 30.2 and 30.3
    // us (the least of 6, before later steps; why 16 and 32 are alike was not found out), while single tokens of many
    // requests, each a run, want waves of their own.
    int64_t range = (int64_t)a.T * 2 * a.c.heads / 8192;
    range = range < 1 ? 1 : range > 16 ? 16 : range;
    const int64_t waves = (a.T + range - 1) / range * a.c.heads;   // below 2^32: T heads <= 2^35
    const int64_t blocks = (waves + kRowWaves - 1) / kRowWaves, wide = 1 << kWide;
    const dim3 grid((unsigned)(blocks < wide ? blocks : wide), 2, (unsigned)((blocks + wide - 1) / wide)), block(kRowThreads);
    const int n = (int)range;
    if (a.c.int8)
        a.fp16 ? quantized_write_kernel<Fp16, true><<<grid, block, 0, stream>>>(a, n)
               : quantized_write_kernel<Bf16, true><<<grid, block, 0, stream>>>(a, n);
    else
        a.fp16 ? quantized_write_kernel<Fp16, false><<<grid, block, 0, stream>>>(a, n)
               : quantized_write_kernel<Bf16, false><<<grid, block, 0, stream>>>(a, n);
    return hipGetLastError();
}

hipError_t launch_quantized_read(const QuantizedRowsArgs &a, int cus, hipStream_t stream)
{
    const int64_t per_token = (int64_t)a.c.heads * (a.c.dim / 8);
    const uint32_t width = per_token < kRowThreads ? (uint32_t)per_token : kRowThreads, rows = kRowThreads / width;
    const int64_t slices = (per_token + kRowThreads - 1) / kRowThreads;   // at most 8192: 65535 heads of 256
    int64_t blocks = ((int64_t)a.T + rows - 1) / rows;
    const int64_t most = (int64_t)cus * 8 / slices;
    if (blocks > (most < 1 ? 1 : most))
        blocks = most < 1 ? 1 : most;
    const dim3 grid((unsigned)blocks, 2, (unsigned)slices), block(kRowThreads);
    if (a.c.int8)
        a.fp16 ? quantized_read_kernel<Fp16, true><<<grid, block, 0, stream>>>(a, width)
               : quantized_read_kernel<Bf16, true><<<grid, block, 0, stream>>>(a, width);
    else
        a.fp16 ? quantized_read_kernel<Fp16, false><<<grid, block, 0, stream>>>(a, width)
               : quantized_read_kernel<Bf16, false><<<grid, block, 0, stream>>>(a, width);
    return hipGetLastError();
}

}  // namespace w4a16
