// What the chunked token mixers share: matrix products of 16-bit values, values split into terms, rows of a
// chunk of tokens as buffers, and running sums over its decays.
#pragma once

#include "mixer_types.h"

namespace w4a16 {

namespace {

constexpr int kChunk = 64;
constexpr float kNone = -193.0f;   // a log decay below counts as this: e^-193 is zero

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma(Bf16, u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(Fp16, u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t pack2(Bf16, float a, float b)
{
    const bf16x2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t pack2(Fp16, float a, float b)
{
    const f16x2 r = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float low(Bf16, uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float high(Bf16, uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
__device__ __forceinline__ float low(Fp16, uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[0]; }
__device__ __forceinline__ float high(Fp16, uint32_t w) { return (float)__builtin_bit_cast(f16x2, w)[1]; }

// Rounds a pair and keeps what that leaves in its place, for the next term. The remainder goes by the bits
// that the product gets: left to itself, the compiler rounds v * d once for one use and twice (float32
// first) for the other.
template <class Type>
__device__ __forceinline__ uint32_t take(Type t, float &a, float &b)
{
    uint32_t both = pack2(t, a, b);
    asm volatile("" : "+v"(both));
    a -= low(t, both);
    b -= high(t, both);
    return both;
}
// The sign's place is set for a value that is not finite (its exponent field, plus one unit of it).
__device__ __forceinline__ uint32_t odd_bits(Bf16, uint32_t w) { return (w & 0x7FFF7FFFu) + 0x00800080u; }
__device__ __forceinline__ uint32_t odd_bits(Fp16, uint32_t w) { return (w & 0x7FFF7FFFu) + 0x04000400u; }
// Keeps a branch that is hardly ever taken a branch, rather than selects on the way past it.
__device__ __forceinline__ void rare() { asm volatile("; rare"); }

// Rows of a chunk as a buffer: `n` of them, `ld` elements apart and `width` long. What lies past the last
// row's end reads as zeros and isn't written, so that a chunk's loads need no branches: where one comes
// between a load and its use, the compiler waits for every load in flight.
typedef __amdgpu_buffer_rsrc_t Rows;
__device__ __forceinline__ Rows rows_of(const void *p, int32_t n, int32_t ld, int width, int bytes)
{
    const uint32_t count = min(max(n, 0), kChunk);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0,
                                             count ? ((count - 1) * (uint32_t)ld + width) * bytes : 0, 0x00027000);
}
__device__ __forceinline__ u32x4 load4(Rows r, uint32_t at)
{
    return __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0);
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, true);
    return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Running sum over the 64 lanes: shifts by 1, 2, 4, 8 inside rows of 16, then the rows' ends.
__device__ __forceinline__ double running_sum(double x)
{
    x = dpp_add<0x111, 0xF>(x);
    x = dpp_add<0x112, 0xF>(x);
    x = dpp_add<0x114, 0xF>(x);
    x = dpp_add<0x118, 0xF>(x);
    x = dpp_add<0x142, 0xA>(x);
    return dpp_add<0x143, 0xC>(x);
}

}  // namespace

}  // namespace w4a16
