// Device-side types of the token mixers: bf16 / fp16 / e4m3 values to and from float.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a16 {

struct Bf16 {
    typedef __bf16 T;
    static __device__ __forceinline__ float f(T x) { return (float)x; }
    static __device__ __forceinline__ T from(float x) { return (T)x; }   // nearest even
};

struct Fp16 {
    typedef _Float16 T;
    static __device__ __forceinline__ float f(T x) { return (float)x; }
    static __device__ __forceinline__ T from(float x) { return (T)x; }
};

// Clamp that keeps NaN.
__device__ __forceinline__ float clamp448(float x)
{
    return x > 448.0f ? 448.0f : x < -448.0f ? -448.0f : x;
}

// Four floats within +-448 (or NaN) to four e4m3 codes, nearest even.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

}  // namespace w4a16
