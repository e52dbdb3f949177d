// cache_mma.cuh -- products with 8-bit codes on mma.m16n8k16: what the attention
// over the cache and its page selection share.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn.h"
#include "cache_codec.cuh"

namespace attn {

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Codes as fp16 pairs, exact.  e4m3: one conversion a pair, as cheap as any
// integer instruction (2 clocks a warp and SM quarter; moving the bits into place
// by hand takes four).  int8: 0x6400 + u is the fp16 1024 + u, u = code + 128.
template <int FMT>
struct Unpack;
template <>
struct Unpack<ATTN_CACHE_E4M3> {
    // bytes (0, 1) and (2, 3) of w
    __device__ __forceinline__ static void quad(uint32_t w, uint32_t &lo, uint32_t &hi) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
    }
};
template <>
struct Unpack<ATTN_CACHE_I8> {
    __device__ __forceinline__ static uint32_t less1152(uint32_t w) {  // 1024 + u -> u - 128
        const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&w),
                                  __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ __forceinline__ static void quad(uint32_t w, uint32_t &lo, uint32_t &hi) {
        const uint32_t u = w ^ 0x80808080u;
        lo = less1152(__byte_perm(u, 0x64646464u, 0x4140));
        hi = less1152(__byte_perm(u, 0x64646464u, 0x4342));
    }
};

// The power of two that puts a row's largest magnitude in [2^14, 2^15), so that
// any fp32 or bf16 exponent fits fp16, and its inverse; 1 for 0 and infinity.
__device__ __forceinline__ void row_power(float amax, float &mul, float &back) {
    int up = 14 - ((int)(__float_as_uint(amax) >> 23) - 127);
    up = up > 126 ? 126 : up;
    if (amax == 0.f || !(amax <= 3.402823466e38f)) up = 0;
    mul = __uint_as_float((uint32_t)(127 + up) << 23);
    back = __uint_as_float((uint32_t)(127 - up) << 23);
}

}  // namespace attn
