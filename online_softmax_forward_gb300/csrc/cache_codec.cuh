// cache_codec.cuh -- the two 8-bit formats of the cache on the device.
//
// A code is an e4m3 number (4-bit exponent, 3-bit mantissa, largest 448) or
// an int8 in -127 .. 127; its value is code * scale.  A scale is a power of
// two (the smallest with amax / scale <= the largest code), so x / scale is
// exact in fp32, rounding happens once (to nearest, ties to even), and a
// larger scale only shifts the codes already held.  A floating code loses
// nothing by it; an int8 code at most one bit against amax / 127.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "attn.h"

namespace attn {

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

namespace codec {

// smallest power of two s >= 2^-126 with amax <= top * s; 0 for amax = 0,
// NaN when amax is not finite.  amax >= 0 or NaN.
template <int FMT>
__device__ __forceinline__ float scale_for(float amax) {
    if (!(amax <= 3.402823466e38f)) return __int_as_float(0x7fc00000);
    if (amax == 0.f) return 0.f;
    // top = m * 2^8 (448 = 1.75 * 2^8) or m * 2^6 (127 = 1.984375 * 2^6)
    constexpr int kExp = FMT == ATTN_CACHE_E4M3 ? 8 : 6;
    constexpr uint32_t kMant = FMT == ATTN_CACHE_E4M3 ? 0x600000u : 0x7e0000u;
    const uint32_t u = __float_as_uint(amax);
    // a subnormal amax has exponent field 0 and lands on the 2^-126 floor
    const int e = (int)(u >> 23) - 127 - kExp + ((u & 0x7fffffu) > kMant ? 1 : 0);
    return __uint_as_float((uint32_t)((e < -126 ? -126 : e) + 127) << 23);
}

// 1 / s (exact for a power of two); 0 for s = 0 or NaN, whose codes are all 0.
__device__ __forceinline__ float inverse_scale(float s) { return s > 0.f ? 1.f / s : 0.f; }

// four values, already divided by the scale, to four packed codes
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (FMT == ATTN_CACHE_E4M3) {
        uint16_t lo, hi;  // the second operand goes to the low byte
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return (uint32_t)lo | ((uint32_t)hi << 16);
    } else {
        const uint32_t x = (uint32_t)__float2int_rn(a) & 0xff, y = (uint32_t)__float2int_rn(b) & 0xff;
        const uint32_t z = (uint32_t)__float2int_rn(c) & 0xff, w = (uint32_t)__float2int_rn(d) & 0xff;
        return x | (y << 8) | (z << 16) | (w << 24);
    }
}

// the numbers of four packed codes
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float *f) {
    if constexpr (FMT == ATTN_CACHE_E4M3) {
        uint32_t a, b;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)(w & 0xffff)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(w >> 16)));
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
        f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = (float)(int)(int8_t)(w >> (8 * i));
    }
}

// Eight consecutive values of a type (DT: 0 fp32, 1 bf16, 2 fp16) as they lie in memory.
template <int DT>
struct Raw8 {
    uint4 u[DT == 0 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p, size_t i) {
        if constexpr (DT == 0) {
            const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<const float *>(p) + i);
            u[0] = q[0];
            u[1] = q[1];
        } else {
            u[0] = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(p) + i);
        }
    }
    __device__ __forceinline__ void widen(float *f) const {
        const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (DT == 0) {
                f[j] = __uint_as_float(w[j]);
            } else if constexpr (DT == 1) {
                f[2 * j] = __uint_as_float(w[j] << 16);
                f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            } else {
                const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
                f[2 * j] = x.x;
                f[2 * j + 1] = x.y;
            }
        }
        if constexpr (DT == 0) {
            f[4] = __uint_as_float(u[1].x); f[5] = __uint_as_float(u[1].y);
            f[6] = __uint_as_float(u[1].z); f[7] = __uint_as_float(u[1].w);
        }
    }
};
template <int DT>
__device__ __forceinline__ void load8(const void *p, size_t i, float *f) {
    Raw8<DT> r;
    r.load(p, i);
    r.widen(f);
}

// Smallest and largest of eight channels over the rows that add() is given; a NaN
// stays.  Pairs of 16-bit values are compared as pairs.
template <int DT>
struct Range8 {
    using P = typename std::conditional<DT == 1, __nv_bfloat162, __half2>::type;
    uint32_t lo[DT == 0 ? 8 : 4], hi[DT == 0 ? 8 : 4];
    __device__ __forceinline__ static uint32_t least(uint32_t a, uint32_t b) {
        if constexpr (DT == 0) {
            float r;
            asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
            return __float_as_uint(r);
        } else {
            const P r = __hmin2_nan(*reinterpret_cast<const P *>(&a), *reinterpret_cast<const P *>(&b));
            return *reinterpret_cast<const uint32_t *>(&r);
        }
    }
    __device__ __forceinline__ static uint32_t most(uint32_t a, uint32_t b) {
        if constexpr (DT == 0) {
            float r;
            asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
            return __float_as_uint(r);
        } else {
            const P r = __hmax2_nan(*reinterpret_cast<const P *>(&a), *reinterpret_cast<const P *>(&b));
            return *reinterpret_cast<const uint32_t *>(&r);
        }
    }
    static constexpr uint32_t kUp = DT == 0 ? 0x7f800000u : DT == 1 ? 0x7f807f80u : 0x7c007c00u;
    static constexpr uint32_t kSign = DT == 0 ? 0x80000000u : 0x80008000u;
    static constexpr int kN = DT == 0 ? 8 : 4;
    __device__ __forceinline__ void clear() {  // +infinity, -infinity
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            lo[j] = kUp;
            hi[j] = kUp | kSign;
        }
    }
    // The largest magnitude of w as the bits of a float; a NaN's exceed infinity's.
    __device__ __forceinline__ static uint32_t largest(const uint32_t (&w)[kN]) {
        uint32_t m = w[0] & ~kSign;
#pragma unroll
        for (int j = 1; j < kN; ++j) m = most(m, w[j] & ~kSign);
        if constexpr (DT == 0) return m;
        float f[8];
        const uint32_t pair[4] = {m, 0, 0, 0};
        widen(pair, f);
        return max(__float_as_uint(f[0]), __float_as_uint(f[1]));
    }
    __device__ __forceinline__ uint32_t largest() const {  // 0 if no row was added
        if (lo[0] == kUp && hi[0] == (kUp | kSign)) return 0;
        uint32_t m[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) m[j] = most(lo[j] & ~kSign, hi[j] & ~kSign);
        return largest(m);
    }
    __device__ __forceinline__ void add(const Raw8<DT> &r) {
        const uint32_t w[8] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w, r.u[DT == 0].x, r.u[DT == 0].y,
                               r.u[DT == 0].z, r.u[DT == 0].w};
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            lo[j] = least(lo[j], w[j]);
            hi[j] = most(hi[j], w[j]);
        }
    }
    // |values| into `m`, which starts at 0
    __device__ __forceinline__ static void add_magnitudes(uint32_t (&m)[kN], const Raw8<DT> &r) {
        const uint32_t w[8] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w, r.u[DT == 0].x, r.u[DT == 0].y,
                               r.u[DT == 0].z, r.u[DT == 0].w};
#pragma unroll
        for (int j = 0; j < kN; ++j) m[j] = most(m[j], w[j] & ~kSign);
    }
    // also over the lanes whose number differs in bit `o`
    __device__ __forceinline__ void join(int o) {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            lo[j] = least(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], o));
            hi[j] = most(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], o));
        }
    }
    __device__ __forceinline__ static void widen(const uint32_t *w, float *f) {
        Raw8<DT> r;
        r.u[0] = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (DT == 0) r.u[1] = make_uint4(w[4], w[5], w[6], w[7]);
        r.widen(f);
    }
};

// x within +-far, NaN kept: a value beyond the output type's range becomes
// its largest finite one (the nearest code to 65504 may stand for 65536)
__device__ __forceinline__ float clamped(float x, float far) {
    return x != x ? x : fminf(fmaxf(x, -far), far);
}

// two fp32 values to a packed pair, clamped, rounded to nearest
template <int DT>
__device__ __forceinline__ uint32_t pack2_clamped(float a, float b) {
    constexpr float far = DT == 1 ? 3.3895314e38f : 65504.f;
    a = clamped(a, far);
    b = clamped(b, far);
    if constexpr (DT == 1) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

}  // namespace codec
}  // namespace attn
