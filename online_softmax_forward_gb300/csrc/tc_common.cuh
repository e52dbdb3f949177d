// tc_common.cuh -- what the tcgen05 kernels share: matrix and instruction
// descriptors, the bounded wait, and a register fence.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_internal.h"
#include "sm100_ptx.cuh"

namespace attn {

// Shared-memory matrix descriptor, 128-byte swizzle.
//   K-major operands: rows of 64 16-bit elements (128 B), 8-row groups
//   1024 B apart (SBO); the K offset inside the atom is added to the start
//   address.  MN-major operands (V for P.V): 64 contiguous N elements per
//   128-byte row, 8 K-rows per 1024-B atom (SBO), atoms along N 16 KB apart
//   (LBO).  The start address occupies the low 14 bits (address / 16), so
//   an offset inside the same shared-memory window is added to the
//   descriptor directly.
__device__ __forceinline__ uint64_t sdesc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
    d |= (uint64_t)1 << 46;  // descriptor version for the sm_100 family
    d |= (uint64_t)2 << 61;  // swizzle: 128 B
    return d;
}

// Instruction descriptor, kind::f16, fp32 accumulate.
__host__ __device__ constexpr uint32_t idesc_f16(bool bf16, int M, int N, bool b_mn_major) {
    return (1u << 4)                          // D format: f32
           | ((bf16 ? 1u : 0u) << 7)          // A format
           | ((bf16 ? 1u : 0u) << 10)         // B format
           | ((b_mn_major ? 1u : 0u) << 16)   // B major-ness
           | ((uint32_t)(N >> 3) << 17)       // N / 8
           | ((uint32_t)(M >> 4) << 24);      // M / 16
}

// Bounded wait shared by all roles.  Returns false if the CTA is aborting
// (another role gave up) or this wait expired (then it starts the abort).
struct Watch {
    volatile int *abort_flag;
    int *status;
    unsigned long long limit;

    __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = ptx::globaltimer_ns();
        while (true) {
#pragma unroll 1
            for (int i = 0; i < 16; ++i)
                if (ptx::mbar_try_wait(bar, parity)) return true;
            if (*abort_flag) return false;
            if (ptx::globaltimer_ns() - t0 > limit) {
                *abort_flag = 1;
                atomicOr(status, kStatusTimeout);
                return false;
            }
        }
    }
    // Waits for hardware completion (TMA / MMA in flight) during teardown,
    // regardless of the abort flag; bounded by the same limit.
    __device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) const {
        const uint64_t t0 = ptx::globaltimer_ns();
        while (!ptx::mbar_try_wait(bar, parity)) {
            if (ptx::globaltimer_ns() - t0 > limit) {
                atomicOr(status, kStatusTimeout);
                return;
            }
        }
    }
};

// Keeps the compiler from reading tcgen05.ld destination registers before
// tcgen05.wait::ld (and from recycling tcgen05.st source registers before
// tcgen05.wait::st when placed after it).
template <int N>
__device__ __forceinline__ void reg_fence(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

}  // namespace attn
