// attn_common.cuh -- what the attention kernels share: packing to the input
// type, tensor-memory reads, the softmax's arithmetic and the bounded wait of
// their pipelines.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "li.h"
#include "ptx.cuh"

namespace li {

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <bool F16>
__device__ __forceinline__ float unpack_lo(uint32_t v)
{
    if constexpr (F16) return __half2float(__ushort_as_half((unsigned short)(v & 0xFFFFu)));
    else return __uint_as_float(v << 16);
}

template <bool F16>
__device__ __forceinline__ float unpack_hi(uint32_t v)
{
    if constexpr (F16) return __half2float(__ushort_as_half((unsigned short)(v >> 16)));
    else return __uint_as_float(v & 0xFFFF0000u);
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Columns 16*CH .. 16*CH+15 of this warp's lanes into r[16*CH ..].
template <int CH, int N>
__device__ __forceinline__ void tmem_ld16_into(uint32_t taddr, uint32_t (&r)[N])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[16 * CH + 0]), "=r"(r[16 * CH + 1]), "=r"(r[16 * CH + 2]), "=r"(r[16 * CH + 3]),
          "=r"(r[16 * CH + 4]), "=r"(r[16 * CH + 5]), "=r"(r[16 * CH + 6]), "=r"(r[16 * CH + 7]),
          "=r"(r[16 * CH + 8]), "=r"(r[16 * CH + 9]), "=r"(r[16 * CH + 10]), "=r"(r[16 * CH + 11]),
          "=r"(r[16 * CH + 12]), "=r"(r[16 * CH + 13]), "=r"(r[16 * CH + 14]), "=r"(r[16 * CH + 15])
        : "r"(taddr + 16 * CH));
}

// 2^x on the special-function unit (relative error about 2^-22, far below
// the 16-bit rounding the weights get next); 2^-inf = 0.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// max of three (one instruction on sm_100)
__device__ __forceinline__ float fmax3(float x, float y, float z)
{
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
    return m;
}

// (d0, d1) = (a0 * b0 + c0, a1 * b1 + c1) as one packed fp32 instruction
__device__ __forceinline__ void ffma2(float &d0, float &d1, float a0, float a1, float b0, float b1, float c0,
                                      float c1)
{
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

// (d0, d1) += (x0, x1) as one packed fp32 instruction
__device__ __forceinline__ void fadd2(float &d0, float &d1, float x0, float x1)
{
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(x0), "f"(x1));
}

// Bounded wait on an mbarrier phase.  A wait that expires (2 s) flags
// LI_DEV_TIMEOUT and sets the CTA's abort flag; from then on every wait of
// the CTA returns after one suspended try (at most about a microsecond), and
// so does a wait of another CTA once it sees the flag in `status`, so a
// broken pipeline ends the kernel promptly (results are then undefined; the
// context stays usable).
__device__ __forceinline__ void wait_phase(uint64_t *bar, uint32_t parity, int32_t *status, volatile int *abort)
{
    // the waiting thread is suspended in hardware (up to 1 us per try) until
    // the phase completes, instead of spinning on the issue slots
    if (mbar_try_wait(bar, parity)) return;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1; !mbar_try_wait_sleep(bar, parity, 1000u); ++it) {
        if (*abort) return;
        // another CTA's timeout, looked at every 256 tries (a global load)
        if ((it & 255u) == 0 && status && (*reinterpret_cast<volatile int32_t *>(status) & LI_DEV_TIMEOUT)) {
            *abort = 1;
            return;
        }
        if ((int64_t)(global_timer_ns() - t0) > 2000000000LL) {
            *abort = 1;
            if (status) atomicOr(status, LI_DEV_TIMEOUT);
            return;
        }
    }
}

}  // namespace li
