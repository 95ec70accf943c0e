// Shared device helpers for libw4a16 (sm_100a only).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "w4a16.h"

#if defined(__CUDA_ARCH__) && (__CUDA_ARCH__ != 1000)
#error "libw4a16 is built for sm_100a only"
#endif

namespace w4 {

// Records the first device-side error of a call in the per-device status word.
__device__ __forceinline__ void record_status(int* status, int code) {
    if (status) atomicCAS(status, 0, code);
}

// 128-bit streaming load that bypasses L1 (weights are read exactly once per call).
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
    uint4 r;
    asm("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "l"(p));
    return r;
}

// 128-bit read-only load that may be cached (activations and metadata shared across CTAs).
__device__ __forceinline__ uint4 ldg_cached(const void* p) {
    uint4 r;
    asm("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
        : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
        : "l"(p));
    return r;
}

// (a & b) | c in one LOP3.
__device__ __forceinline__ uint32_t lop3_and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// (a & b) ^ c in one LOP3.
__device__ __forceinline__ uint32_t lop3_and_xor(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__device__ __forceinline__ uint32_t hsub2_u32(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t hfma2_u32(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The GEMV families' operands: nibbles of bytes 0 and 2 of a word under an exponent, one LOP3 for two, with
// opposite signs in the lower and the upper half:
//     low nibbles (k0, k4; of w >> 8 k2, k6)     1024 + q    and  -(1024 + 15 - q)        = q - 1039
//     high nibbles (k1, k5; of w >> 8 k3, k7)    1024 + 16 q and  -(1024 + 16 (15 - q))   = 16 q - 1264
// Why opposite signs: an MMA cuts its fp32 sums off towards zero, so with offsets of one sign every partial
// sum of a row of one-signed activations (behind a relu, say) lost half a step of 2^17 in the same direction,
// all outputs off by 1.2e-3 (K = 4096) to 3.1e-3 (K = 28672) of their rms on mma.sync and 3.0e-3 (K = 4096)
// to 4.9e-3 (K = 11008) on tcgen05.  With both signs the offsets cancel as they are summed, whatever the
// activations' mean: 1e-5 to 8e-5.
__device__ __forceinline__ uint32_t raw_low(uint32_t w) { return lop3_and_xor(w, 0x000F000Fu, 0xE40F6400u); }
__device__ __forceinline__ uint32_t raw_high(uint32_t w) { return lop3_and_xor(w, 0x00F000F0u, 0xE4F06400u); }

// Eight activations as they are staged for those operands, p = (x0, x4), (x1, x5) / 16, (x2, x6), (x3, x7) / 16:
// what their offsets add to a sum, and the sum of the x.
__device__ __forceinline__ void raw_offsets(const uint4& p, float& C, float& S) {
    auto floats = [](uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); };
    const float2 l0 = floats(p.x), h0 = floats(p.y), l1 = floats(p.z), h1 = floats(p.w);
    const float la = l0.x + l1.x, lb = l0.y + l1.y, ha = h0.x + h1.x, hb = h0.y + h1.y;
    C = fmaf(-1264.0f, hb, fmaf(-1039.0f, lb, 1024.0f * (la + ha)));
    S = fmaf(16.0f, ha + hb, la + lb);
}

// Two fp32 -> packed f16x2 (round to nearest), low half = a.
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Programmatic dependent launch: wait for the preceding kernel's memory to be visible, and
// allow the next kernel in the stream to start launching.  Both are no-ops without the
// launch attribute.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// D = A(16x16, row) * B(16x8, col) + C, fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

}  // namespace w4
