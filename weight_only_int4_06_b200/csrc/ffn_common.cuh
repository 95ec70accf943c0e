// Shared pieces of the feed-forward products (ffn_gemm.cu, ffn_dx.cu).
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace w4 {

// mbar_wait_bounded with long suspended tries (20 us each) and the clock read only after them: two
// dozen warps wait in turn here, and shorter tries took issue slots from the warps that compute.
__device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, volatile int* abort,
                                               uint64_t limit_ns = 2000000000ull) {
    if (mbar_try_wait_suspend(bar, parity, 20000u)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait_suspend(bar, parity, 20000u)) return true;
        if (abort && *abort) return false;
        if (globaltimer_ns() - t0 > limit_ns) return false;
    }
}

// A bounded wait by a whole warp, with one outcome for it (what follows is warp-synchronous).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                          uint64_t limit_ns = 2000000000ull) {
    return __all_sync(0xffffffffu, mbar_wait_long(bar, parity, abort, limit_ns));
}

// Barrier of one warpgroup.
__device__ __forceinline__ void wg_barrier(int id) {  // 1 or 2, as constants: an id in a register is slower
    if (id == 1) asm volatile("bar.sync 1, 128;" ::: "memory");
    else asm volatile("bar.sync 2, 128;" ::: "memory");
}

// Whether any of the warpgroup's threads has `bad` set.
__device__ __forceinline__ bool wg_barrier_any(int id, bool bad) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 128, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"((uint32_t)bad)
                 : "memory");
    return r != 0;
}

// Four fp32 values <-> 8 bytes of fp16.
__device__ __forceinline__ uint2 half4(const float (&f)[4]) { return make_uint2(pack_half2(f[0], f[1]), pack_half2(f[2], f[3])); }
__device__ __forceinline__ void float4_of(const uint2& h, float (&f)[4]) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h.y));
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// Work unit u of `units` = m_tiles * n_tiles * ks: K slice first, then gm m-tiles running down the
// n-tiles together (their activations stay in L2).
struct FfnRaster {
    int m_tiles, n_tiles, gm, ks;
};
struct FfnUnit {
    int mt, nt, slice;
};
__device__ __forceinline__ FfnUnit ffn_unit(const FfnRaster& p, int u) {
    FfnUnit r;
    r.slice = u % p.ks;
    const int t = u / p.ks;
    const int per = p.gm * p.n_tiles;
    const int grp = t / per, first = grp * p.gm;
    const int gm = min(p.gm, p.m_tiles - first);
    const int rem = t - grp * per;
    r.mt = first + rem % gm;
    r.nt = rem / gm;
    return r;
}

inline const __half* hp(const uint16_t* p) { return reinterpret_cast<const __half*>(p); }
inline __half* hp(uint16_t* p) { return reinterpret_cast<__half*>(p); }

}  // namespace w4
