// Input gradients through quantised layers on the tensor cores (w4_gemm_dx, w4_gemm_dx_gated).
//
//   D[k, m] = sum_n W[n, k] dY[m, n]   (for two layers the sum runs over both layers' n)
//
// The contraction runs over the weight's rows, so a group's scale changes along it and cannot be
// applied to sums: each weight (q - z) s is rounded once to fp16 (2^-11 at most, 1.5e-4 in 2-norm)
// before the fp32-accumulating product.  A group whose weights may be beyond fp16 (scale 4368 or more, near
// the limit of fp16 weights) is recorded as W4_ERR_RANGE: an infinite weight would make NaN of zero gradients.
//
// One cluster of two CTAs computes 256 columns k of dX by `tn` (32 ... 256) of its rows m: each CTA
// dequantises its own 128 k (exactly one group: one scale and zero point per weight row) into shared
// memory, n by n as the rows of packed codes come, which is the MN-major A operand; dY is the K-major
// B operand, half of its rows in each CTA.  Shared memory carries, per 128 n and CTA at tn = 256, dY
// in and out 64 KB, codes in and out 16 KB, weights in and out 64 KB: 144 KB in the 1024 cycles of the
// products, 1.1 times what its port moves; that bounds the kernel (the forward product's way, weights
// through tensor memory, needs lanes of k, and eight lanes would share every packed word).
// M = 2048, K = 4096, N = 11008, both layers: 289 us (1277 TFLOP/s) in a short burst, 340 us (1090) called
// without a pause, where the power limit holds the clock down.
//
//   warp 0       TMA producer: per 128 n the dY tile (two boxes of 64 n) and 128 packed rows of 64 bytes
//   warp 1       CTA 0: issues the pair's tcgen05.mma (M = 256, N = tn, K = 16)
//   warp 2       TMEM allocation
//   warps 4-11   dequantise: two warpgroups take the steps in turn, a thread one weight row
//   warps 12-19  epilogue: TMEM -> shared memory -> whole rows, while the next tile's products run
//                (two TMEM buffers of 256 columns)
//
// Few tiles: the n are cut into slices of whole steps, fp32 partial sums to the workspace [slice][M][K],
// added in slice order by dx_reduce_kernel.  Every mbarrier wait is bounded.
#include <algorithm>
#include <mutex>

#include "activation.cuh"
#include "ffn_common.cuh"
#include "internal.h"

namespace w4 {

namespace {

constexpr int DX_THREADS = 640;
constexpr int DX_MAXS = 8;                      // ring stages at most
constexpr int DX_SLOTS = 2;                     // dequantised steps
constexpr uint32_t DX_P_BYTES = 128 * 64;       // packed codes of a step: 128 n x 128 k
constexpr uint32_t DX_W_BYTES = 128 * 128 * 2;  // dequantised
constexpr uint32_t DX_EPI = 32 * 128 * 4;       // an epilogue warpgroup's 32 rows of 128 fp32
constexpr uint32_t DX_SMEM = 227 * 1024;

struct DxArgs {
    const unsigned short* s[2];
    const uint8_t* z[2];
    __half* out;         // dX, or dG
    __half* out2;        // dU
    const __half* G;     // null: dX itself
    const __half* U;
    float* P;            // fp32 partial sums [slice][M][K], or null
    int act;
    int M, N, K;
    int steps1;          // 128-n steps of one layer
    int steps;           // of all layers
    int tn;
    FfnRaster raster;    // n-tiles: 256 k; ks: slices of the steps
    int units;
    int stages;
    int* status;
};

struct DxUnit {
    int m0, k0, slice, i0, i1;
};
__device__ __forceinline__ DxUnit dx_unit(const DxArgs& p, int u) {
    const FfnUnit t = ffn_unit(p.raster, u);
    DxUnit r;
    r.m0 = t.mt * p.tn;
    r.k0 = t.nt * 256;
    r.slice = t.slice;
    r.i0 = (int)((unsigned)t.slice * (unsigned)p.steps / (unsigned)p.raster.ks);  // steps < 2^25, ks <= 16
    r.i1 = (int)((unsigned)(t.slice + 1) * (unsigned)p.steps / (unsigned)p.raster.ks);
    return r;
}

// Finishes four neighbouring outputs of a row (element offset o) from their sums.
template <int ACT>
__device__ __forceinline__ void dx_finish(const float (&d)[4], int64_t o, uint2 gh, uint2 uh, __half* out, __half* out2) {
    if constexpr (ACT < 0) {
        *reinterpret_cast<uint2*>(out + o) = half4(d);
    } else {
        float g[4], u[4], dg[4], du[4];
        float4_of(gh, g);
        float4_of(uh, u);
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            F2 a;
            const F2 h = f2(d[j], d[j + 1]), s = act_grad2<ACT>(f2(g[j], g[j + 1]), a);
            split(mul2(mul2(h, f2(u[j], u[j + 1])), s), dg[j], dg[j + 1]);
            split(mul2(h, a), du[j], du[j + 1]);
        }
        *reinterpret_cast<uint2*>(out + o) = half4(dg);
        *reinterpret_cast<uint2*>(out2 + o) = half4(du);
    }
}

// The smallest fp16 scale (4368) whose largest weight, 15 s, is beyond fp16.
constexpr uint32_t kLargeScale = 0x6C44u;
// Whether a code of this group can have a weight (q - z) s beyond fp16.
__device__ __forceinline__ bool dx_overflows(uint32_t scale, uint32_t z) {
    const __half s = __ushort_as_half((unsigned short)(scale & 0x7FFFu));
    return !(__hmul(s, __int2half_rn(max((int)z, 15 - (int)z))) <= __ushort_as_half((unsigned short)0x7BFFu));
}

// dispatch_act with -1 for "no gate".
template <typename F>
__host__ __device__ __forceinline__ cudaError_t dispatch_gate(bool gated, int act, F&& f) {
    return gated ? dispatch_act(act, f) : f(std::integral_constant<int, -1>{});
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(DX_THREADS, 1)
    ffn_dx_kernel(const __grid_constant__ CUtensorMap tmY0, const __grid_constant__ CUtensorMap tmY1,
                  const __grid_constant__ CUtensorMap tmW0, const __grid_constant__ CUtensorMap tmW1, const DxArgs p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_align1024(smem_raw);
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = cluster_ctarank();
    const int S = p.stages;
    const uint32_t ybytes = (uint32_t)p.tn * 128u;  // tn/2 rows x 128 n x 2 bytes
    const uint32_t stage_bytes = ybytes + DX_P_BYTES;
    const uint32_t w0 = (uint32_t)S * stage_bytes;  // dequantised steps, staging rows, barriers
    const uint32_t epi0 = w0 + DX_SLOTS * DX_W_BYTES;
    const uint32_t bar0 = sbase + epi0 + 2 * DX_EPI;
    auto full_bar = [&](int s) { return bar0 + 8 * s; };
    auto done_bar = [&](int s) { return bar0 + 8 * (DX_MAXS + s); };
    auto a_full = [&](int i) { return bar0 + 8 * (2 * DX_MAXS + i); };
    auto d_full = [&](int i) { return bar0 + 8 * (2 * DX_MAXS + DX_SLOTS + i); };
    auto d_empty = [&](int i) { return bar0 + 8 * (2 * DX_MAXS + DX_SLOTS + 2 + i); };
    unsigned char* tail = smem + epi0 + 2 * DX_EPI + 8 * (2 * DX_MAXS + DX_SLOTS + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 4);

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(done_bar(s), 1);
        }
        for (int i = 0; i < DX_SLOTS; ++i) mbar_init(a_full(i), 8);  // a dequantising warpgroup of each CTA
        for (int i = 0; i < 2; ++i) {
            mbar_init(d_full(i), 1);
            mbar_init(d_empty(i), 16);  // eight epilogue warps of each CTA
        }
        *abort_flag = 0;
        fence_mbarrier_init();
        prefetch_tmap(&tmY0);
        prefetch_tmap(&tmW0);
    }
    if (warp == 2) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    pdl_launch_dependents();

    auto fail = [&]() {
        *abort_flag = 1;
        record_status(p.status, W4_ERR_DEVICE_TIMEOUT);
    };
    const int cluster = (int)blockIdx.x >> 1, n_clusters = (int)gridDim.x >> 1;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer (one lane issuing)
        pdl_wait();  // every role: nothing is read, written or timed beside the preceding kernel
        int it = 0, s = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int u = cluster; u < p.units && ok; u += n_clusters) {
            const DxUnit w = dx_unit(p, u);
            const int my = w.m0 + (int)rank * (p.tn / 2);
            const int kw = (w.k0 + (int)rank * 128) / 8;
            for (int i = w.i0; i < w.i1; ++i, ++it) {
                if (!mbar_wait_long(done_bar(s), ph, abort_flag)) { fail(); ok = false; break; }
                if (elect_one()) {
                    const uint32_t ys = sbase + (uint32_t)s * stage_bytes;
                    const bool second = i >= p.steps1;
                    const int n = (second ? i - p.steps1 : i) * 128;
                    const CUtensorMap* ty = second ? &tmY1 : &tmY0;
                    mbar_arrive_expect_tx(full_bar(s), stage_bytes);
                    tma_load_2d(ys + ybytes, second ? &tmW1 : &tmW0, kw, n, full_bar(s));
                    tma_load_2d(ys, ty, n, my, full_bar(s));
                    tma_load_2d(ys + ybytes / 2, ty, n + 64, my, full_bar(s));
                }
                __syncwarp();
                if (++s == S) { s = 0; ph ^= 1; }
            }
        }
        // Never leave with loads in flight or with the tensor cores still to arrive on this CTA's
        // barriers: wait (bounded) for the last use of every stage.
        for (int i = max(it - S, 0); i < it; ++i) {
            mbar_wait_long(full_bar(i % S), (uint32_t)(i / S) & 1, nullptr, 200000000ull);
            if (ok) mbar_wait_long(done_bar(i % S), (uint32_t)(i / S) & 1, abort_flag);
        }
    } else if (warp == 1 && rank == 0) {
        // ------------------------------------------------------------ MMA issuer (for both CTAs)
        const uint32_t idesc = idesc_f16_f32(256, p.tn) | kIdescAMnMajor;
        pdl_wait();
        int it = 0, s = 0, ut = 0;
        bool ok = true;
        for (int u = cluster; u < p.units && ok; u += n_clusters, ++ut) {
            const DxUnit w = dx_unit(p, u);
            const int b = ut & 1;
            if (!mbar_wait_long(d_empty(b), ((uint32_t)(ut >> 1) & 1) ^ 1, abort_flag)) { fail(); ok = false; break; }
            for (int i = w.i0; i < w.i1; ++i, ++it) {
                const int a = it % DX_SLOTS;
                if (!mbar_wait_long(a_full(a), (uint32_t)(it / DX_SLOTS) & 1, abort_flag)) { fail(); ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t ad = sw128_mnmajor_desc(sbase + w0 + (uint32_t)a * DX_W_BYTES, DX_W_BYTES / 2);
                    const uint64_t bd = sw128_kmajor_desc(sbase + (uint32_t)s * stage_bytes);
                    const uint64_t half = (uint64_t)(ybytes / 2) >> 4;  // the second 64 n
#pragma unroll
                    for (int j = 0; j < 8; ++j)  // 16 n: 16 rows of 128 bytes of A, 32 bytes along B's rows
                        mma_f16_ss_pair(tmem + b * 256, ad + j * (2048 >> 4), bd + (j >> 2) * half + 2 * (j & 3), idesc,
                                        i != w.i0 || j != 0);
                    tc_commit_pair(done_bar(s));
                    if (i == w.i1 - 1) tc_commit_pair(d_full(b));
                }
                __syncwarp();
                if (++s == S) s = 0;
            }
        }
        // on an abort nobody else waits for what was issued: the pair's TMEM is freed after it
        if (!ok && it > 0) mbar_wait_long(done_bar((it - 1) % S), (uint32_t)((it - 1) / S) & 1, nullptr, 200000000ull);
    } else if (warp >= 4 && warp < 12) {
        // ------------------------------------------------------------ dequantisation
        const int wg = (warp - 4) >> 2;
        const int r = tid & 127;  // row n of the step
        const uint32_t sw = (uint32_t)(r >> 1) & 3, c0 = ybytes + (uint32_t)r * 64;
        const uint32_t wrow = w0 + (uint32_t)wg * DX_W_BYTES + (uint32_t)r * 128;  // DX_SLOTS == 2: a slot each
        const uint32_t remote = map_shared(a_full(wg), 0);
        const int64_t G = p.K >> 7;
        pdl_wait();
        bool ok = true;
        int it = wg, s = wg, sa = wg;  // step, its ring stage, the ring stage of step it - 2
        uint32_t ph = 0, pa = 0;
        int skip = wg;
        // scale and zero point of this thread's row in step i of the unit's column of groups
        auto meta = [&](int i, int g, uint32_t& sc, uint32_t& z) {
            sc = 0;
            z = 0;
            const bool second = i >= p.steps1;
            const int64_t n = (int64_t)(second ? i - p.steps1 : i) * 128 + r;
            if (n < p.N && g < G) {
                sc = __ldg(p.s[second ? 1 : 0] + n * G + g);
                z = __ldg(p.z[second ? 1 : 0] + n * G + g);
                if ((sc & 0x7FFFu) >= kLargeScale && dx_overflows(sc, z)) record_status(p.status, W4_ERR_RANGE);
            }
        };
        for (int u = cluster; u < p.units; u += n_clusters) {
            const DxUnit w = dx_unit(p, u);
            const int g = (w.k0 >> 7) + (int)rank;
            int i = w.i0 + skip;
            uint32_t sc = 0, z = 0, scn, zn;
            if (i < w.i1) meta(i, g, sc, z);
            for (; i < w.i1; i += 2) {
                if (i + 2 < w.i1) meta(i + 2, g, scn, zn);  // the next step's, while this one is dequantised
                else scn = zn = 0;
                const uint32_t s2 = sc * 0x10001u;
                const uint32_t zl = (0x6400u + z) * 0x10001u, zh = (0xD400u | (z << 4)) * 0x10001u;
                if (ok && !warp_wait(full_bar(s), ph, abort_flag)) { fail(); ok = false; }
                if (it >= 2) {  // the slot's last step has been multiplied
                    if (ok && !warp_wait(done_bar(sa), pa, abort_flag)) { fail(); ok = false; }
                    sa += 2;
                    if (sa >= S) { sa -= S; pa ^= 1; }
                }
                const unsigned char* st = smem + (uint32_t)s * stage_bytes + c0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {  // 16 bytes: 32 k
                    const uint4 v = *reinterpret_cast<const uint4*>(st + (((uint32_t)c ^ sw) << 4));
                    const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t wd = words[j], w8 = wd >> 8;
                        uint32_t lo0 = hsub2_u32(lop3_and_or(wd, 0x000F000Fu, 0x64006400u), zl);              // k0, k4
                        uint32_t hi0 = hfma2_u32(lop3_and_or(wd, 0x00F000F0u, 0x64006400u), 0x2C002C00u, zh);  // k1, k5
                        uint32_t lo1 = hsub2_u32(lop3_and_or(w8, 0x000F000Fu, 0x64006400u), zl);              // k2, k6
                        uint32_t hi1 = hfma2_u32(lop3_and_or(w8, 0x00F000F0u, 0x64006400u), 0x2C002C00u, zh);  // k3, k7
                        lo0 = hmul2_u32(lo0, s2);
                        hi0 = hmul2_u32(hi0, s2);
                        lo1 = hmul2_u32(lo1, s2);
                        hi1 = hmul2_u32(hi1, s2);
                        // the pairs as they come: eight k are stored in the order 0 4 1 5 2 6 3 7, which orders the
                        // product's rows; the epilogue puts them back
                        const uint4 o = make_uint4(lo0, hi0, lo1, hi1);
                        const uint32_t ch = (uint32_t)(4 * c + j);  // 8-k chunk 0 .. 15: block of 64 k, chunk in it
                        *reinterpret_cast<uint4*>(smem + wrow + (ch >> 3) * (DX_W_BYTES / 2) +
                                                  (((ch & 7) ^ ((uint32_t)r & 7)) << 4)) = o;
                    }
                }
                fence_proxy_async_shared();  // the stores are in place for the tensor cores: before the arrival (mbar_arrive_cluster)
                __syncwarp();
                if (ok && lane == 0) mbar_arrive_cluster(remote);
                sc = scn;
                z = zn;
                it += 2;
                s += 2;
                if (s >= S) { s -= S; ph ^= 1; }
            }
            skip = i - w.i1;
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------ epilogue
        const int f = (warp - 12) >> 2, q = warp & 3;
        const int r = q * 32 + lane;
        const int ncol = p.tn / 2;
        const uint32_t remote = map_shared(d_empty(0), 0);
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(f * ncol);
        float* st = reinterpret_cast<float*>(smem + epi0 + (uint32_t)f * DX_EPI);
        pdl_wait();
        const int kr = (r & ~7) | ((r & 7) >> 1) | ((r & 1) << 2);  // the k of this lane's row of the product
        bool ok = true;
        int ut = 0;
        for (int u = cluster; u < p.units; u += n_clusters, ++ut) {
            const DxUnit w = dx_unit(p, u);
            const int b = ut & 1;
            // a whole tile's products: the limit grows with its steps (under 1 us each)
            const uint64_t limit = 2000000000ull + 10000ull * (uint64_t)(w.i1 - w.i0);
            if (ok && !warp_wait(d_full(b), (uint32_t)(ut >> 1) & 1, abort_flag, limit)) { fail(); ok = false; }
            if (wg_barrier_any(1 + f, !ok)) { ok = false; continue; }  // all four warps agree before the staging barriers
            tc_fence_after();
            const int m0 = w.m0 + f * ncol, kb = w.k0 + (int)rank * 128, k = kb + 4 * lane;
            float* P = p.P ? p.P + (int64_t)w.slice * p.M * p.K : nullptr;
#pragma unroll 1
            for (int c = 0; c < ncol; c += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(taddr + (uint32_t)(b * 256 + c), v);  // columns past tn/2: never stored
                tmem_wait_ld();
                if (c + 32 >= ncol) {  // all read: the buffer is free
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(remote + 8u * (uint32_t)b);
                }
                const int rows = min(min(32, ncol - c), p.M - m0 - c);
#pragma unroll
                for (int i = 0; i < 32; ++i) st[i * 128 + kr] = __uint_as_float(v[i]);
                wg_barrier(1 + f);
                int64_t o = (int64_t)(m0 + c + q) * p.K + k;
                const float* sr = st + q * 128 + 4 * lane;
                dispatch_gate(p.G != nullptr && !P, p.act, [&](auto act) {
                    constexpr int ACT = decltype(act)::value;
#pragma unroll 1
                    for (int i = 0; i < 8; i += 2) {  // rows q, q + 4, ...: two rows' loads in flight together
                        const int left = k < p.K ? rows - q - 4 * i : 0;
                        uint2 gh[2] = {}, uh[2] = {};
                        if (ACT >= 0) {
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (4 * j < left) {
                                    gh[j] = *reinterpret_cast<const uint2*>(p.G + o + (int64_t)(4 * j) * p.K);
                                    uh[j] = *reinterpret_cast<const uint2*>(p.U + o + (int64_t)(4 * j) * p.K);
                                }
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if (4 * j < left) {
                                const float4 a = *reinterpret_cast<const float4*>(sr + 4 * (i + j) * 128);
                                if (P) {
                                    *reinterpret_cast<float4*>(P + o) = a;
                                } else {
                                    const float d[4] = {a.x, a.y, a.z, a.w};
                                    dx_finish<ACT>(d, o, gh[j], uh[j], p.out, p.out2);
                                }
                            }
                            o += (int64_t)4 * p.K;
                        }
                    }
                    return cudaSuccess;
                });
                wg_barrier(1 + f);
            }
        }
    }
    __syncthreads();
    cluster_sync();  // nothing of the pair's products or arrivals is outstanding in either CTA
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// The slices' partial sums [slice][M][K] in slice order, then the outputs.  A programmatic dependent
// of the kernel that writes the partials.
template <int ACT>
__global__ void __launch_bounds__(256) dx_reduce_kernel(const float* P, int slices, int64_t mk, const __half* G,
                                                        const __half* U, __half* out, __half* out2) {
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; e < mk; e += (int64_t)gridDim.x * 1024) {
        uint2 gh = {}, uh = {};
        if (ACT >= 0) {
            gh = *reinterpret_cast<const uint2*>(G + e);
            uh = *reinterpret_cast<const uint2*>(U + e);
        }
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < slices; ++s) {
            const float4 b = *reinterpret_cast<const float4*>(P + (int64_t)s * mk + e);
            d[0] += b.x; d[1] += b.y; d[2] += b.z; d[3] += b.w;
        }
        dx_finish<ACT>(d, e, gh, uh, out, out2);
    }
}

struct DxPlan {
    int tn, ks, stages, m_tiles, k_tiles, units, steps1, steps;
    uint32_t smem;
};

DxPlan dx_plan(int64_t M, int64_t N, int64_t K, int n_layers) {
    const int64_t pairs = std::max(1, device_sm_count() / 2);
    DxPlan best = {};
    best.steps1 = (int)((N + 127) / 128);
    best.steps = best.steps1 * n_layers;
    const int64_t k_tiles = (K + 255) / 256;
    double best_t = -1.0;
    for (int tn : {32, 64, 128, 256}) {
        if (tn > 32 && tn / 2 >= M) break;
        const int64_t m_tiles = (M + tn - 1) / tn, tiles = m_tiles * k_tiles;
        for (int ks = 1; ks <= 16 && ks <= best.steps; ++ks) {
            if (ks > 1 && (tiles * (ks - 1) >= pairs || best.steps / ks < 4)) break;
            const int64_t units = tiles * ks, waves = (units + pairs - 1) / pairs;
            // cycles per step: the products or the dequantising warps; per unit: filling and the last
            // epilogue; a second launch and its traffic when the n are cut
            const double step = std::max(4.5 * tn, 500.0);
            double t = (double)waves * ((double)((best.steps + ks - 1) / ks) * step + 2000.0);
            if (ks > 1) t += 4000.0 + (double)ks * (double)M * (double)K * 8.0 / 3000.0;
            if (best_t < 0.0 || t < best_t) {
                best_t = t;
                best.tn = tn;
                best.ks = ks;
                best.m_tiles = (int)m_tiles;
                best.k_tiles = (int)k_tiles;
                best.units = (int)units;
            }
        }
    }
    const uint32_t stage = (uint32_t)best.tn * 128u + DX_P_BYTES;
    const uint32_t fixed = DX_SLOTS * DX_W_BYTES + 2 * DX_EPI + 512;
    best.stages = (int)std::min<uint32_t>((DX_SMEM - 1024 - fixed) / stage, DX_MAXS);
    best.smem = stage * (uint32_t)best.stages + fixed + 1024;
    return best;
}

cudaError_t dx_setup() {
    static std::once_flag once[64];
    static cudaError_t err[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&]() {
        err[dev] = cudaFuncSetAttribute(ffn_dx_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)DX_SMEM);
    });
    return err[dev];
}

}  // namespace

size_t ffn_dx_workspace(int64_t M, int64_t N, int64_t K, int n_layers) {
    const DxPlan pl = dx_plan(M, N, K, n_layers);
    return pl.ks > 1 ? (size_t)pl.ks * (size_t)M * (size_t)K * 4 : 0;
}

cudaError_t launch_ffn_dx(const uint16_t* dY, const W4Layer& w, const uint16_t* dY2, const W4Layer* w2, int64_t M,
                          int64_t N, int64_t K, const W4GateGrad* gate, uint16_t* dX, void* ws, int* status,
                          cudaStream_t stream) {
    const DxPlan pl = dx_plan(M, N, K, w2 ? 2 : 1);
    if (pl.ks > 1 && !ws) return cudaErrorInvalidValue;
    cudaError_t e = dx_setup();
    if (e != cudaSuccess) return e;
    CUtensorMap ty[2], tw[2];
    for (int l = 0; l < (w2 ? 2 : 1); ++l) {
        if (!make_tensor_map_2d(&ty[l], l ? dY2 : dY, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, (uint64_t)N, (uint64_t)M, 64,
                                (uint32_t)(pl.tn / 2), CU_TENSOR_MAP_SWIZZLE_128B) ||
            !make_tensor_map_2d(&tw[l], l ? w2->packed : w.packed, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, (uint64_t)(K / 8),
                                (uint64_t)N, 16, 128, CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
    }
    if (!w2) {
        ty[1] = ty[0];
        tw[1] = tw[0];
    }
    DxArgs a = {};
    a.s[0] = w.scales;
    a.z[0] = w.zeros;
    a.s[1] = w2 ? w2->scales : w.scales;
    a.z[1] = w2 ? w2->zeros : w.zeros;
    a.out = hp(gate ? gate->dG : dX);
    a.out2 = gate ? hp(gate->dU) : nullptr;
    a.G = gate ? hp(gate->G) : nullptr;
    a.U = gate ? hp(gate->U) : nullptr;
    a.P = pl.ks > 1 ? static_cast<float*>(ws) : nullptr;
    a.act = gate ? gate->activation : 0;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.steps1 = pl.steps1;
    a.steps = pl.steps;
    a.tn = pl.tn;
    a.raster.m_tiles = pl.m_tiles;
    a.raster.n_tiles = pl.k_tiles;
    a.raster.ks = pl.ks;
    // m-tiles whose dY stays in L2 (about 48 MB) run along the k-tiles together
    a.raster.gm = (int)std::max<int64_t>(1, std::min<int64_t>(pl.m_tiles, (48ll << 20) / ((int64_t)pl.tn * N * 2 * (w2 ? 2 : 1))));
    a.units = pl.units;
    a.stages = pl.stages;
    a.status = status;
    const int clusters = std::min(pl.units, std::max(1, device_sm_count() / 2));
    cudaLaunchConfig_t cfg = {};  // both launches: programmatic dependents of what precedes them
    cfg.gridDim = dim3((unsigned)(2 * clusters), 1, 1);
    cfg.blockDim = dim3(DX_THREADS, 1, 1);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, ffn_dx_kernel, ty[0], ty[1], tw[0], tw[1], a);
    if (e != cudaSuccess || pl.ks == 1) return e;
    const int64_t mk = M * K;
    const int64_t want = (mk / 4 + 255) / 256, cap = (int64_t)device_sm_count() * 8;
    cfg.gridDim = dim3((unsigned)std::min(want, cap), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return dispatch_gate(gate != nullptr, a.act, [&](auto act) {
        return cudaLaunchKernelEx(&cfg, dx_reduce_kernel<decltype(act)::value>, (const float*)a.P, pl.ks, mk, a.G, a.U, a.out,
                                  a.out2);
    });
}

}  // namespace w4
