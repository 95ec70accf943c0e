// Forward products of the feed-forward operators on the tensor cores (w4_gemm_fused, w4_gemm_gated).
//
//   D[n, m] = sum_g s[n, g] * sum_{k in g} (q[n, k] - z[n, g]) X[m, k]
//
// The codes' differences q - z are whole numbers of at most 15, exact in fp16, so the tensor cores sum
// exact products in fp32 and the scale multiplies each group's sum in fp32: no weight is ever rounded
// (a weight (q - z) s rounded to fp16 costs 1.5e-4 of the result in 2-norm, as much again as the
// output's own rounding; in the gated product it enters twice).
//
// One cluster of two CTAs computes a tile of 256 weight rows by `tn` (32 ... NMAX) rows of X. The
// weights are the A operand, written by the dequantising threads straight into tensor memory (thread
// = weight row = TMEM lane); X is the B operand, half of its rows in each CTA's shared memory.  Why
// this way round: the weights never pass through shared memory as fp16, which a 256 x 192 tile's
// shared-memory port could not carry beside the tensor cores' own reads (per group of 128 and CTA:
// X in 24 KB, X out 24 KB, codes in and out 16 KB, 64 KB in the 768 cycles of its products; weights
// as fp16 would add 64 KB); a thread owns one weight row, so a group has one scale per thread; and
// small batches cost products of 32 columns, not 128.
//
//   warp 0       TMA producer of its CTA: per group X (two boxes of 64 k) and the packed rows
//   warp 1       CTA 0: one thread issues the pair's tcgen05.mma (M = 256, N = tn, K = 16)
//   warp 2       TMEM allocation
//   warps 4-11   dequantise: the first four warps each group's k 0-63, the other four its k 64-127;
//                64 codes of a row -> 32 TMEM columns
//   warps 12-19  fold: the first four take columns 0 .. tn/2 - 1, the others the rest: read a group's
//                sums from TMEM, acc += s * sum in registers; after the last group the epilogue
// The group sums alternate between two TMEM buffers, the dequantised halves between four, so a
// group's products, the next one's dequantisation and the last one's fold overlap.
//
// Gated: the 32 lanes of a warp hold 16 gate rows and the 16 up rows of the same n, so g and u of an
// output meet by one shuffle between lanes i and i + 16.
//
// Few tiles: K is cut into slices of whole groups, their fp32 sums go to the workspace [slice][layer]
// [M][N] and ffn_reduce_kernel adds them in slice order and runs the epilogue: deterministic.
//
// Every mbarrier wait is bounded; on timeout the kernel records W4_ERR_DEVICE_TIMEOUT and drains.
#include <algorithm>
#include <mutex>

#include "activation.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace w4 {

namespace {

constexpr int FG_THREADS = 640;
constexpr int FG_MAXS = 16;                        // ring stages at most
constexpr uint32_t FG_P_BYTES = 128 * 64;          // packed codes of one group: 128 rows x 64 bytes
constexpr uint32_t FG_SMEM = 227 * 1024;
constexpr int FG_ASLOTS = 4;                       // dequantised half groups (32 TMEM columns each)
// registers per thread: launch allotment 96 x 640; the fold warps' accumulators take what the others
// give up (32 + 72 + 72 + 152 + 152 = 5 x 96)
constexpr int FG_REGS_LAUNCH = 96, FG_REGS_MISC = 32, FG_REGS_DEQ = 72, FG_REGS_FOLD = 152;

struct FgArgs {
    const unsigned short* s0;
    const uint8_t* z0;
    const unsigned short* s1;  // gated: the up projection's
    const uint8_t* z1;
    const __half* bias;
    const __half* residual;
    __half* Y;
    __half* Z;
    __half* U;
    float* P;  // fp32 partial sums [slice][layer][M][N], or null: epilogue in place
    int act;
    int M, N, G;
    int tn;           // X rows per tile
    int m_tiles, n_tiles, gm;  // raster: gm m-tiles run down the n-tiles together
    int ks;           // K slices
    int units;        // m_tiles * n_tiles * ks
    int stages;
    int vec;          // metadata rows allow 4-group vector loads
    int early;        // weights may be read before the preceding kernel has finished
    int* status;
};

struct FgUnit {
    int m0, nt, slice, g0, g1;
};

__device__ __forceinline__ FgUnit fg_unit(const FgArgs& p, int u) {
    FgUnit r;
    r.slice = u % p.ks;
    const int t = u / p.ks;
    const int per = p.gm * p.n_tiles;
    const int grp = t / per, first = grp * p.gm;
    const int gm = min(p.gm, p.m_tiles - first);
    const int rem = t - grp * per;
    r.m0 = (first + rem % gm) * p.tn;
    r.nt = rem / gm;
    r.g0 = (int)((int64_t)r.slice * p.G / p.ks);
    r.g1 = (int)((int64_t)(r.slice + 1) * p.G / p.ks);
    return r;
}

// Four consecutive groups' scales (fp16) of a row in one 64-bit word, starting at g & ~3.
__device__ __forceinline__ uint64_t fg_scales4(const unsigned short* row, int g, int G, bool vec) {
    const int b = g & ~3;
    if (vec) return __ldg(reinterpret_cast<const unsigned long long*>(row + b));
    uint64_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (b + i < G) v |= (uint64_t)__ldg(row + b + i) << (16 * i);
    return v;
}
__device__ __forceinline__ uint32_t fg_zeros4(const uint8_t* row, int g, int G, bool vec) {
    const int b = g & ~3;
    if (vec) return __ldg(reinterpret_cast<const unsigned int*>(row + b));
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (b + i < G) v |= (uint32_t)__ldg(row + b + i) << (8 * i);
    return v;
}

// acc (two fp32) += s * v, one packed FMA.
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t v, uint64_t s) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}
__device__ __forceinline__ uint64_t pack_f32x2(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}

// One tile's outputs from this thread's accumulators: weight row / output column n, X rows m0 ..
// m0 + 16 NCH - 1 (acc[c]).  Lanes of a warp are neighbouring n: stores of one m are contiguous.
template <int ACT, int NACC>
__device__ __forceinline__ void fg_epilogue_plain(const FgArgs& p, const uint64_t (&acc)[NACC / 2], int ncol, int m0, int n) {
    if (n >= p.N) return;
    const float b = p.bias ? __half2float(p.bias[n]) : 0.0f;
    const int64_t o = (int64_t)m0 * p.N + n;
    __half* y = p.Y + o;
    __half* z = p.Z ? p.Z + o : nullptr;
    const __half* r = p.residual ? p.residual + o : nullptr;
    const int rows = min(ncol, p.M - m0);
#pragma unroll
    for (int c = 0; c < NACC; c += 8) {
        if (c < rows) {
            float res[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                res[i] = r && c + i < rows ? __half2float(*r) : 0.0f;
                if (r) r += p.N;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float v[2];
                unpack_f32x2(acc[(c + i) / 2], v[0], v[1]);
                const float pre = v[i & 1] + b;
                if (c + i < rows) {
                    *y = __float2half_rn(act_fwd<ACT>(pre) + res[i]);
                    if (z) *z = __float2half_rn(pre);
                }
                y += p.N;
                if (z) z += p.N;
            }
        }
    }
}

// Gated: lanes 0-15 hold g, lanes 16-31 u of the same 16 columns n; a lower lane finishes the even X
// row of each pair, an upper lane the odd one.
template <int ACT, int NACC>
__device__ __forceinline__ void fg_epilogue_gated(const FgArgs& p, const uint64_t (&acc)[NACC / 2], int ncol, int m0, int n,
                                                  bool upper) {
    const bool nv = n < p.N;
    const int rows = nv ? min(ncol, p.M - m0) : 0;
    const int64_t o = (int64_t)m0 * p.N + n;
    __half* h = p.Y + o + (upper ? p.N : 0);
    __half* pre = p.Z ? (upper ? p.U : p.Z) + o : nullptr;
    const int odd = upper ? 1 : 0;
#pragma unroll
    for (int c = 0; c < NACC; c += 2) {
        if (c < ncol) {  // uniform over the warp
            float v[2];
            unpack_f32x2(acc[c / 2], v[0], v[1]);
            const float other = __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[1], 16);
            const float g = upper ? other : v[0], u = upper ? v[1] : other;
            if (c + odd < rows) *h = __float2half_rn(act_fwd<ACT>(g) * u);
            h += 2 * (int64_t)p.N;
            if (pre) {
                if (c < rows) *pre = __float2half_rn(v[0]);
                if (c + 1 < rows) pre[p.N] = __float2half_rn(v[1]);
                pre += 2 * (int64_t)p.N;
            }
        }
    }
}

template <bool GATED, int NMAX>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FG_THREADS, 1)
    ffn_gemm_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW0,
                    const __grid_constant__ CUtensorMap tmW1, const FgArgs p) {
    constexpr int NACC = NMAX / 2;            // columns per fold thread
    constexpr uint32_t TCOLS = NMAX > 64 ? 512 : 256;
    constexpr uint32_t ACOL = 2 * NMAX;       // TMEM column of the first dequantised half group
    constexpr bool SETREGS = NMAX > 64;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_align1024(smem_raw);
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int S = p.stages;
    const uint32_t xbytes = (uint32_t)p.tn * 128u;  // tn/2 rows x 128 k x 2 bytes
    const uint32_t stage_bytes = xbytes + FG_P_BYTES;
    auto x_addr = [&](int s) { return sbase + (uint32_t)s * stage_bytes; };
    auto p_off = [&](int s) { return (uint32_t)s * stage_bytes + xbytes; };
    const uint32_t bar0 = sbase + (uint32_t)S * stage_bytes;
    auto full_bar = [&](int s) { return bar0 + 8 * s; };
    auto empty_bar = [&](int s) { return bar0 + 8 * (FG_MAXS + s); };
    auto a_full = [&](int i) { return bar0 + 8 * (2 * FG_MAXS + i); };
    auto a_empty = [&](int i) { return bar0 + 8 * (2 * FG_MAXS + FG_ASLOTS + i); };
    auto d_full = [&](int i) { return bar0 + 8 * (2 * FG_MAXS + 2 * FG_ASLOTS + i); };
    auto d_empty = [&](int i) { return bar0 + 8 * (2 * FG_MAXS + 2 * FG_ASLOTS + 2 + i); };
    unsigned char* tail = smem + (uint32_t)S * stage_bytes + 8 * (2 * FG_MAXS + 2 * FG_ASLOTS + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 4);

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int i = 0; i < FG_ASLOTS; ++i) {
            mbar_init(a_full(i), 8);   // four warps of each CTA
            mbar_init(a_empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(d_full(i), 1);
            mbar_init(d_empty(i), 16);  // eight warps of each CTA
        }
        *abort_flag = 0;
        fence_mbarrier_init();
        prefetch_tmap(&tmX);
        prefetch_tmap(&tmW0);
        if (GATED) prefetch_tmap(&tmW1);
    }
    if (warp == 2) {
        tmem_alloc_pair(smem_u32(tmem_slot), TCOLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();

    auto fail = [&]() {
        *abort_flag = 1;
        record_status(p.status, W4_ERR_DEVICE_TIMEOUT);
    };
    const int cluster = (int)blockIdx.x >> 1, n_clusters = (int)gridDim.x >> 1;

    if (warp < 4) {
        if (SETREGS) regs_dec<FG_REGS_MISC>();
        if (warp == 0 && lane == 0) {
            // -------------------------------------------------------- TMA producer
            auto load_w = [&](const FgUnit& u, int g, int s) {
                const uint32_t dst = sbase + p_off(s);
                if constexpr (GATED) {
                    const int n = u.nt * 128 + (int)rank * 64;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        tma_load_2d(dst + q * 2048, &tmW0, g * 16, n + 16 * q, full_bar(s));
                        tma_load_2d(dst + q * 2048 + 1024, &tmW1, g * 16, n + 16 * q, full_bar(s));
                    }
                } else {
                    tma_load_2d(dst, &tmW0, g * 16, u.nt * 256 + (int)rank * 128, full_bar(s));
                }
            };
            if (!p.early) pdl_wait();
            int it = 0, ahead = 0;
            if (p.early) {  // the first ring's weights, before the preceding kernel has finished
                for (int u = cluster; u < p.units && ahead < S; u += n_clusters) {
                    const FgUnit w = fg_unit(p, u);
                    for (int g = w.g0; g < w.g1 && ahead < S; ++g, ++ahead) {
                        mbar_arrive_expect_tx(full_bar(ahead), stage_bytes);
                        load_w(w, g, ahead);
                    }
                }
                pdl_wait();
            }
            bool ok = true;
            for (int u = cluster; u < p.units && ok; u += n_clusters) {
                const FgUnit w = fg_unit(p, u);
                const int mx = w.m0 + (int)rank * (p.tn / 2);
                for (int g = w.g0; g < w.g1; ++g, ++it) {
                    const int s = it % S;
                    const uint32_t ph = (uint32_t)(it / S) & 1;
                    if (it >= ahead) {
                        if (!mbar_wait_cluster(empty_bar(s), ph ^ 1, abort_flag)) { fail(); ok = false; break; }
                        mbar_arrive_expect_tx(full_bar(s), stage_bytes);
                        load_w(w, g, s);
                    }
                    tma_load_2d(x_addr(s), &tmX, g * 128, mx, full_bar(s));
                    tma_load_2d(x_addr(s) + xbytes / 2, &tmX, g * 128 + 64, mx, full_bar(s));
                }
            }
            // Never leave with loads in flight or with the tensor cores still to arrive on this CTA's
            // barriers: wait (bounded) for the last use of every stage and of every dequantised slot.
            for (int i = max(it - S, 0); i < it; ++i) {
                mbar_wait_bounded(full_bar(i % S), (uint32_t)(i / S) & 1, nullptr, 200000000ull);
                if (ok) mbar_wait_cluster(empty_bar(i % S), (uint32_t)(i / S) & 1, abort_flag);
            }
            for (int i = max(it - 2, 0); i < it && ok; ++i)
                for (int h = 0; h < 2; ++h)
                    mbar_wait_cluster(a_empty(2 * (i & 1) + h), (uint32_t)(i >> 1) & 1, abort_flag);
        } else if (warp == 1 && lane == 0 && rank == 0) {
            // -------------------------------------------------------- MMA issuer (for both CTAs)
            const uint32_t idesc = idesc_f16_f32(256, p.tn);
            pdl_wait();
            int it = 0;
            bool ok = true;
            for (int u = cluster; u < p.units && ok; u += n_clusters) {
                const FgUnit w = fg_unit(p, u);
                for (int g = w.g0; g < w.g1 && ok; ++g, ++it) {
                    const int s = it % S, b = it & 1;
                    const uint32_t ph = (uint32_t)(it >> 1) & 1;
                    if (!mbar_wait_cluster(d_empty(b), ph ^ 1, abort_flag)) { fail(); ok = false; break; }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int a = 2 * b + h;
                        if (!mbar_wait_cluster(a_full(a), ph, abort_flag)) { fail(); ok = false; break; }
                        tc_fence_after();
                        const uint64_t bd = sw128_kmajor_desc(x_addr(s) + h * (xbytes / 2));
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_f16_ts_pair(tmem + b * NMAX, tmem + ACOL + a * 32 + j * 8, bd + 2 * j, idesc, (h | j) != 0);
                        tc_commit_pair(a_empty(a));
                    }
                    if (!ok) break;
                    tc_commit_pair(empty_bar(s));
                    tc_commit_pair(d_full(b));
                }
            }
            // on an abort nobody else waits for what was issued: the pair's TMEM is freed after it
            if (!ok && it > 0)
                mbar_wait_cluster(d_full((it - 1) & 1), (uint32_t)((it - 1) >> 1) & 1, nullptr, 200000000ull);
        }
    } else if (warp < 12) {
        if (SETREGS) regs_dec<FG_REGS_DEQ>();
        // ------------------------------------------------------------ dequantisation
        const int h = (warp - 4) >> 2, q = warp & 3;
        const int r = q * 32 + lane;  // row of the CTA's 128 = TMEM lane
        const uint32_t sw = (uint32_t)(r >> 1) & 3;  // 64-byte TMA swizzle
        const uint32_t c0 = (uint32_t)r * 64 + (((2 * h) ^ sw) << 4), c1 = (uint32_t)r * 64 + (((2 * h + 1) ^ sw) << 4);
        const uint8_t* zbase = GATED && lane >= 16 ? p.z1 : p.z0;
        const uint32_t remote = map_shared(a_full(h), 0);  // slot h, then 2 + h
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + ACOL + (uint32_t)h * 32;
        pdl_wait();  // no bounded wait runs beside the preceding kernel
        bool ok = true;
        int it = 0;
        for (int u = cluster; u < p.units; u += n_clusters) {
            const FgUnit w = fg_unit(p, u);
            const int n = GATED ? w.nt * 128 + (int)rank * 64 + 16 * q + (lane & 15) : w.nt * 256 + (int)rank * 128 + r;
            const bool nv = n < p.N;
            const uint8_t* zrow = zbase + (int64_t)(nv ? n : 0) * p.G;
            uint32_t z4 = nv ? fg_zeros4(zrow, w.g0, p.G, p.vec) : 0;
            uint32_t z4n = 0;
            for (int g = w.g0; g < w.g1; ++g, ++it) {
                const int s = it % S, b = it & 1;
                // the next four groups' zero points are fetched while these four are used
                if ((g & 3) == 0 && g > w.g0) z4 = z4n;
                if (((g & 3) == 0 || g == w.g0) && nv && (g & ~3) + 4 < p.G) z4n = fg_zeros4(zrow, (g & ~3) + 4, p.G, p.vec);
                const uint32_t z = (z4 >> (8 * (g & 3))) & 0xFFu;
                // q - z = (1024 + q) - (1024 + z) from a low nibble, (1024 + 16 q) / 16 - (64 + z) from a
                // high one: exact
                const uint32_t zl = (0x6400u + z) * 0x10001u, zh = (0xD400u | (z << 4)) * 0x10001u;
                if (ok && !mbar_wait_bounded(full_bar(s), (uint32_t)(it / S) & 1, abort_flag)) { fail(); ok = false; }
                if (ok && !mbar_wait_cluster(a_empty(2 * b + h), ((uint32_t)(it >> 1) & 1) ^ 1, abort_flag)) { fail(); ok = false; }
                if (!ok) continue;
                const uint4 wa = *reinterpret_cast<const uint4*>(smem + p_off(s) + c0);
                const uint4 wb = *reinterpret_cast<const uint4*>(smem + p_off(s) + c1);
                const uint32_t words[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
                uint32_t o[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint32_t wd = words[c], w8 = wd >> 8;
                    const uint32_t lo0 = hsub2_u32(lop3_and_or(wd, 0x000F000Fu, 0x64006400u), zl);              // k0, k4
                    const uint32_t hi0 = hfma2_u32(lop3_and_or(wd, 0x00F000F0u, 0x64006400u), 0x2C002C00u, zh);  // k1, k5
                    const uint32_t lo1 = hsub2_u32(lop3_and_or(w8, 0x000F000Fu, 0x64006400u), zl);              // k2, k6
                    const uint32_t hi1 = hfma2_u32(lop3_and_or(w8, 0x00F000F0u, 0x64006400u), 0x2C002C00u, zh);  // k3, k7
                    o[4 * c + 0] = __byte_perm(lo0, hi0, 0x5410);  // k0, k1
                    o[4 * c + 1] = __byte_perm(lo1, hi1, 0x5410);  // k2, k3
                    o[4 * c + 2] = __byte_perm(lo0, hi0, 0x7632);  // k4, k5
                    o[4 * c + 3] = __byte_perm(lo1, hi1, 0x7632);  // k6, k7
                }
                tmem_st_32x32b_x32(taddr + (uint32_t)b * 64, o);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(remote + 16u * b);
            }
        }
    } else {
        if (SETREGS) regs_inc<FG_REGS_FOLD>();
        // ------------------------------------------------------------ fold and epilogue
        const int f = (warp - 12) >> 2, q = warp & 3;
        const int r = q * 32 + lane;
        const int ncol = p.tn / 2;
        const bool upper = lane >= 16;
        const unsigned short* sbase_row = GATED && upper ? p.s1 : p.s0;
        const uint32_t remote = map_shared(d_empty(0), 0);
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(f * ncol);
        pdl_wait();  // the outputs may be read, the residual written, by the preceding kernel
        bool ok = true;
        int it = 0;
        for (int u = cluster; u < p.units; u += n_clusters) {
            const FgUnit w = fg_unit(p, u);
            const int n = GATED ? w.nt * 128 + (int)rank * 64 + 16 * q + (lane & 15) : w.nt * 256 + (int)rank * 128 + r;
            const bool nv = n < p.N;
            const unsigned short* srow = sbase_row + (int64_t)(nv ? n : 0) * p.G;
            uint64_t s4 = nv ? fg_scales4(srow, w.g0, p.G, p.vec) : 0, s4n = 0;
            uint64_t acc[NACC / 2];
#pragma unroll
            for (int i = 0; i < NACC / 2; ++i) acc[i] = 0;
            for (int g = w.g0; g < w.g1; ++g, ++it) {
                const int b = it & 1;
                if ((g & 3) == 0 && g > w.g0) s4 = s4n;
                if (((g & 3) == 0 || g == w.g0) && nv && (g & ~3) + 4 < p.G) s4n = fg_scales4(srow, (g & ~3) + 4, p.G, p.vec);
                const float sc = __half2float(__ushort_as_half((unsigned short)(s4 >> (16 * (g & 3)))));
                const uint64_t sc2 = pack_f32x2(__float_as_uint(sc), __float_as_uint(sc));
                if (ok && !mbar_wait_cluster(d_full(b), (uint32_t)(it >> 1) & 1, abort_flag)) { fail(); ok = false; }
                if (!ok) continue;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < NACC; c += 16) {
                    if (c < ncol) {
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(taddr + (uint32_t)(b * NMAX + c), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i += 2) fma2(acc[(c + i) / 2], pack_f32x2(v[i], v[i + 1]), sc2);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(remote + 8u * b);
            }
            if (!ok) continue;
            const int m0 = w.m0 + f * ncol;
            if (p.P) {
                float* P = p.P + ((int64_t)w.slice * (GATED ? 2 : 1) + (GATED && upper ? 1 : 0)) * p.M * p.N;
#pragma unroll
                for (int c = 0; c < NACC; c += 2) {
                    float v[2];
                    unpack_f32x2(acc[c / 2], v[0], v[1]);
                    if (c < ncol && nv && m0 + c < p.M) P[(int64_t)(m0 + c) * p.N + n] = v[0];
                    if (c < ncol && nv && m0 + c + 1 < p.M) P[(int64_t)(m0 + c + 1) * p.N + n] = v[1];
                }
            } else {
                auto epilogue = [&](auto act) {
                    if constexpr (GATED) fg_epilogue_gated<decltype(act)::value, NACC>(p, acc, ncol, m0, n, upper);
                    else fg_epilogue_plain<decltype(act)::value, NACC>(p, acc, ncol, m0, n);
                    return cudaSuccess;
                };
                dispatch_act(p.act, epilogue);
            }
        }
    }
    __syncthreads();
    cluster_sync();  // nothing of the pair's products or arrivals is outstanding in either CTA
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TCOLS);
    }
}

// The K slices' partial sums [slice][layer][M][N] added in slice order, then the epilogue.  No
// slices (an empty K): the epilogue of zeros.  Launched as a programmatic dependent of the kernel
// that writes the partials.
template <int ACT, bool GATED>
__global__ void __launch_bounds__(256) ffn_reduce_kernel(const float* P, int slices, int64_t mn, int N, const __half* bias,
                                                         const __half* residual, __half* Y, __half* Z, __half* U) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int L = GATED ? 2 : 1;
    for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; e < mn; e += (int64_t)gridDim.x * 1024) {
        float4 a[L];
#pragma unroll
        for (int l = 0; l < L; ++l) a[l] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s = 0; s < slices; ++s) {
#pragma unroll
            for (int l = 0; l < L; ++l) {
                const float4 b = *reinterpret_cast<const float4*>(P + ((int64_t)s * L + l) * mn + e);
                a[l].x += b.x; a[l].y += b.y; a[l].z += b.z; a[l].w += b.w;
            }
        }
        float z[4] = {a[0].x, a[0].y, a[0].z, a[0].w}, y[4];
        if (!GATED && bias) {
            const int n = (int)(e % N);
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] += __half2float(bias[n + i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = act_fwd<ACT>(z[i]);
        if constexpr (GATED) {
            const float u[4] = {a[1].x, a[1].y, a[1].z, a[1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] *= u[i];
            if (U) *reinterpret_cast<uint2*>(U + e) = make_uint2(pack_half2(u[0], u[1]), pack_half2(u[2], u[3]));
        }
        if (residual) {
            const uint2 r = *reinterpret_cast<const uint2*>(residual + e);
            const float2 r0 = __half22float2(*reinterpret_cast<const __half2*>(&r.x));
            const float2 r1 = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
            y[0] += r0.x; y[1] += r0.y; y[2] += r1.x; y[3] += r1.y;
        }
        *reinterpret_cast<uint2*>(Y + e) = make_uint2(pack_half2(y[0], y[1]), pack_half2(y[2], y[3]));
        if (Z) *reinterpret_cast<uint2*>(Z + e) = make_uint2(pack_half2(z[0], z[1]), pack_half2(z[2], z[3]));
    }
}

const __half* hp(const uint16_t* p) { return reinterpret_cast<const __half*>(p); }
__half* hp(uint16_t* p) { return reinterpret_cast<__half*>(p); }

struct FgPlan {
    int tn, ks, stages, m_tiles, n_tiles, units;
    bool wide;  // the 192-column instantiation
    uint32_t smem;
};

FgPlan fg_plan(int64_t M, int64_t N, int64_t K, bool gated) {
    const int64_t pairs = std::max(1, device_sm_count() / 2), G = K / 128;
    const int64_t rows = gated ? 128 : 256;
    const int64_t n_tiles = (N + rows - 1) / rows;
    FgPlan best = {};
    double best_t = -1.0;
    for (int tn = 32; tn <= 192; tn += 32) {
        if (tn > 32 && tn >= M + 32) break;
        const int64_t m_tiles = (M + tn - 1) / tn;
        const int64_t tiles = m_tiles * n_tiles;
        for (int ks = 1; ks <= 16 && ks <= G; ++ks) {
            if (ks > 1 && (tiles * (ks - 1) >= pairs || G / ks < 4)) break;
            const int64_t units = tiles * ks;
            const int64_t waves = (units + pairs - 1) / pairs;
            // cycles per group: the products (4 tn) or the dequantising warps' issue rate; per unit: filling
            // and the epilogue; a second launch and its traffic when K is cut
            const double group = std::max(4.0 * tn, 380.0);
            double t = (double)waves * ((double)((G + ks - 1) / ks) * group + 1500.0 + 8.0 * tn);
            if (ks > 1) t += 4000.0 + (double)ks * (double)M * (double)N * (gated ? 2 : 1) * 8.0 / 3000.0;
            if (best_t < 0.0 || t < best_t) {
                best_t = t;
                best.tn = tn;
                best.ks = ks;
                best.m_tiles = (int)m_tiles;
                best.n_tiles = (int)n_tiles;
                best.units = (int)units;
            }
        }
    }
    best.wide = best.tn > 64;
    const uint32_t stage = (uint32_t)best.tn * 128u + FG_P_BYTES;
    best.stages = (int)std::min<uint32_t>((FG_SMEM - 1024 - 512) / stage, FG_MAXS);
    best.smem = stage * (uint32_t)best.stages + 512 + 1024;
    return best;
}

template <bool GATED, int NMAX>
cudaError_t fg_setup() {
    static std::once_flag once[64];
    static cudaError_t err[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&]() {
        err[dev] = cudaFuncSetAttribute(ffn_gemm_kernel<GATED, NMAX>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FG_SMEM);
        // the register split must add up to the launch's allotment, or setmaxnreg.inc would wait for good
        cudaFuncAttributes a;
        if (err[dev] == cudaSuccess) err[dev] = cudaFuncGetAttributes(&a, ffn_gemm_kernel<GATED, NMAX>);
        if (err[dev] == cudaSuccess && NMAX > 64 && a.numRegs != FG_REGS_LAUNCH) err[dev] = cudaErrorInvalidConfiguration;
    });
    return err[dev];
}

template <bool GATED, int NMAX>
cudaError_t fg_launch(const CUtensorMap& tx, const CUtensorMap& t0, const CUtensorMap& t1, const FgArgs& args,
                      const FgPlan& pl, cudaStream_t stream) {
    const cudaError_t e = fg_setup<GATED, NMAX>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * std::min(pl.units, std::max(1, device_sm_count() / 2))), 1, 1);
    cfg.blockDim = dim3(FG_THREADS, 1, 1);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = args.early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<GATED, NMAX>, tx, t0, t1, args);
}

}  // namespace

cudaError_t launch_ffn_reduce(const float* P, int slices, int64_t M, int64_t N, bool gated, const W4Epilogue& ep,
                              cudaStream_t stream) {
    const int64_t mn = M * N;
    const int64_t want = (mn / 4 + 255) / 256, cap = (int64_t)device_sm_count() * 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min(want, cap), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = slices > 0 ? 1 : 0;
    return dispatch_act(ep.activation, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        if (gated)
            return cudaLaunchKernelEx(&cfg, ffn_reduce_kernel<ACT, true>, P, slices, mn, (int)N, hp(ep.bias),
                                      hp(ep.residual), hp(ep.Y), hp(ep.Z), hp(ep.U));
        return cudaLaunchKernelEx(&cfg, ffn_reduce_kernel<ACT, false>, P, slices, mn, (int)N, hp(ep.bias), hp(ep.residual),
                                  hp(ep.Y), hp(ep.Z), hp(ep.U));
    });
}

size_t ffn_gemm_workspace(int64_t M, int64_t N, int64_t K, bool gated) {
    const FgPlan pl = fg_plan(M, N, K, gated);
    return pl.ks > 1 ? (size_t)pl.ks * (size_t)M * (size_t)N * (gated ? 8 : 4) : 0;
}

cudaError_t launch_ffn_gemm(const uint16_t* X, int64_t M, int64_t N, int64_t K, const W4Layer& w, const W4Layer* w2,
                            const W4Epilogue& ep, void* ws, bool weights_static, int* status, cudaStream_t stream) {
    const bool gated = w2 != nullptr;
    const FgPlan pl = fg_plan(M, N, K, gated);
    if (pl.ks > 1 && !ws) return cudaErrorInvalidValue;
    CUtensorMap tx, t0, t1;
    if (!make_tensor_map_2d(&tx, X, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, (uint64_t)K, (uint64_t)M, 64, (uint32_t)(pl.tn / 2),
                            CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    const uint32_t box = gated ? 16 : 128;
    if (!make_tensor_map_2d(&t0, w.packed, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, (uint64_t)(K / 8), (uint64_t)N, 16, box,
                            CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    t1 = t0;
    if (gated && !make_tensor_map_2d(&t1, w2->packed, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, (uint64_t)(K / 8), (uint64_t)N, 16,
                                     box, CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    const int64_t G = K / 128;
    auto vec_ok = [&](const W4Layer& l) {  // 4-group vectors at multiples of 4 groups of every row
        return G % 4 == 0 && (reinterpret_cast<uintptr_t>(l.scales) & 7) == 0 && (reinterpret_cast<uintptr_t>(l.zeros) & 3) == 0;
    };
    FgArgs a = {};
    a.s0 = w.scales;
    a.z0 = w.zeros;
    a.s1 = gated ? w2->scales : w.scales;
    a.z1 = gated ? w2->zeros : w.zeros;
    a.bias = hp(ep.bias);
    a.residual = hp(ep.residual);
    a.Y = hp(ep.Y);
    a.Z = hp(ep.Z);
    a.U = hp(ep.U);
    a.P = pl.ks > 1 ? static_cast<float*>(ws) : nullptr;
    a.act = ep.activation;
    a.M = (int)M;
    a.N = (int)N;
    a.G = (int)G;
    a.tn = pl.tn;
    a.m_tiles = pl.m_tiles;
    a.n_tiles = pl.n_tiles;
    // m-tiles whose X stays in L2 (about 48 MB) run down the weights together
    a.gm = (int)std::max<int64_t>(1, std::min<int64_t>(pl.m_tiles, (48ll << 20) / ((int64_t)pl.tn * K * 2)));
    a.ks = pl.ks;
    a.units = pl.units;
    a.stages = pl.stages;
    a.vec = vec_ok(w) && (!gated || vec_ok(*w2)) ? 1 : 0;
    a.early = weights_static ? 1 : 0;
    a.status = status;
    cudaError_t e;
    if (gated) e = pl.wide ? fg_launch<true, 192>(tx, t0, t1, a, pl, stream) : fg_launch<true, 64>(tx, t0, t1, a, pl, stream);
    else e = pl.wide ? fg_launch<false, 192>(tx, t0, t1, a, pl, stream) : fg_launch<false, 64>(tx, t0, t1, a, pl, stream);
    if (e != cudaSuccess || pl.ks == 1) return e;
    return launch_ffn_reduce(a.P, pl.ks, M, N, gated, ep, stream);
}

}  // namespace w4
