// Forward products of the feed-forward operators on the tensor cores (w4_gemm_fused, w4_gemm_gated).
//
//   D[n, m] = sum_g s[n, g] * sum_{k in g} (q[n, k] - z[n, g]) X[m, k]
//
// The codes' differences q - z are whole numbers of at most 15, exact in fp16, so the tensor cores sum
// exact products in fp32 and the scale multiplies each group's sum in fp32: no weight is ever rounded
// (a weight (q - z) s rounded to fp16 costs 1.5e-4 of the result in 2-norm, as much again as the
// output's own rounding; in the gated product it enters twice).
//
// The weights are the A operand (256 or 128 rows), dequantised once per tile; X is the B operand (`tn`
// rows).  Why this way round: a thread owns one weight row, so a group has one scale per thread, and small
// batches cost products of 32 columns, not 128.  Two instantiations:
//   NMAX 256  large batches: two CTAs share a tile of 256 weight rows by up to 256 rows of X, each with half
//             of both in its shared memory (cta_group::2).  The weights go through shared memory as fp16:
//             144 KB a group and CTA pass its port (X in and out 64, codes in and out 16, weights in and
//             out 64) beside 1024 cycles of products, so port and tensor cores are about equally busy.
//             Weights in tensor memory would spare the port 64 KB but leave columns for 192 rows of X only,
//             whose group took 1152 cycles where 256 take 1258: slower by a fifth.
//   NMAX 64   small batches: one CTA, 128 weight rows by up to 64 rows of X, the weights in tensor memory,
//             two groups a step.  Bound by the dequantisation (a step's codes come in, are converted and
//             stored to tensor memory; two steps in flight): 780 cycles a group, in 340 of which the ALU pipe
//             converts, where HBM would allow 370; 48 us at M = 32, K = 28672, N = 8192.
// At M = 2048, K = 4096, N = 11008, in a short burst: gated 289 us (1280 TFLOP/s), plain 145 us; called without
// a pause, where the power limit holds the clock down, gated 347 us (1065 TFLOP/s).
//
//   warp 0       TMA producer of its CTA: X (boxes of 64 k) and the packed rows of a step
//   warp 1       first CTA: issues the tcgen05.mma (N = tn, K = 16) and one commit a step
//   warp 2       TMEM allocation
//   next 4 DW    dequantise: a thread takes a row's 128 codes of a group
//   last 8       fold: four take columns 0 .. tn/2 - 1, four the rest: read a group's sums from TMEM,
//                acc += s * sum in registers; after the last group the epilogue
// The group sums rotate through NB TMEM buffers, the dequantised steps through AG, so a step's
// products, the next one's dequantisation and the last one's fold overlap.  One barrier per ring
// stage (committed once by the tensor cores) tells the producer that the stage, the dequantising warps
// that the dequantised step is free, and the fold warps that the sums are there.
//
// Epilogue: the fold warps pass 16 columns at a time through shared memory as fp32 [m][n], two buffers of
// them, so that the output, residual and pre-activation rows are read and written as whole 256-byte rows
// (from the accumulators' own layout, thread = n, a warp's stores were 64-byte pieces: 25 cycles each).
// Gated: the 32 lanes of a warp hold 16 gate rows and the 16 up rows of the same n, so both factors of
// an output lie in one CTA's rows.
//
// Few tiles: K is cut into slices of whole groups, their fp32 sums go to the workspace [slice][layer]
// [M][N] and ffn_reduce_kernel adds them in slice order and runs the epilogue: deterministic.
// Small batches with a nearly empty last wave: equal shares of all tiles' steps instead (FgShares).
//
// Every mbarrier wait is bounded; on timeout the kernel records W4_ERR_DEVICE_TIMEOUT and drains.
#include <algorithm>
#include <mutex>

#include "activation.cuh"
#include "ffn_common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace w4 {

namespace {

constexpr int FG_MAXS = 16;                        // ring stages at most
constexpr uint32_t FG_P_BYTES = 128 * 64;          // packed codes of one group: 128 rows x 64 bytes
constexpr uint32_t FG_SMEM = 227 * 1024;
constexpr uint32_t FG_EPI = 32 * 128 * 4;          // a fold warpgroup's 32 rows of 128 fp32

// NMAX columns at most.
// 256 (large batches): the dequantised groups lie in shared memory (K-major, 128-byte swizzle).
// 64 (small batches): in tensor memory; a step is two groups, because a group's products are shorter
// than the waits, round trips and the issue of a step, and because TMA moves a 128-byte row in the
// time of a 64-byte one.
// Every thread launches with kRegs registers; the fold warps take what the others give up (in
// warpgroup shares: 24 + 80 + 2 x 200 = 504 of 4 x 128, and 24 + 2 x 80 + 2 x 144 = 472 of 5 x 96).
// No kernel may spill: with 28 KB of L1 left a reload is an L2 round trip in the group loop.
template <int NMAX>
struct FgCfg {
    static constexpr bool kWide = NMAX > 64;
    static constexpr int kCtas = kWide ? 2 : 1;     // CTAs that share a tile
    static constexpr int kGPS = kWide ? 1 : 2;      // groups per step
    static constexpr int kDW = kWide ? 1 : 2;       // dequantising warpgroups, taking the steps in turn
    static constexpr int kNB = 2;                   // steps whose sums TMEM holds
    static constexpr int kAG = 2;                   // dequantised steps
    static constexpr int kThreads = 128 * (1 + kDW + 2);
    static constexpr uint32_t kACol = kNB * kGPS * NMAX;  // 64: first TMEM column of the dequantised groups (64 each)
    static constexpr uint32_t kWBytes = kWide ? 128 * 128 * 2 : 0;  // 256: shared memory of one
    static constexpr int kRegs = kWide ? 128 : 96;
    static constexpr int kRegsMisc = 24, kRegsDeq = 80, kRegsFold = kWide ? 200 : 144;
    static_assert(kRegsMisc + kDW * kRegsDeq + 2 * kRegsFold <= (3 + kDW) * kRegs, "register shares");
    static_assert(kNB * kGPS * NMAX + (kWide ? 0 : 64 * kAG * kGPS) <= 512, "TMEM");
};

// Small batches whose tiles leave a last wave nearly empty: the steps of all tiles laid end to end and
// cut into equal shares, one per CTA.  A tile that lies in one share is finished there; the parts of
// the others go to the workspace, in the order of their steps, and ffn_reduce_kernel adds them.
struct FgShares {
    int ctas;   // shares; 0: none
    int steps;  // of a tile
    int total;  // of all tiles; total * ctas < 2^29
    __host__ __device__ int start(int c) const { return c * total / ctas; }
    __host__ __device__ int owner(int step) const { return ((step + 1) * ctas - 1) / total; }
    __host__ __device__ int first(int tile) const { return owner(tile * steps); }
    __host__ __device__ int parts(int tile) const { return owner(tile * steps + steps - 1) - first(tile) + 1; }
};

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
    FfnRaster raster;  // ks: slices of K
    FgShares shares;
    int units;
    int stages;
    int vec;          // metadata rows allow 4-group vector loads
    int early;        // weights may be read before the preceding kernel has finished
    int* status;
};

// Arrival on the issuing CTA's barrier.
template <int CTAS>
__device__ __forceinline__ void fg_arrive(uint32_t bar) {
    if constexpr (CTAS == 2) mbar_arrive_cluster(bar);
    else mbar_arrive(bar);
}

struct FgUnit {
    int m0, nt, slice, g0, g1;
};

// A share's tiles are its CTA's units in turn (u = share + i * ctas); those past its end are empty.
template <bool SHARES>
__device__ __forceinline__ FgUnit fg_unit(const FgArgs& p, int u) {
    FgUnit r;
    if (SHARES && p.shares.ctas) {
        const FgShares& h = p.shares;
        const int c = u % h.ctas, begin = h.start(c), end = h.start(c + 1);
        r.nt = begin / h.steps + u / h.ctas;
        r.m0 = 0;
        r.slice = c - h.first(r.nt);
        r.g0 = 2 * max(begin - r.nt * h.steps, 0);
        r.g1 = max(min(2 * (end - r.nt * h.steps), p.G), r.g0);
        return r;
    }
    const FfnUnit t = ffn_unit(p.raster, u);
    r.slice = t.slice;
    r.nt = t.nt;
    r.m0 = t.mt * p.tn;
    r.g0 = t.slice * p.G / p.raster.ks;  // G < 2^24, ks <= 16
    r.g1 = (t.slice + 1) * p.G / p.raster.ks;
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

// 16 columns' sums, ordered before their use by the wait.
__device__ __forceinline__ void fg_tie(uint32_t (&v)[16]) {
    asm volatile("" : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                      "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]));
}

// Four neighbouring outputs of a row (element offset o) from their sums.
template <int ACT, bool GATED>
__device__ __forceinline__ void fg_finish(const FgArgs& p, const float4& s0, const float4& s1, const uint2& bias, const uint2& res,
                                          int64_t o) {
    F2 z[2] = {f2(s0.x, s0.y), f2(s0.z, s0.w)}, y[2];
    float f[4];
    if constexpr (GATED) {
        const F2 u[2] = {f2(s1.x, s1.y), f2(s1.z, s1.w)};
        y[0] = mul2(act_fwd2<ACT>(z[0]), u[0]);
        y[1] = mul2(act_fwd2<ACT>(z[1]), u[1]);
        const float uf[4] = {s1.x, s1.y, s1.z, s1.w};
        if (p.U) *reinterpret_cast<uint2*>(p.U + o) = half4(uf);
    } else {
        if (p.bias) {
            float4_of(bias, f);
            z[0] = add2(z[0], f2(f[0], f[1]));
            z[1] = add2(z[1], f2(f[2], f[3]));
        }
        y[0] = act_fwd2<ACT>(z[0]);
        y[1] = act_fwd2<ACT>(z[1]);
        if (p.residual) {
            float4_of(res, f);
            y[0] = add2(y[0], f2(f[0], f[1]));
            y[1] = add2(y[1], f2(f[2], f[3]));
        }
    }
    split(y[0], f[0], f[1]);
    split(y[1], f[2], f[3]);
    *reinterpret_cast<uint2*>(p.Y + o) = half4(f);
    if (p.Z) {
        split(z[0], f[0], f[1]);
        split(z[1], f[2], f[3]);
        *reinterpret_cast<uint2*>(p.Z + o) = half4(f);
    }
}

// Columns 16 i ... 16 i + 15 of the accumulators (i not a constant) to 16 staged rows.
template <int NACC, int I = 0>
__device__ __forceinline__ void fg_stage(const F2 (&acc)[NACC / 2], int i, float* st) {
    if constexpr (16 * I < NACC) {
        if (i == I) {
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                float a, b;
                split(acc[(16 * I + j) / 2], a, b);
                st[j * 128] = a;
                st[(j + 1) * 128] = b;
            }
        } else {
            fg_stage<NACC, I + 1>(acc, i, st);
        }
    }
}

// One tile's outputs.  acc: this thread's weight row (r of the CTA's 128) by ncol X rows from m0; nb:
// the CTA's first output column; st_off: the warpgroup's staging rows, two buffers of 16, so that the
// next 16 columns are staged while these are finished.  Staged rows are [128 n] or, gated, [64 gate n |
// 64 up n with bit 4 flipped] (conflict-free stores).
template <int ACT, bool GATED, int NACC>
__device__ __forceinline__ void fg_epilogue(const FgArgs& p, const F2 (&acc)[NACC / 2], int ncol, int m0, int nb,
                                            unsigned char* smem, uint32_t st_off, int r, int bar) {
    // opaque to the compiler: what follows from it is computed here, once a tile, and not kept in
    // registers (or spilled) across the group loop
    asm volatile("" : "+r"(r), "+r"(st_off));
    float* st = reinterpret_cast<float*>(smem + st_off);
    const int w = r >> 5, lane = r & 31;
    const int col = GATED ? ((r & 16) ? 64 : 0) + (((r >> 5) * 16 + (r & 15)) ^ (r & 16)) : r;
    const int n4 = GATED ? 4 * (lane & 15) : 4 * lane;  // this thread's four columns of the rows it finishes
    const int n = nb + n4;
    uint2 bias = make_uint2(0u, 0u);
    if (!GATED && p.bias && n < p.N) bias = *reinterpret_cast<const uint2*>(p.bias + n);
    constexpr int RPW = GATED ? 2 : 1, RT = 4 / RPW;  // rows a warp finishes at once, rows of a thread
    const int row0 = RPW * w + (GATED ? lane >> 4 : 0);
    const int rows = n < p.N ? min(ncol, p.M - m0) : 0;  // of the tile
    fg_stage<NACC>(acc, 0, st + col);
    wg_barrier(bar);
#pragma unroll 1
    for (int i = 0; 16 * i < ncol; ++i) {
        const float* sr = st + (i & 1) * 2048 + row0 * 128 + n4;
        const int left = rows - 16 * i - row0;  // of this thread's rows 0, 4 RPW, ... those below it exist
        int64_t o = (int64_t)(m0 + 16 * i + row0) * p.N + n;
        const int64_t step = (int64_t)(4 * RPW) * p.N;
        if (16 * (i + 1) < ncol) fg_stage<NACC>(acc, i + 1, st + ((i + 1) & 1) * 2048 + col);
#pragma unroll
        for (int k = 0; k < RT; k += 2) {  // two rows at a time: more do not fit beside the accumulators
            uint2 res[2];
            float4 s0[2], s1[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (!GATED && p.residual && 4 * RPW * (k + j) < left)
                    res[j] = *reinterpret_cast<const uint2*>(p.residual + o + j * step);
                s0[j] = *reinterpret_cast<const float4*>(sr + 4 * RPW * (k + j) * 128);
                if (GATED) s1[j] = *reinterpret_cast<const float4*>(sr + 4 * RPW * (k + j) * 128 + 64 + (n4 ^ 16) - n4);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (4 * RPW * (k + j) < left) fg_finish<ACT, GATED>(p, s0[j], s1[j], bias, res[j], o);
                o += step;
            }
        }
        wg_barrier(bar);
    }
}

template <bool GATED, int NMAX>
__global__ void __cluster_dims__(FgCfg<NMAX>::kCtas, 1, 1) __launch_bounds__(FgCfg<NMAX>::kThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW0,
                    const __grid_constant__ CUtensorMap tmW1, const FgArgs p) {
    using C = FgCfg<NMAX>;
    constexpr int NACC = NMAX / 2;            // columns per fold thread
    constexpr int NB = C::kNB, AG = C::kAG, GPS = C::kGPS, DW = C::kDW, CTAS = C::kCtas;
    constexpr int TROWS = 128 * CTAS;         // weight rows of a tile
    constexpr int TN = GATED ? TROWS / 2 : TROWS;  // outputs n of a tile; TN / CTAS in each CTA
    constexpr int FOLD_WARP = 4 + 4 * C::kDW;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = smem_align1024(smem_raw);
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform: the issuing loops stay in uniform registers
    const uint32_t rank = CTAS == 2 ? cluster_ctarank() : 0;
    const int S = p.stages;
    const int xrows = p.tn / CTAS;                  // X rows in this CTA
    const uint32_t xbytes = (uint32_t)xrows * 256u;  // 128 k x 2 bytes each
    // a stage: X of the step's groups, then their packed codes, rows of 64 GPS bytes
    const uint32_t p_off = GPS * xbytes, stage_bytes = GPS * (xbytes + FG_P_BYTES);
    const uint32_t w0 = (uint32_t)S * stage_bytes;    // dequantised groups, the epilogue's staging rows, the barriers
    const uint32_t epi0 = w0 + AG * C::kWBytes;
    const uint32_t bar0 = sbase + epi0 + 2 * FG_EPI;
    auto full_bar = [&](int s) { return bar0 + 8 * s; };
    auto done_bar = [&](int s) { return bar0 + 8 * (FG_MAXS + s); };
    auto a_full = [&](int i) { return bar0 + 8 * (2 * FG_MAXS + i); };
    auto d_empty = [&](int i) { return bar0 + 8 * (2 * FG_MAXS + 4 + i); };
    unsigned char* tail = smem + epi0 + 2 * FG_EPI + 8 * (2 * FG_MAXS + 8);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 4);

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(done_bar(s), 1);
        }
        for (int i = 0; i < AG; ++i) mbar_init(a_full(i), 4 * CTAS);  // a warpgroup of each CTA
        for (int i = 0; i < NB; ++i) mbar_init(d_empty(i), 8 * CTAS);  // eight fold warps of each CTA
        *abort_flag = 0;
        fence_mbarrier_init();
        prefetch_tmap(&tmX);
        prefetch_tmap(&tmW0);
        if (GATED) prefetch_tmap(&tmW1);
    }
    if (warp == 2) {
        if constexpr (CTAS == 2) {
            tmem_alloc_pair(smem_u32(tmem_slot), 512);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_slot), 512);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    pdl_launch_dependents();

    auto fail = [&]() {
        *abort_flag = 1;
        record_status(p.status, W4_ERR_DEVICE_TIMEOUT);
    };
    const int cluster = (int)blockIdx.x / CTAS, n_clusters = (int)gridDim.x / CTAS;

    if (warp < 4) {
        regs_dec<C::kRegsMisc>();
        if (warp == 0) {
            // -------------------------------------------------------- TMA producer (one lane issuing)
            // a step's packed rows (all GPS groups' bytes: past the last group of an odd count too)
            auto load_w = [&](const FgUnit& u, int g, int n_groups, int s) {
                mbar_arrive_expect_tx(full_bar(s), (uint32_t)n_groups * xbytes + GPS * FG_P_BYTES);
                const uint32_t dst = sbase + (uint32_t)s * stage_bytes + p_off;
                if constexpr (GATED) {
                    const int n = u.nt * TN + (int)rank * 64;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        tma_load_2d(dst + q * (2048 * GPS), &tmW0, g * 16, n + 16 * q, full_bar(s));
                        tma_load_2d(dst + q * (2048 * GPS) + 1024 * GPS, &tmW1, g * 16, n + 16 * q, full_bar(s));
                    }
                } else {
                    tma_load_2d(dst, &tmW0, g * 16, u.nt * TN + (int)rank * 128, full_bar(s));
                }
            };
            if (!p.early) pdl_wait();
            int ahead = 0;
            if (p.early) {  // the first ring's weights, before the preceding kernel has finished
                for (int u = cluster; u < p.units && ahead < S; u += n_clusters) {
                    const FgUnit w = fg_unit<!C::kWide>(p, u);
                    for (int g = w.g0; g < w.g1 && ahead < S; g += GPS, ++ahead) {
                        if (elect_one()) load_w(w, g, min(GPS, w.g1 - g), ahead);
                        __syncwarp();
                    }
                }
                pdl_wait();
            }
            int it = 0, s = 0;
            uint32_t ph = 1;
            bool ok = true;
            for (int u = cluster; u < p.units && ok; u += n_clusters) {
                const FgUnit w = fg_unit<!C::kWide>(p, u);
                const int mx = w.m0 + (int)rank * xrows;
                for (int g = w.g0; g < w.g1; g += GPS, ++it) {
                    if (it >= ahead && !mbar_wait_long(done_bar(s), ph, abort_flag)) { fail(); ok = false; break; }
                    if (elect_one()) {
                        const int n_groups = min(GPS, w.g1 - g);
                        if (it >= ahead) load_w(w, g, n_groups, s);
#pragma unroll
                        for (int j = 0; j < GPS; ++j) {
                            if (j >= n_groups) break;
                            const uint32_t xs = sbase + (uint32_t)s * stage_bytes + (uint32_t)j * xbytes;
                            tma_load_2d(xs, &tmX, (g + j) * 128, mx, full_bar(s));
                            tma_load_2d(xs + xbytes / 2, &tmX, (g + j) * 128 + 64, mx, full_bar(s));
                        }
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
            // -------------------------------------------------------- MMA issuer (for both CTAs)
            const uint32_t idesc = idesc_f16_f32(TROWS, p.tn);
            pdl_wait();
            int it = 0, s = 0;
            bool ok = true;
            for (int u = cluster; u < p.units && ok; u += n_clusters) {
                const FgUnit w = fg_unit<!C::kWide>(p, u);
                for (int g = w.g0; g < w.g1; g += GPS, ++it) {
                    const int b = it % NB, a = it % AG;
                    // the fold of the step NB ago usually comes last: it is waited for last
                    if (!mbar_wait_long(a_full(a), (uint32_t)(it / AG) & 1, abort_flag) ||
                        !mbar_wait_long(d_empty(b), ((uint32_t)(it / NB) & 1) ^ 1, abort_flag)) {
                        fail();
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t half = (uint64_t)(xbytes / 2) >> 4;  // the second 64 k
#pragma unroll
                        for (int i = 0; i < GPS; ++i) {
                            if (i > 0 && g + i >= w.g1) break;
                            const uint64_t bd = sw128_kmajor_desc(sbase + (uint32_t)s * stage_bytes + (uint32_t)i * xbytes);
                            const uint64_t ad = sw128_kmajor_desc(sbase + w0 + (uint32_t)a * C::kWBytes);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint64_t bj = bd + (j >> 2) * half + 2 * (j & 3);
                                if constexpr (C::kWide)
                                    mma_f16_ss_pair(tmem + b * NMAX, ad + (j >> 2) * (C::kWBytes / 2 >> 4) + 2 * (j & 3), bj, idesc,
                                                    j != 0);
                                else
                                    mma_f16_ts(tmem + (b * GPS + i) * NMAX, tmem + C::kACol + (a * GPS + i) * 64 + j * 8, bj, idesc,
                                               j != 0);
                            }
                        }
                        if constexpr (CTAS == 2) tc_commit_pair(done_bar(s));
                        else tc_commit(done_bar(s));
                    }
                    __syncwarp();
                    if (++s == S) s = 0;
                }
            }
            // on an abort nobody else waits for what was issued: the TMEM is freed after it
            if (!ok && it > 0) mbar_wait_long(done_bar((it - 1) % S), (uint32_t)((it - 1) / S) & 1, nullptr, 200000000ull);
        }
    } else if (warp < FOLD_WARP) {
        regs_dec<C::kRegsDeq>();
        // ------------------------------------------------------------ dequantisation
        // a warpgroup takes every DW-th step: while one waits (for codes, its slot, its stores), another computes
        const int wg = (warp - 4) >> 2, q = warp & 3;
        const int r = q * 32 + lane;  // row of the CTA's 128 = TMEM lane
        // TMA swizzle of the row's 16-byte pieces: 64-byte rows by bits 1-2 of the row, 128-byte ones by 0-2
        const uint32_t sw = GPS == 1 ? (uint32_t)(r >> 1) & 3 : (uint32_t)r & 7;
        const uint32_t c0 = p_off + (uint32_t)r * (64 * GPS);
        const uint8_t* zbase = GATED && lane >= 16 ? p.z1 : p.z0;
        const uint32_t remote = CTAS == 2 ? map_shared(a_full(0), 0) : a_full(0);
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + C::kACol;
        pdl_wait();  // no bounded wait runs beside the preceding kernel
        bool ok = true;
        int it = 0, s = 0, sa = 0;  // step, its ring stage, the ring stage of step it - AG (S >= AG)
        uint32_t ph = 0, pa = 0;
        for (int u = cluster; u < p.units; u += n_clusters) {
            const FgUnit w = fg_unit<!C::kWide>(p, u);
            const int n = w.nt * TN + (GATED ? (int)rank * 64 + 16 * q + (lane & 15) : (int)rank * 128 + r);
            const bool nv = n < p.N;
            const uint8_t* zrow = zbase + (int64_t)(nv ? n : 0) * p.G;
            const int gf = w.g0 + GPS * ((wg + it) % DW);  // this warpgroup's first group (DW <= 2: wg - it = wg + it)
            uint32_t z4 = nv && gf < w.g1 ? fg_zeros4(zrow, gf, p.G, p.vec) : 0, z4n = 0;
            int zb = gf & ~3;  // z4 holds groups zb ... zb + 3, z4n the next four
            if (nv && zb + 4 < p.G) z4n = fg_zeros4(zrow, zb + 4, p.G, p.vec);
            for (int gs = w.g0; gs < w.g1; gs += GPS, ++it) {
                auto next_stage = [&]() {
                    if (it >= AG && ++sa == S) { sa = 0; pa ^= 1; }
                    if (++s == S) { s = 0; ph ^= 1; }
                };
                if (DW > 1 && it % DW != wg) {
                    next_stage();
                    continue;
                }
                const uint32_t slot = (uint32_t)(it % AG);
                // two of the row's four 16-byte pieces: half h of group j's codes
                auto load = [&](int j, int h, uint32_t (&words)[8]) {
                    const unsigned char* st = smem + (uint32_t)s * stage_bytes + c0;
                    const uint4 a = *reinterpret_cast<const uint4*>(st + (((4 * j + 2 * h) ^ sw) << 4));
                    const uint4 b = *reinterpret_cast<const uint4*>(st + (((4 * j + 2 * h + 1) ^ sw) << 4));
                    words[0] = a.x; words[1] = a.y; words[2] = a.z; words[3] = a.w;
                    words[4] = b.x; words[5] = b.y; words[6] = b.z; words[7] = b.w;
                };
                auto free_slot = [&]() {  // the step that used this slot AG steps ago has been multiplied
                    if (it >= AG && ok && !warp_wait(done_bar(sa), pa, abort_flag)) { fail(); ok = false; }
                };
                auto zero_add = [&](int g) {  // -(1024 + z), -(64 + z)
                    if ((g & ~3) != zb) {  // the next four groups' zero points are fetched while these are used
                        z4 = z4n;
                        zb = g & ~3;
                        if (nv && zb + 4 < p.G) z4n = fg_zeros4(zrow, zb + 4, p.G, p.vec);
                    }
                    const uint32_t z = (z4 >> (8 * (g & 3))) & 0xFFu;
                    return (0xE400u + z) | ((0xD400u | (z << 4)) << 16);
                };
                uint32_t zadd = C::kWide ? zero_add(gs) : 0;  // before the wait: 1 % faster in large tiles, slower in small ones
                if (ok && !warp_wait(full_bar(s), ph, abort_flag)) { fail(); ok = false; }
                uint32_t words[8];
                load(0, 0, words);
                uint32_t next[8];
                if (C::kWide) {
                    load(0, 1, next);
                    free_slot();
                }
#pragma unroll
                for (int j = 0; j < GPS; ++j) {
                    const int g = gs + j;
                    if (j > 0 && g >= w.g1) break;
                    if (!C::kWide) zadd = zero_add(g);
                    // A byte in both halves of a word, the low nibble kept in the lower and the high one in the
                    // upper, under the exponent of 1024: the pair 1024 + q, 1024 + 16 q'.  Then (1024 + q) * 1 - (1024
                    // + z) and (1024 + 16 q') / 16 - (64 + z): q - z and q' - z, exact.  Three instructions a pair.
                    auto dequant = [&](uint32_t wd, uint32_t* o) {
                        o[0] = hfma2_u32(lop3_and_or(__byte_perm(wd, 0, 0x0000), 0x00F0000Fu, 0x64006400u), 0x2C003C00u, zadd);
                        o[1] = hfma2_u32(lop3_and_or(__byte_perm(wd, 0, 0x1111), 0x00F0000Fu, 0x64006400u), 0x2C003C00u, zadd);
                        o[2] = hfma2_u32(lop3_and_or(__byte_perm(wd, 0, 0x2222), 0x00F0000Fu, 0x64006400u), 0x2C003C00u, zadd);
                        o[3] = hfma2_u32(lop3_and_or(__byte_perm(wd, 0, 0x3333), 0x00F0000Fu, 0x64006400u), 0x2C003C00u, zadd);
                    };
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (C::kWide) {
                            unsigned char* row = smem + w0 + slot * C::kWBytes + (uint32_t)h * (C::kWBytes / 2) + (uint32_t)r * 128;
#pragma unroll
                            for (int c = 0; c < 8; ++c) {  // 8-k chunks of the block of 64 k
                                uint32_t o[4];
                                dequant(words[c], o);
                                *reinterpret_cast<uint4*>(row + ((c ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                            }
#pragma unroll
                            for (int c = 0; c < 8; ++c) words[c] = next[c];
                        } else {
                            uint32_t o[32];
#pragma unroll
                            for (int c = 0; c < 8; ++c) dequant(words[c], o + 4 * c);
                            if (h == 0) load(j, 1, words);
                            else if (j + 1 < GPS) load(j + 1, 0, words);
                            if (j == 0 && h == 0) free_slot();
                            if (ok) tmem_st_32x32b_x32(taddr + (slot * GPS + j) * 64 + h * 32, o);
                        }
                    }
                }
                if constexpr (C::kWide) {
                    fence_proxy_async_shared();  // the stores are in place for the tensor cores: before the arrival (mbar_arrive_cluster)
                } else if (ok) {
                    tmem_wait_st();
                    tc_fence_before();
                }
                __syncwarp();
                if (ok && lane == 0) fg_arrive<CTAS>(remote + 8u * slot);
                next_stage();
            }
        }
    } else {
        regs_inc<C::kRegsFold>();
        // ------------------------------------------------------------ fold and epilogue
        const int f = (warp - FOLD_WARP) >> 2, q = warp & 3;
        const int r = q * 32 + lane;
        const int ncol = p.tn / 2;
        const bool upper = lane >= 16;
        const unsigned short* sbase_row = GATED && upper ? p.s1 : p.s0;
        const uint32_t remote = CTAS == 2 ? map_shared(d_empty(0), 0) : d_empty(0);
        const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(f * ncol);
        pdl_wait();  // the outputs may be read, the residual written, by the preceding kernel
        bool ok = true;
        int b = 0, s = 0;  // TMEM buffer and ring stage of the group
        uint32_t ph = 0;
        for (int u = cluster; u < p.units; u += n_clusters) {
            const FgUnit w = fg_unit<!C::kWide>(p, u);
            const int n = w.nt * TN + (GATED ? (int)rank * 64 + 16 * q + (lane & 15) : (int)rank * 128 + r);
            const bool nv = n < p.N;
            const unsigned short* srow = sbase_row + (int64_t)(nv ? n : 0) * p.G;
            uint64_t s4 = nv ? fg_scales4(srow, w.g0, p.G, p.vec) : 0, s4n = 0;
            int sb = w.g0 & ~3;  // s4 holds groups sb ... sb + 3, s4n the next four
            if (nv && sb + 4 < p.G) s4n = fg_scales4(srow, sb + 4, p.G, p.vec);
            F2 acc[NACC / 2];
#pragma unroll
            for (int i = 0; i < NACC / 2; ++i) acc[i].v = 0;
            for (int g = w.g0; g < w.g1; g += GPS) {
                const bool two = GPS == 2 && g + 1 < w.g1;
                F2 sc[GPS];
#pragma unroll
                for (int j = 0; j < GPS; ++j) {
                    if (((g + j) & ~3) != sb && g + j < w.g1) {
                        s4 = s4n;
                        sb += 4;
                        if (nv && sb + 4 < p.G) s4n = fg_scales4(srow, sb + 4, p.G, p.vec);
                    }
                    sc[j] = f2(__half2float(__ushort_as_half((unsigned short)(s4 >> (16 * ((g + j) & 3))))));
                }
                if (ok && !warp_wait(done_bar(s), ph, abort_flag)) { fail(); ok = false; }
                if (++s == S) { s = 0; ph ^= 1; }
                if (ok) {
                    tc_fence_after();
                    const uint32_t src = taddr + (uint32_t)(b * GPS * NMAX);
                    // rounds of 32 columns (of both groups), each one wait; columns past tn hold old sums: never
                    // stored.  Longer rounds take registers that the dequantising warps use better (48: 3 % slower)
                    constexpr int RC = 32;
#pragma unroll
                    for (int c = 0; c < NACC; c += RC) {
                        if (c < ncol) {
                            constexpr int KR = RC / 16;
                            uint32_t v[GPS][KR][16];
#pragma unroll
                            for (int k = 0; k < KR; ++k)
                                if (C::kWide || c + 16 * k < ncol) tmem_ld_32x32b_x16(src + (uint32_t)(c + 16 * k), v[0][k]);
                            if (two) {
#pragma unroll
                                for (int k = 0; k < KR; ++k)
                                    if (c + 16 * k < ncol) tmem_ld_32x32b_x16(src + (uint32_t)(NMAX + c + 16 * k), v[GPS - 1][k]);
                            }
                            tmem_wait_ld();
                            if (c + RC >= ncol) {  // all read: the buffer is free
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) fg_arrive<CTAS>(remote + 8u * (uint32_t)b);
                            }
#pragma unroll
                            for (int j = 0; j < GPS; ++j) {
                                if (j == 1 && !two) continue;
#pragma unroll
                                for (int k = 0; k < KR; ++k) {
                                    if (!C::kWide && c + 16 * k >= ncol) continue;
                                    fg_tie(v[j][k]);
#pragma unroll
                                    for (int i = 0; i < 16; i += 2)
                                        acc[(c + 16 * k + i) / 2] =
                                            fma2(f2(__uint_as_float(v[j][k][i]), __uint_as_float(v[j][k][i + 1])), sc[j],
                                                 acc[(c + 16 * k + i) / 2]);
                                }
                            }
                        }
                    }
                }
                if (++b == NB) b = 0;
            }
            if (!C::kWide && w.g0 == w.g1) continue;  // past the end of the CTA's share
            if (wg_barrier_any(1 + f, !ok)) continue;  // all four warps agree before the staging barriers
            const int m0 = w.m0 + f * ncol;
            if (p.P && (C::kWide || !p.shares.ctas || w.g1 - w.g0 < p.G)) {
                float* P = p.P + ((int64_t)w.slice * (GATED ? 2 : 1) + (GATED && upper ? 1 : 0)) * p.M * p.N;
#pragma unroll
                for (int c = 0; c < NACC; c += 2) {
                    float v[2];
                    split(acc[c / 2], v[0], v[1]);
                    if (c < ncol && nv && m0 + c < p.M) P[(int64_t)(m0 + c) * p.N + n] = v[0];
                    if (c < ncol && nv && m0 + c + 1 < p.M) P[(int64_t)(m0 + c + 1) * p.N + n] = v[1];
                }
            } else {
                const int nb = w.nt * TN + (int)rank * (TN / CTAS);
                dispatch_act(p.act, [&](auto act) {
                    fg_epilogue<decltype(act)::value, GATED, NACC>(p, acc, ncol, m0, nb, smem, epi0 + (uint32_t)f * FG_EPI, r, 1 + f);
                    return cudaSuccess;
                });
            }
        }
    }
    __syncthreads();
    if constexpr (CTAS == 2) cluster_sync();  // nothing of the pair's products or arrivals is outstanding in either CTA
    if (warp == 2) {
        tc_fence_after();
        if constexpr (CTAS == 2) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

// The K slices' partial sums [slice][layer][M][N] added in slice order, then the epilogue.  No
// slices (an empty K): the epilogue of zeros.  With shares: only the tiles (of `rows` outputs n) that were
// cut, from as many parts as each has.  Launched as a programmatic dependent of the kernel that writes
// the partials.
template <int ACT, bool GATED>
__global__ void __launch_bounds__(256) ffn_reduce_kernel(const float* P, int slices, FgShares shares, int rows, int64_t mn, int N, const __half* bias,
                                                         const __half* residual, __half* Y, __half* Z, __half* U) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int L = GATED ? 2 : 1;
    for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; e < mn; e += (int64_t)gridDim.x * 1024) {
        if (shares.ctas) {
            slices = shares.parts((int)(e % N) / rows);
            if (slices == 1) continue;
        }
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
        split(act_fwd2<ACT>(f2(z[0], z[1])), y[0], y[1]);
        split(act_fwd2<ACT>(f2(z[2], z[3])), y[2], y[3]);
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

struct FgPlan {
    int tn, ks, stages, m_tiles, n_tiles, units;
    bool wide;  // the 256-column instantiation
    int parts;  // partial sums of an output at most: ks, or of the shares
    FgShares shares;
    uint32_t smem;
};

FgPlan fg_plan(int64_t M, int64_t N, int64_t K, bool gated) {
    const int64_t sms = std::max(2, device_sm_count()), G = K / 128;
    constexpr double kSmallGroup = 630.0;
    FgPlan best = {};
    double best_t = -1.0;
    for (int tn = 32; tn <= 256; tn += 32) {
        if (tn > 32 && tn >= M + 32) break;
        const bool wide = tn > 64;
        const int64_t slots = wide ? sms / 2 : sms;  // tiles at a time
        const int64_t rows = (wide ? 256 : 128) / (gated ? 2 : 1);
        const int64_t m_tiles = (M + tn - 1) / tn, n_tiles = (N + rows - 1) / rows;
        const int64_t tiles = m_tiles * n_tiles;
        for (int ks = 1; ks <= 16 && ks <= G; ++ks) {
            if (ks > 1 && (tiles * (ks - 1) >= slots || G / ks < 4)) break;
            const int64_t units = tiles * ks;
            const int64_t waves = (units + slots - 1) / slots;
            // cycles per group; per unit: filling and the epilogue (33 per column); a second launch and its
            // traffic when K is cut.  Large tiles: 1258 measured at tn = 256, and the other widths by the line
            // through it: 0.79, 0.83, 0.87, 0.91, 0.96 of it at tn = 96, 128, 160, 192, 224, where full waves
            // (M = 8 tn, N = 18944, K = 8192 less 4096) measured 0.80, 0.81, 0.86, 0.88, 0.97 (700, 708, 752, 767,
            // 844 ns against 871).  Small tiles: 780 a group measured
            // with the start and end of the kernel; 630 chooses best between the two instantiations.  700 gives
            // M = 96, K = N = 4096 to large tiles (23.5 us, 19.5 in small ones) and the gated M = 96, K = 4096, N =
            // 11008 (55, 51); 560 leaves the gated M = 192, K = 4096, N = 11008 to small ones (63, 61 in large).
            const double group = wide ? 830.0 + 1.67 * tn : kSmallGroup;
            double t = (double)waves * ((double)((G + ks - 1) / ks) * group + 1500.0 + 33.0 * tn);
            if (ks > 1) t += 4000.0 + (double)ks * (double)M * (double)N * (gated ? 2 : 1) * 8.0 / 3000.0;
            if (best_t < 0.0 || t < best_t) {
                best_t = t;
                best.tn = tn;
                best.ks = ks;
                best.m_tiles = (int)m_tiles;
                best.n_tiles = (int)n_tiles;
                best.units = (int)units;
                best.parts = ks;
                best.shares = {};
            }
        }
        // shares: one for each SM, with a fill and an epilogue for each tile that a share touches, and its
        // first and last tile's partial sums written and read
        // (M = 32: gated K = 8192, N = 28672 99.9 us in whole tiles, 89.8 in shares; gated K = 4096, N = 11008
        // 29.4, 26.2; plain K = 28672, N = 8192 51.4 in two slices, 50.2 in shares; M = 64: gated K = 8192, N =
        // 28672 107.1, 96.3; where the rule is near its edge either is up to 2 us better)
        const int64_t steps = (G + 1) / 2, total = n_tiles * steps, len = total / sms;
        if (wide || m_tiles > 1 || len < 4 || total * sms >= (1ll << 29)) continue;
        const int64_t longest = (total + sms - 1) / sms, per = (longest + steps - 2) / steps + 1;
        const double t = (double)longest * 2.0 * kSmallGroup + (double)per * (1500.0 + 33.0 * tn) + 4000.0 +
                         (double)sms * 2.0 * 128.0 * (double)M * 8.0 / 3000.0;
        if (t < best_t) {
            best_t = t;
            best.tn = tn;
            best.ks = 1;
            best.m_tiles = 1;
            best.n_tiles = (int)n_tiles;
            best.units = (int)(sms * per);
            best.parts = (int)((steps + len - 1) / len + 1);
            best.shares = {(int)sms, (int)steps, (int)total};
        }
    }
    best.wide = best.tn > 64;
    const uint32_t group = (uint32_t)best.tn * (best.wide ? 128u : 256u) + FG_P_BYTES;
    const uint32_t stage = group * (uint32_t)(best.wide ? FgCfg<256>::kGPS : FgCfg<64>::kGPS);
    const uint32_t fixed = (best.wide ? FgCfg<256>::kAG * FgCfg<256>::kWBytes : 0) + 2 * FG_EPI + 512;
    best.stages = (int)std::min<uint32_t>((FG_SMEM - 1024 - fixed) / stage, FG_MAXS);
    best.smem = stage * (uint32_t)best.stages + fixed + 1024;
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
        if (err[dev] == cudaSuccess && a.numRegs != FgCfg<NMAX>::kRegs) err[dev] = cudaErrorInvalidConfiguration;
    });
    return err[dev];
}

template <bool GATED, int NMAX>
cudaError_t fg_launch(const CUtensorMap& tx, const CUtensorMap& t0, const CUtensorMap& t1, const FgArgs& args,
                      const FgPlan& pl, cudaStream_t stream) {
    const cudaError_t e = fg_setup<GATED, NMAX>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    constexpr int ctas = FgCfg<NMAX>::kCtas;
    cfg.gridDim = dim3((unsigned)(ctas * std::min(pl.units, std::max(1, device_sm_count() / ctas))), 1, 1);
    cfg.blockDim = dim3(FgCfg<NMAX>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = pl.smem;
    cfg.stream = stream;
    // A programmatic dependent of whatever precedes it: set-up overlaps the predecessor's end; every
    // role waits for that end before it touches global memory (but for static weights, `early`)
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, ffn_gemm_kernel<GATED, NMAX>, tx, t0, t1, args);
}

cudaError_t fg_reduce(const float* P, int slices, const FgShares& shares, int64_t M, int64_t N, bool gated, const W4Epilogue& ep,
                      cudaStream_t stream) {
    const int64_t mn = M * N;
    const int rows = gated ? 64 : 128;  // outputs n of a shared tile
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
            return cudaLaunchKernelEx(&cfg, ffn_reduce_kernel<ACT, true>, P, slices, shares, rows, mn, (int)N, hp(ep.bias),
                                      hp(ep.residual), hp(ep.Y), hp(ep.Z), hp(ep.U));
        return cudaLaunchKernelEx(&cfg, ffn_reduce_kernel<ACT, false>, P, slices, shares, rows, mn, (int)N, hp(ep.bias), hp(ep.residual),
                                  hp(ep.Y), hp(ep.Z), hp(ep.U));
    });
}

}  // namespace

cudaError_t launch_ffn_reduce(const float* P, int slices, int64_t M, int64_t N, bool gated, const W4Epilogue& ep,
                              cudaStream_t stream) {
    return fg_reduce(P, slices, {}, M, N, gated, ep, stream);
}

size_t ffn_gemm_workspace(int64_t M, int64_t N, int64_t K, bool gated) {
    const FgPlan pl = fg_plan(M, N, K, gated);
    return pl.parts > 1 ? (size_t)pl.parts * (size_t)M * (size_t)N * (gated ? 8 : 4) : 0;
}

cudaError_t launch_ffn_gemm(const uint16_t* X, int64_t M, int64_t N, int64_t K, const W4Layer& w, const W4Layer* w2,
                            const W4Epilogue& ep, void* ws, bool weights_static, int* status, cudaStream_t stream) {
    const bool gated = w2 != nullptr;
    const FgPlan pl = fg_plan(M, N, K, gated);
    if (pl.parts > 1 && !ws) return cudaErrorInvalidValue;
    CUtensorMap tx, t0, t1;
    if (!make_tensor_map_2d(&tx, X, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, (uint64_t)K, (uint64_t)M, 64,
                            (uint32_t)(pl.wide ? pl.tn / 2 : pl.tn),
                            CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    // packed rows in pieces of a step's groups: 64 bytes each
    auto packed_map = [&](CUtensorMap* t, const uint32_t* packed) {
        return make_tensor_map_2d(t, packed, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, (uint64_t)(K / 8), (uint64_t)N,
                                  16u * (uint32_t)(pl.wide ? FgCfg<256>::kGPS : FgCfg<64>::kGPS), gated ? 16 : 128,
                                  pl.wide ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (!packed_map(&t0, w.packed)) return cudaErrorInvalidValue;
    t1 = t0;
    if (gated && !packed_map(&t1, w2->packed)) return cudaErrorInvalidValue;
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
    a.P = pl.parts > 1 ? static_cast<float*>(ws) : nullptr;
    a.act = ep.activation;
    a.M = (int)M;
    a.N = (int)N;
    a.G = (int)G;
    a.tn = pl.tn;
    a.raster.m_tiles = pl.m_tiles;
    a.raster.n_tiles = pl.n_tiles;
    a.raster.ks = pl.ks;
    // m-tiles whose X stays in L2 (about 48 MB) run down the weights together
    a.raster.gm = (int)std::max<int64_t>(1, std::min<int64_t>(pl.m_tiles, (48ll << 20) / ((int64_t)pl.tn * K * 2)));
    a.shares = pl.shares;
    a.units = pl.units;
    a.stages = pl.stages;
    a.vec = vec_ok(w) && (!gated || vec_ok(*w2)) ? 1 : 0;
    a.early = weights_static ? 1 : 0;
    a.status = status;
    cudaError_t e;
    if (gated) e = pl.wide ? fg_launch<true, 256>(tx, t0, t1, a, pl, stream) : fg_launch<true, 64>(tx, t0, t1, a, pl, stream);
    else e = pl.wide ? fg_launch<false, 256>(tx, t0, t1, a, pl, stream) : fg_launch<false, 64>(tx, t0, t1, a, pl, stream);
    if (e != cudaSuccess || pl.parts == 1) return e;
    return fg_reduce(a.P, pl.ks, pl.shares, M, N, gated, ep, stream);
}

}  // namespace w4
