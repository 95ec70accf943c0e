// Backward pass of the activations beside w4_gemm_fused and w4_gemm_gated.
//
//   dZ = dY * act'(Z), dbias[n] = sum_m dZ[m, n]          (U null)
//   dG = dH * U * act'(G), dU = dH * act(G)               (gated: Z holds G, dY holds dH)
//
// The gated form is bound by HBM (10 bytes per element; silu 0.93 of the copy rate).  The plain form moves 6
// bytes against ten to thirty fp32 operations, and with gelu it is bound by the issue of instructions and the
// latency of loads, not by one unit (counters at 1999 x 11000: 65 % of the issue slots of active cycles, FMA
// 45 %, ALU 41 %, special functions 33 %, HBM 33 to 38 %; with sums an SM is active 82 % of the time).  A
// thread takes 8 neighbouring columns (16-byte loads and stores) of every rl-th row of its CTA's block of
// rows, two or four rows' loads in flight together (outputs may be the inputs' own buffers, so nothing moves a
// load over a store).  A CTA is cw column vectors by rl = 256 / cw row lanes, so narrow matrices fill it too.
//
// For dbias (SUM) the thread keeps its columns' sums in registers (fp32, row order), the CTA's row lanes are
// added in order in shared memory, the row blocks' sums go to the workspace and a second launch adds them in
// a fixed order: deterministic, no atomics.  dZ enters the sums unrounded.  The blocks' sums are read
// again, so SUM takes few long blocks, one wave of four CTAs per SM; the others take 4 rows a thread
// (measured at 2048 x 11008, us: gelu 32 against 39 with 16 rows, gated silu 39 against 41; with dbias 51
// against 41).
#include <algorithm>

#include "activation.cuh"
#include "internal.h"

namespace w4 {

namespace {

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
}

constexpr int AB_THREADS = 256;
constexpr int AB_SUM_CTAS = 4;  // per SM, where sums are kept

// blockIdx.y: block of `rows` rows; blockIdx.x: cw (a power of two) column vectors.
template <int ACT, bool GATED, bool SUM>
__global__ void __launch_bounds__(AB_THREADS, AB_SUM_CTAS) act_backward_kernel(const uint4* dY, const uint4* Z, const uint4* U,
                                                                  int64_t M, int64_t N8, int64_t rows, int cw, uint4* dZ,
                                                                  uint4* dU, float* part) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int AB_ROWS = SUM ? 4 : 2;  // rows a thread loads together
    const int rl = AB_THREADS / cw, lane = threadIdx.x / cw;
    const int64_t c = (int64_t)blockIdx.x * cw + threadIdx.x % cw;
    const int64_t m0 = (int64_t)blockIdx.y * rows, m1 = m0 + rows < M ? m0 + rows : M;
    F2 sum[4] = {};
    if (c < N8) {
        for (int64_t mb = m0 + lane; mb < m1; mb += (int64_t)AB_ROWS * rl) {
            uint4 vy[AB_ROWS], vz[AB_ROWS] = {}, vu[AB_ROWS];
#pragma unroll
            for (int i = 0; i < AB_ROWS; ++i) {
                const int64_t m = mb + (int64_t)i * rl;
                if (m < m1) {
                    vy[i] = dY[m * N8 + c];
                    if (Z) vz[i] = Z[m * N8 + c];
                    if (GATED) vu[i] = U[m * N8 + c];
                }
            }
#pragma unroll
            for (int i = 0; i < AB_ROWS; ++i) {
                const int64_t m = mb + (int64_t)i * rl;
                if (m >= m1) break;
                float dy[8], z[8], u[8], dz[8], du[8];
                unpack8(vy[i], dy);
                unpack8(vz[i], z);
                if (GATED) unpack8(vu[i], u);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    F2 a;
                    const F2 y = f2(dy[j], dy[j + 1]), d = act_grad2<ACT>(f2(z[j], z[j + 1]), a);
                    if (GATED) {
                        split(mul2(mul2(y, f2(u[j], u[j + 1])), d), dz[j], dz[j + 1]);
                        split(mul2(y, a), du[j], du[j + 1]);
                    } else {
                        const F2 r = mul2(y, d);
                        if (SUM) sum[j / 2] = add2(sum[j / 2], r);
                        split(r, dz[j], dz[j + 1]);
                    }
                }
                if (dZ) dZ[m * N8 + c] = pack8(dz);
                if (GATED) dU[m * N8 + c] = pack8(du);
            }
        }
    }
    if constexpr (SUM) {
        __shared__ float sh[AB_THREADS][9];
#pragma unroll
        for (int j = 0; j < 8; j += 2) split(sum[j / 2], sh[threadIdx.x][j], sh[threadIdx.x][j + 1]);
        __syncthreads();
        for (int i = threadIdx.x; i < cw * 8; i += AB_THREADS) {  // column i % 8 of vector i / 8
            const int64_t cc = (int64_t)blockIdx.x * cw + i / 8;
            if (cc >= N8) continue;
            float s = 0.0f;
            for (int l = 0; l < rl; ++l) s += sh[l * cw + i / 8][i % 8];
            part[((int64_t)blockIdx.y * N8 + cc) * 8 + i % 8] = s;
        }
    }
}

// dbias[n] = sum of the row blocks' partials: eight threads of a column take every eighth block, then
// their sums are added in order.  A programmatic dependent of the kernel that writes the partials.
__global__ void __launch_bounds__(AB_THREADS) column_sum_kernel(const float* part, int64_t blocks, int64_t N, float* dbias) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float sh[8][32];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t n = (int64_t)blockIdx.x * 32 + x;
    float s = 0.0f;
    if (n < N)
        for (int64_t b = y; b < blocks; b += 8) s += part[b * N + n];
    sh[y][x] = s;
    __syncthreads();
    if (y == 0 && n < N) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sh[i][x];
        dbias[n] = s;
    }
}

struct AbPlan {
    int cw;
    int64_t rows, blocks;
};
AbPlan ab_plan(int64_t M, int64_t N, bool sum) {
    AbPlan p;
    p.cw = 1;
    while (p.cw < AB_THREADS && p.cw < N / 8) p.cw *= 2;
    const int64_t rl = AB_THREADS / p.cw, columns = (N / 8 + p.cw - 1) / p.cw;
    // row blocks: one wave with sums; else 4 rows a thread, as far as the grid's 65535 reach
    const int64_t most = sum ? std::max<int64_t>(1, (int64_t)device_sm_count() * AB_SUM_CTAS / columns) : 32768;
    const int64_t per = (M + most * rl - 1) / (most * rl);
    p.rows = rl * (sum ? per : std::max<int64_t>(4, per));
    p.blocks = (M + p.rows - 1) / p.rows;
    return p;
}

}  // namespace

size_t act_backward_workspace(int64_t M, int64_t N) {
    return M == 0 || N == 0 ? 0 : (size_t)ab_plan(M, N, true).blocks * (size_t)N * 4;
}

cudaError_t launch_act_backward(const uint16_t* dY, const uint16_t* Z, const uint16_t* U, int64_t M, int64_t N,
                                int activation, uint16_t* dZ, uint16_t* dU, float* dbias, void* ws,
                                cudaStream_t stream) {
    const AbPlan pl = ab_plan(M, N, dbias != nullptr);
    const int64_t N8 = N / 8;
    const dim3 grid((unsigned)((N8 + pl.cw - 1) / pl.cw), (unsigned)pl.blocks);
    float* part = dbias ? static_cast<float*>(ws) : nullptr;
    auto p = [](const uint16_t* q) { return reinterpret_cast<const uint4*>(q); };
    auto o = [](uint16_t* q) { return reinterpret_cast<uint4*>(q); };
    cudaLaunchConfig_t cfg = {};  // both launches: programmatic dependents of what precedes them
    cfg.gridDim = grid;
    cfg.blockDim = dim3(AB_THREADS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const uint4* none = nullptr;
    cudaError_t e = dispatch_act(activation, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        if (U)
            return cudaLaunchKernelEx(&cfg, act_backward_kernel<ACT, true, false>, p(dY), p(Z), p(U), M, N8, pl.rows, pl.cw,
                                      o(dZ), o(dU), part);
        if (dbias)
            return cudaLaunchKernelEx(&cfg, act_backward_kernel<ACT, false, true>, p(dY), p(Z), none, M, N8, pl.rows, pl.cw,
                                      o(dZ), o(nullptr), part);
        return cudaLaunchKernelEx(&cfg, act_backward_kernel<ACT, false, false>, p(dY), p(Z), none, M, N8, pl.rows, pl.cw,
                                  o(dZ), o(nullptr), part);
    });
    if (e != cudaSuccess || !dbias) return e;
    cfg.gridDim = dim3((unsigned)((N + 31) / 32), 1, 1);
    return cudaLaunchKernelEx(&cfg, column_sum_kernel, (const float*)part, pl.blocks, N, dbias);
}

}  // namespace w4
