// Input gradients dX[m, k] = sum_n dY[m, n] W[n, k] (one layer or the sum of two) as plain tiled
// products on the CUDA cores: 64 x 64 output tiles, 4 x 4 fp32 sums per thread, the contraction in
// steps of 16 through shared memory.  Every weight is (q - z) * s in fp32 (exact), every sum fp32,
// one rounding at the store.
#include "activation.cuh"
#include "internal.h"

namespace w4 {

namespace {

struct Layer {
    const uint32_t* packed;
    const __half* scales;
    const uint8_t* zeros;
};

__device__ __forceinline__ float weight_at(const Layer& w, int64_t n, int64_t k, int64_t K) {
    const uint32_t word = w.packed[n * (K >> 3) + (k >> 3)];
    const int q = (word >> (4 * (k & 7))) & 15;
    const int64_t g = n * (K >> 7) + (k >> 7);
    return (float)(q - (int)w.zeros[g]) * __half2float(w.scales[g]);
}

constexpr int ST = 64, SK = 16;

// One 64 x 64 tile of sum_c A[m, c] B(o, c): DX: o = k, c = n; else o = n, c = k.
template <bool DX>
__device__ __forceinline__ void simple_tile(const __half* A, const Layer& w, int64_t M, int64_t N, int64_t K, int64_t m0,
                                            int64_t o0, float (&acc)[4][4], float (*sa)[ST + 1], float (*sb)[ST + 1]) {
    const int64_t O = DX ? K : N, C = DX ? N : K;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t c0 = 0; c0 < C; c0 += SK) {
        for (int i = threadIdx.x; i < ST * SK; i += 256) {
            const int c = i & (SK - 1), r = i >> 4;
            sa[c][r] = m0 + r < M && c0 + c < C ? __half2float(A[(m0 + r) * C + c0 + c]) : 0.0f;
            float b = 0.0f;
            if (o0 + r < O && c0 + c < C) b = DX ? weight_at(w, c0 + c, o0 + r, K) : weight_at(w, o0 + r, c0 + c, K);
            sb[c][r] = b;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < SK; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[c][ty * 4 + i], sb[c][tx * 4 + j], acc[i][j]);
        }
        __syncthreads();
    }
}

// ACT < 0: dX itself; else the gate's backward pass on it.
template <int ACT>
__global__ void __launch_bounds__(256) simple_dx_kernel(const __half* dY, Layer w, const __half* dY2, Layer w2, int64_t M,
                                                        int64_t N, int64_t K, const __half* G, const __half* U,
                                                        __half* dX, __half* dU) {
    __shared__ float sa[SK][ST + 1], sb[SK][ST + 1];
    const int64_t m0 = (int64_t)blockIdx.y * ST, k0 = (int64_t)blockIdx.x * ST;
    float acc[4][4] = {};
    simple_tile<true>(dY, w, M, N, K, m0, k0, acc, sa, sb);
    if (dY2) simple_tile<true>(dY2, w2, M, N, K, m0, k0, acc, sa, sb);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + (threadIdx.x >> 4) * 4 + i, k = k0 + (threadIdx.x & 15) * 4 + j;
            if (m >= M || k >= K) continue;
            const int64_t e = m * K + k;
            if constexpr (ACT < 0) {
                dX[e] = __float2half_rn(acc[i][j]);
            } else {
                const float dh = acc[i][j], u = __half2float(U[e]);
                float a;
                const float d = act_grad<ACT>(__half2float(G[e]), a);
                dX[e] = __float2half_rn(dh * u * d);
                dU[e] = __float2half_rn(dh * a);
            }
        }
}

Layer layer(const W4Layer& l) { return {l.packed, reinterpret_cast<const __half*>(l.scales), l.zeros}; }
const __half* h(const uint16_t* p) { return reinterpret_cast<const __half*>(p); }
__half* h(uint16_t* p) { return reinterpret_cast<__half*>(p); }

}  // namespace

cudaError_t launch_dx_simple(const uint16_t* dY, const W4Layer& w, const uint16_t* dY2, const W4Layer* w2, int64_t M,
                             int64_t N, int64_t K, const W4GateGrad* gate, uint16_t* dX, cudaStream_t stream) {
    const dim3 grid((unsigned)((K + ST - 1) / ST), (unsigned)((M + ST - 1) / ST));
    const Layer a = layer(w), b = w2 ? layer(*w2) : a;
    if (!gate) {
        simple_dx_kernel<-1><<<grid, 256, 0, stream>>>(h(dY), a, h(dY2), b, M, N, K, nullptr, nullptr, h(dX), nullptr);
        return cudaGetLastError();
    }
    return dispatch_act(gate->activation, [&](auto act) {
        simple_dx_kernel<decltype(act)::value><<<grid, 256, 0, stream>>>(h(dY), a, nullptr, b, M, N, K, h(gate->G),
                                                                         h(gate->U), h(gate->dG), h(gate->dU));
        return cudaGetLastError();
    });
}

}  // namespace w4
