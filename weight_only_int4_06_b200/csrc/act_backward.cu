// Backward pass of the activations beside w4_gemm_fused and w4_gemm_gated.
//
//   dZ = dY * act'(Z), dbias[n] = sum_m dZ[m, n]          (U null)
//   dG = dH * U * act'(G), dU = dH * act(G)               (gated: Z holds G, dY holds dH)
//
// Bound by HBM: 6 bytes per element (10 gated) against about ten fp32 operations.  A thread takes 8
// neighbouring columns (16-byte loads and stores).  For dbias a CTA walks down a block of rows with
// its columns' sums in registers (fp32, row order), the row blocks' partials go to the workspace and
// a second launch adds them in block order: deterministic, no atomics.  dZ enters the sum unrounded.
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

// blockIdx.y: block of `rows` rows; blockIdx.x: 8 AB_THREADS columns.  Outputs may be the inputs'
// own buffers (every element is read before it is written, by one thread).
template <int ACT, bool GATED>
__global__ void __launch_bounds__(AB_THREADS) act_backward_kernel(const uint4* dY, const uint4* Z, const uint4* U,
                                                                  int64_t M, int64_t N8, int64_t rows, uint4* dZ,
                                                                  uint4* dU, float* part) {
    const int64_t c = (int64_t)blockIdx.x * AB_THREADS + threadIdx.x;
    if (c >= N8) return;
    const int64_t m0 = (int64_t)blockIdx.y * rows, m1 = m0 + rows < M ? m0 + rows : M;
    float sum[8] = {};
    for (int64_t m = m0; m < m1; ++m) {
        const int64_t e = m * N8 + c;
        float dy[8], z[8] = {}, u[8], dz[8], du[8];
        unpack8(dY[e], dy);
        if (Z) unpack8(Z[e], z);
        if (GATED) unpack8(U[e], u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float a;
            const float d = act_grad<ACT>(z[i], a);
            if (GATED) {
                dz[i] = dy[i] * u[i] * d;
                du[i] = dy[i] * a;
            } else {
                dz[i] = dy[i] * d;
                sum[i] += dz[i];
            }
        }
        if (dZ) dZ[e] = pack8(dz);
        if (GATED) dU[e] = pack8(du);
    }
    if (!GATED && part) {
        float4* p = reinterpret_cast<float4*>(part + ((int64_t)blockIdx.y * N8 + c) * 8);
        p[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        p[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
    }
}

__global__ void __launch_bounds__(AB_THREADS) column_sum_kernel(const float* part, int64_t blocks, int64_t N, float* dbias) {
    const int64_t n = (int64_t)blockIdx.x * AB_THREADS + threadIdx.x;
    if (n >= N) return;
    float s = 0.0f;
    for (int64_t b = 0; b < blocks; ++b) s += part[b * N + n];
    dbias[n] = s;
}

// Rows per CTA and row blocks: a function of M alone, so that the workspace size needs no device.
int64_t ab_rows(int64_t M) { return M <= 4096 ? 16 : (M + 255) / 256; }
int64_t ab_blocks(int64_t M) { return (M + ab_rows(M) - 1) / ab_rows(M); }

}  // namespace

size_t act_backward_workspace(int64_t M, int64_t N) { return (size_t)ab_blocks(M) * (size_t)N * 4; }

cudaError_t launch_act_backward(const uint16_t* dY, const uint16_t* Z, const uint16_t* U, int64_t M, int64_t N,
                                int activation, uint16_t* dZ, uint16_t* dU, float* dbias, void* ws,
                                cudaStream_t stream) {
    const int64_t N8 = N / 8;
    const dim3 grid((unsigned)((N8 + AB_THREADS - 1) / AB_THREADS), (unsigned)ab_blocks(M));
    float* part = dbias ? static_cast<float*>(ws) : nullptr;
    auto p = [](const uint16_t* q) { return reinterpret_cast<const uint4*>(q); };
    auto o = [](uint16_t* q) { return reinterpret_cast<uint4*>(q); };
    cudaError_t e = dispatch_act(activation, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        if (U)
            act_backward_kernel<ACT, true>
                <<<grid, AB_THREADS, 0, stream>>>(p(dY), p(Z), p(U), M, N8, ab_rows(M), o(dZ), o(dU), nullptr);
        else
            act_backward_kernel<ACT, false>
                <<<grid, AB_THREADS, 0, stream>>>(p(dY), p(Z), p(U), M, N8, ab_rows(M), o(dZ), o(dU), part);
        return cudaGetLastError();
    });
    if (e != cudaSuccess || !dbias) return e;
    column_sum_kernel<<<(unsigned)((N + AB_THREADS - 1) / AB_THREADS), AB_THREADS, 0, stream>>>(part, ab_blocks(M), N,
                                                                                               dbias);
    return cudaGetLastError();
}

}  // namespace w4
