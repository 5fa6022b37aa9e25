// router_linear.cuh -- the backward of the router's linear map logits = x W (x [T][D], W [D][C]):
//   dW[d][c] = sum_t x[t][d] G[t][c]   with x from an 8-bit checkpoint
//   dx[t][d] = sum_c G[t][c] W[d][c]
// for the dense logit gradient G [T][C] (the balance term reaches every expert of every token).
#pragma once
#include "checkpoint.cuh"

namespace beam {

constexpr int kLinTile = 64, kLinK = 16;

// out[m][n] = sum_k a(m, k) b(n, k) on 64 x 64 tiles, 16 outputs per thread.
template <typename FA, typename FB, typename FO>
__device__ __forceinline__ void lin_tile(int m0, int n0, int Kd, FA a, FB b, FO out)
{
    __shared__ float sa[kLinK][kLinTile + 1], sb[kLinK][kLinTile + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < Kd; k0 += kLinK) {
        for (int i = threadIdx.x; i < kLinTile * kLinK; i += 256) {
            const int r = i & (kLinTile - 1), k = i / kLinTile;
            sa[k][r] = k0 + k < Kd ? a(m0 + r, k0 + k) : 0.f;
            sb[k][r] = k0 + k < Kd ? b(n0 + r, k0 + k) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kLinK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) out(m0 + ty + 16 * i, n0 + tx + 16 * j, acc[i][j]);
}

// dW: m = d, n = c, k = t.  dw is [parts][D][C / parts].
template <typename T>
__global__ void __launch_bounds__(256)
router_weight_grad_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                          int n_tok, int D, int nb, const T* __restrict__ g, long long ldg, int C,
                          int cp, float* __restrict__ dw)
{
    pdl_wait();
    lin_tile(blockIdx.x * kLinTile, blockIdx.y * kLinTile, n_tok,
        [&](int d, int t) {
            return d < D ? (float)q[((long long)t * nb) * kCkptBlock + d] *
                           ckpt_step(scale[(long long)t * nb + d / kCkptBlock]) : 0.f;
        },
        [&](int c, int t) { return c < C ? to_float(g[t * ldg + c]) : 0.f; },
        [&](int d, int c, float v) {
            if (d < D && c < C) dw[((long long)(c / cp) * D + d) * cp + c % cp] = v;
        });
    pdl_launch_dependents();
}

// dx: m = t, n = d, k = c.
template <typename T, typename TW>
__global__ void __launch_bounds__(256)
router_input_grad_kernel(const T* __restrict__ g, long long ldg, int n_tok, int C,
                         const TW* __restrict__ w, long long ldw, int D, float* __restrict__ dx)
{
    pdl_wait();
    lin_tile(blockIdx.x * kLinTile, blockIdx.y * kLinTile, C,
        [&](int t, int c) { return t < n_tok ? to_float(g[t * ldg + c]) : 0.f; },
        [&](int d, int c) { return d < D ? to_float(w[d * ldw + c]) : 0.f; },
        [&](int t, int d, float v) { if (t < n_tok && d < D) dx[(long long)t * D + d] = v; });
    pdl_launch_dependents();
}

}  // namespace beam
