// ckpt_route_grad.cuh -- the routing's slot gradients from 8-bit expert outputs (checkpoint.cuh):
// the formulas of route_grad.cuh with the expert outputs E_i(x_t) of every (token, slot) read
// from a checkpoint in slot order [T K][D] instead of the handle's last forward.
//   s_tk = <dy_t, Y_tk>;  over a decision's tokens (one token, or a segment of S):
//   dg_k = m_k sum s_tk, m_k = [l_k >= 0];  dmh_k = g_k sum s_tk + n reg
//   d_l_k = dmh_k sigmoid(l_k)(1 - sigmoid(l_k));  d_r_k = g_k (dg_k - sum_j g_j dg_j)
// The decision's gradients go to its first token; the others of a segment get 0.
#pragma once
#include "checkpoint.cuh"

namespace beam {

// One warp per (token, slot): the dot product.
template <typename T>
__global__ void __launch_bounds__(256)
ckpt_dot_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ scale, int n_tok, int K,
                int D, int nb, const T* __restrict__ dy, long long lddy, float* __restrict__ s_out)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i < (long long)n_tok * K) {
        const long long t = i / K;
        float acc = 0.f;
        for (int b = 0; b < nb; ++b) {
            const int c = b * kCkptBlock + lane;
            if (c < D)
                acc = fmaf((float)q[(i * nb + b) * kCkptBlock + lane] * ckpt_step(scale[i * nb + b]),
                           to_float(dy[t * lddy + c]), acc);
        }
        acc = warp_sum(acc);
        if (lane == 0) s_out[i] = acc;
    }
    pdl_launch_dependents();
}

// One warp per decision, lane = slot.
__global__ void __launch_bounds__(256)
ckpt_slot_grad_kernel(const float* __restrict__ s, int n_tok, int K, int S,
                      const float* __restrict__ gate, const float* __restrict__ mlogit, float reg,
                      float* __restrict__ d_r, float* __restrict__ d_l)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const long long t0 = r * S, t1 = min((long long)n_tok, t0 + S);
    if (t0 < n_tok) {
        const bool on = lane < K;
        float run = 0.f;
        for (long long t = t0; t < t1; ++t) {
            if (on) run += s[t * K + lane];
            if (on && t != t0) { d_r[t * K + lane] = 0.f; d_l[t * K + lane] = 0.f; }
        }
        const float g = on ? gate[t0 * K + lane] : 0.f, l = on ? mlogit[t0 * K + lane] : 0.f;
        const float dg = (on && l >= 0.f) ? run : 0.f;
        const float c = warp_sum(g * dg);
        const float sg = sigmoid_f(l);
        if (on) {
            d_r[t0 * K + lane] = g * (dg - c);
            d_l[t0 * K + lane] = fmaf(run, g, (float)(t1 - t0) * reg) * (sg * (1.f - sg));
        }
    }
    pdl_launch_dependents();
}

}  // namespace beam
