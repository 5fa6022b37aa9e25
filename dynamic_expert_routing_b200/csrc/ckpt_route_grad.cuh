// ckpt_route_grad.cuh -- the routing's slot gradients from 8-bit expert outputs (checkpoint.cuh):
// the formulas of route_grad.cuh with the expert outputs E_i(x_t) of every (token, slot) read
// from a checkpoint in slot order [T K][D] instead of the handle's last forward.
//   s_tk = <dy_t, Y_tk>;  over a decision's tokens (one token, or a segment of S):
//   dg_k = m_k sum s_tk, m_k = [l_k >= 0];  dmh_k = g_k sum s_tk + n reg
//   d_l_k = dmh_k sigmoid(l_k) sigmoid(-l_k);  d_r_k = g_k (dg_k - sum_j g_j dg_j)
// The decision's gradients go to its first token; the others of a segment get 0.
// HBM-bound: one byte per expert-output value and dy once; at K = 16 the unpacking (a byte permute
// and half an add per value) and the multiply-adds (half an instruction) are within a factor of two of the
// memory time, so nothing else may enter the inner loop.
//
// Measured on B200: 8192 tokens x 16 slots x 1536, float32 dy: 47.3 us, 261 MB, 5.5 TB/s (84 % of the measured
// copy rate; the loads without the arithmetic take 44).  8-byte loads of q for all slots at once, 141 registers: 95 us;
// four slots in flight instead of eight, at any occupancy: 54-65 us; q and dy through a shared-memory ring of
// asynchronous copies, 90 KB per SM in flight: 57 us; two warps per token, eight slots each: 50 us.
// bf16 dy 46.7 us: its bytes fall by a tenth (floor 36), the instructions stay.  In segments of 16 48.3 us, with
// the second launch.  33 x 2 x 4096: 2.25 us with eight warps per token, 5.7 with one.
#pragma once
#include "checkpoint.cuh"

namespace beam {

constexpr int kDotThreads = 256, kDotWarps = kDotThreads / 32;
constexpr int kDotCols = 16 * 32;   // columns of one strip: 16 per lane, one 16-byte load of q

// The slot gradients of one decision, lane = slot: run = sum of s over its n tokens.
__device__ __forceinline__ void slot_grads(bool on, float run, float g, float l, int n, float reg,
                                           float& gr, float& gl)
{
    const float dg = (on && l >= 0.f) ? run : 0.f;
    const float c = warp_sum(on ? g * dg : 0.f);
    gr = g * (dg - c);
    gl = fmaf(run, g, (float)n * reg) * (sigmoid_f(l) * sigmoid_f(-l));   // 1 - sigmoid(l) would cancel for a large l
}

// Sums v[0..N) over the warp's lanes: afterwards lane k (k < N) holds the total of v[k].  Each
// step halves the values a lane carries, N - 1 + log2(32 / N) shuffles instead of 5 N.
template <int N>
__device__ __forceinline__ float warp_sum_slots(float* v, int lane)
{
#pragma unroll
    for (int o = N / 2; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    float r = v[0];
#pragma unroll
    for (int o = N; o < 32; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    return r;
}

// Sixteen columns of a dy row from column c, zeros past D.
template <typename T>
__device__ __forceinline__ void load_dy16(const T* __restrict__ row, int c, int D, bool vec, float* f)
{
    if (vec && c + 16 <= D) {
#pragma unroll
        for (int j = 0; j < 16; j += Vec<T>::N)
            Vec<T>::widen(__ldg(reinterpret_cast<const uint4*>(row + c + j)), f + j);
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = c + j < D ? to_float(row[c + j]) : 0.f;
    }
}

// Two floats in a register pair: the f32x2 instructions add, or multiply and add, both in one issue slot, each
// rounded by itself.
__device__ __forceinline__ unsigned long long f32_pair(float lo, float hi)
{
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
// a += the word's four values times f: the even columns in the lower half, the odd ones in the upper.
__device__ __forceinline__ void dot4_pairs(uint32_t w, const float* f, unsigned long long& a)
{
    const unsigned long long off = f32_pair(-8388736.f, -8388736.f);   // ckpt_unpack4's
    w ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        unsigned long long v = f32_pair(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + 2 * i)),
                                        __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441 + 2 * i)));
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(v), "l"(off));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(v), "l"(f32_pair(f[2 * i], f[2 * i + 1])));
    }
}

// The scale bytes of a strip (512 columns, 16 blocks from block b0 on) of up to eight slots, four blocks of a slot
// per lane: one load where rows of scales are 4-byte aligned.  (A byte per lane and slot instead: 4 us of 49, for
// 8192 x 16 x 1536.)
__device__ __forceinline__ uint32_t load_scales(const uint8_t* __restrict__ st, int nb, int k0, int slots, int b0, int lane,
                                                bool words)
{
    const int b = b0 + 4 * (lane & 3);
    const uint8_t* p = st + (long long)(k0 + min(lane >> 2, slots - 1)) * nb + b;
    if (b >= nb) return 0u;
    if (words) return __ldg(reinterpret_cast<const uint32_t*>(p));
    uint32_t r = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (b + i < nb) r |= (uint32_t)__ldg(p + i) << (8 * i);
    return r;
}
// 2^k of the lane's block (lane / 2) of slot k.
__device__ __forceinline__ float strip_step(uint32_t scales, int k, int lane)
{
    const uint32_t w = __shfl_sync(0xffffffffu, scales, 4 * k + (lane >> 3));
    return __uint_as_float(__byte_perm(w, 0u, ((lane >> 1 & 3) << 12) | 0x0444) >> 1);
}

// KM: the smallest of 2, 4, 8, 16, 32 that holds K.  WPT warps share a token, each taking every
// WPT-th strip of its columns for all K slots (dy is read once per token); their sums are added in
// warp order.  U strips are loaded together: two where K <= 2 and a warp has them (4096 x 2 x 4096 20.0 us, one
// by one 22.1).  With one-token decisions (grads) the slot gradients follow in the same kernel.
template <typename T, int KM, int U>
__global__ void __launch_bounds__(kDotThreads, KM <= 16 ? 2 : 1)
ckpt_dot_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ scale, int n_tok, int K,
                int D, int nb, const T* __restrict__ dy, long long lddy, int vec, int wpt,
                const float* __restrict__ gate, const float* __restrict__ mlogit, float reg,
                int grads, float* __restrict__ s_out, float* __restrict__ d_r, float* __restrict__ d_l)
{
    __shared__ float s_part[kDotWarps][32];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp % wpt;
    const long long t = (long long)blockIdx.x * (kDotWarps / wpt) + warp / wpt;
    const bool live = t < n_tok;
    const bool lead = live && sub == 0 && lane < K;
    const long long o = t * K + lane;
    float g = 0.f, l = 0.f;
    if (lead && grads) { g = __ldg(gate + o); l = __ldg(mlogit + o); }
    float acc[KM];
#pragma unroll
    for (int k = 0; k < KM; ++k) acc[k] = 0.f;
    if (live) {
        constexpr int B = KM < 8 ? KM : 8;   // slots whose loads are in flight together, in U strips
        const T* dyr = dy + t * lddy;
        const int Dp = nb * kCkptBlock;
        const int8_t* qt = q + t * K * Dp;
        const uint8_t* st = scale + t * K * nb;
        const bool words = (nb & 3) == 0 && (reinterpret_cast<uintptr_t>(scale) & 3) == 0;
#pragma unroll 1
        for (int c0 = sub * kDotCols; c0 < Dp; c0 += U * wpt * kDotCols) {
            float f[U][16];
#pragma unroll
            for (int u = 0; u < U; ++u) load_dy16(dyr, c0 + u * wpt * kDotCols + lane * 16, D, vec, f[u]);
#pragma unroll
            for (int k0 = 0; k0 < KM; k0 += B) {
                if (k0 >= K) break;
                uint4 w[U][B];
                uint32_t scales[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int cu = c0 + u * wpt * kDotCols, c = min(cu + lane * 16, Dp - 16);
                    scales[u] = load_scales(st, nb, k0, min(B, K - k0), cu / kCkptBlock, lane, words);
#pragma unroll
                    for (int k = 0; k < B; ++k)
                        // slots past K repeat the last one: no branch, and their sums are dropped
                        w[u][k] = __ldcs(reinterpret_cast<const uint4*>(qt + c + min(k0 + k, K - 1) * Dp));
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int k = 0; k < B; ++k) {
                        const uint32_t x[4] = {w[u][k].x, w[u][k].y, w[u][k].z, w[u][k].w};
                        unsigned long long a = 0ull;
#pragma unroll
                        for (int j = 0; j < 4; ++j) dot4_pairs(x[j], f[u] + 4 * j, a);
                        float a0, a1;
                        asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
                        // lanes past the row: dy and the scale are 0
                        acc[k0 + k] = fmaf(a0 + a1, strip_step(scales[u], k, lane), acc[k0 + k]);
                    }
            }
        }
    }
    float s = warp_sum_slots<KM>(acc, lane);
    if (wpt > 1) {
        s_part[warp][lane] = s;
        __syncthreads();
        if (sub == 0)
            for (int i = 1; i < wpt; ++i) s += s_part[warp + i][lane];
    }
    if (live && sub == 0) {
        if (lane < K) s_out[o] = s;
        if (grads) {
            float gr, gl;
            slot_grads(lane < K, s, g, l, 1, reg, gr, gl);
            if (lane < K) { d_r[o] = gr; d_l[o] = gl; }
        }
    }
    pdl_launch_dependents();
}

// Segments: a CTA per decision adds the tokens' dots in 64 bits (thread = slot and every 256/KP-th token, KP
// the power of two that holds K; then the partials in thread order), and zeroes the gradients
// of the segment's other tokens.
__global__ void __launch_bounds__(kDotThreads)
ckpt_slot_grad_kernel(const float* __restrict__ s, int n_tok, int K, int kp, int S,
                      const float* __restrict__ gate, const float* __restrict__ mlogit, float reg,
                      float* __restrict__ d_r, float* __restrict__ d_l)
{
    __shared__ double s_part[kDotThreads];
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    const long long t0 = (long long)blockIdx.x * S, t1 = min((long long)n_tok, t0 + S);
    const int k = tid & (kp - 1), step = kDotThreads / kp;
    double run = 0.0;
    if (k < K)
#pragma unroll 4
        for (long long t = t0 + tid / kp; t < t1; t += step) run += __ldg(s + t * K + k);
    s_part[tid] = run;
    for (long long i = (t0 + 1) * K + tid; i < t1 * K; i += kDotThreads) { d_r[i] = 0.f; d_l[i] = 0.f; }
    __syncthreads();
    if (tid < 32) {
        const bool on = lane < K;
        run = 0.0;
        if (on)
            for (int i = 0; i < step; ++i) run += s_part[i * kp + lane];
        const float g = on ? gate[t0 * K + lane] : 0.f, l = on ? mlogit[t0 * K + lane] : 0.f;
        float gr, gl;
        slot_grads(on, (float)run, g, l, (int)(t1 - t0), reg, gr, gl);
        if (on) { d_r[t0 * K + lane] = gr; d_l[t0 * K + lane] = gl; }
    }
    pdl_launch_dependents();
}

}  // namespace beam
