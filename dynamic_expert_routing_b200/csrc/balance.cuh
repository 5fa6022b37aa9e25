// balance.cuh -- the load-balance loss L_bal of the training objective L = L_lm + alpha L_bal +
// beta L_reg (BEAM article on aitrends.kr, training paragraph, which names the term without a
// formula): the widely used product of an expert's share of the assignments and its mean
// router probability.  Over the valid tokens of a group g (the whole batch, or one of the packed
// sequences), with p_t = softmax(logits_t) and K slots per token:
//   n_g tokens;  c_ge = slots that chose expert e;  f_ge = c_ge E / (K n_g)
//   P_ge = (1 / n_g) sum_t p_te;  L_bal = mean over the non-empty groups of sum_e f_ge P_ge
// (1 for a uniform assignment).  f is a count, so the gradient goes through P alone:
//   dlogits_tj = scale / (G' n_g) p_tj (f_gj - sum_i f_gi p_ti),  G' = non-empty groups.
// Replacing f by f - 1 = (c E - K n) / (K n) leaves that gradient unchanged (sum_j p_tj = 1) and
// removes the cancellation of two numbers near 1: the numerator is an exact integer.
//
// Kernels:
//   balance_partial_kernel   a CTA takes a fixed run of tokens and writes, for each group that
//                            the run meets, the sums of p, the counts and the token count.
//                            Run c and group g meet in slot c + g: along the tokens one of the
//                            two grows at every step, so the slots are distinct and fewer than
//                            runs + groups.
//   balance_reduce_kernel    a CTA per group adds its slots in order and forms f, P and L_g; the
//                            last CTA to finish (a ticket) takes the mean over the groups.
//   balance_grad_kernel      a warp per token: the gradient above, and optionally the scattered
//                            slot gradients of the routing beside it.
// All float sums have a fixed order; the atomics count integers or elect the last CTA.
#pragma once
#include "common.cuh"

namespace beam {

constexpr int kBalRun = 64;      // tokens per CTA of the first pass
constexpr int kBalThreads = 256;

// Group bounds [cu[g], cu[g+1]) clamped to the batch; one group [0, T) without cu.
__device__ __forceinline__ int bal_bound(const int* __restrict__ cu, int g, int T)
{
    return min(max(__ldg(cu + g), 0), T);
}
// The first group whose end is past token t (n_seq when t is behind the last sequence).
__device__ __forceinline__ int bal_group(const int* __restrict__ cu, int n_seq, int t)
{
    int lo = 0, hi = n_seq;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(cu + mid + 1) > t) hi = mid; else lo = mid + 1;
    }
    return lo;
}

// softmax of one row held as v[j] = logit lane + 32 j (-inf past E); a row without a logit
// above -inf has probability 0 everywhere.
template <int EPL>
__device__ __forceinline__ void bal_softmax(float* v)
{
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) m = fmaxf(m, v[j]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) {
        // fmaxf ignores a NaN: only a row of -inf alone is empty
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) t += isnan(v[j]) ? v[j] : 0.f;
        t = warp_sum(t);
#pragma unroll
        for (int j = 0; j < EPL; ++j) v[j] = t;
        return;
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) { v[j] = expf(v[j] - m); s += v[j]; }
    s = warp_sum(s);
    const float inv = 1.0f / s;
#pragma unroll
    for (int j = 0; j < EPL; ++j) v[j] *= inv;
}

template <typename T, int EPL>
__global__ void __launch_bounds__(kBalThreads)
balance_partial_kernel(const T* __restrict__ logits, long long ldl, int n_tok, int E,
                       const int* __restrict__ topk, int K, const uint8_t* __restrict__ valid,
                       const int* __restrict__ cu, int n_seq, float* __restrict__ part_p,
                       int* __restrict__ part_c, int* __restrict__ part_n, int* __restrict__ ticket)
{
    __shared__ float s_p[kBalThreads / 32][EPL * 32];
    __shared__ int s_c[EPL * 32];
    __shared__ int s_n;
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
    const int t0 = blockIdx.x * kBalRun, t1 = min(n_tok, t0 + kBalRun);
    const int g_end = cu ? n_seq : 1;
    for (int g = cu ? bal_group(cu, n_seq, t0) : 0; g < g_end; ++g) {
        const int a = cu ? max(t0, bal_bound(cu, g, n_tok)) : t0;
        const int b = cu ? min(t1, bal_bound(cu, g + 1, n_tok)) : t1;
        if (a >= t1) break;
        if (a >= b) continue;
        for (int e = threadIdx.x; e < E; e += kBalThreads) s_c[e] = 0;
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
        float acc[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
        int n = 0;
        for (int t = a + warp; t < b; t += kBalThreads / 32) {
            if (valid && !valid[t]) continue;
            ++n;
            float v[EPL];
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int e = lane + 32 * j;
                v[j] = e < E ? to_float(logits[(long long)t * ldl + e]) : -INFINITY;
            }
            bal_softmax<EPL>(v);
#pragma unroll
            for (int j = 0; j < EPL; ++j) acc[j] += v[j];
            if (lane < K) {
                const int id = topk[(long long)t * K + lane];
                if (id >= 0 && id < E) atomicAdd(&s_c[id], 1);
            }
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) s_p[warp][lane + 32 * j] = acc[j];
        if (lane == 0 && n) atomicAdd(&s_n, n);
        __syncthreads();
        const long long slot = (long long)blockIdx.x + g;
        for (int e = threadIdx.x; e < E; e += kBalThreads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kBalThreads / 32; ++w) s += s_p[w][e];
            part_p[slot * E + e] = s;
            part_c[slot * E + e] = s_c[e];
        }
        if (threadIdx.x == 0) part_n[slot] = s_n;
        __syncthreads();
    }
    pdl_launch_dependents();
}

__global__ void __launch_bounds__(256)
balance_reduce_kernel(const float* __restrict__ part_p, const int* __restrict__ part_c,
                      const int* __restrict__ part_n, int n_tok, int E, int K,
                      const int* __restrict__ cu, float* __restrict__ loss_g,
                      int* __restrict__ ticket, float* __restrict__ prob, int* __restrict__ counts,
                      int* __restrict__ tokens, float* __restrict__ loss)
{
    __shared__ float s_l[8];
    __shared__ int s_n, s_last;
    pdl_wait();
    const int g = blockIdx.x;
    const int a = cu ? bal_bound(cu, g, n_tok) : 0, b = cu ? bal_bound(cu, g + 1, n_tok) : n_tok;
    const int c0 = a / kBalRun, c1 = b > a ? (b - 1) / kBalRun + 1 : c0;
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    int n = 0;
    for (int c = c0 + threadIdx.x; c < c1; c += blockDim.x) n += part_n[c + g];
    if (n) atomicAdd(&s_n, n);
    __syncthreads();
    n = s_n;
    float l = 0.f;
    const int e = threadIdx.x;
    if (e < E) {
        float s = 0.f;
        int cnt = 0;
        for (int c = c0; c < c1; ++c) {
            s += part_p[(long long)(c + g) * E + e];
            cnt += part_c[(long long)(c + g) * E + e];
        }
        const float p = n ? s / (float)n : 0.f;
        prob[(long long)g * E + e] = p;
        counts[(long long)g * E + e] = cnt;
        if (n) l = p * ((float)((double)cnt * E / ((double)K * n)));
    }
    l = warp_sum(l);
    if ((threadIdx.x & 31) == 0) s_l[threadIdx.x >> 5] = l;
    __syncthreads();
    if (threadIdx.x == 0) {
        float s = 0.f;
        for (int w = 0; w < 8; ++w) s += s_l[w];
        loss_g[g] = s;
        tokens[g] = n;
        __threadfence();
        s_last = atomicAdd(ticket, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (s_last && threadIdx.x < 32) {
        __threadfence();
        float s = 0.f;
        int act = 0;
        for (int i = threadIdx.x; i < (int)gridDim.x; i += 32) {
            s += __ldcg(loss_g + i);
            act += __ldcg(tokens + i) > 0;
        }
        s = warp_sum(s);
        act = __reduce_add_sync(0xffffffffu, act);
        if (threadIdx.x == 0) *loss = act ? s / (float)act : 0.f;
    }
    pdl_launch_dependents();
}

template <typename T, int EPL>
__global__ void __launch_bounds__(kBalThreads)
balance_grad_kernel(const T* __restrict__ logits, long long ldl, int n_tok, int E,
                    const int* __restrict__ topk, int K, const uint8_t* __restrict__ valid,
                    const int* __restrict__ cu, int n_seq, const int* __restrict__ counts,
                    const int* __restrict__ tokens, float scale, const float* __restrict__ d_r,
                    const float* __restrict__ d_l, float* __restrict__ out)
{
    __shared__ int s_act;
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) s_act = 0;
    __syncthreads();
    const int G = cu ? n_seq : 1;
    int act = 0;
    for (int i = threadIdx.x; i < G; i += kBalThreads) act += tokens[i] > 0;
    if (act) atomicAdd(&s_act, act);
    __syncthreads();
    act = s_act;
    const long long t = (long long)blockIdx.x * (kBalThreads / 32) + warp;
    if (t < n_tok) {
        float d[EPL], dm[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) d[j] = dm[j] = 0.f;
        const int g = cu ? bal_group(cu, n_seq, (int)t) : 0;
        const bool in = g < G && (!cu || bal_bound(cu, g, n_tok) <= t) && (!valid || valid[t]);
        const int n = in ? tokens[g] : 0;
        if (n > 0) {
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int e = lane + 32 * j;
                d[j] = e < E ? to_float(logits[t * ldl + e]) : -INFINITY;
            }
            bal_softmax<EPL>(d);
            const float inv_kn = 1.0f / ((float)K * (float)n);
            float f[EPL], dot = 0.f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int e = lane + 32 * j;
                f[j] = e < E ? (float)((long long)counts[(long long)g * E + e] * E - (long long)K * n) * inv_kn : 0.f;
                dot += f[j] * d[j];
            }
            dot = warp_sum(dot);
            const float coef = scale / ((float)act * (float)n);
#pragma unroll
            for (int j = 0; j < EPL; ++j) d[j] = coef * d[j] * (f[j] - dot);
        }
        const int ldo = d_r ? 2 * E : E;
        if (d_r) {
            for (int k = 0; k < K; ++k) {
                const long long o = t * K + k;
                const int id = topk[o];
                const float gr = d_r[o], gl = d_l[o];
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    if (id == lane + 32 * j) { d[j] += gr; dm[j] += gl; }
            }
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane + 32 * j;
            if (e < E) {
                out[t * ldo + e] = d[j];
                if (d_r) out[t * ldo + E + e] = dm[j];
            }
        }
    }
    pdl_launch_dependents();
}

}  // namespace beam
