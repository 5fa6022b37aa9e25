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
// Kernels (LPR lanes share a row of logits, 8 values each, so that a warp takes 32 / LPR rows at once
// and few lanes idle whatever E):
//   balance_partial_kernel   a CTA takes a run of tokens and writes, for each group that the run
//                            meets, the sums of p, the counts and the token count.  Run c and
//                            group g meet in slot c + g: along the tokens one of the two grows at
//                            every step, so the slots are distinct and fewer than runs + groups.
//                            A batch of one run and one group is finished here, in one launch.
//   balance_reduce_kernel    a CTA per group and 32 experts adds their slots in order and forms f, P
//                            and the experts' part of L_g; the last CTA to finish (a ticket) adds the
//                            parts and takes the mean over the groups.
//   balance_grad_kernel      the gradient above, and optionally the slot gradients of the routing
//                            scattered beside it; a warp's rows are put together in shared memory
//                            and leave as one contiguous piece.
// All float sums have a fixed order; the atomics count integers or elect the last CTA.
//
// Measured on B200 (device time, L2 warm; the floor is the bytes read and written at the measured copy
// rate): 64 tokens of 8 experts 3.0 us in one launch (two launches and a warp per row: 10.6);
// 16384 x 60 bf16 in 24 sequences 12.4 us (floor 0.4: two dependent launches, each a chain of five or
// six round trips to memory; adding the runs through a cluster's shared memory in one launch is not built); 65536 x 60 float32 15 us (floor 2.6; with a warp per row and one CTA to
// reduce: 164).  The gradient of 8192 x 212 with slot gradients 8.9 us (floor 3.4), of 65536 x 60 12.3 us
// (floor 4.8): two fifths of the copy rate, the rest being the softmax's two chains of shuffles per row.
#pragma once
#include "common.cuh"

namespace beam {

constexpr int kBalThreads = 256, kBalWarps = kBalThreads / 32;
constexpr int kBalPer = 8;            // logits per lane
constexpr int kBalRuns = 296;         // most runs of a large batch: two CTAs per SM
constexpr int kBalReduceThreads = 512;

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

// softmax of one row held by LPR lanes as v[j] = logit r + LPR j, r the lane's place in the row (-inf
// past E); a row without a logit above -inf has probability 0 everywhere.
template <int LPR>
__device__ __forceinline__ void bal_softmax(float* v)
{
    float m = v[0], s = 0.f, bad = 0.f;
#pragma unroll
    for (int j = 1; j < kBalPer; ++j) m = fmaxf(m, v[j]);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const bool none = m == -INFINITY;   // fmaxf passes over a NaN: such a row has -inf and NaN only
#pragma unroll
    for (int j = 0; j < kBalPer; ++j) {
        if (none) bad += isnan(v[j]) ? v[j] : 0.f;
        v[j] = none ? 0.f : expf(v[j] - m);
        s += v[j];
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        bad += __shfl_xor_sync(0xffffffffu, bad, o);
    }
    const float inv = none ? bad : 1.0f / s;
#pragma unroll
    for (int j = 0; j < kBalPer; ++j) v[j] = none ? inv : v[j] * inv;
}

template <typename T, int LPR>
__device__ __forceinline__ void bal_load(float* v, const T* __restrict__ row, int r, int E, bool on)
{
#pragma unroll
    for (int j = 0; j < kBalPer; ++j) {
        const int e = r + LPR * j;
        v[j] = on && e < E ? to_float(row[e]) : -INFINITY;
    }
}

// Sum over the block of one value per thread (blockDim a multiple of 32, at most 1024), in a fixed order; in
// all threads.
__device__ __forceinline__ float bal_block_sum(float v, float* s_w)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = v;
    __syncthreads();
    const int w = threadIdx.x & 31;
    return warp_sum(w < (int)(blockDim.x >> 5) ? s_w[w] : 0.f);
}

// prob, counts and (expert 0) tokens of one group from the sums of a thread's expert (none: e >= E), and
// the block's share of the group's loss.
__device__ __forceinline__ float bal_finish(int g, int e, int E, int K, float sum, int cnt, int n,
                                            float* __restrict__ prob, int* __restrict__ counts,
                                            int* __restrict__ tokens, float* s_w)
{
    float l = 0.f;
    if (e < E) {
        const float p = n ? sum / (float)n : 0.f;
        prob[(long long)g * E + e] = p;
        counts[(long long)g * E + e] = cnt;
        if (n) l = p * (float)((double)cnt * E / ((double)K * n));
    }
    if (e == 0) tokens[g] = n;
    return bal_block_sum(l, s_w);
}

template <typename T, int LPR>
__global__ void __launch_bounds__(kBalThreads)
balance_partial_kernel(const T* __restrict__ logits, long long ldl, int n_tok, int E, int run,
                       const int* __restrict__ topk, int K, const uint8_t* __restrict__ valid,
                       const int* __restrict__ cu, int n_seq, float* __restrict__ part_p,
                       int* __restrict__ part_c, int* __restrict__ part_n, int* __restrict__ ticket,
                       float* __restrict__ prob, int* __restrict__ counts, int* __restrict__ tokens,
                       float* __restrict__ loss)
{
    constexpr int R = 32 / LPR;                       // rows of a warp
    __shared__ float s_p[kBalWarps][LPR * kBalPer];
    __shared__ int s_c[256];
    __shared__ int s_n;
    __shared__ float s_w[kBalWarps];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane % LPR;
    const int t0 = (int)min((long long)blockIdx.x * run, (long long)n_tok);
    const int t1 = (int)min((long long)t0 + run, (long long)n_tok);
    const bool alone = gridDim.x == 1 && !cu;         // one run, one group: finished here, without scratch
    if (alone) pdl_launch_dependents();
    if (!alone && blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;
    const int g_end = cu ? n_seq : 1;
    for (int g = cu ? bal_group(cu, n_seq, t0) : 0; g < g_end; ++g) {
        const int a = cu ? max(t0, bal_bound(cu, g, n_tok)) : t0;
        const int b = cu ? min(t1, bal_bound(cu, g + 1, n_tok)) : t1;
        if (a >= t1 && !alone) break;
        if (a >= b && !alone) continue;
        if (threadIdx.x < E) s_c[threadIdx.x] = 0;
        if (threadIdx.x == 0) s_n = 0;
        __syncthreads();
        float acc[kBalPer], v[kBalPer];
#pragma unroll
        for (int j = 0; j < kBalPer; ++j) acc[j] = 0.f;
        int n = 0;
        // rows of this lane, kBalWarps * R apart; the next row is loaded before this one is used.  A row
        // that does not count is loaded like the others (no load waits for another) and dropped.
        int t = a + warp * R + lane / LPR;
        bool on = t < b && (!valid || valid[t]);
        bal_load<T, LPR>(v, logits + (long long)t * ldl, r, E, t < b);
        // counts: one thread per (token, slot)
        const int* ids = topk + (long long)a * K;
        for (int i = threadIdx.x; i < (b - a) * K; i += kBalThreads) {
            const int id = __ldg(ids + i);
            const bool counts_too = !valid || valid[a + i / K];
            if (id >= 0 && id < E && counts_too) atomicAdd(&s_c[id], 1);
        }
        for (int base = a + warp * R; base < b; base += kBalWarps * R) {
            float w[kBalPer];
            const bool cur = on;
            t += kBalWarps * R;
            on = t < b && (!valid || valid[t]);
            bal_load<T, LPR>(w, logits + (long long)t * ldl, r, E, t < b);
            bal_softmax<LPR>(v);
            if (cur) {
                ++n;
#pragma unroll
                for (int j = 0; j < kBalPer; ++j) acc[j] += v[j];
            }
#pragma unroll
            for (int j = 0; j < kBalPer; ++j) v[j] = w[j];
        }
#pragma unroll
        for (int j = 0; j < kBalPer; ++j) {
#pragma unroll
            for (int o = LPR; o < 32; o <<= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
            if (lane < LPR) s_p[warp][r + LPR * j] = acc[j];
        }
        if (r == 0 && n) atomicAdd(&s_n, n);
        __syncthreads();
        const int e = threadIdx.x;
        float sum = 0.f;
        if (e < E)
#pragma unroll
            for (int w = 0; w < kBalWarps; ++w) sum += s_p[w][e];
        if (alone) {
            const float l = bal_finish(0, e, E, K, sum, e < E ? s_c[e] : 0, s_n, prob, counts, tokens, s_w);
            if (threadIdx.x == 0) *loss = l;
            break;
        }
        const long long slot = (long long)blockIdx.x + g;
        if (e < E) {
            part_p[slot * E + e] = sum;
            part_c[slot * E + e] = s_c[e];
        }
        if (e == 0) part_n[slot] = s_n;
        __syncthreads();
    }
    if (!alone) pdl_launch_dependents();
}

// EP: the power of two that holds min(E, 32); 512 / EP threads share an expert's slots.  (One CTA per
// group would read all slots through one SM: 600 KB for 16384 tokens of 256 experts.)
__global__ void __launch_bounds__(kBalReduceThreads)
balance_reduce_kernel(const float* __restrict__ part_p, const int* __restrict__ part_c,
                      const int* __restrict__ part_n, int n_tok, int E, int EP, int K, int run,
                      const int* __restrict__ cu, float* __restrict__ loss_part,
                      int* __restrict__ ticket, float* __restrict__ prob, int* __restrict__ counts,
                      int* __restrict__ tokens, float* __restrict__ loss)
{
    __shared__ float s_p[kBalReduceThreads];
    __shared__ int s_c[kBalReduceThreads];
    __shared__ float s_w[kBalReduceThreads / 32];
    __shared__ int s_n, s_last;
    pdl_wait();
    const int g = blockIdx.x, tid = threadIdx.x, e0 = blockIdx.y * 32;
    const int a = cu ? bal_bound(cu, g, n_tok) : 0, b = cu ? bal_bound(cu, g + 1, n_tok) : n_tok;
    const int c0 = a / run, c1 = b > a ? (b - 1) / run + 1 : c0;
    if (tid == 0) s_n = 0;
    __syncthreads();
    int n = 0;
    for (int c = c0 + tid; c < c1; c += kBalReduceThreads) n += part_n[c + g];
    if (n) atomicAdd(&s_n, n);
    const int e = e0 + (tid & (EP - 1)), subs = kBalReduceThreads / EP, sub = tid / EP;
    float sum = 0.f;
    int cnt = 0;
    if (e < E) {
        constexpr int B = 8;   // slots in flight (most groups have no more per thread)
        for (int b0 = c0 + sub; b0 < c1; b0 += B * subs) {
            float p[B];
            int k[B];
#pragma unroll
            for (int j = 0; j < B; ++j) {
                const int c = b0 + j * subs;
                p[j] = c < c1 ? __ldg(part_p + (long long)(c + g) * E + e) : 0.f;
                k[j] = c < c1 ? __ldg(part_c + (long long)(c + g) * E + e) : 0;
            }
#pragma unroll
            for (int j = 0; j < B; ++j) { sum += p[j]; cnt += k[j]; }
        }
    }
    s_p[tid] = sum;
    s_c[tid] = cnt;
    __syncthreads();
    // halve the threads that share an expert until one is left: the same order whatever the timing
    for (int o = kBalReduceThreads / 2; o >= EP; o >>= 1) {
        if (tid < o) { s_p[tid] += s_p[tid + o]; s_c[tid] += s_c[tid + o]; }
        __syncthreads();
    }
    const float l = bal_finish(g, tid < EP ? e : E, E, K, s_p[tid], s_c[tid], s_n, prob, counts, tokens, s_w);
    if (tid == 0) {
        loss_part[(long long)g * gridDim.y + blockIdx.y] = l;
        __threadfence();
        s_last = atomicAdd(ticket, 1) == (int)(gridDim.x * gridDim.y) - 1;
    }
    __syncthreads();
    if (s_last) {
        __threadfence();
        float s = 0.f, act = 0.f;
        for (long long i = tid; i < (long long)gridDim.x * gridDim.y; i += kBalReduceThreads) s += __ldcg(loss_part + i);
        for (int i = tid; i < (int)gridDim.x; i += kBalReduceThreads) act += __ldcg(tokens + i) > 0 ? 1.f : 0.f;
        s = bal_block_sum(s, s_w);
        act = bal_block_sum(act, s_w);
        if (tid == 0) *loss = act > 0.f ? s / act : 0.f;
    }
    pdl_launch_dependents();
}

// One (row of the warp, slot) pair per lane: its expert and gradients.
struct BalSlot { int id; float gr, gl; };
__device__ __forceinline__ BalSlot bal_slot(int i, int n, const int* __restrict__ ids, const float* __restrict__ d_r,
                                            const float* __restrict__ d_l)
{
    BalSlot s = {-1, 0.f, 0.f};
    if (i < n) s = {__ldg(ids + i), __ldg(d_r + i), __ldg(d_l + i)};
    return s;
}
// Adds the lanes' pairs to the rows in shared memory (row = pair / K), in slot order where a row has
// chosen an expert twice.
__device__ __forceinline__ void bal_add_slots(float* rows, const BalSlot& s, int row, int E, int lane)
{
    const bool on = s.id >= 0 && s.id < E;
    const int key = on ? row * 256 + s.id : -1 - lane;
    const unsigned same = __match_any_sync(0xffffffffu, key);
    const bool twice = __any_sync(0xffffffffu, (same & (same - 1)) != 0);
    float* p = rows + row * 2 * E + s.id;
    if (!twice) {
        if (on) { p[0] += s.gr; p[E] += s.gl; }
    } else {
        for (int k = 0; k < 32; ++k) {
            if (lane == k && on) { p[0] += s.gr; p[E] += s.gl; }
            __syncwarp();
        }
    }
    __syncwarp();
}

template <typename T, int LPR>
__global__ void __launch_bounds__(kBalThreads)
balance_grad_kernel(const T* __restrict__ logits, long long ldl, int n_tok, int E, int run,
                    const int* __restrict__ topk, int K, const uint8_t* __restrict__ valid,
                    const int* __restrict__ cu, int n_seq, const int* __restrict__ counts,
                    const int* __restrict__ tokens, float scale, const float* __restrict__ d_r,
                    const float* __restrict__ d_l, float* __restrict__ out)
{
    constexpr int R = 32 / LPR;
    __shared__ __align__(16) float s_rows[kBalWarps][R * 2 * LPR * kBalPer];   // read as float4
    __shared__ int s_act;
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane % LPR;
    const int G = cu ? n_seq : 1;
    if (threadIdx.x == 0) s_act = 0;
    __syncthreads();
    int act = 0;
    if (G > 1) {
        for (int i = threadIdx.x; i < G; i += kBalThreads) act += tokens[i] > 0;
        if (act) atomicAdd(&s_act, act);
    }
    const long long t0 = (long long)blockIdx.x * run, t1 = min(t0 + run, (long long)n_tok);
    int g = cu ? bal_group(cu, n_seq, (int)t0) : 0;   // moves on with the lane's rows
    float v[kBalPer], f[kBalPer];
    float coef = 0.f;
    int g_of_f = -1;
    const int width = d_r ? 2 * E : E;
    float* rows = s_rows[warp];
    long long t = t0 + warp * R + lane / LPR;
    bool here = t < t1;
    bal_load<T, LPR>(v, logits + t * ldl, r, E, here);
    __syncthreads();
    act = G > 1 ? s_act : 1;   // one group: the tokens that use it make it a non-empty one
    for (long long base = t0 + warp * R; base < t1; base += kBalWarps * R) {
        // the row's group, and f of that group where it is another than the last row's
        bool in = here && (!valid || valid[t]);
        if (cu && in) {
            while (g < G && __ldg(cu + g + 1) <= t) ++g;
            in = g < G && bal_bound(cu, g, n_tok) <= t;
        }
        if (in && g != g_of_f) {
            const int n = tokens[g];
            const float inv_kn = n > 0 ? 1.0f / ((float)K * (float)n) : 0.f;
            coef = n > 0 ? scale / ((float)act * (float)n) : 0.f;
#pragma unroll
            for (int j = 0; j < kBalPer; ++j) {
                const int e = r + LPR * j;
                f[j] = e < E ? (float)((long long)counts[(long long)g * E + e] * E - (long long)K * n) * inv_kn : 0.f;
            }
            g_of_f = g;
        }
        float w[kBalPer];
        const bool cur = in && coef != 0.f;
        // the first 32 slots of the warp's rows, on their way while the softmax runs
        const int n_rows = (int)min((long long)R, t1 - base), n_slots = d_r ? n_rows * K : 0;
        const int* ids = topk + base * K;
        const float *gr = d_r + base * K, *gl = d_l + base * K;
        const BalSlot first = bal_slot(lane, n_slots, ids, gr, gl);
        t += kBalWarps * R;
        here = t < t1;
        bal_load<T, LPR>(w, logits + t * ldl, r, E, here);
        bal_softmax<LPR>(v);
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < kBalPer; ++j) dot += cur ? f[j] * v[j] : 0.f;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        float* row = rows + (lane / LPR) * width;
#pragma unroll
        for (int j = 0; j < kBalPer; ++j) {
            const int e = r + LPR * j;
            if (e < E) {
                row[e] = cur ? coef * v[j] * (f[j] - dot) : 0.f;
                if (d_r) row[E + e] = 0.f;
            }
        }
        __syncwarp();
        if (d_r) {
            bal_add_slots(rows, first, lane / K, E, lane);
            for (int i = 32; i < n_slots; i += 32)
                bal_add_slots(rows, bal_slot(i + lane, n_slots, ids, gr, gl), (i + lane) / K, E, lane);
        }
        // the rows are contiguous in memory
        float* o = out + base * width;
        const int total = n_rows * width;
        if ((reinterpret_cast<uintptr_t>(o) & 15) == 0 && (total & 3) == 0) {
            for (int i = lane; i < total / 4; i += 32)
                reinterpret_cast<float4*>(o)[i] = reinterpret_cast<const float4*>(rows)[i];
        } else {
            for (int i = lane; i < total; i += 32) o[i] = rows[i];
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kBalPer; ++j) v[j] = w[j];
    }
    pdl_launch_dependents();
}

}  // namespace beam
