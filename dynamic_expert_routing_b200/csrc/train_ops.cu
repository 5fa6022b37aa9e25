// train_ops.cu -- C ABI of the training operators that belong to no handle: the load-balance loss,
// 8-bit activation checkpoints, the routing's slot gradients from a checkpoint and the router's
// linear backward.  Every call enqueues its kernels on the given stream and allocates nothing;
// scratch comes from the caller.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "host.cuh"
#include "balance.cuh"
#include "checkpoint.cuh"
#include "ckpt_route_grad.cuh"
#include "router_linear.cuh"

using namespace beam;

#define FAIL_ARG(...) return beam_host_fail(BEAM_ERR_INVALID_ARG, __VA_ARGS__)
#define TRY(call)                                \
    do {                                         \
        const beam_status_t s_ = (call);         \
        if (s_ != BEAM_OK) return s_;            \
    } while (0)

constexpr int kMaxExperts = 256, kMaxSlots = 32, kMaxWidth = 65536, kMaxLogits = 1 << 20;

static long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
static long long align256(long long n) { return (n + 255) & ~255LL; }

static int elem_size(int dtype)
{
    return dtype == BEAM_DTYPE_F32 ? 4 : (dtype == BEAM_DTYPE_BF16 || dtype == BEAM_DTYPE_F16) ? 2 : 0;
}
static bool misaligned(const void* p, int a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// A row-major input of `rows` rows of `cols` values, rows ld apart.
static beam_status_t check_matrix(const char* name, const void* p, int dtype, bool f16, long long rows,
                                  long long cols, long long ld)
{
    if (!elem_size(dtype) || (dtype == BEAM_DTYPE_F16 && !f16))
        FAIL_ARG("%s: unsupported data type %d", name, dtype);
    if (ld < cols) FAIL_ARG("%s: row stride %lld is below its %lld columns", name, ld, cols);
    if (rows > 0 && cols > 0 && !p) FAIL_ARG("%s is NULL", name);
    if (misaligned(p, elem_size(dtype))) FAIL_ARG("%s is not aligned to its elements", name);
    return BEAM_OK;
}

static beam_status_t check_ckpt(const int8_t* q, const uint8_t* scale, long long rows, int d)
{
    if (d < 1 || d > kMaxWidth) FAIL_ARG("checkpoint: d=%d must be in [1, %d]", d, kMaxWidth);
    if (rows < 0 || rows > (1LL << 31) - 1) FAIL_ARG("checkpoint: %lld rows are out of range", rows);
    if (rows > 0 && (!q || !scale)) FAIL_ARG("checkpoint: q or scale is NULL");
    if (misaligned(q, 16)) FAIL_ARG("checkpoint: q must be 16-byte aligned");
    return BEAM_OK;
}

// Calls f(T()) with the C++ type of a data type that check_matrix accepted.
template <typename F>
static cudaError_t with_type(int dtype, F f)
{
    if (dtype == BEAM_DTYPE_F32) return f(float());
    return f(__nv_bfloat16());
}
template <typename F>
static cudaError_t with_type3(int dtype, F f)
{
    if (dtype == BEAM_DTYPE_F16) return f(__half());
    return with_type(dtype, f);
}

// SMs of the current device.
static int num_sms()
{
    static std::atomic<int> cached[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 1;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// ---------------------------------------------------------------- balance loss
struct BalArgs {
    const void* logits; int dtype, T, E; long long ldl; const int32_t* topk; int K;
    const uint8_t* valid; const int32_t* cu; int n_seq;
};

// ids: whether topk_id is read.
static beam_status_t check_balance(const BalArgs& a, bool ids)
{
    if (a.T < 0 || a.T > (1 << 30)) FAIL_ARG("T=%d outside [0, 2^30]", a.T);
    if (a.E < 1 || a.E > kMaxExperts) FAIL_ARG("E=%d must be in [1, %d]", a.E, kMaxExperts);
    if (a.K < 1 || a.K > kMaxSlots) FAIL_ARG("K=%d must be in [1, %d]", a.K, kMaxSlots);
    if ((long long)a.T * a.K > (1LL << 31) - 1) FAIL_ARG("T*K=%lld assignments are too many for int32 counts", (long long)a.T * a.K);
    if (a.cu ? (a.n_seq < 1 || a.n_seq > 65536) : a.n_seq != 0)
        FAIL_ARG("n_seq=%d: 1 to 65536 sequences with cu_seqlens, 0 without", a.n_seq);
    TRY(check_matrix("logits", a.logits, a.dtype, false, a.T, a.E, a.ldl));
    if (ids && a.T > 0 && !a.topk) FAIL_ARG("topk_id is NULL");
    if (misaligned(a.topk, 4) || misaligned(a.cu, 4)) FAIL_ARG("the int32 arrays must be 4-byte aligned");
    return BEAM_OK;
}

// Lanes that share a row of E logits, 8 values each.
static int bal_lanes(int E)
{
    int l = 1;
    while (l * kBalPer < E) l *= 2;
    return l;
}
// Tokens of a run: whole passes of a CTA's rows, as few as keep the runs at kBalRuns or below.
static int bal_run(int T, int E)
{
    const long long pass = (long long)kBalWarps * (32 / bal_lanes(E));
    return (int)std::max(pass, ceil_div(ceil_div(T, kBalRuns), pass) * pass);
}
static long long bal_runs(int T, int E) { return std::max(1LL, ceil_div(T, bal_run(T, E))); }

// Workspace: part_p, part_c [slots][E], part_n [slots], the groups' losses, the ticket.
struct BalWork { long long slots, p, c, n, lg, ticket, bytes; };
static BalWork bal_work(int T, int E, int n_seq)
{
    BalWork w;
    const int G = std::max(1, n_seq);
    w.slots = bal_runs(T, E) + G;
    w.p = 0;
    w.c = align256(w.p + w.slots * E * 4);
    w.n = align256(w.c + w.slots * E * 4);
    w.lg = align256(w.n + w.slots * 4);
    w.ticket = align256(w.lg + G * ceil_div(E, 32) * 4);
    w.bytes = w.ticket + 256;
    if (bal_runs(T, E) == 1 && n_seq == 0) w.bytes = 0;   // finished by its only CTA
    return w;
}

// Calls FN<T, LPR>(...) for the row width.
#define BAL_DISPATCH(FN, ...)                                                                   \
    with_type(a.dtype, [&](auto z) -> cudaError_t {                                             \
        using T_ = decltype(z);                                                                 \
        switch (bal_lanes(a.E)) {                                                               \
            case 1: return FN<T_, 1>(__VA_ARGS__);                                              \
            case 2: return FN<T_, 2>(__VA_ARGS__);                                              \
            case 4: return FN<T_, 4>(__VA_ARGS__);                                              \
            case 8: return FN<T_, 8>(__VA_ARGS__);                                              \
            case 16: return FN<T_, 16>(__VA_ARGS__);                                            \
            default: return FN<T_, 32>(__VA_ARGS__);                                            \
        }                                                                                       \
    })

struct BalOut { float *loss, *prob; int32_t *counts, *tokens; };

template <typename T, int LPR>
static cudaError_t launch_balance(const BalArgs& a, char* ws, const BalWork& w, const BalOut& o, cudaStream_t st)
{
    return launch_free(balance_partial_kernel<T, LPR>, dim3((unsigned)bal_runs(a.T, a.E)), dim3(kBalThreads), 0, st,
                       (const T*)a.logits, a.ldl, a.T, a.E, bal_run(a.T, a.E), a.topk, a.K, a.valid, a.cu, a.n_seq,
                       (float*)(ws + w.p), (int*)(ws + w.c), (int*)(ws + w.n), (int*)(ws + w.ticket), o.prob,
                       o.counts, o.tokens, o.loss);
}

template <typename T, int LPR>
static cudaError_t launch_balance_grad(const BalArgs& a, const int32_t* counts, const int32_t* tokens, float scale,
                                       const float* dr, const float* dl, float* out, cudaStream_t st)
{
    // as many CTAs as are resident (four per SM): 8192 x 212 with slots 8.9 us, with eight per SM 9.4, two 10.8
    const long long pass = (long long)kBalWarps * (32 / LPR);
    const int run = (int)std::max(pass, ceil_div(ceil_div(a.T, num_sms() * 4), pass) * pass);
    return launch_free(balance_grad_kernel<T, LPR>, dim3((unsigned)ceil_div(a.T, run)), dim3(kBalThreads), 0, st,
                       (const T*)a.logits, a.ldl, a.T, a.E, run, a.topk, a.K, a.valid, a.cu, a.n_seq, counts, tokens,
                       scale, dr, dl, out);
}

extern "C" {

int64_t beam_balance_workspace(int32_t T, int32_t E, int32_t n_seq)
{
    if (T < 0 || T > (1 << 30) || E < 1 || E > kMaxExperts || n_seq < 0 || n_seq > 65536) return -1;
    return bal_work(T, E, n_seq).bytes;
}

beam_status_t beam_balance_forward(const void* logits, int32_t dtype, int32_t T, int32_t E,
                                   int64_t ld_logits, const int32_t* topk_id, int32_t K,
                                   const uint8_t* valid, const int32_t* cu_seqlens, int32_t n_seq,
                                   float* loss, float* prob, int32_t* counts, int32_t* tokens,
                                   void* workspace, int64_t workspace_bytes, void* stream)
{
    beam_host_clear_error();
    const BalArgs a{logits, dtype, T, E, ld_logits, topk_id, K, valid, cu_seqlens, n_seq};
    TRY(check_balance(a, true));
    if (!loss || !prob || !counts || !tokens) FAIL_ARG("an output pointer is NULL");
    if (misaligned(loss, 4) || misaligned(prob, 4) || misaligned(counts, 4) || misaligned(tokens, 4))
        FAIL_ARG("the outputs must be 4-byte aligned");
    const BalWork w = bal_work(T, E, n_seq);
    if (w.bytes > 0 && (!workspace || workspace_bytes < w.bytes || misaligned(workspace, 16)))
        FAIL_ARG("the workspace must be 16-byte aligned and hold %lld bytes", w.bytes);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    const BalOut o{loss, prob, counts, tokens};
    BEAM_HOST_CUDA(BAL_DISPATCH(launch_balance, a, ws, w, o, st));
    if (w.bytes == 0) return BEAM_OK;
    int ep = 1;
    while (ep < std::min(E, 32)) ep *= 2;
    const dim3 grid((unsigned)std::max(1, n_seq), (unsigned)ceil_div(E, 32));
    BEAM_HOST_CUDA(launch_free(balance_reduce_kernel, grid, dim3(kBalReduceThreads), 0,
                               st, (const float*)(ws + w.p), (const int*)(ws + w.c), (const int*)(ws + w.n), T, E, ep,
                               K, bal_run(T, E), cu_seqlens, (float*)(ws + w.lg), (int*)(ws + w.ticket), prob, counts,
                               tokens, loss));
    return BEAM_OK;
}

beam_status_t beam_balance_backward(const void* logits, int32_t dtype, int32_t T, int32_t E,
                                    int64_t ld_logits, const int32_t* topk_id, int32_t K,
                                    const uint8_t* valid, const int32_t* cu_seqlens, int32_t n_seq,
                                    const int32_t* counts, const int32_t* tokens, float scale,
                                    const float* d_gate_logit, const float* d_mask_logit,
                                    float* dlogits, void* stream)
{
    beam_host_clear_error();
    const BalArgs a{logits, dtype, T, E, ld_logits, topk_id, K, valid, cu_seqlens, n_seq};
    TRY(check_balance(a, d_gate_logit != nullptr));
    if (!std::isfinite(scale)) FAIL_ARG("scale must be finite");
    if (!d_gate_logit != !d_mask_logit) FAIL_ARG("d_gate_logit and d_mask_logit come together");
    if (T > 0 && (!counts || !tokens || !dlogits)) FAIL_ARG("counts, tokens and dlogits are required");
    if (misaligned(counts, 4) || misaligned(tokens, 4) || misaligned(dlogits, 4) || misaligned(d_gate_logit, 4) ||
        misaligned(d_mask_logit, 4))
        FAIL_ARG("the arrays must be 4-byte aligned");
    if (T == 0) return BEAM_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    BEAM_HOST_CUDA(BAL_DISPATCH(launch_balance_grad, a, counts, tokens, scale, d_gate_logit, d_mask_logit, dlogits, st));
    return BEAM_OK;
}

// ---------------------------------------------------------------- 8-bit checkpoints
}  // extern "C"

static dim3 ckpt_grid(long long units, int unroll)
{
    return dim3((unsigned)ceil_div(units, kCkptThreads * unroll));
}

extern "C" {

beam_status_t beam_checkpoint_save(const void* x, int32_t dtype, int64_t rows, int32_t d, int64_t ld_x,
                                   int8_t* q, uint8_t* scale, void* stream)
{
    beam_host_clear_error();
    TRY(check_ckpt(q, scale, rows, d));
    TRY(check_matrix("x", x, dtype, true, rows, d, ld_x));
    if (rows == 0) return BEAM_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int nb = (int)ceil_div(d, kCkptBlock);
    BEAM_HOST_CUDA(with_type3(dtype, [&](auto z) {
        using T = decltype(z);
        constexpr int V = Vec<T>::N;
        const bool aligned = !misaligned(x, 16) && ld_x % V == 0;
        auto kernel = !aligned                           ? ckpt_save_kernel<T, CKPT_ANY>
                      : ld_x == d && d % kCkptBlock == 0 ? ckpt_save_kernel<T, CKPT_FLAT>
                      : d % V == 0                       ? ckpt_save_kernel<T, CKPT_ROWS>
                                                         : ckpt_save_kernel<T, CKPT_TAIL>;
        return launch_free(kernel, ckpt_grid(rows * nb * (kCkptBlock / V), aligned ? kCkptUnroll : 2), dim3(kCkptThreads),
                           0, st, (const T*)x, (long long)ld_x, (long long)rows, d, nb, q, scale);
    }));
    return BEAM_OK;
}

beam_status_t beam_checkpoint_load(const int8_t* q, const uint8_t* scale, int64_t rows, int32_t d, void* y,
                                   int32_t dtype, void* stream)
{
    beam_host_clear_error();
    TRY(check_ckpt(q, scale, rows, d));
    TRY(check_matrix("y", y, dtype, true, rows, d, d));
    if (misaligned(y, 16)) FAIL_ARG("y must be 16-byte aligned");
    if (rows == 0) return BEAM_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int nb = (int)ceil_div(d, kCkptBlock);
    BEAM_HOST_CUDA(with_type3(dtype, [&](auto z) {
        using T = decltype(z);
        constexpr int V = Vec<T>::N;
        auto kernel = d % kCkptBlock == 0 ? ckpt_load_kernel<T, CKPT_FLAT>
                      : d % V == 0        ? ckpt_load_kernel<T, CKPT_ROWS>
                                          : ckpt_load_any_kernel<T>;
        const long long units = d % V == 0 ? rows * nb * (kCkptBlock / V) : ceil_div(rows * d, V);
        return launch_free(kernel, ckpt_grid(units, kCkptUnroll), dim3(kCkptThreads), 0, st, q, scale, (long long)rows, d,
                           nb, (T*)y);
    }));
    return BEAM_OK;
}

// ---------------------------------------------------------------- slot gradients from a checkpoint
beam_status_t beam_checkpoint_route_grad(const int8_t* q, const uint8_t* scale, int32_t T, int32_t K, int32_t d,
                                         const float* gate, const float* mask_logit, const void* dy, int32_t dtype,
                                         int64_t ld_dy, int32_t segment_len, float reg_scale, float* dghat,
                                         float* d_gate_logit, float* d_mask_logit, void* stream)
{
    beam_host_clear_error();
    if (T < 0) FAIL_ARG("T=%d is negative", T);
    if (K < 1 || K > kMaxSlots) FAIL_ARG("K=%d must be in [1, %d]", K, kMaxSlots);
    TRY(check_ckpt(q, scale, (long long)T * K, d));
    TRY(check_matrix("dy", dy, dtype, false, T, d, ld_dy));
    if (segment_len < 0 || segment_len > 65536) FAIL_ARG("segment_len=%d outside [0, 65536]", segment_len);
    if (!std::isfinite(reg_scale)) FAIL_ARG("reg_scale must be finite");
    if (T > 0 && (!gate || !mask_logit || !dghat || !d_gate_logit || !d_mask_logit))
        FAIL_ARG("gate, mask_logit and the outputs are required");
    if (misaligned(gate, 4) || misaligned(mask_logit, 4) || misaligned(dghat, 4) || misaligned(d_gate_logit, 4) ||
        misaligned(d_mask_logit, 4))
        FAIL_ARG("the float32 arrays must be 4-byte aligned");
    if (T == 0) return BEAM_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int S = std::max(1, segment_len), nb = (int)ceil_div(d, kCkptBlock);
    const float reg = (float)((double)reg_scale / ((double)T * K));
    // warps per token: the fewest that give every SM 16 warps, as long as each has a strip of columns
    int wpt = 1;
    const int enough = num_sms() * 16;
    while (wpt < kDotWarps && (long long)T * wpt < enough && wpt * kDotCols < d) wpt *= 2;
    const bool grads = S == 1;
    BEAM_HOST_CUDA(with_type(dtype, [&](auto z) {
        using TY = decltype(z);
        auto go = [&](auto kernel) {
            return launch_free(kernel, dim3((unsigned)ceil_div(T, kDotWarps / wpt)), dim3(kDotThreads), 0, st, q, scale, T,
                               K, d, nb, (const TY*)dy, (long long)ld_dy, (int)(!misaligned(dy, 16) && ld_dy % Vec<TY>::N == 0),
                               wpt, gate, mask_logit, reg, (int)grads, dghat, d_gate_logit, d_mask_logit);
        };
        if (K <= 2 && d > wpt * kDotCols) return go(ckpt_dot_kernel<TY, 2, 2>);
        if (K <= 2) return go(ckpt_dot_kernel<TY, 2, 1>);
        if (K <= 4) return go(ckpt_dot_kernel<TY, 4, 1>);
        if (K <= 8) return go(ckpt_dot_kernel<TY, 8, 1>);
        if (K <= 16) return go(ckpt_dot_kernel<TY, 16, 1>);
        return go(ckpt_dot_kernel<TY, 32, 1>);
    }));
    if (!grads) {
        int kp = 1;
        while (kp < K) kp *= 2;
        BEAM_HOST_CUDA(launch_free(ckpt_slot_grad_kernel, dim3((unsigned)ceil_div(T, S)), dim3(kDotThreads), 0, st,
                                   (const float*)dghat, T, K, kp, S, gate, mask_logit, reg, d_gate_logit, d_mask_logit));
    }
    return BEAM_OK;
}

// ---------------------------------------------------------------- the router's linear backward
}  // extern "C"

// Slices of k: as many as fill the pairs of SMs, each of at least kChain steps.
static void plan_slices(lin::Params& p, int pairs)
{
    const long long tiles = (long long)p.m_tiles * p.n_tiles;
    const long long most = std::max(1LL, ceil_div(p.k_steps, lin::kChain));
    const long long want = std::min(most, std::max(1LL, pairs / tiles));
    p.split_steps = (int)ceil_div(p.k_steps, want);
    p.units = (int)(tiles * ceil_div(p.k_steps, p.split_steps));
}

static lin::Params lin_params(int M, int N, int K, bool narrow = false)
{
    lin::Params p = {};
    p.M = M; p.N = N; p.K = K;
    p.m_tiles = (int)ceil_div(M, lin::BM);
    p.n_tiles = (int)ceil_div(N, narrow ? lin::kBN / 2 : lin::kBN);
    p.k_steps = (int)ceil_div(K, lin::BK);
    p.split_steps = p.k_steps;
    p.units = p.m_tiles * p.n_tiles;
    p.last = 1;
    return p;
}

static lin::Operand operand(const void* x, int dtype, long long ld, long long cols)
{
    const int v = 16 / elem_size(dtype);
    return {x, nullptr, ld, !misaligned(x, 16) && ld % v == 0 && cols % v == 0};
}

// Ranges of n per m tile for a resident A: each pair's time is about the tiles it walks plus one for
// converting A per unit; the fewest rounds times that wins.
static void plan_ranges(lin::Params& p, int pairs)
{
    long long best = -1;
    for (int r = 1; r <= p.n_tiles && r <= 4 * pairs; ++r) {
        const int len = (int)ceil_div(p.n_tiles, r), ranges = (int)ceil_div(p.n_tiles, len);
        const long long cost = ceil_div((long long)p.m_tiles * ranges, pairs) * (len + 1);
        if (best < 0 || cost < best) {
            best = cost;
            p.range = len;
            p.ranges = ranges;
            p.units = p.m_tiles * ranges;
        }
    }
}

template <int SA, bool MNA, int SB, bool MNB, bool VEC, bool RES, bool NARROW = false>
static cudaError_t launch_lin_as(const lin::Params& p, int pairs, cudaStream_t st)
{
    auto kernel = lin::lin_gemm_kernel<SA, MNA, SB, MNB, VEC, RES, NARROW>;
    const int smem = RES ? lin::res_bytes<SA, SB>(p.k_steps) : lin::smem_bytes<SA, SB>();
    static std::atomic<unsigned long long> ready;   // devices whose attribute is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, lin::kSmemLimit);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ULL << dev, std::memory_order_relaxed);
    }
    return launch_free(kernel, dim3(2 * (unsigned)std::min(p.units, pairs)), dim3(lin::kThreads), smem, st, p);
}

// k is not cut (dx).
template <int SA, bool MNA, int SB, bool MNB>
static cudaError_t launch_rows(lin::Params p, int pairs, cudaStream_t st)
{
    const bool vec = p.a.vec && p.b.vec;
    if (p.n_tiles > 1 && p.k_steps <= lin::res_steps<SA, SB>()) {
        plan_ranges(p, pairs);
        return vec ? launch_lin_as<SA, MNA, SB, MNB, true, true>(p, pairs, st)
                   : launch_lin_as<SA, MNA, SB, MNB, false, true>(p, pairs, st);
    }
    return vec ? launch_lin_as<SA, MNA, SB, MNB, true, false>(p, pairs, st)
               : launch_lin_as<SA, MNA, SB, MNB, false, false>(p, pairs, st);
}

// Tiles of 64 columns for dW's n.
static bool narrow(int N) { return N <= lin::kBN / 2; }
// k may be cut into slices (dW).
template <int SA, bool MNA, int SB, bool MNB>
static cudaError_t launch_slices(const lin::Params& p, int pairs, cudaStream_t st)
{
    const bool vec = p.a.vec && p.b.vec;
    if (narrow(p.N))
        return vec ? launch_lin_as<SA, MNA, SB, MNB, true, false, true>(p, pairs, st)
                   : launch_lin_as<SA, MNA, SB, MNB, false, false, true>(p, pairs, st);
    return vec ? launch_lin_as<SA, MNA, SB, MNB, true, false>(p, pairs, st)
               : launch_lin_as<SA, MNA, SB, MNB, false, false>(p, pairs, st);
}

// Workspace of the weight gradient: the slices' partial tiles.
static int weight_ld(int C) { return (C + 7) & ~7; }
static lin::Params weight_params(int T, int C, int d)
{
    lin::Params p = lin_params(d, C, T, narrow(C));
    plan_slices(p, std::max(1, num_sms() / 2));
    return p;
}
static long long weight_bytes(const lin::Params& p)
{
    const long long slices = p.units / ((long long)p.m_tiles * p.n_tiles);
    return slices > 1 ? slices * p.M * weight_ld(p.N) * 4 : 0;
}

static beam_status_t check_sizes(int T, int C, int d)
{
    if (T < 0 || T > (1 << 30)) FAIL_ARG("T=%d outside [0, 2^30]", T);
    if (C < 1 || C > kMaxLogits) FAIL_ARG("C=%d must be in [1, %d]", C, kMaxLogits);
    if (d < 1 || d > kMaxWidth) FAIL_ARG("d=%d must be in [1, %d]", d, kMaxWidth);
    if (ceil_div(T, lin::BM) * ceil_div(d, lin::kBN) > (1LL << 30))
        FAIL_ARG("T=%d rows of %d values are too many", T, d);
    return BEAM_OK;
}
static beam_status_t check_linear(int T, int C, int d, const void* g, int dtype, long long ldg)
{
    TRY(check_sizes(T, C, d));
    return check_matrix("dlogits", g, dtype, false, T, C, ldg);
}

static beam_status_t check_dx(const float* dx, int T, int d, long long ld_dx)
{
    if ((T > 0 && !dx) || misaligned(dx, 4)) FAIL_ARG("dx must be a 4-byte aligned pointer");
    if (ld_dx < d || ld_dx > (1LL << 31) - 1) FAIL_ARG("dx: row stride %lld is below its %d columns, or too long", ld_dx, d);
    return BEAM_OK;
}

beam_status_t beam_host_input_grad_rows(const float* dlogits, int64_t ld_dlogits, int32_t T, int32_t C, const void* w,
                                        int32_t w_dtype, int64_t ld_w, int32_t d, float* dx, int64_t ld_dx, void* stream)
{
    TRY(check_linear(T, C, d, dlogits, BEAM_DTYPE_F32, ld_dlogits));
    TRY(check_dx(dx, T, d, ld_dx));
    if (T == 0) return BEAM_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    lin::Params p = lin_params(T, d, C);
    p.a = operand(dlogits, BEAM_DTYPE_F32, ld_dlogits, C);
    p.b = operand(w, w_dtype, ld_w, d);
    p.out = dx;
    p.cp = (int)ld_dx;
    const int pairs = std::max(1, num_sms() / 2);
    BEAM_HOST_CUDA((w_dtype == BEAM_DTYPE_F32 ? launch_rows<lin::SRC_F32, false, lin::SRC_F32, true>(p, pairs, st)
                                              : launch_rows<lin::SRC_F32, false, lin::SRC_BF16, true>(p, pairs, st)));
    return BEAM_OK;
}

extern "C" {

int64_t beam_router_weight_grad_workspace(int32_t T, int32_t d, int32_t C)
{
    if (check_sizes(T, C, d) != BEAM_OK) return -1;
    return T == 0 ? 0 : weight_bytes(weight_params(T, C, d));
}

beam_status_t beam_router_weight_grad(const int8_t* q, const uint8_t* scale, int32_t T, int32_t d,
                                      const void* dlogits, int32_t dtype, int64_t ld_dlogits, int32_t C,
                                      int32_t parts, float* dw, void* workspace, int64_t workspace_bytes,
                                      void* stream)
{
    beam_host_clear_error();
    TRY(check_linear(T, C, d, dlogits, dtype, ld_dlogits));
    TRY(check_ckpt(q, scale, T, d));
    if (parts < 1 || C % parts) FAIL_ARG("parts=%d must divide C=%d", parts, C);
    if (!dw || misaligned(dw, 4)) FAIL_ARG("dw must be a 4-byte aligned pointer");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        BEAM_HOST_CUDA(cudaMemsetAsync(dw, 0, (size_t)d * C * 4, st));
        return BEAM_OK;
    }
    lin::Params p = weight_params(T, C, d);
    const long long need = weight_bytes(p);
    if (need > 0 && (!workspace || workspace_bytes < need || misaligned(workspace, 16)))
        FAIL_ARG("the workspace must be 16-byte aligned and hold %lld bytes", need);
    p.a = {q, scale, ceil_div(d, kCkptBlock) * kCkptBlock, 1};
    p.b = operand(dlogits, dtype, ld_dlogits, C);
    const int ldp = weight_ld(C), cp = C / parts;
    p.out = need ? static_cast<float*>(workspace) : dw;
    p.slice = (long long)d * ldp;
    p.cp = need ? ldp : cp;
    p.last = need == 0;
    const int pairs = std::max(1, num_sms() / 2);
    const cudaError_t e = dtype == BEAM_DTYPE_F32 ? launch_slices<lin::SRC_CKPT, true, lin::SRC_F32, true>(p, pairs, st)
                                                  : launch_slices<lin::SRC_CKPT, true, lin::SRC_BF16, true>(p, pairs, st);
    BEAM_HOST_CUDA(e);
    if (need) {
        const long long n = (long long)d * ceil_div(C, 4);
        BEAM_HOST_CUDA(launch_free(lin::lin_reduce_kernel, dim3((unsigned)ceil_div(n, 256)), dim3(256), 0, st,
                                   (const float*)p.out, (int)(need / (p.slice * 4)), p.slice, d, C, ldp, cp, dw));
    }
    return BEAM_OK;
}

beam_status_t beam_router_input_grad(const void* dlogits, int32_t dtype, int64_t ld_dlogits, int32_t T, int32_t C,
                                     const void* w, int32_t w_dtype, int64_t ld_w, int32_t d, float* dx,
                                     int64_t ld_dx, void* stream)
{
    beam_host_clear_error();
    TRY(check_linear(T, C, d, dlogits, dtype, ld_dlogits));
    TRY(check_matrix("w", w, w_dtype, false, d, C, ld_w));
    TRY(check_dx(dx, T, d, ld_dx));
    if (T == 0) return BEAM_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    lin::Params p = lin_params(T, d, C);
    p.a = operand(dlogits, dtype, ld_dlogits, C);
    p.b = operand(w, w_dtype, ld_w, C);
    p.out = dx;
    p.cp = (int)ld_dx;
    const int pairs = std::max(1, num_sms() / 2);
    const bool g32 = dtype == BEAM_DTYPE_F32, w32 = w_dtype == BEAM_DTYPE_F32;
    const cudaError_t e =
        g32 ? (w32 ? launch_rows<lin::SRC_F32, false, lin::SRC_F32, false>(p, pairs, st)
                   : launch_rows<lin::SRC_F32, false, lin::SRC_BF16, false>(p, pairs, st))
            : (w32 ? launch_rows<lin::SRC_BF16, false, lin::SRC_F32, false>(p, pairs, st)
                   : launch_rows<lin::SRC_BF16, false, lin::SRC_BF16, false>(p, pairs, st));
    BEAM_HOST_CUDA(e);
    return BEAM_OK;
}

}  // extern "C"
