// ckpt_handle.cuh -- the state that a training forward leaves in a layer handle, written out as a
// checkpoint: the expert outputs E_k(x_t) of every (token, slot) in 8 bits (checkpoint.cuh), in slot
// order instead of the expert order of Y_perm, and the router's logits.
#pragma once
#include "checkpoint.cuh"
#include "stream_experts.cuh"

namespace beam {

constexpr int kCkptHandleUnroll = 4;

// Row t K + k of q / scale = Y_perm row inv[t][k], split-K slices added in slice order.  A thread takes 4
// columns, 8 lanes a block; D is a multiple of 4.  Each output is read once (2 bytes per value from the
// tensor-core path) and written in one byte, but not at the copy rate: the 8-byte loads wait for the row's
// place.  8192 tokens x 16 slots x 1536: 285 us with the routing's copies, 610 MB, 2.1 TB/s (floor 93 us).
template <typename TY>
__global__ void __launch_bounds__(kCkptThreads)
ckpt_experts_kernel(const TY* __restrict__ yperm, int splits, long long stride, const int* __restrict__ inv,
                    long long rows, int D, int nb, int8_t* __restrict__ q, uint8_t* __restrict__ scale)
{
    constexpr int L = kCkptBlock / 4;
    pdl_wait();
    const int per_row = nb * L, D4 = D >> 2;
    const long long n = rows * per_row, s4 = stride >> 2;
    const long long u0 = (long long)blockIdx.x * (kCkptThreads * kCkptHandleUnroll) + threadIdx.x;
    float4 v[kCkptHandleUnroll];
    RowPos pos(u0, kCkptThreads, per_row);
#pragma unroll
    for (int i = 0; i < kCkptHandleUnroll; ++i) {
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (u0 + i * kCkptThreads < n && pos.at < D4) {
            const int p = __ldg(inv + pos.row);
            if (p >= 0) {   // a training forward evaluates every slot
                const size_t at = (size_t)p * D4 + pos.at;
                v[i] = load4(yperm, at);
                for (int s = 1; s < splits; ++s) {
                    const float4 w = load4(yperm, s * s4 + at);
                    v[i].x += w.x; v[i].y += w.y; v[i].z += w.z; v[i].w += w.w;
                }
            }
        }
        pos.advance();
    }
#pragma unroll
    for (int i = 0; i < kCkptHandleUnroll; ++i) {
        const long long u = u0 + i * kCkptThreads;
        const float f[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t a = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) a = max(a, __float_as_uint(f[j]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < L; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
        const int byte = ckpt_scale_byte(a);
        if (u < n) {
            *reinterpret_cast<uint32_t*>(q + u * 4) = ckpt_quant4(f, byte);
            if ((threadIdx.x & (L - 1)) == 0) scale[u / L] = (uint8_t)byte;
        }
    }
    pdl_launch_dependents();
}

// logits [rows][cols] = the router's K slices [splits][rows][ld], added in slice order as the routing does.
__global__ void __launch_bounds__(256)
ckpt_logits_kernel(const float* __restrict__ L, int splits, long long stride, int ld, long long rows, int cols,
                   float* __restrict__ logits)
{
    pdl_wait();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long r = i / cols;
    if (r < rows) {
        const float* p = L + r * ld + (i - r * cols);
        float v = *p;
        for (int s = 1; s < splits; ++s) v += p[s * stride];
        logits[i] = v;
    }
    pdl_launch_dependents();
}

}  // namespace beam
