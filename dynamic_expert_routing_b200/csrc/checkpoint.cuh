// checkpoint.cuh -- 8-bit activation checkpoints: rows of a tensor kept in one byte per value
// between the forward and the backward, with one power-of-two scale per 32 columns.
//
// Block of 32 columns with a = max |x|: k = the smallest integer >= -120 with a <= 127 * 2^k,
// q = x * 2^-k rounded to nearest even (|q| <= 127), stored as int8, and the byte k + 127.  The
// block stands for q * 2^k.  Scaling by a power of two is exact, so the one rounding is the
// integer's, half a step 2^(k-1) at most, and every value q * 2^k has at most 7 significant bits:
// it is exact in bfloat16, which lets the weight gradient feed it to the tensor cores unrounded.
// (A scale a / 127 would save up to one bit of the step, but its products are rounded twice and
// exact in no narrower type.)  A block that holds an infinity or a NaN gets the byte 255 and
// reads back as NaN.  k = 122, the largest, limits |q| to 63: 64 * 2^122 is past float32.
// Rows of q are padded with zeros to a whole block, so that every row starts 32-byte aligned.
#pragma once
#include "common.cuh"

namespace beam {

constexpr int kCkptBlock = 32;       // columns per scale
constexpr int kCkptMinExp = -120;    // smallest scale exponent
constexpr int kCkptBias = 127;
constexpr int kCkptNan = 255;        // scale byte of a block with a non-finite value

// Scale byte of a block whose largest magnitude has the float bits `a` (sign cleared).
// a = m * 2^e, 1 <= m < 2, and 127 = 1.984375 * 2^6: k = e - 6, one more when m > 1.984375
// (fraction field above 0x7e0000, which is where adding 0x1ffff carries into the exponent).
__device__ __forceinline__ int ckpt_scale_byte(uint32_t a)
{
    if (a >= 0x7f800000u) return kCkptNan;
    const int e = (int)((a + 0x1ffffu) >> 23);   // biased exponent, carried
    return max(e - 6, kCkptMinExp + kCkptBias);
}
// 2^-k and 2^k of a scale byte (both normal floats for k in [-120, 122]); NaN for byte 255.
__device__ __forceinline__ float ckpt_inv_step(int byte)
{
    return byte == kCkptNan ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)(254 - byte) << 23);
}
__device__ __forceinline__ float ckpt_step(int byte)
{
    return byte == kCkptNan ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)byte << 23);
}
__device__ __forceinline__ int ckpt_quant(float x, float inv_step, int byte)
{
    const int lim = byte == 122 + kCkptBias ? 63 : 127;
    const int q = __float2int_rn(x * inv_step);   // NaN (a 255 block) converts to 0
    return max(-lim, min(lim, q));
}

// One warp per (row, block), lane = column.
template <typename T>
__global__ void __launch_bounds__(256)
ckpt_save_kernel(const T* __restrict__ x, long long ldx, long long rows, int D, int nb,
                 int8_t* __restrict__ q, uint8_t* __restrict__ scale)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long n = rows * nb;
    for (long long b = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); b < n; b += (long long)gridDim.x * 8) {
        const long long r = b / nb;
        const int c = (int)(b - r * nb) * kCkptBlock + lane;
        const float v = c < D ? to_float(x[r * ldx + c]) : 0.f;
        const uint32_t a = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
        const int byte = ckpt_scale_byte(a);
        q[b * kCkptBlock + lane] = (int8_t)ckpt_quant(v, ckpt_inv_step(byte), byte);
        if (lane == 0) scale[b] = (uint8_t)byte;
    }
    pdl_launch_dependents();
}

// Largest finite value of the read-back types: a value that rounds past it saturates (float16
// only: its range ends at 65504, while a block whose maximum is 65504 may round up to 65536).
template <typename T> __device__ __forceinline__ T ckpt_value(float v) { return from_float<T>(v); }
template <> __device__ __forceinline__ __half ckpt_value<__half>(float v)
{
    return __float2half_rn(v > 65504.f ? 65504.f : (v < -65504.f ? -65504.f : v));
}

template <typename T>
__global__ void __launch_bounds__(256)
ckpt_load_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ scale, long long rows,
                 int D, int nb, T* __restrict__ y)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long n = rows * nb;
    for (long long b = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); b < n; b += (long long)gridDim.x * 8) {
        const long long r = b / nb;
        const int c = (int)(b - r * nb) * kCkptBlock + lane;
        if (c < D) y[r * D + c] = ckpt_value<T>((float)q[b * kCkptBlock + lane] * ckpt_step(scale[b]));
    }
    pdl_launch_dependents();
}

}  // namespace beam
