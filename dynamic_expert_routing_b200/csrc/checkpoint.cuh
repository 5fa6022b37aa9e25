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
//
// Measured on B200 (save + load of 8192 x 4096, L2 warm): float16 29.0 us for 203 MB moved (7.0 TB/s: part of
// q is still in L2 when it is read back), float32 51.5 us for 337 MB (6.5 TB/s), at the measured copy rate;
// 20000 x 1413 bf16 (no row aligned on the way out) 45 us for 171 MB; a warp per block with single values took
// 213 and 125 us.  With values widened to float32 one by one the integer pipe was busy for 80 % of the time
// (save 19.9, load 18.1 us alone and cold); in pairs of 16 bits 15.6 and 15.2 us.
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
// 2^-k of a scale byte (a normal float for k in [-120, 122]), for the blocks that are quantised.
__device__ __forceinline__ float ckpt_inv_step(int byte)
{
    return __uint_as_float((uint32_t)(254 - byte) << 23);
}
// 2^k; an infinity for byte 255, whose block holds q = 0: every product with it is NaN.
__device__ __forceinline__ float ckpt_step(int byte) { return __uint_as_float((uint32_t)byte << 23); }
// Four quantised values, one per byte.  Adding 1.5 * 2^23 rounds to an integer (nearest even) and
// leaves it in the low mantissa bits, in two's complement; x * inv_step is exact, so the fused
// multiply-add is the one rounding.  (The conversion instruction would run at a quarter of the
// rate.)  |x * inv_step| <= 127 by the choice of the scale.
__device__ __forceinline__ uint32_t ckpt_quant4(const float* x, int byte)
{
    constexpr float kRound = 12582912.f;
    float v[4] = {x[0], x[1], x[2], x[3]};
    if (byte >= 122 + kCkptBias) {   // hardly ever taken: the largest exponent, or a block of NaN
        if (byte == kCkptNan) return 0u;
        const float lim = 63.f * ckpt_step(byte);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fminf(fmaxf(v[i], -lim), lim);
    }
    const float inv_step = ckpt_inv_step(byte);
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(fmaf(v[i], inv_step, kRound));
    return __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
}
// The four integers of a word as floats: byte ^ 0x80 = q + 128 under the exponent of 2^23.
__device__ __forceinline__ void ckpt_unpack4(uint32_t w, float* f)
{
    w ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + i)) - 8388736.f;
}

// q 2^k in pairs of bf16.  With u = q + 128 = 128 h + l, the byte l under 0x43 is the bf16 number 128 + l, and
// the byte 128 (1 - h) under 0x43 is 128 or 256: their difference is q, exactly (8 significant bits), and so
// is its product with 2^k.  (Going by float32 takes half as many instructions again.)  sel: 0x4140 for the
// word's lower two bytes, 0x4342 for the upper two.
__device__ __forceinline__ uint32_t ckpt_pair(uint32_t w, uint32_t sel, __nv_bfloat162 step)
{
    const uint32_t a = __byte_perm(w & 0x7f7f7f7fu, 0x43u, sel), c = __byte_perm(w & 0x80808080u, 0x43u, sel);
    const __nv_bfloat162 q = __hsub2(reinterpret_cast<const __nv_bfloat162&>(a), reinterpret_cast<const __nv_bfloat162&>(c));
    const __nv_bfloat162 v = __hmul2(q, step);
    return reinterpret_cast<const uint32_t&>(v);
}
__device__ __forceinline__ __nv_bfloat162 ckpt_step_pair(int byte)
{
    const uint32_t k = (uint32_t)byte << 7, k2 = k | k << 16;
    return reinterpret_cast<const __nv_bfloat162&>(k2);
}
// The same in float16 for scale bytes in [103, 136], where 2^k is a float16 and no product passes its range:
// q + 128 under 0x64 is 1024 + (q + 128).  Products below 2^-14 round like any float16.
__device__ __forceinline__ uint32_t ckpt_pair(uint32_t w, uint32_t sel, __half2 step)
{
    const uint32_t a = __byte_perm(w ^ 0x80808080u, 0x64u, sel);
    const __half2 v = __hmul2(__hsub2(reinterpret_cast<const __half2&>(a), __float2half2_rn(1152.f)), step);
    return reinterpret_cast<const uint32_t&>(v);
}

// ---------------------------------------------------------------- one 16-byte vector of the wide type
// The arithmetic below is what bounded the copies before it was done in pairs (the integer pipe at 80 %).
// A key of the largest magnitude in a vector, ordered like it (NaN on top), ...
__device__ __forceinline__ uint32_t ckpt_amax(const uint4& v, float)
{
    float m = 0.f;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(__uint_as_float(w[i]))));
    return __float_as_uint(m);
}
__device__ __forceinline__ uint32_t ckpt_amax16(const uint4& v)
{
    const uint32_t k = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & k, v.y & k), __vmaxu2(v.z & k, v.w & k));
    return max(m & 0xffffu, m >> 16);
}
__device__ __forceinline__ uint32_t ckpt_amax(const uint4& v, __half) { return ckpt_amax16(v); }
__device__ __forceinline__ uint32_t ckpt_amax(const uint4& v, __nv_bfloat16) { return ckpt_amax16(v); }
// ... and its float32 bits.
__device__ __forceinline__ uint32_t ckpt_key_bits(uint32_t key, float) { return key; }
__device__ __forceinline__ uint32_t ckpt_key_bits(uint32_t key, __nv_bfloat16) { return key << 16; }
__device__ __forceinline__ uint32_t ckpt_key_bits(uint32_t key, __half)
{
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)key)));
}

// The vector's V quantised bytes (float32: the lower word).
template <typename T>
__device__ __forceinline__ uint2 ckpt_quant(const uint4& raw, int byte)
{
    constexpr int V = Vec<T>::N;
    float v[8];
    Vec<T>::widen(raw, v);
    return make_uint2(ckpt_quant4(v, byte), V == 8 ? ckpt_quant4(v + V - 4, byte) : 0u);
}
// float16: 1.5 * 2^10 rounds to an integer as 1.5 * 2^23 does in float32, where 2^-k is a float16.
template <>
__device__ __forceinline__ uint2 ckpt_quant<__half>(const uint4& raw, int byte)
{
    if (byte < kCkptBias - 15 || byte > kCkptBias + 10) {
        float v[8];
        Vec<__half>::widen(raw, v);
        return make_uint2(ckpt_quant4(v, byte), ckpt_quant4(v + 4, byte));
    }
    const __half2 inv = __float2half2_rn(ckpt_inv_step(byte)), round = __float2half2_rn(1536.f);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __hfma2(reinterpret_cast<const __half2&>(w[i]), inv, round);
        r[i] = reinterpret_cast<const uint32_t&>(h);
    }
    return make_uint2(__byte_perm(r[0], r[1], 0x6420), __byte_perm(r[2], r[3], 0x6420));
}

// Position of a unit u of a [rows][per_row] grid, advanced by a fixed step without dividing.
struct RowPos {
    long long row;
    int at, per_row;
    long long d_row;
    int d_at;
    __device__ RowPos(long long u, long long step, int per_row_) : per_row(per_row_)
    {
        row = u / per_row; at = (int)(u - row * per_row);
        d_row = step / per_row; d_at = (int)(step - d_row * per_row);
    }
    __device__ void advance()
    {
        row += d_row; at += d_at;
        if (at >= per_row) { at -= per_row; ++row; }
    }
};

// Both directions move one 16-byte vector of the wide type per thread and step (V = 4 or 8
// columns, so 8 or 4 lanes share a block) and V bytes of q: every access of a warp is contiguous.
// HBM-bound: 2 + 1 + 1/32 bytes per value for a 16-bit type.  kCkptUnroll vectors are in flight
// per thread.
constexpr int kCkptThreads = 256, kCkptUnroll = 4;

// How rows of the wide tensor are reached (8192 x 4096 float16, save + load: 31.6 us FLAT, 42.9 when saved
// value by value; 20000 x 1413 bf16: 47.5 TAIL, 52.3 ANY): FLAT, rows contiguous, 16-byte aligned and a multiple of 32
// values long, so that no row index is needed; ROWS, every row starts and ends at a 16-byte boundary; TAIL,
// every row starts at one; ANY, one value at a time.
enum CkptRows { CKPT_FLAT = 0, CKPT_ROWS = 1, CKPT_TAIL = 2, CKPT_ANY = 3 };

template <typename T, int ROWS>
__global__ void __launch_bounds__(kCkptThreads)
ckpt_save_kernel(const T* __restrict__ x, long long ldx, long long rows, int D, int nb,
                 int8_t* __restrict__ q, uint8_t* __restrict__ scale)
{
    constexpr int V = Vec<T>::N, L = kCkptBlock / V;   // L lanes hold a block
    constexpr int U = ROWS == CKPT_ANY ? 2 : kCkptUnroll;
    pdl_wait();
    const int per_row = nb * L;
    const long long n = rows * per_row;   // a multiple of L: a block's lanes are in or out together
    const long long u0 = (long long)blockIdx.x * (kCkptThreads * U) + threadIdx.x;
    union Values { T t[V]; uint4 u; } raw[U];
    RowPos pos(ROWS == CKPT_FLAT ? 0 : u0, kCkptThreads, per_row);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const long long u = u0 + i * kCkptThreads;
        raw[i].u = make_uint4(0u, 0u, 0u, 0u);
        if (ROWS == CKPT_FLAT) {
            if (u < n) raw[i].u = ldg_stream(x + u * V);
        } else {
            const int c = pos.at * V;
            const T* p = x + pos.row * ldx + c;
            if (ROWS == CKPT_ANY) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (u < n && c + j < D) raw[i].t[j] = p[j];
            } else if (u < n && c + V <= D) {
                raw[i].u = ldg_stream(p);
            }
            pos.advance();
        }
    }
    if (ROWS == CKPT_TAIL) {   // the vectors that a row's end cuts, after the others are on their way
        RowPos tail(u0, kCkptThreads, per_row);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = tail.at * V;
            if (u0 + i * kCkptThreads < n && c < D && c + V > D) {
                const T* p = x + tail.row * ldx + c;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (c + j < D) raw[i].t[j] = p[j];
            }
            tail.advance();
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const long long u = u0 + i * kCkptThreads;
        uint32_t a = ckpt_amax(raw[i].u, T());
#pragma unroll
        for (int o = 1; o < L; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
        const int byte = ckpt_scale_byte(ckpt_key_bits(a, T()));
        const uint2 b = ckpt_quant<T>(raw[i].u, byte);
        if (u < n) {
            if (V == 8) *reinterpret_cast<uint2*>(q + u * V) = b;
            else *reinterpret_cast<uint32_t*>(q + u * V) = b.x;
            if ((threadIdx.x & (L - 1)) == 0) scale[u / L] = (uint8_t)byte;
        }
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

// V consecutive values of the read-back type in one 16-byte vector.
template <typename T>
__device__ __forceinline__ uint4 ckpt_pack(const float* f)
{
    constexpr int V = Vec<T>::N;
    union { T t[V]; uint4 u; } o;
#pragma unroll
    for (int j = 0; j < V; ++j) o.t[j] = ckpt_value<T>(f[j]);
    return o.u;
}

// V values of one block from their bytes.
template <typename T>
__device__ __forceinline__ uint4 ckpt_values(const uint2& q, int byte)
{
    constexpr int V = Vec<T>::N;
    float f[8];
    ckpt_unpack4(q.x, f);
    if (V == 8) ckpt_unpack4(q.y, f + 4);
    const float step = ckpt_step(byte);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] *= step;
    return ckpt_pack<T>(f);
}
template <typename S>
__device__ __forceinline__ uint4 ckpt_pairs(const uint2& q, S step)
{
    return make_uint4(ckpt_pair(q.x, 0x4140, step), ckpt_pair(q.x, 0x4342, step), ckpt_pair(q.y, 0x4140, step),
                      ckpt_pair(q.y, 0x4342, step));
}
template <>
__device__ __forceinline__ uint4 ckpt_values<__nv_bfloat16>(const uint2& q, int byte)
{
    return ckpt_pairs(q, ckpt_step_pair(byte));
}
template <>
__device__ __forceinline__ uint4 ckpt_values<__half>(const uint2& q, int byte)
{
    if (byte >= kCkptBias - 24 && byte <= kCkptBias + 9) return ckpt_pairs(q, __float2half2_rn(ckpt_step(byte)));
    float f[8];
    ckpt_unpack4(q.x, f);
    ckpt_unpack4(q.y, f + 4);
    const float step = ckpt_step(byte);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= step;
    return ckpt_pack<__half>(f);
}

// y [rows][D] contiguous and 16-byte aligned.  FLAT: D a multiple of 32; ROWS: of V.
template <typename T, int ROWS>
__global__ void __launch_bounds__(kCkptThreads)
ckpt_load_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ scale, long long rows,
                 int D, int nb, T* __restrict__ y)
{
    constexpr int V = Vec<T>::N, L = kCkptBlock / V;
    pdl_wait();
    const int per_row = nb * L;
    const long long n = rows * per_row;
    const long long u0 = (long long)blockIdx.x * (kCkptThreads * kCkptUnroll) + threadIdx.x;
    uint2 raw[kCkptUnroll];
    int byte[kCkptUnroll];
#pragma unroll
    for (int i = 0; i < kCkptUnroll; ++i) {
        const long long u = u0 + i * kCkptThreads;
        raw[i] = make_uint2(0u, 0u);
        byte[i] = kCkptBias;
        if (u < n) {
            if (V == 8) raw[i] = __ldg(reinterpret_cast<const uint2*>(q + u * V));
            else raw[i].x = __ldg(reinterpret_cast<const uint32_t*>(q + u * V));
            byte[i] = __ldg(scale + u / L);
        }
    }
    RowPos pos(ROWS == CKPT_FLAT ? 0 : u0, kCkptThreads, per_row);
#pragma unroll
    for (int i = 0; i < kCkptUnroll; ++i) {
        const long long u = u0 + i * kCkptThreads;
        const uint4 v = ckpt_values<T>(raw[i], byte[i]);
        if (ROWS == CKPT_FLAT) {
            if (u < n) *reinterpret_cast<uint4*>(y + u * V) = v;
        } else {
            if (u < n && pos.at * V < D) *reinterpret_cast<uint4*>(y + pos.row * D + pos.at * V) = v;
            pos.advance();
        }
    }
    pdl_launch_dependents();
}

// Any D: a thread makes one 16-byte vector of the flat y, wherever its V values start in a row, from the
// aligned words of q that hold them, so that every store is whole (stores of single values would each
// touch a sector: 8 times the write traffic).  A vector that spans two rows goes value by value.
template <typename T>
__global__ void __launch_bounds__(kCkptThreads)
ckpt_load_any_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ scale, long long rows,
                     int D, int nb, T* __restrict__ y)
{
    constexpr int V = Vec<T>::N;
    pdl_wait();
    const long long total = rows * D;
    const long long f0 = ((long long)blockIdx.x * (kCkptThreads * kCkptUnroll) + threadIdx.x) * V;
    RowPos pos(f0, kCkptThreads * V, D);
#pragma unroll
    for (int i = 0; i < kCkptUnroll; ++i) {
        const long long at = f0 + (long long)i * kCkptThreads * V;
        const int c = pos.at;
        float f[8];
        if (at < total && c + V <= D) {
            const int8_t* p = q + pos.row * nb * kCkptBlock + c;
            const uint8_t* s = scale + pos.row * nb;
            const uint32_t* w = reinterpret_cast<const uint32_t*>(p - (c & 3));
            const int sh = 8 * (c & 3);
            uint32_t lo = __ldg(w);
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                // the next word holds values of this vector, or (sh = 0, the last time) is not read
                const uint32_t hi = sh || j + 4 < V ? __ldg(w + j / 4 + 1) : 0u;
                ckpt_unpack4(__funnelshift_r(lo, hi, sh), f + j);
                lo = hi;
            }
            const int first = kCkptBlock - (c & (kCkptBlock - 1));   // values in the first block
            const float s0 = ckpt_step(__ldg(s + c / kCkptBlock)), s1 = ckpt_step(__ldg(s + (c + V - 1) / kCkptBlock));
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] *= j < first ? s0 : s1;
        } else {
            long long r = pos.row;
            int k = c;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                f[j] = 0.f;
                if (at + j < total)
                    f[j] = (float)q[r * nb * kCkptBlock + k] * ckpt_step(__ldg(scale + r * nb + k / kCkptBlock));
                if (++k == D) { k = 0; ++r; }
            }
        }
        if (at + V <= total) {
            *reinterpret_cast<uint4*>(y + at) = ckpt_pack<T>(f);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (at + j < total) y[at + j] = ckpt_value<T>(f[j]);
        }
        pos.advance();
    }
    pdl_launch_dependents();
}

}  // namespace beam
