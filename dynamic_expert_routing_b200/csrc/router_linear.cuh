// router_linear.cuh -- the backward of the router's linear map logits = x W (x [T][D], W [D][C]):
//   dW[d][c] = sum_t x[t][d] G[t][c]   with x from an 8-bit checkpoint
//   dx[t][d] = sum_c G[t][c] W[d][c]
// for the dense logit gradient G [T][C] (the balance term reaches every expert of every token).
//
// Both run on the tensor cores (tcgen05, bf16 operands, fp32 accumulation) and keep float32's
// precision.  A checkpoint value q 2^k and a bf16 value are bf16 operands as they are.  A float32
// value is the exact sum of three bf16 numbers cut from its 24 significant bits, 8 at a time (its
// upper half; the upper half of the rest; the rest): cut, not rounded, the second reaches 2^-7 of the value and the
// third 2^-15.  The product of two operands is taken limb by limb, all pairs but the two third limbs', which
// stays below 2^-30 of it (leaving out the pairs of a second and a third limb too, 2^-22 each and of one
// sign, would cost a float32 x float32 product 2^-21).  The tensor cores add into their accumulator with truncation, an error of one sign that
// grows with the number of additions: the leading product therefore has an accumulator of
// its own (the small ones share another), and every kChain steps of 64 the accumulators are
// drained into float32 sums in registers, rounded to nearest.
//
// One kernel computes out[m][n] = sum_k A(m, k) B(n, k) on 256 x 128 tiles (256 x 64 for dW of up to 64
// logits), 64 of k per step:
//   dW: m = d, n = c, k = t: A and B lie in memory with m, n contiguous ("MN-major");
//   dx: m = t, n = d, k = c: k contiguous ("K-major"; MN-major for a repacked W [C][D]).
// Two CTAs share a tile (cta_group::2): each converts its 128 rows of A and half of B, so an operand
// value is converted half as often, which is what bounds the kernel beside the MMAs: the operands are
// not bf16 in memory, so TMA could not bring them.  16 warps per CTA write them into shared memory in
// the 128-byte-swizzled layout that tcgen05.mma reads (a block of rows of 128 bytes; the major-ness
// is a bit of the instruction descriptor); each thread loads the next step's piece as it converts
// this one's.  One warp of the first CTA issues the MMAs of both (two of the second pass on what its warps
// have ready); 8 warps in each drain its rows' accumulators from TMEM (two sets, so that a drain overlaps
// the next steps) and store.  The grid is
// persistent; when the tiles are fewer than the CTA pairs, k is cut into slices whose partial tiles
// lin_reduce_kernel adds in order.  Where k is short (dx: k = c), a pair converts its rows of A once, keeps
// them in shared memory and walks a range of n with B alone in the ring.
// Every wait is bounded: when one runs out, the pair's tiles that are not yet stored are set to NaN.
//
// Measured on B200 (device time):
//   dW 8192 x 1536 x 424, float32 G: 38.4 us, 278 TFLOP/s of dW's own operations, 0.83 PFLOP/s with the limbs;
//     unsliced 92 us.  What bounds it is the loaders' work per step (converting and storing 40 KB per CTA):
//     the MMAs alone take 20 of them.  bf16 G 32 us.  1003 x 2048 x 128, bf16 G: 9.1 us (unsliced 11.6).
//   dx 8192 x 2048 x 128, float32 G, bf16 W: 19.8 us, 67 MB written (floor 11 us at the copy rate); with A
//     converted again for every n tile 34 us; float32 W 27.8.  8192 x 1536 x 424 (float32 G is too long to stay):
//     55 us, W as [C][D] 52, float32 W 69, bf16 G and W 24.
//   Error against 64 bits at 8192 x 1536 x 424: 1.1e-7; with the accumulator drained every 16 steps 2.1e-7,
//     never 3.0e-6 (2.3e-6 of it towards zero), with one accumulator for all products 8.5e-7.
#pragma once
#include <type_traits>
#include "checkpoint.cuh"
#include "tc_ptx.cuh"

namespace beam {
namespace lin {

constexpr int BM = 256, kBN = 128, BK = 64;   // the tile of a CTA pair (BN = 64 where n is short, see NARROW)
constexpr int kRowsA = BM / 2;                // a CTA's share of A, half a tile like that of B
constexpr int kLimbA = kRowsA * BK * 2, kLimbB = kBN / 2 * BK * 2;   // bytes of one limb of a share
constexpr int kChain = 4;                     // steps added in the tensor cores' accumulator
// Warpgroups of 4 warps: 4 that load and convert, one whose first warp issues the MMAs, 2 that drain.
// The kernel is launched with 72 registers a thread (7 x 128 x 72 of the SM's 65536); the
// epilogue, which keeps 64 sums per thread, takes some from the others: 512 x 64 + 128 x 24 + 256 x 112
// = 64512 registers, the launch's own total.
constexpr int kLoadWarps = 16, kEpiWarps = 8, kMmaWarp = kLoadWarps, kEpiWarp0 = kLoadWarps + 4;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kLaunchRegs = 72, kLoadRegs = 64, kMmaRegs = 24, kEpiRegs = 112;
static_assert(32 * kLoadWarps * kLoadRegs + 128 * kMmaRegs + 32 * kEpiWarps * kEpiRegs <= kThreads * kLaunchRegs,
              "the register shares must fit the launch's");
constexpr int kMaxStages = 4;
constexpr int kStagePitch = 36;               // epilogue staging: 32 x 32 sub-tiles, 16-byte accesses without
                                              // conflicts both ways
constexpr int kEpiBytes = kEpiWarps * 32 * kStagePitch * 4;
constexpr int kSmemLimit = 227 * 1024;

enum Src { SRC_CKPT = 0, SRC_F32 = 1, SRC_BF16 = 2 };
__host__ __device__ constexpr int limbs(int src) { return src == SRC_F32 ? 3 : 1; }

template <int SA, int SB> __host__ __device__ constexpr int stage_bytes() { return limbs(SA) * kLimbA + limbs(SB) * kLimbB; }
template <int SA, int SB> __host__ __device__ constexpr int stages()
{
    constexpr int n = (kSmemLimit - kEpiBytes - 2048) / stage_bytes<SA, SB>();
    return n < kMaxStages ? n : kMaxStages;
}
template <int SA, int SB> __host__ __device__ constexpr int accs() { return limbs(SA) * limbs(SB) > 1 ? 2 : 1; }
constexpr int kSmemExtra = kEpiBytes + 1024 /* alignment */ + 256 /* barriers */;
template <int SA, int SB> __host__ __device__ constexpr int smem_bytes()
{
    return stages<SA, SB>() * stage_bytes<SA, SB>() + kSmemExtra;
}
// A resident: all k steps of A's share stay in shared memory while the pair walks a range of n, and the
// ring holds B alone.
template <int SB> __host__ __device__ constexpr int res_stages() { return limbs(SB) > 1 ? 2 : 4; }
template <int SA, int SB> __host__ __device__ constexpr int res_steps()   // the most k steps that fit
{
    return (kSmemLimit - kSmemExtra - res_stages<SB>() * limbs(SB) * kLimbB) / (limbs(SA) * kLimbA);
}
template <int SA, int SB> __host__ __device__ constexpr int res_bytes(int k_steps)
{
    return k_steps * limbs(SA) * kLimbA + res_stages<SB>() * limbs(SB) * kLimbB + kSmemExtra;
}

struct Operand {
    const void* p;
    const uint8_t* scale;   // checkpoint: [rows][ld / 32]
    long long ld;           // elements between rows
    int vec;                // rows start and end at 16-byte boundaries
};

struct Params {
    Operand a, b;
    int M, N, K;
    int m_tiles, n_tiles, k_steps;
    // Work units of a CTA pair: a tile over a slice of k (split_steps steps), or, with A resident, the
    // tiles of one m over a range of n (range tiles; k is not cut).
    int split_steps, range, ranges;
    int units;
    // Element (m, n) of slice s is at out + s * slice + ((n / cp) * M + m) * cp + n % cp.
    float* out;
    long long slice;
    int cp;
    int last;               // no reduction follows
};

// ---------------------------------------------------------------- operands
// Eight consecutive values of a row, as loaded.
template <int SRC> struct Raw;
template <> struct Raw<SRC_F32> { uint4 a, b; };
template <> struct Raw<SRC_BF16> { uint4 a; };
template <> struct Raw<SRC_CKPT> { uint2 w; int byte; };

// Loads that a predicate turns into zeros, without a branch: a branch would merge loaded registers
// with zeroed ones, and the copies would wait for the load that the next step is to use.
__device__ __forceinline__ uint4 ldg16_if(const void* p, bool on)
{
    uint4 r;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
                 "mov.b32 %0, 0; mov.b32 %1, 0; mov.b32 %2, 0; mov.b32 %3, 0;\n\t"
                 "@p ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
                 : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w) : "l"(p), "r"((int)on));
    return r;
}
__device__ __forceinline__ uint2 ldg8_if(const void* p, bool on)
{
    uint2 r;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b32 %0, 0; mov.b32 %1, 0;\n\t"
                 "@p ld.global.nc.v2.u32 {%0,%1}, [%2];\n\t}"
                 : "=&r"(r.x), "=&r"(r.y) : "l"(p), "r"((int)on));
    return r;
}
__device__ __forceinline__ uint32_t ldg4_if(const void* p, bool on)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t"
                 "@p ld.global.nc.u32 %0, [%1];\n\t}" : "=&r"(r) : "l"(p), "r"((int)on));
    return r;
}
__device__ __forceinline__ uint32_t ldg2_if(const void* p, bool on)
{
    unsigned short r;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b16 %0, 0;\n\t"
                 "@p ld.global.nc.u16 %0, [%1];\n\t}" : "=&h"(r) : "l"(p), "r"((int)on));
    return r;
}
__device__ __forceinline__ int ldg1_if(const void* p, bool on)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t"
                 "@p ld.global.nc.u8 %0, [%1];\n\t}" : "=&r"(r) : "l"(p), "r"((int)on));
    return (int)r;
}

// Eight values, all of them there (off: the distance of the second half where it exists, else 0).
__device__ __forceinline__ void raw_load_all(Raw<SRC_F32>& r, const char* p, const uint8_t*, int off)
{
    r.a = __ldg(reinterpret_cast<const uint4*>(p));
    r.b = __ldg(reinterpret_cast<const uint4*>(p + off));
}
__device__ __forceinline__ void raw_load_all(Raw<SRC_BF16>& r, const char* p, const uint8_t*, int)
{
    r.a = __ldg(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ void raw_load_all(Raw<SRC_CKPT>& r, const char* p, const uint8_t* scale, int)
{
    r.w = __ldg(reinterpret_cast<const uint2*>(p));
    r.byte = __ldg(scale);
}

// The first n values from p on (n <= 0: none), the rest 0.  VEC: p is 16-byte aligned and n ends at a
// 16-byte boundary.
template <bool VEC>
__device__ __forceinline__ void raw_load(Raw<SRC_F32>& r, const char* p, const uint8_t*, int n)
{
    if (VEC) {
        r.a = ldg16_if(p, n > 0);
        r.b = ldg16_if(p + 16, n > 4);
    } else {
        r.a = make_uint4(ldg4_if(p, n > 0), ldg4_if(p + 4, n > 1), ldg4_if(p + 8, n > 2), ldg4_if(p + 12, n > 3));
        r.b = make_uint4(ldg4_if(p + 16, n > 4), ldg4_if(p + 20, n > 5), ldg4_if(p + 24, n > 6), ldg4_if(p + 28, n > 7));
    }
}
template <bool VEC>
__device__ __forceinline__ void raw_load(Raw<SRC_BF16>& r, const char* p, const uint8_t*, int n)
{
    if (VEC) {
        r.a = ldg16_if(p, n > 0);
    } else {
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = ldg2_if(p + 2 * j, n > j);
        r.a = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
    }
}
// Checkpoint rows are 32-byte aligned and padded with zeros to whole blocks.
template <bool VEC>
__device__ __forceinline__ void raw_load(Raw<SRC_CKPT>& r, const char* p, const uint8_t* scale, int n)
{
    r.w = ldg8_if(p, n > 0);
    r.byte = ldg1_if(scale, n > 0);
}

// The upper halves of two words.
__device__ __forceinline__ uint32_t pack_hi(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x7632); }

// bf16 limbs of the eight values, most significant first.
__device__ __forceinline__ void raw_limbs(const Raw<SRC_BF16>& r, uint4* o) { o[0] = r.a; }
__device__ __forceinline__ void raw_limbs(const Raw<SRC_CKPT>& r, uint4* o)
{
    o[0] = ckpt_pairs(r.w, ckpt_step_pair(r.byte));
}
__device__ __forceinline__ void raw_limbs(const Raw<SRC_F32>& r, uint4* o)
{
    const uint32_t x[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    uint32_t mid[8], low[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float rest = __uint_as_float(x[j]) - __uint_as_float(x[j] & 0xffff0000u);   // exact
        mid[j] = __float_as_uint(rest);
        low[j] = __float_as_uint(rest - __uint_as_float(mid[j] & 0xffff0000u));           // exact, 8 bits
    }
    o[0] = make_uint4(pack_hi(x[0], x[1]), pack_hi(x[2], x[3]), pack_hi(x[4], x[5]), pack_hi(x[6], x[7]));
    o[1] = make_uint4(pack_hi(mid[0], mid[1]), pack_hi(mid[2], mid[3]), pack_hi(mid[4], mid[5]), pack_hi(mid[6], mid[7]));
    o[2] = make_uint4(pack_hi(low[0], low[1]), pack_hi(low[2], low[3]), pack_hi(low[4], low[5]), pack_hi(low[6], low[7]));
}

// ---------------------------------------------------------------- units and steps
struct Unit { int m0, nt, nt1, slice, s0, s1; };

template <bool RES>
__device__ __forceinline__ bool get_unit(const Params& p, int u, Unit& t)
{
    if (u >= p.units) return false;
    const int width = RES ? p.ranges : p.n_tiles;
    const int c = u % width, r = u / width;
    t.nt = RES ? c * p.range : c;
    t.nt1 = RES ? min(p.n_tiles, t.nt + p.range) : c + 1;
    t.m0 = (RES ? r : r % p.m_tiles) * BM;
    t.slice = RES ? 0 : r / p.m_tiles;
    t.s0 = RES ? 0 : t.slice * p.split_steps;
    t.s1 = RES ? p.k_steps : min(p.k_steps, t.s0 + p.split_steps);
    return true;
}

// The pieces of one operand share (ROWS of m or n) that a loader thread brings: one 8-value chunk of
// kPieces rows of the share's blocks of rows.  MN-major: 64 rows (k) x ROWS / 8 chunks; K-major: ROWS
// rows (m or n) x 8 chunks.  A quarter warp stores 8 different chunks of one row: no bank conflict.
// Past the operand, k reads as zero; m and n read anything (those outputs are never stored).
template <int SRC, bool MN, int ROWS> struct Cursor {
    static constexpr int ES = SRC == SRC_CKPT ? 1 : (SRC == SRC_F32 ? 4 : 2);
    static constexpr int kChunks = MN ? ROWS / 8 : 8;
    static constexpr int kRows = 32 * kLoadWarps / kChunks;        // rows of a block between pieces
    static constexpr int kSpan = MN ? BK : ROWS;                   // rows of a block
    static constexpr int kPieces = kSpan > kRows ? kSpan / kRows : 1;
    static_assert(kPieces <= 2, "one distance between pieces");
    // The threads that have a piece: all, or the first warps where the share is small.
    static __device__ __forceinline__ bool busy(int tid) { return kSpan >= kRows || tid < kSpan * kChunks; }
    static_assert(kSpan * kChunks % 32 == 0, "whole warps");
    const char* p;           // piece 0 of the current step
    const uint8_t* sc;
    long long next;          // bytes from piece 0 to piece 1
    int k;                   // the first k of piece 0
    int n;                   // MN-major: values that the chunk has (<= 0: none);  K-major: rows from piece 0 on
    int off;                 // distance of a chunk's second 16 bytes
    __device__ __forceinline__ void start(const Operand& o, int tid, int x0, int xs, int k0)
    {
        const int chunk = tid % kChunks, row = tid / kChunks;
        int x = x0 + (MN ? 8 * chunk : row);
        k = k0 + (MN ? row : 8 * chunk);
        n = xs - x;
        if (n <= 0) x = MN ? (xs - 1) & ~7 : xs - 1;   // a place that can be read
        off = MN && n <= 4 ? 0 : 16;
        const long long r = MN ? k : x, c = MN ? x : k;
        p = static_cast<const char*>(o.p) + (r * o.ld + c) * ES;
        next = MN || kRows < n ? kRows * o.ld * ES : 0;
        if (SRC == SRC_CKPT) sc = o.scale + r * (o.ld >> 5) + (c >> 5);
    }
    __device__ __forceinline__ void advance(const Operand& o)
    {
        k += BK;
        p += (MN ? BK * o.ld : BK) * ES;
        if (SRC == SRC_CKPT) sc += MN ? BK * (o.ld >> 5) : BK >> 5;
    }
    // Piece i where the whole step lies inside k.
    __device__ __forceinline__ void load_all(Raw<SRC>& r, int i) const
    {
        raw_load_all(r, p + (i ? next : 0), SRC == SRC_CKPT ? sc + (i ? (next >> 5) : 0) : nullptr, off);
    }
    template <bool VEC> __device__ __forceinline__ void load(Raw<SRC>& r, int i, int K) const
    {
        const int ki = MN ? k + i * kRows : k, have = MN ? n : n - i * kRows;
        raw_load<VEC>(r, p + (i ? next : 0), SRC == SRC_CKPT ? sc + (i ? (next >> 5) : 0) : nullptr,
                      have > 0 && ki < K ? (MN ? n : K - k) : 0);
    }
    // Byte offset of piece 0 in a limb's swizzled tile; piece i is kRows * 128 bytes on (a multiple of
    // the 8-row swizzle period).
    __device__ static __forceinline__ uint32_t offset(int tid)
    {
        const int chunk = tid % kChunks, row = tid / kChunks;
        return (chunk >> 3) * (BK * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
    }
};
static_assert(kCkptBlock == 32, "the scale of a value is found by shifts of 5");

// at: an address of the shared window.
template <int SRC, int LIMB>
__device__ __forceinline__ void piece_store(const Raw<SRC>& r, uint32_t at)
{
    uint4 l[limbs(SRC)];
    raw_limbs(r, l);
#pragma unroll
    for (int i = 0; i < limbs(SRC); ++i)
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + i * LIMB), "r"(l[i].x), "r"(l[i].y),
                     "r"(l[i].z), "r"(l[i].w) : "memory");
}

// Shared-memory descriptor of an MN-major tile: blocks of 64 values (128 bytes) of m or n, 64 rows of k
// each (leading byte offset: the next block), groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr)
{
    return tc::sw128_desc(saddr) - ((uint64_t)1 << 16) + ((uint64_t)((BK * 128) >> 4) << 16);
}

// NARROW: tiles of 64 columns, for n <= 64 (MN-major B only: a share's 32 columns take the lower half of each
// 128-byte row).  dW 4096 x 4096 x 16 15.3 us, with 128 columns 16.5.
template <int SA, bool MNA, int SB, bool MNB, bool VEC, bool RES, bool NARROW>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
lin_gemm_kernel(const __grid_constant__ Params p)
{
    constexpr int BN = NARROW ? kBN / 2 : kBN, kRowsB = BN / 2;
    static_assert(!NARROW || (MNB && !RES), "not built");
    constexpr int LA = limbs(SA), LB = limbs(SB), ST = RES ? res_stages<SB>() : stages<SA, SB>(), ACC = accs<SA, SB>();
    constexpr int kStage = RES ? LB * kLimbB : stage_bytes<SA, SB>();   // bytes of a ring stage
    constexpr int kTmemCols = 512;   // 2 sets of ACC accumulators of BN columns, at the same place in both CTAs
    static_assert(2 * ACC * BN <= kTmemCols, "accumulators");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = tc::smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw_addr);
    const uint32_t ring = RES ? p.k_steps * (LA * kLimbA) : 0;           // where the ring starts, behind a resident A
    const uint32_t bpart = RES ? 0 : LA * kLimbA;                        // B's place in a stage
    float* epi_buf = reinterpret_cast<float*>(gbase + ring + ST * kStage);
    const uint32_t bars = base + ring + ST * kStage + kEpiBytes;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (ST + s); };
    auto tfull_bar = [&](int a) { return bars + 8u * (2 * ST + a); };
    auto tempty_bar = [&](int a) { return bars + 8u * (2 * ST + 2 + a); };
    const uint32_t drain_bar = bars + 8u * (2 * ST + 4);
    const uint32_t afree_bar = bars + 8u * (2 * ST + 5);   // RES: the MMAs on the resident A have finished
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + (bars - base) + 8 * (2 * ST + 6));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = tc::cluster_rank();                 // CTA of the pair; 0 issues the MMAs
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        // full and tempty take the arrivals of the CTA's own warps, and in CTA 0 one more: a warp of CTA 1
        // passes on its own barrier's completed phases.  empty and tfull are signalled in both
        // CTAs by the MMAs' completion.
        const int other = rank == 0 ? 1 : 0;
        for (int s = 0; s < ST; ++s) { tc::mbar_init(full_bar(s), kLoadWarps + other); tc::mbar_init(empty_bar(s), 1); }
        for (int a = 0; a < 2; ++a) { tc::mbar_init(tfull_bar(a), 1); tc::mbar_init(tempty_bar(a), kEpiWarps + other); }
        tc::mbar_init(drain_bar, 1);
        tc::mbar_init(afree_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(tc::smem_u32(tmem_slot)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc::tc_fence_before();
    tc::cluster_sync();
    tc::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();
    // The next launch may begin now, behind this grid, where it is another operator's (input grad 64 x 256 x 16:
    // 5.2 us against 5.9); lin_reduce_kernel's many CTAs, started early, cost the MMAs more than they gain.
    if (p.last) pdl_launch_dependents();

    if (warp < kLoadWarps) {
        // ------------------------------------------------ loaders: global -> bf16 limbs -> shared
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
        const int tid = threadIdx.x;
        using CA = Cursor<SA, MNA, kRowsA>;
        using CB = Cursor<SB, MNB, kRowsB>;
        constexpr int PA = CA::kPieces, PB = CB::kPieces;
        static_assert(CA::kSpan >= CA::kRows, "every thread has pieces of A");
        const bool b_on = CB::busy(tid);
        const uint32_t oa = CA::offset(tid), ob = CB::offset(tid) + ring + bpart;
        CA ca;
        CB cb;
        // The registers of one step: each piece is loaded again as soon as it is converted.  (Two sets, a step
        // further ahead, measured slower: 40 against 38 us for 8192 x 1536 x 424.)
        struct Set { Raw<SA> a[RES ? 1 : PA]; Raw<SB> b[PB]; } set;
        Unit t = {};
        int u = pair, left = 0;
        auto start_tile = [&]() {
            if (!RES) ca.start(p.a, tid, t.m0 + rank * kRowsA, p.M, t.s0 * BK);
            cb.start(p.b, tid, t.nt * BN + rank * kRowsB, p.N, t.s0 * BK);
            left = t.s1 - t.s0;
        };
        bool more = get_unit<RES>(p, u, t);   // the cursors are at a step that is not loaded (or, at the end, at the last)
        start_tile();
        auto next = [&]() {
            if (!more) return;
            if (left > 1) {
                --left;
                if (!RES) ca.advance(p.a);
                cb.advance(p.b);
            } else if (RES && t.nt + 1 < t.nt1) {
                ++t.nt;
                start_tile();
            } else {
                u += pairs;
                more = get_unit<RES>(p, u, t);
                if (more) start_tile();
            }
        };
        auto fill = [&](Set& r) {
            if (!RES)
#pragma unroll
                for (int i = 0; i < PA; ++i) ca.template load<VEC>(r.a[RES ? 0 : i], i, p.K);
            if (b_on)
#pragma unroll
                for (int i = 0; i < PB; ++i) cb.template load<VEC>(r.b[i], i, p.K);
        };
        int s = 0;
        uint32_t ph = 0;
        // Converts and stores the step in `r` and loads the one at the cursors into the same registers,
        // piece by piece.  ALL: that one lies inside k: plain loads.
        auto body = [&](Set& r, auto all) {
            constexpr bool ALL = decltype(all)::value;
            const uint32_t sm = base + s * kStage;
            if (!RES)
#pragma unroll
                for (int i = 0; i < PA; ++i) {
                    Raw<SA>& v = r.a[RES ? 0 : i];
                    piece_store<SA, kLimbA>(v, sm + oa + i * (CA::kRows * 128));
                    if (ALL) ca.load_all(v, i);
                    else ca.template load<VEC>(v, i, p.K);
                }
            if (b_on)
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                piece_store<SB, kLimbB>(r.b[i], sm + ob + i * (CB::kRows * 128));
                if (ALL) cb.load_all(r.b[i], i);
                else cb.template load<VEC>(r.b[i], i, p.K);
            }
        };
        // RES: the unit whose steps are being stored, its steps to come, and the units before it
        int cu = pair, rest = 0, units = 0;
        auto process = [&](Set& r) {
            if (RES && rest == 0) {
                Unit c;
                get_unit<RES>(p, cu, c);
                if (units > 0 && !tc::mbar_wait(afree_bar, (units - 1) & 1, abort_flag)) return false;
                ca.start(p.a, tid, c.m0 + rank * kRowsA, p.M, 0);
                for (int k = 0; k < p.k_steps; ++k) {
                    Raw<SA> v[PA];
#pragma unroll
                    for (int i = 0; i < PA; ++i) ca.template load<VEC>(v[i], i, p.K);
#pragma unroll
                    for (int i = 0; i < PA; ++i)
                        piece_store<SA, kLimbA>(v[i], base + k * (LA * kLimbA) + oa + i * (CA::kRows * 128));
                    ca.advance(p.a);
                }
                rest = (c.nt1 - c.nt) * p.k_steps;
                cu += pairs;
                ++units;
            }
            if (RES) --rest;
            if (!tc::mbar_wait(empty_bar(s), ph ^ 1u, abort_flag)) return false;
            if (VEC && (t.s1 - left + 1) * BK <= p.K) body(r, std::true_type());
            else body(r, std::false_type());
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(full_bar(s));
            if (++s == ST) { s = 0; ph ^= 1u; }
            return true;
        };
        fill(set);
        next();
        while (true) {
            const bool v0 = more;
            if (!process(set)) break;
            next();
            if (!v0) break;
        }
    } else if (warp < kEpiWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
        if (warp == kMmaWarp && rank == 0) {
            // -------------------------------------------- MMA issuer.  The whole warp walks the
            // steps, so that descriptors stay in uniform registers; one elected lane issues.
            // The descriptors of a stage differ from the first stage's in the address field alone.
            const bool leader = tc::elect_one();
            constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((MNA ? 1u : 0u) << 15) |
                                       ((MNB ? 1u : 0u) << 16) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
            const uint64_t da = MNA ? mn_desc(base) : tc::sw128_desc(base);
            const uint64_t db = MNB ? mn_desc(base + ring + bpart) : tc::sw128_desc(base + ring + bpart);
            int s = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true, issued = false;
            Unit t;
            for (int u = pair; ok && get_unit<RES>(p, u, t); u += pairs) {
                int at = 0;
                const int steps = t.s1 - t.s0, total = RES ? (t.nt1 - t.nt) * steps : steps;
                for (int i = 0, step = t.s0; i < total; ++i) {
                    const uint32_t d0 = tmem_base + (uint32_t)(buf * ACC * BN);
                    if (at == 0) {
                        if (!tc::mbar_wait<true>(tempty_bar(buf), bph ^ 1u, abort_flag)) { ok = false; break; }
                    }
                    if (!tc::mbar_wait<true>(full_bar(s), ph, abort_flag)) { ok = false; break; }
                    tc::fence_acquire_shared();
                    tc::tc_fence_after();
                    const uint64_t sa = da + (uint32_t)(RES ? step * (LA * kLimbA >> 4) : s * (kStage >> 4));
                    const uint64_t sb = db + (uint32_t)(s * (kStage >> 4));
                    const int k_left = p.K - step * BK;
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk) {
                            if (16 * kk >= k_left) break;
                            // 16 of k: 32 bytes of a K-major row, 16 rows of an MN-major block
                            constexpr int KA = (MNA ? 2048 : 32) >> 4, KB = (MNB ? 2048 : 32) >> 4;
                            bool low = false;   // whether a small product of this kk was issued
#pragma unroll
                            for (int i = 0; i < LA; ++i)
#pragma unroll
                                for (int j = 0; j < LB; ++j) {
                                    if (i + j > 3) continue;   // below 2^-30 of the product
                                    const uint64_t ad = sa + (uint32_t)(i * (kLimbA >> 4) + kk * KA);
                                    const uint64_t bd = sb + (uint32_t)(j * (kLimbB >> 4) + kk * KB);
                                    const bool add = kk > 0 || at > 0;
                                    if (i + j == 0) {
                                        tc::tc_mma_f16_pair(d0, ad, bd, idesc, add);
                                    } else {
                                        tc::tc_mma_f16_pair(d0 + BN, ad, bd, idesc, add || low);
                                        low = true;
                                    }
                                }
                        }
                        tc::tc_commit_pair(empty_bar(s));
                    }
                    issued = true;
                    __syncwarp();
                    if (++s == ST) { s = 0; ph ^= 1u; }
                    const bool last = ++step == t.s1;      // of a tile
                    if (++at == kChain || last) {
                        if (leader) {
                            tc::tc_commit_pair(tfull_bar(buf));
                            if (RES && i + 1 == total) tc::tc_commit_pair(afree_bar);
                        }
                        __syncwarp();
                        at = 0;
                        if (++buf == 2) { buf = 0; bph ^= 1u; }
                    }
                    if (last) step = t.s0;
                }
            }
            if (!ok && issued && leader) {
                tc::tc_commit_pair(drain_bar);   // completes when every MMA issued so far has finished
                const unsigned long long t0 = tc::globaltimer();
                while (!tc::mbar_try_wait(drain_bar, 0) && tc::globaltimer() - t0 < tc::kWaitLimitNs) {}
            }
            __syncwarp();
        } else if (rank == 1 && warp <= kMmaWarp + 1 && lane == 0) {
            // -------------------------------------------- CTA 1: two threads pass on to the MMA issuer in CTA 0
            // what the loaders (the first) and the epilogue (the second) have completed.  A release at cluster scope
            // alone orders the issuer behind another CTA's threads (a local arrival's ends with the CTA); a loader's
            // own would wait for the loads of its next step, these threads have none in flight: dW 8192 x 1536 x
            // 424 38.4 us, with the loaders' own 42.  A phase is passed on before its barrier can complete the
            // next, which needs the MMAs behind this arrival.
            const bool steps = warp == kMmaWarp;
            int left = 0;
            Unit t;
            for (int u = pair; get_unit<RES>(p, u, t); u += pairs)
                left += (t.nt1 - t.nt) * (steps ? t.s1 - t.s0 : (t.s1 - t.s0 + kChain - 1) / kChain);
            const uint32_t first = steps ? full_bar(0) : tempty_bar(0), end = steps ? full_bar(ST) : tempty_bar(2);
            uint32_t bar = first, ph = 0;
            for (; left > 0 && tc::mbar_wait(bar, ph, abort_flag); --left) {
                tc::tc_fence_after();
                tc::tc_fence_before();
                tc::fence_release_shared();
                tc::mbar_arrive_cluster(bar, 0);
                if ((bar += 8u) == end) { bar = first; ph ^= 1u; }
            }
        }
    } else {
        // ------------------------------------------------ epilogue: TMEM -> float32 sums -> global
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        const int lb = 32 * (warp & 3);                    // TMEM lanes this warp may access
        const int half = (warp - kEpiWarp0) / 4;           // which half of the columns
        int buf = 0;
        uint32_t bph = 0;
        bool ok = true;
        Unit t;
        float* buf32 = epi_buf + (warp - kEpiWarp0) * (32 * kStagePitch);
        for (int u = pair; get_unit<RES>(p, u, t); u += pairs)
        for (int nt = t.nt; nt < t.nt1; ++nt) {
            float sum[BN / 2];
#pragma unroll
            for (int j = 0; j < BN / 2; ++j) sum[j] = 0.f;
            for (int c = t.s0; c < t.s1; c += kChain) {
                if (ok) ok = tc::mbar_wait(tfull_bar(buf), bph, abort_flag);
                if (!ok) break;
                tc::tc_fence_after();
                const uint32_t d0 = tmem_base + ((uint32_t)lb << 16) + (uint32_t)(buf * ACC * BN + BN / 2 * half);
#pragma unroll
                for (int a = ACC - 1; a >= 0; --a)     // the small products first
#pragma unroll
                    for (int h = 0; h < BN / 2; h += 16) {   // 16 at a time: 64 sums stay in registers
                        float v[16];
                        tc::tmem_ld16(d0 + a * BN + h, v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[h + j] += v[j];
                    }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(tempty_bar(buf));
                if (++buf == 2) { buf = 0; bph ^= 1u; }
            }
            if (!ok)
#pragma unroll
                for (int j = 0; j < BN / 2; ++j) sum[j] = __uint_as_float(0x7fffffffu);
            // 32 x 32 sub-tiles through shared memory (lane = row in, so that every store instruction writes
            // whole rows of a sub-tile: four as 16-byte vectors where the output's rows allow, else one)
            const int m0 = t.m0 + rank * kRowsA + lb, rows = min(32, p.M - m0);
            float* out = p.out + t.slice * p.slice;
#pragma unroll
            for (int h = 0; h < BN / 64; ++h) {
                const int c0 = nt * BN + BN / 2 * half + 32 * h;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<float4*>(buf32 + lane * kStagePitch + j) =
                        make_float4(sum[32 * h + j], sum[32 * h + j + 1], sum[32 * h + j + 2], sum[32 * h + j + 3]);
                __syncwarp();
                if ((p.cp & 3) == 0 && (p.N & 3) == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0) {
                    const int n = c0 + 4 * (lane & 7), r0 = lane >> 3;
                    if (n < p.N) {
                        const int part = n / p.cp;
                        float* o = out + ((long long)part * p.M + m0 + r0) * p.cp + (n - part * p.cp);
                        const float* v = buf32 + 4 * (lane & 7);
#pragma unroll 4
                        for (int r = r0; r < rows; r += 4, o += 4LL * p.cp)
                            *reinterpret_cast<float4*>(o) = *reinterpret_cast<const float4*>(v + r * kStagePitch);
                    }
                } else {
                    const int n = c0 + lane;
                    if (n < p.N) {
                        const int part = n / p.cp;
                        float* o = out + ((long long)part * p.M + m0) * p.cp + (n - part * p.cp);
#pragma unroll 4
                        for (int r = 0; r < rows; ++r, o += p.cp) *o = buf32[r * kStagePitch + lane];
                    }
                }
            }
        }
    }
    __syncwarp();
    tc::tc_fence_before();
    tc::cluster_sync();   // neither CTA leaves while the other may signal or read it
    if (warp == kMmaWarp) {
        __syncwarp();
        tc::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
    }
    if (!p.last) pdl_launch_dependents();
}

// dw = the slices' partial tiles [slices][M][ld], added in slice order.
__global__ void __launch_bounds__(256)
lin_reduce_kernel(const float* __restrict__ part, int slices, long long slice, int M, int N, int ld, int cp,
                  float* __restrict__ out)
{
    pdl_wait();
    pdl_launch_dependents();   // the next operator's launch overlaps this grid (13.2 us against 14.3 at 5001 x 1000 x 77)
    const int n4 = (N + 3) / 4;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const int m = (int)(i / n4), n = (int)(i - (long long)m * n4) * 4;
    if (m < M) {
        const float4* src = reinterpret_cast<const float4*>(part + (long long)m * ld + n);
        float4 s = __ldcg(src);
#pragma unroll 4
        for (int k = 1; k < slices; ++k) {
            const float4 v = __ldcg(src + k * (slice >> 2));
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        const float r[4] = {s.x, s.y, s.z, s.w};
        const int p0 = n / cp, at = n - p0 * cp;
        float* dst = out + ((long long)p0 * M + m) * cp + at;
        if (at + 4 <= cp && n + 4 <= N && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
            *reinterpret_cast<float4*>(dst) = s;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < N) out[((long long)((n + j) / cp) * M + m) * cp + (n + j) % cp] = r[j];
        }
    }
}

}  // namespace lin
}  // namespace beam
