// qli_paged_chunk.cu -- the paged attention of qli_paged_attention.cu for many rows that read the same KV head (chunks
// of prompts, several new tokens, wide groups of query heads), on the tcgen05 tensor cores.
//
// A CTA takes up to 256 consecutive (token, query head) rows of a sequence and one KV head, and walks the cached
// positions that some of them see in tiles of 128:
//
//     S = Q K^T  (128 x 128 x D)     P = 2^(S f - m), zero where the row does not see the position     O += P V
//
// with the rows of a product on its M side.  Two streams of products keep the tensor cores busy while the other's
// softmax runs: with more than 128 rows each stream has its own 128 and both walk all tiles; with fewer both share
// the rows, each takes every other tile, and their results are joined at the end.  Roles:
//   * one warp copies the KV head's bytes of a tile's positions by TMA, 16 positions of a page a box;
//   * 4 converter warps, a position per thread, decode them into fp16 operands in shared memory: rows of positions
//     for K and for V (V enters the product with its positions as the K dimension, "MN-major"; its elements come in the
//     order in which a lane of the output's warps reads them); they also copy the queries in and turn them into fp16 there;
//   * one warp issues the products: Q, K and V from shared memory, logits and accumulators in tensor memory, P in the
//     place of the logits it came from;
//   * 4 softmax warps per stream, a row per thread: masked logits, running maximum (raised only when the sum of 64 probabilities
//     passes 65000, which P would not hold much longer: then the rows of O are rescaled), sum in fp32, P to fp16;
//     for float16 outputs what that rounding drops stands beside P in the logits' place and is a product of its own with V
//     (chunks 828 -> 1138 us, prompts 1071 -> 1443: half as many products again).
//   * one warp looks after the work: a CTA that is through takes over CTAs of the grid that have not begun, and the next block's
//     positions and queries are under way while the last one's rows are written.  A sequence's later rows, which see more, begin
//     first; sequences begin in the reverse of the batch's order, whatever their length (chunks of 512, 1000, 33 and 2047 tokens
//     behind 8k to 30k 821 us, the same four in the opposite order 879).
// Where there are few blocks of rows a cluster of CTAs shares a block's tiles, and the partial results are joined
// through distributed shared memory in a fixed order.
//
// Bound by the products (4 D operations a logit): 4 prompts of 15360 tokens in all, 64 / 8 heads of 128, 1.46e12 operations over what
// the rows see, 1086 us, 1.35 PFLOP/s (0.70 of a library's large product); chunks of 3592 tokens behind 67000 cached ones, 32 / 8
// heads, 821 us, 1.51 PFLOP/s (0.78); the prompts with windows of 1024, 495 us, 0.92 PFLOP/s.  What is above the products' time: the
// chain from a stream's logits through its softmax to its next logits, about 3400 cycles a tile for two streams of which the products
// 2048 (tensor memory holds two of S and two of O, so that a stream's S waits for its P to be used), and about 5 us a block of rows
// (the queries, the first and last tiles' masks, 2 us for the output).  So the logits' loads run beside the exponentials (each wait
// for tensor memory costs about 260 cycles), a block's queries and tiles are under way while the last one's rows are written, and
// what is rare stands in calls.  Measured and not kept: S in two halves of 64 positions (1101 us for the chunks, then 925: an operand
// of 128 rows is read from shared memory again for each), two warps that issue products (1190, then 849), P handed on in halves
// (909, then 848), quarters of a tile at a time (1011, then 854), outputs in pieces of 32 bytes a lane (826, then 817).
//
// Masks, pages outside the pool and NaN scales as in qli_paged_attention.cu.  Every wait is bounded (0.2 s, those for
// a task and for the end of one 100 s); on expiry the kernel records kErrTimeout, writes NaN and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cstring>

#include "qli_paged.cuh"

namespace qli {

namespace {

constexpr int kM = 128, kTile = 128;                   // rows and positions of a product
constexpr int kTileChunks = kTile / kChunk;
constexpr int kSoftWarps = 8, kConvWarp = 8, kConvWarps = 4, kMmaWarp = 12, kCopyWarp = 13;      // and one for work
constexpr int kThreads = 32 * 15;
constexpr int kRing = 4, kMaxRaw = 2;
constexpr int kMaxSplits = 8;
constexpr uint32_t kTmemCols = 512, kColO = 256;       // logits of stream q at 128 q
// Probabilities enter the second product in fp16.  The maximum in use is set to 6 below the largest of a row's first 128 logits
// (base 2), so that its sum stands at 2^6 or above from the first tile on, and what becomes 0 (2^-25) lies 2^-31 below it: 100000
// positions 25 bits below one whose value is 0 count (from 2^0 on they were lost).  It is raised when 64 probabilities add up to more
// than fp16 is sure to hold; the warp's other rows then catch up with their largest sum so far, since their next records are near.
// us for 8 / 7 / 6 / 5 below, chunks and prompts: queries of normal values 837 / 837 / 837 / 850 and 1097 / 1095 / 1097 / 1104, with
// twice that spread 884 / 872 / 859 / 855 and 1223 / 1164 / 1130 / 1122 (each row raised alone, 8 below, 1081 and 1672).
constexpr float kBelow = 6.0f, kUnit6 = 1.0f / 64.0f;
constexpr float kMostSum = 65000.0f;
constexpr uint64_t kWaitLimitNs = 200000000ull, kTaskLimitNs = 100000000000ull;     // (the length of a task: 2^31 positions)

struct Layout {
    int32_t rows;          // of a block: 128 or 256
    int32_t blocks;        // BSND: blocks per sequence
    int32_t splits;        // CTAs of a cluster
    uint32_t block_recip;
};

// A block of rows and a KV head
struct Task {
    RowBlock blk;
    KeyRange range;
    int32_t kvh;
    int32_t n;                                         // tiles of this CTA, or one of these
    int32_t tok0;
    uint32_t rest;                                     // global head row of row i: `base` + i + (tokens before it) (heads_q - group)
    int64_t base;
};
constexpr int32_t kNoMore = -1, kBadSums = -2;

struct Shared {
    uint4 taken;                                       // the answer to a request for a pending CTA
    uint64_t rawfull[kMaxRaw], rawfree[kMaxRaw], opfull[kRing], opfree[kRing], sfull[2], pfull[2];
    uint64_t taskfull[2], taskfree[2], qfull, qfree, odone, oread, joined, copied, answer;
    uint32_t tmem, abort;
    uint8_t valid[8];                                  // chunks of a tile that lie in the pool
    Task task[2];
    uint32_t held, asking;                             // 1 + the CTA whose work is not in a task yet; a request is out
    float factor[2][2 * kM];
    float2 ml[2][2][kM];                               // maximum and sum of the streams' shared rows
};

template <int D>
struct Sizes {
    static constexpr int atom = kM * 128;              // 128 rows of 64 fp16 in the 128-byte swizzle
    static constexpr int operand = D / 64 * atom;      // 128 rows of D
    // the KV head's bytes of a position, from a multiple of 16 on (heads of 72 bytes start on a multiple of 8)
    static constexpr int raw_row = D == 128 ? 144 : 80;
    static constexpr int raw = kTile * raw_row;
    // Q (one or two blocks of rows), a ring of operands, and copied bytes: one stage, or two in place of the second
    // block of rows
    static constexpr int shared_at = (2 + kRing) * operand + raw;
    static constexpr int smem = shared_at + (int)sizeof(Shared);
    static_assert(kMaxRaw * raw <= operand + raw, "copied bytes");
};

__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile uint32_t* abort, uint32_t* err,
                                             uint64_t limit = kWaitLimitNs)
{
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = ptx::globaltimer();
    while (!__all_sync(0xffffffffu, ptx::mbar_try_wait_sleep(bar, parity, 100000u))) {
        if (__any_sync(0xffffffffu, *abort != 0)) return false;
        if (__any_sync(0xffffffffu, ptx::globaltimer() - t0 > limit)) {
            *abort = 1;
            if (err) atomicOr(err, kErrTimeout);
            return false;
        }
    }
    return true;
}

// `kBelow` under a logit, rounded up: logits that fp32 holds in steps of 16 have their largest at 2^0, not at 2^16
__device__ __forceinline__ float below(float top) { return __fadd_ru(top, -kBelow); }

// ln of a row's sum of exponentials, held as `sum` of 2^(z - m)
__device__ __forceinline__ float lse_of(float m, float sum)
{
    return sum == 0.0f ? -INFINITY : (m + kBelow + log2f(sum * kUnit6)) * 0.6931471805599453f;
}

// What a row's accumulators are multiplied by, and its lse
__device__ __noinline__ float2 end_of_row(float m, float sum)
{
    sum = sum_that_counts(m, sum);
    return make_float2(sum == 0.0f ? 0.0f : 1.0f / sum, lse_of(m, sum));
}

// Wait for this thread's loads from tensor memory; the registers pass through it, so that nothing that uses
// them moves in front
template <int N>
__device__ __forceinline__ void wait_loaded(uint32_t (&r)[N])
{
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Byte offset of 16-byte piece `piece` (eight fp16) of row r in an operand
template <int D>
__device__ __forceinline__ uint32_t operand_at(int r, int piece)
{
    return (piece >> 3) * Sizes<D>::atom + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
}

// The low n bits, n clamped to [0, 16]
__device__ __forceinline__ uint32_t low16(int n) { return (1u << min(max(n, 0), 16)) - 1; }

// Bits of the chunk's positions that a row with end `hi` sees
__device__ __forceinline__ uint32_t chunk_bits(const PagedArgs& a, const KeyRange& range, int chunk, int hi)
{
    const int pos = range.position(chunk);
    uint32_t bits = low16(min(hi, range.limit(chunk)) - pos);
    if (a.window > 0) bits &= ~low16(hi - a.window - pos) | low16(a.sinks - pos);
    return bits;
}

// Eight scale bytes times 16-element blocks: prepared pairs
template <bool E2M1, int N>
__device__ __forceinline__ void scale_pairs(const uint32_t (&w)[N], bool finite, PairScale (&g)[4 * N])
{
#pragma unroll
    for (int i = 0; i < 2 * N; ++i) {
        uint32_t h = e4m3x2_to_f16x2(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu);
        if (finite) h = finite_f16x2(h);
        g[2 * i] = pair_scale<E2M1>(__byte_perm(h, 0, 0x1010));
        g[2 * i + 1] = pair_scale<E2M1>(__byte_perm(h, 0, 0x3232));
    }
}

// One position's codes of K or V: for D = 128 16 bytes at a time (eight lanes' rows, 144 bytes apart, lie in
// different banks), heads of 72 bytes 8 at a time
template <int D>
__device__ __forceinline__ void load_codes(const uint8_t* src, uint32_t (&w)[D / 8])
{
    if constexpr (D == 128) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint4 x = reinterpret_cast<const uint4*>(src)[i];
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint2 x = reinterpret_cast<const uint2*>(src)[i];
            w[2 * i] = x.x, w[2 * i + 1] = x.y;
        }
    }
}

// One position's codes (D / 8 words) times their scales into row `row` of an operand
template <bool E2M1, int D>
__device__ __forceinline__ void store_row(uint8_t* operand, int row, const uint32_t (&code)[D / 8], const PairScale (&g)[D / 16])
{
    uint8_t* dst = operand + row * 128;
    const int flip = (row & 7) << 4;
#pragma unroll
    for (int p = 0; p < D / 8; ++p) {
        uint32_t o[4];
        decode_pairs<E2M1>(code[p], g[p / 2], o);
        *reinterpret_cast<uint4*>(dst + (p >> 3) * Sizes<D>::atom + (((p & 7) << 4) ^ flip)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// The same of V, with the elements of each 32 in an order of their own: pair k of word c (of four) is columns 8 k + 2 c and the
// next, so that a lane that reads those of k = 0 ... 3 from the accumulators has a word's eight elements
template <bool E2M1, int D>
__device__ __forceinline__ void store_values(uint8_t* operand, int row, const uint32_t (&code)[D / 8], const PairScale (&g)[D / 16])
{
    uint8_t* dst = operand + row * 128;
    const int flip = (row & 7) << 4;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
        uint32_t o[4][4];
#pragma unroll
        for (int c = 0; c < 4; ++c) decode_pairs<E2M1>(code[4 * b + c], g[2 * b + c / 2], o[c]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(dst + (b >> 1) * Sizes<D>::atom + ((((b & 1) * 4 + k) << 4) ^ flip)) =
                make_uint4(o[0][k], o[1][k], o[2][k], o[3][k]);
    }
}

// Probabilities 2^(s f - m) of 32 of a row's logits, in fp16 pairs, and their sum onto `part`; F16: what the rounding dropped, too
template <bool F16>
__device__ __forceinline__ void soft_part(const uint32_t (&s)[32], float f, float m, uint32_t* p, uint32_t* rest, uint64_t (&part)[2])
{
    const uint64_t F = ptx::pack2(f, f), M = ptx::pack2(-m, -m);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        float zx, zy;
        ptx::unpack2(ptx::fma2(ptx::pack2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), F, M), zx, zy);
        const float px = ptx::ex2(zx), py = ptx::ex2(zy);
        part[e >> 1 & 1] = ptx::add2(part[e >> 1 & 1], ptx::pack2(px, py));
        p[e / 2] = float2_to_act2<true>(px, py);
        if constexpr (F16) rest[e / 2] = remainder_f16x2(px, py, p[e / 2]);
    }
}
__device__ __forceinline__ float sum_of(const uint64_t (&part)[2])
{
    float sum, other;
    ptx::unpack2(ptx::add2(part[0], part[1]), sum, other);
    return sum + other;
}

// The rarer steps are calls, so that they take no registers from the ones above.

// The largest of a row's 64 logits (NaN: of the others)
__device__ __noinline__ float max_half(uint32_t cols)
{
    uint32_t s[2][32];
    QLI_TMEM_LD_X32(cols, s[0]);
    QLI_TMEM_LD_X32(cols + 32, s[1]);
    wait_loaded(s[0]);
    wait_loaded(s[1]);
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < 32; ++e) top = ptx::max3(top, __uint_as_float(s[0][e]), __uint_as_float(s[1][e]));
    return top;
}

// The probabilities of a row's 64 logits from column `cols` on into the 32 columns from `to` on (F16: what their rounding dropped
// into the 32 behind these), and their sum
template <bool F16>
__device__ __noinline__ float soft_half(uint32_t cols, uint32_t to, float f, float m)
{
    uint32_t s[2][32], p[32], rest[32];
    QLI_TMEM_LD_X32(cols, s[0]);
    QLI_TMEM_LD_X32(cols + 32, s[1]);
    wait_loaded(s[0]);
    wait_loaded(s[1]);
    uint64_t part[2] = {0, 0};
    soft_part<F16>(s[0], f, m, p, rest, part);
    soft_part<F16>(s[1], f, m, p + 16, rest + 16, part);
    QLI_TMEM_ST_X32(to, p);
    if constexpr (F16) QLI_TMEM_ST_X32(to + 32, rest);
    ptx::tmem_wait_st();
    return sum_of(part);
}

// -infinity for those of a row's 64 logits whose bit is not set
__device__ __noinline__ void mask_half(uint32_t cols, uint32_t bits0, uint32_t bits1)
{
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
        const uint32_t bits = c ? bits1 : bits0;
        uint32_t s[32];
        QLI_TMEM_LD_X32(cols + 32 * c, s);
        wait_loaded(s);
#pragma unroll
        for (int e = 0; e < 32; ++e) s[e] = bits & (1u << e) ? s[e] : 0xFF800000u;
        QLI_TMEM_ST_X32(cols + 32 * c, s);
    }
    ptx::tmem_wait_st();
}

// A row's accumulators (32 n columns) times g
__device__ __noinline__ void scale_row(uint32_t cols, int n, float g)
{
#pragma unroll 1
    for (int x = 0; x < n; ++x) {
        uint32_t o[32];
        QLI_TMEM_LD_X32(cols + 32 * x, o);
        wait_loaded(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * g);
        QLI_TMEM_ST_X32(cols + 32 * x, o);
    }
}

// A row's 64 probabilities times g (F16: with what their rounding dropped, rounded anew)
template <bool F16>
__device__ __noinline__ void scale_half(uint32_t cols, float g)
{
    uint32_t o[32], rest[32];
    ptx::tmem_wait_st();
    QLI_TMEM_LD_X32(cols, o);
    if constexpr (F16) QLI_TMEM_LD_X32(cols + 32, rest);
    wait_loaded(o);
    if constexpr (F16) wait_loaded(rest);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
        float2 v = act2_to_float2<true>(o[e]);
        if constexpr (F16) {
            const float2 r = act2_to_float2<true>(rest[e]);
            v.x += r.x, v.y += r.y;                        // (exact: 22 bits)
        }
        o[e] = float2_to_act2<true>(v.x * g, v.y * g);
        if constexpr (F16) rest[e] = remainder_f16x2(v.x * g, v.y * g, o[e]);
    }
    QLI_TMEM_ST_X32(cols, o);
    if constexpr (F16) QLI_TMEM_ST_X32(cols + 32, rest);
}

// A lane's eight elements of a row (of 32 columns, in the order of store_values), times f
template <bool E2M1>
__device__ __forceinline__ float element(const uint32_t (&o)[16], int half, int e)
{
    return __uint_as_float(E2M1 ? o[4 * (e >> 1) + 2 * half + (e & 1)] : o[4 * (e & 3) + 2 * half + (e >> 2)]);
}

// Columns [32 from, 32 to) of a warp's 32 rows' accumulators from `acc` on, times f0 (with `both`, and those D further times
// f1; without `some`, zeros): times g into the output, or as fp32 into `partial`.  A lane has eight elements of rows lane / 4 + 8 i, which
// begin at elements at0 ... at3 (-1: none); f0 and f1 are those of row `lane`.
template <bool F16, bool E2M1, int D>
__device__ __noinline__ void write_rows(uint32_t acc, int from, int to, bool both, bool some, float f0, float f1, float g, uint16_t* dst, int64_t at0,
                                        int64_t at1, int64_t at2, int64_t at3, float* partial)
{
    constexpr int kStride = D + 4;
    const int lane = threadIdx.x & 31, r = lane >> 2;
    const int64_t at[4] = {at0, at1, at2, at3};
    float a0[4], a1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a0[i] = __shfl_sync(0xffffffffu, f0, r + 8 * i);
        a1[i] = __shfl_sync(0xffffffffu, f1, r + 8 * i);
    }
    auto put = [&](int x, int i, const float (&v)[8]) {
        if (partial) {
            float4* to4 = reinterpret_cast<float4*>(partial + (r + 8 * i) * kStride + 32 * x + 8 * (lane & 3));
            to4[0] = make_float4(v[0], v[1], v[2], v[3]);
            to4[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else if (at[i] >= 0) {
            *reinterpret_cast<uint4*>(dst + at[i] + 32 * x) =
                make_uint4(float2_to_act2<F16>(v[0] * g, v[1] * g), float2_to_act2<F16>(v[2] * g, v[3] * g),
                           float2_to_act2<F16>(v[4] * g, v[5] * g), float2_to_act2<F16>(v[6] * g, v[7] * g));
        }
    };
    // two blocks of 32 columns, or one of both accumulators
#pragma unroll 1
    for (int x = from; x < to; x += both ? 1 : 2) {
        uint32_t o[2][2][16];
        const uint32_t second = both ? acc + D + 32 * x : acc + 32 * x + 32;
        if (some) {
            QLI_TMEM_LD_16X256_X4(acc + 32 * x, o[0][0]);
            QLI_TMEM_LD_16X256_X4(acc + 32 * x + (16u << 16), o[0][1]);
            QLI_TMEM_LD_16X256_X4(second, o[1][0]);
            QLI_TMEM_LD_16X256_X4(second + (16u << 16), o[1][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) wait_loaded(o[i >> 1][i & 1]);
        } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) o[i >> 5][i >> 4 & 1][i & 15] = 0;
        }
        if (both) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = fmaf(a0[i], element<E2M1>(o[0][i >> 1], i & 1, e), a1[i] * element<E2M1>(o[1][i >> 1], i & 1, e));
                put(x, i, v);
            }
        } else {
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = a0[i] * element<E2M1>(o[y][i >> 1], i & 1, e);
                    put(x + y, i, v);
                }
        }
    }
    __syncwarp();
}

// The block number `slot`, found by a warp (as find_rows); false: the prefix sums are invalid.  `checked`: they have been looked
// at as a whole (and will have been), so that a search finds the sequence: of 50000 without new tokens each number costs a few
// loads, not 1563.
__device__ __forceinline__ bool find_rows_warp(const PagedArgs& a, uint32_t slot, int blocks, int M, int group, bool& checked,
                                               RowBlock& r)
{
    const Params& p = a.p;
    const int lane = threadIdx.x & 31;
    int b, block;
    if (!p.layout_tnd) {
        b = (int)(slot / (uint32_t)blocks);
        block = (int)(slot - (uint32_t)b * blocks);
    } else if (checked) {
        // the number of sequences that begin at or before the block lies in [b, b + n]: each lane asks for the last of a piece
        b = 0;
        for (uint32_t n = (uint32_t)p.batch; n > 0;) {
            const uint32_t step = (n + 31) / 32;
            const int i = b + (int)min((lane + 1) * step, n) - 1;
            const bool before = (int64_t)a.seq_lens_q[i] * group / M + i + 1 <= (int64_t)slot;
            const uint32_t past = min(__popc(__ballot_sync(0xffffffffu, before)) * step, n);
            b += (int)past;
            n = past < n ? min(step, n - past) - 1 : 0;    // (that piece's last is not among them)
        }
        const int64_t done = b > 0 ? a.seq_lens_q[b - 1] : 0;
        block = (int)((int64_t)slot - (done * group / M + b));
    } else {
        bool bad = false;
        b = 0;
        for (int i0 = 0; i0 < p.batch; i0 += 32) {
            const int i = i0 + lane;
            bool before = false;
            if (i < p.batch) {
                const int64_t lo = i > 0 ? a.seq_lens_q[i - 1] : 0, hi = a.seq_lens_q[i];
                if (lo < 0 || hi < lo || hi > p.total_q) bad = true;
                else before = hi * group / M + i + 1 <= (int64_t)slot;
            }
            b += __popc(__ballot_sync(0xffffffffu, before));
        }
        if (__any_sync(0xffffffffu, bad)) return false;
        checked = true;
        const int64_t done = b > 0 ? a.seq_lens_q[b - 1] : 0;
        block = (int)((int64_t)slot - (done * group / M + b));
    }
    rows_of_block(a, b, block, M, group, lane == 0, r);
    return true;
}

// The rare step of a row's 64 logits at cols + 64 h, whose probabilities add up to too much for fp16 in some row of the warp: raise the
// maximum to the logits that are left of the tile, of rows that do not need it also so that their largest sum stands near 2^6,
// rescale sums, accumulators (32 n columns from `acc` on) and the tile's first half of P, and take the probabilities again.
struct Running {
    float m, l, best;                                      // maximum in use, sum, largest sum of 64
};
template <bool F16>
__device__ __noinline__ Running raise_rows(uint32_t cols, int h, int half_cols, uint32_t acc, int n, float f, float sum, Running r)
{
    const float top = below((h == 0 ? fmaxf(max_half(cols), max_half(cols + 64)) : max_half(cols + 64)) * f);
    const float more = r.best > 2 / kUnit6 ? (float)(int)(__float_as_uint(r.best) >> 23) - (127 + kBelow) : 0.0f;
    const float up = fmaxf(top, sum > kMostSum ? r.m : __fadd_rd(r.m, more));
    const float g = ptx::ex2(r.m - up);
    r.m = up;
    if (h == 1) scale_half<F16>(cols, g);
    scale_row(acc, n, g);
    const float now = soft_half<F16>(cols + 64 * h, cols + half_cols * h, f, up);
    r.l = r.l * g + now;
    r.best = fmaxf(r.best * g, now);
    return r;
}

template <bool F16, bool E2M1, int D>
__device__ __noinline__ uint32_t turn_row(uint8_t* base, int row)
{
    constexpr int kPieces = D / 8;
    uint32_t ex = 127;
    uint4 w[kPieces];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) w[p] = *reinterpret_cast<const uint4*>(base + operand_at<D>(row, p));
    float down = 1.0f;
    if constexpr (!F16) {
        uint32_t most = 0;                                 // magnitudes order like integers
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            most = __vmaxu2(most, __vmaxu2(w[p].x & 0x7FFF7FFFu, w[p].y & 0x7FFF7FFFu));
            most = __vmaxu2(most, __vmaxu2(w[p].z & 0x7FFF7FFFu, w[p].w & 0x7FFF7FFFu));
        }
        most = max(most & 0xFFFFu, most >> 16);
        ex = min(max(most >> 7, 1u), 253u);
        down = __uint_as_float((254u - ex) << 23);         // 2^-(exponent of the largest)
    }
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        uint32_t o[4] = {w[p].x, w[p].y, w[p].z, w[p].w};
        if constexpr (!F16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 v = act2_to_float2<F16>(o[e]);
                o[e] = float2_to_act2<true>(v.x * down, v.y * down);
            }
        }
        *reinterpret_cast<uint4*>(base + operand_at<D>(row, p)) =
            E2M1 ? make_uint4(o[0], o[1], o[2], o[3])
                 : make_uint4(__byte_perm(o[0], o[2], 0x5410), __byte_perm(o[0], o[2], 0x7632), __byte_perm(o[1], o[3], 0x5410),
                              __byte_perm(o[1], o[3], 0x7632));
    }
    return ex;
}

template <bool F16, bool E2M1, int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ Layout L,
                       const __grid_constant__ CUtensorMap pages)
{
    using Z = Sizes<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem + Z::shared_at);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = a.heads_q / a.heads_kv;
    const int rank = L.splits > 1 ? (int)ptx::cluster_rank() : 0;
    uint8_t* const ring = smem + (L.rows == kM ? 1 : 2) * Z::operand;
    uint8_t* const raw = ring + kRing * Z::operand;
    const int raw_stages = L.rows == kM ? kMaxRaw : 1;

    if (tid == 0) {
        for (int i = 0; i < kMaxRaw; ++i) {
            ptx::mbar_init(&sh.rawfull[i], 1);
            ptx::mbar_init(&sh.rawfree[i], kConvWarps);
        }
        for (int i = 0; i < kRing; ++i) {
            ptx::mbar_init(&sh.opfull[i], kConvWarps);
            ptx::mbar_init(&sh.opfree[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sh.sfull[i], 1);
            ptx::mbar_init(&sh.pfull[i], 4);
            ptx::mbar_init(&sh.taskfull[i], 1);
            ptx::mbar_init(&sh.taskfree[i], kSoftWarps + kConvWarps + 2);
            sh.task[i].blk.rows = 0;
        }
        ptx::mbar_init(&sh.qfull, kConvWarps);
        ptx::mbar_init(&sh.qfree, 1);
        ptx::mbar_init(&sh.odone, 1);
        ptx::mbar_init(&sh.oread, kSoftWarps);
        ptx::mbar_init(&sh.joined, kSoftWarps);
        ptx::mbar_init(&sh.copied, 1);
        ptx::mbar_init(&sh.answer, 1);
        sh.held = blockIdx.x / (uint32_t)L.splits + 1;
        sh.asking = 0;
        sh.abort = 0;
        ptx::fence_mbar_init();
    }
    ptx::pdl_wait();
    if (warp == kMmaWarp) {                                // (not before: kernels that still run may need it)
        ptx::tmem_alloc(&sh.tmem, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sh.tmem;

    // whether the streams share a task's rows, and a stream's steps and tiles
    auto shares = [](const Task& k) { return k.blk.rows <= kM; };
    auto steps_of = [&](const Task& k, int q) { return shares(k) ? (k.n - q + 1) / 2 : k.n; };
    auto tile_of = [&](const Task& k, int q, int j) { return shares(k) ? 2 * j + q : j; };
    // global head row of a task's row i: `base` + i + (tokens before it) (heads_q - group)
    const uint32_t recip = (1u << 22) / group + 1;         // exact quotients of numbers below 512 by up to 256
    auto set_heads = [&](Task& k) {
        k.tok0 = k.blk.first / group;
        k.rest = (uint32_t)(k.blk.first - k.tok0 * group);
        k.base = (k.blk.row0 + k.tok0) * a.heads_q + k.kvh * group + k.rest;
    };
    auto head_of = [&](const Task& h, int i) { return h.base + i + (int)((h.rest + i) * recip >> 22) * (a.heads_q - group); };
    // the next task; false when a wait gave up.  (The softmax warps read theirs in place and hand it back at its end.)
    auto next_task = [&](int it, Task& k) {
        if (!wait_bounded(&sh.taskfull[it & 1], it >> 1 & 1, &sh.abort, a.err, kTaskLimitNs)) return false;
        k = sh.task[it & 1];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh.taskfree[it & 1]);
        return true;
    };
    uint16_t* const dst = static_cast<uint16_t*>(a.out);
    constexpr int kStride = D + 4;                         // of partial rows (splits), in floats
    float* const part_o = reinterpret_cast<float*>(smem);  // [2 * kM][kStride], then the rows' (maximum, sum)
    float2* const part_ml = reinterpret_cast<float2*>(part_o + 2 * kM * kStride);
    static_assert(2 * kM * (kStride * 4 + 8) <= Z::shared_at, "partial results in the operands' place");
    Task task;
    // columns from the probabilities of a tile's first 64 positions to the others': F16, what their rounding dropped stands between
    constexpr int kHalfCols = F16 ? 64 : 32;

    if (warp < kSoftWarps) {
        // ---------------------------------------------------------------- softmax
        const int q = warp >> 2, lane_row = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21), cols = lanes + kTile * q, out = lanes + kColO;
        uint32_t step = 0, tiles = 0, turn = 0;            // steps, tiles and tasks with tiles so far
        uint32_t joins = 0;
        for (int it = 0;; ++it) {
            const Task& task = sh.task[it & 1];
            if (!wait_bounded(&sh.taskfull[it & 1], it >> 1 & 1, &sh.abort, a.err, kTaskLimitNs) || task.n < 0) break;

            const bool shared = shares(task);
            const int row = (shared ? 0 : q * kM) + lane_row, steps = steps_of(task, q);
            const bool idle = (row & ~31) >= task.blk.rows;
            Running run = {-FLT_MAX, 0.0f, 0.0f};
            bool ok = true;
            if (task.n > 0) {
                const int hi = seen_end(a, task.blk, task.tok0 + (int)((task.rest + row) * recip >> 22));
                if (!wait_bounded(&sh.qfull, turn & 1, &sh.abort, a.err)) break;
                const float f = sh.factor[turn & 1][row];
                for (int j = 0; j < steps; ++j, ++step) {
                    const int t = tile_of(task, q, j), ch = kTileChunks * (t * L.splits + rank);
                    ok = wait_bounded(&sh.sfull[q], step & 1, &sh.abort, a.err);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    // (a warp without rows hands its part of P on as it is: it weighs in no row that counts)
                    if (idle) {
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&sh.pfull[q]);
                        continue;
                    }
                    const uint32_t valid = sh.valid[(tiles + t) & 7];
                    const bool whole = valid == 0xFFu && task.range.all_see(ch, kTileChunks);
                    if (!whole) {
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            uint32_t bits[2];
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const int x = 4 * h + 2 * c;
                                bits[c] = chunk_bits(a, task.range, ch + x, hi) | chunk_bits(a, task.range, ch + x + 1, hi) << 16;
                                if (!(valid >> x & 1)) bits[c] &= 0xFFFF0000u;
                                if (!(valid >> (x + 1) & 1)) bits[c] &= 0x0000FFFFu;
                            }
                            mask_half(cols + 64 * h, bits[0], bits[1]);
                        }
                    }
                    if (j == 0) run.m = fmaxf(run.m, below(fmaxf(max_half(cols), max_half(cols + 64)) * f));
                    // half a tile at a time, each 32 logits on their way while those before are worked on
                    uint32_t s[2][32];
                    QLI_TMEM_LD_X32(cols, s[0]);
                    wait_loaded(s[0]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t p[32], rest[32];
                        uint64_t part[2] = {0, 0};
                        QLI_TMEM_LD_X32(cols + 64 * h + 32, s[1]);
                        soft_part<F16>(s[0], f, run.m, p, rest, part);
                        wait_loaded(s[1]);
                        if (h == 0) QLI_TMEM_LD_X32(cols + 64, s[0]);
                        soft_part<F16>(s[1], f, run.m, p + 16, rest + 16, part);
                        if (h == 0) wait_loaded(s[0]);
                        const float sum = sum_of(part);
                        if (__any_sync(0xffffffffu, sum > kMostSum)) {
                            // (The stream's last product was issued before these logits, and has ended.  What is in registers
                            // does not live through the call.)
                            run = raise_rows<F16>(cols, h, kHalfCols, out + D * q, j > 0 ? D / 32 : 0, f, sum, run);
                            QLI_TMEM_LD_X32(cols + 64, s[0]);
                            wait_loaded(s[0]);
                        } else {
                            run.l += sum;
                            run.best = fmaxf(run.best, sum);
                            QLI_TMEM_ST_X32(cols + kHalfCols * h, p);     // in the place of the logits that are through
                            if constexpr (F16) QLI_TMEM_ST_X32(cols + kHalfCols * h + 32, rest);
                        }
                    }
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(&sh.pfull[q]);
                }
                if (!ok) break;
            }
            // ---- the rows' outputs.  Shared rows: each stream's warps join half of the elements of both accumulators.
            // (What there is to know before the last products end.)
            float g[2] = {1.0f, 0.0f};
            float top = run.m, sum = run.l;
            const bool both = shared && steps_of(task, 1) > 0;
            if (both) {
                sh.ml[joins & 1][q][lane_row] = make_float2(run.m, run.l);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sh.joined);
                if (!wait_bounded(&sh.joined, joins & 1, &sh.abort, a.err)) break;
                const float2 u = sh.ml[joins & 1][0][lane_row], v = sh.ml[joins & 1][1][lane_row];
                ++joins;
                top = fmaxf(u.x, v.x);
                g[0] = ptx::ex2(u.x - top);
                g[1] = ptx::ex2(v.x - top);
                sum = fmaf(g[0], u.y, g[1] * v.y);
            }
            // (a stream without steps of its own leaves shared rows to the other)
            const bool writes = !shared || both || q == 0;
            const int from = both ? q * (D / 64) : 0, to = both ? from + D / 64 : D / 32;
            const uint32_t acc = out + (shared ? 0 : D * q);
            int64_t at[4];                                 // of the rows that this lane writes
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int w = (row & ~31) + (lane >> 2) + 8 * i;
                at[i] = w < task.blk.rows ? head_of(task, w) * D + 8 * (lane & 3) : -1;
            }
            const float2 end = L.splits > 1 ? make_float2(1.0f, 0.0f) : end_of_row(top, sum);
            const float inv = end.x;
            if (L.splits == 1 && writes && from == 0 && row < task.blk.rows && a.lse)
                a.lse[head_of(task, row)] = end.y;
            if (task.n > 0) {
                if (!wait_bounded(&sh.odone, turn & 1, &sh.abort, a.err)) break;
                ptx::tc_fence_after();
            }
            // (the operands' place is free now)
            if (L.splits > 1 && writes && from == 0) part_ml[row] = make_float2(top, sum);
            if (writes && !idle)
                write_rows<F16, E2M1, D>(acc, from, to, both, task.n > 0, g[0] * inv, g[1] * inv, a.v_scale, dst, at[0], at[1], at[2], at[3],
                                         L.splits > 1 ? part_o + (row & ~31) * kStride : nullptr);
            if (task.n > 0) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sh.oread);
            }
            tiles += task.n;
            turn += task.n > 0;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sh.taskfree[it & 1]);
        }
    } else if (warp < kMmaWarp) {
        // ---------------------------------------------------------------- converters, a position per thread
        const int row = tid - 32 * kConvWarp;
        const bool stall = a.p.test_stall == 1;            // test switch: no tile is handed on, the waits run out
        int rs = 0;
        uint32_t rp = 0, tiles = 0, turn = 0;
        // the task's queries as operands: row m is row blk.first + m of the sequence, in fp16 (float16 as it is, bfloat16
        // times a power of two of its largest magnitude; for int4 each eight elements in the order 0 4 1 5 2 6 3 7, as its
        // codes come).  They are copied into place, and what there is to change is changed there, a row per thread.
        auto queries = [&](const Task& task) {
            if (turn > 0 && !wait_bounded(&sh.qfree, turn - 1 & 1, &sh.abort, a.err)) return false;
            constexpr int kPieces = D / 8;
            const int mine = 32 * (warp - kConvWarp), halves = shares(task) ? 1 : 2;
            const int64_t first = task.tok0;
            for (int h = 0; h < halves; ++h)
#pragma unroll 4
                for (int x = lane / kPieces; x < 32; x += 32 / kPieces) {
                    const int m = kM * h + mine + x, piece = lane % kPieces;
                    const uint32_t i = task.rest + m, tok = i * recip >> 22;
                    const bool some = m < task.blk.rows;
                    const uint16_t* src = static_cast<const uint16_t*>(a.query);
                    if (some) src += (task.blk.row0 + first + tok) * a.q_stride + (task.kvh * group + (int)(i - tok * group)) * D + 8 * piece;
                    ptx::cp_async16(smem + h * Z::operand + operand_at<D>(mine + x, piece), src, some);
                }
            ptx::cp_async_wait_all();
            __syncwarp();
            for (int h = 0; h < halves; ++h) {
                uint8_t* const base = smem + h * Z::operand;
                const uint32_t ex = F16 && E2M1 ? 127u : turn_row<F16, E2M1, D>(base, row);
                // (above zero: the mask's -infinity times it stays -infinity)
                sh.factor[turn & 1][kM * h + row] =
                    fminf(fmaxf(__uint_as_float(ex << 23) * (a.softmax_scale * a.k_scale * 1.4426950408889634f), 1.0e-30f), 3.0e38f);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sh.qfull);
            return true;
        };
        for (int it = 0;; ++it) {
            if (!next_task(it, task) || task.n < 0) break;
            if (task.n == 0) continue;
            const int lo = task.kvh * kv_unit_bytes(D) & 8;                    // (heads of 72 bytes)
            bool ok = true;
            for (int t = 0;; ++t, ++tiles) {
                // (behind the first tile, or before it: the queries of the task before are needed until its last logits are there)
                if (t == (turn > 0)) ok = queries(task);
                if (!ok || t == task.n) break;
                // the position's bytes into registers: the next tile's may land
                const uint8_t* src = raw + rs * Z::raw + row * Z::raw_row + lo;
                ok = wait_bounded(&sh.rawfull[rs], rp, &sh.abort, a.err);
                if (!ok) break;
                uint32_t kc[D / 8], vc[D / 8], ks[D / 64], vs[D / 64];
                load_codes<D>(src, kc);
                load_codes<D>(src + D / 2, vc);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    ks[i] = reinterpret_cast<const uint32_t*>(src + D)[i];
                    vs[i] = reinterpret_cast<const uint32_t*>(src + D + D / 16)[i];
                    // a NaN (0x7F or 0xFF) among the values' scales becomes one of the keys'
                    ks[i] |= __vcmpeq4(vs[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sh.rawfree[rs]);
                if (++rs == raw_stages) rs = 0, rp ^= 1;
                // fills 2 tiles and 2 tiles + 1 of the ring
                const int sk = 2 * tiles & 3, sv = sk + 1;
                const uint32_t free_phase = (tiles >> 1 & 1) ^ 1;
                PairScale g[D / 16];
                scale_pairs<E2M1>(ks, false, g);
                ok = wait_bounded(&sh.opfree[sk], free_phase, &sh.abort, a.err);
                if (!ok) break;
                store_row<E2M1, D>(ring + sk * Z::operand, row, kc, g);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && !stall) ptx::mbar_arrive(&sh.opfull[sk]);
                scale_pairs<E2M1>(vs, true, g);
                ok = wait_bounded(&sh.opfree[sv], free_phase, &sh.abort, a.err);
                if (!ok) break;
                store_values<E2M1, D>(ring + sv * Z::operand, row, vc, g);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && !stall) ptx::mbar_arrive(&sh.opfull[sv]);
            }
            if (!ok) break;
            ++turn;
        }
    } else if (warp == kCopyWarp) {
        // ---------------------------------------------------------------- copies, a chunk per lane
        int rs = 0;
        uint32_t rp = 1, tiles = 0;
        for (int it = 0;; ++it) {
            if (!next_task(it, task) || task.n < 0) break;
            const int32_t* table = a.block_table + (int64_t)task.blk.batch * a.p.max_blocks_per_seq;
            const int x = (task.kvh * kv_unit_bytes(D) & ~15) / 8;
            int at = 0, page = INT32_MIN;
            if (task.n > 0 && lane < kTileChunks) page = chunk_page(a, task.range, table, L.block_recip, kTileChunks * rank + lane, &at);
            bool ok = true;
            for (int t = 0; t < task.n; ++t, ++tiles) {
                const int pg = page, ps = at;
                const bool here = pg >= 0 && pg < a.p.num_blocks;
                if (!here && pg != INT32_MIN && a.err) atomicOr(a.err, kErrPage);
                const uint32_t live = __ballot_sync(0xffffffffu, here);
                if (t + 1 < task.n && lane < kTileChunks)
                    page = chunk_page(a, task.range, table, L.block_recip, kTileChunks * ((t + 1) * L.splits + rank) + lane, &at);
                ok = wait_bounded(&sh.rawfree[rs], rp, &sh.abort, a.err);
                if (!ok) break;
                if (lane == 0) {
                    sh.valid[tiles & 7] = (uint8_t)live;
                    ptx::mbar_arrive_expect_tx(&sh.rawfull[rs], __popc(live) * kChunk * Z::raw_row);
                }
                __syncwarp();
                if (here) ptx::tma_load_3d(raw + rs * Z::raw + lane * kChunk * Z::raw_row, &pages, x, ps, pg, &sh.rawfull[rs]);
                __syncwarp();
                if (++rs == raw_stages) rs = 0, rp ^= 1;
            }
            if (!ok) break;
            if (lane == 0) ptx::mbar_arrive(&sh.copied);
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- products
        const uint32_t idesc_s = ptx::idesc_f16_f32(kM, kTile), idesc_o = ptx::idesc_f16_f32(kM, D) | ptx::kIdescMajorB;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t qd = ptx::sdesc_kmajor_sw128(ptx::smem_addr(smem));
        const uint64_t kd = ptx::sdesc_kmajor_sw128(ptx::smem_addr(ring));
        const uint64_t vd = ptx::sdesc_mnmajor_sw128(ptx::smem_addr(ring), Z::atom);
        uint32_t tiles = 0, turn = 0, step0 = 0, step1 = 0;
        for (int it = 0;; ++it) {
            if (!next_task(it, task) || task.n < 0) break;
            if (task.n == 0) continue;
            const bool shared = shares(task);
            const int s0 = steps_of(task, 0), s1 = steps_of(task, 1);
            int left = s0 + s1;                            // logits to issue
            auto logits = [&](int q, int j) {
                const uint32_t t = tiles + tile_of(task, q, j);
                const int stage = 2 * t & 3;
                if (!wait_bounded(&sh.opfull[stage], t >> 1 & 1, &sh.abort, a.err)) return false;
                ptx::tc_fence_after();
                --left;
                if (ptx::elect_one()) {
                    const uint64_t qo = qd + ((shared ? 0 : q * Z::operand) >> 4), ko = kd + (stage * Z::operand >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int off = (kk >> 2) * Z::atom + (kk & 3) * 32;
                        ptx::mma_f16_ss(tm + kTile * q, qo + (off >> 4), ko + (off >> 4), idesc_s, kk > 0);
                    }
                    ptx::mma_commit(&sh.sfull[q]);
                    if (shared || q == 1) ptx::mma_commit(&sh.opfree[stage]);
                    if (left == 0) ptx::mma_commit(&sh.qfree);
                }
                __syncwarp();
                return true;
            };
            auto output = [&](int q, int j) {
                const uint32_t t = tiles + tile_of(task, q, j);
                const int stage = (2 * t & 3) + 1;
                if (!wait_bounded(&sh.opfull[stage], t >> 1 & 1, &sh.abort, a.err) ||
                    !wait_bounded(&sh.pfull[q], (q ? step1 : step0) + j & 1, &sh.abort, a.err))
                    return false;
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
                    const uint64_t vo = vd + (stage * Z::operand >> 4);
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
#pragma unroll
                        for (int e = 0; e < (F16 ? 2 : 1); ++e)
                            ptx::mma_f16_ts(tm + kColO + D * q, tm + kTile * q + kHalfCols * (kk >> 2) + 8 * (kk & 3) + 32 * e,
                                            vo + (kk * 16 * 128 >> 4), idesc_o, j > 0 || kk > 0 || e > 0);
                    if (shared || q == 1) ptx::mma_commit(&sh.opfree[stage]);
                }
                __syncwarp();
                return true;
            };
            bool ok = wait_bounded(&sh.qfull, turn & 1, &sh.abort, a.err) && logits(0, 0);
            if (ok && s1 > 0) ok = logits(1, 0);
            // (the accumulators of the task before have been read)
            if (ok && turn > 0) ok = wait_bounded(&sh.oread, turn - 1 & 1, &sh.abort, a.err);
            // a stream's next logits follow its output, so that the other's products run beside its softmax
            for (int j = 0; ok && j < s0; ++j) {
                ok = output(0, j);
                if (ok && j + 1 < s0) ok = logits(0, j + 1);
                if (ok && j < s1) ok = output(1, j);
                if (ok && j + 1 < s1) ok = logits(1, j + 1);
            }
            if (!ok) break;
            if (ptx::elect_one()) ptx::mma_commit(&sh.odone);
            __syncwarp();
            tiles += task.n, step0 += s0, step1 += s1, ++turn;
        }
    } else {
        // ---------------------------------------------------------------- work.  Later rows of a sequence see more of it:
        // they start first.
        const uint32_t tasks = gridDim.x / (uint32_t)L.splits;
        uint32_t id = blockIdx.x / (uint32_t)L.splits, asked = 0;
        bool more = true, ok = true, checked = false;
        for (int it = 0; more; ++it) {
            Task k;
            k.n = k.blk.rows = 0;
            const uint32_t at = tasks - 1 - id, slot = at / (uint32_t)a.heads_kv;
            k.kvh = (int)(at - slot * a.heads_kv);
            if (!find_rows_warp(a, slot, L.blocks, L.rows, group, checked, k.blk)) {
                k.n = kBadSums;
                more = false;
            } else if (k.blk.rows > 0) {
                k.range = key_range(a, k.blk, group);
                const int all = (k.range.chunks + kTileChunks - 1) / kTileChunks;
                k.n = max(0, (all - rank + L.splits - 1) / L.splits);
            }
            if (k.n < 0 || k.blk.rows > 0) {
                set_heads(k);
                if (k.n > 0 && it > 0) {
                    // the queries on their way to L2
                    const int64_t first = k.tok0;
                    for (int i = lane; i < k.blk.rows; i += 32) {
                        const uint32_t tok = (k.rest + i) * recip >> 22;
                        const uint16_t* src = static_cast<const uint16_t*>(a.query) + (k.blk.row0 + first + tok) * a.q_stride +
                                              (k.kvh * group + (int)(k.rest + i - tok * group)) * D;
#pragma unroll
                        for (int x = 0; x < D; x += 64) ptx::prefetch_l2(src + x);
                    }
                }
                ok = wait_bounded(&sh.taskfree[it & 1], (it >> 1 & 1) ^ 1, &sh.abort, a.err, kTaskLimitNs);
                if (!ok) break;
                if (lane == 0) {
                    sh.task[it & 1] = k;
                    sh.held = 0;
                    ptx::mbar_arrive(&sh.taskfull[it & 1]);
                }
                __syncwarp();
            } else {
                --it;                                      // (a number that no block has)
                if (lane == 0) sh.held = 0;
            }
            if (!more) break;
            more = false;
            if (L.splits == 1) {
                // (not before the task's last copy, a few tiles ahead of its end: 472 blocks of 100 to 400 us 1099 us when
                // the next one is taken at once)
                if (it >= 0) ok = wait_bounded(&sh.copied, it & 1, &sh.abort, a.err, kTaskLimitNs);
                if (!ok) break;
                if (lane == 0) {
                    sh.asking = 1;
                    ptx::mbar_arrive_expect_tx(&sh.answer, 16);
                    ptx::take_pending_cta(&sh.taken, &sh.answer);
                }
                __syncwarp();
                ok = wait_bounded(&sh.answer, asked & 1, &sh.abort, a.err);
                if (!ok) break;
                ++asked;
                more = ptx::taken_cta(&sh.taken, id);
                if (lane == 0) sh.asking = 0, sh.held = more ? id + 1 : 0;
                ptx::fence_proxy_async_smem();             // (the next answer lands in the same place)
                __syncwarp();
            }
            if (!more) {
                const int end = it + 1;
                ok = wait_bounded(&sh.taskfree[end & 1], (end >> 1 & 1) ^ 1, &sh.abort, a.err, kTaskLimitNs);
                if (ok && lane == 0) {
                    sh.task[end & 1].n = kNoMore;
                    sh.task[end & 1].blk.rows = 0;
                    ptx::mbar_arrive(&sh.taskfull[end & 1]);
                }
                __syncwarp();
            }
        }
    }

    // ---- the end
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (sh.abort != 0) {
        if (warp == kMmaWarp) {                            // products and copies that are still under way end first
            const uint64_t t0 = ptx::globaltimer();
            while (ptx::globaltimer() - t0 < kWaitLimitNs) {
            }
        }
        __syncthreads();
        // NaN for the rows of every task that this CTA may have left
        auto fail_rows = [&](const Task& k) {
            for (int i = tid; i < k.blk.rows * (D / 8); i += kThreads)
                reinterpret_cast<uint4*>(dst + head_of(k, i / (D / 8)) * D)[i % (D / 8)] =
                    make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
            if (a.lse)
                for (int i = tid; i < k.blk.rows; i += kThreads) a.lse[head_of(k, i)] = __int_as_float(0x7FC00000);
        };
        if (rank == 0) {
            fail_rows(sh.task[0]);
            fail_rows(sh.task[1]);
            uint32_t held = sh.held, id;
            if (sh.asking && ptx::taken_cta(&sh.taken, id)) held = id + 1;
            if (held > 0) {
                const uint32_t at = gridDim.x / (uint32_t)L.splits - held, slot = at / (uint32_t)a.heads_kv;
                task.kvh = (int)(at - slot * a.heads_kv);
                bool checked = false;
                if (find_rows_warp(a, slot, L.blocks, L.rows, group, checked, task.blk)) {
                    set_heads(task);
                    fail_rows(task);
                }
            }
        }
    } else if (sh.task[0].n == kBadSums) {
        clear_rows(a, D, (int64_t)blockIdx.x * kThreads + tid, (int64_t)gridDim.x * kThreads);
    }
    if (L.splits > 1) {
        // join the cluster's partial results (of its only task)
        const bool failed = sh.abort != 0;
        const Task& k = sh.task[0];
        if (failed) {
            for (int i = tid; i < 2 * kM; i += kThreads) part_ml[i] = make_float2(0.0f, __int_as_float(0x7FC00000));
        }
        ptx::cluster_sync();
        const int pieces = (k.n >= 0 ? k.blk.rows : 0) * (D / 4);
        for (int z = rank * kThreads + tid; z < pieces; z += L.splits * kThreads) {
            const int i = z / (D / 4), d4 = z % (D / 4);
            float top = -FLT_MAX, sum = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float2 ml[kMaxSplits];
            float4 v[kMaxSplits];
#pragma unroll
            for (int x = 0; x < kMaxSplits; ++x) {
                ml[x] = make_float2(-FLT_MAX, 0.0f);
                v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (x < L.splits) {
                    ml[x] = ptx::ld_cluster2(ptx::cluster_addr(ptx::smem_addr(part_ml + i), x));
                    v[x] = ptx::ld_cluster4(ptx::cluster_addr(ptx::smem_addr(part_o + i * kStride + 4 * d4), x));
                }
                top = fmaxf(top, ml[x].x);
            }
#pragma unroll
            for (int x = 0; x < kMaxSplits; ++x) {
                const float g = ptx::ex2(ml[x].x - top);
                sum = fmaf(g, ml[x].y, sum);
                acc.x = fmaf(g, v[x].x, acc.x), acc.y = fmaf(g, v[x].y, acc.y);
                acc.z = fmaf(g, v[x].z, acc.z), acc.w = fmaf(g, v[x].w, acc.w);
            }
            const int64_t head = head_of(k, i);
            sum = sum_that_counts(top, sum);
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum, g = a.v_scale;
            *reinterpret_cast<uint2*>(dst + head * D + 4 * d4) =
                make_uint2(float2_to_act2<F16>(acc.x * inv * g, acc.y * inv * g), float2_to_act2<F16>(acc.z * inv * g, acc.w * inv * g));
            if (a.lse && d4 == 0) a.lse[head] = lse_of(top, sum);
        }
        __syncwarp();
        ptx::cluster_sync();                               // no CTA leaves while another reads its partial results
    }
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <bool F16, bool E2M1, int D>
cudaError_t launch_shape(const PagedArgs& a, int64_t most_rows, int sms, cudaStream_t st)
{
    using Z = Sizes<D>;
    static_assert(Z::smem <= 227 * 1024, "shared memory of an SM");
    const int group = a.heads_q / a.heads_kv;
    Layout L;
    L.block_recip = (uint32_t)((UINT64_C(1) << 32) / (uint32_t)a.p.block_size);
    L.rows = most_rows <= kM ? kM : 2 * kM;
    const int64_t slots = row_slots(a, L.rows, group, &L.blocks);
    const int64_t tiles = ceil_div64(most_positions(a, L.rows, group), kTile);
    // blocks that hold rows (TND: most of the numbers past these have none)
    const int64_t full = a.p.layout_tnd ? std::min<int64_t>(slots, a.p.batch * ceil_div64(most_rows, L.rows)) : slots;
    // CTAs that all run at once: clusters leave some SMs of each group of 18 to 20 out.  us for splits 2 / 4 / 8: 4 sequences of
    // 16k-32k positions (32 blocks and heads) 122 / 69 / -, 2 of 30000 and 9000 (16) 126 / 70 / 66, one of 16384 (16) - / 66 / 82
    L.splits = 1;
    auto room = [&](int splits) { return splits == 2 ? sms : splits == 4 ? sms * 27 / 32 : sms * 3 / 4; };
    while (L.splits < kMaxSplits && full * a.heads_kv * L.splits * 2 <= room(2 * L.splits) && tiles >= 4 * L.splits) L.splits *= 2;
    const int64_t grid = slots * a.heads_kv * L.splits;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    CUtensorMap pages;
    std::memset(&pages, 0, sizeof(pages));
    if (a.p.batch > 0 && !encode_page_map(&pages, a.kv, a.entry_bytes, a.p.block_size, a.page_bytes, a.p.num_blocks, Z::raw_row, kChunk))
        return cudaErrorUnknown;
    auto kernel = paged_chunk_kernel<F16, E2M1, D>;
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? UINT64_C(1) << dev : 0;
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::smem);
        if (e != cudaSuccess) return e;
        raised.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Z::smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = L.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = L.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, L, pages);
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedArgs& a, int head_dim, bool f16, bool e2m1, int64_t most_rows, int sms, cudaStream_t st)
{
    if (head_dim == 64) {
        if (f16) return e2m1 ? launch_shape<true, true, 64>(a, most_rows, sms, st) : launch_shape<true, false, 64>(a, most_rows, sms, st);
        return e2m1 ? launch_shape<false, true, 64>(a, most_rows, sms, st) : launch_shape<false, false, 64>(a, most_rows, sms, st);
    }
    if (f16) return e2m1 ? launch_shape<true, true, 128>(a, most_rows, sms, st) : launch_shape<true, false, 128>(a, most_rows, sms, st);
    return e2m1 ? launch_shape<false, true, 128>(a, most_rows, sms, st) : launch_shape<false, false, 128>(a, most_rows, sms, st);
}

}  // namespace qli
