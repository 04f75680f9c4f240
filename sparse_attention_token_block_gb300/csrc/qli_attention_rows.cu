// qli_attention_rows.cu -- the sparse attention for blocks of neighbouring rows whose lists cover a large
// part of their keys (a prefill): the same operator as qli_attention.cu, on the tcgen05 tensor cores.
//
// A CTA takes R consecutive rows x G query heads of one KV head after another: R * G <= 128 rows of a
// product.  It turns the rows' lists into bit masks over the positions of their sequence, walks the
// tiles of 64 positions in which some row has an entry, and runs per tile
//
//     S = Q K^T  (128 x 64 x D)     P = 2^(S f - m), zero where the row's bit is not set     O += P V
//
// so that a key is decoded once for R rows instead of once per row that lists it.  Roles:
//   * one warp copies the KV head's bytes of a tile's entries by TMA, 16 positions (of one page) a box,
//     where any of the 16 is listed (the mask covers what else lies there, finite values);
//   * 2 + 2 converter warps decode them into fp16 operands in shared memory: K rows as they are, V
//     transposed (a lane takes eight entries x 16 elements and pairs the nibbles of two entries, as
//     qli_attention.cu does);
//   * one warp issues the products: Q, K and V from shared memory, the logits twice in tensor memory, P in
//     the place of the logits it came from;
//   * 4 softmax warps, a row of the product per thread: masked logits, running maximum (raised only when
//     a logit passes it by more than 2^8, then the row of O is rescaled), sum in fp32, P to fp16; with float16
//     activations what that rounding dropped follows P as a second operand, where the other half of the
//     logits was (1024 + 2048 rows of up to 1024 entries 212 us instead of 184; the errors as in
//     qli_attention.cu).
// Two CTAs share an SM (half its shared and tensor memory each): what a tile costs is mostly the way from
// role to role, and one CTA's masks, queries and outputs overlap the other's products.
//
// A position that a row lists n times counts n times: where the lists of a block hold duplicates (more
// entries than mask bits), the masks hold one binary digit of the counts a round, digit d's logits raised by
// d (2^d p), so that a round is needed for each digit that occurs, at most twelve.  (2432 rows of 2048 entries,
// 294 us: one row that names one position 2048 times 400 us, every row's second half position 0 651 us; a round
// for each repetition took 138 ms for the former.)  Further rounds also take the rows of a block that belong to
// another batch and the positions past the masks' width.
//
// A zero of P times a NaN would be a NaN, in rows that do not list the entry: an entry with a NaN among its
// scales (the cache write makes none) is taken as NaN keys, which the mask hides from the other rows, and
// finite values.
//
// What bounds it: latency, not a pipe.  A tile takes a CTA about 4000 cycles from role to role (two CTAs:
// 2000 an SM) of which its products take 512; the SM issues in 46 % of its cycles.  Without the arithmetic
// of softmax and decoding at all an earlier form (one CTA, tiles of 128) still took two thirds of its time.
// Building the masks is an eighth, staging the queries a twentieth.  Measured on a GB300, 64 query heads
// over 8 KV heads, E2M1, causal: 1024 + 2048 + 4096 rows of up to 2048 entries 612 us (one row at a time
// 1764), with 8192 more, which take two masks, 2311 us (4327); 1024 + 2048 rows of up to 1024 190 us (434), the
// same for one KV head 199 us (469), for groups of four 137 us (432), int4 204 us (577); one CTA an SM takes 816
// us for the first, the CTAs in the order of the rows 737, tiles whose logits are loaded in two parts 761.
//
// Every wait is bounded (0.2 s); on expiry the kernel records kErrTimeout, writes NaN and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cstring>

#include "qli_kv.cuh"

namespace qli {

namespace {

constexpr int kD = 128;
constexpr int kM = 128, kTile = 64;                    // rows and keys of a product
constexpr int kSoftWarps = 4, kKeyWarp = 4, kValueWarp = 6, kMmaWarp = 8, kCopyWarp = 9;
constexpr int kThreads = 320;
constexpr int kUnit = kv_unit_bytes(kD), kRaw = kTile * kUnit;             // a tile's entries of one KV head
// shared memory: operands (rows of 64 fp16 in the 128-byte swizzle, 128 bytes each), the copied entries, masks
constexpr int kAtomQ = kM * 128, kAtomK = kTile * 128, kAtomV = kD * 128;
constexpr int kSmemK = 2 * kAtomQ, kSmemV = kSmemK + 2 * kAtomK, kSmemRaw = kSmemV + 2 * kAtomV, kSmemMask = kSmemRaw + 2 * kRaw;
constexpr int kMaxRows = 32;                           // of a block
constexpr int kMaskBytes = 12 * 1024;
constexpr int kMaxWords = 128;                         // of a row's mask
constexpr uint32_t kColS = 0, kColO = 2 * kTile, kTmemCols = 256;
constexpr uint32_t kNone = 0xffffffffu;
constexpr float kRescale = 8.0f;
constexpr uint64_t kWaitLimitNs = 200000000ull;

struct RowsLayout {
    int32_t rows;          // rows of a block
    int32_t words;         // mask words per row (whole tiles)
    int32_t heads;         // KV heads per CTA
    int32_t slices;        // CTAs per block
    uint32_t block_recip;
};

struct Shared {
    uint64_t rawfull[2], rawfree[2], kfull, vfull[2], sfull[2], pfull[2], vfree[2], pvdone;
    uint32_t tmem, abort, tiles, entries, bits, next;
    uint32_t digits, row_digits[kMaxRows];             // binary digits that occur among a range's counts, and each row's
    int32_t batch[kMaxRows];
    float factor[kM];
    alignas(16) int32_t slot[2 * kMaxWords];           // slot of the pool of every 16th position, -1: none of the 16 is listed
    uint8_t list[kMaxWords / 2];                       // tiles with an entry
};

// The whole warp waits for the phase of a barrier; false (for every lane) when a wait gave up.  (Inline: a
// call would send what the roles hold in registers through local memory.)
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile uint32_t* abort, uint32_t* err)
{
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = ptx::globaltimer();
    while (!__all_sync(0xffffffffu, ptx::mbar_try_wait_sleep(bar, parity, 100000u))) {
        if (__any_sync(0xffffffffu, *abort != 0)) return false;
        if (__any_sync(0xffffffffu, ptx::globaltimer() - t0 > kWaitLimitNs)) {
            *abort = 1;
            if (err) atomicOr(err, kErrTimeout);
            return false;
        }
    }
    return true;
}

// Wait for this thread's loads from tensor memory; the registers pass through it, so that nothing that uses
// them moves in front
__device__ __forceinline__ void wait_loaded(uint32_t (&r)[32])
{
    ptx::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}

// Byte offset of 16-byte piece `piece` (eight fp16) of row r in an operand of swizzled blocks of `atom` bytes
__device__ __forceinline__ uint32_t operand_at(int r, int piece, int atom)
{
    return (piece >> 3) * atom + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
}

// Masks of digit `digit` of how often each of `rows` lists names each position from + [0, width), and the
// digits that occur at all (with digit 0).  The counts, 16 bits a position (a list has at most 2048), lie at
// `space`; after digit 0 only the rows that have the digit are counted.  (A call keeps the plain masks' code
// together: 2 % of a short prefill.)
__device__ __noinline__ void count_rows(const int32_t* idx, int k, uint32_t from, uint32_t width, int words, int rows, int digit,
                                        uint8_t* space, uint32_t* mask, uint32_t* row_digits, uint32_t* digits)
{
    const int tid = threadIdx.x, line = 32 * words;
    uint32_t* count = reinterpret_cast<uint32_t*>(space);
    for (int i = tid; i < rows * line / 8; i += kThreads) reinterpret_cast<uint4*>(count)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (digit == 0 && tid < rows) row_digits[tid] = 0;
    __syncthreads();
    for (int r = 0; r < rows; ++r, idx += k) {
        if (digit > 0 && !(row_digits[r] >> digit & 1)) continue;
        for (int e = tid; e < k; e += kThreads) {
            const uint32_t at = (uint32_t)idx[e] - from;
            if (idx[e] >= 0 && at < width) atomicAdd(count + ((r * line + at) >> 1), at & 1 ? 0x10000u : 1u);
        }
    }
    __syncthreads();
    for (int i = tid; i < rows * words; i += kThreads) {
        uint32_t word = 0, some = 0;
#pragma unroll 1
        for (int z = 0; z < 16; ++z) {
            const uint32_t c = count[16 * i + z];
            word |= ((c >> digit & 1u) | (c >> (16 + digit) & 1u) << 1) << (2 * z);
            some |= c;
        }
        mask[i] = word;
        some = (some | some >> 16) & 0xFFFFu;
        if (digit == 0 && some) {
            atomicOr(row_digits + i / words, some);
            atomicOr(digits, some);
        }
    }
}

template <bool F16, bool E2M1>
__global__ void __launch_bounds__(kThreads, 2)
    attention_rows_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ RowsLayout L,
                          const __grid_constant__ CUtensorMap pages)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* qs = smem;
    uint32_t* mask = reinterpret_cast<uint32_t*>(smem + kSmemMask);
    Shared& sh = *reinterpret_cast<Shared*>(smem + kSmemMask + kMaskBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = a.heads_q / a.heads_kv, k = a.p.sparse_count;
    // later rows of a sequence attend to more of it: they start first
    const uint32_t cta = gridDim.x - 1 - blockIdx.x;
    const int64_t block = cta / (uint32_t)L.slices;
    const int slice = (int)(cta - block * L.slices);
    const int64_t r0 = block * L.rows;
    const int nrows = (int)min((int64_t)L.rows, a.p.rows - r0);
    const int head0 = slice * L.heads, head1 = min(a.heads_kv, head0 + L.heads);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sh.rawfull[i], 1);
            ptx::mbar_init(&sh.rawfree[i], 4);
            ptx::mbar_init(&sh.vfull[i], 2);
            ptx::mbar_init(&sh.sfull[i], 1);
            ptx::mbar_init(&sh.pfull[i], kSoftWarps);
            ptx::mbar_init(&sh.vfree[i], 1);
        }
        ptx::mbar_init(&sh.kfull, 2);
        ptx::mbar_init(&sh.pvdone, 1);
        sh.abort = 0;
        ptx::fence_mbar_init();
    }
    ptx::pdl_wait();
    if (warp == kMmaWarp) {                            // (not before: kernels that still run may need it)
        ptx::tmem_alloc(&sh.tmem, kTmemCols);
        ptx::tmem_relinquish();
    }
    if (tid < L.rows) sh.batch[tid] = tid < nrows ? (int32_t)row_batch(a.p, a.seq_lens_q, r0 + tid) : -1;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sh.tmem;
    // rows of no batch: any index is an error
    for (int r = 0; r < nrows; ++r) {
        if (sh.batch[r] >= 0) continue;
        for (int e = tid; e < k; e += kThreads)
            if (a.idx[(r0 + r) * k + e] != -1 && a.err) atomicOr(a.err, kErrLength);
    }

    uint32_t done = 0;                                 // tiles walked so far: every role counts the same
    bool standing = false;                             // the masks are those of all rows and all their positions
    for (int kvh = head0; kvh < head1; ++kvh) {
        // ---- the head's queries as an operand: row m is query head m % group of row m / group, in fp16 (float16 as
        // it is, bfloat16 times a power of two of its largest magnitude)
        constexpr int kPerWarp = 16;
        if (warp < kM / kPerWarp) {
            // lane: 4 elements (for int4 2 x 2 of each eight: its codes come in the order 0 4 1 5 2 6 3 7)
            const int c8 = lane >> 1, half = lane & 1;
            uint2 raw[kPerWarp];
#pragma unroll
            for (int x = 0; x < kPerWarp; ++x) {
                const int m = kPerWarp * warp + x, r = m / group, h = kvh * group + m - r * group;
                raw[x] = make_uint2(0u, 0u);
                if (r >= nrows) continue;
                const uint16_t* src = static_cast<const uint16_t*>(a.query) + (r0 + r) * a.q_stride + (int64_t)h * kD + 8 * c8;
                if (E2M1) {
                    raw[x] = *reinterpret_cast<const uint2*>(src + 4 * half);
                } else {
                    raw[x] = make_uint2(*reinterpret_cast<const uint32_t*>(src + 2 * half),
                                        *reinterpret_cast<const uint32_t*>(src + 4 + 2 * half));
                }
            }
#pragma unroll
            for (int x = 0; x < kPerWarp; ++x) {
                const int m = kPerWarp * warp + x;
                if (!E2M1) raw[x] = make_uint2(__byte_perm(raw[x].x, raw[x].y, 0x5410), __byte_perm(raw[x].x, raw[x].y, 0x7632));
                uint32_t ex = 127;
                if constexpr (F16) {
                    *reinterpret_cast<uint2*>(qs + operand_at(m, c8, kAtomQ) + 8 * half) = raw[x];
                } else {
                    const float2 u = act2_to_float2<F16>(raw[x].x), v = act2_to_float2<F16>(raw[x].y);
                    float big = fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(v.x), fabsf(v.y)));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                    ex = min(max(__float_as_uint(big) >> 23, 1u), 253u);
                    const float down = __uint_as_float((254u - ex) << 23);              // 2^-(exponent of big)
                    *reinterpret_cast<uint2*>(qs + operand_at(m, c8, kAtomQ) + 8 * half) =
                        make_uint2(float2_to_act2<true>(u.x * down, u.y * down), float2_to_act2<true>(v.x * down, v.y * down));
                }
                // (above zero: the mask's -infinity times it stays -infinity)
                if (lane == 0)
                    sh.factor[m] = fminf(fmaxf(__uint_as_float(ex << 23) * (a.softmax_scale * a.k_scale * 1.4426950408889634f), 1.0e-30f),
                                         3.0e38f);
            }
        }
        ptx::fence_proxy_async_smem();
        float m_run = -FLT_MAX, l_run = 0.0f;          // softmax threads
        bool fresh = true;                             // no product has written O for this head yet
        int first = 0;                                 // rows of the round: [first, last)
        while (first < nrows && !sh.abort) {
            const int b = sh.batch[first];
            int last = first + 1;
            while (last < nrows && sh.batch[last] == b) ++last;
            const int64_t limit = b >= 0 ? index_limit(a.p, a.seq_lens_k, b) : 0;
            const int32_t* table = a.block_table + (int64_t)max(b, 0) * a.p.max_blocks_per_seq;
            int64_t from = 0;                          // first position of the masks
            bool counted = false;                      // the lists hold duplicates: the masks hold digits of counts
            const int words = L.words;
            // (a list of a batch without positions is still looked at: its indices are errors)
            for (int digit = 0; b >= 0;) {
                while (!standing) {
                    // ---- masks of this round
                    __syncthreads();                   // (every thread has read what the last round left)
                    if (tid == 0) sh.entries = sh.bits = 0, sh.next = counted ? sh.next : kNone;
                    __syncthreads();
                    uint32_t bits = 0, entries = 0, set = 0, next = kNone;     // next: first valid index past the masks
                    const uint32_t width = (uint32_t)max((int64_t)0, min((int64_t)(32 * words), limit - from));
                    constexpr int kMapBytes = kSmemMask - kSmemK;
                    const int line = 32 * words;
                    if (!counted) {
                        // a byte per position in the operands' space, then the bytes to bits (with an atomic OR
                        // per entry into the masks a prefill takes 628 us instead of 620)
                        constexpr int kAtOnce = 16;
                        uint8_t* map = smem + kSmemK;
                        const int fit = kMapBytes / line;
                        for (int ra = first; ra < last; ra += fit) {
                            const int rows = min(fit, last - ra);
                            if (ra > first) __syncthreads();
                            for (int i = tid; i < rows * line / 16; i += kThreads)
                                reinterpret_cast<uint4*>(map)[i] = make_uint4(0u, 0u, 0u, 0u);
                            __syncthreads();
                            for (int e = tid; e < k; e += kThreads) {
#pragma unroll 1
                                for (int rb = 0; rb < rows; rb += kAtOnce) {
                                    const int32_t* src = a.idx + (r0 + ra + rb) * k + e;
                                    int32_t j[kAtOnce];
#pragma unroll
                                    for (int r = 0; r < kAtOnce; ++r) j[r] = rb + r < rows ? src[r * k] : -1;
                                    uint8_t* m = map + rb * line;
#pragma unroll
                                    for (int r = 0; r < kAtOnce; ++r) {
                                        const uint32_t at = (uint32_t)j[r] - (uint32_t)from;
                                        if (j[r] >= 0 && at < width) {
                                            m[r * line + at] = 1;
                                            ++entries;
                                        } else if (j[r] != -1) {
                                            if (j[r] < 0 || j[r] >= limit) bits |= kErrLength;
                                            else if (j[r] >= from) next = min(next, (uint32_t)j[r]);
                                        }
                                    }
                                }
                            }
                            __syncthreads();
                            for (int i = tid; i < rows * words; i += kThreads) {
                                const uint4 x = reinterpret_cast<const uint4*>(map)[2 * i], y = reinterpret_cast<const uint4*>(map)[2 * i + 1];
                                const uint32_t b[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                                uint32_t word = 0;
#pragma unroll
                                for (int z = 0; z < 8; ++z) word |= (b[z] * 0x01020408u >> 24) << (4 * z);       // byte i of b to bit i
                                mask[ra * words + i] = word;
                            }
                        }
                        ptx::fence_proxy_async_smem();         // before copies land in the same place
                    } else {
                        for (int ra = first; ra < last; ra += kMapBytes / (2 * line)) {
                            if (ra > first) __syncthreads();
                            count_rows(a.idx + (r0 + ra) * k, k, (uint32_t)from, width, words, min(kMapBytes / (2 * line), last - ra), digit,
                                       smem + kSmemK, mask + ra * words, sh.row_digits + ra, &sh.digits);
                        }
                        ptx::fence_proxy_async_smem();
                    }
                    next = __reduce_min_sync(0xffffffffu, next);
                    if (lane == 0 && next != kNone) atomicMin(&sh.next, next);
                    entries = __reduce_add_sync(0xffffffffu, entries);
                    if (lane == 0 && entries) atomicAdd(&sh.entries, entries);
                    __syncthreads();
                    // what some row lists; positions on bad pages leave the masks (16 positions share a page)
                    for (int w = tid; w < words; w += kThreads) {
                        uint32_t o = 0;
                        for (int r = first; r < last; ++r) {
                            const uint32_t x = mask[r * words + w];
                            o |= x;
                            set += __popc(x);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            int slot = -1;
                            if (o >> (16 * h) & 0xFFFFu) {
                                const uint32_t at = (uint32_t)from + 32 * w + 16 * h, bs = (uint32_t)a.p.block_size;
                                uint32_t blk = __umulhi(at, L.block_recip);
                                if (at - blk * bs >= bs) ++blk;
                                const int page = table[blk];
                                if (page < 0 || page >= a.p.num_blocks) {
                                    bits |= kErrPage;
                                    for (int r = first; r < last; ++r) reinterpret_cast<uint16_t*>(mask)[2 * (r * words + w) + h] = 0;
                                } else {
                                    slot = page * a.p.block_size + (int)(at - blk * bs);
                                }
                            }
                            sh.slot[2 * w + h] = slot;
                        }
                    }
                    set = __reduce_add_sync(0xffffffffu, set);
                    if (lane == 0 && set) atomicAdd(&sh.bits, set);
                    if (bits && a.err) atomicOr(a.err, bits);
                    __syncthreads();
                    if (!counted && sh.entries != sh.bits) {           // more entries than bits: again, with counts
                        counted = true;
                        if (tid == 0) sh.digits = 0;
                        continue;
                    }
                    if (warp == 0) {
                        int n = 0;
                        for (int t0 = 0; t0 < words / 2; t0 += 32) {
                            const int t = t0 + lane;
                            bool some = false;
                            if (t < words / 2) {
                                const int4 x = *reinterpret_cast<const int4*>(sh.slot + 4 * t);
                                some = (x.x & x.y & x.z & x.w) >= 0;
                            }
                            const uint32_t live = __ballot_sync(0xffffffffu, some);
                            if (some) sh.list[n + __popc(live & ((1u << lane) - 1))] = (uint8_t)t;
                            n += __popc(live);
                        }
                        if (lane == 0) sh.tiles = n;
                    }
                    break;
                }
                __syncthreads();
                const int n = (int)sh.tiles;
                if (warp < kSoftWarps) {
                    // ------------------------------------------------------------ softmax
                    const int r = tid / group;
                    const uint32_t lanes = tmem + ((uint32_t)warp << 21);
                    const float f = sh.factor[tid];
                    const bool mine = r >= first && r < last;
                    const uint32_t* row_mask = mask + (mine ? r : 0) * words;
                    // logits raised by the digit: the maximum lowered by it for the round
                    m_run -= (float)digit;
                    for (int i = 0; i < n; ++i) {
                        const uint32_t t = done + i, buf = t & 1, cols = lanes + kColS + kTile * buf;
                        uint2 w = *reinterpret_cast<const uint2*>(row_mask + 2 * sh.list[i]);
                        if (!mine) w = make_uint2(0u, 0u);
                        if (!wait_bounded(&sh.sfull[buf], (t >> 1) & 1, &sh.abort, a.err)) break;
                        ptx::tc_fence_after();
                        bool ok = true;
                        uint32_t p[32], rest[F16 ? 32 : 1];
                        while (true) {
                            float best[2] = {-INFINITY, -INFINITY};
                            uint64_t part[2] = {0, 0};
                            const uint64_t F = ptx::pack2(f, f), M = ptx::pack2(-m_run, -m_run);
                            uint32_t s[2][32];
                            QLI_TMEM_LD_X32(cols, s[0]);
                            QLI_TMEM_LD_X32(cols + 32, s[1]);
                            wait_loaded(s[0]);
                            wait_loaded(s[1]);
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const uint32_t bits = q ? w.y : w.x;
                                if (!__all_sync(0xffffffffu, bits == 0xffffffffu)) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        s[q][e] = __float_as_uint(bits & (1u << e) ? __uint_as_float(s[q][e]) : -INFINITY);
                                }
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float x = __uint_as_float(s[q][e]), y = __uint_as_float(s[q][e + 1]);
                                    best[e >> 1 & 1] = fmaxf(best[e >> 1 & 1], fmaxf(x, y));
                                    float zx, zy;
                                    ptx::unpack2(ptx::fma2(ptx::pack2(x, y), F, M), zx, zy);
                                    const float px = ptx::ex2(zx), py = ptx::ex2(zy);
                                    part[e >> 1 & 1] = ptx::add2(part[e >> 1 & 1], ptx::pack2(px, py));
                                    const int at = 16 * q + e / 2;
                                    p[at] = float2_to_act2<true>(px, py);
                                    if constexpr (F16) rest[at] = remainder_f16x2(px, py, p[at]);
                                }
                            }
                            float sum, other;
                            ptx::unpack2(ptx::add2(part[0], part[1]), sum, other);
                            sum += other;
                            const float top = fmaxf(best[0], best[1]);
                            const float up = top * f;
                            const bool over = fmaf(top, f, -m_run) > kRescale && up > m_run;
                            if (!__any_sync(0xffffffffu, over)) {
                                l_run += sum;
                                break;
                            }
                            // raise the maximum of the rows that need it, rescale their sums and accumulators
                            const float g = over ? ptx::ex2(m_run - up) : 1.0f;
                            if (over) m_run = up;
                            l_run *= g;
                            if (fresh && i == 0) continue;
                            ok = wait_bounded(&sh.pvdone, (t - 1) & 1, &sh.abort, a.err);
                            if (!ok) break;
                            ptx::tc_fence_after();
#pragma unroll 1
                            for (int q = 0; q < 4; ++q) {
                                uint32_t o[32];
                                QLI_TMEM_LD_X32(lanes + kColO + 32 * q, o);
                                wait_loaded(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * g);
                                QLI_TMEM_ST_X32(lanes + kColO + 32 * q, o);
                            }
                        }
                        if (!ok) break;
                        // in the place of the logits (in parts of 16 columns where the registers of p and rest are
                        // those that the logits leave)
                        if constexpr (F16) {
                            QLI_TMEM_ST_X16(cols, p);
                            QLI_TMEM_ST_X16(cols + 16, (p + 16));
                            QLI_TMEM_ST_X16(cols + 32, rest);
                            QLI_TMEM_ST_X16(cols + 48, (rest + 16));
                        } else {
                            QLI_TMEM_ST_X32(cols, p);
                        }
                        ptx::tmem_wait_st();
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&sh.pfull[buf]);
                    }
                    m_run += (float)digit;
                } else if (warp < kValueWarp) {
                    // ------------------------------------------------------------ converters of the keys
                    // a lane takes a quarter of four positions, eight neighbouring lanes eight positions: their
                    // loads (144 bytes apart) and stores (swizzled rows) meet all banks once
                    const int row = 32 * (warp - kKeyWarp) + (lane & 7), quarter = lane >> 3;
                    const bool stall = a.p.test_stall == 1;        // test switch: no tile is handed on, the waits run out
                    const uint32_t off0 = kSmemK + operand_at(row, 4 * quarter, kAtomK);
                    for (int i = 0; i < n; ++i) {
                        const uint32_t t = done + i, buf = t & 1;
                        const uint8_t* src = smem + kSmemRaw + buf * kRaw + row * kUnit;
                        if (!wait_bounded(&sh.rawfull[buf], (t >> 1) & 1, &sh.abort, a.err)) break;
                        // the operand is free once the logits of the tile before are there
                        if (t > 0 && !wait_bounded(&sh.sfull[buf ^ 1], ((t - 1) >> 1) & 1, &sh.abort, a.err)) break;
#pragma unroll
                        for (int x = 0; x < 4; ++x, src += 8 * kUnit) {
                            const uint4 code = reinterpret_cast<const uint4*>(src)[quarter];
                            uint32_t scale = reinterpret_cast<const uint16_t*>(src + kD)[quarter];
                            const uint32_t vscale = reinterpret_cast<const uint16_t*>(src + kD + kD / 16)[quarter];
                            // a NaN (0x7F or 0xFF) among two of the values' scales
                            if (__vcmpeq4(vscale & 0x7F7Fu, 0x00007F7Fu) & 0xFFFFu) scale = 0x7F7Fu;
                            const uint32_t h = e4m3x2_to_f16x2(scale), w[4] = {code.x, code.y, code.z, code.w};
                            const PairScale g[2] = {pair_scale<E2M1>(__byte_perm(h, 0, 0x1010)), pair_scale<E2M1>(__byte_perm(h, 0, 0x3232))};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t o[4];
                                decode_pairs<E2M1>(w[e], g[e >> 1], o);
                                *reinterpret_cast<uint4*>(smem + ((off0 ^ (e << 4)) + 8 * 128 * x)) =
                                    make_uint4(o[0], o[1], o[2], o[3]);
                            }
                        }
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && !stall) {
                            ptx::mbar_arrive(&sh.kfull);
                            ptx::mbar_arrive(&sh.rawfree[buf]);
                        }
                    }
                } else if (warp < kMmaWarp) {
                    // ------------------------------------------------------------ converters of the values
                    // a lane takes one block of 16 elements of eight positions, in odd blocks the elements in the
                    // order 4 5 6 7 0 1 2 3, so that the stores of eight neighbouring lanes meet all banks once
                    const int vg = (lane & 3) + 4 * (warp - kValueWarp), vb = lane >> 2;
                    const bool stall = a.p.test_stall == 1;
                    const uint32_t turn = vb & 1 ? 0x1032 : 0x3210;
                    // operand_at of its first element; of element e: 128 e further, and the column with e flipped
                    const uint32_t off0 = operand_at(16 * vb + 4 * (vb & 1), vg, kAtomV);
                    for (int i = 0; i < n; ++i) {
                        const uint32_t t = done + i, buf = t & 1;
                        const uint8_t* src = smem + kSmemRaw + buf * kRaw + 8 * vg * kUnit + kD / 2;
                        if (!wait_bounded(&sh.rawfull[buf], (t >> 1) & 1, &sh.abort, a.err)) break;
                        uint32_t w[2][8], scale[8];
                        PairScale g[4];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint2 code = reinterpret_cast<const uint2*>(src + e * kUnit)[vb];
                            w[0][e] = __byte_perm(code.x, 0, turn);
                            w[1][e] = __byte_perm(code.y, 0, turn);
                            scale[e] = src[e * kUnit + kD / 2 + kD / 16 + vb];
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t h = e4m3x2_to_f16x2(scale[2 * e] | scale[2 * e + 1] << 8);
                            asm("max.f16x2 %0, %0, %1;" : "+r"(h) : "r"(0xDF00DF00u));        // -448: NaN to a number
                            g[e] = pair_scale<E2M1>(h);
                        }
                        if (t >= 2 && !wait_bounded(&sh.vfree[buf], ((t >> 1) - 1) & 1, &sh.abort, a.err)) break;
                        uint8_t* dst = smem + kSmemV + buf * kAtomV;
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            uint32_t o[4][8];
#pragma unroll
                            for (int e = 0; e < 4; ++e) decode_across<E2M1>(w[y][2 * e], w[y][2 * e + 1], g[e], o[e]);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4*>(dst + (off0 ^ (e << 7 | e << 4)) + 8 * 128 * y) =
                                    make_uint4(o[0][e], o[1][e], o[2][e], o[3][e]);
                        }
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && !stall) {
                            ptx::mbar_arrive(&sh.vfull[buf]);
                            ptx::mbar_arrive(&sh.rawfree[buf]);
                        }
                    }
                } else if (warp == kCopyWarp) {
                    // ------------------------------------------------------------ copies, 16 positions each
                    for (int i = 0; i < n; ++i) {
                        const uint32_t t = done + i, buf = t & 1;
                        const int32_t slot = lane < 4 ? sh.slot[4 * sh.list[i] + lane] : -1;
                        const uint32_t live = __popc(__ballot_sync(0xffffffffu, slot >= 0));
                        if (t >= 2 && !wait_bounded(&sh.rawfree[buf], ((t >> 1) - 1) & 1, &sh.abort, a.err)) break;
                        if (lane == 0) ptx::mbar_arrive_expect_tx(&sh.rawfull[buf], live * 16 * kUnit);
                        __syncwarp();
                        if (slot >= 0) {
                            uint32_t page = __umulhi((uint32_t)slot, L.block_recip), pos = (uint32_t)slot - page * a.p.block_size;
                            if (pos >= (uint32_t)a.p.block_size) ++page, pos -= a.p.block_size;
                            ptx::tma_load_3d(smem + kSmemRaw + buf * kRaw + lane * 16 * kUnit, &pages, kvh * (kUnit / 8), (int)pos, (int)page,
                                             &sh.rawfull[buf]);
                        }
                        __syncwarp();
                    }
                } else {
                    // ------------------------------------------------------------ products
                    const uint32_t idesc_s = ptx::idesc_f16_f32(kM, kTile), idesc_o = ptx::idesc_f16_f32(kM, kD);
                    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
                    const uint64_t qd = ptx::sdesc_kmajor_sw128(ptx::smem_addr(qs));
                    const uint64_t kd = ptx::sdesc_kmajor_sw128(ptx::smem_addr(smem + kSmemK));
                    bool ok = true;
                    for (int i = 0; i <= n; ++i) {
                        if (i < n) {
                            // logits of tile i; P of the tile before last lies where they go
                            const uint32_t t = done + i, buf = t & 1;
                            ok = wait_bounded(&sh.kfull, t & 1, &sh.abort, a.err) &&
                                 (i < 2 || wait_bounded(&sh.pvdone, t & 1, &sh.abort, a.err));
                            if (!ok) break;
                            ptx::tc_fence_after();
                            if (ptx::elect_one()) {
#pragma unroll
                                for (int kk = 0; kk < kD / 16; ++kk) {
                                    ptx::mma_f16_ss(tm + kColS + kTile * buf, qd + (((kk >> 2) * kAtomQ + (kk & 3) * 32) >> 4),
                                                    kd + (((kk >> 2) * kAtomK + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
                                }
                                ptx::mma_commit(&sh.sfull[buf]);
                            }
                            __syncwarp();
                        }
                        if (i > 0) {
                            // output of tile i - 1
                            const uint32_t t = done + i - 1, buf = t & 1;
                            ok = wait_bounded(&sh.vfull[buf], (t >> 1) & 1, &sh.abort, a.err) &&
                                 wait_bounded(&sh.pfull[buf], (t >> 1) & 1, &sh.abort, a.err);
                            if (!ok) break;
                            ptx::tc_fence_after();
                            const uint64_t vd = ptx::sdesc_kmajor_sw128(ptx::smem_addr(smem + kSmemV + buf * kAtomV));
                            const bool add = !(fresh && i == 1);
                            if (ptx::elect_one()) {
#pragma unroll
                                for (int kk = 0; kk < (F16 ? 2 : 1) * kTile / 16; ++kk)
                                    ptx::mma_f16_ts(tm + kColO, tm + kColS + kTile * buf + 8 * kk, vd + (kk % 4 * 32 >> 4), idesc_o, add || kk > 0);
                                ptx::mma_commit(&sh.vfree[buf]);
                                ptx::mma_commit(&sh.pvdone);
                            }
                            __syncwarp();
                        }
                    }
                    // every product is done before anything of this round is touched again
                    if (ok && n > 0) wait_bounded(&sh.pvdone, (done + n - 1) & 1, &sh.abort, a.err);
                }
                done += n;
                if (n > 0) fresh = false;
                ptx::tc_fence_before();
                __syncthreads();
                ptx::tc_fence_after();
                if (sh.abort) break;
                standing = !counted && from == 0 && first == 0 && last == nrows && sh.next == kNone;
                if (counted && sh.digits >> (digit + 1) != 0) {
                    digit += __ffs(sh.digits >> (digit + 1));
                    continue;
                }
                if (sh.next == kNone) break;
                from = sh.next & ~(uint32_t)(kTile - 1);
                digit = 0;
                counted = false;
            }
            first = last;
        }
        // ---- output of this head
        const bool failed = sh.abort != 0;
        if (warp < kSoftWarps) {
            const int r = tid / group, h = kvh * group + tid - r * group;
            const float sum = failed ? __int_as_float(0x7FC00000) : l_run;
            const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
            const bool live = r < nrows;
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + ((r0 + (live ? r : 0)) * a.heads_q + h) * kD);
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t o[32];
                if (fresh) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0;
                } else {
                    QLI_TMEM_LD_X32(tmem + ((uint32_t)warp << 21) + kColO + 32 * q, o);
                    wait_loaded(o);
                }
                if (live) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t w[4];
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            w[z] = sum == 0.0f ? 0u : float2_to_act2<F16>(__uint_as_float(o[8 * e + 2 * z]) * inv,
                                                                         __uint_as_float(o[8 * e + 2 * z + 1]) * inv);
                        dst[4 * q + e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();                          // the loads above take the whole warp
            }
            if (live && a.lse)
                a.lse[(r0 + r) * a.heads_q + h] = sum == 0.0f ? -INFINITY : (m_run + log2f(sum)) * 0.6931471805599453f;
        }
        ptx::tc_fence_before();
        __syncthreads();
        ptx::tc_fence_after();
    }
    if (warp == kMmaWarp) {
        if (sh.abort) {                                // products that are still under way end before the memory goes
            const uint64_t t0 = ptx::globaltimer();
            while (ptx::globaltimer() - t0 < kWaitLimitNs) {
            }
        }
        ptx::tmem_dealloc(tmem, kTmemCols);
    }
}

template <bool F16, bool E2M1>
cudaError_t launch_rows(const AttentionArgs& a, const RowsLayout& L, int64_t grid, cudaStream_t st)
{
    auto kernel = attention_rows_kernel<F16, E2M1>;
    constexpr int kSmem = kSmemMask + kMaskBytes + (int)sizeof(Shared);
    static_assert(kSmem <= 113 * 1024, "shared memory of half an SM");
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? UINT64_C(1) << dev : 0;
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        raised.fetch_or(bit, std::memory_order_relaxed);
    }
    CUtensorMap pages;
    std::memset(&pages, 0, sizeof(pages));
    if (a.p.num_blocks > 0 && !encode_page_map(&pages, a.kv, a.entry_bytes, a.p.block_size, a.page_bytes, a.p.num_blocks, kUnit, 16))
        return cudaErrorUnknown;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), kSmem, st, a, L, pages);
}

}  // namespace

namespace {

// Positions that a row's list may name: the longest sequence, or what the block_table holds
int64_t positions(const AttentionArgs& a)
{
    const int64_t held = (int64_t)a.p.max_blocks_per_seq * a.p.block_size;
    return a.seq_lens_k ? std::min(held, ((int64_t)a.p.max_seqlen_k + a.p.cmp_ratio - 1) / a.p.cmp_ratio) : held;
}

}  // namespace

// A tile costs the same whatever the rows list of it, so the lists have to be a large part of the positions:
// 4096 positions, lists of 1024: 435 us against 681 one row at a time; of 500: 415 against 382.  A CTA has
// 10-20 us of latency around its tiles, so they have to be several (lists of 256, 1024 rows: 57 and 57 us; of
// 512: 60 and 92; 32 sequences of 64 rows and positions: 77 and 47), the blocks have to fill the GPU (256 rows:
// 18.5 and 16.2; 305 rows: 22.2 and 26.8) and mostly hold one sequence's rows (64 sequences of 17 rows: 56 and
// 25; 8 of 64 rows with 2048 positions: 68 and 114).
bool attention_in_rows(const AttentionArgs& a, int head_dim, int sms)
{
    const int group = a.heads_q / a.heads_kv;
    if (head_dim != kD || group > kM || !a.kv) return false;
    const int64_t rows = a.p.rows, per = std::min(kMaxRows, kM / group), blocks = (rows + per - 1) / per;
    return rows >= 4 * per * a.p.batch && blocks * a.heads_kv >= sms && a.p.sparse_count >= 512 &&
           positions(a) <= 4 * (int64_t)a.p.sparse_count;
}

namespace {

RowsLayout rows_layout(const AttentionArgs& a, int sms)
{
    const int group = a.heads_q / a.heads_kv;
    RowsLayout L;
    L.rows = std::min(kMaxRows, kM / group);
    const int64_t words = std::max<int64_t>(1, (positions(a) + kTile - 1) / kTile) * 2;
    const int space = kMaskBytes / 4 / L.rows;
    L.words = (int32_t)std::min<int64_t>(words, std::min(kMaxWords, space) & ~1);
    L.block_recip = (uint32_t)((UINT64_C(1) << 32) / (uint32_t)a.p.block_size);
    const int64_t blocks = ((int64_t)a.p.rows + L.rows - 1) / L.rows;
    // KV heads per CTA: more share a list's mask, fewer balance better; four waves (prefill of 7168 rows, eight
    // heads: two 694 us, four 620, eight 624; of 1024 + 2048 rows: 222, 194, 215)
    L.slices = 1;
    while (L.slices < a.heads_kv && blocks * L.slices < 4 * (int64_t)sms) L.slices *= 2;
    L.heads = (a.heads_kv + L.slices - 1) / L.slices;
    L.slices = (a.heads_kv + L.heads - 1) / L.heads;
    return L;
}

}  // namespace

RowsShape attention_rows_shape(const AttentionArgs& a, int sms)
{
    const RowsLayout L = rows_layout(a, sms);
    return {L.rows, L.heads, 32 * L.words};
}

cudaError_t launch_attention_rows(const AttentionArgs& a, bool f16, bool e2m1, int sms, cudaStream_t st)
{
    const RowsLayout L = rows_layout(a, sms);
    const int64_t grid = ((int64_t)a.p.rows + L.rows - 1) / L.rows * L.slices;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    if (f16) return e2m1 ? launch_rows<true, true>(a, L, grid, st) : launch_rows<true, false>(a, L, grid, st);
    return e2m1 ? launch_rows<false, true>(a, L, grid, st) : launch_rows<false, false>(a, L, grid, st);
}

}  // namespace qli
