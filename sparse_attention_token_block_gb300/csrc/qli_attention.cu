// qli_attention.cu -- attention of each query row over the KV-cache entries that its index list
// names, the entries held in 4 bits:
//     z_i = scale * q_h . K_i,   out_h = sum_i softmax(z)_i V_i,   lse_h = ln sum_i exp(z_i)
//
// A cluster of `splits` CTAs works on one row (or a slice of its KV heads), each on a slice of the
// list.  A CTA first resolves its slice -- index, bounds, block_table -- into rows of the pool.  Each
// of its eight warps then carries one unit, a KV head with up to 8 * NT of its query heads, over its
// share of the entries, 32 a step, and meets no other warp until the end: its head's bytes of those
// entries come into a ring of its own by TMA row gathers, four entries an instruction.  (In a probe
// from L2, 16-byte asynchronous copies of a head's 144 bytes stop at 7.8 TB/s, a shared-memory write
// per 32-byte sector; row gathers of them reach 14.5 TB/s.  A bulk copy per entry costs about 45 issue
// slots.)  Where the eight warps of a CTA carry eight KV heads side by side (kShared), the ring is the
// CTA's: every warp gathers four whole entries a step, one instruction instead of eight, and the warps
// hand the stages on through barriers.
//
//   * logits:  S^T (16 entries x 8 heads) = K Q^T.  A lane decodes 4-bit keys straight into the A
//     fragment: lane (r, c) of a warp holds rows r and r + 8, so it takes 1/4 of two key vectors as one
//     shared-memory load each; which of its columns meets which step of the product is free as long as
//     the query fragment, loaded once, follows the same order.
//   * softmax: running maximum and sum per head in fp32 (base 2).  The accumulators are rescaled only
//     when some logit exceeds the maximum in use by more than 8 (then p stays within 2^8, inside
//     fp16's range at full precision), so most tiles skip the exchange between lanes.
//   * output:  O^T (D x 8 heads) += V^T P^T.  P, rounded to fp16, goes from accumulator to B fragment by 8 x 8
//     transposes; with float16 activations what the rounding dropped follows as a product of its own.  (The
//     error of a float16 output is then its rounding's, 2.1e-4 of its size instead of 2.8e-4, and 32 rows of
//     2048 entries take 23.2 us instead of 21.6; of a bfloat16 output it is 1.619e-3 without, and 1.611e-3 in
//     fp32 throughout.)  V^T's A fragment pairs two entries per register: the nibbles of two entries are
//     interleaved before they are decoded.
//
// Heads never fill the M side of a product, entries do, so groups of 8 query heads waste nothing of
// the tensor cores.  4-bit values times e4m3 scales are exact in fp16 (E2M1: at most 6 significant bits, 2^-10
// to 2688; int4: 7, 2^-9 to 3136), and so are float16 queries; bfloat16 queries are scaled by a power of two of
// their head's largest magnitude, so that they fit fp16 (elements below 2^-17 of the largest are off by up to
// 2^-25 of it).
//
// What bounds it: from L2 (a prefill), the SM's arithmetic.  A step of 32 entries x 8 query heads is 535
// instructions, of which 128 conversions of code pairs, 128 scale products and 32 tensor products; a
// probe gives 2, 2 and 7.1 cycles for these per sub-partition, products and scale products on one pipe,
// so about 570 cycles, and a step takes about 900.  (Dropping the scale products of V alone takes 8 %
// off; giving the keys' to the integer pipe adds 6 %: both pipes are near full.)  From HBM (a decode),
// the gathers' latency and the start: list, entries, join.  Measured on a GB300, 64 query heads over 8 KV
// heads of 128, E2M1, 2048 entries a row: 1 row 7.1 us, 8 rows 11.0, 32 rows (8k-32k keys) 21.4 (3.6 TB/s),
// 64 rows 36.4 (4.2), 128 rows 65.1 (4.7); prefill of 1024 + 2048 + 4096 rows 1.76 ms (166 TFLOP/s; such calls
// go to qli_attention_rows.cu, 0.61 ms); int4 27.1 us at 32 rows: its codes take seven integer operations per
// eight, E2M1's four.
//
// Partial results of the warps and CTAs that share a unit meet in shared memory (distributed over
// the cluster) and are joined in a fixed order.  Every wait for a copy is bounded (0.2 s): on expiry the
// kernel records kErrTimeout, writes NaN, lets its copies land and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstring>

#include "qli_kv.cuh"

namespace qli {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxPerThread = kMaxSparse / kThreads;
constexpr int kMaxSplits = 8;                     // a portable cluster
constexpr int kMaxSmem = 220 * 1024;              // dynamic, of a CTA
constexpr uint64_t kWaitLimitNs = 200000000ull;
constexpr float kRescale = 8.0f;                  // logits (base 2) above the maximum in use

// How a launch is laid out (host)
struct Layout {
    int32_t chunks;        // units per KV head: ceil(group / (8 NT))
    int32_t units;         // heads_kv * chunks
    int32_t per_cta;       // units per CTA, at most kWarps
    int32_t ctas;          // CTAs a row's units take: ceil(units / per_cta)
    int32_t parts;         // warps that share a unit: kWarps / per_cta
    int32_t splits;        // CTAs of the cluster, each with a slice of the list
    int32_t per_split;     // list positions per slice
    uint32_t block_recip;  // floor(2^32 / block_size)
    int32_t page_rows;     // entries from one page to the next; 0: no whole number, no row gathers
    int32_t mask_off, ring_off;   // shared-memory offsets of the masks and the rings, behind the list
};

// One KV head's bytes of an entry, from a multiple of 16 on (heads of 72 bytes start on a multiple of
// 8), and their stride in a ring: 32 or 96 beyond a multiple of 128
constexpr int head_bytes(int d) { return d == 128 ? 144 : 80; }
constexpr int row_bytes(int d, bool shared)
{
    return shared ? kWarps * kv_unit_bytes(d) + 32 : (d == 128 ? 160 : 96);
}
constexpr int kStages = 2;                                          // steps in a ring

// Resident CTAs per SM, as the accumulators (D x 8 NT fp32 per warp) and the rings allow.  (D = 64 with
// three: int4 prefill of 1024 and 2048 rows 237 -> 212 us against two.)
constexpr int ctas_per_sm(int d, int nt) { return nt * d <= 64 ? 3 : (nt * d <= 128 ? 2 : 1); }

// The whole warp waits for the phase of a barrier; false (for every lane) when a wait gave up
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile uint32_t* abort, uint32_t* err)
{
    const uint64_t t0 = ptx::globaltimer();
    while (true) {
        const bool done = ptx::mbar_try_wait_sleep(bar, parity, 100000u);
        if (__all_sync(0xffffffffu, done)) return true;
        if (__any_sync(0xffffffffu, *abort != 0)) return false;
        if (__any_sync(0xffffffffu, ptx::globaltimer() - t0 > kWaitLimitNs)) {
            *abort = 1;
            if (err) atomicOr(err, kErrTimeout);
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile uint32_t* abort, uint32_t* err)
{
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    return wait_slow(bar, parity, abort, err);
}

// Entry (of a group of eight) that row r of an 8-row fragment holds.  Rows 2c and 2c + 1 hold entries
// c and 4 + (c + 2) % 4: with an entry stride of 32 or 96 modulo 128 bytes, the four entries that a
// quarter-warp reads of V and the two that it reads of K then lie in different banks.
__device__ __forceinline__ int entry_of_row(int r) { return (r & 1) ? 4 + (((r >> 1) + 2) & 3) : r >> 1; }

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N])
{
    static_assert(N == 1 || N == 2 || N == 4, "4, 8 or 16 bytes");
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

template <bool F16, bool E2M1, int D, int NT, bool kShared>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NT))
    attention_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ Layout L,
                     const __grid_constant__ CUtensorMap rows)
{
    constexpr int kUnit = kv_unit_bytes(D);
    constexpr int NW = D / 32;                    // words of key codes per lane and entry
    constexpr int MO = D / 16;                    // 16-row tiles of the output
    constexpr int kHeadStride = D + 4;            // of partial outputs, in floats
    constexpr int kRow = row_bytes(D, kShared), kStep = 32 * kRow;
    // of each warp's ring; kShared: [0] the ring's, [1] its stages handed back
    __shared__ uint64_t bars[kWarps][kStages];
    __shared__ uint32_t abort;
    extern __shared__ __align__(128) uint8_t smem[];
    int32_t* list = reinterpret_cast<int32_t*>(smem);
    uint32_t* masks = reinterpret_cast<uint32_t*>(smem + L.mask_off);
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = L.splits > 1 ? (int)ptx::cluster_rank() : 0;
    const uint32_t task = blockIdx.x / (uint32_t)L.splits, row = task / (uint32_t)L.ctas;
    const int u0 = (int)(task - row * L.ctas) * L.per_cta, nu = min(L.per_cta, L.units - u0);
    const int group = a.heads_q / a.heads_kv, active = nu * L.parts;       // warps with work
    if (tid == 0) abort = 0;
    if (lane == 0) {
        for (int x = 0; x < kStages; ++x) ptx::mbar_init(&bars[wid][x], kShared ? kWarps : (L.page_rows ? 1 : 32));
        ptx::fence_mbar_init();
    }
    if (tid == 0 && L.page_rows) ptx::prefetch_tensormap(&rows);
    const int unit = wid / L.parts, part = wid - unit * L.parts;
    const int kvh = (u0 + unit) / L.chunks;
    const int h0 = kvh * group + (u0 + unit - kvh * L.chunks) * 8 * NT;      // the unit's first query head
    const int nh = min(8 * NT, (kvh + 1) * group - h0);
    const int r = lane >> 2, c = lane & 3;
    ptx::pdl_wait();
    // the query heads' elements, under way while the list is resolved: head r of each block of eight,
    // this lane's quarter of D
    uint4 qraw[NT][NW];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            qraw[t][j] = make_uint4(0u, 0u, 0u, 0u);
            if (wid < active && 8 * t + r < nh)
                qraw[t][j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.query) + (int64_t)row * a.q_stride +
                                                             (int64_t)(h0 + 8 * t + r) * D + c * (D / 4) + 8 * j);
        }

    // ---- the slice's entries as rows of the pool, 32 positions of the list per warp at a time: the mask
    // of the valid ones, and in the others' places a valid one's row (what is copied from there is
    // masked), so that every byte a step reads is some listed entry's
    const int k0 = rank * L.per_split, n = max(0, min(L.per_split, a.p.sparse_count - k0));
    const int chunks = (n + 31) / 32;             // of the list
    {
        const int32_t* idx = a.idx + (int64_t)row * a.p.sparse_count + k0;
        int32_t j[kMaxPerThread], page[kMaxPerThread];
#pragma unroll
        for (int e = 0; e < kMaxPerThread; ++e) {
            const int at = 32 * (wid + kWarps * e) + lane;
            j[e] = at < n ? idx[at] : -1;
        }
        const int64_t b = row_batch(a.p, a.seq_lens_q, row);
        const int64_t limit = b >= 0 ? index_limit(a.p, a.seq_lens_k, b) : -1;
        const int32_t* table = a.block_table + b * a.p.max_blocks_per_seq;
        const uint32_t bs = (uint32_t)a.p.block_size;
        uint32_t bits = 0;
#pragma unroll
        for (int e = 0; e < kMaxPerThread; ++e) {
            const bool ok = j[e] >= 0 && j[e] < limit;
            if (j[e] != -1 && !ok) bits |= kErrLength;
            // j / block_size: the reciprocal rounded down gives the quotient or one less
            uint32_t blk = __umulhi((uint32_t)j[e], L.block_recip), pos = (uint32_t)j[e] - blk * bs;
            if (pos >= bs) ++blk, pos -= bs;
            page[e] = ok ? table[blk] : -1;
            j[e] = ok ? (int32_t)pos : -1;
        }
#pragma unroll
        for (int e = 0; e < kMaxPerThread; ++e) {
            const int st = wid + kWarps * e;
            if (st >= chunks) break;
            const bool ok = j[e] >= 0 && page[e] >= 0 && page[e] < a.p.num_blocks;
            if (j[e] >= 0 && !ok) bits |= kErrPage;
            const uint32_t mask = __ballot_sync(0xffffffffu, ok);
            // (without row gathers the row is page * block_size + position, taken apart again below)
            const int32_t at = page[e] * (L.page_rows ? L.page_rows : a.p.block_size) + j[e];
            const int32_t some = __shfl_sync(0xffffffffu, at, mask ? __ffs(mask) - 1 : 0);
            list[32 * st + lane] = ok ? at : some;
            if (lane == 0) masks[st] = mask;
        }
        bits = __reduce_or_sync(0xffffffffu, bits);
        if (bits && lane == 0 && a.err) atomicOr(a.err, bits);
    }
    __syncthreads();

    float o[NT][MO][4], m[NT][2], l[NT][2];
    if (wid < active) {
        // the chunks of 32 positions part, part + parts, ... are this warp's steps; a chunk without a valid
        // entry is not copied
        const int steps = (chunks - part + L.parts - 1) / L.parts, lo = (kShared ? u0 : kvh) * kUnit & ~15;
        uint8_t* ring = smem + L.ring_off + (kShared ? 0 : wid * kStages * kStep);
        uint64_t* bar = bars[kShared ? 0 : wid];
        auto copy_step = [&](int st, int stage) {
            const int ch = st * L.parts + part;
            const bool go = masks[ch] != 0;
            const bool stall = a.p.test_stall == 1;            // test switch: nothing arrives, the waits run out
            if constexpr (kShared) {
                if (ptx::elect_one()) {
                    ptx::mbar_arrive_expect_tx(&bar[stage], go ? 4 * kRow : 0);
                    const int4 y = *reinterpret_cast<const int4*>(list + 32 * ch + 4 * wid);
                    if (go && !stall) ptx::tma_gather4(ring + stage * kStep + 4 * wid * kRow, &rows, lo / 8, y.x, y.y, y.z, y.w, &bar[stage]);
                }
                __syncwarp();
            } else if (L.page_rows) {
                if (ptx::elect_one()) {
                    ptx::mbar_arrive_expect_tx(&bar[stage], go ? kStep : 0);
                    if (go && !stall) {
                        int4 y[8];                // all loads first: the gathers keep the compiler from moving them up
#pragma unroll
                        for (int g = 0; g < 8; ++g) y[g] = reinterpret_cast<const int4*>(list + 32 * ch)[g];
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            ptx::tma_gather4(ring + stage * kStep + 4 * g * kRow, &rows, lo / 8, y[g].x, y[g].y, y[g].z, y[g].w,
                                             &bar[stage]);
                    }
                }
                __syncwarp();
            } else if (!stall) {
                // a lane per entry, 16 bytes at a time
                if (go) {
                    const int slot = list[32 * ch + lane], pg = slot / a.p.block_size;
                    const uint8_t* src = a.kv + pg * a.page_bytes + (int64_t)(slot - pg * a.p.block_size) * a.entry_bytes + lo;
#pragma unroll
                    for (int x = 0; x < head_bytes(D); x += 16)
                        ptx::cp_async<16>(ring + stage * kStep + lane * kRow + x, src + x);
                }
                ptx::cp_async_arrive_noinc(&bar[stage]);
            }
        };
        if (steps > 0) copy_step(0, 0);
        // query fragments: float16 as they are, bfloat16 scaled by a power of two
        uint32_t q[NT][NW][4];
        float f[NT][2];                           // base-2 logit factor of heads 2c and 2c + 1
        const float factor = a.softmax_scale * a.k_scale * 1.4426950408889634f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            uint32_t w[NW][4];
#pragma unroll
            for (int j = 0; j < NW; ++j) w[j][0] = qraw[t][j].x, w[j][1] = qraw[t][j].y, w[j][2] = qraw[t][j].z, w[j][3] = qraw[t][j].w;
            if constexpr (F16) {
#pragma unroll
                for (int j = 0; j < NW; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)     // elements 2i, 2i + 1 or i, i + 4
                        q[t][j][i] = E2M1 ? w[j][i] : __byte_perm(w[j][i / 2], w[j][2 + i / 2], i & 1 ? 0x7632 : 0x5410);
                f[t][0] = f[t][1] = fminf(factor, 3.0e38f);
            } else {
                float big = 0.0f;
#pragma unroll
                for (int j = 0; j < NW; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 v = act2_to_float2<F16>(w[j][i]);
                        big = fmaxf(big, fmaxf(fabsf(v.x), fabsf(v.y)));
                    }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                const uint32_t ex = min(max(__float_as_uint(big) >> 23, 1u), 253u);
                const float down = __uint_as_float((254u - ex) << 23);          // 2^-(exponent of big)
#pragma unroll
                for (int j = 0; j < NW; ++j) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 v = act2_to_float2<F16>(w[j][i]);
                        x[2 * i] = v.x * down;
                        x[2 * i + 1] = v.y * down;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        q[t][j][i] = E2M1 ? float2_to_act2<true>(x[2 * i], x[2 * i + 1]) : float2_to_act2<true>(x[i], x[i + 4]);
                }
                const float up = __uint_as_float(ex << 23) * factor;
                f[t][0] = fminf(__shfl_sync(0xffffffffu, up, 8 * c), 3.0e38f);
                f[t][1] = fminf(__shfl_sync(0xffffffffu, up, 8 * c + 4), 3.0e38f);
            }
#pragma unroll
            for (int i = 0; i < MO; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][i][e] = 0.0f;
            m[t][0] = m[t][1] = -FLT_MAX;
            l[t][0] = l[t][1] = 0.0f;
        }
        for (int st = 1; st < min(kStages, steps); ++st) copy_step(st, st);
        const int tk = entry_of_row(r), ta = c, tb = 4 + ((c + 2) & 3);
        const uint8_t* head = ring + kvh * kUnit - lo;
        const uint8_t* kc0 = head + tk * kRow + (D / 8) * c;                       // the lane's key codes and scales,
        const uint8_t* ks0 = head + tk * kRow + D + (D == 128 ? 2 * c : c);
        const uint8_t* vc0 = head + ta * kRow + D / 2 + (D / 16) * r;              // value codes and scales
        const uint8_t* vs0 = head + ta * kRow + D + D / 16 + (D == 128 ? r : r >> 1);
        const int vb = (tb - ta) * kRow;
        int stage = 0, parity = 0;
#pragma unroll 1
        for (int st = 0; st < steps; ++st) {
            if (kShared && st > 0 && st - 1 + kStages < steps) {
                // the step before freed its stage (of the other parity when it was the last of a round)
                const int freed = stage == 0 ? kStages - 1 : stage - 1;
                if (!wait_bounded(&bars[1][freed], stage == 0 ? parity ^ 1 : parity, &abort, a.err)) break;
                copy_step(st - 1 + kStages, freed);
            }
            if (!wait_bounded(&bar[stage], parity, &abort, a.err)) break;
            const uint32_t mask = masks[st * L.parts + part];
            if (mask) {
            const uint8_t* kc = kc0 + stage * kStep;
            const uint8_t* ks = ks0 + stage * kStep;
            const uint8_t* va = vc0 + stage * kStep;
            const uint8_t* vs = vs0 + stage * kStep;
            // ---- logits of two tiles of 16 entries
            float s[2][NT][4];
            uint32_t w[2][2][NW];                  // tile, row r or r + 8: codes
            PairScale g[2][2][D / 64];             // and the scales of the lane's blocks
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    load_words<NW>(kc + (16 * u + 8 * y) * kRow, w[u][y]);
                    const uint8_t* x = ks + (16 * u + 8 * y) * kRow;
                    if constexpr (D == 128) {
                        const uint32_t h = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(x));
                        g[u][y][0] = pair_scale<E2M1>(__byte_perm(h, 0, 0x1010));
                        g[u][y][1] = pair_scale<E2M1>(__byte_perm(h, 0, 0x3232));
                    } else {
                        g[u][y][0] = pair_scale<E2M1>(__byte_perm(e4m3x2_to_f16x2(*x), 0, 0x1010));
                    }
                }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t) s[u][t][0] = s[u][t][1] = s[u][t][2] = s[u][t][3] = 0.0f;
#pragma unroll
            for (int j = 0; j < NW; ++j)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t x[4], y[4];
                    decode_pairs<E2M1>(w[u][0][j], g[u][0][j / 2], x);
                    decode_pairs<E2M1>(w[u][1][j], g[u][1][j / 2], y);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        ptx::mma_16816(s[u][t], x[0], y[0], x[1], y[1], q[t][j][0], q[t][j][1]);
                        ptx::mma_16816(s[u][t], x[2], y[2], x[3], y[3], q[t][j][2], q[t][j][3]);
                    }
                }
            // ---- softmax: masked entries get -infinity
            float z[2][NT][4], over = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[u][t][e] = fmaf(s[u][t][e], f[t][e & 1], -m[t][e & 1]);
            if (mask != 0xffffffffu) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(mask >> (16 * u + 8 * (e >> 1) + tk) & 1)) z[u][t][e] = -INFINITY;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    over = fmaxf(over, fmaxf(fmaxf(z[u][t][0], z[u][t][1]), fmaxf(z[u][t][2], z[u][t][3])));
            if (__any_sync(0xffffffffu, over > kRescale)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = m[t][e];
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int y = e; y < 4; y += 2)
                                if (z[u][t][y] > -INFINITY) top = fmaxf(top, s[u][t][y] * f[t][e]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        const float down = ptx::ex2(m[t][e] - top);
                        m[t][e] = top;
                        l[t][e] *= down;
#pragma unroll
                        for (int i = 0; i < MO; ++i) {
                            o[t][i][e] *= down;
                            o[t][i][e + 2] *= down;
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int y = e; y < 4; y += 2)
                                if (z[u][t][y] > -INFINITY) z[u][t][y] = fmaf(s[u][t][y], f[t][e], -top);
                    }
            }
            // each probability rounded to fp16 (the sum keeps the unrounded ones), and what that dropped
            constexpr int kParts = F16 ? 2 : 1;
            uint32_t pb[kParts][2][NT][2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[u][t][e] = ptx::ex2(z[u][t][e]);
                    l[t][0] += z[u][t][0] + z[u][t][2];
                    l[t][1] += z[u][t][1] + z[u][t][3];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t p = float2_to_act2<true>(z[u][t][2 * y], z[u][t][2 * y + 1]);
                        pb[0][u][t][y] = ptx::transpose_8x8(p);
                        if constexpr (F16) pb[1][u][t][y] = ptx::transpose_8x8(remainder_f16x2(z[u][t][2 * y], z[u][t][2 * y + 1], p));
                    }
                }
            // ---- output
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t* x0 = vs + 16 * u * kRow;
                const PairScale sab = pair_scale<E2M1>(e4m3x2_to_f16x2(x0[0] | (uint32_t)x0[vb] << 8));
                const PairScale scd = pair_scale<E2M1>(e4m3x2_to_f16x2(x0[8 * kRow] | (uint32_t)x0[vb + 8 * kRow] << 8));
                uint32_t wa[NW / 2], wb[NW / 2], wc[NW / 2], wd[NW / 2];
                load_words<NW / 2>(va + 16 * u * kRow, wa);
                load_words<NW / 2>(va + 16 * u * kRow + vb, wb);
                load_words<NW / 2>(va + (16 * u + 8) * kRow, wc);
                load_words<NW / 2>(va + (16 * u + 8) * kRow + vb, wd);
#pragma unroll
                for (int j = 0; j < NW / 2; ++j) {
                    uint32_t x[8], y[8];
                    decode_across<E2M1>(wa[j], wb[j], sab, x);
                    decode_across<E2M1>(wc[j], wd[j], scd, y);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < kParts; ++e)
                                ptx::mma_16816(o[t][4 * j + i], x[2 * i], x[2 * i + 1], y[2 * i], y[2 * i + 1], pb[e][u][t][0], pb[e][u][t][1]);
                }
            }
            }
            __syncwarp();                          // every lane is done with the stage
            if constexpr (kShared) {
                if (lane == 0) ptx::mbar_arrive(&bars[1][stage]);
            } else if (st + kStages < steps) {
                copy_step(st + kStages, stage);
            }
            if (++stage == kStages) {
                stage = 0;
                parity ^= 1;
            }
        }
        // the sums over the lanes that share a head's column
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 4);
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 8);
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 16);
            }
    }

    // ---- join and write.  Lane (r, c) holds elements r * D / 8 ... of heads 2c and 2c + 1 of each block.
    __syncthreads();                               // the rings are free
    const bool failed = abort != 0;
    if (failed) {                                  // copies that are still under way land before the CTA ends
        // (which phase a barrier is in is not known here: give the copies the time of a wait)
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < kWaitLimitNs) {
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t) l[t][0] = l[t][1] = __int_as_float(0x7FC00000);
    }
    uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)row * a.heads_q * D;
    if (L.parts * L.splits == 1) {
        if (wid >= active) return;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = 8 * t + 2 * c + e;
                if (h >= nh) continue;
                const float sum = l[t][e];
                const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
                uint32_t w[MO];
#pragma unroll
                for (int i = 0; i < MO; ++i) w[i] = float2_to_act2<F16>(o[t][i][e] * inv, o[t][i][e + 2] * inv);
                uint4* dst = reinterpret_cast<uint4*>(out + (int64_t)(h0 + h) * D + r * (D / 8));
#pragma unroll
                for (int i = 0; i < MO / 4; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                if (a.lse && r == 0)
                    a.lse[(int64_t)row * a.heads_q + h0 + h] = sum == 0.0f ? -INFINITY : (m[t][e] + log2f(sum)) * 0.6931471805599453f;
            }
        return;
    }
    // partial outputs [warp][8 NT heads][kHeadStride], (maximum, sum) [warp][8 NT heads], and the same
    // pairs of the CTA's units once its warps are joined
    float* part_o = reinterpret_cast<float*>(smem + L.ring_off);
    float2* part_ml = reinterpret_cast<float2*>(part_o + kWarps * 8 * NT * kHeadStride);
    float2* unit_ml = part_ml + kWarps * 8 * NT;
    if (wid < active) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = wid * 8 * NT + 8 * t + 2 * c + e;
                float4* dst = reinterpret_cast<float4*>(part_o + h * kHeadStride + r * (D / 8));
#pragma unroll
                for (int i = 0; i < MO / 2; ++i)
                    dst[i] = make_float4(o[t][2 * i][e], o[t][2 * i][e + 2], o[t][2 * i + 1][e], o[t][2 * i + 1][e + 2]);
                if (r == 0) (L.parts > 1 ? part_ml : unit_ml)[h] = make_float2(m[t][e], l[t][e]);
            }
    }
    const int pieces = nu * 8 * NT * (D / 4);      // 4 elements of a head
    auto finish = [&](int hh, int d4, const float4& v, float top, float sum) {
        const int un = hh / (8 * NT), h = hh - un * 8 * NT, kv = (u0 + un) / L.chunks;
        const int head = kv * group + (u0 + un - kv * L.chunks) * 8 * NT + h;
        if (head >= (kv + 1) * group) return;
        const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
        *reinterpret_cast<uint2*>(out + (int64_t)head * D + 4 * d4) =
            make_uint2(float2_to_act2<F16>(v.x * inv, v.y * inv), float2_to_act2<F16>(v.z * inv, v.w * inv));
        if (a.lse && d4 == 0)
            a.lse[(int64_t)row * a.heads_q + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    };
    if (L.parts > 1) {
        // the warps of each unit; the joined result replaces the first warp's
        __syncthreads();
        for (int i = tid; i < pieces; i += kThreads) {
            const int hh = i / (D / 4), d4 = i % (D / 4), un = hh / (8 * NT);
            const int at = hh + un * (L.parts - 1) * 8 * NT;       // of the unit's first warp
            float2 ml[kWarps];
            float4 v[kWarps];
            float top = -FLT_MAX, sum = 0.0f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                ml[x] = make_float2(-FLT_MAX, 0.0f);
                v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (x < L.parts) {
                    ml[x] = part_ml[at + x * 8 * NT];
                    v[x] = *reinterpret_cast<const float4*>(part_o + (at + x * 8 * NT) * kHeadStride + 4 * d4);
                }
                top = fmaxf(top, ml[x].x);
            }
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const float g = ptx::ex2(ml[x].x - top);
                sum = fmaf(g, ml[x].y, sum);
                acc.x = fmaf(g, v[x].x, acc.x), acc.y = fmaf(g, v[x].y, acc.y);
                acc.z = fmaf(g, v[x].z, acc.z), acc.w = fmaf(g, v[x].w, acc.w);
            }
            if (L.splits == 1) {
                finish(hh, d4, acc, top, sum);
            } else {
                *reinterpret_cast<float4*>(part_o + at * kHeadStride + 4 * d4) = acc;
                if (d4 == 0) unit_ml[at] = make_float2(top, sum);
            }
        }
        if (L.splits == 1) return;
        __syncwarp();
    }
    ptx::cluster_sync();
    for (int i = rank * kThreads + tid; i < pieces; i += L.splits * kThreads) {
        const int hh = i / (D / 4), d4 = i % (D / 4), un = hh / (8 * NT);
        const int at = hh + un * (L.parts - 1) * 8 * NT;
        const uint32_t from_ml = ptx::smem_addr(unit_ml + at), from_o = ptx::smem_addr(part_o + at * kHeadStride + 4 * d4);
        float2 ml[kMaxSplits];
        float4 v[kMaxSplits];
        float top = -FLT_MAX, sum = 0.0f;
#pragma unroll
        for (int x = 0; x < kMaxSplits; ++x) {
            ml[x] = make_float2(-FLT_MAX, 0.0f);
            v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (x < L.splits) {
                ml[x] = ptx::ld_cluster2(ptx::cluster_addr(from_ml, x));
                v[x] = ptx::ld_cluster4(ptx::cluster_addr(from_o, x));
            }
        }
#pragma unroll
        for (int x = 0; x < kMaxSplits; ++x) top = fmaxf(top, ml[x].x);
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int x = 0; x < kMaxSplits; ++x) {
            const float g = ptx::ex2(ml[x].x - top);
            sum = fmaf(g, ml[x].y, sum);
            acc.x = fmaf(g, v[x].x, acc.x), acc.y = fmaf(g, v[x].y, acc.y);
            acc.z = fmaf(g, v[x].z, acc.z), acc.w = fmaf(g, v[x].w, acc.w);
        }
        finish(hh, d4, acc, top, sum);
    }
    __syncwarp();
    ptx::cluster_sync();                           // no CTA leaves while another reads its partial results
}

template <bool F16, bool E2M1, int D, int NT, bool kShared>
cudaError_t launch_layout(const AttentionArgs& a, Layout L, cudaStream_t st)
{
    const int64_t rows = a.p.rows;
    const int steps = (L.per_split + 31) / 32;
    L.block_recip = (uint32_t)((UINT64_C(1) << 32) / (uint32_t)a.p.block_size);
    L.mask_off = 4 * 32 * steps;
    L.ring_off = (L.mask_off + 4 * steps + 127) & ~127;
    int ring = (kShared ? 1 : kWarps) * kStages * 32 * row_bytes(D, kShared);
    CUtensorMap rows_map;
    std::memset(&rows_map, 0, sizeof(rows_map));
    if (L.page_rows && !encode_row_map(&rows_map, a.kv, a.entry_bytes,
                                       (int64_t)L.page_rows * (a.p.num_blocks - 1) + a.p.block_size, row_bytes(D, kShared)))
        return cudaErrorUnknown;
    const int join = kWarps * 8 * NT * ((D + 4) + 2 + 2) * 4;        // partial outputs, (maximum, sum) twice
    if (L.parts * L.splits > 1 && ring < join) ring = join;
    const int smem = L.ring_off + ring;
    const int64_t grid = rows * L.ctas * L.splits;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    auto kernel = attention_kernel<F16, E2M1, D, NT, kShared>;
    // the kernel's shared-memory limit, raised once per device
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? UINT64_C(1) << dev : 0;
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        raised.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
    return cudaLaunchKernelEx(&cfg, kernel, a, L, rows_map);
}

template <bool F16, bool E2M1, int D, int NT>
cudaError_t launch_shape(const AttentionArgs& a, int sms, cudaStream_t st)
{
    const int group = a.heads_q / a.heads_kv;
    Layout L;
    L.chunks = (group + 8 * NT - 1) / (8 * NT);
    L.units = a.heads_kv * L.chunks;
    const int k = a.p.sparse_count;
    const int64_t rows = a.p.rows;
    // CTAs per row: as many slices of the units as still run in one wave (fewer units per CTA: more warps
    // share a unit, so each reads a shorter part of the list.  8 units, 2048 entries; 32 rows: 8 units
    // per CTA 73 us, 4 42, 2 24.1, 1 21.5; 64 rows: 73, 42.8, 36.4, 40.9; 128 rows: 75, 65.1, 69, 69.6).
    // The list itself is split over a cluster while each SM has at most one CTA and each warp keeps a
    // step of its own (1 row: 13.1 us unsplit, 7.1 with 8 splits; 8 rows: 13.8 unsplit, 11.0 with 2, 11.4
    // with 4, 17.1 with 8).
    const int slots = ctas_per_sm(D, NT) * sms;
    L.per_cta = 1;
    while (L.per_cta < kWarps && rows * ((L.units + L.per_cta - 1) / L.per_cta) > slots) L.per_cta *= 2;
    L.ctas = (L.units + L.per_cta - 1) / L.per_cta;
    L.per_cta = (L.units + L.ctas - 1) / L.ctas;
    L.parts = kWarps / L.per_cta;
    L.splits = 1;
    while (L.splits < kMaxSplits && rows * L.ctas * L.splits * 2 <= sms && k >= 32 * L.parts * L.splits * 2) L.splits *= 2;
    L.per_split = (k + L.splits - 1) / L.splits;
    // row gathers need one stride for all entries of the pool
    L.page_rows = 0;
    if (a.kv && a.page_bytes % a.entry_bytes == 0 && a.page_bytes / a.entry_bytes * a.p.num_blocks <= INT32_MAX)
        L.page_rows = (int32_t)(a.page_bytes / a.entry_bytes);
    if constexpr (NT == 1) {
        if (L.page_rows && L.chunks == 1 && L.per_cta == kWarps && L.units % kWarps == 0)
            return launch_layout<F16, E2M1, D, NT, true>(a, L, st);
    }
    return launch_layout<F16, E2M1, D, NT, false>(a, L, st);
}

template <bool F16, bool E2M1>
cudaError_t launch_type(const AttentionArgs& a, int head_dim, int sms, cudaStream_t st)
{
    // query heads per unit: as few blocks of eight as hold the group, within the registers (an
    // accumulator of D x 8 NT fp32 per warp)
    const int group = a.heads_q / a.heads_kv;
    if (head_dim == 64) {
        if (group <= 8) return launch_shape<F16, E2M1, 64, 1>(a, sms, st);
        if (group <= 16) return launch_shape<F16, E2M1, 64, 2>(a, sms, st);
        return launch_shape<F16, E2M1, 64, 4>(a, sms, st);
    }
    return group <= 8 ? launch_shape<F16, E2M1, 128, 1>(a, sms, st) : launch_shape<F16, E2M1, 128, 2>(a, sms, st);
}

}  // namespace

cudaError_t launch_attention(const AttentionArgs& a, int head_dim, bool f16, bool e2m1, int sms, cudaStream_t st)
{
    if (attention_in_rows(a, head_dim, sms)) return launch_attention_rows(a, f16, e2m1, sms, st);
    if (f16) return e2m1 ? launch_type<true, true>(a, head_dim, sms, st) : launch_type<true, false>(a, head_dim, sms, st);
    return e2m1 ? launch_type<false, true>(a, head_dim, sms, st) : launch_type<false, false>(a, head_dim, sms, st);
}

}  // namespace qli
