// qli_paged_attention.cu -- attention of each sequence's new tokens over the cached positions that they see: all
// of them up to the row's own (causal), or a sliding window of them and the first few (sinks); the entries are
// held in 4 bits:
//     z_j = scale * q_h . K_j,   out_h = sum_j softmax(z)_j V_j,   lse_h = ln sum_j exp(z_j)
//
// A unit is a KV head with up to 8 * NT of the (token, query head) rows that read it; a warp carries it over its
// share of the positions, 32 a step:
//   * logits:  S^T (16 positions x 8 rows) = K Q^T, keys decoded from shared memory straight into the fragment;
//   * softmax: running maximum and sum per row in fp32 (base 2); the accumulators are rescaled only when a logit
//     exceeds the maximum in use by more than 15;
//   * output:  O^T (D x 8 rows) += V^T P^T, P rounded to fp16 (values of codes times scales are exact in fp16), for float16
//     outputs with a second product of what that rounding dropped (decode 162 -> 177 us, over int4 206 -> 231).
// The units of `per_cta` KV heads of the same rows share a CTA, and a copy warp brings their bytes of 16 positions
// of a page by one TMA box; warps that are left over (`parts`) and the CTAs of a cluster (`splits`) share the
// steps in turn, and their partial results are joined in shared memory in a fixed order.
//
// Bound by the cache's bytes: 32 sequences of 8k-32k positions, 64 / 8 heads of 128, 732 MB in 164 us, 4.5 TB/s (0.66 of a copy); the
// steady state reads 6.9 TB/s.  The rest is what a CTA does once (its rows 1 us, the first bytes 3 us, the join 1 to 5 us) and
// sequences of uneven length: clusters of CTAs on a sequence even these out and pay the join.  Entries are decoded in registers, each
// key once for its 8 or 16 rows: with the entries on the M side no part of a product is padding, and 8 rows cost what one does.
// Windows of 4096 of the same batch 37 us (4.1 TB/s: 256 CTAs, two on some SMs, where instructions count: shorter tests for NaN and
// masks gave 5 %).  96 tokens' rows over 128 / 512 / 1024 positions of an int4 cache, float16, 10 / 16 / 25 us: 2.1 us a step of a warp;
// one row of 256, one step a warp, 6 us.  Measured and not kept: the pages' numbers and queries loaded before the lengths are known
// (no gain), copies by lanes on their own (slower).
//
// Positions that a step holds beyond what a row sees are masked, and so are those on pages outside the pool (of
// which nothing is copied).  What lies there is arbitrary: scales of NaN among the values are taken as numbers
// and their positions' keys as NaN instead, which the mask hides from the rows that do not see them.
//
// Every wait is bounded (0.2 s): on expiry the kernel records kErrTimeout, writes NaN, lets its copies land and
// returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cstring>

#include "qli_paged.cuh"

namespace qli {

namespace {

constexpr int kWarps = 8;                         // with a unit each, and one that copies
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStep = 2 * kChunk;                 // positions
constexpr int kMaxSplits = 16;                    // the largest cluster
constexpr int kMaxStages = 6;
constexpr int kHalfSmem = 112 * 1024;             // dynamic, of one of two CTAs on an SM
constexpr int kMostSmem = 220 * 1024;
constexpr uint64_t kWaitLimitNs = 200000000ull;
// Probabilities enter the products in fp16, where a row's largest stands between 2^11 and 2^15: the maximum in use is raised to 11
// below the largest logit (base 2) when one lies more than 15 above it.  So fp16's normal range (2^-14) reaches 2^-25 of the largest
// at least, and 2^-36 of it is what becomes 0: however many positions lie 27 bits down, they count.  (Raised to the largest logit
// itself 2^-25 became 0: 50000 positions below one whose value is 0 were lost.)
constexpr float kRescale = 15.0f, kBelow = 11.0f, kUnit11 = 1.0f / 2048.0f;

// How a launch is laid out (host)
struct Layout {
    int32_t blocks;        // BSND: row blocks per sequence
    int32_t per_cta;       // KV heads of a CTA
    int32_t slices;        // CTAs a block's heads take
    int32_t parts;         // warps that share a unit: kWarps / per_cta
    int32_t splits;        // CTAs of a cluster
    int32_t stages;        // of a ring
    int32_t row_bytes;     // from one position to the next in a ring
    uint32_t block_recip;
};

constexpr int ctas_per_sm(int d, int nt) { return nt * d <= 128 ? 2 : 1; }

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

// ln of a row's sum of exponentials, held as `sum` of 2^(z - m)
__device__ __forceinline__ float lse_of(float m, float sum)
{
    return sum == 0.0f ? -INFINITY : (m + kBelow + log2f(sum * kUnit11)) * 0.6931471805599453f;
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N])
{
    static_assert(N == 1 || N == 2 || N == 4, "4, 8 or 16 bytes");
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

template <bool F16, bool E2M1, int D, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NT))
    paged_attention_kernel(const __grid_constant__ PagedArgs a, const __grid_constant__ Layout L,
                           const __grid_constant__ CUtensorMap pages)
{
    constexpr int kUnit = kv_unit_bytes(D);
    constexpr int M = 8 * NT;                     // rows of a unit
    constexpr int NW = D / 32;                    // words of key codes per lane and position
    constexpr int MO = D / 16;                    // 16-row tiles of the output
    constexpr int kHeadStride = D + 4;            // of partial outputs, in floats
    __shared__ uint64_t full[kWarps][kMaxStages], freed[kWarps][kMaxStages];
    __shared__ uint32_t live[kWarps][kMaxStages];         // which 16 of a step's positions lie in the pool
    __shared__ uint32_t abort;
    __shared__ RowBlock blk;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = L.splits > 1 ? (int)ptx::cluster_rank() : 0;
    const int group = a.heads_q / a.heads_kv;
    if (tid == 0) abort = 0;
    if (tid < kWarps) {
        for (int x = 0; x < L.stages; ++x) {
            ptx::mbar_init(&full[tid][x], 1);
            ptx::mbar_init(&freed[tid][x], L.per_cta);
        }
        ptx::fence_mbar_init();
    }
    ptx::pdl_wait();
    const uint32_t task = blockIdx.x / (uint32_t)L.splits, slot = task / (uint32_t)L.slices;
    const int u0 = (int)(task - slot * L.slices) * L.per_cta, nu = min(L.per_cta, a.heads_kv - u0);
    if (!find_rows(a, slot, L.blocks, M, group, &blk)) {
        // prefix sums that are not: every row is zero
        clear_rows(a, D, (int64_t)blockIdx.x * kThreads + tid, (int64_t)gridDim.x * kThreads);
        return;
    }
    if (blk.rows == 0) return;                    // (the whole cluster)
    const KeyRange range = key_range(a, blk, group);
    // the steps of this CTA and part: numbers part + parts * (rank + splits * i)
    const int lanes_of = L.parts * L.splits, all_steps = (range.chunks + 1) / 2;
    auto steps_of = [&](int part) { return max(0, (all_steps - (rank * L.parts + part) + lanes_of - 1) / lanes_of); };

    const int unit = wid / L.parts, part = wid - unit * L.parts;
    const int r = lane >> 2, c = lane & 3;
    const bool works = wid < kWarps && unit < nu;
    float o[NT][MO][4], m[NT][2], l[NT][2];
    if (wid == kWarps) {
        // ---------------------------------------------------------------- copies: a lane per part and chunk of its steps
        const int p = min(lane >> 1, L.parts - 1), x = lane & 1, n = lane < 2 * L.parts ? steps_of(p) : 0, lo = u0 * kUnit & ~15;
        const bool stall = a.p.test_stall == 1;                // test switches: nothing arrives, the waits run out
        const bool late = a.p.test_stall == 3;                 // second lanes' own tests of a stage fail
        const int32_t* table = a.block_table + (int64_t)blk.batch * a.p.max_blocks_per_seq;
        const uint32_t bytes = kChunk * L.row_bytes;
        uint8_t* const ring = smem + p * L.stages * 2 * bytes + x * bytes;
        // pages, and positions in them, of the next step's chunk and of the one after it
        int page[2], at[2];
        auto resolve = [&](int i, int& pg, int& ps) {
            pg = INT32_MIN;
            if (i < n) pg = chunk_page(a, range, table, L.block_recip, 2 * ((i * L.splits + rank) * L.parts + p) + x, &ps);
        };
        resolve(0, page[0], at[0]);
        resolve(1, page[1], at[1]);
        int i = 0, stage = 0;
        uint32_t parity = 1;
        uint64_t since = ptx::globaltimer();
        while (__any_sync(0xffffffffu, i < n)) {
            // those parts whose next stage is free go on: the first lane of the pair that copies for a part tells (two tests of
            // a barrier that is about to change may differ, and a lane that went on alone would arm it for half the bytes)
            bool ready = i < n && !(late && x) && ptx::mbar_test_wait(&freed[p][stage], parity);
            ready = __shfl_sync(0xffffffffu, ready, lane & ~1);
            if (!__any_sync(0xffffffffu, ready)) {
                if (__any_sync(0xffffffffu, *(volatile uint32_t*)&abort != 0)) break;
                if (__any_sync(0xffffffffu, ptx::globaltimer() - since > kWaitLimitNs)) {
                    abort = 1;
                    if (a.err) atomicOr(a.err, kErrTimeout);
                    break;
                }
                __nanosleep(50);
                continue;
            }
            const bool here = ready && page[0] >= 0 && page[0] < a.p.num_blocks;
            if (ready && !here && page[0] != INT32_MIN && a.err) atomicOr(a.err, kErrPage);
            const uint32_t mask = __ballot_sync(0xffffffffu, here) >> (lane & ~1) & 3;
            if (ready && x == 0) {
                live[p][stage] = mask;
                ptx::mbar_arrive_expect_tx(&full[p][stage], stall ? bytes : __popc(mask) * bytes);
            }
            __syncwarp();
            if (here && !stall) ptx::tma_load_3d(ring + 2 * stage * bytes, &pages, lo / 8, at[0], page[0], &full[p][stage]);
            if (ready) {
                if (++stage == L.stages) stage = 0, parity ^= 1;
                ++i;
                page[0] = page[1], at[0] = at[1];
                resolve(i + 1, page[1], at[1]);
            }
            since = ptx::globaltimer();
        }
        __syncwarp();
    } else if (works) {
        const int kvh = u0 + unit;
        // query fragments: row r of each block of eight, this lane's quarter of D; float16 as they are, bfloat16
        // in fp16, scaled by a power of two of the row's largest magnitude
        uint32_t q[NT][NW][4];
        float f[NT][2];                           // base-2 logit factor of rows 2c and 2c + 1
        int hi[NT][2];                            // positions that they see
        const float factor = a.softmax_scale * a.k_scale * 1.4426950408889634f;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int i = blk.first + 8 * t + r, tok = i / group;
            uint4 raw[NW];
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                raw[j] = make_uint4(0u, 0u, 0u, 0u);
                if (8 * t + r < blk.rows)
                    raw[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.query) + (blk.row0 + tok) * a.q_stride +
                                                             (int64_t)(kvh * group + i - tok * group) * D + c * (D / 4) + 8 * j);
            }
            uint32_t w[NW][4];
#pragma unroll
            for (int j = 0; j < NW; ++j) w[j][0] = raw[j].x, w[j][1] = raw[j].y, w[j][2] = raw[j].z, w[j][3] = raw[j].w;
            if constexpr (F16) {
#pragma unroll
                for (int j = 0; j < NW; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)     // elements 2e, 2e + 1 or e, e + 4
                        q[t][j][e] = E2M1 ? w[j][e] : __byte_perm(w[j][e / 2], w[j][2 + e / 2], e & 1 ? 0x7632 : 0x5410);
                f[t][0] = f[t][1] = fminf(factor, 3.0e38f);
            } else {
                float big = 0.0f;
#pragma unroll
                for (int j = 0; j < NW; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 v = act2_to_float2<F16>(w[j][e]);
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
                    for (int e = 0; e < 4; ++e) {
                        const float2 v = act2_to_float2<F16>(w[j][e]);
                        x[2 * e] = v.x * down;
                        x[2 * e + 1] = v.y * down;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        q[t][j][e] = E2M1 ? float2_to_act2<true>(x[2 * e], x[2 * e + 1]) : float2_to_act2<true>(x[e], x[e + 4]);
                }
                const float up = __uint_as_float(ex << 23) * factor;
                f[t][0] = fminf(__shfl_sync(0xffffffffu, up, 8 * c), 3.0e38f);
                f[t][1] = fminf(__shfl_sync(0xffffffffu, up, 8 * c + 4), 3.0e38f);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) hi[t][e] = seen_end(a, blk, (blk.first + 8 * t + 2 * c + e) / group);
#pragma unroll
            for (int i2 = 0; i2 < MO; ++i2)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][i2][e] = 0.0f;
            m[t][0] = m[t][1] = -FLT_MAX;
            l[t][0] = l[t][1] = 0.0f;
        }
        const int steps = steps_of(part), step_bytes = kStep * L.row_bytes, row = L.row_bytes;
        // rows r of a fragment are positions r of each eight, columns 2c and 2c + 1 of the values' too
        const uint8_t* head = smem + part * L.stages * step_bytes + kvh * kUnit - (u0 * kUnit & ~15);
        const uint8_t* kc0 = head + r * row + (D / 8) * c;                         // the lane's key codes and scales,
        const uint8_t* ks0 = head + r * row + D + (D == 128 ? 2 * c : c);
        const uint8_t* vc0 = head + 2 * c * row + D / 2 + (D / 16) * r;               // value codes and scales
        const uint8_t* vs0 = head + 2 * c * row + D + D / 16 + (D == 128 ? r : r >> 1);
        // steps that every row sees whole (of those behind the sinks')
        const int whole_from = range.sink_chunks + (max(0, range.high - range.base) + kChunk - 1) / kChunk;
        const int whole_to = range.sink_chunks + max(0, range.low - range.base) / kChunk - 1;
        int stage = 0, parity = 0;
#pragma unroll 1
        for (int st = 0; st < steps; ++st) {
            const int ch = 2 * ((st * L.splits + rank) * L.parts + part);
            if (!wait_bounded(&full[part][stage], parity, &abort, a.err)) break;
            const uint32_t mask = live[part][stage];
            const uint8_t* kc = kc0 + stage * step_bytes;
            const uint8_t* ks = ks0 + stage * step_bytes;
            const uint8_t* va = vc0 + stage * step_bytes;
            const uint8_t* vs = vs0 + stage * step_bytes;
            // ---- logits of two tiles of 16 positions
            float s[2][NT][4];
            uint32_t w[2][2][NW];                  // tile, row r or r + 8: codes
            PairScale g[2][2][D / 64];             // and the scales of the lane's blocks
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    load_words<NW>(kc + (16 * u + 8 * y) * row, w[u][y]);
                    const uint8_t* x = ks + (16 * u + 8 * y) * row;
                    // a NaN (0x7F or 0xFF) among the values' scales becomes one of the keys'
                    if constexpr (D == 128) {
                        uint32_t b = *reinterpret_cast<const uint16_t*>(x);
                        const uint32_t v = *reinterpret_cast<const uint16_t*>(x + D / 16);
                        if ((v & 0x7F7Fu) + 0x0101u & 0x8080u) b = 0x7F7Fu;
                        const uint32_t h = e4m3x2_to_f16x2(b);
                        g[u][y][0] = pair_scale<E2M1>(__byte_perm(h, 0, 0x1010));
                        g[u][y][1] = pair_scale<E2M1>(__byte_perm(h, 0, 0x3232));
                    } else {
                        uint32_t b = *x;
                        if ((x[D / 16] & 0x7F) == 0x7F) b = 0x7F;
                        g[u][y][0] = pair_scale<E2M1>(__byte_perm(e4m3x2_to_f16x2(b), 0, 0x1010));
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
            // ---- softmax: masked positions get -infinity
            float z[2][NT][4], over = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[u][t][e] = fmaf(s[u][t][e], f[t][e & 1], -m[t][e & 1]);
            if (mask != 3u || ch < whole_from || ch >= whole_to) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int pos = range.position(ch + u), limit = mask >> u & 1 ? range.limit(ch + u) : 0;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = pos + 8 * (e >> 1) + r;
                            if (j >= limit || !sees(a, hi[t][e & 1], j)) z[u][t][e] = -INFINITY;
                        }
                }
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
                        float top = -FLT_MAX;
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int y = e; y < 4; y += 2)
                                if (z[u][t][y] > -INFINITY) top = fmaxf(top, s[u][t][y] * f[t][e]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        // (rounded up: logits that fp32 holds in steps of 16 have their largest at 2^0, not at 2^16)
                        top = fmaxf(m[t][e], __fadd_ru(top, -kBelow));
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
            // each probability rounded to fp16 (the sum keeps the unrounded ones), for float16 outputs, which would show it, with
            // what that dropped
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
                const uint8_t* x0 = vs + 16 * u * row;
                const PairScale sab = pair_scale<E2M1>(finite_f16x2(e4m3x2_to_f16x2(x0[0] | (uint32_t)x0[row] << 8)));
                const PairScale scd = pair_scale<E2M1>(finite_f16x2(e4m3x2_to_f16x2(x0[8 * row] | (uint32_t)x0[9 * row] << 8)));
                uint32_t wa[NW / 2], wb[NW / 2], wc[NW / 2], wd[NW / 2];
                load_words<NW / 2>(va + 16 * u * row, wa);
                load_words<NW / 2>(va + (16 * u + 1) * row, wb);
                load_words<NW / 2>(va + (16 * u + 8) * row, wc);
                load_words<NW / 2>(va + (16 * u + 9) * row, wd);
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
            __syncwarp();                          // every lane is done with the stage
            if (lane == 0) ptx::mbar_arrive(&freed[part][stage]);
            if (++stage == L.stages) stage = 0, parity ^= 1;
        }
        // the sums over the lanes that share a row's column
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 4);
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 8);
                l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], 16);
            }
    } else {
        // a warp without a unit hands its stages straight back (the barriers count per_cta warps)
        const int steps = unit < L.per_cta ? steps_of(part) : 0;
        int stage = 0, parity = 0;
        for (int st = 0; st < steps; ++st) {
            if (!wait_bounded(&full[part][stage], parity, &abort, a.err)) break;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&freed[part][stage]);
            if (++stage == L.stages) stage = 0, parity ^= 1;
        }
    }

    // ---- join and write.  Lane (r, c) holds elements r * D / 8 ... of rows 2c and 2c + 1 of each block.
    __syncthreads();                               // the rings are free
    const bool failed = abort != 0;
    if (failed) {                                  // copies that are still under way land before the CTA ends
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < kWaitLimitNs) {
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t) l[t][0] = l[t][1] = __int_as_float(0x7FC00000);
    }
    uint16_t* out = static_cast<uint16_t*>(a.out);
    // element 0 of row `i` of unit `un` in the output, in heads of D
    auto out_head = [&](int un, int i) {
        const int at = blk.first + i, tok = at / group;
        return (blk.row0 + tok) * a.heads_q + (u0 + un) * group + at - tok * group;
    };
    if (L.parts * L.splits == 1) {
        if (!works) return;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 8 * t + 2 * c + e;
                if (i >= blk.rows) continue;
                const float sum = sum_that_counts(m[t][e], l[t][e]);
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                uint32_t w[MO];
#pragma unroll
                for (int x = 0; x < MO; ++x) w[x] = float2_to_act2<F16>(o[t][x][e] * inv * a.v_scale, o[t][x][e + 2] * inv * a.v_scale);
                const int64_t at = out_head(unit, i);
                uint4* dst = reinterpret_cast<uint4*>(out + at * D + r * (D / 8));
#pragma unroll
                for (int x = 0; x < MO / 4; ++x) dst[x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
                if (a.lse && r == 0) a.lse[at] = lse_of(m[t][e], sum);
            }
        return;
    }
    // partial outputs [warp][M rows][kHeadStride], (maximum, sum) [warp][M rows], and the same pairs of the CTA's
    // units once its warps are joined
    float* part_o = reinterpret_cast<float*>(smem);
    float2* part_ml = reinterpret_cast<float2*>(part_o + kWarps * M * kHeadStride);
    float2* unit_ml = part_ml + kWarps * M;
    if (works) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = wid * M + 8 * t + 2 * c + e;
                float4* dst = reinterpret_cast<float4*>(part_o + h * kHeadStride + r * (D / 8));
#pragma unroll
                for (int i = 0; i < MO / 2; ++i)
                    dst[i] = make_float4(o[t][2 * i][e], o[t][2 * i][e + 2], o[t][2 * i + 1][e], o[t][2 * i + 1][e + 2]);
                if (r == 0) (L.parts > 1 ? part_ml : unit_ml)[h] = make_float2(m[t][e], l[t][e]);
            }
    }
    const int pieces = nu * M * (D / 4);           // 4 elements of a row
    auto finish = [&](int hh, int d4, const float4& v, float top, float sum) {
        const int un = hh / M, i = hh - un * M;
        if (i >= blk.rows) return;
        sum = sum_that_counts(top, sum);
        const int64_t at = out_head(un, i);
        // (two steps: a factor near the smallest number over the sum would not be one that fp32 holds)
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum, g = a.v_scale;
        *reinterpret_cast<uint2*>(out + at * D + 4 * d4) =
            make_uint2(float2_to_act2<F16>(v.x * inv * g, v.y * inv * g), float2_to_act2<F16>(v.z * inv * g, v.w * inv * g));
        if (a.lse && d4 == 0) a.lse[at] = lse_of(top, sum);
    };
    if (L.parts > 1) {
        // the warps of each unit; the joined result replaces the first warp's
        __syncthreads();
        for (int i = tid; i < pieces; i += kThreads) {
            const int hh = i / (D / 4), d4 = i % (D / 4), un = hh / M;
            const int at = hh + un * (L.parts - 1) * M;            // of the unit's first warp
            float2 ml[kWarps];
            float4 v[kWarps];
            float top = -FLT_MAX, sum = 0.0f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                ml[x] = make_float2(-FLT_MAX, 0.0f);
                v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (x < L.parts) {
                    ml[x] = part_ml[at + x * M];
                    v[x] = *reinterpret_cast<const float4*>(part_o + (at + x * M) * kHeadStride + 4 * d4);
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
        const int hh = i / (D / 4), d4 = i % (D / 4), un = hh / M;
        const int at = hh + un * (L.parts - 1) * M;
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

// Row stride in a ring of `heads` KV heads' bytes, with room for a start that is no multiple of 16: an odd multiple of 16,
// so that the four positions that a half-warp reads of V lie in different banks (of K two share them; strides for both
// would take a quarter of the ring)
int ring_row(int heads, int unit)
{
    return ((heads * unit + 15 & ~15) + (heads * unit % 16 ? 16 : 0)) | 16;
}

template <bool F16, bool E2M1, int D, int NT>
cudaError_t launch_shape(const PagedArgs& a, int sms, cudaStream_t st)
{
    constexpr int M = 8 * NT;
    const int group = a.heads_q / a.heads_kv;
    Layout L;
    L.block_recip = (uint32_t)((UINT64_C(1) << 32) / (uint32_t)a.p.block_size);
    const int64_t slots = row_slots(a, M, group, &L.blocks);
    const int64_t steps = ceil_div64(most_positions(a, M, group), kStep);         // of a row block
    // row blocks that hold rows (TND: most of the numbers past these have none)
    const int64_t full = a.p.layout_tnd ? std::min<int64_t>(slots, a.p.batch * ceil_div64(most_rows(a), M) + 1) : slots;
    const int room = ctas_per_sm(D, NT) * sms;
    L.per_cta = 1;
    while (L.per_cta < kWarps && full * ceil_div64(a.heads_kv, L.per_cta) > room) L.per_cta *= 2;
    L.per_cta = std::min<int>(L.per_cta, a.heads_kv);
    L.slices = (int)ceil_div64(a.heads_kv, L.per_cta);
    L.per_cta = (int)ceil_div64(a.heads_kv, L.slices);
    L.parts = kWarps / L.per_cta;
    // a cluster shares the steps while its CTAs fit the GPU together, and further (so that sequences of different lengths
    // balance) while a warp keeps 16 steps.  us, 64 / 8 heads, splits 1 / 2 / 4 / 8: 32 sequences of 8k-32k 210 / 183 / 175 /
    // 195, 32 windows of 4096 41 / 49 / 58 / 86, 64 of 1k-4k 63 / 68 / 90 / 144, 8 of 8k-32k 151 / 81 / 66 / 66.
    L.splits = 1;
    while (L.splits < kMaxSplits) {
        const int64_t ctas = full * L.slices * L.splits * 2, each = steps / (L.parts * L.splits * 2);
        if (!(ctas <= room && L.splits < 8 ? each >= 1 : each >= 16 && ctas <= 4 * room)) break;
        L.splits *= 2;
    }
    L.row_bytes = ring_row(L.per_cta, kv_unit_bytes(D));
    const int step = L.parts * kStep * L.row_bytes;
    // (a CTA that has its SM to itself takes all of it; clusters do not: fewer of them would fit the GPU at a time, 16 CTAs
    // of one 131072-position sequence's 8 heads 101 us instead of 71)
    const bool alone = ctas_per_sm(D, NT) == 1 || (L.splits == 1 && full * L.slices <= sms);
    L.stages = std::max(2, std::min(kMaxStages, (alone ? kMostSmem : kHalfSmem) / step));
    const int join = L.parts * L.splits > 1 ? kWarps * M * ((D + 4) + 2 + 2) * 4 : 0;       // partial outputs, pairs twice
    const int smem = std::max(L.stages * step, join);
    const int64_t grid = slots * L.slices * L.splits;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    CUtensorMap pages;
    std::memset(&pages, 0, sizeof(pages));
    if (a.p.batch > 0 && !encode_page_map(&pages, a.kv, a.entry_bytes, a.p.block_size, a.page_bytes, a.p.num_blocks, L.row_bytes, 16))
        return cudaErrorUnknown;
    auto kernel = paged_attention_kernel<F16, E2M1, D, NT>;
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? UINT64_C(1) << dev : 0;
    if (!(raised.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
    return cudaLaunchKernelEx(&cfg, kernel, a, L, pages);
}

template <bool F16, bool E2M1>
cudaError_t launch_type(const PagedArgs& a, int head_dim, int sms, cudaStream_t st)
{
    // rows per unit: as few blocks of eight as hold a sequence's, within the registers (an accumulator of D x 8 NT
    // fp32 per warp)
    const int64_t rows = most_rows(a);
    if (head_dim == 64) {
        if (rows <= 8) return launch_shape<F16, E2M1, 64, 1>(a, sms, st);
        if (rows <= 16) return launch_shape<F16, E2M1, 64, 2>(a, sms, st);
        return launch_shape<F16, E2M1, 64, 4>(a, sms, st);
    }
    return rows <= 8 ? launch_shape<F16, E2M1, 128, 1>(a, sms, st) : launch_shape<F16, E2M1, 128, 2>(a, sms, st);
}

}  // namespace

// A block of 128 rows of the tensor cores costs what 19 rows of this kernel do, and their kernel a few us more.  us for this
// kernel and for that one, 8 KV heads of 128: 32 sequences of 16384 positions, 16 rows each 218 and 246, 24 rows 404 and 247; 4
// sequences of 16384, 16 rows 33 and 43, 24 rows 63 and 43; 24 of 512, 32 rows 21 and 22, 64 rows 29 and 22; 4 of 512, 64 rows
// 10 and 14, 128 rows 14 and 16; 4 heads of 64, 16 sequences of 12000, 28 rows 47 and 45, 42 rows 91 and 45.
bool paged_in_chunks(const PagedArgs& a)
{
    if (most_rows(a) <= 16) return false;
    const int group = a.heads_q / a.heads_kv;
    int32_t blocks;
    const int64_t few = row_slots(a, 16, group, &blocks) * most_positions(a, 16, group);
    const int64_t many = row_slots(a, 128, group, &blocks) * most_positions(a, 128, group);
    return a.heads_kv * (5 * few - 6 * many) > 900000;
}

cudaError_t launch_paged_attention(const PagedArgs& a, int head_dim, bool f16, bool e2m1, int sms, cudaStream_t st)
{
    if (a.route ? a.route == 2 : paged_in_chunks(a)) return launch_paged_chunk(a, head_dim, f16, e2m1, most_rows(a), sms, st);
    if (f16) return e2m1 ? launch_type<true, true>(a, head_dim, sms, st) : launch_type<true, false>(a, head_dim, sms, st);
    return e2m1 ? launch_type<false, true>(a, head_dim, sms, st) : launch_type<false, false>(a, head_dim, sms, st);
}

}  // namespace qli
