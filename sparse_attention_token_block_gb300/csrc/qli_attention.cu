// qli_attention.cu -- attention of each query row over the KV-cache entries that its index list
// names, the entries held in 4 bits:
//     z_i = scale * q_h . K_i,   out_h = sum_i softmax(z)_i V_i,   lse_h = ln sum_i exp(z_i)
//
// A cluster of `splits` CTAs works on one row (or a slice of its KV heads), each on a slice of the
// list.  A CTA first resolves its slice -- index, bounds, block_table -- into a compact list of the
// valid entries' addresses.  Each of its eight warps then carries one unit, a KV head with up to
// 8 * NT of its query heads, over its share of the entries, 16 at a time, on its own: it copies its
// head's bytes of each entry (144 for D = 128) into a ring of its own with 16-byte asynchronous
// copies, kStages tiles deep, and meets no other warp until the end.  (One bulk copy per entry from
// a producer warp, all heads in one copy, measured slower: an SM takes about 44 cycles per bulk copy
// whatever its size.)
//
//   * logits:  S^T (16 entries x 8 heads) = K Q^T.  A lane decodes 4-bit keys straight into the A
//     fragment: lane (r, c) of a warp holds rows r and r + 8, so it takes 1/4 of two key vectors as one
//     shared-memory load each; which of its columns meets which step of the product is free as long as
//     the query fragment, loaded once, follows the same order.
//   * softmax: running maximum and sum per head in fp32 (base 2).  The accumulators are rescaled only
//     when some logit exceeds the maximum in use by more than 8 (then p stays within 2^8, inside
//     fp16's range at full precision), so most tiles skip the exchange between lanes.
//   * output:  O^T (D x 8 heads) += V^T P^T.  P goes from accumulator to B fragment by 8 x 8
//     transposes.  V^T's A fragment pairs two entries per register: the nibbles of two entries are
//     interleaved before they are decoded.
//
// Heads never fill the M side of a product, entries do, so groups of 8 query heads waste nothing of
// the tensor cores.  4-bit values times e4m3 scales are exact in fp16 (at most 6 significant bits,
// 2^-10 to 2688); queries are scaled by a power of two of their head's largest magnitude, so that
// bfloat16 fits fp16 too (elements below 2^-14 of the largest lose bits of 2^-25 of it).
//
// Partial results of the warps and CTAs that share a unit meet in shared memory (distributed over
// the cluster) and are joined in a fixed order.
#include <cuda_runtime.h>

#include <cfloat>

#include "qli_kv.cuh"

namespace qli {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxPerThread = kMaxSparse / kThreads;
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
    int32_t ring_off;      // shared-memory offset of the rings, behind the list
};

// One KV head's bytes of an entry, widened to 16-byte pieces (they start on a multiple of 8 for
// D = 64), and the stride of entries in a ring: 32 or 96 beyond a multiple of 128
constexpr int pieces_of(int d) { return d == 128 ? 9 : 5; }
constexpr int row_bytes_of(int d) { return d == 128 ? 160 : 96; }
constexpr int stages_of(int d) { return d == 128 ? 2 : 3; }          // of 32 entries each (two CTAs fit an SM)

// Entry (of a group of eight) that row r of an 8-row fragment holds.  Rows 2c and 2c + 1 hold entries
// c and 4 + (c + 2) % 4: with an entry stride of 32 or 96 modulo 128 bytes, the four entries that a
// quarter-warp reads of V and the two that it reads of K then lie in different banks.
__device__ __forceinline__ int entry_of_row(int r) { return (r & 1) ? 4 + (((r >> 1) + 2) & 3) : r >> 1; }

// A value of another CTA's shared memory (of this CTA's when there is no cluster)
__device__ __forceinline__ float peer_load(const float* p, int rank, int splits)
{
    return splits > 1 ? __uint_as_float(ptx::ld_cluster(ptx::cluster_addr(p, rank))) : *p;
}

__device__ __forceinline__ float4 peer_load4(const float* p, int rank, int splits)
{
    return splits > 1 ? ptx::ld_cluster4(ptx::cluster_addr(p, rank)) : *reinterpret_cast<const float4*>(p);
}

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

template <bool F16, bool E2M1, int D, int NT>
__global__ void __launch_bounds__(kThreads, NT * D <= 128 ? 2 : 1)
    attention_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ Layout L)
{
    constexpr int kUnit = kv_unit_bytes(D);
    constexpr int NW = D / 32;                    // words of key codes per lane and entry
    constexpr int MO = D / 16;                    // 16-row tiles of the output
    constexpr int kHeadStride = D + 4;            // of partial outputs, in floats
    constexpr int kPieces = pieces_of(D), kRow = row_bytes_of(D), kPair = 32 * kRow, kStages = stages_of(D);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int32_t warp_count[kWarps];
    int64_t* list = reinterpret_cast<int64_t*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int rank = L.splits > 1 ? (int)ptx::cluster_rank() : 0;
    const int64_t task = blockIdx.x / L.splits, row = task / L.ctas;
    const int u0 = (int)(task - row * L.ctas) * L.per_cta, nu = min(L.per_cta, L.units - u0);
    const int group = a.heads_q / a.heads_kv;
    ptx::pdl_wait();

    // ---- the slice's valid entries, in list order, as byte offsets into the pool
    const int k0 = rank * L.per_split, n = max(0, min(L.per_split, a.p.sparse_count - k0));
    int32_t j[kMaxPerThread], page[kMaxPerThread];
    int mine = 0;
    const uint32_t bs = (uint32_t)a.p.block_size;
    {
        const int64_t b = row_batch(a.p, a.seq_lens_q, row);
        const int64_t limit = b >= 0 ? index_limit(a.p, a.seq_lens_k, b) : -1;
        const int32_t* idx = a.idx + row * a.p.sparse_count + k0;
        const int32_t* table = a.block_table + b * a.p.max_blocks_per_seq;
        const int per = (n + kThreads - 1) / kThreads, at = tid * per;
        uint32_t bits = 0;
#pragma unroll
        for (int e = 0; e < kMaxPerThread; ++e) j[e] = e < per && at + e < n ? idx[at + e] : -1;
#pragma unroll
        for (int e = 0; e < kMaxPerThread; ++e) {
            const bool ok = j[e] >= 0 && j[e] < limit;
            if (j[e] != -1 && !ok) bits |= kErrLength;
            page[e] = ok ? table[(uint32_t)j[e] / bs] : -1;
            if (!ok) j[e] = -1;
        }
#pragma unroll
        for (int e = 0; e < kMaxPerThread; ++e) {
            const bool ok = j[e] >= 0 && page[e] >= 0 && page[e] < a.p.num_blocks;
            if (j[e] >= 0 && !ok) bits |= kErrPage;
            if (!ok) j[e] = -1;
            mine += ok ? 1 : 0;
        }
        bits = __reduce_or_sync(0xffffffffu, bits);
        if (bits && lane == 0 && a.err) atomicOr(a.err, bits);
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane == 31) warp_count[wid] = sum;
        mine = sum - mine;                        // entries of the warp's earlier lanes
    }
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == wid) mine += total;
        total += warp_count[w];
    }
#pragma unroll
    for (int e = 0; e < kMaxPerThread; ++e)
        if (j[e] >= 0) {
            const int64_t at = page[e] * a.page_bytes + (int64_t)((uint32_t)j[e] % bs) * a.entry_bytes;
            list[mine++] = at;
            if (mine == total)                    // filled up to 32 with the last one (masked below)
                for (int x = mine; x & 31; ++x) list[x] = at;
        }
    __syncthreads();

    const int active = nu * L.parts;              // consumer warps with work
    const int unit = wid / L.parts, part = wid - unit * L.parts;
    const int kvh = (u0 + unit) / L.chunks;
    const int h0 = kvh * group + (u0 + unit - kvh * L.chunks) * 8 * NT;      // the unit's first query head
    const int nh = min(8 * NT, (kvh + 1) * group - h0);
    const int r = lane >> 2, c = lane & 3;
    float o[NT][MO][4], m[NT][2], l[NT][2];
    if (wid < active) {
        // The lane's 16-byte copies of 32 entries: four lanes take 64 bytes in a row of one entry, eight
        // entries at a time, and the one piece that is left over goes by entry = lane.  Code bytes of odd
        // heads start 16 bytes past a sector, so there the left-over piece is the first one.
        const int pairs = (total + 31) / 32;
        const int head_lo = kvh * kUnit & ~15;
        const int quad_at = (D == 128 && (kvh & 1)) ? 16 : 0, rest_at = quad_at ? 0 : 16 * (kPieces - 1);
        uint8_t* ring = smem + L.ring_off + wid * kStages * kPair;
        const uint8_t* src = a.kv + head_lo + quad_at + 16 * (lane & 3);
        const uint8_t* src_rest = a.kv + head_lo + rest_at;
        uint8_t* dst = ring + (lane >> 2) * kRow + quad_at + 16 * (lane & 3);
        uint8_t* dst_rest = ring + lane * kRow + rest_at;
        auto copy_pair = [&](int pi, int stage) {
            if (pi < pairs) {
                const int64_t* at = list + 32 * pi;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint8_t* x = src + at[(lane >> 2) + 8 * i];
#pragma unroll
                    for (int y = 0; y < kPieces / 4; ++y)
                        ptx::cp_async<16>(dst + stage * kPair + 8 * i * kRow + 64 * y, x + 64 * y);
                }
                ptx::cp_async<16>(dst_rest + stage * kPair, src_rest + at[lane]);
            }
            ptx::cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) copy_pair(part + i * L.parts, i);
        // query fragments: head r of each block of eight, this lane's quarter of D, scaled by a power of two
        uint32_t q[NT][NW][4];
        float f[NT][2];                           // base-2 logit factor of heads 2c and 2c + 1
        const uint16_t* qrow = static_cast<const uint16_t*>(a.query) + row * a.q_stride + (int64_t)h0 * D;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            uint32_t w[NW][4];
            const bool live = 8 * t + r < nh;
#pragma unroll
            for (int j = 0; j < NW; ++j) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (live) v = *reinterpret_cast<const uint4*>(qrow + (int64_t)(8 * t + r) * D + c * (D / 4) + 8 * j);
                w[j][0] = v.x;
                w[j][1] = v.y;
                w[j][2] = v.z;
                w[j][3] = v.w;
            }
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
            const float up = __uint_as_float(ex << 23) * (a.softmax_scale * a.k_scale * 1.4426950408889634f);
            f[t][0] = fminf(__shfl_sync(0xffffffffu, up, 8 * c), 3.0e38f);
            f[t][1] = fminf(__shfl_sync(0xffffffffu, up, 8 * c + 4), 3.0e38f);
#pragma unroll
            for (int i = 0; i < MO; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][i][e] = 0.0f;
            m[t][0] = m[t][1] = -FLT_MAX;
            l[t][0] = l[t][1] = 0.0f;
        }
        const int tk = entry_of_row(r), ta = c, tb = 4 + ((c + 2) & 3);
        const uint8_t* kp = ring + kvh * kUnit - head_lo + tk * kRow;          // the lane's key rows, value entries
        const uint8_t* vp = ring + kvh * kUnit - head_lo;
        int stage = 0;
#pragma unroll 1
        for (int pi = part; pi < pairs; pi += L.parts) {
            ptx::cp_async_wait<kStages - 2>();     // the lane's copies of these entries have landed ...
            __syncwarp();                          // ... and the others'; the entries before them are done with
            copy_pair(pi + (kStages - 1) * L.parts, stage == 0 ? kStages - 1 : stage - 1);
            const uint8_t* kx = kp + stage * kPair;
            const uint8_t* vx = vp + stage * kPair;
            stage = stage == kStages - 1 ? 0 : stage + 1;
            // ---- logits of two tiles of 16 entries
            float s[2][NT][4];
            uint32_t w[2][2][NW], g[2][2][2];      // tile, row r or r + 8: codes and the two halves' scales
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint8_t* x = kx + (16 * u + 8 * y) * kRow;
                    load_words<NW>(x + (D / 8) * c, w[u][y]);
                    if constexpr (D == 128) {
                        const uint32_t h = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(x + D + 2 * c));
                        g[u][y][0] = __byte_perm(h, 0, 0x1010);
                        g[u][y][1] = __byte_perm(h, 0, 0x3232);
                    } else {
                        g[u][y][0] = g[u][y][1] = __byte_perm(e4m3x2_to_f16x2(x[D + c]), 0, 0x1010);
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
                    decode_pairs<E2M1>(w[u][0][j], x);
                    decode_pairs<E2M1>(w[u][1][j], y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = ptx::mul_f16x2(x[i], g[u][0][j / (NW / 2)]);
                        y[i] = ptx::mul_f16x2(y[i], g[u][1][j / (NW / 2)]);
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        ptx::mma_16816(s[u][t], x[0], y[0], x[1], y[1], q[t][j][0], q[t][j][1]);
                        ptx::mma_16816(s[u][t], x[2], y[2], x[3], y[3], q[t][j][2], q[t][j][3]);
                    }
                }
            // ---- softmax: entries past the end get -infinity
            const int left = total - 32 * pi;      // 32 or more except in the last pair
            float z[2][NT][4], over = -INFINITY;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[u][t][e] = fmaf(s[u][t][e], f[t][e & 1], -m[t][e & 1]);
            if (left < 32) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (16 * u + 8 * (e >> 1) + tk >= left) z[u][t][e] = -INFINITY;
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
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[u][t][e] = ptx::ex2(z[u][t][e]);
                    l[t][0] += z[u][t][0] + z[u][t][2];
                    l[t][1] += z[u][t][1] + z[u][t][3];
                    // one rounding to fp16 of each probability (the sum keeps the unrounded ones)
                    pb[u][t][0] = ptx::transpose_8x8(float2_to_act2<true>(z[u][t][0], z[u][t][1]));
                    pb[u][t][1] = ptx::transpose_8x8(float2_to_act2<true>(z[u][t][2], z[u][t][3]));
                }
            // ---- output
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t* va = vx + (16 * u + ta) * kRow;
                const uint8_t* vb = vx + (16 * u + tb) * kRow;
                const int off = D / 2 + r * (D / 16), soff = D + D / 16 + (D == 128 ? r : r >> 1);
                const uint32_t sab = e4m3x2_to_f16x2(va[soff] | (uint32_t)vb[soff] << 8);
                const uint32_t scd = e4m3x2_to_f16x2(va[8 * kRow + soff] | (uint32_t)vb[8 * kRow + soff] << 8);
                uint32_t wa[NW / 2], wb[NW / 2], wc[NW / 2], wd[NW / 2];
                load_words<NW / 2>(va + off, wa);
                load_words<NW / 2>(vb + off, wb);
                load_words<NW / 2>(va + 8 * kRow + off, wc);
                load_words<NW / 2>(vb + 8 * kRow + off, wd);
#pragma unroll
                for (int j = 0; j < NW / 2; ++j) {
                    uint32_t x[8], y[8];
                    decode_across<E2M1>(wa[j], wb[j], x);
                    decode_across<E2M1>(wc[j], wd[j], y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a0 = ptx::mul_f16x2(x[2 * i], sab), a1 = ptx::mul_f16x2(x[2 * i + 1], sab);
                        const uint32_t a2 = ptx::mul_f16x2(y[2 * i], scd), a3 = ptx::mul_f16x2(y[2 * i + 1], scd);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            ptx::mma_16816(o[t][4 * j + i], a0, a1, a2, a3, pb[u][t][0], pb[u][t][1]);
                    }
                }
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
    uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.heads_q * D;
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
                    a.lse[row * a.heads_q + h0 + h] = sum == 0.0f ? -INFINITY : (m[t][e] + log2f(sum)) * 0.6931471805599453f;
            }
        return;
    }
    // partial outputs [warp][8 NT heads][kHeadStride], then (maximum, sum) [warp][8 NT heads]
    __syncthreads();                               // the rings are free
    float* part_o = reinterpret_cast<float*>(smem + L.ring_off);
    float* part_ml = part_o + active * 8 * NT * kHeadStride;
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
                if (r == 0) {
                    part_ml[2 * h] = m[t][e];
                    part_ml[2 * h + 1] = l[t][e];
                }
            }
    }
    if (L.splits > 1) ptx::cluster_sync();
    else __syncthreads();
    // every CTA: the weight 2^(m - top) * v_scale / sum of each partial result of each head
    float* weight = part_ml + active * 8 * NT * 2;          // [split * parts + part][nu * 8 NT]
    const int heads = nu * 8 * NT, partials = L.splits * L.parts;
    for (int hh = tid; hh < heads; hh += kThreads) {
        const int un = hh / (8 * NT), h = hh - un * 8 * NT;
        const int kv = (u0 + un) / L.chunks, first = kv * group + (u0 + un - kv * L.chunks) * 8 * NT;
        float top = -FLT_MAX, sum = 0.0f;
#pragma unroll 4
        for (int x = 0; x < partials; ++x) {
            const int sp = x / L.parts;
            const float pm = peer_load(part_ml + 2 * ((un * L.parts + x - sp * L.parts) * 8 * NT + h), sp, L.splits);
            weight[x * heads + hh] = pm;
            top = fmaxf(top, pm);
        }
#pragma unroll 4
        for (int x = 0; x < partials; ++x) {
            const int sp = x / L.parts;
            const float pl = peer_load(part_ml + 2 * ((un * L.parts + x - sp * L.parts) * 8 * NT + h) + 1, sp, L.splits);
            const float g = ptx::ex2(weight[x * heads + hh] - top);
            weight[x * heads + hh] = g;
            sum = fmaf(g, pl, sum);
        }
        const float inv = sum == 0.0f ? 0.0f : a.v_scale / sum;
        for (int x = 0; x < partials; ++x) weight[x * heads + hh] *= inv;
        if (a.lse && rank == 0 && first + h < (kv + 1) * group)
            a.lse[row * a.heads_q + first + h] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
    __syncthreads();
    for (int i = rank * kThreads + tid; i < heads * (D / 8); i += L.splits * kThreads) {      // 8 elements of a head
        const int hh = i / (D / 8), d8 = i - hh * (D / 8), un = hh / (8 * NT), h = hh - un * 8 * NT;
        const int kv = (u0 + un) / L.chunks, first = kv * group + (u0 + un - kv * L.chunks) * 8 * NT;
        if (first + h >= (kv + 1) * group) continue;
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
        for (int x = 0; x < partials; ++x) {
            const int sp = x / L.parts;
            const float* from = part_o + ((un * L.parts + x - sp * L.parts) * 8 * NT + h) * kHeadStride + 8 * d8;
            const float4 v = peer_load4(from, sp, L.splits), w = peer_load4(from + 4, sp, L.splits);
            const float g = weight[x * heads + hh];
            acc[0] = fmaf(g, v.x, acc[0]), acc[1] = fmaf(g, v.y, acc[1]), acc[2] = fmaf(g, v.z, acc[2]);
            acc[3] = fmaf(g, v.w, acc[3]), acc[4] = fmaf(g, w.x, acc[4]), acc[5] = fmaf(g, w.y, acc[5]);
            acc[6] = fmaf(g, w.z, acc[6]), acc[7] = fmaf(g, w.w, acc[7]);
        }
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = float2_to_act2<F16>(acc[2 * e], acc[2 * e + 1]);
        *reinterpret_cast<uint4*>(out + (int64_t)(first + h) * D + 8 * d8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    if (L.splits > 1) ptx::cluster_sync();         // no CTA leaves while another reads its partial results
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
    L.ctas = (L.units + kWarps - 1) / kWarps;
    L.per_cta = (L.units + L.ctas - 1) / L.ctas;
    L.splits = 1;
    const int slots = (NT * D <= 128 ? 2 : 1) * sms;
    while (L.splits < 8 && rows * L.ctas * L.splits * 2 <= slots && k > 64 * L.splits) L.splits *= 2;
    L.ctas = (L.units + L.per_cta - 1) / L.per_cta;
    L.parts = kWarps / L.per_cta;
    L.per_split = (k + L.splits - 1) / L.splits;
    L.ring_off = 8 * ((L.per_split + 31) & ~31);
    int ring = kWarps * stages_of(D) * 32 * row_bytes_of(D);
    const int join = kWarps * 8 * NT * ((D + 4) + 2 + L.splits) * 4;      // partial outputs, (m, l), weights
    if (L.parts * L.splits > 1 && ring < join) ring = join;
    const int smem = L.ring_off + ring;
    const int64_t grid = rows * L.ctas * L.splits;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    auto kernel = attention_kernel<F16, E2M1, D, NT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
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
    return cudaLaunchKernelEx(&cfg, kernel, a, L);
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
    if (f16) return e2m1 ? launch_type<true, true>(a, head_dim, sms, st) : launch_type<true, false>(a, head_dim, sms, st);
    return e2m1 ? launch_type<false, true>(a, head_dim, sms, st) : launch_type<false, false>(a, head_dim, sms, st);
}

}  // namespace qli
