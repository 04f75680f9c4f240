// qli_paged.cuh -- which (token, query head) rows a CTA of the dense paged attention works on, and which cached
// positions they see.
#pragma once

#include <cfloat>

#include "qli_kv.cuh"

namespace qli {

struct PagedArgs {
    Params p;
    const void* query;
    int64_t q_stride;                      // elements between rows
    const int32_t* seq_lens_q;
    const int32_t* seq_lens_k;
    const int32_t* block_table;
    const uint8_t* kv;
    void* out;
    float* lse;                            // optional
    uint32_t* err;                         // optional sticky error word
    int64_t page_bytes;
    int32_t entry_bytes;
    int32_t heads_q, heads_kv;
    int32_t window, sinks;                 // window 0: everything up to the row's own position
    int32_t route;                         // test switch: 1 the kernel of few rows, 2 that of many
    float softmax_scale, k_scale, v_scale;
};

// A block of consecutive rows of one sequence: row i of a sequence is query head i % group (of each KV head) of
// its new token i / group
struct RowBlock {
    int32_t batch;
    int32_t first, rows;                   // of the sequence's rows
    int32_t sq, sk, lc;                    // live tokens (0 for an invalid sequence), cached tokens, positions
    int64_t row0;                          // global row of the sequence's token 0
};

// Blocks of M rows in a call (`blocks`: per sequence, BSND).  TND: sequence b's blocks begin at number
// floor(cum[b - 1] group / M) + b, which leaves it at least ceil(Sq group / M) of them, and is found without a
// scan; the rows behind the last sequence count as one more.
inline int64_t row_slots(const PagedArgs& a, int M, int group, int32_t* blocks)
{
    if (!a.p.layout_tnd) {
        *blocks = (int32_t)ceil_div64((int64_t)a.p.s1 * group, M);
        return (int64_t)a.p.batch * *blocks;
    }
    *blocks = 0;
    return (int64_t)a.p.total_q * group / M + a.p.batch + 1;
}

// Block `block` of sequence b (p.batch: of the rows behind the last); `reports`: sets the error bit of an invalid one
__device__ __forceinline__ void rows_of_block(const PagedArgs& a, int b, int block, int M, int group, bool reports, RowBlock& r)
{
    const Params& p = a.p;
    r.batch = b;
    r.sq = r.sk = r.lc = 0;
    int64_t tokens = p.s1;
    if (b >= p.batch) {
        r.row0 = p.batch > 0 ? a.seq_lens_q[p.batch - 1] : 0;
        tokens = p.total_q - r.row0;
    } else {
        const BatchExtent e = batch_extent(p, a.seq_lens_q, a.seq_lens_k, b);
        r.row0 = e.first;
        if (p.layout_tnd) tokens = e.sq;
        if (e.ok) r.sq = e.sq, r.sk = e.sk, r.lc = e.lc;
        else if (reports && a.err) atomicOr(a.err, kErrLength);
    }
    const int64_t first = (int64_t)block * M, left = tokens * group - first;
    r.first = (int32_t)min(first, (int64_t)INT32_MAX);
    r.rows = (int32_t)max((int64_t)0, min((int64_t)M, left));
}

// Block number `slot`, found by the whole CTA; rows = 0 for a number that no block has.  False: the prefix sums
// are invalid.
__device__ __forceinline__ bool find_rows(const PagedArgs& a, uint32_t slot, int blocks, int M, int group, RowBlock* out)
{
    const Params& p = a.p;
    int b, block;
    if (!p.layout_tnd) {
        b = (int)(slot / (uint32_t)blocks);
        block = (int)(slot - (uint32_t)b * blocks);
    } else {
        // sequences that begin at or before the block
        bool bad = false;
        b = 0;
        for (int i0 = 0; i0 < p.batch; i0 += blockDim.x) {
            const int i = i0 + threadIdx.x;
            bool before = false;
            if (i < p.batch) {
                const int64_t lo = i > 0 ? a.seq_lens_q[i - 1] : 0, hi = a.seq_lens_q[i];
                if (lo < 0 || hi < lo || hi > p.total_q) bad = true;
                else before = hi * group / M + i + 1 <= (int64_t)slot;
            }
            b += __syncthreads_count(before);
        }
        if (__syncthreads_or(bad)) return false;
        const int64_t done = b > 0 ? a.seq_lens_q[b - 1] : 0;
        block = (int)((int64_t)slot - (done * group / M + b));
    }
    if (threadIdx.x == 0) rows_of_block(a, b, block, M, group, true, *out);
    __syncthreads();
    return true;
}

// Positions [0, end) that the sequence's new token `token` sees (apart from the window)
__device__ __forceinline__ int seen_end(const PagedArgs& a, const RowBlock& b, int token)
{
    return (int)visible_keys(a.p.sparse_mode, a.p.cmp_ratio, b.sq, b.sk, b.lc, token, a.p.complete_blocks);
}

__device__ __forceinline__ bool sees(const PagedArgs& a, int end, int j)
{
    return j < end && (a.window == 0 || j >= end - a.window || j < a.sinks);
}

// The positions that some row of a block sees, in chunks of 16 (which share a page): first those of the sinks that
// lie before the windows, then from the first window's start (rounded down to 16) on
constexpr int kChunk = 16;
struct KeyRange {
    int base, end, chunks;
    int sink_end, sink_chunks;
    int low, high;                         // positions [high, low) are seen by every row

    __device__ __forceinline__ int position(int chunk) const
    {
        return chunk < sink_chunks ? kChunk * chunk : base + kChunk * (chunk - sink_chunks);
    }
    // end of what a chunk may count (a position is not counted as a sink and as part of the window)
    __device__ __forceinline__ int limit(int chunk) const { return chunk < sink_chunks ? sink_end : end; }
    // whether every row sees all of chunks [chunk, chunk + n)
    __device__ __forceinline__ bool all_see(int chunk, int n) const
    {
        const int pos = position(chunk), last = pos + kChunk * n;
        return last <= low && (chunk >= sink_chunks ? pos >= high : last <= sink_end);
    }
};

__device__ __forceinline__ KeyRange key_range(const PagedArgs& a, const RowBlock& b, int group)
{
    KeyRange r;
    const int t0 = b.first / group, t1 = min((b.first + b.rows - 1) / group, b.sq - 1);
    const int first = t0 < b.sq ? seen_end(a, b, t0) : 0;
    // (rows of a block behind the live ones see nothing)
    r.low = (b.first + b.rows - 1) / group < b.sq ? first : 0;
    r.end = t0 < b.sq ? seen_end(a, b, t1) : 0;
    r.high = a.window > 0 ? max(0, r.end - a.window) : 0;
    r.base = a.window > 0 ? max(0, first - a.window) & ~(kChunk - 1) : 0;
    r.sink_end = min(a.sinks, r.base);
    r.sink_chunks = (r.sink_end + kChunk - 1) / kChunk;
    r.chunks = r.end > 0 ? r.sink_chunks + (r.end - r.base + kChunk - 1) / kChunk : 0;
    return r;
}

// Page of a chunk and its position there; INT32_MIN: no row sees any of the chunk
__device__ __forceinline__ int chunk_page(const PagedArgs& a, const KeyRange& r, const int32_t* table, uint32_t block_recip, int chunk,
                                          int* at)
{
    const uint32_t bs = (uint32_t)a.p.block_size, j = (uint32_t)r.position(chunk);
    uint32_t b = __umulhi(j, block_recip);         // the reciprocal rounded down gives the quotient or one less
    if (j - b * bs >= bs) ++b;
    *at = (int)(j - b * bs);
    return chunk < r.chunks && (int)j < r.limit(chunk) ? table[b] : INT32_MIN;
}

// Most positions that a block of M rows goes over
inline int64_t most_positions(const PagedArgs& a, int M, int group)
{
    int64_t n = compressed_keys(a.p.max_seqlen_k, a.p.cmp_ratio);
    if (a.window > 0 && (int64_t)a.window + a.sinks + M / group + 32 < n) n = (int64_t)a.window + a.sinks + M / group + 32;
    return n;
}

// A row's sum as it counts.  Exponentials take s f - m at once, with m near the largest s f in fp32: from 2^28 on (base 2) fp32 holds
// every 32nd number, and 2^(s f - m) of the largest itself leaves fp16's range.  Such rows are NaN (m = -FLT_MAX: nothing seen).
__device__ __forceinline__ float sum_that_counts(float m, float sum)
{
    return fabsf(m) < 268435456.0f || m == -FLT_MAX ? sum : __int_as_float(0x7FC00000);
}

// Every row zero, shared between all threads of the launch (`thread` of `threads`)
__device__ __forceinline__ void clear_rows(const PagedArgs& a, int dim, int64_t thread, int64_t threads)
{
    if (thread == 0 && a.err) atomicOr(a.err, kErrLength);
    const int64_t heads = (int64_t)a.p.rows * a.heads_q, n = heads * dim / 8;
    for (int64_t i = thread; i < n; i += threads) static_cast<uint4*>(a.out)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse)
        for (int64_t i = thread; i < heads; i += threads) a.lse[i] = -INFINITY;
}

// NaN among two fp16 numbers made a number (scales: e4m3 has no infinity)
__device__ __forceinline__ uint32_t finite_f16x2(uint32_t h)
{
    asm("max.f16x2 %0, %0, %1;" : "+r"(h) : "r"(0xDF00DF00u));     // -448
    return h;
}

// Rows that read a KV head of one sequence, at most
inline int64_t most_rows(const PagedArgs& a)
{
    const int64_t tokens = a.p.layout_tnd ? (a.p.max_seqlen_q < a.p.total_q ? a.p.max_seqlen_q : a.p.total_q) : a.p.s1;
    return (tokens > 1 ? tokens : 1) * (a.heads_q / a.heads_kv);
}

// For many such rows (qli_paged_chunk.cu), and whether a call goes there
bool paged_in_chunks(const PagedArgs& a);
cudaError_t launch_paged_chunk(const PagedArgs& a, int head_dim, bool f16, bool e2m1, int64_t most_rows, int sms, cudaStream_t st);
cudaError_t launch_paged_attention(const PagedArgs& a, int head_dim, bool f16, bool e2m1, int sms, cudaStream_t st);

}  // namespace qli
