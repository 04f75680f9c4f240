// qli_attention.cu -- attention of each query row over the KV-cache entries that its index list
// names, the entries held in 4 bits:
//     z_i = scale * q_h . K_i,   out_h = sum_i softmax(z)_i V_i,   lse_h = ln sum_i exp(z_i)
//
// One CTA per (row, KV head, eight of its query heads).  A tile of 32 listed entries is decoded
// into shared memory in fp32; each of the four warps carries two query heads, one entry per lane for
// the logits and D / 32 output elements per lane for the weighted sum, with the running maximum and
// sum of the softmax.
#include <cuda_runtime.h>

#include "qli_kv.cuh"

namespace qli {

namespace {

constexpr int kAttnThreads = 128;
constexpr int kAttnTile = 32;
constexpr int kAttnHeads = 8;

template <bool F16, bool E2M1, int D>
__global__ void __launch_bounds__(kAttnThreads) attention_kernel(AttentionArgs a)
{
    __shared__ float ks[kAttnTile][D + 1], vs[kAttnTile][D];
    __shared__ float qs[kAttnHeads][D];
    __shared__ int64_t src[kAttnTile];
    ptx::pdl_wait();
    const int group = a.heads_q / a.heads_kv, chunks = (group + kAttnHeads - 1) / kAttnHeads;
    const int64_t unit = (int64_t)a.heads_kv * chunks, r = blockIdx.x / unit;
    const int uh = (int)(blockIdx.x - r * unit), kvh = uh / chunks, h0 = kvh * group + (uh - kvh * chunks) * kAttnHeads;
    const int nh = min(kAttnHeads, (kvh + 1) * group - h0);
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const uint16_t* q = static_cast<const uint16_t*>(a.query) + r * a.q_stride + (int64_t)h0 * D;
    for (int i = tid; i < kAttnHeads * D / 2; i += kAttnThreads) {
        const int h = 2 * i / D;
        float2 f = make_float2(0.0f, 0.0f);
        if (h < nh) f = act2_to_float2<F16>(reinterpret_cast<const uint32_t*>(q)[i]);
        qs[h][2 * i % D] = f.x * a.softmax_scale;              // (first, so that the products stay in range)
        qs[h][2 * i % D + 1] = f.y * a.softmax_scale;
    }
    const int64_t b = row_batch(a.p, a.seq_lens_q, r);
    const int64_t limit = b >= 0 ? index_limit(a.p, a.seq_lens_k, b) : -1;
    const int k = a.p.sparse_count;
    const int32_t* idx = a.idx + r * k;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, acc[2][D / 32];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < D / 32; ++e) acc[j][e] = 0.0f;
    uint32_t bits = 0;
    for (int t0 = 0; t0 < k; t0 += kAttnTile) {
        __syncthreads();
        if (tid < kAttnTile) {
            const int j = t0 + tid < k ? idx[t0 + tid] : -1;
            src[tid] = j == -1 ? -1
                               : kv_entry_offset(a.p, a.block_table, b, j, limit, a.page_bytes, a.entry_bytes, &bits);
        }
        __syncthreads();
        for (int i = tid; i < kAttnTile * D / 8; i += kAttnThreads) {
            const int t = i / (D / 8), c = i - t * (D / 8);
            float kf[8] = {0, 0, 0, 0, 0, 0, 0, 0}, vf[8] = {0, 0, 0, 0, 0, 0, 0, 0}, sk = 0.0f, sv = 0.0f;
            if (src[t] >= 0) {
                const uint8_t* e = a.kv + src[t] + kvh * kv_unit_bytes(D);
                decode8<E2M1>(*reinterpret_cast<const uint32_t*>(e + 4 * c), kf);
                decode8<E2M1>(*reinterpret_cast<const uint32_t*>(e + D / 2 + 4 * c), vf);
                sk = e4m3_to_float(e[D + c / 2]) * a.k_scale;
                sv = e4m3_to_float(e[D + D / 16 + c / 2]) * a.v_scale;
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                ks[t][8 * c + x] = kf[x] * sk;
                vs[t][8 * c + x] = vf[x] * sv;
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int h = 2 * wid + j;
            if (h >= nh) continue;
            float z = 0.0f;
            for (int d = 0; d < D; ++d) z = fmaf(qs[h][d], ks[lane][d], z);
            z = src[lane] >= 0 ? z : -INFINITY;
            float top = z;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float mn = fmaxf(m[j], top);
            if (mn == -INFINITY) continue;                     // nothing valid so far
            const float p = __expf(z - mn), f = __expf(m[j] - mn);
            m[j] = mn;
            l[j] = l[j] * f + p;                               // per lane; summed at the end
#pragma unroll
            for (int e = 0; e < D / 32; ++e) acc[j][e] *= f;
            for (int t = 0; t < kAttnTile; ++t) {
                const float pt = __shfl_sync(0xffffffffu, p, t);
#pragma unroll
                for (int e = 0; e < D / 32; ++e) acc[j][e] = fmaf(pt, vs[t][32 * e + lane], acc[j][e]);
            }
        }
    }
    bits = __reduce_or_sync(0xffffffffu, bits);
    if (bits && lane == 0 && a.err) atomicOr(a.err, bits);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int h = 2 * wid + j;
        if (h >= nh) continue;
        float total = l[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        const float inv = total > 0.0f ? 1.0f / total : 0.0f;
        uint16_t* out = static_cast<uint16_t*>(a.out) + (r * a.heads_q + h0 + h) * D;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
            out[32 * e + lane] = (uint16_t)float2_to_act2<F16>(acc[j][e] * inv, 0.0f);
        if (a.lse && lane == 0) a.lse[r * a.heads_q + h0 + h] = total > 0.0f ? m[j] + logf(total) : -INFINITY;
    }
}

template <bool F16, bool E2M1>
cudaError_t launch_type(const AttentionArgs& a, int head_dim, cudaStream_t st)
{
    const int group = a.heads_q / a.heads_kv, chunks = (group + kAttnHeads - 1) / kAttnHeads;
    const int64_t grid = (int64_t)a.p.rows * a.heads_kv * chunks;
    auto kernel = head_dim == 64 ? attention_kernel<F16, E2M1, 64> : attention_kernel<F16, E2M1, 128>;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kAttnThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_attention(const AttentionArgs& a, int head_dim, bool f16, bool e2m1, int, cudaStream_t st)
{
    if (f16) return e2m1 ? launch_type<true, true>(a, head_dim, st) : launch_type<true, false>(a, head_dim, st);
    return e2m1 ? launch_type<false, true>(a, head_dim, st) : launch_type<false, false>(a, head_dim, st);
}

}  // namespace qli
