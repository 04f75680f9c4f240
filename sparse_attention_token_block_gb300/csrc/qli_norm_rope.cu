// qli_norm_rope.cu -- norm of each query and key head and the position rotation in one pass:
//     y = x / sqrt(mean(x^2) + eps) * w,   (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)
// over the R leading elements (pairs (i, i + R/2) or (2i, 2i + 1)), fp32 throughout, rounded once.
//
// A stream over HBM: 2 bytes read and 2 written per element and a table row per token.  A CTA works
// on one token (few tokens: several CTAs on one, by heads), so the rotation's factors and the weights
// stay in registers; D / 8 lanes share a head vector, and each does kHeads heads at a time with all their
// loads under way before the first is used.  A lane has two chunks of four elements of a vector,
// chosen so that it holds both elements of its pairs: in the half layout lane l < R/8 takes 4l.. and
// R/2 + 4l.., in the interleaved layout (and past R) eight consecutive elements.  So the rotation
// needs no exchange between lanes and the norm only a sum over the group.
#include <cuda_runtime.h>

#include "qli_kv.cuh"

namespace qli {

namespace {

constexpr int kNormThreads = 256;

template <bool F16>
__device__ __forceinline__ void unpack8(const uint2& u, const uint2& v, float (&y)[8])
{
    const uint32_t w[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = act2_to_float2<F16>(w[i]);
        y[2 * i] = f.x;
        y[2 * i + 1] = f.y;
    }
}

template <bool F16, int D, bool kInterleaved, int kHeads>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(NormRopeArgs a)
{
    constexpr int G = D / 8, kGroups = kNormThreads / G;           // lanes per vector, vectors at a time
    ptx::pdl_wait();
    const int lane = threadIdx.x % G, R = a.rotary;
    const int64_t t = blockIdx.x;
    const int heads = a.heads[0] + a.heads[1], step = kGroups * gridDim.y;
    const int h_first = blockIdx.y * kGroups + threadIdx.x / G;
    // the lane's chunks [c0, c0 + 4) and [c1, c1 + 4)
    const bool rot = 8 * lane < R;
    const int c0 = (kInterleaved || !rot) ? 8 * lane : 4 * lane;
    const int c1 = (kInterleaved || !rot) ? c0 + 4 : R / 2 + 4 * lane;
    // (the key side's pointers start that many heads earlier, so that one head number serves both)
    const uint16_t* const in_q = static_cast<const uint16_t*>(a.in[0]) + t * a.in_stride[0];
    const uint16_t* const in_k = static_cast<const uint16_t*>(a.in[1]) + t * a.in_stride[1] - (int64_t)a.heads[0] * D;
    uint16_t* const out_q = static_cast<uint16_t*>(a.out[0]) + t * a.out_stride[0];
    uint16_t* const out_k = static_cast<uint16_t*>(a.out[1]) + t * a.out_stride[1] - (int64_t)a.heads[0] * D;
    uint2 w[2][2] = {};
    const int pos = a.positions[t];
    const bool ok = pos >= 0 && pos < a.max_positions;
    if (!ok && a.err && h_first == 0 && lane == 0) atomicOr(a.err, kErrLength);
    float cs[8] = {1, 1, 1, 1, 0, 0, 0, 0};                        // cosines, sines of the lane's pairs
    for (int h0 = h_first; h0 - h_first < heads; h0 += kHeads * step) {        // (a whole group leaves together)
        uint2 x[kHeads][2];
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = h0 + u * step, side = h >= a.heads[0];
            x[u][0] = x[u][1] = make_uint2(0u, 0u);
            if (h < heads) {
                const uint16_t* p = (side ? in_k : in_q) + h * D;
                x[u][0] = *reinterpret_cast<const uint2*>(p + c0);
                x[u][1] = *reinterpret_cast<const uint2*>(p + c1);
            }
        }
        if (h0 == h_first) {
            if (a.norm) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint16_t* p = static_cast<const uint16_t*>(a.weight[s]);
                    if (p) {
                        w[s][0] = *reinterpret_cast<const uint2*>(p + c0);
                        w[s][1] = *reinterpret_cast<const uint2*>(p + c1);
                    }
                }
            }
            if (ok && rot) {
                const float* p = a.cos_sin + (int64_t)pos * R + 4 * lane;
                const float4 c = *reinterpret_cast<const float4*>(p), s = *reinterpret_cast<const float4*>(p + R / 2);
                cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
                cs[4] = s.x, cs[5] = s.y, cs[6] = s.z, cs[7] = s.w;
            }
        }
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = h0 + u * step, side = h >= a.heads[0];
            float y[8];
            unpack8<F16>(x[u][0], x[u][1], y);
            if (a.norm) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
                for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float r = rsqrtf(ss * (1.0f / D) + a.eps);
                float g[8];
                unpack8<F16>(side ? w[1][0] : w[0][0], side ? w[1][1] : w[0][1], g);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = y[i] * r * g[i];
            }
            if (h >= heads) continue;
            // pairs (i, i + 4) of the lane's elements, or (2i, 2i + 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = kInterleaved ? 2 * i : i, q = kInterleaved ? 2 * i + 1 : i + 4;
                const float ya = y[p], yb = y[q];
                if (rot) {
                    y[p] = ya * cs[i] - yb * cs[4 + i];
                    y[q] = yb * cs[i] + ya * cs[4 + i];
                }
            }
            uint2 lo = make_uint2(float2_to_act2<F16>(y[0], y[1]), float2_to_act2<F16>(y[2], y[3]));
            uint2 hi = make_uint2(float2_to_act2<F16>(y[4], y[5]), float2_to_act2<F16>(y[6], y[7]));
            if (!ok) lo = hi = make_uint2(0u, 0u);
            uint16_t* p = (side ? out_k : out_q) + h * D;
            *reinterpret_cast<uint2*>(p + c0) = lo;
            *reinterpret_cast<uint2*>(p + c1) = hi;
        }
    }
}

template <bool F16, bool kInterleaved>
cudaError_t launch_type(const NormRopeArgs& a, int head_dim, int sms, cudaStream_t st)
{
    // CTAs per token: as many as leave each group of lanes one head, once there are enough tokens five
    // heads (prefill of 15360 tokens, 72 heads of 128: 143 us with one, 107 with five)
    const int groups = kNormThreads / (head_dim / 8), heads = a.heads[0] + a.heads[1];
    int64_t slices = ceil_div64(heads, groups);
    const bool many = slices > 1 && a.tokens * slices > 4 * sms;
    if (many) slices = ceil_div64(slices, 5);
    auto kernel = many ? (head_dim == 64 ? norm_rope_kernel<F16, 64, kInterleaved, 5>
                                         : (head_dim == 128 ? norm_rope_kernel<F16, 128, kInterleaved, 5>
                                                            : norm_rope_kernel<F16, 256, kInterleaved, 5>))
                       : (head_dim == 64 ? norm_rope_kernel<F16, 64, kInterleaved, 1>
                                         : (head_dim == 128 ? norm_rope_kernel<F16, 128, kInterleaved, 1>
                                                            : norm_rope_kernel<F16, 256, kInterleaved, 1>));
    return launch_pdl(kernel, dim3((unsigned)a.tokens, (unsigned)slices), dim3(kNormThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int head_dim, bool f16, int sms, cudaStream_t st)
{
    if (f16) return a.interleaved ? launch_type<true, true>(a, head_dim, sms, st) : launch_type<true, false>(a, head_dim, sms, st);
    return a.interleaved ? launch_type<false, true>(a, head_dim, sms, st) : launch_type<false, false>(a, head_dim, sms, st);
}

}  // namespace qli
