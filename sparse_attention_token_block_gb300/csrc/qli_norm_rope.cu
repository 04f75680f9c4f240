// qli_norm_rope.cu -- norm of each query and key head and the position rotation in one pass:
//     y = x / sqrt(mean(x^2) + eps) * w,   (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)
// over the R leading elements (pairs (i, i + R/2) or (2i, 2i + 1)), fp32 throughout, rounded once.
//
// A stream over HBM: 2 bytes read and 2 written per element and a table row per token.  A CTA works
// on one token (few tokens: several CTAs on one, by heads), so the rotation's factors stay in registers
// and the weights, as fp32, in shared memory; D / 8 lanes share a head vector, and each does kHeads heads
// at a time with all their loads under way before the first is used.  A lane has two chunks of four elements of a vector,
// chosen so that it holds both elements of its pairs: in the half layout lane l < R/8 takes 4l.. and
// R/2 + 4l.., in the interleaved layout (and past R) eight consecutive elements.  So the rotation
// needs no exchange between lanes and the norm only a sum over the group.  The arithmetic runs two
// elements at a time in packed fp32.  Measured on a GB300: 15360 tokens with 72 heads of 128 (574 MB)
// 96 us = 6.0 TB/s, 0.88 of a copy's rate; one token 1.9 us.
#include <cuda_runtime.h>

#include "qli_norm_rope.cuh"

namespace qli {

namespace {

constexpr int kNormThreads = 128;
constexpr int kMostHeads = 9;              // heads of a lane under way together: 64 registers, eight CTAs an SM

template <bool F16, int D, bool kInterleaved, int kHeads>
__global__ void __launch_bounds__(kNormThreads, kHeads > 1 ? 8 : 1) norm_rope_kernel(NormRopeArgs a)
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
    __shared__ __align__(16) float weight[2][D];
    if (a.norm) {
        for (int i = threadIdx.x; i < D; i += kNormThreads) {
            const int s = i >= D / 2, e = i - s * (D / 2);         // two elements of one side's weights
            const uint32_t* w = static_cast<const uint32_t*>(a.weight[s]);
            const float2 f = w ? act2_to_float2<F16>(w[e]) : make_float2(0.0f, 0.0f);
            *reinterpret_cast<float2*>(&weight[s][2 * e]) = f;
        }
    }
    const int pos = a.positions[t];
    const bool ok = pos >= 0 && pos < a.max_positions;
    if (!ok && a.err && h_first == 0 && lane == 0) atomicOr(a.err, kErrLength);
    float cs[8] = {1, 1, 1, 1, 0, 0, 0, 0};                        // cosines, sines of the lane's pairs
    if (ok && rot) {
        const float* p = a.cos_sin + (int64_t)pos * R + 4 * lane;
        const float4 c = *reinterpret_cast<const float4*>(p), s = *reinterpret_cast<const float4*>(p + R / 2);
        cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
        cs[4] = s.x, cs[5] = s.y, cs[6] = s.z, cs[7] = s.w;
    }
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
        if (h0 == h_first) __syncthreads();                        // the weights (behind the first loads)
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
            const int h = h0 + u * step, side = h >= a.heads[0];
            if (h0 - h_first + u * step >= heads) break;           // the same for every thread
            uint64_t y[2][2];                                      // the two chunks, in pairs
            unpack4<F16>(x[u][0], y[0]);
            unpack4<F16>(x[u][1], y[1]);
            norm_and_turn<D, kInterleaved>(y, a.norm, a.eps, &weight[side][c0], &weight[side][c1], rot, cs);
            if (h >= heads) continue;
            uint2 lo = pack4<F16>(y[0]), hi = pack4<F16>(y[1]);
            if (!ok) lo = hi = make_uint2(0u, 0u);
            uint16_t* p = (side ? out_k : out_q) + h * D;
            *reinterpret_cast<uint2*>(p + c0) = lo;
            *reinterpret_cast<uint2*>(p + c1) = hi;
        }
    }
}

using Kernel = void (*)(NormRopeArgs);

// The build whose lanes take `heads` heads at a time, 1 ... kMostHeads (of 6 and 8: 7 and 9)
template <bool F16, int D, bool kInterleaved>
Kernel kernel_of(int heads)
{
    if (heads == 1) return norm_rope_kernel<F16, D, kInterleaved, 1>;
    if (heads == 2) return norm_rope_kernel<F16, D, kInterleaved, 2>;
    if (heads == 3) return norm_rope_kernel<F16, D, kInterleaved, 3>;
    if (heads == 4) return norm_rope_kernel<F16, D, kInterleaved, 4>;
    if (heads == 5) return norm_rope_kernel<F16, D, kInterleaved, 5>;
    return heads <= 7 ? norm_rope_kernel<F16, D, kInterleaved, 7> : norm_rope_kernel<F16, D, kInterleaved, kMostHeads>;
}

template <bool F16, bool kInterleaved>
cudaError_t launch_type(const NormRopeArgs& a, int head_dim, int sms, cudaStream_t st)
{
    // CTAs per token: as many as leave each group of lanes one head; with many tokens as few as take at most
    // kMostHeads heads a lane, in the build that holds no more.  us for 8000 tokens, one head a lane / 3 / 4 / 5 /
    // 6 / 7 / 9: 72 heads of 128 83 / 62 / 62 / 60 / 62 / 63 / 53, 40 of 128 48 / 40 / 40 / 33 / 34 / 35 / 37, 32 of
    // 128 39 / 34 / 27 / 30 / 30 / 31 / 33, 24 of 256 62 / 46 / 46 / 51 / 39 / 40 / 42; 4000 tokens, 104 of 128
    // 60 / 46 / 43 / 44 / 45 / 41 / 44.
    const int groups = kNormThreads / (head_dim / 8), heads = a.heads[0] + a.heads[1];
    int64_t slices = ceil_div64(heads, groups);
    int each = 1;
    if (slices > 1 && a.tokens * slices > 16 * sms) {
        const int64_t all = slices;
        slices = ceil_div64(all, kMostHeads);
        each = (int)ceil_div64(all, slices);
    }
    const Kernel kernel = head_dim == 64 ? kernel_of<F16, 64, kInterleaved>(each)
                                         : (head_dim == 128 ? kernel_of<F16, 128, kInterleaved>(each) : kernel_of<F16, 256, kInterleaved>(each));
    return launch_pdl(kernel, dim3((unsigned)a.tokens, (unsigned)slices), dim3(kNormThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int head_dim, bool f16, int sms, cudaStream_t st)
{
    if (f16) return a.interleaved ? launch_type<true, true>(a, head_dim, sms, st) : launch_type<true, false>(a, head_dim, sms, st);
    return a.interleaved ? launch_type<false, true>(a, head_dim, sms, st) : launch_type<false, false>(a, head_dim, sms, st);
}

}  // namespace qli
