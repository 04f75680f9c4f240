// qli_norm_rope.cu -- norm of each query and key head and the position rotation in one pass:
//     y = x / sqrt(mean(x^2) + eps) * w,   (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)
// over the R leading elements (pairs (i, i + R/2) or (2i, 2i + 1)), fp32 throughout, rounded once.
//
// A stream over HBM: 2 bytes read and 2 written per element and a table row per token.  D / 8 lanes
// share a head vector, each with two chunks of four elements chosen so that it holds both elements
// of its pairs: in the half layout lane l < R/8 takes 4l.. and R/2 + 4l.., in the interleaved layout
// (and past R) eight consecutive elements.  So the rotation needs no exchange between lanes and
// the norm only a sum over the group.
#include <cuda_runtime.h>

#include "qli_kv.cuh"

namespace qli {

namespace {

constexpr int kNormThreads = 256;

template <bool F16, int D>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(NormRopeArgs a)
{
    constexpr int G = D / 8;                               // lanes per vector
    ptx::pdl_wait();
    const int lane = threadIdx.x & (G - 1);
    const int heads = a.heads[0] + a.heads[1];
    const int64_t vec = ((int64_t)blockIdx.x * kNormThreads + threadIdx.x) / G;
    const bool live = vec < a.tokens * heads;              // (every lane takes part in the sums)
    const int64_t t = live ? vec / heads : 0;
    int h = (int)(live ? vec - t * heads : 0);
    const int side = h >= a.heads[0] ? 1 : 0;
    if (side) h -= a.heads[0];
    // the lane's chunks [c0, c0 + 4) and [c1, c1 + 4)
    const int R = a.rotary;
    const bool rot = 8 * lane < R;
    const int c0 = (a.interleaved || !rot) ? 8 * lane : 4 * lane;
    const int c1 = (a.interleaved || !rot) ? c0 + 4 : R / 2 + 4 * lane;
    float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (live) {
        const uint16_t* x = static_cast<const uint16_t*>(a.in[side]) + t * a.in_stride[side] + (int64_t)h * D;
        const uint2 u = *reinterpret_cast<const uint2*>(x + c0), v = *reinterpret_cast<const uint2*>(x + c1);
        const uint32_t w[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = act2_to_float2<F16>(w[i]);
            y[2 * i] = f.x;
            y[2 * i + 1] = f.y;
        }
    }
    if (a.norm) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.0f / D) + a.eps);
        const uint16_t* wt = static_cast<const uint16_t*>(a.weight[side]);
        const uint2 u = *reinterpret_cast<const uint2*>(wt + c0), v = *reinterpret_cast<const uint2*>(wt + c1);
        const uint32_t w[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = act2_to_float2<F16>(w[i]);
            y[2 * i] = y[2 * i] * r * f.x;
            y[2 * i + 1] = y[2 * i + 1] * r * f.y;
        }
    }
    if (!live) return;
    const int pos = a.positions[t];
    const bool ok = pos >= 0 && pos < a.max_positions;
    if (!ok) {
        if (lane == 0 && a.err) atomicOr(a.err, kErrLength);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.0f;
    } else if (rot) {
        const float* cs = a.cos_sin + (int64_t)pos * R + 4 * lane;
        const float4 c = *reinterpret_cast<const float4*>(cs), s = *reinterpret_cast<const float4*>(cs + R / 2);
        const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float ya = a.interleaved ? y[2 * i] : y[i], yb = a.interleaved ? y[2 * i + 1] : y[i + 4];
            const float oa = ya * cv[i] - yb * sv[i], ob = yb * cv[i] + ya * sv[i];
            if (a.interleaved) {
                y[2 * i] = oa;
                y[2 * i + 1] = ob;
            } else {
                y[i] = oa;
                y[i + 4] = ob;
            }
        }
    }
    uint16_t* o = static_cast<uint16_t*>(a.out[side]) + t * a.out_stride[side] + (int64_t)h * D;
    *reinterpret_cast<uint2*>(o + c0) = make_uint2(float2_to_act2<F16>(y[0], y[1]), float2_to_act2<F16>(y[2], y[3]));
    *reinterpret_cast<uint2*>(o + c1) = make_uint2(float2_to_act2<F16>(y[4], y[5]), float2_to_act2<F16>(y[6], y[7]));
}

template <bool F16>
cudaError_t launch_type(const NormRopeArgs& a, int head_dim, cudaStream_t st)
{
    const int64_t lanes = a.tokens * (a.heads[0] + a.heads[1]) * (head_dim / 8);
    const int64_t grid = ceil_div64(lanes, kNormThreads);
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    auto kernel = head_dim == 64 ? norm_rope_kernel<F16, 64>
                                 : (head_dim == 128 ? norm_rope_kernel<F16, 128> : norm_rope_kernel<F16, 256>);
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kNormThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int head_dim, bool f16, int, cudaStream_t st)
{
    return f16 ? launch_type<true>(a, head_dim, st) : launch_type<false>(a, head_dim, st);
}

}  // namespace qli
