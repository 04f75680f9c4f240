// qli_norm_rope.cuh -- norm and rotation of a vector that D / 8 lanes share, and its activations in pairs.
#pragma once

#include "qli_kv.cuh"

namespace qli {

// Four activations in two words as two packed pairs
template <bool F16>
__device__ __forceinline__ void unpack4(const uint2& u, uint64_t (&y)[2])
{
    const float2 a = act2_to_float2<F16>(u.x), b = act2_to_float2<F16>(u.y);
    y[0] = ptx::pack2(a.x, a.y);
    y[1] = ptx::pack2(b.x, b.y);
}

template <bool F16>
__device__ __forceinline__ uint2 pack4(const uint64_t (&y)[2])
{
    float a, b, c, d;
    ptx::unpack2(y[0], a, b);
    ptx::unpack2(y[1], c, d);
    return make_uint2(float2_to_act2<F16>(a, b), float2_to_act2<F16>(c, d));
}

// Two chunks of four elements of a vector of D, y[0] and y[1] (in pairs), normalised (weights at w0 and w1) and
// turned by the factors cs (four cosines, four sines).  The D / 8 lanes of the vector call it together.  A
// rotating lane's chunks hold both elements of its pairs: half layout, elements i and R / 2 + i in one chunk
// each; interleaved, neighbours.
template <int D, bool kInterleaved>
__device__ __forceinline__ void norm_and_turn(uint64_t (&y)[2][2], bool norm, float eps, const float* w0, const float* w1,
                                              bool rot, const float (&cs)[8])
{
    constexpr int G = D / 8;
    if (norm) {
        uint64_t sq = ptx::mul2(y[0][0], y[0][0]);
        sq = ptx::fma2(y[0][1], y[0][1], sq);
        sq = ptx::fma2(y[1][0], y[1][0], sq);
        sq = ptx::fma2(y[1][1], y[1][1], sq);
        float ss, odd;
        ptx::unpack2(sq, ss, odd);
        ss += odd;
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.0f / D) + eps);
        const uint64_t rr = ptx::pack2(r, r);
        const float4 g0 = *reinterpret_cast<const float4*>(w0);
        const float4 g1 = *reinterpret_cast<const float4*>(w1);
        y[0][0] = ptx::mul2(ptx::mul2(y[0][0], rr), ptx::pack2(g0.x, g0.y));
        y[0][1] = ptx::mul2(ptx::mul2(y[0][1], rr), ptx::pack2(g0.z, g0.w));
        y[1][0] = ptx::mul2(ptx::mul2(y[1][0], rr), ptx::pack2(g1.x, g1.y));
        y[1][1] = ptx::mul2(ptx::mul2(y[1][1], rr), ptx::pack2(g1.z, g1.w));
    }
    if (rot) {
        if (kInterleaved) {
            // a pair of elements is a pair of the rotation
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float ya, yb;
                ptx::unpack2(y[i >> 1][i & 1], ya, yb);
                y[i >> 1][i & 1] = ptx::pack2(ya * cs[i] - yb * cs[4 + i], yb * cs[i] + ya * cs[4 + i]);
            }
        } else {
            // the first chunk's elements turn with the second's
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint64_t c = ptx::pack2(cs[2 * i], cs[2 * i + 1]), s = ptx::pack2(cs[4 + 2 * i], cs[5 + 2 * i]);
                const uint64_t ns = ptx::pack2(-cs[4 + 2 * i], -cs[5 + 2 * i]), ya = y[0][i], yb = y[1][i];
                y[0][i] = ptx::fma2(ya, c, ptx::mul2(yb, ns));
                y[1][i] = ptx::fma2(yb, c, ptx::mul2(ya, s));
            }
        }
    }
}

}  // namespace qli
