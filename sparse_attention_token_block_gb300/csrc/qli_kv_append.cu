// qli_kv_append.cu -- a step's new tokens in one pass: norm and position rotation of the query and key heads
// (as qli_norm_rope.cu), the queries written out, the keys and values quantised into the paged 4-bit cache (as
// qli_kv_cache.cu):
//     y = x / sqrt(mean(x^2) + eps) * w,   (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s),   K = quant(y / k_scale)
// fp32 throughout: a key is rounded once, to its code.
//
// A stream over HBM: 2 bytes read per element, 2 written per query element and 0.5625 per cached one.  A CTA
// works on one token (few tokens: several CTAs on one, by heads); D / 8 lanes share a head vector, query heads
// first, then key heads, then value heads, and each lane does kHeads vectors at a time with all their loads under way
// before the first is used, the token's places (batch, position, block_table: three dependent loads) behind
// them.  The rotation wants a lane to hold elements i and R / 2 + i, the quantiser eight consecutive ones (half
// a block): a key's vector changes hands through shared memory.
//
// 15360 tokens of 64 + 8 + 8 heads of 128: 584 MB in 118 us, 4.9 TB/s (0.73 of a copy; 65 % of the issue slots: norm, rotation and
// quantisation, no pipe above 46 %); as two calls 94.6 and 23.5 us, 118 together, the keys going out and in again in 16 bits
// between them: for many tokens the pass saves the keys' rounding to 16 bits, not time.  One token 2.5 us, as two calls 3.5; with a
// call that reads it back 4.0, a launch and three dependent loads each.
#include <cuda_runtime.h>

#include "qli_norm_rope.cuh"

namespace qli {

namespace {

constexpr int kAppendThreads = 128;

// Cosines and sines of a lane's pairs at a position
__device__ __forceinline__ void load_factors(const NormRopeArgs& a, int pos, int lane, float (&cs)[8])
{
    const float* p = a.cos_sin + (int64_t)pos * a.rotary + 4 * lane;
    const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + a.rotary / 2);
    cs[0] = x.x, cs[1] = x.y, cs[2] = x.z, cs[3] = x.w;
    cs[4] = y.x, cs[5] = y.y, cs[6] = y.z, cs[7] = y.w;
}

// kQ query vectors and kC cached ones (keys, then values) of a group of lanes under way together
template <bool F16, bool E2M1, int D, bool kInterleaved, int kQ, int kC>
__global__ void __launch_bounds__(kAppendThreads, kQ == 8 ? 6 : (kQ == 4 ? 8 : 1))
    kv_append_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ KvArgs c, const uint16_t* __restrict__ v,
                     uint8_t* __restrict__ pool)
{
    constexpr int G = D / 8, kGroups = kAppendThreads / G, kUnit = kv_unit_bytes(D);
    __shared__ __align__(16) float weight[2][D];
    __shared__ __align__(16) float turned[kGroups][D];
    ptx::pdl_wait();
    const int lane = threadIdx.x % G, group = threadIdx.x / G, R = a.rotary;
    const int64_t t = blockIdx.x;
    const int queries = a.heads[0], keys = a.heads[1], step = kGroups * gridDim.y, first = blockIdx.y * kGroups + group;
    // the lane's chunks [c0, c0 + 4) and [c1, c1 + 4) of a rotated vector; of a value's, eight elements in a row
    const bool rot = 8 * lane < R;
    const int c0 = (kInterleaved || !rot) ? 8 * lane : 4 * lane;
    const int c1 = (kInterleaved || !rot) ? c0 + 4 : R / 2 + 4 * lane;
    const uint16_t* const in_q = static_cast<const uint16_t*>(a.in[0]) + t * a.in_stride[0];
    const uint16_t* const in_k = static_cast<const uint16_t*>(a.in[1]) + t * a.in_stride[1];
    const uint16_t* const in_v = v + t * c.stride[1];
    uint16_t* const out_q = static_cast<uint16_t*>(a.out[0]) + t * a.out_stride[0];
    if (a.norm) {
        for (int i = threadIdx.x; i < D; i += kAppendThreads) {
            const int s = i >= D / 2, e = i - s * (D / 2);
            const uint32_t* w = static_cast<const uint32_t*>(a.weight[s]);
            const float2 f = w ? act2_to_float2<F16>(w[e]) : make_float2(0.0f, 0.0f);
            *reinterpret_cast<float2*>(&weight[s][2 * e]) = f;
        }
    }
    const int pos = a.positions[t], batch = c.token_batch[t], place = c.token_pos[t];
    // (one vector a group: the cached ones' groups follow the queries')
    const int first_c = kQ == 1 ? first - queries : first;
    uint2 xc[kC][2];
    auto load_cached = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kC; ++u) {
            const int i = i0 + u * step;
            xc[u][0] = xc[u][1] = make_uint2(0u, 0u);
            if (i >= 0 && i < keys) {
                xc[u][0] = *reinterpret_cast<const uint2*>(in_k + i * D + c0);
                xc[u][1] = *reinterpret_cast<const uint2*>(in_k + i * D + c1);
            } else if (i >= keys && i < 2 * keys) {
                const uint4 w = *reinterpret_cast<const uint4*>(in_v + (i - keys) * D + 8 * lane);
                xc[u][0] = make_uint2(w.x, w.y);
                xc[u][1] = make_uint2(w.z, w.w);
            }
        }
    };
    load_cached(first_c);
    const bool ok = pos >= 0 && pos < a.max_positions;
    float cs[8] = {1, 1, 1, 1, 0, 0, 0, 0};
    int64_t entry = -1;                                            // the token's place in the pool, -1: nothing is written
    auto begin = [&]() {
        if (ok && rot) load_factors(a, pos, lane, cs);
        uint32_t bits = 0;
        entry = kv_entry_offset(c.p, c.block_table, batch, place, (int64_t)c.p.max_blocks_per_seq * c.p.block_size, c.page_bytes,
                                c.entry_bytes, &bits);
        if (!ok) {
            bits |= kErrLength;
            entry = -1;
        }
        if (bits && c.err && first == 0 && lane == 0) atomicOr(c.err, bits);
        __syncthreads();                                           // the weights
    };
    // (whole groups go through the loops together; the vectors past the end are zeros that nobody stores)
    for (int h0 = first; h0 - first < queries; h0 += kQ * step) {
        uint2 x[kQ][2];
#pragma unroll
        for (int u = 0; u < kQ; ++u) {
            const int h = h0 + u * step;
            x[u][0] = x[u][1] = make_uint2(0u, 0u);
            if (h < queries) {
                x[u][0] = *reinterpret_cast<const uint2*>(in_q + h * D + c0);
                x[u][1] = *reinterpret_cast<const uint2*>(in_q + h * D + c1);
            }
        }
        if (h0 == first) begin();                                  // (behind the first loads)
        if (kQ == 1 && !__any_sync(0xffffffffu, h0 < queries)) break;
#pragma unroll
        for (int u = 0; u < kQ; ++u) {
            const int h = h0 + u * step;
            if (h0 - first + u * step >= queries) break;           // the same for every thread
            uint64_t y[2][2];
            unpack4<F16>(x[u][0], y[0]);
            unpack4<F16>(x[u][1], y[1]);
            norm_and_turn<D, kInterleaved>(y, a.norm, a.eps, &weight[0][c0], &weight[0][c1], rot, cs);
            if (h >= queries) continue;
            uint2 lo = pack4<F16>(y[0]), hi = pack4<F16>(y[1]);
            if (!ok) lo = hi = make_uint2(0u, 0u);
            *reinterpret_cast<uint2*>(out_q + h * D + c0) = lo;
            *reinterpret_cast<uint2*>(out_q + h * D + c1) = hi;
        }
    }
    if (queries == 0) begin();
    if (kQ == 1 && !__any_sync(0xffffffffu, first_c >= 0)) return;
    for (int i0 = first_c; i0 - first_c < 2 * keys; i0 += kC * step) {
        if (i0 != first_c) load_cached(i0);
#pragma unroll
        for (int u = 0; u < kC; ++u) {
            const int i = i0 + u * step, kv = i >= keys, hc = i - (kv ? keys : 0);
            if (i0 - first_c + u * step >= 2 * keys) break;          // the same for every thread
            uint64_t y[2][2];
            unpack4<F16>(xc[u][0], y[0]);
            unpack4<F16>(xc[u][1], y[1]);
            if (__any_sync(0xffffffffu, !kv)) {
                norm_and_turn<D, kInterleaved>(y, a.norm, a.eps, &weight[1][c0], &weight[1][c1], rot, cs);
                if (kv) {                                          // (values beside keys in a warp: as they came)
                    unpack4<F16>(xc[u][0], y[0]);
                    unpack4<F16>(xc[u][1], y[1]);
                }
            }
            float z[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) ptx::unpack2(y[e >> 1][e & 1], z[2 * e], z[2 * e + 1]);
            if (!kInterleaved && __any_sync(0xffffffffu, !kv)) {
                __syncwarp();                                      // (what was read of the last vector)
                *reinterpret_cast<float4*>(&turned[group][kv ? 8 * lane : c0]) = make_float4(z[0], z[1], z[2], z[3]);
                *reinterpret_cast<float4*>(&turned[group][kv ? 8 * lane + 4 : c1]) = make_float4(z[4], z[5], z[6], z[7]);
                __syncwarp();
                const float4 lo = *reinterpret_cast<const float4*>(&turned[group][8 * lane]);
                const float4 hi = *reinterpret_cast<const float4*>(&turned[group][8 * lane + 4]);
                z[0] = lo.x, z[1] = lo.y, z[2] = lo.z, z[3] = lo.w;
                z[4] = hi.x, z[5] = hi.y, z[6] = hi.z, z[7] = hi.w;
            }
            float amax = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(z[e]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            divide_by_factor<E2M1>(z, amax, kv ? c.scale[1] : c.scale[0], kv ? c.inverse[1] : c.inverse[0]);
            uint32_t scale;
            const uint32_t code = quantize8<E2M1>(z, amax, scale);
            if (i >= 0 && i < 2 * keys && entry >= 0) {
                uint8_t* dst = pool + entry + hc * kUnit;
                *reinterpret_cast<uint32_t*>(dst + kv * (D / 2) + 4 * lane) = code;
                if (!(lane & 1)) dst[D + kv * (D / kKvBlock) + lane / 2] = (uint8_t)scale;
            }
        }
    }
}

using Kernel = void (*)(NormRopeArgs, KvArgs, const uint16_t*, uint8_t*);

template <bool F16, bool E2M1, int D>
Kernel kernel_of(bool interleaved, int each)
{
    if (each == 1) return interleaved ? kv_append_kernel<F16, E2M1, D, true, 1, 1> : kv_append_kernel<F16, E2M1, D, false, 1, 1>;
    if (each == 4) return interleaved ? kv_append_kernel<F16, E2M1, D, true, 4, 1> : kv_append_kernel<F16, E2M1, D, false, 4, 1>;
    return interleaved ? kv_append_kernel<F16, E2M1, D, true, 8, 2> : kv_append_kernel<F16, E2M1, D, false, 8, 2>;
}

template <bool F16, bool E2M1>
cudaError_t launch_type(const NormRopeArgs& a, const KvArgs& c, const void* v, void* kv, int sms, cudaStream_t st)
{
    const int groups = kAppendThreads / (c.head_dim / 8);
    // CTAs per token: as many as leave each group of lanes one vector; with many tokens one that takes them in turn, four
    // or eight query vectors at a time.  15360 tokens (written and read back), us for 5 of any kind / 4 queries and a cached
    // vector / 8 and 2: 64 + 8 + 8 heads of 128 160 / 144 / 136, 28 + 4 + 4 83 / 73 / 89.
    int64_t slices = ceil_div64(a.heads[0] + 2 * a.heads[1], groups);
    int each = 1;
    if (slices > 1 && a.tokens * slices > 16 * sms) {
        each = ceil_div64(a.heads[0], groups) > 4 ? 8 : 4;
        slices = ceil_div64(a.heads[0] > 2 * a.heads[1] ? a.heads[0] : 2 * a.heads[1], groups * each);
    }
    const Kernel kernel = c.head_dim == 64 ? kernel_of<F16, E2M1, 64>(a.interleaved, each) : kernel_of<F16, E2M1, 128>(a.interleaved, each);
    return launch_pdl(kernel, dim3((unsigned)a.tokens, (unsigned)slices), dim3(kAppendThreads), 0, st, a, c,
                      static_cast<const uint16_t*>(v), static_cast<uint8_t*>(kv));
}

}  // namespace

cudaError_t launch_kv_append(const NormRopeArgs& a, const KvArgs& c, const void* v, void* kv, int sms, cudaStream_t st)
{
    if (c.f16) return c.e2m1 ? launch_type<true, true>(a, c, v, kv, sms, st) : launch_type<true, false>(a, c, v, kv, sms, st);
    return c.e2m1 ? launch_type<false, true>(a, c, v, kv, sms, st) : launch_type<false, false>(a, c, v, kv, sms, st);
}

}  // namespace qli
