// qli_kv_cache.cu -- the paged KV cache in 4 bits: quantising keys and values as they are written
// through the block_table, and reading them back.
//
// Per block of 16 elements:  y = x / g (g = k_scale or v_scale);  s = e4m3(min(max |y| / Q, 448)),
// Q = 7 (int4) or 6 (E2M1);  code = y / s in fp32 rounded to nearest even and saturated to +-Q.
//
// Streams over HBM: 2 bytes per element on the activations' side and 0.5625 on the cache's.  One
// thread per block of 16 elements: its maximum needs no exchange between lanes, and a token's
// blocks (K heads, then V heads) follow one another over the threads, so both sides coalesce.
#include <cuda_runtime.h>

#include "qli_kv.cuh"

namespace qli {

namespace {

constexpr int kKvThreads = 256;

// Block i of a token: K or V (kv), head h, block b of D / 16
struct BlockPos {
    int kv, h, b;
};
__device__ __forceinline__ BlockPos block_pos(int i, int heads, int nb)
{
    BlockPos r;
    r.kv = i >= heads * nb ? 1 : 0;
    i -= r.kv * heads * nb;
    r.h = i / nb;
    r.b = i - r.h * nb;
    return r;
}

// The entry of token t: byte offset into the pool, or -1 with the error bit set (once per token)
__device__ __forceinline__ int64_t token_entry(const KvArgs& a, int64_t t, bool report)
{
    uint32_t bits = 0;
    const int64_t off = kv_entry_offset(a.p, a.block_table, a.token_batch[t], a.token_pos[t],
                                        (int64_t)a.p.max_blocks_per_seq * a.p.block_size, a.page_bytes, a.entry_bytes, &bits);
    if (bits && report && a.err) atomicOr(a.err, bits);
    return off;
}

template <bool F16, bool E2M1>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(KvArgs a, const uint16_t* __restrict__ k,
                                                              const uint16_t* __restrict__ v, uint8_t* __restrict__ pool,
                                                              int tokens_per_cta)
{
    ptx::pdl_wait();
    const int nb = a.head_dim / kKvBlock, blocks = 2 * a.heads_kv * nb, unit = kv_unit_bytes(a.head_dim);
    constexpr float kTop = E2M1 ? 6.0f : 7.0f;
    for (int i = threadIdx.x; i < tokens_per_cta * blocks; i += kKvThreads) {
        const int tl = i / blocks, ib = i - tl * blocks;
        const int64_t t = (int64_t)blockIdx.x * tokens_per_cta + tl;
        if (t >= a.tokens) break;
        const int64_t entry = token_entry(a, t, ib == 0);
        if (entry < 0) continue;
        const BlockPos w = block_pos(ib, a.heads_kv, nb);
        const uint4* src = reinterpret_cast<const uint4*>((w.kv ? v : k) + t * a.stride[w.kv] +
                                                          (int64_t)w.h * a.head_dim + w.b * kKvBlock);
        const uint4 u0 = src[0], u1 = src[1];
        const uint32_t x[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
        const float g = w.kv ? a.v_scale : a.k_scale;
        float y[16], amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 f = act2_to_float2<F16>(x[j]);
            y[2 * j] = __fdiv_rn(f.x, g);
            y[2 * j + 1] = __fdiv_rn(f.y, g);
            amax = fmaxf(amax, fmaxf(fabsf(y[2 * j]), fabsf(y[2 * j + 1])));
        }
        const uint32_t sb = float_to_e4m3(fminf(__fdiv_rn(amax, kTop), 448.0f));
        const float s = e4m3_to_float(sb);
        uint32_t code[2] = {0u, 0u};
        if (s > 0.0f) {
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const float q0 = __fdiv_rn(y[j], s), q1 = __fdiv_rn(y[j + 1], s);
                uint32_t byte;
                if (E2M1) {
                    asm("{\n\t.reg .b8 d;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %1, %2;\n\t"
                        "mov.b32 %0, {d, 0, 0, 0};\n\t}"
                        : "=r"(byte)
                        : "f"(q1), "f"(q0));
                } else {
                    const int c0 = __float2int_rn(fminf(fmaxf(q0, -7.0f), 7.0f));
                    const int c1 = __float2int_rn(fminf(fmaxf(q1, -7.0f), 7.0f));
                    byte = (c0 & 15) | ((c1 & 15) << 4);
                }
                code[j >> 3] |= byte << ((j & 7) * 4);
            }
        }
        uint8_t* dst = pool + entry + w.h * unit;
        *reinterpret_cast<uint2*>(dst + w.kv * (a.head_dim / 2) + w.b * 8) = make_uint2(code[0], code[1]);
        dst[a.head_dim + w.kv * nb + w.b] = (uint8_t)sb;
    }
}

template <bool F16, bool E2M1>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(KvArgs a, const uint8_t* __restrict__ pool,
                                                             uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                                                             int tokens_per_cta)
{
    ptx::pdl_wait();
    const int nb = a.head_dim / kKvBlock, blocks = 2 * a.heads_kv * nb, unit = kv_unit_bytes(a.head_dim);
    for (int i = threadIdx.x; i < tokens_per_cta * blocks; i += kKvThreads) {
        const int tl = i / blocks, ib = i - tl * blocks;
        const int64_t t = (int64_t)blockIdx.x * tokens_per_cta + tl;
        if (t >= a.tokens) break;
        const int64_t entry = token_entry(a, t, ib == 0);
        const BlockPos w = block_pos(ib, a.heads_kv, nb);
        uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (entry >= 0) {
            const uint8_t* src = pool + entry + w.h * unit;
            const uint2 c = *reinterpret_cast<const uint2*>(src + w.kv * (a.head_dim / 2) + w.b * 8);
            const float s = e4m3_to_float(src[a.head_dim + w.kv * nb + w.b]), g = w.kv ? a.v_scale : a.k_scale;
            float f[8];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                decode8<E2M1>(j ? c.y : c.x, f);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[4 * j + e] = float2_to_act2<F16>(f[2 * e] * s * g, f[2 * e + 1] * s * g);
            }
        }
        uint4* dst = reinterpret_cast<uint4*>((w.kv ? v : k) + t * a.stride[w.kv] + (int64_t)w.h * a.head_dim +
                                              w.b * kKvBlock);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

int tokens_per_cta(const KvArgs& a)
{
    const int blocks = 2 * a.heads_kv * (a.head_dim / kKvBlock);
    return blocks >= kKvThreads ? 1 : kKvThreads / blocks;
}

}  // namespace

cudaError_t launch_kv_write(const KvArgs& a, const void* k, const void* v, void* kv, cudaStream_t st)
{
    const int tpc = tokens_per_cta(a);
    auto kernel = a.f16 ? (a.e2m1 ? kv_write_kernel<true, true> : kv_write_kernel<true, false>)
                        : (a.e2m1 ? kv_write_kernel<false, true> : kv_write_kernel<false, false>);
    return launch_pdl(kernel, dim3((unsigned)ceil_div64(a.tokens, tpc)), dim3(kKvThreads), 0, st, a,
                      static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), static_cast<uint8_t*>(kv), tpc);
}

cudaError_t launch_kv_read(const KvArgs& a, const void* kv, void* k, void* v, cudaStream_t st)
{
    const int tpc = tokens_per_cta(a);
    auto kernel = a.f16 ? (a.e2m1 ? kv_read_kernel<true, true> : kv_read_kernel<true, false>)
                        : (a.e2m1 ? kv_read_kernel<false, true> : kv_read_kernel<false, false>);
    return launch_pdl(kernel, dim3((unsigned)ceil_div64(a.tokens, tpc)), dim3(kKvThreads), 0, st, a,
                      static_cast<const uint8_t*>(kv), static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), tpc);
}

}  // namespace qli
