// qli_kv_cache.cu -- the paged KV cache in 4 bits: quantising keys and values as they are written
// through the block_table, and reading them back.
//
// Per block of 16 elements:  y = x / g (g = k_scale or v_scale);  s = e4m3(min(max |y| / Q, 448)),
// Q = 7 (int4) or 6 (E2M1);  code = y / s in fp32 rounded to nearest even and saturated to +-Q.
//
// Streams over HBM: 2 bytes per element on the activations' side and 0.5625 on the cache's.  A thread
// holds half a block, eight elements: 16 bytes of activations and 4 of codes, so every load and store
// of a warp is one contiguous range of a token (a whole block per thread wrote 16 bytes at a stride of
// 32), and a block's maximum takes one exchange with the neighbouring lane.  A token's half-blocks (K
// heads, then V heads) follow one another over the threads.  A CTA looks up the entries of up to
// kMaxTokens tokens first (batch, position, block_table, pool are four dependent loads; one lookup per
// four tokens left the read of 65536 tokens at 89 us), then each thread streams its half-block of
// those tokens, kUnroll at a time.  Measured on a GB300, 8 KV heads of 128, E2M1: reading 65536 tokens
// (344 MB) 61.7 us = 5.6 TB/s, 0.82 of a copy's rate; writing 15360 tokens (81 MB) and reading them back 36
// us (the write is bound by its 118 instructions per eight elements at 42 % occupancy, and by its
// length: five CTAs per SM instead of four, or two or eight tokens under way, change nothing).
#include <cuda_runtime.h>

#include <cfloat>

#include "qli_kv.cuh"

namespace qli {

namespace {

constexpr int kKvThreads = 256;
constexpr int kMaxTokens = 32;             // tokens of a CTA
constexpr int kUnroll = 4;                 // half-blocks of a thread under way

// Half-block i of a token: byte offsets in the entry, element offset in K or V
struct HalfPos {
    int kv;                                // 0: K, 1: V
    int element, code, scale;
};
__device__ __forceinline__ HalfPos half_pos(int i, int heads, int dim)
{
    const int per = dim / 8;               // half-blocks of a vector
    HalfPos r;
    r.kv = i >= heads * per ? 1 : 0;
    i -= r.kv * heads * per;
    const int h = i / per, x = i - h * per, unit = kv_unit_bytes(dim);
    r.element = 8 * i;
    r.code = h * unit + r.kv * (dim / 2) + 4 * x;
    r.scale = h * unit + dim + r.kv * (dim / kKvBlock) + x / 2;
    return r;
}

// The entries of the CTA's n tokens from t0 on: byte offsets into the pool, -1 for invalid tokens (with
// the error bit)
__device__ __forceinline__ void find_entries(const KvArgs& a, int64_t t0, int n, int64_t* entry)
{
    if (threadIdx.x < n) {
        uint32_t bits = 0;
        const int64_t t = t0 + threadIdx.x;
        entry[threadIdx.x] = kv_entry_offset(a.p, a.block_table, a.token_batch[t], a.token_pos[t],
                                             (int64_t)a.p.max_blocks_per_seq * a.p.block_size, a.page_bytes,
                                             a.entry_bytes, &bits);
        if (bits && a.err) atomicOr(a.err, bits);
    }
}

// y <- y / d for eight elements whose largest quotient is `top`: a reciprocal and remainder corrections
// where they give the correctly rounded quotient, else divisions.  The corrections can lose the sign
// of a zero quotient; kSign keeps it.
template <bool kSign>
__device__ __forceinline__ void divide8(float (&y)[8], float d, float top)
{
    if (top <= FLT_MAX && ptx::reciprocal_ok(d)) {
        const float r = __frcp_rn(d);
        const uint64_t R = ptx::pack2(r, r), NS = ptx::pack2(-d, -d);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float lo, hi;
            ptx::unpack2(ptx::quotient2(ptx::pack2(y[i], y[i + 1]), R, NS), lo, hi);
            y[i] = kSign ? copysignf(lo, y[i]) : lo;
            y[i + 1] = kSign ? copysignf(hi, y[i + 1]) : hi;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(y[i], d);
    }
}

// The correctly rounded quotients y / d of a finite y and a d of at most four significant bits (a scale,
// 6 or 7), from r within an ulp of 1 / d: q = RN(y r) is within two ulps of y / d, its remainder
// y - q d is exact in a fused multiply-add, and q + (y - q d) r lies within 2^-21 ulp of y / d.
// Rounded, that is the quotient rounded: y / d is no midpoint of two fp32 numbers (a 25-bit number
// times d has more bits than y) and no nearer to one than 2^-5 ulp.  Quotients below 2^-126 may
// differ, but give code 0 and scale 0 either way.
__device__ __forceinline__ uint64_t short_quotient2(uint64_t Y, uint64_t R, uint64_t ND)
{
    const uint64_t Q = ptx::mul2(Y, R);
    return ptx::fma2(ptx::fma2(Q, ND, Y), R, Q);
}

// Codes of eight elements y and the scale byte of their block, whose largest magnitude is amax
template <bool E2M1>
__device__ __forceinline__ uint32_t quantize8(const float (&y)[8], float amax, uint32_t& scale)
{
    constexpr float kTop = E2M1 ? 6.0f : 7.0f, kTopInv = 1.0f / kTop;
    if (!(amax <= FLT_MAX)) {                          // y = x / g overflowed: the largest scale, codes +-Q or 0
        scale = 0x7E;
        uint32_t code = 0;
        for (int i = 0; i < 8; ++i) {
            const float q = fminf(fmaxf(__fdiv_rn(y[i], 448.0f), -kTop), kTop);
            uint32_t c = (uint32_t)__float2int_rn(q) & 15u;
            if (E2M1) {
                asm("{\n\t.reg .b8 d;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %1, %2;\n\tmov.b32 %0, {d, 0, 0, 0};\n\t}"
                    : "=r"(c)
                    : "f"(0.0f), "f"(q));
                c &= 15u;
            }
            code |= c << (4 * i);
        }
        return code;
    }
    float s, dummy;
    ptx::unpack2(short_quotient2(ptx::pack2(amax, 0.0f), ptx::pack2(kTopInv, kTopInv), ptx::pack2(-kTop, -kTop)), s, dummy);
    scale = float_to_e4m3(fminf(s, 448.0f));
    s = e4m3_to_float(scale);
    if (s == 0.0f) return 0u;
    const float r = ptx::rcp_approx(s);
    const uint64_t R = ptx::pack2(r, r), NS = ptx::pack2(-s, -s);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) ptx::unpack2(short_quotient2(ptx::pack2(y[i], y[i + 1]), R, NS), q[i], q[i + 1]);
    uint32_t code = 0;
    if (E2M1) {
        uint32_t byte[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // (the correction can lose the sign of a zero quotient, which the code keeps)
            const float lo = copysignf(q[2 * i], y[2 * i]), hi = copysignf(q[2 * i + 1], y[2 * i + 1]);
            asm("{\n\t.reg .b8 d;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %1, %2;\n\tmov.b32 %0, {d, 0, 0, 0};\n\t}"
                : "=r"(byte[i])
                : "f"(hi), "f"(lo));
        }
        code = __byte_perm(__byte_perm(byte[0], byte[1], 0x0040), __byte_perm(byte[2], byte[3], 0x0040), 0x5410);
    } else {
        // q + 1.5 * 2^23 rounds q to an integer (ties to even), whose two's complement ends the sum's bits
#pragma unroll
        for (int i = 0; i < 8; ++i)
            code |= (__float_as_uint(fminf(fmaxf(q[i], -7.0f), 7.0f) + 12582912.0f) & 15u) << (4 * i);
    }
    return code;
}

template <bool F16, bool E2M1>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(KvArgs a, const uint16_t* __restrict__ k,
                                                              const uint16_t* __restrict__ v, uint8_t* __restrict__ pool,
                                                              int slots, int tokens)
{
    __shared__ int64_t entry[kMaxTokens];
    ptx::pdl_wait();
    const int halves = 2 * a.heads_kv * (a.head_dim / 8);
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)min((int64_t)tokens, a.tokens - t0);
    const int covered = slots * halves;
    for (int base = 0; base < covered; base += kKvThreads) {
        // (threads past the end follow along with nothing to load or store: whole warps take part in the exchange)
        const int i = min(base + (int)threadIdx.x, covered - 1), slot = i / halves, ih = i - slot * halves;
        const bool live = base + (int)threadIdx.x < covered;
        const HalfPos w = half_pos(ih, a.heads_kv, a.head_dim);
        const int64_t stride = a.stride[w.kv];
        const uint16_t* src = (w.kv ? v : k) + w.element + t0 * stride;
        const float g = w.kv ? a.scale[1] : a.scale[0], gi = w.kv ? a.inverse[1] : a.inverse[0];
        for (int l0 = 0; l0 < n; l0 += kUnroll * slots) {
            uint4 x[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int l = l0 + slot + u * slots;
                x[u] = make_uint4(0u, 0u, 0u, 0u);
                if (live && l < n) x[u] = __ldcs(reinterpret_cast<const uint4*>(src + l * stride));
            }
            if (base == 0 && l0 == 0) {                                // (behind the first loads)
                find_entries(a, t0, n, entry);
                __syncthreads();
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (l0 + u * slots >= n) break;                        // the same for every thread
                const int l = l0 + slot + u * slots;
                const uint32_t word[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                float y[8], amax = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = act2_to_float2<F16>(word[j]);
                    y[2 * j] = f.x;
                    y[2 * j + 1] = f.y;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(y[j]));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                if (gi != 0.0f) {
                    // a power of two: the product with its reciprocal is the quotient
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] *= gi;
                    amax *= gi;
                } else {
                    // (the division is monotone: the largest quotient is the largest magnitude's)
                    amax = __fdiv_rn(amax, g);
                    divide8<E2M1>(y, g, amax);
                }
                uint32_t scale;
                const uint32_t code = quantize8<E2M1>(y, amax, scale);
                const int64_t at = live && l < n ? entry[l] : -1;
                if (at >= 0) {
                    *reinterpret_cast<uint32_t*>(pool + at + w.code) = code;
                    if (!(ih & 1)) pool[at + w.scale] = (uint8_t)scale;
                }
            }
        }
    }
}

template <bool F16, bool E2M1>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(KvArgs a, const uint8_t* __restrict__ pool,
                                                             uint16_t* __restrict__ k, uint16_t* __restrict__ v, int slots,
                                                             int tokens)
{
    __shared__ int64_t entry[kMaxTokens];
    ptx::pdl_wait();
    const int halves = 2 * a.heads_kv * (a.head_dim / 8);
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)min((int64_t)tokens, a.tokens - t0);
    find_entries(a, t0, n, entry);
    __syncthreads();
    for (int i = threadIdx.x; i < slots * halves; i += kKvThreads) {
        const int slot = i / halves, ih = i - slot * halves;
        const HalfPos w = half_pos(ih, a.heads_kv, a.head_dim);
        const int64_t stride = a.stride[w.kv];
        uint16_t* dst = (w.kv ? v : k) + w.element + t0 * stride;
        const float g = w.kv ? a.scale[1] : a.scale[0];
        for (int l0 = slot; l0 < n; l0 += kUnroll * slots) {
            uint32_t code[kUnroll], scale[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int l = l0 + u * slots;
                const int64_t at = l < n ? entry[l] : -1;
                code[u] = at >= 0 ? *reinterpret_cast<const uint32_t*>(pool + at + w.code) : 0u;
                scale[u] = at >= 0 ? pool[at + w.scale] : 0u;             // (an invalid token: zeros times zero)
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int l = l0 + u * slots;
                if (l >= n) break;
                const float s = e4m3_to_float(scale[u]);
                float f[8];
                decode8<E2M1>(code[u], f);
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = float2_to_act2<F16>(f[2 * e] * s * g, f[2 * e + 1] * s * g);
                __stcs(reinterpret_cast<uint4*>(dst + l * stride), make_uint4(o[0], o[1], o[2], o[3]));
            }
        }
    }
}

// Token slots that a CTA's threads cover at once, and the tokens of a CTA: up to kMaxTokens while about
// eight CTAs per SM remain
struct Split {
    int slots, tokens;
};
Split split_of(const KvArgs& a, int sms)
{
    const int halves = 2 * a.heads_kv * (a.head_dim / 8);
    Split s;
    s.slots = halves >= kKvThreads ? 1 : kKvThreads / halves;
    if (s.slots > kMaxTokens) s.slots = kMaxTokens;
    const int64_t per = ceil_div64(a.tokens, 8 * sms);
    s.tokens = per < s.slots ? s.slots : (per > kMaxTokens ? kMaxTokens : (int)per);
    return s;
}

}  // namespace

cudaError_t launch_kv_write(const KvArgs& a, int sms, const void* k, const void* v, void* kv, cudaStream_t st)
{
    const Split s = split_of(a, sms);
    auto kernel = a.f16 ? (a.e2m1 ? kv_write_kernel<true, true> : kv_write_kernel<true, false>)
                        : (a.e2m1 ? kv_write_kernel<false, true> : kv_write_kernel<false, false>);
    return launch_pdl(kernel, dim3((unsigned)ceil_div64(a.tokens, s.tokens)), dim3(kKvThreads), 0, st, a,
                      static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), static_cast<uint8_t*>(kv), s.slots, s.tokens);
}

cudaError_t launch_kv_read(const KvArgs& a, int sms, const void* kv, void* k, void* v, cudaStream_t st)
{
    const Split s = split_of(a, sms);
    auto kernel = a.f16 ? (a.e2m1 ? kv_read_kernel<true, true> : kv_read_kernel<true, false>)
                        : (a.e2m1 ? kv_read_kernel<false, true> : kv_read_kernel<false, false>);
    return launch_pdl(kernel, dim3((unsigned)ceil_div64(a.tokens, s.tokens)), dim3(kKvThreads), 0, st, a,
                      static_cast<const uint8_t*>(kv), static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), s.slots, s.tokens);
}

}  // namespace qli
