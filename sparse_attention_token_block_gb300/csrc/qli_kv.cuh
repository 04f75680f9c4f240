// qli_kv.cuh -- the 4-bit codes of the KV cache: quantising one block of 16 elements, decoding codes
// and scales, and finding an entry through the block_table.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qli_internal.cuh"
#include "qli_ptx.cuh"

namespace qli {

// Two activations packed in a word -> fp32 (exact), and back (rounded to nearest even)
template <bool F16>
__device__ __forceinline__ float2 act2_to_float2(uint32_t w)
{
    if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <bool F16>
__device__ __forceinline__ uint32_t float2_to_act2(float lo, float hi)
{
    if (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// What the rounding of lo and hi to the fp16 pair p left, rounded to fp16
__device__ __forceinline__ uint32_t remainder_f16x2(float lo, float hi, uint32_t p)
{
    const float2 r = act2_to_float2<true>(p);
    float x, y;
    ptx::unpack2(ptx::fma2(ptx::pack2(r.x, r.y), ptx::pack2(-1.0f, -1.0f), ptx::pack2(lo, hi)), x, y);
    return float2_to_act2<true>(x, y);
}

// Two scale bytes as fp16 (exact), the low byte in the low half
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t bytes)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(bytes)));
    return h;
}

// A scale byte (float8_e4m3fn) as fp32, and the scale of a block: e4m3(min(a, 448)) as a byte
__device__ __forceinline__ float e4m3_to_float(uint32_t byte)
{
    return __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(byte) & 0xFFFFu)));
}

__device__ __forceinline__ uint32_t float_to_e4m3(float a)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(a));
    return r & 0xFFu;
}

// Eight E2M1 codes in a word -> f16x2 words of elements (0, 1), (2, 3), (4, 5), (6, 7) (exact)
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&o)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}

// Code c of a word as fp32
template <bool E2M1>
__device__ __forceinline__ void decode8(uint32_t w, float (&v)[8])
{
    if (E2M1) {
        uint32_t h[4];
        e2m1x8_to_f16x2(w, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)((int32_t)(w << (28 - 4 * i)) >> 28);
    }
}

// Scales of two elements as fp16, prepared for the codes they multiply.  An int4 nibble u = code + 8 is
// placed at bits 4-7 of the fp16 number x = 1024 + 16 u, so code * s = x * (s / 16) - 72 s, one fused
// multiply-add.  All of it is exact: s has at most four significant bits, 72 s at most eight, the result
// at most seven, and the smallest numbers (2^-13) are normal or multiples of fp16's spacing.
struct PairScale {
    uint32_t mul, add;
};
template <bool E2M1>
__device__ __forceinline__ PairScale pair_scale(uint32_t s)
{
    if (E2M1) return {s, 0u};
    return {ptx::mul_f16x2(s, 0x2C002C00u), ptx::mul_f16x2(s, 0xD480D480u)};        // s / 16, -72 s
}

// Eight codes of one vector in a word, times their scale, as four fp16 pairs, exactly: E2M1 elements
// (2i, 2i + 1), int4 elements (i, i + 4)
template <bool E2M1>
__device__ __forceinline__ void decode_pairs(uint32_t w, const PairScale& s, uint32_t (&o)[4])
{
    if (E2M1) {
        e2m1x8_to_f16x2(w, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = ptx::mul_f16x2(o[i], s.mul);
        return;
    }
    const uint32_t at[4] = {w << 4, w, w >> 4, w >> 8};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // (w & 0xF0) with its top bit flipped (u = code + 8), under the exponent of 1024
        const uint32_t x = (at[i] & 0x00F000F0u) ^ 0x64806480u;
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(o[i]) : "r"(x), "r"(s.mul), "r"(s.add));
    }
}

// The low nibble of every byte of a, the high nibble of every byte of b (one instruction)
__device__ __forceinline__ uint32_t select_low_nibbles(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, 0x0F0F0F0F, 0xE4;" : "=r"(r) : "r"(a), "r"(b));        // (a & c) | (b & ~c)
    return r;
}

// Eight codes each of two vectors, times their scales (s: a's, b's), as eight fp16 pairs (a's element e,
// b's element e), exactly
template <bool E2M1>
__device__ __forceinline__ void decode_across(uint32_t a, uint32_t b, const PairScale& s, uint32_t (&o)[8])
{
    uint32_t x[4], y[4];
    if (E2M1) {
        // bytes of (a's nibble, b's nibble) for the even and the odd elements
        const uint32_t even = select_low_nibbles(a, b << 4), odd = select_low_nibbles(a >> 4, b);
        decode_pairs<true>(even, s, x);
        decode_pairs<true>(odd, s, y);
    } else {
        // elements 0-3 of both in one word, 4-7 in another
        decode_pairs<false>(__byte_perm(a, b, 0x5410), s, x);
        decode_pairs<false>(__byte_perm(a, b, 0x7632), s, y);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[E2M1 ? 2 * i : i] = x[i];
        o[E2M1 ? 2 * i + 1 : 4 + i] = y[i];
    }
}

// Byte offset of compressed position `pos` of batch `b` in the pool, -1 when the batch, the
// position (against `limit`) or the page is invalid (with the error bit)
__device__ __forceinline__ int64_t kv_entry_offset(const Params& p, const int32_t* block_table, int64_t b, int64_t pos,
                                                   int64_t limit, int64_t page_bytes, int64_t entry_bytes,
                                                   uint32_t* bits)
{
    if (b < 0 || b >= p.batch || pos < 0 || pos >= limit) {
        *bits |= kErrLength;
        return -1;
    }
    const uint32_t bs = (uint32_t)p.block_size, block = (uint32_t)pos / bs;       // pos < 2^31
    const int64_t page = block_table[b * p.max_blocks_per_seq + block];
    if (page < 0 || page >= p.num_blocks) {
        *bits |= kErrPage;
        return -1;
    }
    return page * page_bytes + (int64_t)((uint32_t)pos - block * bs) * entry_bytes;
}

// Tensor map (a CUtensorMap) of a paged pool: 8-byte elements, boxes of `box_entries` entries of a page, `box_bytes`
// wide
bool encode_page_map(void* tmap, const void* pool, int64_t entry_bytes, int block_size, int64_t page_bytes, int num_blocks,
                     int box_bytes, int box_entries);

// Sparse attention over blocks of neighbouring rows (qli_attention_rows.cu): whether it suits a call, and
// its launch
bool attention_in_rows(const AttentionArgs& a, int head_dim, int sms);
cudaError_t launch_attention_rows(const AttentionArgs& a, bool f16, bool e2m1, int sms, cudaStream_t st);
// How that launch is laid out: rows of a block, KV heads of a CTA, positions of a mask
struct RowsShape {
    int32_t rows, heads, positions;
};
RowsShape attention_rows_shape(const AttentionArgs& a, int sms);

}  // namespace qli
