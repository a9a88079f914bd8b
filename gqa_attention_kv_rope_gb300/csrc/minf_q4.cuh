// minf_q4.cuh -- Q4 block arithmetic shared by the store, read and attention kernels.
//
// A Q4 block is 32 consecutive values of a row, kept as one binary16 scale and 32 codes of 4 bits.  With m the
// value of largest magnitude (the positive one of two), the store takes d = m / -8 rounded to 8 significant bits
// (bfloat16, then binary16), q = round(x * (1/d)) within -8 .. 7 (halves away from zero; d = 0 gives q = 0) and the
// code u = q + 8; a value reads back as d * q.  The scale is m / -8, not max|x| / 7, so that all sixteen codes are
// used and m itself reads back to 2^-9.
//
// d has 8 significant bits and q at most 3 (or is -8), so every value is exactly a binary16 number: the attention's
// products take it as one tensor-core operand, where a Q8_0 value needs two halves, and a read back to binary16 loses
// nothing.  A full binary16 scale would change a value by 2^-9 of itself at most, against the quantisation's 2^-4 of
// the block's largest.  Blocks that hold a NaN, an infinity or a magnitude of 65408 and more (d would be 8192, and -8 d
// not a binary16 number) get the scale NaN: they read back as NaN.
//
// Row layout: the codes, W/2 bytes, each 8 values a 32-bit word; then the W/32 scales, then zeros to a multiple of 16
// bytes.  In a word nibble i < 4 is value 2i and nibble 4 + i value 2i + 1: the word and its shifts by 4, 8 and 12 hold
// the pairs of neighbours in the low nibbles of their halves, where one mask leaves a pair for a half2.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "minf_common.cuh"

namespace minf {

struct Q4 {};  // storage tag: Q4 rows

// What a block's scale follows from: the largest magnitude in the upper 31 bits (infinities and NaN above every
// number), and whether it is positive; of several values' keys the largest is the block's.
__device__ __forceinline__ uint32_t q4_key(float x) {
    const uint32_t b = __float_as_uint(x);
    return (b << 1) | ((b >> 31) ^ 1u);
}
__device__ __forceinline__ uint32_t q4_key4(float4 x) { return max(max(q4_key(x.x), q4_key(x.y)), max(q4_key(x.z), q4_key(x.w))); }

// The scale of a block with this key, and r = 1/d (0 for a block of zeros or without numbers).
__device__ __forceinline__ __half q4_scale(uint32_t key, float &r) {
    const float m = __uint_as_float((key >> 1) | (key & 1u ? 0u : 0x80000000u));
    const float d8 = __bfloat162float(__float2bfloat16_rn(m * -0.125f));
    r = 0.0f;
    if (!(fabsf(d8) < 8192.0f)) return __ushort_as_half(0x7fffu);  // NaN
    const __half d = __float2half_rn(d8);
    const float f = __half2float(d);
    if (f == 0.0f) return __ushort_as_half(0);
    r = __fdiv_rn(1.0f, f);
    return d;
}

__device__ __forceinline__ uint32_t q4_code(float x, float r) {
    return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(roundf(__fmul_rn(x, r)), -8.0f), 7.0f)) + 8);
}
// Values 4i .. 4i+3 of a word (i 0 or 1), at their places in it.
__device__ __forceinline__ uint32_t q4_codes(float4 x, float r, int i) {
    const uint32_t a = q4_code(x.x, r) | (q4_code(x.y, r) << 16), b = q4_code(x.z, r) | (q4_code(x.w, r) << 16);
    return (a | (b << 4)) << (8 * i);
}

// One block held as four values by each of eight consecutive lanes (mask: exactly those lanes): its codes as words, in
// the even ones of the lanes, and its scale.
__device__ __forceinline__ uint32_t q4_quant4(float4 x, unsigned mask, __half &d) {
    uint32_t key = q4_key4(x);
    key = max(key, __shfl_xor_sync(mask, key, 1));
    key = max(key, __shfl_xor_sync(mask, key, 2));
    key = max(key, __shfl_xor_sync(mask, key, 4));
    float r;
    d = q4_scale(key, r);
    const uint32_t w = q4_codes(x, r, threadIdx.x & 1);
    return w | __shfl_xor_sync(mask, w, 1);
}

// A Q4 row's zero padding after its scales (up to 14 bytes).
__device__ __forceinline__ void q4_pad(unsigned char *row, int W, long long rb) {
    for (long long b = W / 2 + W / 16; b < rb; b += 2) *reinterpret_cast<uint16_t *>(row + b) = 0;
}

// Elements 4*i4 .. 4*i4+3 of a Q4 row (row: its first byte; W: values in the row).
__device__ __forceinline__ float4 ld4_q4(const unsigned char *row, int W, int i4) {
    const uint32_t w = reinterpret_cast<const uint32_t *>(row)[i4 >> 1] >> (8 * (i4 & 1));
    const float d = __half2float(reinterpret_cast<const __half *>(row + W / 2)[i4 >> 3]);
    auto val = [&](int bit) { return d * static_cast<float>(static_cast<int>((w >> bit) & 15u) - 8); };
    return make_float4(val(0), val(16), val(4), val(20));
}

// The eight values of a word as half2 pairs, in order; d2: the scale in both halves.  A nibble under 0x6400 is 1024 + u
// (or 1024 + 16 u where it stands four bits higher), u - 8 is exact, and so is its product with d.  (Codes put under a
// binary16 number's exponent, the bias taken off in arithmetic: Kim, Henry, Fahim and Awadalla, "Who Says Elephants Can't
// Run: Bringing Large Scale MoE Models into Cloud Scale Production", 2022.)
__device__ __forceinline__ uint32_t q4_lop(uint32_t w, uint32_t mask) {  // (w & mask) | 0x64006400
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, 0x64006400, 0xea;" : "=r"(y) : "r"(w), "r"(mask));
    return y;
}
__device__ __forceinline__ void q4_quants(uint32_t w, uint32_t (&q)[4]) {  // u - 8 as binary16
    const __half2 off = __half2half2(__ushort_as_half(0xe408)), off16 = __half2half2(__ushort_as_half(0xd480));  // -1032, -72
    const __half2 sixteenth = __half2half2(__ushort_as_half(0x2c00));
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint32_t x = i ? w >> 8 : w, a = q4_lop(x, 0x000f000fu), b = q4_lop(x, 0x00f000f0u);
        const __half2 ya = __hadd2(*reinterpret_cast<const __half2 *>(&a), off);
        const __half2 yb = __hfma2(*reinterpret_cast<const __half2 *>(&b), sixteenth, off16);
        q[i] = *reinterpret_cast<const uint32_t *>(&ya);
        q[i + 1] = *reinterpret_cast<const uint32_t *>(&yb);
    }
}
__device__ __forceinline__ void q4_values(uint32_t w, uint32_t d2, uint32_t (&h)[4]) {
    q4_quants(w, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 y = __hmul2_rn(*reinterpret_cast<const __half2 *>(&h[i]), *reinterpret_cast<const __half2 *>(&d2));
        h[i] = *reinterpret_cast<const uint32_t *>(&y);
    }
}

}  // namespace minf
