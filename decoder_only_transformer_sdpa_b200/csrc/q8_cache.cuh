// q8_cache.cuh -- the 8-bit block cache of keys and values as the kernels see
// it: where each part of a block lies, and the checks of what callers keep on
// the device (sequence lengths, block lists).
//
// Blocks of 64 tokens are quantised when they are full ("closed"), one scale
// for the keys and one for the values of a block and head:
//
//   scale = max|x| / 127,  code = 128 + rint(127 x / max|x|),
//   x is held as (code - 128) * scale.
//
// 127 x is exact in float32 (15 significant bits), and a quotient of a 15-bit
// and an 8-bit number is either half-way between two whole numbers or further
// from it than float32's rounding, so the rounded division decides every tie
// as real arithmetic does (to even).  A held value is off by at most half a
// step, max|x| / 254.  A block with an infinity or a NaN takes a NaN scale.
//
// Keys of a block lie as [D / S][64][S] bytes with S = min(D, 64), values as
// [D][64]: 64 consecutive bytes are what four lanes of a tensor-core fragment
// take, so both operands of the two products are read from shared memory with
// 16-byte loads that touch every bank once.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"
#include "sm100.cuh"

namespace attn {
namespace q8 {

constexpr int kBlock = kQ8Block;    // tokens of a block
constexpr int kRing = 2 * kBlock;   // positions kept in bf16 (position p in row p mod 128)

__host__ __device__ constexpr int slab(int D) { return D < 64 ? D : 64; }

// Byte offset of channel `ch` of token `t` in a block's keys.
template <int D>
__device__ __forceinline__ int key_offset(int t, int ch) {
    constexpr int S = slab(D);
    return (ch / S) * (kBlock * S) + t * S + ch % S;
}

// The length of sequence b, or -1 (recorded in the error word) when it is
// negative or beyond what the cache holds.
__device__ __forceinline__ int checked_length(const int32_t *lens, int b, int blocks, int *err) {
    const int L = lens[b];
    if (L < 0 || L / kBlock > blocks) {
        if (threadIdx.x == 0) atomicExch(err, kErrLength);
        return -1;
    }
    return L;
}

// Two code bytes (0, 1 or 2, 3 of a word) as an f16 pair of code - 128: the
// byte under 0x64 is 1024 + code, and 1152 is subtracted exactly.
template <int Half>
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t w) {
    uint32_t h;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(h) : "r"(w), "r"(0x64646464u), "n"(Half ? 0x4342 : 0x4140));
    uint32_t r;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
    return r;
}

// rint(127 x / most) for |x| <= most, most > 0 and finite (both bf16).  Above
// 2^120 both are brought down by 2^10 first, so that 127 x stays finite; that
// is exact but for values whose quotient rounds to 0 either way.
__device__ __forceinline__ int code_number(float x, float most) {
    const float f = most >= 1.329227995784916e36f ? 0.0009765625f : 1.f;
    return __float2int_rn(__fdiv_rn(127.f * (x * f), most * f));
}

// A float's place in the order of all floats, as an unsigned number (the two
// zeros are one; NaN comes above everything but kFirst).
constexpr uint32_t kFirst = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return kFirst - 1;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

}  // namespace q8
}  // namespace attn
