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

#include "q8.h"
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

// A sequence's length L, or -1 (recorded in the error word) when it is negative
// or beyond what the cache holds.
__device__ __forceinline__ int checked_length(int L, int blocks, int *err) {
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
    uint32_t h, r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(h) : "r"(w), "r"(0x64646464u), "n"(Half ? 0x4342 : 0x4140));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
    return r;
}

// Codes of numbers against one maximum `most` (bf16, positive and finite):
// rint(127 x / most) for |x| <= most, ties to even, without a division each.
// With f = 2^-e that brings most near 1 (so that nothing below over- or
// underflows), a = 127 f x and d = f most are exact, and with the rounded
// reciprocal c of d
//   t = c a is off by at most 2^-22 t,  r = a - t d is exact (the leading bits
//   cancel),  t + c r is the quotient but for its last rounding
// (a residual correction, as in Markstein's division).  A quotient half-way
// between two whole numbers has at most eight bits, so it comes out exactly;
// any other quotient is further from half-way than 2^-9 of its size.  1.5 2^23
// + 128 added then leaves code number + 128 in the low byte.
struct Coder {
    uint64_t f127, d, c;  // 127 f, -d and c, each as a pair
    __device__ __forceinline__ explicit Coder(float most) {
        int e = (int)(__float_as_uint(most) >> 23) - 127;
        e = max(-120, min(126, e));  // (127 f is finite, and f is no subnormal)
        const float f = __uint_as_float((uint32_t)(127 - e) << 23), near = most * f, inv = __frcp_rn(near);
        f127 = sm100::f2pack(127.f * f, 127.f * f);
        d = sm100::f2pack(-near, -near);
        c = sm100::f2pack(inv, inv);
    }
    // The codes of a bf16 pair in the low bytes of the two words.
    __device__ __forceinline__ uint2 operator()(uint32_t pair) const {
        const uint64_t x = sm100::f2pack(__uint_as_float(pair << 16), __uint_as_float(pair & 0xffff0000u));
        const uint64_t a = sm100::fmul2(f127, x), t = sm100::fmul2(c, a);
        const uint64_t q = sm100::ffma2(c, sm100::ffma2(t, d, a), t);
        const float2 r = sm100::f2unpack(sm100::fadd2(q, sm100::f2pack(12583040.f, 12583040.f)));
        return make_uint2(__float_as_uint(r.x), __float_as_uint(r.y));
    }
    // Of two pairs, as the bytes of a word.
    __device__ __forceinline__ uint32_t operator()(uint32_t first, uint32_t second) const {
        const uint2 a = (*this)(first), b = (*this)(second);
        return __byte_perm(__byte_perm(a.x, a.y, 0x0040), __byte_perm(b.x, b.y, 0x0040), 0x5410);
    }
};

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
