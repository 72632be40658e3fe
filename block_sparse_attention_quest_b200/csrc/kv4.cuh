// The 4-bit cache: its format, and the code that writes one token or one block
// of it.
//
// A group of 64 channels of a token's key (or value) is held as
//   x = zero + scale * code,  scale = bf16((max - min) * fp32(1/15)),
//   zero = bf16(min),  code = rint((x - zero) / scale) in 0..15 (0 where the
//   scale is 0),
// all in fp32 arithmetic. Sixteen tokens (one block of the block-sparse
// method) form one record of 16 * (D + 8 * D / 64) bytes,
//   [key codes][value codes][scales and zeros],
// contiguous, so that one bulk copy brings a block and one warp computes it:
//   keys    token 8h + r, channel 64g + 16c + 8j + i: nibble i of 32-bit word
//           [g][r][c][2h + j];
//   values  token 8h + 2c + o, channel 64g + 16m + 8e + r: nibble e + 2h + 4o
//           of word [g][r][c][m];
//   scales  token 8h + r, group g: [r][h][g] of {key scale, key zero, value
//           scale, value zero} in bf16.
// Lane (r, c) = 4r + c of a warp thus finds its operand fragments of the
// m16n8k16 product in one 16-byte word group per 64 channels: a mask of
// 0x000f000f or 0x00f000f0 (after a shift by 8 for the upper bytes) leaves the
// two codes of one operand register, 16 bits apart. Read as bf16 those bits
// are the subnormal numbers code * 2^-133 (or 16 * code * 2^-133), exact, so a
// code costs no conversion; the power of two and the group's scale are applied
// to the fp32 sums.
#pragma once

#include "launch.h"

namespace resa {

constexpr int kKv4Group = 64;                    // channels per scale and zero point
constexpr float kKv4Inv15 = 1.0f / 15.0f;

__host__ __device__ constexpr int kv4_record_bytes(int D) {
  return kBlock * (D + 8 * (D / kKv4Group));
}
__host__ __device__ constexpr int kv4_code_bytes(int D) { return 512 * (D / kKv4Group); }
// byte offsets inside a record
__device__ __forceinline__ int kv4_meta_at(int D, int t, int g) {
  return 2 * kv4_code_bytes(D) + (((t & 7) * 2 + (t >> 3)) * (D / kKv4Group) + g) * 8;
}
// first of the words that hold value codes of token t, channels 64g + 16m + 8e + r
// (the word of r is 64 bytes further for each r)
__device__ __forceinline__ int kv4_value_word_at(int D, int t, int g, int m) {
  return kv4_code_bytes(D) + g * 512 + ((t & 7) >> 1) * 16 + m * 4;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 8 consecutive channels of one token as floats
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
  Chunk<__nv_bfloat16>::unpack(ld_stream16(p), f);
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
  const uint4 a = ld_stream16(p), b = ld_stream16(p + 4);
  Chunk<float>::unpack(a, f);
  Chunk<float>::unpack(b, f + 4);
}

// Scale, zero (as their bf16 values) and the eight codes (nibble i = channel i)
// of this lane's 8 channels; the group's 8 lanes are lane & ~7 .. lane | 7 and
// all of them call this together.
//
// code = rint(fl((x - zero) / scale)) needs the correctly rounded quotient
// only next to a half: the product with the reciprocal is within 15 * 2^-22 of
// it, so unless some product lies within 2^-16 of a half its rounding is the
// quotient's, and the eight divisions (about ten instructions each, more than
// the copy's bandwidth leaves per element) are done only then.
__device__ __forceinline__ uint32_t kv4_encode8(const float (&x)[8], float& scale, float& zero) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) { lo = fminf(lo, x[i]); hi = fmaxf(hi, x[i]); }
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  zero = __bfloat162float(__float2bfloat16_rn(lo));
  scale = __bfloat162float(__float2bfloat16_rn(__fmul_rn(__fsub_rn(hi, lo), kKv4Inv15)));
  constexpr float kMagic = 12582912.f;           // 1.5 * 2^23: adding it rounds to an integer
  const float inv = __frcp_rn(scale);
  float worst = 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = fminf(fmaxf((x[i] - zero) * inv, 0.f), 15.f);
    const float r = q + kMagic;
    worst = fmaxf(worst, fabsf(q - (r - kMagic)));
    w |= (__float_as_uint(r) & 15u) << (4 * i);
  }
  if (!(worst < 0.5f - 1.0f / 65536.f) || !(scale > 1e-30f)) {
    w = 0;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      // (a loop over one copy of the division: this path is rare)
      float xi = x[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) xi = i == e ? x[e] : xi;
      const float q = scale > 0.f ? __fdiv_rn(__fsub_rn(xi, zero), scale) : 0.f;
      w |= static_cast<uint32_t>(fminf(fmaxf(rintf(q), 0.f), 15.f)) << (4 * i);
    }
  }
  return w;
}

// bf16 {scale, zero} of one tensor as the record holds them
__device__ __forceinline__ uint32_t kv4_pack_meta(float scale, float zero) {
  return (__float_as_uint(scale) >> 16) | (__float_as_uint(zero) & 0xffff0000u);
}

}  // namespace resa
