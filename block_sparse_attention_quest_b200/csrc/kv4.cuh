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

// Eight codes (nibble i = channel i) of x for a group's scale and zero:
// rint(fl((x - zero) / scale)), with inv = 1 / scale to one unit in the last
// place.
//
// The rounded quotient comes without a division. With d = fl(x - zero) and
// q0 = fl(d inv), which is within 2^-22 of d / scale relatively, the residual
// d - q0 scale is exact in one fused operation (scale has 8 significant bits,
// so q0 scale has 32, of which the upper 22 cancel), and q0 + residual inv is
// within 2^-44 of the quotient before its one rounding. A quotient of a 24-bit
// by an 8-bit number that is not itself half-way between two fp32 numbers is
// at least 2^-34 away from there, so that rounding is the quotient's. This
// needs inv and the residual to be normal numbers: scales outside 1e-30 ..
// 1e30 take the division (a constant group's scale is 0, its codes are 0).
//
// EXACT_ZERO: x holds bf16 values, whose minimum the zero is; then no quotient
// leaves [0, 15.5) and nothing is clamped.
template <bool EXACT_ZERO>
__device__ __forceinline__ uint32_t kv4_codes8(const float (&x)[8], float scale, float zero,
                                               float inv) {
  constexpr float kMagic = 12582912.f;           // 1.5 * 2^23: adding it rounds to an integer
  const uint64_t nz = f2_pack(-zero, -zero), iv = f2_pack(inv, inv);
  const uint64_t ns = f2_pack(-scale, -scale);
  const uint64_t up = f2_pack(kMagic, kMagic), down = f2_pack(-kMagic, -kMagic);
  // (2^23 on the pairs' first halves: the sums below then hold the codes in
  // their low bits)
  const uint64_t down0 = f2_pack(8388608.f - kMagic, -kMagic), k256 = f2_pack(256.f, 256.f);
  uint64_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t d = f2_add(f2_pack(x[2 * i], x[2 * i + 1]), nz);
    const uint64_t q0 = f2_mul(d, iv);
    uint64_t q = f2_fma(f2_fma(q0, ns, d), iv, q0);
    if constexpr (!EXACT_ZERO) {
      float a, b;
      f2_unpack(q, a, b);
      q = f2_pack(fminf(fmaxf(a, 0.f), 15.f), fminf(fmaxf(b, 0.f), 15.f));
    }
    c[i] = f2_add(f2_add(q, up), i & 1 ? down : down0);
  }
  // four codes at a time as one number below 2^16, exact in fp32
  float e0, o0, e1, o1;
  f2_unpack(f2_fma(c[1], k256, c[0]), e0, o0);
  f2_unpack(f2_fma(c[3], k256, c[2]), e1, o1);
  uint32_t w = __byte_perm(__float_as_uint(fmaf(o0, 16.f, e0)), __float_as_uint(fmaf(o1, 16.f, e1)),
                           0x5410);
  if (!(scale > 1e-30f && scale < 1e30f)) {
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

__device__ __forceinline__ float kv4_scale(float lo, float hi) {
  return __bfloat162float(__float2bfloat16_rn(__fmul_rn(__fsub_rn(hi, lo), kKv4Inv15)));
}
__device__ __forceinline__ float kv4_reciprocal(float scale) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(scale));
  return y;
}

// Scale, zero and codes of this lane's 8 channels; the group's 8 lanes are
// lane & ~7 .. lane | 7 and all of them call this together.
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
  scale = kv4_scale(lo, hi);
  return kv4_codes8<false>(x, scale, zero, kv4_reciprocal(scale));
}
// The same for eight bf16 values as they lie in memory (minima and maxima two
// at a time).
__device__ __forceinline__ uint32_t kv4_encode8(const uint4& raw, float& scale, float& zero) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  const uint32_t lo2 = bf16x2_min(bf16x2_min(w[0], w[1]), bf16x2_min(w[2], w[3]));
  const uint32_t hi2 = bf16x2_max(bf16x2_max(w[0], w[1]), bf16x2_max(w[2], w[3]));
  // (minimum, -maximum) in one word from here on
  uint32_t v = bf16x2_min(__byte_perm(lo2, hi2, 0x5410) ^ 0x80000000u,
                          __byte_perm(lo2, hi2, 0x7632) ^ 0x80000000u);
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) v = bf16x2_min(v, __shfl_xor_sync(0xffffffffu, v, m));
  zero = bf16_lo(v);
  scale = kv4_scale(zero, -bf16_hi(v));
  float x[8];
  Chunk<__nv_bfloat16>::unpack(raw, x);
  return kv4_codes8<true>(x, scale, zero, kv4_reciprocal(scale));
}

// Transpose of an 8 x 8 matrix of nibbles: nibble c of word r <-> nibble r of
// word c.
__device__ __forceinline__ void nibble_transpose(uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {                  // 4 x 4 halves
    const uint32_t a = w[i], b = w[i + 4];
    w[i] = __byte_perm(a, b, 0x5410);
    w[i + 4] = __byte_perm(a, b, 0x7632);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i & 2) continue;                         // 2 x 2 bytes
    const uint32_t a = w[i], b = w[i + 2];
    w[i] = __byte_perm(a, b, 0x6240);
    w[i + 2] = __byte_perm(a, b, 0x7351);
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {               // nibbles of a byte
    const uint32_t a = w[i], b = w[i + 1];
    w[i] = (a & 0x0f0f0f0fu) | ((b & 0x0f0f0f0fu) << 4);
    w[i + 1] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
  }
}

// bf16 {scale, zero} of one tensor as the record holds them
__device__ __forceinline__ uint32_t kv4_pack_meta(float scale, float zero) {
  return (__float_as_uint(scale) >> 16) | (__float_as_uint(zero) & 0xffff0000u);
}

}  // namespace resa
