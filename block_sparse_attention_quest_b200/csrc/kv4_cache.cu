// Writing and reading back the 4-bit cache: whole rows, and the token a decode
// step appends. The format is described in kv4.cuh.
#include "kv4.cuh"

namespace resa {

// Rows to records. One warp per (record, K or V): a lane owns 8 channels of a
// token, the 8 lanes of a 64-channel group find its minimum and maximum with
// three shuffles each. The key words of a lane's 8 channels are whole words of
// the record; the value words mix four tokens and two times eight channels,
// one 8 x 8 transpose of nibbles for each (group, token pair, 16 channels),
// done by one lane on words taken from shared memory. Tokens past the row's
// length count as zeros (code 0, scale 0, zero 0).
//
// Bound by instruction issue: 128K tokens of 8 heads, d = 128, take 149 us (688
// MB, 105 us at the copy rate) at 3.0 of 4 instructions per cycle, about 14
// per 32 elements; see kv4_codes8 for what that takes (with divisions 327 us).
template <typename T> struct Kv4Raw;
template <> struct Kv4Raw<__nv_bfloat16> {
  uint4 x;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = ld_stream16(p); }
  __device__ __forceinline__ void clear() { x = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ uint32_t encode(float& scale, float& zero) const {
    return kv4_encode8(x, scale, zero);
  }
};
template <> struct Kv4Raw<float> {
  float x[8];
  __device__ __forceinline__ void load(const float* p) { load8<float>(p, x); }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
  }
  __device__ __forceinline__ uint32_t encode(float& scale, float& zero) const {
    return kv4_encode8(x, scale, zero);
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_quantize_kernel(const T* __restrict__ k,
                                                           const T* __restrict__ v,
                                                           uint8_t* __restrict__ kv4, int64_t L_max,
                                                           int Mmax, int M, int64_t len,
                                                           int64_t total, const int32_t* lens,
                                                           int H) {
  constexpr int NG = D / kKv4Group;
  constexpr int LPR = D / 8;                     // lanes per token
  constexpr int TPP = 32 / LPR;                  // tokens per pass
  constexpr int PASSES = kBlock / TPP;
  constexpr int REC = kv4_record_bytes(D);
  __shared__ __align__(16) uint8_t stage[4][REC];   // one record per pair of warps
  __shared__ __align__(16) uint32_t vcode[4][kBlock][D / 8 + 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = warp >> 1;
  const bool is_v = warp & 1;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + pair;
  const int64_t bh = id / M;
  const int j = static_cast<int>(id % M);
  int64_t len_b = 0;
  if (id < total) len_b = row_len(lens, len, static_cast<int>(bh / H));
  const int64_t t0 = static_cast<int64_t>(j) * kBlock;
  const bool live = id < total && t0 < len_b;
  const int valid = live ? static_cast<int>(len_b - t0 < kBlock ? len_b - t0 : kBlock) : 0;
  const int chunk = lane % LPR;                  // channels 8 * chunk .. + 7
  const int r0 = lane / LPR;
  const int g = chunk / 8, x8 = chunk % 8;       // 64-channel group, 8-channel part of it
  uint8_t* rec = stage[pair];
  if (live) {
    const T* src = (is_v ? v : k) + (bh * L_max + t0) * D + chunk * 8;
    Kv4Raw<T> x[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int t = r0 + p * TPP;
      if (t < valid) x[p].load(src + static_cast<int64_t>(t) * D);
      else x[p].clear();
    }
    // token t = r0 + p * TPP = 8h + r of pass p: h = p / HALF, r from the rest
    constexpr int HALF = PASSES / 2;
    uint8_t* codes = is_v ? reinterpret_cast<uint8_t*>(&vcode[pair][r0][chunk])
                          : rec + g * 512 + (r0 * 4 + (x8 >> 1)) * 16 + (x8 & 1) * 4;
    // (from one pass to the next of a half, and from one half to the other)
    const int step = is_v ? TPP * static_cast<int>(sizeof(vcode[0][0])) : TPP * 64;
    const int hop = is_v ? 8 * static_cast<int>(sizeof(vcode[0][0])) : 8;
    uint8_t* meta = rec + 2 * kv4_code_bytes(D) + (r0 * 2 * NG + g) * 8 + (is_v ? 4 : 0);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      float scale, zero;
      const uint32_t w = x[p].encode(scale, zero);
      *reinterpret_cast<uint32_t*>(codes + (p % HALF) * step + (p / HALF) * hop) = w;
      if (x8 == 0)
        *reinterpret_cast<uint32_t*>(meta + (p % HALF) * (TPP * 2 * NG * 8) + (p / HALF) * (NG * 8)) =
            kv4_pack_meta(scale, zero);
    }
    if (is_v) {
      __syncwarp();
      // lane (g, c, m): nibble e + 2h + 4o of the words r = 0 .. 7 is token
      // 8h + 2c + o, channel 16m + 8e + r
      const int gg = lane >> 4, c = (lane >> 2) & 3, m = lane & 3;
      if (gg < NG) {
        uint32_t w[8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const uint2 cd = *reinterpret_cast<const uint2*>(
                &vcode[pair][8 * h + 2 * c + o][gg * 8 + 2 * m]);
            w[2 * h + 4 * o] = cd.x;
            w[1 + 2 * h + 4 * o] = cd.y;
          }
        nibble_transpose(w);
        uint8_t* dst = rec + kv4_value_word_at(D, 2 * c, gg, m);
#pragma unroll
        for (int r = 0; r < 8; ++r) *reinterpret_cast<uint32_t*>(dst + r * 64) = w[r];
      }
    }
  }
  __syncthreads();
  if (live) {
    uint8_t* dst = kv4 + (bh * Mmax + j) * REC;
    for (int i = lane + (is_v ? 32 : 0); i < REC / 16; i += 64)
      *reinterpret_cast<uint4*>(dst + i * 16) = *reinterpret_cast<const uint4*>(rec + i * 16);
  }
}

// Eight values zero + scale * code of a word's nibbles, in fp32 (the product
// is exact; a code becomes a float as the low bits of 2^23 + code).
__device__ __forceinline__ void kv4_decode8(uint32_t w, uint32_t meta, float (&f)[8]) {
  const float s = bf16_lo(meta), z = bf16_hi(meta);
  const uint64_t s2 = f2_pack(s, s), z2 = f2_pack(z, z), down = f2_pack(-8388608.f, -8388608.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __uint_as_float(((w >> (8 * i)) & 15u) | 0x4b000000u);
    const float b = __uint_as_float(((w >> (8 * i + 4)) & 15u) | 0x4b000000u);
    f2_unpack(f2_fma(f2_add(f2_pack(a, b), down), s2, z2), f[2 * i], f[2 * i + 1]);
  }
}

// 16 consecutive channels of a token
__device__ __forceinline__ void store16(float* p, bool, const float (&a)[8], const float (&b)[8]) {
  float4* q = reinterpret_cast<float4*>(p);
  q[0] = make_float4(a[0], a[1], a[2], a[3]);
  q[1] = make_float4(a[4], a[5], a[6], a[7]);
  q[2] = make_float4(b[0], b[1], b[2], b[3]);
  q[3] = make_float4(b[4], b[5], b[6], b[7]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, bool wide, const float (&a)[8],
                                        const float (&b)[8]) {
  const uint4 x = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                             pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
  const uint4 y = make_uint4(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]),
                             pack_bf16x2(b[4], b[5]), pack_bf16x2(b[6], b[7]));
  if (wide) {                                     // a whole sector from one lane
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"l"(p), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(y.x), "r"(y.y), "r"(y.z),
                   "r"(y.w)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = x;
    reinterpret_cast<uint4*>(p)[1] = y;
  }
}

// Records to rows, rounded once to the cache type. One warp per (record, K or
// V); lane (g, c, m) has the sixteen channels 64g + 16m .. + 15 of four
// tokens, for values the four of an inverse transpose of nibbles. Bound by HBM
// (128K tokens of 8 heads, d = 128: 102 us for 688 MB).
template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_dequantize_kernel(const uint8_t* __restrict__ kv4,
                                                             T* __restrict__ k, T* __restrict__ v,
                                                             int64_t L_max, int Mmax, int M,
                                                             int64_t len, int64_t total,
                                                             const int32_t* lens, int H) {
  constexpr int REC = kv4_record_bytes(D);
  constexpr int NG = D / kKv4Group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool is_v = warp & 1;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + (warp >> 1);
  if (id >= total) return;
  const int64_t bh = id / M;
  const int j = static_cast<int>(id % M);
  const int64_t len_b = row_len(lens, len, static_cast<int>(bh / H));
  const int64_t t0 = static_cast<int64_t>(j) * kBlock;
  if (t0 >= len_b) return;
  const int valid = static_cast<int>(len_b - t0 < kBlock ? len_b - t0 : kBlock);
  const int g = lane >> 4, c = (lane >> 2) & 3, m = lane & 3;
  if (g >= NG) return;
  // (the caches are 16-byte aligned; 32-byte stores need twice that)
  const bool wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31) == 0;
  const uint8_t* rec = kv4 + (bh * Mmax + j) * REC;
  T* dst = (is_v ? v : k) + (bh * L_max + t0) * D + g * 64 + m * 16;
  if (is_v) {
    uint32_t w[8];
    const uint8_t* src = rec + kv4_value_word_at(D, 2 * c, g, m);
#pragma unroll
    for (int r = 0; r < 8; ++r) w[r] = __ldg(reinterpret_cast<const uint32_t*>(src + r * 64));
    uint32_t meta[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)                   // token 8 (i / 2) + 2c + i % 2
      meta[i] = __ldg(reinterpret_cast<const uint32_t*>(
          rec + kv4_meta_at(D, 8 * (i >> 1) + 2 * c + (i & 1), g) + 4));
    nibble_transpose(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 8 * (i >> 1) + 2 * c + (i & 1);
      if (t >= valid) continue;
      float a[8], b[8];
      kv4_decode8(w[2 * (i >> 1) + 4 * (i & 1)], meta[i], a);
      kv4_decode8(w[1 + 2 * (i >> 1) + 4 * (i & 1)], meta[i], b);
      store16(dst + static_cast<int64_t>(t) * D, wide, a, b);
    }
  } else {
    // words [r][m][2h], [r][m][2h + 1] of token 8h + r; lane's tokens c, c + 4, ...
    uint2 w[4];
    uint32_t meta[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = c + 4 * i;
      w[i] = __ldg(reinterpret_cast<const uint2*>(rec + g * 512 + ((t & 7) * 4 + m) * 16 + (t >> 3) * 8));
      meta[i] = __ldg(reinterpret_cast<const uint32_t*>(rec + kv4_meta_at(D, t, g)));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = c + 4 * i;
      if (t >= valid) continue;
      float a[8], b[8];
      kv4_decode8(w[i].x, meta[i], a);
      kv4_decode8(w[i].y, meta[i], b);
      store16(dst + static_cast<int64_t>(t) * D, wide, a, b);
    }
  }
}

// The token a decode step appends: its key and value into slot len - 1 of the
// records, its key into the block's descriptor (when there is one). Grid
// (H, B), 64 threads: warp 0 the key, warp 1 the value. A token that opens a
// block clears the block's value words, so no code of an earlier use remains.
template <typename T, int D>
__global__ void __launch_bounds__(64) kv4_append_kernel(const T* __restrict__ k_new,
                                                        const T* __restrict__ v_new,
                                                        uint8_t* __restrict__ kv4,
                                                        T* __restrict__ desc, int H, int Mmax,
                                                        int64_t len, const int32_t* lens) {
  constexpr int LPR = D / 8;
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool is_v = warp == 1;
  const int64_t bh = static_cast<int64_t>(blockIdx.y) * H + blockIdx.x;
  const int64_t tok = row_len(lens, len, blockIdx.y) - 1;
  const int64_t blk = tok / kBlock;
  const int t = static_cast<int>(tok % kBlock);
  uint8_t* rec = kv4 + (bh * Mmax + blk) * kv4_record_bytes(D);
  const int chunk = lane % LPR;                  // (lanes past the token's repeat it and store nothing)
  const bool own = lane < LPR;
  const int g = chunk / 8, x8 = chunk % 8;
  float x[8];
  load8<T>((is_v ? v_new : k_new) + bh * D + chunk * 8, x);
  float scale, zero;
  const uint32_t w = kv4_encode8(x, scale, zero);
  if (own && x8 == 0)
    *reinterpret_cast<uint32_t*>(rec + kv4_meta_at(D, t, g) + (is_v ? 4 : 0)) =
        kv4_pack_meta(scale, zero);
  if (!is_v) {
    if (own)
      *reinterpret_cast<uint32_t*>(
          rec + g * 512 + ((t & 7) * 4 + (x8 >> 1)) * 16 + ((t >> 3) * 2 + (x8 & 1)) * 4) = w;
    if (desc != nullptr && own) {
      T* d = desc + (bh * Mmax + blk) * 2 * D + chunk * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float lo = x[i], hi = x[i];
        if (t != 0) {
          lo = fminf(Dt<T>::to_f(d[i]), lo);
          hi = fmaxf(Dt<T>::to_f(d[D + i]), hi);
        }
        d[i] = Dt<T>::from_f(lo);
        d[D + i] = Dt<T>::from_f(hi);
      }
    }
    return;
  }
  // value word [g][r][c][m], nibbles 2h + 4o (channels r) and 1 + 2h + 4o
  // (channels 8 + r): the even one of two neighbouring lanes writes both
  const uint32_t w1 = __shfl_down_sync(0xffffffffu, w, 1);
  if (own && (x8 & 1) == 0) {
    const int sh = 4 * (2 * (t >> 3) + 4 * (t & 1));
    uint8_t* at = rec + kv4_value_word_at(D, t, g, x8 >> 1);
    const bool opens = t == 0;
    uint32_t old[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      old[r] = opens ? 0u : *reinterpret_cast<const uint32_t*>(at + r * 64);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const uint32_t two = ((w >> (4 * r)) & 15u) | (((w1 >> (4 * r)) & 15u) << 4);
      *reinterpret_cast<uint32_t*>(at + r * 64) = (old[r] & ~(255u << sh)) | (two << sh);
    }
    if (opens) {
      // the words of the block's other token pairs (c = 1, 2, 3)
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int c = 1; c < 4; ++c) *reinterpret_cast<uint32_t*>(at + r * 64 + c * 16) = 0u;
    }
  }
}

template <typename T, int D>
static cudaError_t quantize_t(const Shape& s, const void* k, const void* v, void* kv4, int64_t len,
                              const int32_t* lens, cudaStream_t st) {
  const int M = static_cast<int>((len + kBlock - 1) / kBlock);
  const int64_t total = static_cast<int64_t>(s.B) * s.H * M;
  kv4_quantize_kernel<T, D><<<static_cast<unsigned>((total + 3) / 4), 256, 0, st>>>(
      static_cast<const T*>(k), static_cast<const T*>(v), static_cast<uint8_t*>(kv4), s.L_max,
      s.Mmax, M, len, total, lens, s.H);
  return cudaGetLastError();
}

cudaError_t launch_kv4_quantize(const Shape& s, const void* k, const void* v, void* kv4,
                                int64_t len, const int32_t* lens, cudaStream_t st) {
  if (s.bf16)
    return s.D == 128 ? quantize_t<__nv_bfloat16, 128>(s, k, v, kv4, len, lens, st)
                      : quantize_t<__nv_bfloat16, 64>(s, k, v, kv4, len, lens, st);
  return s.D == 128 ? quantize_t<float, 128>(s, k, v, kv4, len, lens, st)
                    : quantize_t<float, 64>(s, k, v, kv4, len, lens, st);
}

template <typename T, int D>
static cudaError_t dequantize_t(const Shape& s, const void* kv4, void* k, void* v, int64_t len,
                                const int32_t* lens, cudaStream_t st) {
  const int M = static_cast<int>((len + kBlock - 1) / kBlock);
  const int64_t total = static_cast<int64_t>(s.B) * s.H * M;
  kv4_dequantize_kernel<T, D><<<static_cast<unsigned>((total + 3) / 4), 256, 0, st>>>(
      static_cast<const uint8_t*>(kv4), static_cast<T*>(k), static_cast<T*>(v), s.L_max, s.Mmax, M,
      len, total, lens, s.H);
  return cudaGetLastError();
}

cudaError_t launch_kv4_dequantize(const Shape& s, const void* kv4, void* k, void* v, int64_t len,
                                  const int32_t* lens, cudaStream_t st) {
  if (s.bf16)
    return s.D == 128 ? dequantize_t<__nv_bfloat16, 128>(s, kv4, k, v, len, lens, st)
                      : dequantize_t<__nv_bfloat16, 64>(s, kv4, k, v, len, lens, st);
  return s.D == 128 ? dequantize_t<float, 128>(s, kv4, k, v, len, lens, st)
                    : dequantize_t<float, 64>(s, kv4, k, v, len, lens, st);
}

template <typename T, int D>
static cudaError_t append_t(const Shape& s, const void* k_new, const void* v_new, void* kv4,
                            void* desc, int64_t len, const int32_t* lens, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.H, s.B);
  cfg.blockDim = dim3(64);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_append_kernel<T, D>, static_cast<const T*>(k_new),
                            static_cast<const T*>(v_new), static_cast<uint8_t*>(kv4),
                            static_cast<T*>(desc), s.H, s.Mmax, len, lens);
}

cudaError_t launch_kv4_append(const Shape& s, const void* k_new, const void* v_new, void* kv4,
                              void* desc, int64_t len, const int32_t* lens, cudaStream_t st) {
  if (s.bf16)
    return s.D == 128 ? append_t<__nv_bfloat16, 128>(s, k_new, v_new, kv4, desc, len, lens, st)
                      : append_t<__nv_bfloat16, 64>(s, k_new, v_new, kv4, desc, len, lens, st);
  return s.D == 128 ? append_t<float, 128>(s, k_new, v_new, kv4, desc, len, lens, st)
                    : append_t<float, 64>(s, k_new, v_new, kv4, desc, len, lens, st);
}

}  // namespace resa
