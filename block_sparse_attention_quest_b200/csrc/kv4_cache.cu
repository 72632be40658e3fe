// Writing and reading back the 4-bit cache: whole rows, and the token a decode
// step appends. The format is described in kv4.cuh.
#include "kv4.cuh"

namespace resa {

// Rows to records. One warp per (record, K or V): a lane owns 8 channels of a
// token, the 8 lanes of a 64-channel group find its minimum and maximum with
// three shuffles each. The key words of a lane's 8 channels are whole words of
// the record; the value words mix four tokens and two channels, so the value
// codes pass through shared memory. Tokens past the row's length count as
// zeros (code 0, scale 0, zero 0).
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
  __shared__ __align__(16) uint32_t vcode[4][kBlock][D / 8];
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
    float x[PASSES][8];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int t = r0 + p * TPP;
      if (t < valid) {
        load8<T>(src + static_cast<int64_t>(t) * D, x[p]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[p][e] = 0.f;
      }
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int t = r0 + p * TPP;
      float scale, zero;
      const uint32_t w = kv4_encode8(x[p], scale, zero);
      if (is_v) {
        vcode[pair][t][chunk] = w;
      } else {
        // word [g][r][c][2h + j]: r = t % 8, c = x8 / 2, h = t / 8, j = x8 % 2
        *reinterpret_cast<uint32_t*>(
            rec + g * 512 + ((t & 7) * 4 + (x8 >> 1)) * 16 + ((t >> 3) * 2 + (x8 & 1)) * 4) = w;
      }
      if (x8 == 0)
        *reinterpret_cast<uint32_t*>(rec + kv4_meta_at(D, t, g) + (is_v ? 4 : 0)) =
            kv4_pack_meta(scale, zero);
    }
    if (is_v) {
      __syncwarp();
      // lane (r, c): word m of group g holds tokens 2c, 2c + 1, 2c + 8, 2c + 9
      // of channels 16m + r and 16m + 8 + r
      const int r = lane >> 2, c = lane & 3;
#pragma unroll
      for (int gg = 0; gg < NG; ++gg) {
        uint32_t out[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          uint32_t w = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const uint2 cd = *reinterpret_cast<const uint2*>(
                  &vcode[pair][8 * h + 2 * c + o][gg * 8 + 2 * m]);
              w |= ((cd.x >> (4 * r)) & 15u) << (4 * (2 * h + 4 * o));
              w |= ((cd.y >> (4 * r)) & 15u) << (4 * (1 + 2 * h + 4 * o));
            }
          out[m] = w;
        }
        *reinterpret_cast<uint4*>(rec + kv4_code_bytes(D) + gg * 512 + lane * 16) =
            make_uint4(out[0], out[1], out[2], out[3]);
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

// Records to rows: one warp per record; zero + scale * code in fp32 (the
// product is exact), rounded once to the cache type.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv4_dequantize_kernel(const uint8_t* __restrict__ kv4,
                                                             T* __restrict__ k, T* __restrict__ v,
                                                             int64_t L_max, int Mmax, int M,
                                                             int64_t len, int64_t total,
                                                             const int32_t* lens, int H) {
  constexpr int REC = kv4_record_bytes(D);
  constexpr int LPR = D / 8;
  constexpr int TPP = 32 / LPR;
  __shared__ __align__(16) uint8_t stage[8][REC];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  if (id >= total) return;
  const int64_t bh = id / M;
  const int j = static_cast<int>(id % M);
  const int64_t len_b = row_len(lens, len, static_cast<int>(bh / H));
  const int64_t t0 = static_cast<int64_t>(j) * kBlock;
  if (t0 >= len_b) return;
  const int valid = static_cast<int>(len_b - t0 < kBlock ? len_b - t0 : kBlock);
  const uint8_t* src = kv4 + (bh * Mmax + j) * REC;
  uint8_t* rec = stage[warp];
  for (int i = lane; i < REC / 16; i += 32)
    *reinterpret_cast<uint4*>(rec + i * 16) = ld_stream16(src + i * 16);
  __syncwarp();
  const int chunk = lane % LPR, r0 = lane / LPR;
  const int g = chunk / 8, x8 = chunk % 8;
  auto store = [&](T* dst, const float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(dst) = make_float4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                  pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
  };
#pragma unroll 2
  for (int t = r0; t < valid; t += TPP) {
    const uint2 meta = *reinterpret_cast<const uint2*>(rec + kv4_meta_at(D, t, g));
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(
        rec + g * 512 + ((t & 7) * 4 + (x8 >> 1)) * 16 + ((t >> 3) * 2 + (x8 & 1)) * 4);
    const int m = x8 >> 1, e = x8 & 1;
    const int sh = 4 * (e + 2 * (t >> 3) + 4 * (t & 1));
    float fk[8], fv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t vw =
          *reinterpret_cast<const uint32_t*>(rec + kv4_value_word_at(D, t, g, m) + i * 64);
      fk[i] = fmaf(bf16_lo(meta.x), static_cast<float>((kw >> (4 * i)) & 15u), bf16_hi(meta.x));
      fv[i] = fmaf(bf16_lo(meta.y), static_cast<float>((vw >> sh) & 15u), bf16_hi(meta.y));
    }
    const int64_t at = (bh * L_max + t0 + t) * D + chunk * 8;
    store(k + at, fk);
    store(v + at, fv);
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
  kv4_dequantize_kernel<T, D><<<static_cast<unsigned>((total + 7) / 8), 256, 0, st>>>(
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
