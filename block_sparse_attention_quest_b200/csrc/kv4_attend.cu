// Decode attention over the 4-bit cache (format: kv4.cuh): every query head of
// a KV group over all of a row's tokens, or over a list of its blocks.
//
// With x = zero + scale * code per token t and 64-channel group a,
//   q . k_t   = sum_a [ ks_ta * sum_{c in a} q_c kcode_tc + kz_ta * sum_{c in a} q_c ]
//   out_c     = sum_t (p_t vs_ta) vcode_tc + sum_t p_t vz_ta        (c in a)
// so both products run on the codes themselves (m16n8k16 on bf16: 16 tokens x
// 8 heads, then 16 channels x 8 heads), and the scales and zeros enter as fp32
// factors of the sums, two per token and head. A code is used as the bf16
// subnormal its bits are (code * 2^-133): one mask per two codes and no
// conversion; q and p enter multiplied by 2^64 so that every sum stays a
// normal number, and 2^69 is taken out of the results. Codes, q (bf16) and
// their products are exact. p * vs is rounded to bf16 (relative error 2^-9 per
// term, as the bf16 cache's attention rounds p); the zero part keeps fp32 p.
// fp32 queries and fp32 p * vs enter as three bf16 parts each (24 bits), so an
// fp32 call keeps fp32 accuracy.
//
// Work split: the blocks of every (row, KV head) in turn form one range, cut
// into equal parts, one per CTA; a CTA walks the one or more (row, head)
// pieces of its part. Rows of different lengths therefore load every CTA
// alike. A piece that is not a whole (row, head) is left as a partial
// (max, sum, accumulator) and the last CTA to arrive merges them in the order
// of the range, so results do not depend on the arrival order.
//
// Each warp streams whole records (one bulk copy per 16-token block, four in
// flight) through its own ring in shared memory.
#include "kv4.cuh"

#include "attend_core.cuh"

namespace resa {

struct Kv4K {
  const void* q;
  const uint8_t* kv4;
  const int32_t* sel;      // [B][H][n_sel] or nullptr (every block)
  const int32_t* lens;     // optional per-row lengths [B]
  float* part_o;           // [2 * CTAs][G][D]
  float* part_ml;          // [2 * CTAs][G][2]
  int* counters;           // [B * H], zero between calls
  Ctrl* ctrl;
  void* out;
  float* lse;
  int64_t len;             // length, or the bound on the rows' lengths
  double r;                // with lens and sel: Eq. 5 of each row (r > 0)
  int n_min;
  int B, H, G, Hq, Mmax, n_sel;
  float scale_log2;
};

constexpr int kKv4Warps = 8;
constexpr int kKv4Stages = 4;
constexpr int kKv4MinBlocks = 8;   // blocks per CTA below which fewer CTAs are used

template <int D>
struct Kv4Cfg {
  static constexpr int kRec = kv4_record_bytes(D);
  static constexpr int kRing = kKv4Warps * kKv4Stages * kRec;
  static constexpr int kMerge = merge_floats(D, kKv4Warps) * 4;
  static constexpr int kSmem = (kRing > kMerge ? kRing : kMerge) + 128;
  static_assert(kRing >= (8 * (kKv4MaxCtas + 2) + 8) * 4, "weights of the parts");
};

// blocks of row b that its heads attend to
__device__ __forceinline__ int kv4_row_blocks(const Kv4K& a, int b) {
  const int64_t l = row_len(a.lens, a.len, b);
  if (a.sel == nullptr) return static_cast<int>((l + kBlock - 1) / kBlock);
  return a.lens != nullptr ? num_selected_dev(l, a.r, a.n_min) : a.n_sel;
}

// One warp finds the row that holds position `x` of the range (or, with
// x < 0, only the total).
__device__ __forceinline__ void kv4_find(const Kv4K& a, long long x, long long& total, int& row,
                                         long long& row_start) {
  const int lane = threadIdx.x & 31;
  if (a.lens == nullptr) {
    const long long per = static_cast<long long>(a.H) * kv4_row_blocks(a, 0);
    total = per * a.B;
    row = x < 0 ? 0 : static_cast<int>(x / per);
    row_start = row * per;
    return;
  }
  long long run = 0;
  row = a.B;
  row_start = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    const long long mine = b < a.B ? static_cast<long long>(a.H) * kv4_row_blocks(a, b) : 0;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const long long begin = run + inc - mine;
    const bool here = x >= begin && x < begin + mine;
    const unsigned who = __ballot_sync(0xffffffffu, here);
    if (who) {
      const int src = __ffs(who) - 1;
      row = b0 + src;
      row_start = __shfl_sync(0xffffffffu, begin, src);
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  total = run;
}

// first position of CTA i's part
__device__ __forceinline__ long long kv4_cut(long long total, int ctas, int i) {
  return total * i / ctas;
}
// the CTA whose part holds position x
__device__ __forceinline__ int kv4_owner(long long total, int ctas, long long x) {
  int i = static_cast<int>((x * ctas) / total);
  while (i + 1 < ctas && kv4_cut(total, ctas, i + 1) <= x) ++i;
  while (kv4_cut(total, ctas, i) > x) --i;
  return i;
}

// Merge of the partials of (row, head) u, whose blocks are [u0, u1) of the
// range, by one CTA. The parts' (max, sum) pairs are turned into weights first,
// then every thread sums pairs of output columns over the parts.
template <typename T, int D>
__device__ __forceinline__ void kv4_merge(const Kv4K& a, float* sm, long long total, int ctas,
                                          long long u0, long long u1, int64_t head0) {
  constexpr int NT = kKv4Warps * 32;
  const int first = kv4_owner(total, ctas, u0), last = kv4_owner(total, ctas, u1 - 1);
  const int n = last - first + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto slot = [&](int s) -> int64_t {
    // a part that began before the unit's first block holds it as its last piece
    return 2 * static_cast<int64_t>(first + s) +
           (s == 0 && kv4_cut(total, ctas, first) < u0 ? 1 : 0);
  };
  float* w_s = sm;                      // [n][8] weights
  float* l_h = sm + 8 * (kKv4MaxCtas + 2);
  for (int h = warp; h < a.G; h += kKv4Warps) {
    float m = -INFINITY;
    for (int s = lane; s < n; s += 32) m = fmaxf(m, __ldcg(a.part_ml + (slot(s) * a.G + h) * 2));
    m = warp_max_xor(m, 16, 1);
    float l = 0.f;
    for (int s = lane; s < n; s += 32) {
      const float ms = __ldcg(a.part_ml + (slot(s) * a.G + h) * 2);
      const float w = ms == -INFINITY ? 0.f : exp2f(ms - m);
      w_s[s * 8 + h] = w;
      l = fmaf(w, __ldcg(a.part_ml + (slot(s) * a.G + h) * 2 + 1), l);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      l_h[h] = l;
      if (a.lse != nullptr) a.lse[head0 + h] = (m + log2f(l)) * 0.69314718055994531f;
    }
  }
  __syncthreads();
  T* out = static_cast<T*>(a.out);
  for (int i = threadIdx.x; i < a.G * (D / 2); i += NT) {
    const int h = i / (D / 2), c = (i % (D / 2)) * 2;
    float o0 = 0.f, o1 = 0.f;
    for (int s0 = 0; s0 < n; s0 += 16) {
      float2 x[16];
#pragma unroll
      for (int u = 0; u < 16; ++u)
        if (s0 + u < n)
          x[u] = __ldcg(reinterpret_cast<const float2*>(a.part_o + (slot(s0 + u) * a.G + h) * D + c));
#pragma unroll
      for (int u = 0; u < 16; ++u)
        if (s0 + u < n) {
          const float w = w_s[(s0 + u) * 8 + h];
          o0 = fmaf(w, x[u].x, o0);
          o1 = fmaf(w, x[u].y, o1);
        }
    }
    const float inv = 1.f / l_h[h];
    out[(head0 + h) * D + c] = Dt<T>::from_f(o0 * inv);
    out[(head0 + h) * D + c + 1] = Dt<T>::from_f(o1 * inv);
  }
}

// A value as the sum of PARTS bf16 numbers (the first is its rounding, each
// next one the rounding of what is left).
template <int PARTS>
__device__ __forceinline__ void bf16_parts(float x, float (&p)[PARTS]) {
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    p[i] = __bfloat162float(__float2bfloat16_rn(x));
    x -= p[i];
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kKv4Warps * 32, sizeof(T) == 2 ? 2 : 1)
    kv4_attend_kernel(Kv4K a) {
  using C = Kv4Cfg<D>;
  constexpr int PARTS = sizeof(T) == 2 ? 1 : 3;    // bf16 parts of q and of p * scale
  constexpr int NG = D / kKv4Group;
  constexpr int NW = kKv4Warps, ST = kKv4Stages, REC = C::kRec;
  constexpr float kUp = 18446744073709551616.f;                 // 2^64
  constexpr float kDown = 5.9029581035870565e+20f;              // 2^69
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[NW][ST];
  __shared__ long long s_total, s_row_start;
  __shared__ int s_row, s_last;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) &
                                             ~static_cast<uintptr_t>(127));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, cq = lane & 3;
  if (lane == 0) {
#pragma unroll
    for (int st = 0; st < ST; ++st) mbar_init(&bars[warp][st], 1);
    fence_mbar_init();
  }
  // everything read below may come from the kernel before this one
  grid_dependency_wait();
  if (warp == 0) {
    long long total, start;
    int row;
    kv4_find(a, -1, total, row, start);
    const long long most = (total + kKv4MinBlocks - 1) / kKv4MinBlocks;
    const int n = static_cast<int>(most < gridDim.x ? most : gridDim.x);
    if (static_cast<int>(blockIdx.x) < n)
      kv4_find(a, kv4_cut(total, n, blockIdx.x), total, row, start);
    if (lane == 0) { s_total = total; s_row = row; s_row_start = start; }
  }
  if (a.lens != nullptr && blockIdx.x == 0)
    for (int b = threadIdx.x; b < a.B; b += NW * 32)
      if (row_len_bad(a.lens, a.len, b)) raise_error(a.ctrl, kErrBadIndex);
  __syncthreads();
  const long long total = s_total;
  const long long most = (total + kKv4MinBlocks - 1) / kKv4MinBlocks;
  const int ctas = static_cast<int>(most < gridDim.x ? most : gridDim.x);
  if (static_cast<int>(blockIdx.x) >= ctas) return;
  const long long part0 = kv4_cut(total, ctas, blockIdx.x);
  const long long part1 = kv4_cut(total, ctas, blockIdx.x + 1);
  int row = s_row;
  long long row_start = s_row_start;
  uint8_t* my_ring = ring + warp * ST * REC;
  uint32_t issued = 0, used = 0;                  // records of this warp's ring, over all pieces
  bool ok = true;

  for (long long x = part0; x < part1;) {
    // ---- the piece [x, x_end) of (row, head) g
    int m_row = kv4_row_blocks(a, row);
    while (x >= row_start + static_cast<long long>(m_row) * a.H) {
      row_start += static_cast<long long>(m_row) * a.H;
      m_row = kv4_row_blocks(a, ++row);
    }
    const int g = static_cast<int>((x - row_start) / m_row);
    const long long u0 = row_start + static_cast<long long>(g) * m_row, u1 = u0 + m_row;
    const long long x_end = u1 < part1 ? u1 : part1;
    const int i0 = static_cast<int>(x - u0), i1 = static_cast<int>(x_end - u0);
    const int64_t bh = static_cast<int64_t>(row) * a.H + g;
    const int64_t len_r = row_len(a.lens, a.len, row);
    const int blocks_r = static_cast<int>((len_r + kBlock - 1) / kBlock);
    const int32_t* selp = a.sel ? a.sel + bh * a.n_sel : nullptr;
    const uint8_t* base = a.kv4 + bh * a.Mmax * REC;
    const int64_t head0 = static_cast<int64_t>(row) * a.Hq + g * a.G;
    const int span = i1 - i0;
    const int count = span > warp ? (span - warp + NW - 1) / NW : 0;
    // this warp's k-th block is number i0 + warp + k NW of the list; lane u
    // holds the ids of blocks 32 w + u of its own sequence
    int ids = -1;
    auto load_ids = [&](int k0) {
      const int k = k0 + lane;
      ids = -1;
      if (k < count) {
        const int i = i0 + warp + k * NW;
        const int j = selp ? __ldg(selp + i) : i;
        ids = j >= 0 && j < blocks_r ? j : -1;
      }
    };
    // the blocks copied run ST ahead of those in use: ids holds the 32 ids
    // around the former, ids_now those around the latter
    load_ids(0);
    int ids_now = ids;
    auto issue = [&](int k) {                     // whole warp
      const int j = __shfl_sync(0xffffffffu, ids, k & 31);
      if (lane == 0) {
        fence_proxy_async_smem();                 // the stage's last reads precede the copy
        uint64_t* bar = &bars[warp][issued % ST];
        mbar_arrive_expect_tx(bar, REC);
        // (a bad id still fills the stage, with block 0)
        bulk_load(my_ring + (issued % ST) * REC, base + static_cast<int64_t>(j < 0 ? 0 : j) * REC,
                  REC, bar);
      }
      ++issued;
    };
    for (int k = 0; k < count && k < ST; ++k) issue(k);

    // ---- q fragments and the group sums of q
    uint32_t qb[PARTS][NG * 4][2];
    float qs0[NG], qs1[NG];
    {
      const T* qg = static_cast<const T*>(a.q) + head0 * D;
#pragma unroll
      for (int g2 = 0; g2 < NG; ++g2) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float f[8];
          if (gq < a.G) {
            const T* p = qg + gq * D + g2 * 64 + cq * 16 + j * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = Dt<T>::to_f(p[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) sum += f[i];
          float part[8][PARTS];
#pragma unroll
          for (int i = 0; i < 8; ++i) bf16_parts<PARTS>(f[i] * kUp, part[i]);
          // word j: product step 2j takes nibbles 0, 4 and 1, 5 (the latter
          // read 16 times too large), step 2j + 1 nibbles 2, 6 and 3, 7
#pragma unroll
          for (int p = 0; p < PARTS; ++p)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              qb[p][g2 * 4 + 2 * j + s][0] = pack_bf16x2(part[2 * s][p], part[2 * s + 4][p]);
              qb[p][g2 * 4 + 2 * j + s][1] =
                  pack_bf16x2(part[2 * s + 1][p] * 0.0625f, part[2 * s + 5][p] * 0.0625f);
            }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        // heads 2 cq and 2 cq + 1 of the result layout, in the sums' scale
        qs0[g2] = __shfl_sync(0xffffffffu, sum, 8 * cq) / kDown;
        qs1[g2] = __shfl_sync(0xffffffffu, sum, 8 * cq + 4) / kDown;
      }
    }
    const float to_log2 = a.scale_log2 * kDown;

    float o[NG * 4][4], zo0[NG], zo1[NG];
#pragma unroll
    for (int i = 0; i < NG * 4; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) { zo0[i] = 0.f; zo1[i] = 0.f; }
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    for (int k = 0; k < count; ++k) {
      if ((k & 31) == 0) ids_now = ids;           // (loaded when block k was issued)
      const int st = used % ST;
      const bool arrived = mbar_wait_bounded(&bars[warp][st], (used / ST) & 1, a.ctrl);
      if (!__all_sync(0xffffffffu, arrived)) { ok = false; break; }
      ++used;
      const int j = __shfl_sync(0xffffffffu, ids_now, k & 31);
      const uint8_t* rec = my_ring + st * REC;
      uint4 kw[NG], vw[NG];
      uint2 meta[2][NG];                          // [token half][group]: {ks kz}, {vs vz}
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        kw[i] = *reinterpret_cast<const uint4*>(rec + i * 512 + lane * 16);
        vw[i] = *reinterpret_cast<const uint4*>(rec + kv4_code_bytes(D) + i * 512 + lane * 16);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NG; ++i)
          meta[h][i] = *reinterpret_cast<const uint2*>(rec + 2 * kv4_code_bytes(D) +
                                                       ((gq * 2 + h) * NG + i) * 8);
      __syncwarp();                               // every lane has read the record
      if (k + ST < count) {
        if (((k + ST) & 31) == 0) load_ids(k + ST);
        issue(k + ST);
      }
      if (j < 0) {                                // skip the block, report it
        if (lane == 0) raise_error(a.ctrl, kErrBadIndex);
        continue;
      }
      // ---- logits of tokens gq, gq + 8 and heads 2 cq, 2 cq + 1
      float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t wa[2] = {kw[i].x, kw[i].y}, wb[2] = {kw[i].z, kw[i].w};
#pragma unroll
        for (int w = 0; w < 2; ++w) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t x0 = wa[w] >> (8 * s), x1 = wb[w] >> (8 * s);
            const uint32_t af[4] = {x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u,
                                    x1 & 0x00f000f0u};
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
              mma_bf16_16816(acc, af, qb[p][i * 4 + 2 * w + s][0], qb[p][i * 4 + 2 * w + s][1]);
          }
        }
        const float ka = bf16_lo(meta[0][i].x), za = bf16_hi(meta[0][i].x);
        const float kb = bf16_lo(meta[1][i].x), zb = bf16_hi(meta[1][i].x);
        s0 = fmaf(ka, acc[0], fmaf(za, qs0[i], s0));
        s1 = fmaf(ka, acc[1], fmaf(za, qs1[i], s1));
        s2 = fmaf(kb, acc[2], fmaf(zb, qs0[i], s2));
        s3 = fmaf(kb, acc[3], fmaf(zb, qs1[i], s3));
      }
      s0 *= to_log2; s1 *= to_log2; s2 *= to_log2; s3 *= to_log2;
      // tokens past the end: weight 0, and neither their codes (any four
      // bits are finite) nor their scales (masked below) reach an output
      const int64_t t_lo = static_cast<int64_t>(j) * kBlock + gq;
      const bool va = t_lo < len_r, vb = t_lo + 8 < len_r;
      if (!va) { s0 = -INFINITY; s1 = -INFINITY; }
      if (!vb) { s2 = -INFINITY; s3 = -INFINITY; }
      // the reference moves only when some token exceeds it by 2^8: p, the
      // sums and the outputs stay far inside fp32, and most blocks rescale
      // nothing
      const float b0 = fmaxf(s0, s2), b1 = fmaxf(s1, s3);
      if (__any_sync(0xffffffffu, b0 > m0 + 8.f || b1 > m1 + 8.f)) {
        const float n0 = fmaxf(m0, warp_max_xor(b0, 16, 4));
        const float n1 = fmaxf(m1, warp_max_xor(b1, 16, 4));
        const float al0 = m0 == -INFINITY ? 0.f : exp2f(m0 - n0);
        const float al1 = m1 == -INFINITY ? 0.f : exp2f(m1 - n1);
        m0 = n0; m1 = n1;
        l0 *= al0; l1 *= al1;
#pragma unroll
        for (int i = 0; i < NG * 4; ++i) {
          o[i][0] *= al0; o[i][2] *= al0;
          o[i][1] *= al1; o[i][3] *= al1;
        }
#pragma unroll
        for (int i = 0; i < NG; ++i) { zo0[i] *= al0; zo1[i] *= al1; }
      }
      const float p0 = exp2f(s0 - m0), p1 = exp2f(s1 - m1);
      const float p2 = exp2f(s2 - m0), p3 = exp2f(s3 - m1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      // ---- values
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const float sa = va ? bf16_lo(meta[0][i].y) * kUp : 0.f;
        const float sb = vb ? bf16_lo(meta[1][i].y) * kUp : 0.f;
        const float za = va ? bf16_hi(meta[0][i].y) : 0.f;
        const float zb = vb ? bf16_hi(meta[1][i].y) : 0.f;
        zo0[i] = fmaf(p0, za, fmaf(p2, zb, zo0[i]));
        zo1[i] = fmaf(p1, za, fmaf(p3, zb, zo1[i]));
        uint32_t pb[PARTS][2];
        {
          float e0[PARTS], e1[PARTS], e2[PARTS], e3[PARTS];
          if constexpr (PARTS == 1) {
            e0[0] = p0 * sa; e1[0] = p1 * sa; e2[0] = p2 * sb; e3[0] = p3 * sb;
          } else {
            bf16_parts<PARTS>(p0 * sa, e0);
            bf16_parts<PARTS>(p1 * sa, e1);
            bf16_parts<PARTS>(p2 * sb, e2);
            bf16_parts<PARTS>(p3 * sb, e3);
          }
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            pb[p][0] = movmatrix_trans(pack_bf16x2(e0[p], e1[p]));
            pb[p][1] = movmatrix_trans(pack_bf16x2(e2[p], e3[p]));
          }
        }
        const uint32_t w4[4] = {vw[i].x, vw[i].y, vw[i].z, vw[i].w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t x0 = w4[m], x1 = w4[m] >> 8;
          const uint32_t af[4] = {x0 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x000f000fu,
                                  x1 & 0x00f000f0u};
#pragma unroll
          for (int p = 0; p < PARTS; ++p) mma_bf16_16816(o[i * 4 + m], af, pb[p][0], pb[p][1]);
        }
      }
    }
    if (!ok) {
      // drain this warp's copies in flight (bounded)
      while (used != issued) {
        (void)mbar_wait_bounded(&bars[warp][used % ST], (used / ST) & 1, a.ctrl);
        ++used;
      }
    }
    if (x_end == part1) grid_launch_dependents();
    if (!__syncthreads_and(ok)) return;

    // ---- the warps' results, merged in shared memory (the ring is idle)
    l0 += __shfl_xor_sync(0xffffffffu, l0, 4);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 8);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 16);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 4);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 8);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 16);
#pragma unroll
    for (int i = 0; i < NG; ++i) {
#pragma unroll
      for (int m = 4; m <= 16; m <<= 1) {
        zo0[i] += __shfl_xor_sync(0xffffffffu, zo0[i], m);
        zo1[i] += __shfl_xor_sync(0xffffffffu, zo1[i], m);
      }
    }
    constexpr int OR = merge_row(D);
    float* sm = reinterpret_cast<float*>(ring);
    float* sm_o = sm;                             // [NW][8][OR]
    float* sm_m = sm + NW * 8 * OR;               // [NW][8]
    float* sm_l = sm_m + NW * 8;
    const int h0 = 2 * cq, h1 = 2 * cq + 1;
    if (gq == 0) {
      sm_m[warp * 8 + h0] = m0; sm_l[warp * 8 + h0] = l0;
      sm_m[warp * 8 + h1] = m1; sm_l[warp * 8 + h1] = l1;
    }
    if (h0 < a.G) {
      // rows gq + 8 hold codes read 16 times too large
#pragma unroll
      for (int i = 0; i < NG * 4; ++i) {
        const int ch = i * 16 + gq;
        sm_o[(warp * 8 + h0) * OR + ch] = fmaf(o[i][0], kDown, zo0[i / 4]);
        sm_o[(warp * 8 + h1) * OR + ch] = fmaf(o[i][1], kDown, zo1[i / 4]);
        sm_o[(warp * 8 + h0) * OR + ch + 8] = fmaf(o[i][2], kDown * 0.0625f, zo0[i / 4]);
        sm_o[(warp * 8 + h1) * OR + ch + 8] = fmaf(o[i][3], kDown * 0.0625f, zo1[i / 4]);
      }
    }
    __syncthreads();
    const bool whole = x == u0 && x_end == u1;
    // slot 0: the part's first piece, slot 1: its last one
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (x == part0 ? 0 : 1);
    T* out = static_cast<T*>(a.out);
    for (int i = threadIdx.x; i < a.G * D; i += NW * 32) {
      const int h = i / D, ch = i % D;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) mx = fmaxf(mx, sm_m[w * 8 + h]);
      float v = 0.f, l = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float mw = sm_m[w * 8 + h];
        const float sc = mw == -INFINITY ? 0.f : exp2f(mw - mx);
        v = fmaf(sc, sm_o[(w * 8 + h) * OR + ch], v);
        l = fmaf(sc, sm_l[w * 8 + h], l);
      }
      if (whole) {
        out[(head0 + h) * D + ch] = Dt<T>::from_f(v / l);
        if (a.lse != nullptr && ch == 0)
          a.lse[head0 + h] = (mx + log2f(l)) * 0.69314718055994531f;
      } else {
        a.part_o[(slot * a.G + h) * D + ch] = v;
        if (ch == 0) {
          a.part_ml[(slot * a.G + h) * 2] = mx;
          a.part_ml[(slot * a.G + h) * 2 + 1] = l;
        }
      }
    }
    __syncthreads();
    if (!whole) {
      if (threadIdx.x == 0) {
        const int parts = kv4_owner(total, ctas, u1 - 1) - kv4_owner(total, ctas, u0) + 1;
        s_last = atomic_add_acq_rel(a.counters + bh, 1) == parts - 1;
      }
      __syncthreads();
      if (s_last) {
        kv4_merge<T, D>(a, sm, total, ctas, u0, u1, head0);
        if (threadIdx.x == 0) a.counters[bh] = 0;
      }
      __syncthreads();
    }
    // the next piece's copies overwrite what was just read here
    fence_proxy_async_smem();
    __syncthreads();
    x = x_end;
  }
}

template <typename T, int D>
static cudaError_t kv4_attend_t(const Shape& s, const Kv4K& k, int ctas, cudaStream_t st) {
  using C = Kv4Cfg<D>;
  static std::atomic<bool> attr_set[64];   // per device; launches may come from several host threads
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kv4_attend_kernel<T, D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kKv4Warps * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_attend_kernel<T, D>, k);
}

// CTAs of a launch: one wave (two CTAs per SM for bf16, one for fp32), at most
// kMaxSplits per (row, KV head), none with less than kKv4MinBlocks blocks.
int kv4_ctas(const Shape& s, int64_t blocks_bound, int num_sms) {
  const int64_t units = static_cast<int64_t>(s.B) * s.H;
  int64_t n = static_cast<int64_t>(num_sms) * (s.bf16 ? 2 : 1);
  if (n > kKv4MaxCtas) n = kKv4MaxCtas;
  if (n > units * kMaxSplits) n = units * kMaxSplits;
  const int64_t most = (units * blocks_bound + kKv4MinBlocks - 1) / kKv4MinBlocks;
  return static_cast<int>(n < most ? n : most);
}

cudaError_t launch_kv4_attend(const Shape& s, const Kv4Args& a, cudaStream_t st) {
  Kv4K k{};
  k.q = a.q; k.kv4 = static_cast<const uint8_t*>(a.kv4); k.sel = a.sel; k.lens = a.lens;
  k.part_o = a.part_o; k.part_ml = a.part_ml; k.counters = a.counters; k.ctrl = a.ctrl;
  k.out = a.out; k.lse = a.lse; k.len = a.len; k.r = a.r; k.n_min = a.n_min;
  k.B = s.B; k.H = s.H; k.G = s.G; k.Hq = s.Hq; k.Mmax = s.Mmax; k.n_sel = a.n_sel;
  k.scale_log2 = a.scale * 1.4426950408889634f;
  if (s.bf16)
    return s.D == 128 ? kv4_attend_t<__nv_bfloat16, 128>(s, k, a.ctas, st)
                      : kv4_attend_t<__nv_bfloat16, 64>(s, k, a.ctas, st);
  return s.D == 128 ? kv4_attend_t<float, 128>(s, k, a.ctas, st)
                    : kv4_attend_t<float, 64>(s, k, a.ctas, st);
}

}  // namespace resa
