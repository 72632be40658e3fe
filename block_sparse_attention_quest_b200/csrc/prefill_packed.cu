// Causal attention over packed prompts of different lengths on the 5th
// generation tensor cores, filling the caches and block descriptors that
// decoding starts from.
//
//   out_i = sum_{t <= i} softmax_t(scale q_i . k_t) v_t   inside each sequence
//
// Sequence b is tokens starts[b] .. starts[b + 1] - 1 of q, k and v. A CTA
// takes NT = 2 (or 1) tiles of 128 rows of one sequence: row = query * Gt +
// head, of 128 / Gt consecutive queries of Gt query heads that share a KV head
// (Gt: the largest power of two that divides the group), which is how q lies
// in memory; and walks the key tiles of 128 tokens up to its last query. Both
// tiles use every K and V tile that arrives, so a tile is read from L2 once
// for 256 rows. Bound: the tensor cores and, equally, the exponential unit
// (2 x 128 x 128 exponentials take 2048 cycles of an SM, as do the four 128^3
// products).
//
// NT + 1 warpgroups:
//   NT softmax warpgroups, one tile each, one row per thread (= TMEM lane): S
//             is read into registers whole, the row maximum moves its
//             reference only when it grows by more than 2^8 (O is rescaled in
//             TMEM then), and P = 2^(s - m) goes back as bf16 over the S
//             columns, as the A operand of the second product;
//   4 warps:  one thread issues the products. For each tile the next S is
//             issued right behind the O product that reads the previous P
//             from the same columns: the tensor pipe runs them in order. Its
//             completion therefore also says that O may be rescaled.
//             One thread issues the TMA copies: Q, then K and V tiles through
//             a ring of 128-token slots. Two warps copy this CTA's own tokens
//             of K and V from the packed tensors to the caches and write their
//             block descriptors (one CTA per KV head).
// While one tile's softmax runs, the other tile's products do.
//
// Measured (B200, 32/8 heads, d = 128): 32768 tokens in sequences of 1822,
// 16384 and 14562 tokens 3580 us = 1108 TFLOP/s, tensor pipe active 63 % of
// the cycles, the SMs at about 1.34 GHz under the power cap (cuBLAS holds 1390
// TFLOP/s there); 24 sequences of 0 to 1250 tokens 37 us.
//
// Rows of a key tile past the sequence's end belong to other sequences: their
// scores are masked and their V rows zeroed in shared memory, so nothing of
// another sequence (an infinity times 0) reaches an output.
#include "launch.h"
#include "tc.cuh"

namespace resa {

struct PackedK {
  __nv_bfloat16* out;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* starts;      // [B + 1]
  __nv_bfloat16* k_cache;     // or nullptr
  __nv_bfloat16* v_cache;
  __nv_bfloat16* desc;        // or nullptr
  Ctrl* ctrl;
  int64_t L_max;
  int Mmax;
  int B, T, longest, Hq, H, G;
  int gs;                     // Gt = 1 << gs
  float scale_log2;
};

// NT: 128-row tiles per CTA. Two, one CTA per SM, for long sequences; one, two
// CTAs per SM, for short ones, whose CTAs spend most of their time on the way
// to the first product and from the last (about 7 us; the other CTA's work
// fills it).
template <int D, int NT>
struct PackedCfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfBytes = 128 * 128;          // [128 rows][64 bf16]
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kSlots = NT == 2 || D == 64 ? 5 : 2;
  // (never room for more CTAs than have their TMEM columns: one would wait)
  static constexpr int kLeast = NT == 2 ? 116 * 1024 : 78 * 1024;
  static constexpr int kNeed = (NT + kSlots) * kTileBytes + 1024;
  static constexpr int kSmem = kNeed > kLeast ? kNeed : kLeast;
  static constexpr uint32_t kTmemCols = 256 * NT;        // S and O of each tile, 128 columns each
  // The warps start with 168 registers each (NT = 2, twelve warps) or 128; the
  // softmax warps, which hold a row of S, take 200, the last warpgroup leaves
  // them (2 * 200 + 104 = 3 * 168, 200 + 56 = 2 * 128).
  static constexpr int kThreads = (NT + 1) * 128;
  static constexpr int kRegsSoftmax = 200, kRegsOther = NT == 2 ? 104 : 56;
};

// The ring: copy n (K of tile n / 2 where n is even, V where it is odd) goes to
// slot n % slots. The slot's last tile, copy n - slots, is given back with the
// one before or after it: K 0 alone first (give-back 0), then V t and K t + 1
// together (give-back t + 1). Which give-back copy n waits for, -1 for none:
__host__ __device__ constexpr int packed_waits_for(int n, int slots) {
  return n >= slots && (n == slots || (n - slots) % 2 == 1) ? (n - slots + 1) / 2 : -1;
}
// and how many of them the copies of n_tiles tiles wait for. No other is made:
// its arrival could reach a barrier of a CTA that has ended.
__host__ __device__ constexpr int packed_give_backs(int n_tiles, int slots) {
  return 2 * n_tiles > slots ? (2 * n_tiles - slots) / 2 + 1 : 0;
}
constexpr bool packed_ring_agrees(int slots) {
  for (int tiles = 1; tiles < 40; ++tiles) {
    int next = 0;
    for (int n = 0; n < 2 * tiles; ++n) {
      const int f = packed_waits_for(n, slots);
      if (f >= 0 && f != next++) return false;
      // the give-back that frees the slot is waited for by then
      if (n >= slots && (n - slots + 1) / 2 >= next) return false;
    }
    if (next != packed_give_backs(tiles, slots)) return false;
  }
  return true;
}
static_assert(packed_ring_agrees(2) && packed_ring_agrees(5), "ring of K and V tiles");

__device__ __forceinline__ float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// bounds of sequence b, and whether the starts given are out of order or range
struct SeqBounds {
  int begin, len;
  bool bad;
};
__device__ __forceinline__ SeqBounds seq_bounds(const PackedK& a, int b) {
  const int s0 = a.starts[b], s1 = a.starts[b + 1];
  SeqBounds r;
  r.begin = s0 < 0 ? 0 : (s0 > a.T ? a.T : s0);
  const int end = s1 < r.begin ? r.begin : (s1 > a.T ? a.T : s1);
  r.len = end - r.begin > a.longest ? a.longest : end - r.begin;
  r.bad = r.begin != s0 || r.begin + r.len != s1;
  return r;
}

// V, or K, rows [t0, t0 + n) of a sequence to its cache row, with K the
// descriptors of their blocks (t0 is a multiple of 16); one warp each.
template <int D>
__device__ __forceinline__ void fill_cache(const PackedK& a, bool is_v, int b, int begin, int g,
                                           int t0, int n) {
  constexpr int CPR = D / 8, TPP = 32 / CPR, NP = kBlock / TPP;
  const int lane = threadIdx.x & 31, chunk = lane % CPR, r0 = lane / CPR;
  const int64_t bh = static_cast<int64_t>(b) * a.H + g;
  const int64_t stride = static_cast<int64_t>(a.H) * D;
  __nv_bfloat16* cache = is_v ? a.v_cache : a.k_cache;
  if (cache == nullptr && (is_v || a.desc == nullptr)) return;
  const __nv_bfloat16* src =
      (is_v ? a.v : a.k) + (static_cast<int64_t>(begin + t0) * a.H + g) * D + chunk * 8;
  __nv_bfloat16* dst = cache + (bh * a.L_max + t0) * D + chunk * 8;
#pragma unroll 1
  for (int j = 0; j < n; j += kBlock) {
    const int valid = n - j < kBlock ? n - j : kBlock;
    uint4 x[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (r0 + i * TPP < valid) x[i] = ldg16(src + (j + r0 + i * TPP) * stride);
    if (cache != nullptr) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (r0 + i * TPP < valid)
          *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(j + r0 + i * TPP) * D) = x[i];
    }
    if (is_v || a.desc == nullptr) continue;
    // (bf16 minima and maxima, two at a time: exact)
    uint32_t mn[4], mx[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) { mn[e] = 0x7f807f80u; mx[e] = 0xff80ff80u; }
    auto fold = [&](uint32_t (&lo)[4], uint32_t (&hi)[4], const uint32_t (&u)[4], const uint32_t (&v)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lo[e] = bf16x2_min(lo[e], u[e]);
        hi[e] = bf16x2_max(hi[e], v[e]);
      }
    };
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (r0 + i * TPP < valid) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        fold(mn, mx, w, w);
      }
#pragma unroll
    for (int m = CPR; m < 32; m <<= 1) {
      uint32_t u[4], v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = __shfl_xor_sync(0xffffffffu, mn[e], m);
        v[e] = __shfl_xor_sync(0xffffffffu, mx[e], m);
      }
      fold(mn, mx, u, v);
    }
    if (lane < CPR) {
      __nv_bfloat16* d = a.desc + (bh * a.Mmax + (t0 + j) / kBlock) * 2 * D + chunk * 8;
      *reinterpret_cast<uint4*>(d) = make_uint4(mn[0], mn[1], mn[2], mn[3]);
      *reinterpret_cast<uint4*>(d + D) = make_uint4(mx[0], mx[1], mx[2], mx[3]);
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__((PackedCfg<D, NT>::kThreads), (NT == 2 ? 1 : 2))
    prefill_packed_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, PackedK a) {
  using C = PackedCfg<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_q[NT], bar_full[C::kSlots], bar_free[3];
  __shared__ __align__(8) uint64_t bar_s[NT], bar_p[NT][2], bar_o[NT];   // [tile], P: [tile][half of the keys]
  __shared__ uint32_t tmem_base_sh;
  __shared__ bool s_disorder;
  __shared__ int s_seq, s_block, s_tot[C::kThreads / 32];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  auto sQ = [&](int w) { return base + w * C::kTileBytes; };
  auto slot = [&](int n) { return base + (NT + n % C::kSlots) * C::kTileBytes; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Gt = 1 << a.gs, QT = 128 >> a.gs, QB = NT * QT;   // queries per tile, per CTA
  const int qbs = 7 - a.gs + (NT - 1);            // QB = 1 << qbs
  const int n_hg = a.Hq >> a.gs;
  const int hg = blockIdx.x % n_hg, x = blockIdx.x / n_hg;

  // which sequence and which of its query blocks (the last ones, which see the
  // most keys, first): one sequence per thread, a scan of their block counts
  if (threadIdx.x == 0) { s_seq = -1; s_disorder = false; }
  for (int b0 = 0, run = 0; b0 < a.B; b0 += C::kThreads) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < a.B) {
      const SeqBounds sb = seq_bounds(a, b);
      n = (sb.len + QB - 1) >> qbs;
      if (blockIdx.x == 0 && sb.bad) raise_error(a.ctrl, kErrBadIndex);
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();                              // (the last round's totals are read)
    if (lane == 31) s_tot[warp] = inc;
    if (b < a.B && a.starts[b + 1] < a.starts[b]) s_disorder = true;
    __syncthreads();
    int before = run, all = run;
#pragma unroll
    for (int i = 0; i < C::kThreads / 32; ++i) {
      before += i < warp ? s_tot[i] : 0;
      all += s_tot[i];
    }
    if (x >= before + inc - n && x < before + inc) {
      s_seq = b;
      s_block = before + inc - 1 - x;
    }
    run = all;
    if (run > x && blockIdx.x != 0) break;        // (the first CTA reports every bad entry)
  }
  __syncthreads();
  const int b = s_seq;
  if (b < 0) return;                              // more CTAs than query blocks
  const SeqBounds sb = seq_bounds(a, b);
  // a sequence that begins below an earlier start would share tokens, and the
  // rows of their outputs, with a sequence before it: left out
  if (s_disorder) {
    int top = 0;
#pragma unroll 1
    for (int i = 0; i < b; ++i) top = max(top, a.starts[i]);
    if (top > sb.begin) return;
  }
  const int q0 = s_block * QB;
  const int nq = sb.len - q0 < QB ? sb.len - q0 : QB;
  const int g = (hg << a.gs) / a.G;                  // KV head
  // key tiles of A and of B (none without queries)
  const int nt_a = (q0 + (nq < QT ? nq : QT) - 1) / 128 + 1;
  const int nt_b = NT > 1 && nq > QT ? (q0 + nq - 1) / 128 + 1 : 0;
  const int n_tiles = nt_b > nt_a ? nt_b : nt_a;

  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 0; w < NT; ++w) {
      mbar_init(&bar_q[w], 1);
      mbar_init(&bar_s[w], 1);
      mbar_init(&bar_p[w][0], 128);
      mbar_init(&bar_p[w][1], 128);
      mbar_init(&bar_o[w], 1);
    }
#pragma unroll
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&bar_full[i], 1);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) mbar_init(&bar_free[i], 1);
    fence_mbar_init();
  }
  if (warp == 4 * NT) tc::alloc(&tmem_base_sh, C::kTmemCols);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_base_sh;
  auto tS = [&](int w) { return tmem + 128u * w; };
  auto tO = [&](int w) { return tmem + 128u * NT + 128u * w; };

  if (warp >= 4 * NT) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsOther));
    if (warp == 4 * NT + 1) {
      // ---------------------------------------------------------------- copies
      if (lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        auto load_q = [&](int w) {
          mbar_arrive_expect_tx(&bar_q[w], C::kTileBytes);
#pragma unroll
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_3d(sQ(w) + hf * C::kHalfBytes, &tmQ, hf * 64, hg << a.gs, sb.begin + q0 + w * QT,
                        &bar_q[w]);
        };
        load_q(0);
        int n = 0;                                   // copy n: K (even) or V (odd) of tile n / 2
        bool ok = true;
        for (; n < 2 * n_tiles; ++n) {
          const int i = n % C::kSlots;
          const int f = packed_waits_for(n, C::kSlots);
          if (f >= 0 && !(ok = mbar_wait_bounded(&bar_free[f % 3], (f / 3) & 1, a.ctrl))) break;
          mbar_arrive_expect_tx(&bar_full[i], C::kTileBytes);
          const CUtensorMap* map = n & 1 ? &tmV : &tmK;
#pragma unroll
          for (int hf = 0; hf < C::kHalves; ++hf)
            tma_load_3d(slot(n) + hf * C::kHalfBytes, map, hf * 64, g, sb.begin + (n >> 1) * 128,
                        &bar_full[i]);
          if (NT > 1 && n == 0 && nt_b > 0) load_q(NT - 1);
        }
        if (!ok) {
          // the copies in flight end (within the bound) before this CTA does
          for (int w = 0; w < (nt_b > 0 ? 2 : 1); ++w)
            (void)mbar_wait_bounded(&bar_q[w], 0, a.ctrl);
          for (int m = n >= C::kSlots ? n - C::kSlots : 0; m < n; ++m)
            (void)mbar_wait_bounded(&bar_full[m % C::kSlots], (m / C::kSlots) & 1, a.ctrl);
        }
      }
      __syncwarp();
    } else if (warp == 4 * NT) {
      // -------------------------------------------------------------- products
      if (lane == 0) {
        constexpr uint32_t idS = tc::idesc_bf16(128, 128, false);
        constexpr uint32_t idO = tc::idesc_bf16(128, D, true);
        constexpr uint32_t hi = tc::desc_hi(1024);
        constexpr uint32_t kTileLo = C::kTileBytes >> 4, kHalfLo = C::kHalfBytes >> 4;
        const uint32_t q_lo = tc::desc_lo(smem_u32(sQ(0)), 16);
        const uint32_t k_lo = tc::desc_lo(smem_u32(slot(0)), 16);
        const uint32_t v_lo = tc::desc_lo(smem_u32(slot(0)), C::kHalfBytes);
        // the ring slot in use and its phase; slots are taken in the order they
        // are filled: K 0, V 0, K 1, V 1, ...
        auto qk = [&](int w, uint32_t i) {
          const uint32_t ql = q_lo + w * kTileLo, kl = k_lo + i * kTileLo, d = tS(w);
          tc::mma_ss_lo<false>(d, ql, kl, hi, idS);
#pragma unroll
          for (int kk = 1; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kHalfLo + (kk & 3) * 2;
            tc::mma_ss_lo<true>(d, ql + off, kl + off, hi, idS);
          }
          tc::commit(&bar_s[w]);
        };
        auto pv = [&](int w, int half, uint32_t i, uint32_t acc) {   // 64 keys
          const uint32_t vl = v_lo + i * kTileLo + half * 512, d = tO(w), p = tS(w) + 32u * half;
          tc::mma_ts_lo(d, p, vl, hi, idO, acc);
#pragma unroll
          for (int kk = 1; kk < 4; ++kk) tc::mma_ts_lo(d, p + 8u * kk, vl + kk * 128, hi, idO, 1u);
        };
        bool ok = mbar_wait_bounded(&bar_full[0], 0, a.ctrl);
        for (int w = 0; ok && w < (nt_b > 0 ? 2 : 1); ++w) {
          if (!(ok = mbar_wait_bounded(&bar_q[w], 0, a.ctrl))) break;
          tc::fence_after_sync();
          qk(w, 0);
        }
        const int backs = packed_give_backs(n_tiles, C::kSlots);
        if (ok && backs > 0) tc::commit(&bar_free[0]);
        uint32_t f = 1;                              // give-back t + 1 on barrier f
        uint32_t i = 1, ph = 0;                      // slot and phase of V of tile t
        for (int t = 0; ok && t < n_tiles; ++t) {
          uint32_t i2 = i + 1, ph2 = ph;             // of K of tile t + 1
          if (i2 == C::kSlots) { i2 = 0; ph2 ^= 1u; }
          if (!(ok = mbar_wait_bounded(&bar_full[i], ph, a.ctrl))) break;
          bool have_k = false;
#pragma unroll
          for (int w = 0; w < NT; ++w) {
            const int nt = w == 0 ? nt_a : nt_b;
            if (!ok || t >= nt) continue;
            if (!(ok = mbar_wait_bounded(&bar_p[w][0], t & 1, a.ctrl))) continue;
            tc::fence_after_sync();
            pv(w, 0, i, t > 0);
            if (!(ok = mbar_wait_bounded(&bar_p[w][1], t & 1, a.ctrl))) continue;
            tc::fence_after_sync();
            pv(w, 1, i, 1u);
            if (t + 1 < nt) {
              if (!have_k) {
                if (!(ok = mbar_wait_bounded(&bar_full[i2], ph2, a.ctrl))) continue;
                have_k = true;
                tc::fence_after_sync();
              }
              qk(w, i2);
            } else {
              tc::commit(&bar_o[w]);
            }
          }
          if (!ok) break;
          // both tiles have taken V of tile t and K of tile t + 1
          if (t + 1 < backs) tc::commit(&bar_free[f]);
          if (++f == 3) f = 0;
          i = i2 + 1;
          ph = ph2;
          if (i == C::kSlots) { i = 0; ph ^= 1u; }
        }
      }
      __syncwarp();
    } else if ((hg << a.gs) % a.G == 0) {
      // ------------------------------------------------- caches and descriptors
      fill_cache<D>(a, warp == 4 * NT + 3, b, sb.begin, g, q0, nq);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    // --------------------------------------------------------------- softmax
    const int w = warp >> 2;
    const int nt = w == 0 ? nt_a : nt_b;
    const int row = threadIdx.x & 127;             // TMEM lane
    const int qpos = q0 + w * QT + (row >> a.gs);     // causal limit
    const int qpos_lo = q0 + w * QT;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float sl2 = a.scale_log2;
    // reference and sum of the row; the maximum beyond which the reference moves;
    // what the weights add to s * sl2
    float m_ref = -INFINITY, l = 0.f, limit = -INFINITY, nm = 0.f;
    bool ok = true;
    for (int t = 0; t < nt; ++t) {
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bar_s[w], t & 1, a.ctrl));
      if (!ok) break;
      tc::fence_after_sync();
      float s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::ld32(tS(w) + lane_off + 32 * c, s[c]);
      tc::wait_ld();
      const int key0 = t * 128;
      if (key0 + 127 > qpos_lo) {                  // (the last tiles only)
        const int lim = qpos - key0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c * 32 + i > lim) s[c][i] = -INFINITY;
      }
      if (key0 + 128 > sb.len) {
        // V rows past the sequence's end (both tiles' threads do this: the
        // product of either may come first)
        const int n = 2 * t + 1;
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bar_full[n % C::kSlots],
                                                       (n / C::kSlots) & 1, a.ctrl));
        if (!ok) break;
        if (key0 + row >= sb.len) {
          uint8_t* vt = slot(n) + row * 128;
#pragma unroll
          for (int hf = 0; hf < C::kHalves; ++hf)
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(vt + hf * C::kHalfBytes + c * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      uint64_t sum[2] = {0ull, 0ull};
      // P of 64 keys (the chunks c0, c0 + 1) for the reference m_ref, over the
      // S columns they came from (all of S is in registers)
      auto weights = [&](int c0) {
        const uint64_t sl2_2 = f2_pack(sl2, sl2), nm_2 = f2_pack(nm, nm);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t wd[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float x0 = s[c0 + c][2 * e], x1 = s[c0 + c][2 * e + 1];
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(x0, x1), sl2_2, nm_2), p0, p1);
            p0 = ex2_fast(p0);
            p1 = ex2_fast(p1);
            sum[e & 1] = f2_add(sum[e & 1], f2_pack(p0, p1));
            wd[e] = pack_bf16x2(p0, p1);
          }
          tc::st16(tS(w) + lane_off + (c0 + c) * 16, wd);
        }
      };
      // the row maximum (eight chains of three-input maxima) moves the reference
      // when it exceeds it by 2^8: in the first tile, and rarely later
      float mp[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) mp[j] = fmaxf(s[0][j], s[2][j]);
#pragma unroll
      for (int i = 8; i < 32; ++i) mp[i & 7] = max3(mp[i & 7], s[0][i], s[2][i]);
#pragma unroll
      for (int i = 0; i < 32; ++i) mp[i & 7] = max3(mp[i & 7], s[1][i], s[3][i]);
      const float mx =
          fmaxf(max3(max3(mp[0], mp[1], mp[2]), mp[3], mp[4]), max3(mp[5], mp[6], mp[7])) * sl2;
      if (__any_sync(0xffffffffu, mx > limit)) {
        const bool need = mx > m_ref + 8.f;
        const float m_new = need ? mx : m_ref;
        const float alpha = need ? (m_ref == -INFINITY ? 0.f : ex2_fast(m_ref - m_new)) : 1.f;
        if (t > 0) {
          // (this S is complete, and the O product before it with it)
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            float o[16];
            tc::ld16(tO(w) + lane_off + c * 16, o);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= alpha;
            tc::st16f(tO(w) + lane_off + c * 16, o);
          }
          tc::wait_st();
        }
        l *= alpha;
        m_ref = m_new;
        // Far rows (see tc::kFar) come here with every tile and make s relative to
        // their reference. (A branch of its own for them, which ordinary inputs
        // never take, costs 3 % at 32K tokens.)
        const bool far = fabsf(m_ref) > tc::kFar && m_ref != -INFINITY;
        limit = far ? -INFINITY : m_ref + 8.f;
        // (a row with no visible key yet, -inf - -inf, takes weight 0)
        nm = far || m_ref == -INFINITY ? 0.f : -m_ref;
        if (__any_sync(0xffffffffu, far)) {
          const float inv = 1.f / sl2;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float rel = __fsub_rn(__fmul_rn(s[c][i], sl2), m_ref) * inv;
              s[c][i] = far ? rel : s[c][i];
            }
        }
      }
      // each half of P is handed over by itself: its products run while the
      // other half's exponentials do
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        weights(2 * half);
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(&bar_p[w][half]);
      }
      float s0, s1, s2, s3;
      f2_unpack(sum[0], s0, s1);
      f2_unpack(sum[1], s2, s3);
      l += (s0 + s1) + (s2 + s3);
    }
    if (ok && nt > 0) {
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bar_o[w], 0, a.ctrl));
      if (ok) {
        tc::fence_after_sync();
        // each warp's 32 rows through its part of its tile's query buffer (no
        // product reads it any more), 16-byte unit j of row r at j ^ (r mod 8)
        constexpr int NU = D / 8;                  // 16-byte units per row
        uint4* st = reinterpret_cast<uint4*>(sQ(w)) + (warp & 3) * 32 * NU;
        const float inv = 1.f / l;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tc::ld32(tO(w) + lane_off + c * 32, o);
          tc::wait_ld();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            st[lane * NU + ((c * 4 + k) ^ (lane & 7))] =
                make_uint4(pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv),
                           pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                           pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                           pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
        }
        __syncwarp();
        constexpr int RPI = 32 / NU;               // rows per store instruction
        const int j = lane % NU;
#pragma unroll 4
        for (int it = 0; it < 32 / RPI; ++it) {
          const int r = it * RPI + lane / NU;
          const int rt = (warp & 3) * 32 + r;      // row of the tile
          const int qi = w * QT + (rt >> a.gs);
          if (qi >= nq) continue;
          const int64_t orow = static_cast<int64_t>(sb.begin + q0 + qi) * a.Hq + (hg << a.gs) + (rt & (Gt - 1));
          *reinterpret_cast<uint4*>(a.out + orow * D + j * 8) = st[r * NU + (j ^ (r & 7))];
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 4 * NT) {
    tc::fence_after_sync();
    tc::dealloc(tmem, C::kTmemCols);
  }
}

template <int D, int NT>
static cudaError_t prefill_packed_t(const PackedArgs& r, cudaStream_t st) {
  using C = PackedCfg<D, NT>;
  static std::atomic<bool> attr_set[64];   // per device; launches may come from several host threads
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(prefill_packed_kernel<D, NT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  PackedK k{};
  k.out = static_cast<__nv_bfloat16*>(r.out);
  k.k = static_cast<const __nv_bfloat16*>(r.k);
  k.v = static_cast<const __nv_bfloat16*>(r.v);
  k.starts = r.starts;
  k.k_cache = static_cast<__nv_bfloat16*>(r.k_cache);
  k.v_cache = static_cast<__nv_bfloat16*>(r.v_cache);
  k.desc = static_cast<__nv_bfloat16*>(r.desc);
  k.ctrl = r.ctrl;
  k.L_max = r.L_max; k.Mmax = static_cast<int>(r.L_max / kBlock);
  k.B = r.B; k.T = r.T; k.longest = r.longest; k.Hq = r.Hq; k.H = r.H; k.G = r.G;
  while ((1 << k.gs) < r.Gt) ++k.gs;
  k.scale_log2 = r.scale * 1.4426950408889634f;
  // every sequence has at most one query block that is not full
  const int QB = NT * 128 / r.Gt;
  const int64_t blocks = r.T / QB + r.B;
  prefill_packed_kernel<D, NT><<<static_cast<unsigned>(blocks * (r.Hq / r.Gt)), C::kThreads, C::kSmem, st>>>(
      *r.tm_q, *r.tm_k, *r.tm_v, k);
  return cudaGetLastError();
}

// One or two tiles per CTA, measured on 16384 tokens of equal sequences (32/8
// heads, d = 128; us with one, with two): 32 tokens 176, 256; 100: 148, 168;
// 256: 130, 136; 512: 156, 160; 1024: 208, 208; 2048: 316, 307; 4096: 540, 515;
// 16384: 2150, 1863. A batch counts as long by its mean, or by one long
// sequence, which then holds most of the work.
cudaError_t launch_prefill_packed(const PackedArgs& r, cudaStream_t st) {
  const bool two = r.longest > 2048 || r.T / r.B > 1024;
  if (r.D == 128) return two ? prefill_packed_t<128, 2>(r, st) : prefill_packed_t<128, 1>(r, st);
  return two ? prefill_packed_t<64, 2>(r, st) : prefill_packed_t<64, 1>(r, st);
}

}  // namespace resa
