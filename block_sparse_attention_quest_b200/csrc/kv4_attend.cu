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
// conversion; q enters multiplied by 2^64 and p * vs by 2^62 so that the sums
// are normal numbers, and 2^69 and 2^71 are taken out of the results. Codes, q
// (bf16) and their products are exact. p * vs is rounded to bf16 (relative error 2^-9 per
// term, as the bf16 cache's attention rounds p); the zero part keeps fp32 p.
// fp32 queries and fp32 p * vs enter as three bf16 parts each (24 bits), so an
// fp32 call keeps fp32 accuracy.
//
// Work split, one CTA per SM. With one length for every row each (row, KV
// head) is cut into the same number of parts, one per CTA, wherever that
// leaves few SMs idle. Otherwise the blocks of every (row, head) in turn form
// one range, cut into equal parts; a CTA walks the pieces of its part, so rows
// of different lengths load every CTA alike. (Each (row, head) also counts
// kKv4PieceCost blocks for the fixed cost of a piece.) A piece that is not a
// whole (row, head) is left as a partial (max, sum, accumulator) and the last
// CTA to arrive merges them in the order of the range, so results do not
// depend on the arrival order.
//
// Each warp streams whole records (bulk copies, two blocks per stage) through
// its own ring in shared memory; the copies of a CTA's next piece are under
// way while the warps' results of the last one are merged.
//
// Measured (B200, 32/8 heads, d = 128, bf16): a 128K context 34.7 us (151 MB, 0.67
// of the copy rate), of which about 27 streaming and 8 before the first
// product and in the merges; 1639 of 16384 blocks of a 256K context 14.2 us;
// 16 rows of 1K to 32K tokens 66.7 us (0.69). While it streams it is bound by
// instruction latency: 277 instructions per block and warp, three warps per
// scheduler at 168 registers (sixteen warps at 128 spill and are slower).
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
  int B, H, G, Mmax, n_sel;
  int splits;              // parts per (row, head) with a CTA each, or 0: parts of the range
  int row_blocks;          // with splits: the blocks of every (row, head), their
  int split_per, split_rem;   // quotient and rest by splits
  float scale_log2;
};

// one CTA per SM; warps by the registers a warp needs (fp32 holds three parts
// of q)
template <typename T>
constexpr int kKv4Warps = sizeof(T) == 2 ? 12 : 8;
constexpr int kKv4Stages = 3;      // stages of two records per warp
constexpr int kKv4MinBlocks = 16;  // blocks per CTA below which fewer CTAs are used
// A piece's fixed cost, in blocks: its q, its first records' latency and the
// merge of its warps, 4 us or more where a block takes 72 ns. Measured back to
// back on a batch of 16 rows of 1K to 32K tokens: 69.4 us with 32, 64.4 with 48,
// 64.1 with 64 (with less the CTAs of several short rows end last).
constexpr uint32_t kKv4PieceCost = 64;

template <typename T, int D>
struct Kv4Cfg {
  static constexpr int kRec = kv4_record_bytes(D);
  static constexpr int kRing = kKv4Warps<T> * kKv4Stages * 2 * kRec;
  // the warps' results; then the parts' weights and the threads' sums
  static constexpr int kWarps = merge_floats(D, kKv4Warps<T>) * 4;
  static constexpr int kParts = (8 * (kKv4MaxCtas + 2) + 8 + kKv4Warps<T> * 32 * 4) * 4;
  static constexpr int kSmem = kRing + (kWarps > kParts ? kWarps : kParts);
};

// blocks of row b that its heads attend to
__device__ __forceinline__ uint32_t kv4_row_blocks(const Kv4K& a, int b) {
  const int64_t l = row_len(a.lens, a.len, b);
  if (a.sel == nullptr) return static_cast<uint32_t>((l + kBlock - 1) / kBlock);
  return a.lens != nullptr ? num_selected_dev(l, a.r, a.n_min) : a.n_sel;
}

// The range of all (row, head) units, each kKv4PieceCost + its blocks long, and
// its cut into equal parts (positions stay below 2^32: kv4_range_fits).
struct Kv4Range {
  uint32_t total, per, rem;
  int ctas;
  __device__ __forceinline__ void set(uint32_t n, uint32_t grid) {
    total = n;
    const uint32_t most = (n - 1) / (kKv4MinBlocks + kKv4PieceCost) + 1;
    ctas = static_cast<int>(most < grid ? most : grid);
    per = total / ctas;
    rem = total - per * ctas;
  }
  // first position of CTA i's part
  __device__ __forceinline__ uint32_t cut(uint32_t i) const { return i * per + min(i, rem); }
  // the CTA whose part holds position x
  __device__ __forceinline__ uint32_t owner(uint32_t x) const {
    const uint32_t big = rem * (per + 1);
    return x < big ? x / (per + 1) : rem + (x - big) / per;
  }
};

// One warp finds the range's length and the row that holds position x.
__device__ __forceinline__ void kv4_find(const Kv4K& a, uint32_t x, uint32_t& total, int& row,
                                         uint32_t& row_start) {
  const int lane = threadIdx.x & 31;
  uint32_t run = 0;
  row = 0;
  row_start = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    const uint32_t mine = b < a.B ? a.H * (kv4_row_blocks(a, b) + kKv4PieceCost) : 0u;
    uint32_t inc = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t begin = run + inc - mine;
    const unsigned who = __ballot_sync(0xffffffffu, b < a.B && x >= begin);
    if (who) {                                    // the last row that begins at or before x
      const int src = 31 - __clz(who);
      row = b0 + src;
      row_start = __shfl_sync(0xffffffffu, begin, src);
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  total = run;
}

// 2^x; results below 2^-126 are 0 (weights that small change no sum here)
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Merge of the partials that `parts` consecutive CTAs from `first` on left of one
// (row, head), by one CTA. `late`: the first of them began before this (row,
// head), so it is that CTA's last piece. The (max, sum) pairs are turned into
// weights first, then every thread sums four output columns over its parts.
// (Code that a CTA runs once costs its fetch, some 25 cycles an instruction,
// far more than its execution: loops here and in the rest of a piece's end are
// kept rolled.)
template <typename T, int D>
__device__ __forceinline__ void kv4_merge(const Kv4K& a, float* sm, int first, int parts,
                                          bool late, int64_t head0) {
  constexpr int NW = kKv4Warps<T>, NT = NW * 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto slot = [&](int s) -> int { return 2 * (first + s) + (s == 0 && late ? 1 : 0); };
  float* w_s = sm;                      // [parts][8] weights
  float* l_h = sm + 8 * (kKv4MaxCtas + 2);
  float4* sums = reinterpret_cast<float4*>(l_h + 8);
  // four columns per thread; where the group's columns need fewer threads than
  // there are, every `step`-th part. The first four of a thread's parts are
  // requested ahead of the weights (eight make the kernel spill: 35.9 us at 128K
  // against 35.0; none 35.3).
  static_assert(8 * (D / 4) <= NT, "a thread has at most four columns");
  constexpr int kAhead = 4;
  const int items = a.G * (D / 4), step = NT / items;
  const int i = static_cast<int>(threadIdx.x) % items, from = static_cast<int>(threadIdx.x) / items;
  const int most = from < step ? parts : 0;
  const float4* po = reinterpret_cast<const float4*>(a.part_o) + i;
  float4 x[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int s = from + u * step;
    if (s < most) x[u] = __ldcg(po + static_cast<int64_t>(slot(s)) * items);
  }
  if (warp < a.G) {
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + warp;
    // (mostly at most 32 parts: one load per lane)
    const float2 mine = lane < parts ? __ldcg(ml + slot(lane) * a.G) : make_float2(-INFINITY, 0.f);
    float m = mine.x;
#pragma unroll 1
    for (int s = lane + 32; s < parts; s += 32) m = fmaxf(m, __ldcg(ml + slot(s) * a.G).x);
#pragma unroll 1
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
#pragma unroll 1
    for (int s = lane; s < parts; s += 32) {
      const float2 p = s == lane ? mine : __ldcg(ml + slot(s) * a.G);
      const float w = p.x == -INFINITY ? 0.f : ex2_ftz(p.x - m);
      w_s[s * 8 + warp] = w;
      l = fmaf(w, p.y, l);
    }
#pragma unroll 1
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      l_h[warp] = l;
      if (a.lse != nullptr) a.lse[head0 + warp] = (m + log2f(l)) * 0.69314718055994531f;
    }
  }
  __syncthreads();
  const int h = i / (D / 4);
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& z, float w) {
    y.x = fmaf(w, z.x, y.x); y.y = fmaf(w, z.y, y.y);
    y.z = fmaf(w, z.z, y.z); y.w = fmaf(w, z.w, y.w);
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int s = from + u * step;
    if (s < most) add(x[u], w_s[s * 8 + h]);
  }
#pragma unroll 1
  for (int s = from + kAhead * step; s < most; s += step)
    add(__ldcg(po + static_cast<int64_t>(slot(s)) * items), w_s[s * 8 + h]);
  sums[threadIdx.x] = y;
  __syncthreads();
  if (from == 0) {
#pragma unroll 1
    for (int k = 1; k < step; ++k) {
      const float4 z = sums[threadIdx.x + k * items];
      y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
    }
    const float inv = 1.f / l_h[h];
    T* out = static_cast<T*>(a.out) + head0 * D + i * 4;
    out[0] = Dt<T>::from_f(y.x * inv); out[1] = Dt<T>::from_f(y.y * inv);
    out[2] = Dt<T>::from_f(y.z * inv); out[3] = Dt<T>::from_f(y.w * inv);
  }
  __syncthreads();
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

// What the end of a piece needs, kept in shared memory while its blocks stream.
struct Kv4Done {
  int64_t bh;
  int slot;                // partial slot, or -1 when the piece is the whole unit
  int first, parts, late;  // the unit's partials: see kv4_merge
};

// code - 8 of the low nibbles of both halves, as bf16 numbers (exact)
__device__ __forceinline__ uint32_t signed_codes(uint32_t w) {
  return bf16x2_add((w & 0x000f000fu) | 0x43004300u, 0xc308c308u);   // 128 + code, -136
}

// mma_bf16_16816 with rows 8 .. 15 of the sum left out.
__device__ __forceinline__ void mma_row0(float& d0, float& d1, const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  [[maybe_unused]] float x2, x3;
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%10,%10};"
      : "+f"(d0), "+f"(d1), "=f"(x2), "=f"(x3)
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// A warp takes two blocks at a time (one stage of its ring): the two
// independent chains of products and exponentials hide each other's latency,
// and the barrier, the check of the running maximum and the loop's own
// instructions are shared.
//
// The factor 2^62 of a bf16 call's p * vs, which keeps products with subnormal
// codes normal numbers, is put on vs (exactly), not on p: the sums of p and of
// p * zero are plain fp32 sums, which values up to 2^60 leave far below 2^128.
// p * vs itself is largest at p = 2^8 (the reference is moved beyond that) and
// vs = 2^61 / 15: 2^127.1, still a bf16 number. A product is lost below
// 2^-149, so a code part counts down to 2^-78 beside a weight of 1.
// (With the factor in the exponent of p, 32 equal weights of values 2^59 made
// 2^128; and m - 64 is rounded for references m beyond 2^30, which leaves
// weights of 2^128 or 1 where 2^64 is meant.)
//
// Rounding p * scale to bf16 costs 2^-9 of each term p * scale * code, and the
// codes' common part (their mean is near 8 of 15) would make that error three
// times the bf16 cache's. So the products are taken about code 8: the sum of
// the rounded p * scale (one product with a constant matrix of ones per group)
// times 8 is subtracted at the end, exactly, and zero + 8 * scale takes the
// place of the zero. (Measured at a 128K context: error against 64 bits 4.8e-3
// without, 2.4e-3 with it, 1.7e-3 being the output's own rounding.) An fp32
// call makes bf16 numbers of code - 8 instead, for keys too, so that its sums
// stay small and of both signs: the tensor cores truncate, and a common sign
// would add up (outputs over 65000 tokens: 9.9e-6 off; 8.6e-7 with it, the small
// parts first and running sums that round).
template <typename T, int D, bool SEL>
__global__ void __launch_bounds__(kKv4Warps<T> * 32, 1)
    kv4_attend_kernel(Kv4K a) {
  using C = Kv4Cfg<T, D>;
  constexpr int PARTS = sizeof(T) == 2 ? 1 : 3;    // bf16 parts of q and of p * scale
  constexpr int NG = D / kKv4Group;
  constexpr int NW = kKv4Warps<T>, ST = kKv4Stages, REC = C::kRec;
  constexpr float kUp = PARTS == 1 ? 4611686018427387904.f : 1.f;   // 2^62 on the value scales
  constexpr float kDown = 5.9029581035870565e+20f;              // 2^69
  constexpr uint32_t kOnes = 0x00010001u;                       // code 1 in both halves
  constexpr uint32_t kOne = PARTS == 1 ? kOnes : 0x3f803f80u, kOneHigh = PARTS == 1 ? 0x00100010u : kOne;
  constexpr float kMid = 8.f;                                   // code the products are taken about
  constexpr float kMidK = PARTS == 1 ? 0.f : 8.f;
  constexpr float kKeys = PARTS == 1 ? kDown : 1.f;             // what brings q . code back
  // what brings the running sums back: 2^71 (and 1/16 of it where codes count
  // 16-fold); nothing for fp32, whose value codes are used as numbers
  constexpr float kBack = PARTS == 1 ? 2361183241434822606848.f : 1.f, kRow8 = PARTS == 1 ? 0.0625f : 1.f;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t bars[NW][ST];
  __shared__ uint32_t s_total, s_row_start;
  __shared__ int s_row, s_last;
  __shared__ float s_mx[8], s_l[8];
  __shared__ Kv4Done s_done[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gq = lane >> 2, cq = lane & 3;
  if (lane == 0) {
#pragma unroll
    for (int st = 0; st < ST; ++st) mbar_init(&bars[warp][st], 1);
    fence_mbar_init();
  }
  __syncwarp();
  // everything read below may come from the kernel before this one
  grid_dependency_wait();
  // ---- this CTA's part: one part of one unit (a.splits per unit), or a
  // stretch of the range
  Kv4Range range;
  uint32_t x = 0, part1 = 0, row_start = 0, m_row;
  int row;
  if (a.splits > 0) {                             // grid (splits, H, B)
    m_row = a.row_blocks;
    row = blockIdx.z;
  } else {
    if (a.lens == nullptr) {
      m_row = a.row_blocks;
      const uint32_t per_row = a.H * (m_row + kKv4PieceCost);
      range.set(per_row * a.B, gridDim.x);
      if (static_cast<int>(blockIdx.x) >= range.ctas) return;
      row = static_cast<int>(range.cut(blockIdx.x) / per_row);
      row_start = row * per_row;
    } else {
      if (warp == 0) {
        uint32_t n, start;
        int r;
        kv4_find(a, 0u, n, r, start);
        range.set(n, gridDim.x);
        kv4_find(a, range.cut(blockIdx.x), n, r, start);
        if (lane == 0) { s_total = n; s_row = r; s_row_start = start; }
      } else if (blockIdx.x == 0) {
        for (int b = threadIdx.x - 32; b < a.B; b += (NW - 1) * 32)
          if (row_len_bad(a.lens, a.len, b)) raise_error(a.ctrl, kErrBadIndex);
      }
      __syncthreads();
      range.set(s_total, gridDim.x);
      if (static_cast<int>(blockIdx.x) >= range.ctas) return;
      row = s_row;
      row_start = s_row_start;
      m_row = kv4_row_blocks(a, row);
    }
    x = range.cut(blockIdx.x);
    part1 = range.cut(blockIdx.x + 1);
  }
  const uint32_t part0 = x;
  uint8_t* my_ring = ring + warp * ST * 2 * REC;
  uint32_t used = 0;                              // stages of this warp's ring, over all pieces

  // ---- the piece at hand: entries [i0, i1) of unit bh's blocks (or list)
  int i0, i1, count, tail, part_block, blocks_r, ids = -1, ids_now = -1;
  int64_t bh;
  const uint8_t* base;
  // With a list, lane u of `ids` holds entry u % 2 of this warp's pair
  // 16 w + u / 2 around the pair copied next, `ids_now` those around the pair
  // in use; pair k is entries i0 + 2 (warp + k NW) and the next.
  auto load_ids = [&](int k0) {
    const int i = i0 + 2 * (warp + (k0 + (lane >> 1)) * NW) + (lane & 1);
    ids = -1;
    if (i < i1) {
      const int j = __ldg(a.sel + bh * a.n_sel + i);
      if (j >= 0 && j < blocks_r) ids = j;
      else raise_error(a.ctrl, kErrBadIndex);      // the block is skipped
    }
  };
  auto issue = [&](int k, int st) {               // pair k into stage st; whole warp
    uint64_t* bar = &bars[warp][st];
    uint8_t* dst = my_ring + st * 2 * REC;
    if constexpr (SEL) {
      if ((k & 15) == 0) load_ids(k);
      const int ja = __shfl_sync(0xffffffffu, ids, (2 * k) & 31);
      const int jb = __shfl_sync(0xffffffffu, ids, (2 * k + 1) & 31);
      if (lane == 0) {
        fence_proxy_async_smem();                 // the stage's last reads precede the copy
        mbar_arrive_expect_tx(bar, ((ja >= 0) + (jb >= 0)) * REC);
        if (ja >= 0) bulk_load(dst, base + static_cast<int64_t>(ja) * REC, REC, bar);
        if (jb >= 0) bulk_load(dst + REC, base + static_cast<int64_t>(jb) * REC, REC, bar);
      }
    } else {
      if (lane == 0) {
        const int i = i0 + 2 * (warp + k * NW);
        const uint32_t bytes = i + 1 < i1 ? 2 * REC : REC;
        fence_proxy_async_smem();
        mbar_arrive_expect_tx(bar, bytes);
        bulk_load(dst, base + static_cast<int64_t>(i) * REC, bytes, bar);
      }
    }
  };
  // Moves to the next piece (from x on), starts its copies and notes in
  // `done` what its end needs; false when there is none.
  auto next_piece = [&](Kv4Done& done) -> bool {
    int g;
    if (a.splits > 0) {
      if (x != 0) return false;
      x = 1;
      const int part = blockIdx.x;
      g = blockIdx.y;
      i0 = part * a.split_per + min(part, a.split_rem);
      i1 = i0 + a.split_per + (part < a.split_rem);
      bh = static_cast<int64_t>(row) * a.H + g;
      if (threadIdx.x == 0) {
        done.bh = bh;
        done.first = static_cast<int>(bh) * a.splits;
        done.slot = a.splits == 1 ? -1 : 2 * (done.first + part);
        done.parts = a.splits; done.late = 0;
      }
    } else {
      uint32_t u0, u1, from;
      do {
        if (x >= part1) return false;
        while (x - row_start >= a.H * (m_row + kKv4PieceCost)) {
          row_start += a.H * (m_row + kKv4PieceCost);
          m_row = kv4_row_blocks(a, ++row);
        }
        g = static_cast<int>((x - row_start) / (m_row + kKv4PieceCost));
        u0 = row_start + g * (m_row + kKv4PieceCost);
        u1 = u0 + kKv4PieceCost + m_row;
        from = x;
        x = min(u1, part1);
        i0 = static_cast<int>(max(from, u0 + kKv4PieceCost) - (u0 + kKv4PieceCost));
        i1 = static_cast<int>(max(x, u0 + kKv4PieceCost) - (u0 + kKv4PieceCost));
      } while (i0 >= i1);                         // (a unit's cost without its blocks)
      bh = static_cast<int64_t>(row) * a.H + g;
      if (threadIdx.x == 0) {
        done.bh = bh;
        // slot 0: a part that begins in its first piece's unit; slot 1: its last piece
        done.slot = i0 == 0 && i1 == static_cast<int>(m_row)
                        ? -1 : 2 * static_cast<int>(blockIdx.x) + (from == part0 ? 0 : 1);
        if (done.slot >= 0) {
          done.first = static_cast<int>(range.owner(u0 + kKv4PieceCost));
          done.parts = static_cast<int>(range.owner(u1 - 1)) - done.first + 1;
          done.late = range.cut(done.first) < u0;
        }
      }
    }
    const int64_t len_r = row_len(a.lens, a.len, row);
    blocks_r = static_cast<int>((len_r + kBlock - 1) / kBlock);
    // tokens of the row's last block, and its number where it is not full
    tail = static_cast<int>(len_r & (kBlock - 1));
    part_block = tail ? blocks_r - 1 : -2;
    base = a.kv4 + bh * a.Mmax * REC;
    const int pairs = (i1 - i0 + 1) / 2;
    count = pairs > warp ? (pairs - warp + NW - 1) / NW : 0;
    for (int k = 0; k < count && k < ST; ++k) issue(k, (used + k) % ST);
    return true;
  };

  bool more = next_piece(s_done[0]);
#pragma unroll 1
  for (int piece = 0; more; ++piece) {
    bool ok = true;
    // ---- q fragments and the group sums of q
    uint32_t qb[PARTS][NG * 4][2];
    float qs0[NG], qs1[NG];
    {
      const T* qg = static_cast<const T*>(a.q) + (bh * a.G + gq) * D + cq * 16;
      // word j: product step 2j takes nibbles 0, 4 and 1, 5 (the latter read 16
      // times too large), step 2j + 1 nibbles 2, 6 and 3, 7
#pragma unroll
      for (int g2 = 0; g2 < NG; ++g2) {
        if constexpr (PARTS == 1) {
          uint4 raw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
          if (gq < a.G) {
            raw[0] = ldg16(qg + g2 * 64);
            raw[1] = ldg16(qg + g2 * 64 + 8);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t lo[2] = {raw[j].x, raw[j].y}, hi[2] = {raw[j].z, raw[j].w};
#pragma unroll
            for (int s = 0; s < 2; ++s) {          // times 2^64 and 2^60, exact
              qb[0][g2 * 4 + 2 * j + s][0] = bf16x2_mul(__byte_perm(lo[s], hi[s], 0x5410), 0x5f805f80u);
              qb[0][g2 * 4 + 2 * j + s][1] = bf16x2_mul(__byte_perm(lo[s], hi[s], 0x7632), 0x5d805d80u);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = 0.f;
            if (gq < a.G) load8<T>(qg + g2 * 64 + j * 8, f);
            float part[8][PARTS];
#pragma unroll
            for (int i = 0; i < 8; ++i) bf16_parts<PARTS>(f[i], part[i]);
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
#pragma unroll
              for (int s = 0; s < 2; ++s) {
                qb[p][g2 * 4 + 2 * j + s][0] = pack_bf16x2(part[2 * s][p], part[2 * s + 4][p]);
                qb[p][g2 * 4 + 2 * j + s][1] = pack_bf16x2(part[2 * s + 1][p], part[2 * s + 5][p]);
              }
          }
        }
        // the sums of q of heads 2 cq and 2 cq + 1, as the products with codes
        // of 1 (read as 16 where codes are), in the logits' scale
        const uint32_t one[4] = {kOne, kOne, kOneHigh, kOneHigh};
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = PARTS - 1; p >= 0; --p)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            mma_bf16_16816(acc, one, qb[p][g2 * 4 + s][0], qb[p][g2 * 4 + s][1]);
        qs0[g2] = acc[0];
        qs1[g2] = acc[1];
      }
    }
    const float to_log2 = a.scale_log2 * kKeys;

    float o[NG * 4][4], ones[NG][2], zo0[NG], zo1[NG];
#pragma unroll
    for (int i = 0; i < NG * 4; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      ones[i][0] = 0.f; ones[i][1] = 0.f;
      zo0[i] = 0.f; zo1[i] = 0.f;
    }
    // n = -m with m the reference (log2 units) of the weights 2^(s + n), exactly
    // (finite: logits of minus infinity, as an overflow of fp32 leaves them,
    // weigh 0 before any other has come)
    float n0 = 3.402823466e38f, n1 = 3.402823466e38f, l0 = 0.f, l1 = 0.f;

    int k = 0;
    for (; k < count; ++k) {
      const int st = used % ST;
      if (!__all_sync(0xffffffffu, mbar_try_wait(&bars[warp][st], (used / ST) & 1))) {
        const bool arrived = mbar_wait_bounded(&bars[warp][st], (used / ST) & 1, a.ctrl);
        if (!__all_sync(0xffffffffu, arrived)) { ok = false; break; }
      }
      ++used;
      const uint8_t* rec = my_ring + st * 2 * REC + lane * 16;
      const uint8_t* met = my_ring + st * 2 * REC + 2 * kv4_code_bytes(D) + gq * 16 * NG;
      // tokens of the two blocks that count (16 and 16 but for a row's last
      // block, an odd list's end, an id out of range)
      int ja, jb, va = kBlock, vb = kBlock;
      if constexpr (SEL) {
        if ((k & 15) == 0) ids_now = ids;       // (pairs k .. k + 15, loaded at pair k's issue)
        ja = __shfl_sync(0xffffffffu, ids_now, (2 * k) & 31);
        jb = __shfl_sync(0xffffffffu, ids_now, (2 * k + 1) & 31);
      } else {
        ja = i0 + 2 * (warp + k * NW);
        jb = ja + 1 < i1 ? ja + 1 : -1;
      }
      if (ja == part_block) va = tail;
      if (jb == part_block) vb = tail;
      if (ja < 0) va = 0;
      if (jb < 0) vb = 0;
      const bool whole = va + vb == 2 * kBlock;   // warp-uniform

      // ---- logits of tokens gq, gq + 8 of both blocks, heads 2 cq, 2 cq + 1
      float s[2][4];
      uint32_t vm[2][2][NG];                      // [block][token half][group]: {vs vz}
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
        uint2 meta[2][NG];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < NG; ++i)
            meta[h][i] = *reinterpret_cast<const uint2*>(met + u * REC + (h * NG + i) * 8);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const uint4 kw = *reinterpret_cast<const uint4*>(rec + u * REC + i * 512);
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          const uint32_t wa[2] = {kw.x, kw.y}, wb[2] = {kw.z, kw.w};
          // (the small parts of q first: their sums lose least)
#pragma unroll
          for (int p = PARTS - 1; p >= 0; --p)
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t x0 = wa[w] >> (8 * e), x1 = wb[w] >> (8 * e);
                uint32_t af[4];
                if constexpr (PARTS == 1) {
                  af[0] = x0 & 0x000f000fu; af[1] = x1 & 0x000f000fu;
                  af[2] = x0 & 0x00f000f0u; af[3] = x1 & 0x00f000f0u;
                } else {
                  af[0] = signed_codes(x0); af[1] = signed_codes(x1);
                  af[2] = signed_codes(x0 >> 4); af[3] = signed_codes(x1 >> 4);
                }
                mma_bf16_16816(acc, af, qb[p][i * 4 + 2 * w + e][0], qb[p][i * 4 + 2 * w + e][1]);
              }
          const float ka = bf16_lo(meta[0][i].x), kb = bf16_lo(meta[1][i].x);
          const float za = fmaf(kMidK, ka, bf16_hi(meta[0][i].x));
          const float zb = fmaf(kMidK, kb, bf16_hi(meta[1][i].x));
          s[u][0] = fmaf(ka, acc[0], fmaf(za, qs0[i], s[u][0]));
          s[u][1] = fmaf(ka, acc[1], fmaf(za, qs1[i], s[u][1]));
          s[u][2] = fmaf(kb, acc[2], fmaf(zb, qs0[i], s[u][2]));
          s[u][3] = fmaf(kb, acc[3], fmaf(zb, qs1[i], s[u][3]));
          vm[u][0][i] = meta[0][i].y;
          vm[u][1][i] = meta[1][i].y;
        }
      }
      // tokens that do not count: weight 0, and their scales (which may be
      // anything) with it; their codes are finite whatever the bits
      if (!whole) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int valid = u == 0 ? va : vb;
          if (gq >= valid) { s[u][0] = -INFINITY; s[u][1] = -INFINITY; }
          if (gq + 8 >= valid) { s[u][2] = -INFINITY; s[u][3] = -INFINITY; }
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            if (gq >= valid) vm[u][0][i] = 0u;
            if (gq + 8 >= valid) vm[u][1][i] = 0u;
          }
        }
        if (va + vb == 0) {                       // (both ids out of range)
          __syncwarp();
          if (k + ST < count) issue(k + ST, st);
          continue;
        }
      }
      // The reference moves only when some weight would exceed it by 2^8: the
      // sums stay far inside fp32, and most pairs rescale nothing.
      // (The product is rounded before n is added: with one rounding of both,
      // logits beyond 2^24 would leave a difference of any size.)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[u][e] = __fmul_rn(s[u][e], to_log2);
      const float x0 = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
      const float x1 = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
      if (__any_sync(0xffffffffu, !(x0 + n0 <= 8.f && x1 + n1 <= 8.f))) {
        const float r0 = fminf(n0, -warp_max_xor(x0, 16, 4));
        const float r1 = fminf(n1, -warp_max_xor(x1, 16, 4));
        const float al0 = ex2_ftz(r0 - n0), al1 = ex2_ftz(r1 - n1);
        n0 = r0; n1 = r1;
        l0 *= al0; l1 *= al1;
#pragma unroll
        for (int i = 0; i < NG * 4; ++i) {
          o[i][0] *= al0; o[i][2] *= al0;
          o[i][1] *= al1; o[i][3] *= al1;
        }
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          zo0[i] *= al0; zo1[i] *= al1;
          ones[i][0] *= al0; ones[i][1] *= al1;
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float p0 = ex2_ftz(s[u][0] + n0), p1 = ex2_ftz(s[u][1] + n1);
        const float p2 = ex2_ftz(s[u][2] + n0), p3 = ex2_ftz(s[u][3] + n1);
        l0 += p0 + p2;
        l1 += p1 + p3;
        // ---- values
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const float sa = bf16_lo(vm[u][0][i]), sb = bf16_lo(vm[u][1][i]);
          const float za = fmaf(kMid, sa, bf16_hi(vm[u][0][i]));
          const float zb = fmaf(kMid, sb, bf16_hi(vm[u][1][i]));
          zo0[i] = fmaf(p0, za, fmaf(p2, zb, zo0[i]));
          zo1[i] = fmaf(p1, za, fmaf(p3, zb, zo1[i]));
          uint32_t pb[PARTS][2];
          float e0[PARTS], e1[PARTS], e2[PARTS], e3[PARTS];
          if constexpr (PARTS == 1) {
            const float ua = sa * kUp, ub = sb * kUp;
            e0[0] = p0 * ua; e1[0] = p1 * ua; e2[0] = p2 * ub; e3[0] = p3 * ub;
          } else {
            bf16_parts<PARTS>(p0 * sa, e0);
            bf16_parts<PARTS>(p1 * sa, e1);
            bf16_parts<PARTS>(p2 * sb, e2);
            bf16_parts<PARTS>(p3 * sb, e3);
          }
          const uint32_t one[4] = {kOnes, kOnes, kOnes, kOnes};
#pragma unroll
          for (int p = 0; p < PARTS; ++p) {
            pb[p][0] = movmatrix_trans(pack_bf16x2(e0[p], e1[p]));
            pb[p][1] = movmatrix_trans(pack_bf16x2(e2[p], e3[p]));
            if constexpr (PARTS == 1) mma_row0(ones[i][0], ones[i][1], one, pb[p][0], pb[p][1]);
          }
          const uint4 vw = *reinterpret_cast<const uint4*>(rec + u * REC + kv4_code_bytes(D) + i * 512);
          const uint32_t w4[4] = {vw.x, vw.y, vw.z, vw.w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t x0 = w4[m], x1 = w4[m] >> 8;
            if constexpr (PARTS == 1) {
              const uint32_t af[4] = {x0 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x000f000fu,
                                      x1 & 0x00f000f0u};
              mma_bf16_16816(o[i * 4 + m], af, pb[0][0], pb[0][1]);
            } else {
              // sixteen tokens at a time, added to the running sums by rounded
              // additions (the tensor cores' own truncate)
              const uint32_t af[4] = {signed_codes(x0), signed_codes(x0 >> 4), signed_codes(x1),
                                      signed_codes(x1 >> 4)};
              float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int p = PARTS - 1; p >= 0; --p) mma_bf16_16816(y, af, pb[p][0], pb[p][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[i * 4 + m][e] += y[e];
            }
          }
        }
      }
      __syncwarp();                               // every lane has read the stage
      if (k + ST < count) issue(k + ST, st);
    }
    if (!ok) {
      // wait, within the bound, for this warp's other copies in flight (pairs
      // k + 1 .. of this piece)
      for (int i = 1; i < ST && k + i < count; ++i)
        (void)mbar_wait_bounded(&bars[warp][(used + i) % ST], ((used + i) / ST) & 1, a.ctrl);
      more = false;
    } else {
      more = next_piece(s_done[(piece + 1) & 1]);
    }
    if (!more) grid_launch_dependents();
    // ---- the warps' results, merged in shared memory
#pragma unroll 1
    for (int m = 4; m <= 16; m <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, m);
      l1 += __shfl_xor_sync(0xffffffffu, l1, m);
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        zo0[i] += __shfl_xor_sync(0xffffffffu, zo0[i], m);
        zo1[i] += __shfl_xor_sync(0xffffffffu, zo1[i], m);
      }
    }
    constexpr int OR = merge_row(D);
    float* sm = reinterpret_cast<float*>(ring + C::kRing);
    float* sm_o = sm;                             // [NW][8][OR]
    float* sm_m = sm + NW * 8 * OR;               // [NW][8], then the warps' weights
    float* sm_l = sm_m + NW * 8;
    const int h0 = 2 * cq, h1 = 2 * cq + 1;
    if (gq == 0) {
      sm_m[warp * 8 + h0] = -n0; sm_l[warp * 8 + h0] = l0;
      sm_m[warp * 8 + h1] = -n1; sm_l[warp * 8 + h1] = l1;
    }
    if (h0 < a.G) {
      // rows gq + 8 hold codes read 16 times too large
#pragma unroll
      for (int i = 0; i < NG * 4; ++i) {
        const int ch = i * 16 + gq;
        const float c0 = kMid * ones[i / 4][0], c1 = kMid * ones[i / 4][1];   // (0 for fp32)
        sm_o[(warp * 8 + h0) * OR + ch] = fmaf(o[i][0] - c0, kBack, zo0[i / 4]);
        sm_o[(warp * 8 + h1) * OR + ch] = fmaf(o[i][1] - c1, kBack, zo1[i / 4]);
        sm_o[(warp * 8 + h0) * OR + ch + 8] = fmaf(fmaf(o[i][2], kRow8, -c0), kBack, zo0[i / 4]);
        sm_o[(warp * 8 + h1) * OR + ch + 8] = fmaf(fmaf(o[i][3], kRow8, -c1), kBack, zo1[i / 4]);
      }
    }
    if (!__syncthreads_and(ok)) {
      // the copies of a next piece that a warp began end before it leaves
      if (more)
        for (int k = 0; k < count && k < ST; ++k)
          (void)mbar_wait_bounded(&bars[warp][(used + k) % ST], ((used + k) / ST) & 1, a.ctrl);
      return;
    }
    if (warp < 8) {                               // head `warp`: lane w holds warp w's (m, l)
      const float m = lane < NW ? sm_m[lane * 8 + warp] : -INFINITY;
      float mx = m;
#pragma unroll 1
      for (int i = 8; i >= 1; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
      const float w = m == -INFINITY ? 0.f : ex2_ftz(m - mx);
      float l = lane < NW ? w * sm_l[lane * 8 + warp] : 0.f;
#pragma unroll 1
      for (int i = 8; i >= 1; i >>= 1) l += __shfl_xor_sync(0xffffffffu, l, i);
      __syncwarp();
      if (lane < NW) sm_m[lane * 8 + warp] = w;
      if (lane == 0) { s_mx[warp] = mx; s_l[warp] = l; }
    }
    __syncthreads();
    const Kv4Done dn = s_done[piece & 1];
    T* out = static_cast<T*>(a.out);
    for (int i = threadIdx.x; i < a.G * (D / 2); i += NW * 32) {
      const int h = i / (D / 2), ch = (i % (D / 2)) * 2;
      float v0 = 0.f, v1 = 0.f;
#pragma unroll 4
      for (int w = 0; w < NW; ++w) {
        const float sc = sm_m[w * 8 + h];
        const float2 y = *reinterpret_cast<const float2*>(sm_o + (w * 8 + h) * OR + ch);
        v0 = fmaf(sc, y.x, v0);
        v1 = fmaf(sc, y.y, v1);
      }
      if (dn.slot < 0) {
        const float inv = 1.f / s_l[h];
        out[(dn.bh * a.G + h) * D + ch] = Dt<T>::from_f(v0 * inv);
        out[(dn.bh * a.G + h) * D + ch + 1] = Dt<T>::from_f(v1 * inv);
        if (a.lse != nullptr && ch == 0)
          a.lse[dn.bh * a.G + h] = (s_mx[h] + log2f(s_l[h])) * 0.69314718055994531f;
      } else {
        *reinterpret_cast<float2*>(a.part_o + (static_cast<int64_t>(dn.slot) * a.G + h) * D + ch) =
            make_float2(v0, v1);
        if (ch == 0)
          *reinterpret_cast<float2*>(a.part_ml + (dn.slot * a.G + h) * 2) =
              make_float2(s_mx[h], s_l[h]);
      }
    }
    __syncthreads();
    if (dn.slot >= 0) {
      if (threadIdx.x == 0)
        s_last = atomic_add_acq_rel(a.counters + dn.bh, 1) == dn.parts - 1;
      __syncthreads();
      if (s_last) {
        kv4_merge<T, D>(a, sm, dn.first, dn.parts, dn.late != 0, dn.bh * a.G);
        if (threadIdx.x == 0) a.counters[dn.bh] = 0;
      }
      __syncthreads();
    }
  }
}

template <typename T, int D, bool SEL>
static cudaError_t kv4_attend_t(const Shape& s, const Kv4K& k, int ctas, cudaStream_t st) {
  using C = Kv4Cfg<T, D>;
  static std::atomic<bool> attr_set[64];   // per device; launches may come from several host threads
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kv4_attend_kernel<T, D, SEL>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = k.splits > 0 ? dim3(k.splits, k.H, k.B) : dim3(ctas);
  cfg.blockDim = dim3(kKv4Warps<T> * 32);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_attend_kernel<T, D, SEL>, k);
}

template <typename T, int D>
static cudaError_t kv4_attend_d(const Shape& s, const Kv4K& k, int ctas, cudaStream_t st) {
  return k.sel != nullptr ? kv4_attend_t<T, D, true>(s, k, ctas, st)
                          : kv4_attend_t<T, D, false>(s, k, ctas, st);
}

// CTAs of a launch over at most blocks_bound blocks per (row, KV head): one per
// SM at most, none with less than kKv4MinBlocks blocks where there are more.
// *splits > 0: that many parts of every (row, head); 0: parts of the range.
// A cut of every unit alike leaves up to units - 1 SMs idle; it is taken where
// at least nine tenths of them work (a CTA that crosses from one unit to
// another pays a second piece's fixed cost, about a tenth of a 128K context).
int kv4_ctas(const Shape& s, int64_t blocks_bound, bool ragged, int num_sms, int* splits) {
  const int64_t units = static_cast<int64_t>(s.B) * s.H;
  const int64_t want = (blocks_bound + kKv4MinBlocks - 1) / kKv4MinBlocks;   // parts of one unit
  const int64_t sms = num_sms < kKv4MaxCtas ? num_sms : kKv4MaxCtas;
  int64_t S = units > sms ? 0 : sms / units;
  if (S > want) S = want;
  if (S > kMaxSplits) S = kMaxSplits;
  if (!ragged && S > 0 && (S == want || S == kMaxSplits || units * S * 10 >= sms * 9)) {
    *splits = static_cast<int>(S);
    return static_cast<int>(units * S);
  }
  *splits = 0;
  int64_t n = units * (want < kMaxSplits ? want : kMaxSplits);
  return static_cast<int>(n < sms ? n : sms);
}

// most CTAs of any launch up to blocks_bound blocks, on any device
int kv4_most_ctas(const Shape& s, int64_t blocks_bound) {
  const int64_t want = (blocks_bound + kKv4MinBlocks - 1) / kKv4MinBlocks;
  const int64_t n = static_cast<int64_t>(s.B) * s.H * (want < kMaxSplits ? want : kMaxSplits);
  return static_cast<int>(n < kKv4MaxCtas ? n : kKv4MaxCtas);
}

// (a cache of fewer than 2^31 rows can still have some 2^26 units of a block or
// two, whose fixed costs add up to more)
bool kv4_range_fits(const Shape& s, int64_t blocks_bound) {
  return static_cast<int64_t>(s.B) * s.H * (blocks_bound + kKv4PieceCost) < (1LL << 32);
}

cudaError_t launch_kv4_attend(const Shape& s, const Kv4Args& a, cudaStream_t st) {
  Kv4K k{};
  k.q = a.q; k.kv4 = static_cast<const uint8_t*>(a.kv4); k.sel = a.sel; k.lens = a.lens;
  k.part_o = a.part_o; k.part_ml = a.part_ml; k.counters = a.counters; k.ctrl = a.ctrl;
  k.out = a.out; k.lse = a.lse; k.len = a.len; k.r = a.r; k.n_min = a.n_min;
  k.B = s.B; k.H = s.H; k.G = s.G; k.splits = a.splits; k.Mmax = s.Mmax; k.n_sel = a.n_sel;
  k.scale_log2 = a.scale * 1.4426950408889634f;
  k.row_blocks = a.sel ? a.n_sel : static_cast<int>((a.len + kBlock - 1) / kBlock);
  if (a.splits > 0) {
    k.split_per = k.row_blocks / a.splits;
    k.split_rem = k.row_blocks % a.splits;
  }
  if (s.bf16) return s.D == 128 ? kv4_attend_d<__nv_bfloat16, 128>(s, k, a.ctas, st)
                                : kv4_attend_d<__nv_bfloat16, 64>(s, k, a.ctas, st);
  return s.D == 128 ? kv4_attend_d<float, 128>(s, k, a.ctas, st)
                    : kv4_attend_d<float, 64>(s, k, a.ctas, st);
}

}  // namespace resa
