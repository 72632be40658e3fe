// Accumulated attention weights, and a cache cut to the tokens that gathered
// the most of them.
//
// A decode step's weight of token t for KV group g is the sum over the group's
// heads h of exp(scale q_h . k_t - lse_h). The attention kernel leaves every
// logit (log2 units) and each head's (max m, sum l) in the workspace; the sums
//   w_t += sum_h 2^(logit_ht - m_h) / l_h
// follow in a kernel of their own, because no weight is known before the last
// split has been merged. Reading the logits back (4 bytes per head and token,
// from L2) replaces a second pass over the keys (2 d bytes per token). A 128K
// step of 32/8 heads takes 99.5 us: append 3.5, attention 86, sums about 10.
//
// Eviction keeps, per (row, KV head), the newest `recent` tokens and of the
// others the budget - recent with the largest sums, in their order.
#include <cooperative_groups.h>

#include "select_core.cuh"

namespace resa {

namespace cg = cooperative_groups;

// Grid (tokens / 1024, H, B), 256 threads; a thread adds the weights of four
// tokens 256 apart, so that every load of a warp is one contiguous run, and
// requests all of its logits and sums before it uses any.
template <int G>
__global__ void __launch_bounds__(256) add_weights_kernel(const float* __restrict__ logits,
                                                          const float* __restrict__ ml,
                                                          float* __restrict__ weights, int H,
                                                          int64_t stride, int64_t L_max,
                                                          int64_t len, const int32_t* lens,
                                                          bool fresh) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int g = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * H + g;
  const int64_t len_b = row_len(lens, len, b);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 1024 + threadIdx.x;
  const float* z = logits + (bh * stride + t0) * G;
  float* wp = weights + bh * L_max + t0;
  float x[4][G], old[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (t0 + i * 256 >= len_b) continue;
    const float* zi = z + static_cast<int64_t>(i) * 256 * G;
    if constexpr (G % 4 == 0) {
#pragma unroll
      for (int h = 0; h < G; h += 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(zi + h));
        x[i][h] = y.x; x[i][h + 1] = y.y; x[i][h + 2] = y.z; x[i][h + 3] = y.w;
      }
    } else {
#pragma unroll
      for (int h = 0; h < G; ++h) x[i][h] = __ldcg(zi + h);
    }
    old[i] = wp[i * 256];
  }
  float m[G], inv[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const float2 p = __ldcg(reinterpret_cast<const float2*>(ml) + bh * G + h);
    m[h] = p.x;
    inv[h] = 1.f / p.y;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + i * 256;
    if (t >= len_b) continue;
    float sum = 0.f;
#pragma unroll
    for (int h = 0; h < G; ++h) sum = fmaf(exp2f(x[i][h] - m[h]), inv[h], sum);
    wp[i * 256] = fresh && t == len_b - 1 ? sum : old[i] + sum;
  }
}

template <int G>
static cudaError_t add_weights_t(const Shape& s, const float* logits, const float* ml,
                                 float* weights, int64_t len, const int32_t* lens, bool fresh,
                                 cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((len + 1023) / 1024), s.H, s.B);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, add_weights_kernel<G>, logits, ml, weights, s.H,
                            (len + kBlock - 1) / kBlock * kBlock, s.L_max, len, lens, fresh);
}

cudaError_t launch_add_weights(const Shape& s, const float* logits, const float* ml,
                               float* weights, int64_t len, const int32_t* lens, bool fresh,
                               cudaStream_t st) {
  switch (s.G) {
    case 1: return add_weights_t<1>(s, logits, ml, weights, len, lens, fresh, st);
    case 2: return add_weights_t<2>(s, logits, ml, weights, len, lens, fresh, st);
    case 3: return add_weights_t<3>(s, logits, ml, weights, len, lens, fresh, st);
    case 4: return add_weights_t<4>(s, logits, ml, weights, len, lens, fresh, st);
    case 5: return add_weights_t<5>(s, logits, ml, weights, len, lens, fresh, st);
    case 6: return add_weights_t<6>(s, logits, ml, weights, len, lens, fresh, st);
    case 7: return add_weights_t<7>(s, logits, ml, weights, len, lens, fresh, st);
    default: return add_weights_t<8>(s, logits, ml, weights, len, lens, fresh, st);
  }
}

// ---------------------------------------------------------------------- select
constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvCluster = 8;        // CTAs per (row, KV head) of a long row

// order-preserving key of a weight; NaN below every number
__device__ __forceinline__ uint32_t weight_key(float w) { return w == w ? score_key(w) : 0u; }

// Exclusive prefix sum of x over the CTA's threads; total receives the sum.
__device__ __forceinline__ uint32_t ev_scan(uint32_t x, uint32_t* warp_tot, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  uint32_t c = warp_tot[lane], run = c;          // (one total per lane: 32 warps)
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += y;
  }
  total = __shfl_sync(0xffffffffu, run, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, run - c, warp);
  __syncthreads();
  return before + inc - x;
}

// One CTA (CL = 1) or a cluster of eight per (row, KV head), each CTA with a
// slice of the candidates in registers: KPT per thread, four consecutive ones
// per 16-byte load, so that index order is (load u, thread, element). KPT = 0:
// a slice of any length, read again (from L2) in every pass.
//
// Three radix passes (11, 11 and 10 bits of the keys, from the top) find the
// exact threshold key: every CTA counts its slice into a histogram of its own
// (one per pass), and after a cluster barrier all of them read all eight
// through distributed shared memory and take the same decision. A pass after
// which the threshold bin is taken whole is the last one. Then the keys above
// and those equal to the threshold are counted per (u, warp); one scan over
// those counts and the CTAs' totals gives every kept token its place in the
// list. Latency-bound: 23 us for 8 heads of 128K weights, of which 4.5 per pass
// (1.1 counting, 2.8 barrier and remote reads, 0.6 the decision); one CTA of
// 4K weights 8 us.
template <int CL, int KPT>
__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const float* __restrict__ weights,
                                                                  int32_t* __restrict__ kept, int H,
                                                                  int64_t L_max, int64_t len,
                                                                  const int32_t* lens, int budget,
                                                                  int recent, Ctrl* ctrl) {
  constexpr int U = KPT > 0 ? KPT / 4 : 1;        // loads held per thread
  __shared__ __align__(16) uint32_t hist[3][kBins];
  __shared__ uint32_t warp_tot[kEvWarps];
  __shared__ uint32_t tab[U][kEvWarps];           // per (u, warp): keys above | equal << 16
  __shared__ uint32_t s_prefix, s_remaining, s_whole;
  __shared__ __align__(8) uint32_t s_count[2];    // keys above, equal to the threshold
  cg::cluster_group cluster = cg::this_cluster();
  auto all_sync = [&] {
    if constexpr (CL > 1) cluster.sync();
    else __syncthreads();
  };
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = CL > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  for (int i = tid; i < 3 * kBins / 4; i += kEvThreads)
    reinterpret_cast<uint4*>(&hist[0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
  grid_launch_dependents();                       // the gather waits for this grid's end
  grid_dependency_wait();
  const int g = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * H + g;
  int32_t* out = kept + bh * budget;
  if (rank == 0 && g == 0 && tid == 0 && row_len_bad(lens, len, b)) raise_error(ctrl, kErrBadIndex);
  const int n = static_cast<int>(row_len(lens, len, b));
  const int me = rank * kEvThreads + tid;
  if (n <= budget) {                              // nothing to evict (whole cluster)
    for (int i = me; i < budget; i += CL * kEvThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int cand = n - recent, need = budget - recent;
  for (int i = me; i < recent; i += CL * kEvThreads) out[need + i] = cand + i;
  if (need == 0) return;
  // a slice starts at a multiple of 16 tokens, as rows do (16-byte loads)
  const float* w = weights + bh * L_max;
  const int per = (cand + CL * 16 - 1) / (CL * 16) * 16;
  const int c0 = min(cand, rank * per), c1 = min(cand, c0 + per);
  const int rounds = KPT > 0 ? U : (per + 4 * kEvThreads - 1) / (4 * kEvThreads);
  uint32_t key[4 * U];
  uint32_t in = 0;                                // bit 4u + e: key is a candidate
  auto load = [&](int u, int at) {
    const int j = c0 + (u * kEvThreads + tid) * 4;
    const float4 x = j < c1 ? __ldcg(reinterpret_cast<const float4*>(w + j))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
    const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      key[at + e] = weight_key(y[e]);
      if (j + e < c1) in |= 1u << (at + e);
      else in &= ~(1u << (at + e));
    }
  };
  if constexpr (KPT > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, 4 * u);
  }
  __syncthreads();                                // the histograms are clear
  uint32_t prefix = 0, remaining = static_cast<uint32_t>(need);
  int shift = 21;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    const uint32_t above = pass == 0 ? 0u : (pass == 1 ? 0xffe00000u : 0xfffffc00u);
    uint32_t* h = hist[pass];
    auto count = [&](int at) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (((in >> (at + e)) & 1u) && (key[at + e] & above) == prefix)
          atomicAdd(&h[(key[at + e] >> shift) & mask], 1u);
    };
    if constexpr (KPT > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) count(4 * u);
    } else {
      for (int u = 0; u < rounds; ++u) { load(u, 0); count(0); }
    }
    all_sync();
    // thread t owns bins 2047 - 2t and 2046 - 2t
    uint32_t hi = 0, lo = 0;
    uint2 r[CL];
#pragma unroll
    for (int i = 0; i < CL; ++i) {
      const uint32_t* hr = CL > 1 ? cluster.map_shared_rank(h, i) : h;
      r[i] = *reinterpret_cast<const uint2*>(hr + kBins - 2 - 2 * tid);
    }
#pragma unroll
    for (int i = 0; i < CL; ++i) { hi += r[i].y; lo += r[i].x; }
    uint32_t total;
    const uint32_t before = ev_scan(hi + lo, warp_tot, total);
    if (before < remaining && remaining <= before + hi + lo) {
      const bool first = remaining <= before + hi;
      const uint32_t left = remaining - before - (first ? 0u : hi);
      s_prefix = prefix | (static_cast<uint32_t>(kBins - 1 - 2 * tid - (first ? 0 : 1)) << shift);
      s_remaining = left;
      s_whole = left == (first ? hi : lo);
    }
    __syncthreads();
    prefix = s_prefix;
    remaining = s_remaining;
    const bool whole = s_whole;
    if (whole || pass == 2) break;
    shift = pass == 0 ? 10 : 0;
    __syncthreads();
  }
  // Kept: every key whose bits above `shift` exceed those of T, and the
  // `remaining` of lowest index among those with the same bits (all of them
  // where the bin is taken whole).
  const uint32_t T = prefix >> shift;
  auto marks = [&](int at, uint32_t& gt, uint32_t& eq) {
    gt = 0; eq = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t k = key[at + e] >> shift;
      if ((in >> (at + e)) & 1u) {
        gt |= (k > T ? 1u : 0u) << e;
        eq |= (k == T ? 1u : 0u) << e;
      }
    }
  };
  // counts of a load over this warp's earlier lanes (exclusive) and in all
  auto lane_scan = [&](uint32_t gt, uint32_t eq, uint32_t& all) {
    const uint32_t mine = __popc(gt) | (__popc(eq) << 16);
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    all = __shfl_sync(0xffffffffu, inc, 31);
    return inc - mine;
  };
  uint32_t base_gt = 0, base_eq = 0;              // of this CTA, then running
  // adds the counts of the cluster's earlier CTAs; the barrier that keeps any
  // CTA from leaving while another reads it is waited for at the very end
  auto earlier_ctas = [&] {
    if constexpr (CL > 1) {
      uint2 c[CL];
#pragma unroll
      for (int i = 0; i < CL; ++i)
        c[i] = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(s_count, i));
#pragma unroll
      for (int i = 0; i < CL; ++i) {
        base_gt += i < rank ? c[i].x : 0u;
        base_eq += i < rank ? c[i].y : 0u;
      }
      cluster.barrier_arrive();
    }
  };
  auto place = [&](int u, int at, uint32_t off, uint32_t gt, uint32_t eq) {
    // off: counts before this thread's four keys, within the CTA
    uint32_t g_at = base_gt + (off & 0xffffu), e_at = base_eq + (off >> 16);
    const int j = c0 + (u * kEvThreads + tid) * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if ((gt >> e) & 1u) out[g_at++ + min(e_at, remaining)] = j + e;
      if ((eq >> e) & 1u) {
        if (e_at < remaining) out[g_at + e_at] = j + e;
        ++e_at;
      }
    }
  };
  if constexpr (KPT > 0) {
    uint32_t off[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t gt, eq, all;
      marks(4 * u, gt, eq);
      off[u] = lane_scan(gt, eq, all);
      if (lane == 0) tab[u][warp] = all;
    }
    __syncthreads();
    // scan of the table in (u, warp) order, the packed counts of a CTA fit 16 bits
    if (warp == 0) {
      uint32_t run = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t c = tab[u][lane];
        uint32_t inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        tab[u][lane] = run + inc - c;
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) { s_count[0] = run & 0xffffu; s_count[1] = run >> 16; }
    }
    all_sync();
    earlier_ctas();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t gt, eq;
      marks(4 * u, gt, eq);
      place(u, 4 * u, tab[u][warp] + off[u], gt, eq);
    }
  } else {
    // the CTA's totals first, then round by round
    uint32_t n_gt = 0, n_eq = 0;
    for (int u = 0; u < rounds; ++u) {
      uint32_t gt, eq;
      load(u, 0);
      marks(0, gt, eq);
      n_gt += __popc(gt);
      n_eq += __popc(eq);
    }
    uint32_t t_gt, t_eq;
    (void)ev_scan(n_gt, warp_tot, t_gt);
    (void)ev_scan(n_eq, warp_tot, t_eq);
    if (tid == 0) { s_count[0] = t_gt; s_count[1] = t_eq; }
    all_sync();
    earlier_ctas();
    for (int u = 0; u < rounds; ++u) {
      uint32_t gt, eq, all;
      load(u, 0);
      marks(0, gt, eq);
      const uint32_t off = ev_scan(__popc(gt) | (__popc(eq) << 16), warp_tot, all);
      place(u, 0, off, gt, eq);
      base_gt += all & 0xffffu;
      base_eq += all >> 16;
    }
  }
  if constexpr (CL > 1) cluster.barrier_wait();
}

// ---------------------------------------------------------------------- gather
// One warp per 16-token block of the new cache: its rows are copied from where
// `kept` says, their minimum and maximum become the block's descriptor. 21 us
// for 16384 of 128K tokens of 8 heads, d = 128 (134 MB read and written, rows
// of 256 bytes scattered).
template <typename T, int D>
__global__ void __launch_bounds__(256) evict_gather_kernel(EvictArgs a, int H, int64_t L_max,
                                                           int M, int64_t total) {
  constexpr int CH = Chunk<T>::N;
  constexpr int CPR = D / CH;                     // 16-byte chunks per token row
  constexpr int TPP = 32 / CPR;                   // rows covered by one warp-wide load
  constexpr int NP = kBlock / TPP;
  grid_dependency_wait();
  const int64_t wid = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= total) return;
  const int64_t bh = wid / M;
  const int j = static_cast<int>(wid % M);
  const int64_t n = row_len(a.lens, a.len, static_cast<int>(bh / H));
  const int keep = static_cast<int>(n < a.budget ? n : a.budget);
  const int left = keep - j * kBlock;
  if (left <= 0) return;
  const int valid = left < kBlock ? left : kBlock;
  const int src_mine = lane < valid ? __ldcg(a.kept + bh * a.budget + j * kBlock + lane) : 0;
  const int chunk = lane % CPR, r0 = lane / CPR;
  const T* k = static_cast<const T*>(a.k) + bh * L_max * D + chunk * CH;
  const T* v = static_cast<const T*>(a.v) + bh * L_max * D + chunk * CH;
  uint4 kr[NP], vr[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = r0 + i * TPP;
    const int src = __shfl_sync(0xffffffffu, src_mine, t);
    if (t < valid) {
      kr[i] = ld_stream16(k + static_cast<int64_t>(src) * D);
      vr[i] = ld_stream16(v + static_cast<int64_t>(src) * D);
    }
  }
  if (a.weights_out != nullptr && lane < valid)
    a.weights_out[bh * a.L_out + j * kBlock + lane] = __ldg(a.weights + bh * L_max + src_mine);
  T* ko = static_cast<T*>(a.k_out) + (bh * a.L_out + j * kBlock) * D + chunk * CH;
  T* vo = static_cast<T*>(a.v_out) + (bh * a.L_out + j * kBlock) * D + chunk * CH;
  float mn[CH], mx[CH];
#pragma unroll
  for (int e = 0; e < CH; ++e) { mn[e] = INFINITY; mx[e] = -INFINITY; }
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int t = r0 + i * TPP;
    if (t < valid) {
      *reinterpret_cast<uint4*>(ko + static_cast<int64_t>(t) * D) = kr[i];
      *reinterpret_cast<uint4*>(vo + static_cast<int64_t>(t) * D) = vr[i];
      float f[CH];
      Chunk<T>::unpack(kr[i], f);
#pragma unroll
      for (int e = 0; e < CH; ++e) { mn[e] = fminf(mn[e], f[e]); mx[e] = fmaxf(mx[e], f[e]); }
    }
  }
  if (a.desc_out == nullptr) return;
#pragma unroll
  for (int m = CPR; m < 32; m <<= 1) {
#pragma unroll
    for (int e = 0; e < CH; ++e) {
      mn[e] = fminf(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], m));
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], m));
    }
  }
  if (lane < CPR) {
    T* d = static_cast<T*>(a.desc_out) + (bh * (a.L_out / kBlock) + j) * 2 * D + chunk * CH;
    *reinterpret_cast<uint4*>(d) = Chunk<T>::pack(mn);
    *reinterpret_cast<uint4*>(d + D) = Chunk<T>::pack(mx);
  }
}

template <typename T, int D>
static cudaError_t gather_t(const Shape& s, const EvictArgs& a, cudaStream_t st) {
  const int64_t most = a.len < a.budget ? a.len : a.budget;
  const int M = static_cast<int>((most + kBlock - 1) / kBlock);
  const int64_t total = static_cast<int64_t>(s.B) * s.H * M;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((total * 32 + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_gather_kernel<T, D>, a, s.H, s.L_max, M, total);
}

template <int CL, int KPT>
static cudaError_t evict_select_t(const Shape& s, const EvictArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CL, s.H, s.B);
  cfg.blockDim = dim3(kEvThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<CL, KPT>, a.weights, a.kept, s.H, s.L_max,
                            a.len, a.lens, a.budget, a.recent, a.ctrl);
}

// One CTA up to 8192 tokens (no cluster barriers), eight up to 131072 with
// their slices in registers, eight of any length beyond (32 keys per thread
// spill).
cudaError_t launch_evict(const Shape& s, const EvictArgs& a, cudaStream_t st) {
  cudaError_t e;
  if (a.len <= 8 * kEvThreads) e = evict_select_t<1, 8>(s, a, st);
  else if (a.len <= 8 * kEvCluster * kEvThreads) e = evict_select_t<kEvCluster, 8>(s, a, st);
  else if (a.len <= 16 * kEvCluster * kEvThreads) e = evict_select_t<kEvCluster, 16>(s, a, st);
  else e = evict_select_t<kEvCluster, 0>(s, a, st);
  if (e != cudaSuccess) return e;
  if (s.bf16)
    return s.D == 128 ? gather_t<__nv_bfloat16, 128>(s, a, st) : gather_t<__nv_bfloat16, 64>(s, a, st);
  return s.D == 128 ? gather_t<float, 128>(s, a, st) : gather_t<float, 64>(s, a, st);
}

}  // namespace resa
