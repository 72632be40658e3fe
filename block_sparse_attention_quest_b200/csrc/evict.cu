// Accumulated attention weights, and a cache cut to the tokens that gathered
// the most of them.
//
// A decode step's weight of token t for KV group g is the sum over the group's
// heads h of exp(scale q_h . k_t - lse_h). The attention kernel leaves every
// logit (log2 units) and each head's (max m, sum l) in the workspace; the sums
//   w_t += sum_h 2^(logit_ht - m_h) / l_h
// follow in a kernel of their own, because no weight is known before the last
// split has been merged. Reading the logits back (4 bytes per head and token,
// from L2) replaces a second pass over the keys (2 d bytes per token).
//
// Eviction keeps, per (row, KV head), the newest `recent` tokens and of the
// others the budget - recent with the largest sums, in their order.
#include <cooperative_groups.h>

#include "select_core.cuh"

namespace resa {

namespace cg = cooperative_groups;

// Grid (tokens / 256, H, B): one token per thread.
__global__ void __launch_bounds__(256) add_weights_kernel(const float* __restrict__ logits,
                                                          const float* __restrict__ ml,
                                                          float* __restrict__ weights, int H, int G,
                                                          int64_t stride, int64_t L_max,
                                                          int64_t len, const int32_t* lens,
                                                          bool fresh) {
  __shared__ float s_m[8], s_inv[8];
  grid_dependency_wait();
  grid_launch_dependents();
  const int g = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * H + g;
  if (threadIdx.x < G) {
    const float2 p = __ldcg(reinterpret_cast<const float2*>(ml) + bh * G + threadIdx.x);
    s_m[threadIdx.x] = p.x;
    s_inv[threadIdx.x] = 1.f / p.y;
  }
  __syncthreads();
  const int64_t len_b = row_len(lens, len, b);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (t >= len_b) return;
  const float* z = logits + (bh * stride + t) * G;
  float x[8];
  if ((G & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (4 * i < G) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(z) + i);
        x[4 * i] = y.x; x[4 * i + 1] = y.y; x[4 * i + 2] = y.z; x[4 * i + 3] = y.w;
      }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < G) x[i] = __ldcg(z + i);
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < G) sum = fmaf(exp2f(x[i] - s_m[i]), s_inv[i], sum);
  float* w = weights + bh * L_max + t;
  *w = fresh && t == len_b - 1 ? sum : *w + sum;
}

cudaError_t launch_add_weights(const Shape& s, const float* logits, const float* ml,
                               float* weights, int64_t len, const int32_t* lens, bool fresh,
                               cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((len + 255) / 256), s.H, s.B);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, add_weights_kernel, logits, ml, weights, s.H, s.G,
                            (len + kBlock - 1) / kBlock * kBlock, s.L_max, len, lens, fresh);
}

// ---------------------------------------------------------------------- select
constexpr int kEvThreads = 512;
constexpr int kEvCluster = 8;        // CTAs per (row, KV head), each with a slice of its tokens

// order-preserving key of a weight; NaN below every number
__device__ __forceinline__ uint32_t weight_key(float w) { return w == w ? score_key(w) : 0u; }

// Exclusive prefix sum of x over the CTA's threads; *total receives the sum.
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
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kEvThreads / 32; ++w) {
    const uint32_t c = warp_tot[w];
    before += w < warp ? c : 0u;
    all += c;
  }
  __syncthreads();
  total = all;
  return before + inc - x;
}

// A cluster of eight CTAs per (row, KV head). Three radix passes (11, 11 and
// 10 bits of the keys, from the top) find the exact threshold key: every CTA
// counts its slice into its own histogram, and after a cluster barrier all of
// them read all eight through distributed shared memory and take the same
// decision, so one barrier per pass suffices (each pass has a histogram of its
// own). Then each CTA counts the keys above and equal to the threshold in its
// slice, the eight counts give its place in the list, and warps that own
// contiguous ranges write it in order.
__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const float* __restrict__ weights,
                                                                  int32_t* __restrict__ kept, int H,
                                                                  int64_t L_max, int64_t len,
                                                                  const int32_t* lens, int budget,
                                                                  int recent, Ctrl* ctrl) {
  __shared__ __align__(16) uint32_t hist[3][kBins];
  __shared__ uint32_t warp_tot[kEvThreads / 32];
  __shared__ uint32_t s_prefix, s_remaining;
  __shared__ uint32_t s_count[2];                 // keys above, equal to the threshold
  cg::cluster_group cluster = cg::this_cluster();
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster.block_rank());
  const int g = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * H + g;
  int32_t* out = kept + bh * budget;
  if (rank == 0 && g == 0 && tid == 0 && row_len_bad(lens, len, b)) raise_error(ctrl, kErrBadIndex);
  const int n = static_cast<int>(row_len(lens, len, b));
  const int all = kEvCluster * kEvThreads;
  const int me = rank * kEvThreads + tid;
  if (n <= budget) {                              // nothing to evict (whole cluster)
    for (int i = me; i < budget; i += all) out[i] = i < n ? i : -1;
    return;
  }
  const int cand = n - recent, need = budget - recent;
  for (int i = me; i < recent; i += all) out[need + i] = cand + i;
  if (need == 0) return;
  const float* w = weights + bh * L_max;
  const int per = (cand + kEvCluster * 128 - 1) / (kEvCluster * 128) * 128;
  const int c0 = min(cand, rank * per), c1 = min(cand, c0 + per);
  for (int i = tid; i < 3 * kBins; i += kEvThreads) (&hist[0][0])[i] = 0u;
  if (tid == 0) { s_prefix = 0u; s_remaining = static_cast<uint32_t>(need); }
  __syncthreads();
  // calls f(index, key) for every key of [from, to), four loads at a time
  auto each = [&](auto&& f) {
    for (int j0 = c0 + tid * 4; j0 < c1; j0 += 4 * 4 * kEvThreads) {
      float4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + u * 4 * kEvThreads;
        // (a slice starts at a multiple of 128 and rows hold a multiple of 16)
        if (j < c1) x[u] = __ldcg(reinterpret_cast<const float4*>(w + j));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = j0 + u * 4 * kEvThreads;
        const float y[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < c1) f(weight_key(y[e]));
      }
    }
  };
  uint32_t prefix = 0, remaining = static_cast<uint32_t>(need);
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    const uint32_t above = pass == 0 ? 0u : (pass == 1 ? 0xffe00000u : 0xfffffc00u);
    uint32_t* h = hist[pass];
    each([&](uint32_t key) {
      if ((key & above) == prefix) atomicAdd(&h[(key >> shift) & mask], 1u);
    });
    cluster.sync();
    // thread t owns bins 2047 - 4t .. 2044 - 4t, from the top
    uint32_t c[4] = {0u, 0u, 0u, 0u};
    uint4 r[kEvCluster];
#pragma unroll
    for (int i = 0; i < kEvCluster; ++i)
      r[i] = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(h, i) + kBins - 4 - 4 * tid);
#pragma unroll
    for (int i = 0; i < kEvCluster; ++i) {
      c[0] += r[i].w; c[1] += r[i].z; c[2] += r[i].y; c[3] += r[i].x;
    }
    uint32_t total;
    uint32_t before = ev_scan(c[0] + c[1] + c[2] + c[3], warp_tot, total);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (before < remaining && remaining <= before + c[e]) {
        s_prefix = prefix | (static_cast<uint32_t>(kBins - 1 - 4 * tid - e) << shift);
        s_remaining = remaining - before;
      }
      before += c[e];
    }
    __syncthreads();
    prefix = s_prefix;
    remaining = s_remaining;
    __syncthreads();
  }
  // every key above T, and the `remaining` of lowest index among those equal
  const uint32_t T = prefix;
  const int chunk = per / (kEvThreads / 32) > 32 ? (per / (kEvThreads / 32) + 31) / 32 * 32 : 32;
  const int wb = min(c1, c0 + warp * chunk), we = min(c1, wb + chunk);
  uint32_t gt = 0, eq = 0;
  for (int j0 = wb; j0 < we; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t key = j < we ? weight_key(__ldcg(w + j)) : 0u;
    gt += __popc(__ballot_sync(0xffffffffu, j < we && key > T));
    eq += __popc(__ballot_sync(0xffffffffu, j < we && key == T));
  }
  uint32_t gt_all, eq_all;
  uint32_t gt_at = ev_scan(lane == 0 ? gt : 0u, warp_tot, gt_all);
  uint32_t eq_at = ev_scan(lane == 0 ? eq : 0u, warp_tot, eq_all);
  gt_at = __shfl_sync(0xffffffffu, gt_at, 0);
  eq_at = __shfl_sync(0xffffffffu, eq_at, 0);
  if (tid == 0) { s_count[0] = gt_all; s_count[1] = eq_all; }
  cluster.sync();
  for (int i = 0; i < rank; ++i) {
    const uint32_t* other = cluster.map_shared_rank(s_count, i);
    gt_at += other[0];
    eq_at += other[1];
  }
  cluster.sync();                                 // no CTA leaves while another reads it
  uint32_t pos = gt_at + min(eq_at, remaining);
  const uint32_t lt = (1u << lane) - 1u;
  for (int j0 = wb; j0 < we; j0 += 32) {
    const int j = j0 + lane;
    const uint32_t key = j < we ? weight_key(__ldcg(w + j)) : 0u;
    const uint32_t eqb = __ballot_sync(0xffffffffu, j < we && key == T);
    const bool take = j < we && (key > T || (key == T && eq_at + __popc(eqb & lt) < remaining));
    eq_at += __popc(eqb);
    const uint32_t tb = __ballot_sync(0xffffffffu, take);
    if (take) out[pos + __popc(tb & lt)] = j;
    pos += __popc(tb);
  }
}

// ---------------------------------------------------------------------- gather
// One warp per 16-token block of the new cache: its rows are copied from where
// `kept` says, their minimum and maximum become the block's descriptor.
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

cudaError_t launch_evict(const Shape& s, const EvictArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kEvCluster, s.H, s.B);
  cfg.blockDim = dim3(kEvThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kEvCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a.weights, a.kept, s.H, s.L_max,
                                     a.len, a.lens, a.budget, a.recent, a.ctrl);
  if (e != cudaSuccess) return e;
  if (s.bf16)
    return s.D == 128 ? gather_t<__nv_bfloat16, 128>(s, a, st) : gather_t<__nv_bfloat16, 64>(s, a, st);
  return s.D == 128 ? gather_t<float, 128>(s, a, st) : gather_t<float, 64>(s, a, st);
}

}  // namespace resa
