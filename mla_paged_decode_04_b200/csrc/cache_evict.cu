// Eviction from the paged cache by accumulated attention weight: per entry,
// which keys stay (cache_evict_select_kernel), then their rows onto the pages
// of another table (cache_evict_move_kernel, its programmatic dependent).
//
// Selection. Between the protected first `sinks` and last `recent` keys the
// k = budget - sinks - recent largest weights stay. A weight maps to a 32-bit
// number that orders like it (sign folded, -0 as +0, NaN below everything), and
// three passes over 11, 11 and 10 bits, from the top, find the k-th largest
// exactly: a histogram of the digit among the weights that agree with the
// digits found so far, then the digit at which the count from above reaches k.
// All weights above it stay, and of those equal to it the ones at the lowest
// positions. Positions are then compacted in order: every warp counts its own
// run, the counts before it give where it starts, and a second walk writes.
//
// The weights are read from HBM once (4 bytes a key, little next to the rows
// that move), so what bounds the selection is the latency of its passes. One
// cluster of up to 8 CTAs per entry, each with its stretch of the weights in
// shared memory. After a pass CTA r sums its share of the bins over all
// histograms through distributed shared memory; every CTA then knows the shares'
// totals, reads the one share that holds the digit and finds it itself: two
// cluster barriers a pass. (Every CTA reading all histograms took one barrier
// but 4-byte remote reads of 64 KB a pass: 48 us for 16 x 81,920 weights, of
// which @@SEL@@ now.)
//
// Moving. HBM-bound: 2 * 576 (FP8) or 2 * 1152 bytes per row that stays. A warp
// takes 288 16-byte chunks at a time (8 FP8 or 4 16-bit rows): the lanes look up
// the rows' places together, then each has nine loads in flight before its
// first store.
#include "device_common.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kSelThreads = 512;  // 1024 leave one CTA an SM: of 16 clusters of 8 half waited for the others
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxHeld = 48 * 1024;  // numbers a CTA keeps in shared memory; of longer stretches none

// Orders as the weights do: larger weight, larger number.
__device__ __forceinline__ uint32_t weight_order(float w) {
  if (w != w) return 0u;
  const uint32_t b = w == 0.f ? 0u : __float_as_uint(w);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ int evict_len(const EvictArgs& e, int b, bool flag) {
  int n = e.seq_lens[b];
  const int64_t cap = min(e.cols, (int64_t)e.max_pages_per_seq * kTileKeys);
  if ((n < 0 || (int64_t)n > cap) && flag && e.status) atomicOr(e.status, MLA_DEV_SEQ_TOO_LONG);
  if (n < 0) n = 0;
  return (int64_t)n > cap ? (int)cap : n;
}

__device__ __forceinline__ int ld_cluster(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int4 ld_cluster4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// held: room for the weights of a CTA's stretch (0: read them again at each
// use).
__global__ void __launch_bounds__(kSelThreads, 2) cache_evict_select_kernel(const EvictArgs e, int ctas, int held) {
  extern __shared__ __align__(16) uint32_t held_u[];
  __shared__ __align__(16) int hist[3][kBins];
  __shared__ __align__(16) int share[kBins];  // this CTA's bins, summed over the cluster
  __shared__ int s_share[kMaxCluster];        // the shares' totals, from the top
  __shared__ int s_warp[kSelWarps];
  __shared__ int s_digit, s_left;
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps], s_total[2];
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  ptx::launch_dependents();
  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
  ptx::grid_dep_wait();  // nothing above reads or writes global memory
  const int n = evict_len(e, b, tid == 0 && rank == 0);
  const float* w = e.weights + (int64_t)b * e.weights_stride;
  int32_t* kept = e.kept + (int64_t)b * e.budget;
  float* ow = e.out_weights ? e.out_weights + (int64_t)b * e.out_weights_stride : nullptr;
  auto keep = [&](int i, int j, float x) {
    kept[i] = j;
    if (ow) ow[i] = x;
  };
  // every CTA has read the length when rank 0 writes the new one, after a
  // cluster barrier (out_seq_lens may be seq_lens)
  if (n <= e.budget) {
    for (int i = rank * kSelThreads + tid; i < e.budget; i += ctas * kSelThreads) {
      if (i < n)
        keep(i, i, w[i]);
      else
        kept[i] = -1;
    }
    ptx::cluster_sync();
    if (rank == 0 && tid == 0) e.out_seq_lens[b] = n;
    return;
  }
  const int lo = e.sinks, hi = n - e.recent, k = e.budget - e.sinks - e.recent;
  for (int i = rank * kSelThreads + tid; i < e.sinks; i += ctas * kSelThreads) keep(i, i, w[i]);
  for (int i = rank * kSelThreads + tid; i < e.recent; i += ctas * kSelThreads)
    keep(e.budget - e.recent + i, hi + i, w[hi + i]);
  if (k == 0) {
    ptx::cluster_sync();
    if (rank == 0 && tid == 0) e.out_seq_lens[b] = e.budget;
    return;
  }
  // this CTA's stretch [c0, c1) of the candidates
  const int per_cta = (hi - lo + ctas - 1) / ctas;
  const int c0 = min(hi, lo + rank * per_cta), c1 = min(hi, c0 + per_cta);
  const bool hold = c1 - c0 <= held;
  auto number = [&](int j) -> uint32_t { return hold ? held_u[j - c0] : weight_order(w[j]); };
  __syncthreads();  // the histograms are zero
  constexpr int kAhead = 8;  // loads in flight per thread
  for (int jb = c0; jb < c1; jb += kAhead * kSelThreads) {
    float x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = jb + i * kSelThreads + tid;
      x[i] = j < c1 ? w[j] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int j = jb + i * kSelThreads + tid;
      if (j >= c1) break;
      const uint32_t u = weight_order(x[i]);
      if (hold) held_u[j - c0] = u;
      atomicAdd(&hist[0][u >> 21], 1);
    }
  }
  // the weight of a number; the zeros and the NaNs share one, theirs are read again
  auto weight_of = [&](uint32_t u, int j) -> float {
    if (u == 0u || u == 0x80000000u) return w[j];
    return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
  };
  uint32_t prefix = 0;  // the digits found so far
  int left = k;         // how many of the weights that agree with them stay
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    ptx::cluster_sync();  // every CTA's histogram of this pass is complete
    // CTA r's share: bins [kBins - (r + 1) * size, kBins - r * size), four per thread
    const int size = kBins / ctas;
    if (tid < size / 4) {
      const uint32_t at = ptx::smem_u32(&hist[pass][kBins - (rank + 1) * size + 4 * tid]);
      int4 sum = make_int4(0, 0, 0, 0);
      int4 x[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)  // all in flight before the first is used
        x[r] = r < ctas ? ld_cluster4(ptx::mapa(at, (uint32_t)r)) : make_int4(0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) sum.x += x[r].x, sum.y += x[r].y, sum.z += x[r].z, sum.w += x[r].w;
      *reinterpret_cast<int4*>(&share[4 * tid]) = sum;
      const int t = __reduce_add_sync(0xffffffffu, sum.x + sum.y + sum.z + sum.w);
      if (lane == 0) s_warp[warp] = t;
    }
    __syncthreads();
    if (tid < ctas) {
      int t = 0;
      for (int i = 0; i < size / 128; ++i) t += s_warp[i];
      st_cluster(ptx::mapa(ptx::smem_u32(&s_share[rank]), (uint32_t)tid), t);
    }
    ptx::cluster_sync();  // every share and every total is in place
    int owner = 0, above = 0;
    while (owner < ctas - 1 && above + s_share[owner] < left) above += s_share[owner++];
    // thread t: bins 4t' + 3 .. 4t' of the owner's share, t' counted from the top
    if (tid < size / 4) {
      const int top = size / 4 - 1 - tid;
      const int4 x = ld_cluster4(ptx::mapa(ptx::smem_u32(&share[4 * top]), (uint32_t)owner));
      const int c[4] = {x.w, x.z, x.y, x.x};
      int incl = c[0] + c[1] + c[2] + c[3];
      const int own = incl;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      if (lane == 31) s_warp[warp] = incl;  // (its last readers are behind the cluster barrier)
      if (size > 128) asm volatile("bar.sync 1, %0;" ::"r"(size / 4) : "memory");
      above += incl - own + __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < left && left <= above + c[i]) {
          s_digit = kBins - owner * size - 1 - 4 * tid - i;
          s_left = left - above;
        }
        above += c[i];
      }
    }
    __syncthreads();
    const int bits = pass == 2 ? 10 : 11;
    prefix = (prefix << bits) | (uint32_t)s_digit;
    left = s_left;
    if (pass < 2) {
      const int found = pass == 0 ? 21 : 10;  // bits below the digits found
      auto count = [&](uint32_t u) {
        if ((u >> found) == prefix) atomicAdd(&hist[pass + 1][pass == 0 ? (u >> 10) & 2047u : u & 1023u], 1);
      };
      if (hold) {  // four numbers at a time
        const int n4 = (c1 - c0) >> 2;
        for (int i = tid; i < n4; i += kSelThreads) {
          const uint4 u = reinterpret_cast<const uint4*>(held_u)[i];
          count(u.x), count(u.y), count(u.z), count(u.w);
        }
        if (4 * n4 + tid < c1 - c0) count(held_u[4 * n4 + tid]);
      } else {
        for (int j = c0 + tid; j < c1; j += kSelThreads) count(weight_order(w[j]));
      }
    }
  }
  const uint32_t cut = prefix;
  const int ties = left;  // weights equal to the cut that stay
  const int per = ((c1 - c0 + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int j0 = min(c1, c0 + warp * per), j1 = min(c1, j0 + per);
  int gt = 0, eq = 0;
  for (int j = j0 + lane; j < j1; j += 32) {
    const uint32_t u = number(j);
    gt += u > cut;
    eq += u == cut;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) s_gt[warp] = gt, s_eq[warp] = eq;
  __syncthreads();
  int gt0 = __reduce_add_sync(0xffffffffu, lane < warp ? s_gt[lane] : 0);  // before this warp's run
  int eq0 = __reduce_add_sync(0xffffffffu, lane < warp ? s_eq[lane] : 0);
  if (warp == kSelWarps - 1 && lane == 0) s_total[0] = gt0 + gt, s_total[1] = eq0 + eq;
  ptx::cluster_sync();
  if (rank == 0 && tid == 0) e.out_seq_lens[b] = e.budget;
  {
    const int x = lane < rank ? ld_cluster(ptx::mapa(ptx::smem_u32(&s_total[0]), (uint32_t)lane)) : 0;
    const int y = lane < rank ? ld_cluster(ptx::mapa(ptx::smem_u32(&s_total[1]), (uint32_t)lane)) : 0;
    gt0 += __reduce_add_sync(0xffffffffu, x);
    eq0 += __reduce_add_sync(0xffffffffu, y);
  }
  for (int jb = j0; jb < j1; jb += 32) {
    const int j = jb + lane;
    const uint32_t u = j < j1 ? number(j) : 0u;
    const unsigned g = __ballot_sync(0xffffffffu, j < j1 && u > cut);
    const unsigned q = __ballot_sync(0xffffffffu, j < j1 && u == cut);
    const unsigned before = (1u << lane) - 1u;
    const int eq_before = eq0 + __popc(q & before);
    if (((g >> lane) & 1u) || (((q >> lane) & 1u) && eq_before < ties))
      keep(e.sinks + gt0 + __popc(g & before) + min(eq_before, ties), j, weight_of(u, j));
    gt0 += __popc(g);
    eq0 += __popc(q);
  }
  ptx::cluster_sync();  // no CTA leaves while another may read its shared memory
}

constexpr int kMoveChunks = 9;  // 16-byte chunks of a lane: a warp moves 288 at a time

template <int kRowBytes>
__global__ void __launch_bounds__(256) cache_evict_move_kernel(const EvictArgs e) {
  constexpr int kPer = kRowBytes / 16;                  // chunks of a row
  constexpr int kRows = 32 * kMoveChunks / kPer;        // rows of a warp's step
  static_assert(32 * kMoveChunks % kPer == 0 && kTileKeys % kRows == 0, "whole rows, within a page");
  const int steps = (e.budget + kTileKeys - 1) / kTileKeys * (kTileKeys / kRows);  // of an entry, last page's rest too
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  const int64_t total = (int64_t)e.batch * steps;
  ptx::grid_dep_wait();
  for (int64_t it = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < total; it += warps) {
    const int b = (int)(it / steps), i0 = (int)(it - (int64_t)b * steps) * kRows;
    const int len = e.out_seq_lens[b];
    if (i0 >= ((len + kTileKeys - 1) & ~(kTileKeys - 1))) continue;  // (the same for the whole warp)
    const int to = e.out_block_tables[(int64_t)b * e.out_max_pages_per_seq + i0 / kTileKeys];
    if (to < 0 || (int64_t)to >= e.out_num_pages) {
      if (e.status && lane == 0) atomicOr(e.status, MLA_DEV_BAD_PAGE);
      continue;
    }
    // lane r: the source row of row i0 + r, or -1 (past the length, or on a
    // page outside the cache: zeros arrive)
    int64_t from = -1;
    if (lane < kRows && i0 + lane < len) {
      const int j = e.kept[(int64_t)b * e.budget + i0 + lane];
      const int pg = e.block_tables[(int64_t)b * e.max_pages_per_seq + j / kTileKeys];
      if (pg < 0 || (int64_t)pg >= e.num_pages) {
        if (e.status) atomicOr(e.status, MLA_DEV_BAD_PAGE);
      } else {
        from = (int64_t)pg * kTileKeys + j % kTileKeys;
      }
    }
    uint4 v[kMoveChunks];
#pragma unroll
    for (int u = 0; u < kMoveChunks; ++u) {
      const int c = 32 * u + lane, r = c / kPer;
      const int64_t row = __shfl_sync(0xffffffffu, from, r);
      v[u] = row < 0 ? make_uint4(0, 0, 0, 0)
                     : __ldcs(reinterpret_cast<const uint4*>(e.kv_cache + row * kRowBytes + 16 * (c - r * kPer)));
    }
    uint4* dst = reinterpret_cast<uint4*>(e.out_cache + ((int64_t)to * kTileKeys + i0 % kTileKeys) * kRowBytes);
#pragma unroll
    for (int u = 0; u < kMoveChunks; ++u) dst[32 * u + lane] = v[u];
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& e, cudaStream_t stream) {
  // CTAs per entry: as many as the SMs hold at two each, with at least 1024
  // candidates for each
  const int64_t longest = e.cols < (int64_t)e.max_pages_per_seq * kTileKeys ? e.cols
                                                                            : (int64_t)e.max_pages_per_seq * kTileKeys;
  int ctas = 1;
  while (ctas < kMaxCluster && (int64_t)e.batch * ctas * 2 <= 2 * kNumSMs && longest >= 2048 * ctas) ctas *= 2;
  const int64_t stretch = (longest + ctas - 1) / ctas;
  const int held = stretch <= kMaxHeld ? (int)stretch : 0;
  static std::atomic<uint64_t> smem_set{0};
  if (cudaError_t rc = set_max_dynamic_smem((const void*)cache_evict_select_kernel, kMaxHeld * 4, smem_set);
      rc != cudaSuccess)
    return rc;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)e.batch * (unsigned)ctas);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (size_t)held * 4;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaError_t rc = cudaLaunchKernelEx(&cfg, cache_evict_select_kernel, e, ctas, held); rc != cudaSuccess) return rc;
  const int64_t pages = (int64_t)e.batch * ((e.budget + kTileKeys - 1) / kTileKeys);
  const int64_t blocks = (pages * kTileKeys * (e.row_bytes / 16) + 8 * 32 * kMoveChunks - 1) / (8 * 32 * kMoveChunks);
  cfg.gridDim = dim3((unsigned)(blocks < kNumSMs * 8 ? blocks : kNumSMs * 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return e.row_bytes == MLA_D_QK ? cudaLaunchKernelEx(&cfg, cache_evict_move_kernel<MLA_D_QK>, e)
                                 : cudaLaunchKernelEx(&cfg, cache_evict_move_kernel<2 * MLA_D_QK>, e);
}

}  // namespace mla
