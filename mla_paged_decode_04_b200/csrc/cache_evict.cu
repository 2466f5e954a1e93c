// Eviction from the paged cache by accumulated attention weight: per entry,
// which keys stay, then their rows onto the pages of another table.
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
// CTA per entry or a cluster of up to 8, each with its stretch of the weights in
// shared memory. After a pass CTA r sums its share of the bins over all
// histograms through distributed shared memory; every CTA then knows the shares'
// totals, reads the one share that holds the digit and finds it itself: two
// cluster barriers a pass, none where one CTA has the entry to itself.
//
// Moving. HBM-bound: 2 * 576 (FP8) or 2 * 1152 bytes per row that stays. A warp
// takes 288 16-byte chunks at a time (8 FP8 or 4 16-bit rows): the lanes look up
// the rows' places together, then each has nine loads in flight before its
// first store. Where the clusters fill three of four places (two CTAs an SM),
// each moves its own entry's rows as soon as it has chosen them: one launch, and
// entries that are done early keep HBM busy while others select. With fewer a
// second kernel, a programmatic dependent, spreads the rows over all SMs.
//
// Measured (replayed graphs): 16 x 81,920 FP8 weights to 8192 keys 50 us, of
// which the selection 22 and the moving 28 (5.4 TB/s); 64 x 1000..16,384 BF16 to
// 2000 keys 64 us (4.5 TB/s in all); one entry of 1100 keys to 1024 8 us.
#include "device_common.cuh"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kSelThreads = 512;  // 1024 leave one CTA an SM: of 16 clusters of 8 half waited for the others
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelPerSM = MLA_BOUNDS_CHECK ? 1 : 2;  // (the checks take more than 64 registers)
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxHeld = 48 * 1024;  // numbers a CTA keeps in shared memory; of longer stretches none

// Orders as the weights do: larger weight, larger number.
__device__ __forceinline__ uint32_t weight_order(float w) {
  if (w != w) return 0u;
  const uint32_t b = w == 0.f ? 0u : __float_as_uint(w);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Bounds check of the checking build (see in_bounds): whether i lies in [0, n).
__device__ __forceinline__ bool evict_in_bounds(const EvictArgs& e, int64_t i, int64_t n) {
#if MLA_BOUNDS_CHECK
  if (i >= 0 && i < n) return true;
  if (e.status) atomicOr(e.status, MLA_DEV_BOUNDS);
  return false;
#else
  (void)e, (void)i, (void)n;
  return true;
#endif
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
__device__ __forceinline__ void add_cluster(uint32_t addr, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

constexpr int kMoveChunks = 9;  // 16-byte chunks of a lane: a warp moves 288 at a time

// Step `it` of entry b's rows, by one warp. kept and out_len may have been
// written by other CTAs of the cluster or by the kernel before.
template <int kRowBytes>
__device__ __forceinline__ void move_step(const EvictArgs& e, int b, int it, int len) {
  constexpr int kPer = kRowBytes / 16;                  // chunks of a row
  constexpr int kRows = 32 * kMoveChunks / kPer;        // rows of a step
  static_assert(32 * kMoveChunks % kPer == 0 && kTileKeys % kRows == 0, "whole rows, within a page");
  const int lane = threadIdx.x & 31, i0 = it * kRows;
  if (!evict_in_bounds(e, b, e.batch) || !evict_in_bounds(e, i0 / kTileKeys, e.out_max_pages_per_seq)) return;
  const int to = e.out_block_tables[(int64_t)b * e.out_max_pages_per_seq + i0 / kTileKeys];
  if (to < 0 || (int64_t)to >= e.out_num_pages) {
    if (e.status && lane == 0) atomicOr(e.status, MLA_DEV_BAD_PAGE);
    return;
  }
  // lane r: the source row of row i0 + r, or -1 (past the length, or on a page
  // outside the cache: zeros arrive)
  int64_t from = -1;
  if (lane < kRows && i0 + lane < len && evict_in_bounds(e, i0 + lane, e.budget)) {
    const int j = e.kept[(int64_t)b * e.budget + i0 + lane];
    const bool in_table = evict_in_bounds(e, j, (int64_t)e.max_pages_per_seq * kTileKeys);
    const int pg = in_table ? e.block_tables[(int64_t)b * e.max_pages_per_seq + j / kTileKeys] : -1;
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
// Steps that cover `len` rows and the rest of their last page.
template <int kRowBytes>
__device__ __forceinline__ int move_steps(int len) {
  constexpr int kRows = 32 * kMoveChunks * 16 / kRowBytes;
  return (len + kTileKeys - 1) / kTileKeys * (kTileKeys / kRows);
}

template <int kRowBytes>
__global__ void __launch_bounds__(256) cache_evict_move_kernel(const EvictArgs e) {
  const int steps = move_steps<kRowBytes>(e.budget);
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  const int64_t total = (int64_t)e.batch * steps;
  ptx::grid_dep_wait();
  for (int64_t it = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < total; it += warps) {
    const int b = (int)(it / steps), step = (int)(it - (int64_t)b * steps);
    const int len = __ldcg(e.out_seq_lens + b);  // (may be seq_lens, which L1 may hold as it was)
    if (step < move_steps<kRowBytes>(len)) move_step<kRowBytes>(e, b, step, len);
  }
}

// held: room for the weights of a CTA's stretch (0: read them again at each
// use). kRowBytes > 0: the cluster moves its entry's rows too.
template <bool kCluster, int kRowBytes>
__global__ void __launch_bounds__(kSelThreads, kSelPerSM) cache_evict_select_kernel(const EvictArgs e, int ctas_arg, int held) {
  extern __shared__ __align__(16) uint32_t held_u[];
  __shared__ __align__(16) int hist[3][kBins];
  __shared__ __align__(16) int share[kCluster ? kBins / 2 : 4];      // this CTA's bins, summed over the cluster
  __shared__ __align__(16) int s_share[3][kMaxCluster];              // per pass the shares' totals, from the top
  __shared__ int s_warp[kSelWarps];
  __shared__ int s_digit, s_left;
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps], s_total[2];
  const int ctas = kCluster ? ctas_arg : 1;
  const int b = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto barrier = [&]() {
    if constexpr (kCluster) ptx::cluster_sync(); else __syncthreads();
  };
  if (kRowBytes == 0) ptx::launch_dependents();
  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
  if (tid < 3 * kMaxCluster) (&s_share[0][0])[tid] = 0;
  ptx::grid_dep_wait();  // nothing above reads or writes global memory
  const int n = evict_len(e, b, tid == 0 && rank == 0);
  const int len = min(n, e.budget);
  const float* w = e.weights + (int64_t)b * e.weights_stride;
  auto weight_at = [&](int j) -> float { return evict_in_bounds(e, j, e.cols) ? w[j] : 0.f; };
  int32_t* kept = e.kept + (int64_t)b * e.budget;
  float* ow = e.out_weights ? e.out_weights + (int64_t)b * e.out_weights_stride : nullptr;
  auto keep = [&](int i, int j, float x) {
    if (!evict_in_bounds(e, i, e.budget)) return;
    kept[i] = j;
    if (ow) ow[i] = x;
  };
  // When every CTA of the cluster is past a barrier with its share of kept
  // written: the length (only then has every CTA read the old one, and
  // out_seq_lens may be seq_lens), the rows, and a last barrier, since no CTA may
  // leave while another may read its shared memory.
  auto finish = [&]() {
    barrier();
    if (rank == 0 && tid == 0) e.out_seq_lens[b] = len;
    if constexpr (kRowBytes > 0) {
      const int steps = move_steps<kRowBytes>(len);
      for (int it = rank * kSelWarps + warp; it < steps; it += ctas * kSelWarps) move_step<kRowBytes>(e, b, it, len);
    }
  };
  if (n <= e.budget) {
    for (int i = rank * kSelThreads + tid; i < e.budget; i += ctas * kSelThreads) {
      if (i < n)
        keep(i, i, weight_at(i));
      else
        kept[i] = -1;
    }
    finish();
    return;
  }
  const int lo = e.sinks, hi = n - e.recent, k = e.budget - e.sinks - e.recent;
  // the protected keys: position i of the sinks and the recent ones together
  const int safe = e.sinks + e.recent;
  auto keep_safe = [&](int i, float x) {
    if (i < e.sinks) keep(i, i, x); else keep(k + i, hi + i - e.sinks, x);
  };
  auto safe_weight = [&](int i) -> float { return weight_at(i < e.sinks ? i : hi + i - e.sinks); };
  const int safe0 = rank * kSelThreads + tid;
  const float x_safe = safe0 < safe ? safe_weight(safe0) : 0.f;  // (its store comes after the loads below)
  // this CTA's stretch [c0, c1) of the candidates
  const int per_cta = (hi - lo + ctas - 1) / ctas;
  const int c0 = min(hi, lo + rank * per_cta), c1 = min(hi, c0 + per_cta);
  const bool hold = c1 - c0 <= held;
  auto number = [&](int j) -> uint32_t { return hold ? held_u[j - c0] : weight_order(weight_at(j)); };
  if (k > 0) {
    __syncthreads();  // the histograms are zero
    constexpr int kAhead = 12;  // loads in flight per thread
    for (int jb = c0; jb < c1; jb += kAhead * kSelThreads) {
      float x[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = jb + i * kSelThreads + tid;
        x[i] = j < c1 ? weight_at(j) : 0.f;
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
  }
  if (safe0 < safe) keep_safe(safe0, x_safe);
  for (int i = safe0 + ctas * kSelThreads; i < safe; i += ctas * kSelThreads) keep_safe(i, safe_weight(i));
  if (k == 0) {
    finish();
    return;
  }
  uint32_t prefix = 0;  // the digits found so far
  int left = k;         // how many of the weights that agree with them stay
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    barrier();  // every CTA's histogram of this pass is complete
    const int size = kBins / ctas;  // bins of a share, four per thread
    int owner = 0, above = 0;
    if constexpr (kCluster) {
      // CTA r's share: bins [kBins - (r + 1) * size, kBins - r * size)
      if (tid < size / 4) {
        const uint32_t at = ptx::smem_u32(&hist[pass][kBins - (rank + 1) * size + 4 * tid]);
        int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll
        for (int h = 0; h < kMaxCluster; h += 4) {
          int4 x[4];
#pragma unroll
          for (int r = 0; r < 4; ++r)  // in flight together
            x[r] = h + r < ctas ? ld_cluster4(ptx::mapa(at, (uint32_t)(h + r))) : make_int4(0, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; ++r) sum.x += x[r].x, sum.y += x[r].y, sum.z += x[r].z, sum.w += x[r].w;
        }
        *reinterpret_cast<int4*>(&share[4 * tid]) = sum;
        const int t = __reduce_add_sync(0xffffffffu, sum.x + sum.y + sum.z + sum.w);
        if (lane < ctas) add_cluster(ptx::mapa(ptx::smem_u32(&s_share[pass][rank]), (uint32_t)lane), t);
      }
      barrier();  // every share and every total is in place
#pragma unroll
      for (int r = 0; r < kMaxCluster - 1; ++r) {
        const int t = s_share[pass][r];
        if (owner == r && r < ctas - 1 && above + t < left) above += t, ++owner;
      }
    }
    // thread t: bins 4t' + 3 .. 4t' of the owner's share, t' counted from the top
    if (tid < size / 4) {
      const int top = size / 4 - 1 - tid;
      int4 x;
      if constexpr (kCluster)
        x = ld_cluster4(ptx::mapa(ptx::smem_u32(&share[4 * top]), (uint32_t)owner));
      else
        x = *reinterpret_cast<const int4*>(&hist[pass][4 * top]);
      const int c[4] = {x.w, x.z, x.y, x.x};
      int incl = c[0] + c[1] + c[2] + c[3];
      const int own = incl;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      if (lane == 31) s_warp[warp] = incl;  // (its last readers are behind a barrier)
      asm volatile("bar.sync 1, %0;" ::"r"(size / 4) : "memory");
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
    prefix = (prefix << (pass == 2 ? 10 : 11)) | (uint32_t)s_digit;
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
        for (int j = c0 + tid; j < c1; j += kSelThreads) count(weight_order(weight_at(j)));
      }
    }
  }
  const uint32_t cut = prefix;
  const int ties = left;  // weights equal to the cut that stay
  // Every warp takes a run of the stretch, a lane four numbers of every 128.
  const int per = ((c1 - c0 + kSelWarps - 1) / kSelWarps + 127) & ~127;
  const int j0 = min(c1, c0 + warp * per), j1 = min(c1, j0 + per);
  auto four = [&](int j, uint32_t (&u)[4]) {
    if (hold && j + 4 <= j1) {
      const uint4 x = *reinterpret_cast<const uint4*>(&held_u[j - c0]);
      u[0] = x.x, u[1] = x.y, u[2] = x.z, u[3] = x.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = j + i < j1 ? number(j + i) : 0u;
    }
  };
  int gt = 0, eq = 0;
  for (int jb = j0; jb < j1; jb += 128) {
    uint32_t u[4];
    four(jb + 4 * lane, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      gt += u[i] > cut;  // (past the run u = 0: above no cut)
      eq += u[i] == cut && jb + 4 * lane + i < j1;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) s_gt[warp] = gt, s_eq[warp] = eq;
  __syncthreads();
  int gt0 = __reduce_add_sync(0xffffffffu, lane < warp ? s_gt[lane] : 0);  // before this warp's run
  int eq0 = __reduce_add_sync(0xffffffffu, lane < warp ? s_eq[lane] : 0);
  if constexpr (kCluster) {
    if (warp == kSelWarps - 1 && lane == 0) s_total[0] = gt0 + gt, s_total[1] = eq0 + eq;
    barrier();
    const int x = lane < rank ? ld_cluster(ptx::mapa(ptx::smem_u32(&s_total[0]), (uint32_t)lane)) : 0;
    const int y = lane < rank ? ld_cluster(ptx::mapa(ptx::smem_u32(&s_total[1]), (uint32_t)lane)) : 0;
    gt0 += __reduce_add_sync(0xffffffffu, x);
    eq0 += __reduce_add_sync(0xffffffffu, y);
  }
  // Where all of the run's equal weights stay, or none, what stays is u >= cut or
  // u > cut; only the run in which the ties run out counts them one by one.
  const bool mixed = eq0 < ties && eq0 + eq > ties;
  if (hold && !mixed) {
    // The positions that stay, in place at the start of the run (a number is read
    // before anything at or above its place is written), then out to where they
    // go in one coalesced sweep.
    const uint32_t least = eq0 < ties ? cut : cut + 1u;  // (cut + 1: cut is below the largest number)
    uint32_t* list = held_u + (j0 - c0);
    int count = 0;
    for (int jb = j0; jb < j1; jb += 128) {
      const int j = jb + 4 * lane;
      uint32_t u[4];
      four(j, u);
      int at = count;
      bool stays[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        stays[i] = u[i] >= least && j + i < j1;
        const unsigned m = __ballot_sync(0xffffffffu, stays[i]);
        at += __popc(m & ((1u << lane) - 1u));
        count += __popc(m);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (stays[i]) list[at++] = (uint32_t)(j + i);
      __syncwarp();
    }
    const int base = e.sinks + gt0 + min(eq0, ties);
    for (int i = lane; i < count; i += 32) {
      const int j = (int)list[i];
      keep(base + i, j, weight_at(j));
    }
  } else {
    for (int j = j0 + lane; j - lane < j1; j += 32) {
      const uint32_t u = j < j1 ? number(j) : 0u;
      const unsigned g = __ballot_sync(0xffffffffu, j < j1 && u > cut);
      const unsigned q = __ballot_sync(0xffffffffu, j < j1 && u == cut);
      const unsigned before = (1u << lane) - 1u;
      const int eq_before = eq0 + __popc(q & before);
      if (((g >> lane) & 1u) || (((q >> lane) & 1u) && eq_before < ties))
        keep(e.sinks + gt0 + __popc(g & before) + min(eq_before, ties), j, weight_at(j));
      gt0 += __popc(g);
      eq0 += __popc(q);
    }
  }
  finish();  // (its barrier: no CTA leaves while another may read its shared memory)
}

template <bool kCluster, int kRowBytes>
cudaError_t launch_select(const EvictArgs& e, cudaLaunchConfig_t& cfg, int ctas, int held) {
  auto* const kernel = cache_evict_select_kernel<kCluster, kRowBytes>;
  static std::atomic<uint64_t> smem_set{0};
  if (cudaError_t rc = set_max_dynamic_smem((const void*)kernel, kMaxHeld * 4, smem_set); rc != cudaSuccess) return rc;
  return cudaLaunchKernelEx(&cfg, kernel, e, ctas, held);
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& e, cudaStream_t stream) {
  // CTAs per entry: one where the columns or the table hold fewer than 10,240
  // keys, since a cluster's launch and barriers cost 4 to 5 us whatever its entry
  // holds (16 entries of 2500 keys: 12.7 us with one, 16.8 with clusters; of 9000
  // 15.3 and 19.5; of 20,000 20.5 and 19.8), else as many as the SMs hold at two
  // each. The batch is not in the rule: many entries gain from clusters a little
  // earlier (64 of 9000: 68.2 us with one, 65.8 with clusters).
  const int64_t longest = e.cols < (int64_t)e.max_pages_per_seq * kTileKeys ? e.cols
                                                                            : (int64_t)e.max_pages_per_seq * kTileKeys;
  int ctas = 1;
  constexpr int64_t kClusterKeys = 10240;
  while (longest >= kClusterKeys && ctas < kMaxCluster && (int64_t)e.batch * ctas <= kNumSMs) ctas *= 2;
  const int64_t stretch = (longest + ctas - 1) / ctas;
  const int held = stretch <= kMaxHeld ? (int)stretch : 0;
  // (64 entries, 256 CTAs: 64.5 us against 71.3 in two kernels; 16 entries, 128
  // CTAs: 61.4 against 55.1)
  const bool own_rows = (int64_t)e.batch * ctas * 2 >= 3 * kNumSMs;
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
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  constexpr int kFp8 = MLA_D_QK, k16 = 2 * MLA_D_QK;
  const bool fp8 = e.row_bytes == kFp8;
  cudaError_t rc;
  if (own_rows) {
    if (ctas > 1)
      rc = fp8 ? launch_select<true, kFp8>(e, cfg, ctas, held) : launch_select<true, k16>(e, cfg, ctas, held);
    else
      rc = fp8 ? launch_select<false, kFp8>(e, cfg, ctas, held) : launch_select<false, k16>(e, cfg, ctas, held);
    return rc;
  }
  rc = ctas > 1 ? launch_select<true, 0>(e, cfg, ctas, held) : launch_select<false, 0>(e, cfg, ctas, held);
  if (rc != cudaSuccess) return rc;
  const int64_t pages = (int64_t)e.batch * ((e.budget + kTileKeys - 1) / kTileKeys);
  const int64_t blocks = (pages * kTileKeys * (e.row_bytes / 16) + 8 * 32 * kMoveChunks - 1) / (8 * 32 * kMoveChunks);
  cfg.gridDim = dim3((unsigned)(blocks < kNumSMs * 8 ? blocks : kNumSMs * 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return fp8 ? cudaLaunchKernelEx(&cfg, cache_evict_move_kernel<kFp8>, e)
             : cudaLaunchKernelEx(&cfg, cache_evict_move_kernel<k16>, e);
}

}  // namespace mla
