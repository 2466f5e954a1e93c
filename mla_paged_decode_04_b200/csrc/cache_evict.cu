// Eviction from the paged cache by accumulated attention weight: per entry,
// which keys stay (cache_evict_select_kernel), then their rows onto the pages
// of another table (cache_evict_move_kernel).
//
// Selection. Between the protected first `sinks` and last `recent` keys the
// k = budget - sinks - recent largest weights stay. A weight maps to a 32-bit
// number that orders like it (sign folded, -0 as +0, NaN below everything), and
// four passes over 8 bits each, from the top, find the k-th largest exactly:
// a histogram of the digit among the weights that agree with the digits found
// so far, then the digit at which the count from above reaches k. All weights
// above it stay, and of those equal to it the ones at the lowest positions.
// Positions are then compacted in order: every warp counts its own run, a scan
// over the warps gives where it starts, and a second walk writes. One CTA per
// entry.
//
// Moving. One thread per 16 bytes of a row that stays.
#include "device_common.cuh"

namespace mla {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

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

__global__ void __launch_bounds__(kSelThreads) cache_evict_select_kernel(const EvictArgs e) {
  __shared__ int hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = evict_len(e, b, tid == 0);
  const float* w = e.weights + (int64_t)b * e.weights_stride;
  int32_t* kept = e.kept + (int64_t)b * e.budget;
  float* ow = e.out_weights ? e.out_weights + (int64_t)b * e.out_weights_stride : nullptr;
  auto keep = [&](int i, int j) {
    kept[i] = j;
    if (ow) ow[i] = w[j];
  };
  __syncthreads();  // every thread has read the length (out_seq_lens may be seq_lens)
  if (tid == 0) e.out_seq_lens[b] = min(n, e.budget);
  if (n <= e.budget) {
    for (int i = tid; i < e.budget; i += kSelThreads) {
      if (i < n)
        keep(i, i);
      else
        kept[i] = -1;
    }
    return;
  }
  const int lo = e.sinks, hi = n - e.recent, k = e.budget - e.sinks - e.recent;
  for (int i = tid; i < e.sinks; i += kSelThreads) keep(i, i);
  for (int i = tid; i < e.recent; i += kSelThreads) keep(e.budget - e.recent + i, hi + i);
  if (k == 0) return;
  if (tid == 0) s_prefix = 0u, s_left = k;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      const uint32_t u = weight_order(w[j]);
      if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l: digits 255 - 8l down to 248 - 8l
      int c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c[i] = hist[255 - 8 * lane - i];
      int incl = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      const int left = s_left;
      int above = incl - sum;
      __syncwarp();
      if (above < left && left <= incl) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < left && left <= above + c[i]) {
            s_prefix = prefix | ((uint32_t)(255 - 8 * lane - i) << shift);
            s_left = left - above;
          }
          above += c[i];
        }
      }
    }
    __syncthreads();
  }
  const uint32_t cut = s_prefix;
  const int ties = s_left;  // weights equal to the cut that stay
  const int per = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int j0 = min(hi, lo + warp * per), j1 = min(hi, j0 + per);
  int gt = 0, eq = 0;
  for (int j = j0 + lane; j < j1; j += 32) {
    const uint32_t u = weight_order(w[j]);
    gt += u > cut;
    eq += u == cut;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  if (lane == 0) s_gt[warp] = gt, s_eq[warp] = eq;
  __syncthreads();
  int gt0 = 0, eq0 = 0;  // before this warp's run
  for (int i = 0; i < warp; ++i) gt0 += s_gt[i], eq0 += s_eq[i];
  for (int jb = j0; jb < j1; jb += 32) {
    const int j = jb + lane;
    const uint32_t u = j < j1 ? weight_order(w[j]) : 0u;
    const unsigned g = __ballot_sync(0xffffffffu, j < j1 && u > cut);
    const unsigned q = __ballot_sync(0xffffffffu, j < j1 && u == cut);
    const unsigned before = (1u << lane) - 1u;
    const int eq_before = eq0 + __popc(q & before);
    if (((g >> lane) & 1u) || (((q >> lane) & 1u) && eq_before < ties))
      keep(e.sinks + gt0 + __popc(g & before) + min(eq_before, ties), j);
    gt0 += __popc(g);
    eq0 += __popc(q);
  }
}

__global__ void __launch_bounds__(256) cache_evict_move_kernel(const EvictArgs e) {
  const int per_row = e.row_bytes / 16;
  const int rows = ((e.budget + kTileKeys - 1) / kTileKeys) * kTileKeys;  // of an entry, with the last page's rest
  const int64_t total = (int64_t)e.batch * rows * per_row;
  for (int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; idx < total;
       idx += (int64_t)gridDim.x * blockDim.x) {
    const int64_t rr = idx / per_row;
    const int c = (int)(idx - rr * per_row);
    const int b = (int)(rr / rows), i = (int)(rr - (int64_t)b * rows);
    const int len = e.out_seq_lens[b];
    if (i >= ((len + kTileKeys - 1) & ~(kTileKeys - 1))) continue;
    const int to = e.out_block_tables[(int64_t)b * e.out_max_pages_per_seq + i / kTileKeys];
    if (to < 0 || (int64_t)to >= e.out_num_pages) {
      if (e.status) atomicOr(e.status, MLA_DEV_BAD_PAGE);
      continue;
    }
    uint4 v = make_uint4(0, 0, 0, 0);
    if (i < len) {
      const int j = e.kept[(int64_t)b * e.budget + i];
      const int from = e.block_tables[(int64_t)b * e.max_pages_per_seq + j / kTileKeys];
      if (from < 0 || (int64_t)from >= e.num_pages) {
        if (e.status) atomicOr(e.status, MLA_DEV_BAD_PAGE);
      } else {
        v = *reinterpret_cast<const uint4*>(e.kv_cache + ((int64_t)from * kTileKeys + j % kTileKeys) * e.row_bytes +
                                            16 * c);
      }
    }
    *reinterpret_cast<uint4*>(e.out_cache + ((int64_t)to * kTileKeys + i % kTileKeys) * e.row_bytes + 16 * c) = v;
  }
}

}  // namespace

cudaError_t launch_cache_evict(const EvictArgs& e, cudaStream_t stream) {
  cache_evict_select_kernel<<<(unsigned)e.batch, kSelThreads, 0, stream>>>(e);
  if (cudaError_t rc = cudaGetLastError(); rc != cudaSuccess) return rc;
  const int64_t rows = ((int64_t)(e.budget + kTileKeys - 1) / kTileKeys) * kTileKeys;
  const int64_t blocks = ((int64_t)e.batch * rows * (e.row_bytes / 16) + 255) / 256;
  cache_evict_move_kernel<<<(unsigned)(blocks < kNumSMs * 8 ? blocks : kNumSMs * 8), 256, 0, stream>>>(e);
  return cudaGetLastError();
}

}  // namespace mla
