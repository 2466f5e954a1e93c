// Accumulated attention weights on CUDA cores: the simple cross-check kernel
// of mla_key_weights.
//
// Key j of entry b receives sum over the entry's query rows r that see it of
// p_rj = exp(scale q_r . k_j - lse_r), the attention's own probabilities
// rebuilt from its log-sum-exp, so one pass over K is enough and no maximum is
// kept. One CTA per (entry, 64-key page), one warp per key at a time: lanes
// split the 576 dims, the key's row stays in registers and the entry's query
// rows are read one after the other. The sum runs over rows in order, in 64
// bits: a prefill step has up to 131,072 rows (1024 tokens x 128 heads), over
// which an fp32 sum of nearly equal terms drifts (1.2e-4 of the sum on uniform
// attention over 4024 keys), and this form is what the tensor-core one, whose
// partial sums are short, is held against.
#include "device_common.cuh"

namespace mla {
namespace {

template <int DT>
__global__ void __launch_bounds__(256) key_weights_simt_kernel(const KeyWeightArgs k, int tiles) {
  const DecodeArgs& a = k.a;
  const mla_plan& p = a.plan;
  const int b = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const bool flag = tile == 0 && threadIdx.x == 0;
  const int n = effective_seq_len(a, b, flag);
  const EntryQ e = entry_q(a, b, flag);
  const int key0 = tile * kTileKeys;
  const int key1 = (int)min((int64_t)min(n, key0 + kTileKeys), k.cols);
  if (key0 >= key1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sinks = plan_has_sinks(p) ? p.sinks : 0;
  // rows that see some key of this page: the page's table entry is looked at
  // only if there are any
  const int first_last = n - e.qlen;  // newest key of the entry's first token
  const bool seen = e.qlen > 0 && key0 < n && (key1 > row_key_lo(p, first_last) || key0 < sinks);
  int page = 0;
  bool ok = false;
  if (seen && in_bounds(a, b, p.batch) && in_bounds(a, tile, a.max_pages_per_seq)) {
    page = a.block_tables[(int64_t)b * a.max_pages_per_seq + tile];
    ok = page >= 0 && (int64_t)page < a.num_pages;
    if (!ok && threadIdx.x == 0) atomicOr(a.status, MLA_DEV_BAD_PAGE);
  }
  for (int j = key0 + warp; j < key1; j += 8) {
    double sum = 0.;
    if (ok) {
      const int64_t base = ((int64_t)page * kTileKeys + (j - key0)) * MLA_D_QK;
      float kv[MLA_D_QK / 32];
#pragma unroll
      for (int i = 0; i < MLA_D_QK / 32; ++i) kv[i] = load_elem<DT>(a.kv_cache, base + lane + 32 * i);
      for (int t = 0; t < e.qlen; ++t) {
        const int last = first_last + t;
        if (j > last || (j < row_key_lo(p, last) && j >= sinks)) continue;
        for (int h = 0; h < p.num_heads; ++h) {
          const int64_t row = (e.q0 + t) * p.num_heads + h;
          if (!in_bounds(a, row, out_rows(a))) continue;
          const float lse = k.lse[row];
          if (lse == -INFINITY) continue;
          float dot = 0.f;
#pragma unroll
          for (int i = 0; i < MLA_D_QK / 32; ++i)
            dot = fmaf(load_elem<DT>(a.q, row * MLA_D_QK + lane + 32 * i), kv[i], dot);
          sum += exp2f(fmaf(warp_sum(dot), a.score_scale_log2, (float)((double)lse * -1.4426950408889634)));
        }
      }
    }
    if (lane == 0 && in_bounds(a, b, p.batch) && in_bounds(a, j, k.cols)) {
      const float old = k.w_in ? k.decay * k.w_in[(int64_t)b * k.in_stride + j] : 0.f;
      k.w_out[(int64_t)b * k.out_stride + j] = old + (float)sum;
    }
  }
}

}  // namespace

cudaError_t launch_key_weights_simt(const KeyWeightArgs& k, cudaStream_t stream) {
  const mla_plan& p = k.a.plan;
  // as far as effective_seq_len lets a length go: the plan's splits may reach past its longest sequence
  const int64_t keys = min((int64_t)k.a.max_pages_per_seq * kTileKeys, (int64_t)p.split_kv * p.keys_per_split);
  const int tiles = (int)((keys + kTileKeys - 1) / kTileKeys);
  const int64_t grid = (int64_t)p.batch * tiles;
  if (grid == 0) return cudaSuccess;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  switch (p.dtype) {
    case MLA_BF16: key_weights_simt_kernel<MLA_BF16><<<(unsigned)grid, 256, 0, stream>>>(k, tiles); break;
    case MLA_FP16: key_weights_simt_kernel<MLA_FP16><<<(unsigned)grid, 256, 0, stream>>>(k, tiles); break;
    default: key_weights_simt_kernel<MLA_FP8_E4M3><<<(unsigned)grid, 256, 0, stream>>>(k, tiles); break;
  }
  return cudaGetLastError();
}

}  // namespace mla
