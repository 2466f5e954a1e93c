// Accumulated attention weights on the sm_100a tensor cores (mla_key_weights).
//
// Key j of entry b receives sum_r p_rj over the entry's query rows r that see
// it, p_rj = exp(scale q_r . k_j - lse_r): the attention's probabilities
// rebuilt from its log-sum-exp, so that one pass over K is enough and there
// is no running maximum. K is read once (576 dims a key), 2 * 576 operations
// per (row, key): a decode step (up to 128 rows an entry) is bound by HBM, a
// step of many query tokens by the tensor cores.
//
// S is computed transposed, S^T = K Q^T: keys are the M dimension, so a key is
// a TMEM lane and its sum over rows runs along the lane's columns inside one
// thread, in a fixed order and without any exchange. CTA pairs
// (tcgen05.mma.cta_group::2, M = 256, N <= 256): CTA c holds 128 keys (two
// pages) of a 256-key tile and half of the N query rows, and receives its 128
// keys' scores for all N rows.
//
// Both operands are cut into 128-byte column chunks (nine for 16-bit, five
// for FP8, the last one 64 bytes wide) that go through a ring of slots; what
// bounds the ring is the time from a slot's release to its next use (about
// 3000 cycles: the MMAs' commit, the loader, TMA and L2, the peer's half), so
// it has to hold that much MMA time. Three forms:
//   * kRowsStay: an entry's rows fit one group of N <= 256 (16-bit: 128) and
//     stay in shared memory, the key tiles stream. A pair takes a contiguous run
//     of the entries' tiles, so Q is loaded once per entry that it meets.
//   * kKeysStay (FP8, more rows): a key tile stays, the row groups stream. K
//     comes from HBM once; a 16 KB chunk from L2 feeds 256 x 256 x 128 products.
//   * kBothStream (16-bit, more than 128 rows): either resident part would take
//     147 KB and leave a ring of 64 KB, 2048 cycles of MMAs. Without one the ring
//     holds six slots of both operands' chunks, half as much again; K is read per
//     group, from L2 (the FP16 case below: 158 us with keys resident, 143 without).
// With several row groups the sum goes on in registers from group to group,
// and pairs take tiles a grid apart, whose numbers of groups (causal mask,
// window) are alike. A resident operand is replaced slot by slot behind the
// last MMAs that read it.
//
// Roles (384 threads per CTA): warp 0 loads, warp 1 of the leader issues the
// MMAs, warps 2 and 3 write the keys that no row sees (their old weight,
// decayed), warps 4-11 sum: ex2 of the score minus the row's log-sum-exp (one
// FMA), over the rows. Up to 128 rows the two groups of four warps take alternate
// score buffers; above, a buffer's 256 columns take a group as long as its MMAs
// and more, so the two share every buffer (alternate 32 columns) and hand it back
// in half the time (16..32 last tokens x 64 heads over 4 x up to 32,768 FP16
// keys: 127 -> 118 us; 16 x 4 tokens x 64 heads over 81,920 FP8 keys: 207 -> 194 us).
//
// Measured: 16 x 4 tokens x 32 heads over 81,920 FP8 keys 123 to 135 us in
// replayed graphs (5.7 to 6.2 TB/s, 0.87 to 0.95 of the copy bandwidth; 149 us
// where the power limit holds the clock down), 4 x 4 x 32 over 8192 BF16 keys 16 us
// (two tiles a pair, 5.9 us of HBM time). kKeysStay: 16 x 8 tokens x 64 heads over
// 40,960 FP8 keys 204 us (117 of FP8 products at twice the BF16 rate; no unit is
// full: tensor pipe 38 %, ex2 36 %, issue 27 % of the active cycles of a quarter of
// it, so the hand-over between products and sums is what is left), 16..32 tokens x
// 64 heads over 4 x up to 32,768 95 us (45 of products).
// Every wait is bounded as in the attention kernels; a plan with fault_test = 1
// makes them run out (tests). No TMA load uses multicast.
#include <cuda.h>

#include <type_traits>

#include "device_common.cuh"
#include "pair_schedule.cuh"
#include "sm100_ptx.cuh"
#include "tc_common.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kTile = 256;       // keys per pair tile
constexpr int kHalf = 128;       // keys of a tile per CTA
constexpr int kThreads = 384;
enum Form { kRowsStay = 0, kKeysStay = 1, kBothStream = 2 };
constexpr int kMaxEntries = 1024;  // entries of one launch: their tiles and lengths are kept in shared memory
constexpr int kMaxStages = 8;
constexpr int kMaxSlots = 9;     // ring slots a tile is cut into
constexpr uint32_t kChunkBytes = 128 * 128;
// 16-bit scores of few rows (N <= 64) go to four accumulators, of 192, 128, 128
// and 128 dims, added in fp32 afterwards. The tensor cores cut partial sums
// toward zero, at a unit of the sum's own size, and of so few rows no others
// average that out. Worst error of a key's weight, one FP16 head over 4096 random
// keys: 3.5e-6 with one accumulator, 9.6e-7 with four; positive q and k, where
// cuts do not cancel, at scores of 30: 1.1e-4 and 2.1e-5. More rows have one
// accumulator (two score buffers of 256 columns are all of the tensor memory):
// 7e-7 in the norm on 16..32 tokens x 64 heads. FP8 loses nothing measurable.
constexpr int kParts = 4;
constexpr int kPartCols = 64;

// shared memory, from a 1024-aligned base
constexpr uint32_t kStartOff = 0;                                   // int [kMaxEntries + 1]: first tile of an entry
constexpr uint32_t kLenOff = kStartOff + 4 * (kMaxEntries + 32);   // int [kMaxEntries]: keys of an entry
constexpr uint32_t kLseOff = kLenOff + 4 * kMaxEntries;                     // float [group][2][256]: -lse * log2(e)
constexpr uint32_t kLastOff = kLseOff + 4096;                       // int [group][2][256]: newest key of the row
constexpr uint32_t kSumOff = kLastOff + 4096;                       // float [128]: group 1's sums
constexpr uint32_t kScanOff = kSumOff + 512;                        // int [12]
constexpr uint32_t kMiscOff = kScanOff + 64;                        // TMEM address, abort flag, loads issued
constexpr uint32_t kBarOff = kMiscOff + 64;
constexpr int B_FULL = 0;                          // leader, + stage: both CTAs' chunk landed
constexpr int B_EMPTY = B_FULL + kMaxStages;       // both, + stage
constexpr int B_RES_FULL = B_EMPTY + kMaxStages;   // leader, + slot
constexpr int B_RES_EMPTY = B_RES_FULL + kMaxSlots;  // both, + slot
constexpr int B_S_FULL = B_RES_EMPTY + kMaxSlots;  // both, + buffer
constexpr int B_S_EMPTY = B_S_FULL + 2;            // leader, + buffer
constexpr int B_LSE = B_S_EMPTY + 2;               // local, + group: the rows' constants are staged
constexpr int B_SUM = B_LSE + 2;                   // local: group 1's sums are in shared memory
constexpr int B_SUM_READ = B_SUM + 1;              // local: group 0 has read them
constexpr int kNumBars = B_SUM_READ + 1;
constexpr uint32_t kDataOff = 18432;
static_assert(kBarOff + 8 * kNumBars <= kDataOff && kDataOff % 1024 == 0, "layout");
constexpr uint32_t kSmemMax = 232448 - 1024;  // less the slack for the base's alignment

struct KeyWeightParams {
  CUtensorMap tm_q, tm_q_rope, tm_k, tm_k_rope;  // the rope maps: FP8's last 64 dims
  KeyWeightArgs k;
  int b0, nb;        // this launch's entries
  int n_cols;        // N: rows per group (a multiple of 32)
  int parts;         // accumulators the dims are spread over (1 or kParts)
  int stages;
  uint32_t idesc;
};

// One batch entry: keys, new tokens and their place in q, the rows' union of
// visible keys.
struct Entry {
  int b, n, qlen, rows, klo;
  int64_t q0;
};
__device__ __forceinline__ Entry make_entry(const KeyWeightParams& prm, int i, int n, bool flag) {
  const DecodeArgs& a = prm.k.a;
  Entry e;
  e.b = prm.b0 + i;
  e.n = n;
  const EntryQ q = entry_q(a, e.b, flag);
  e.q0 = q.q0;
  e.qlen = q.qlen;
  e.rows = q.qlen * a.plan.num_heads;
  e.klo = a.plan.window > 0 ? max(0, e.n - e.qlen + 1 - a.plan.window) : 0;
  return e;
}
// Tiles that hold a key some row sees: those of the sinks, then those from
// the window's first tile on; one run from tile 0 when the two meet.
__device__ __forceinline__ int entry_tiles(const mla_plan& p, const Entry& e) {
  if (e.n == 0 || e.qlen == 0 || e.klo >= e.n) return 0;
  const int first = e.klo / kTile, nst = (min(plan_has_sinks(p) ? p.sinks : 0, e.klo) + kTile - 1) / kTile;
  return (e.n + kTile - 1) / kTile - first + min(nst, first);
}
// Place in the sequence of an entry's i-th such tile.
__device__ __forceinline__ int entry_tile(const mla_plan& p, const Entry& e, int i) {
  const int first = e.klo / kTile, nst = (min(plan_has_sinks(p) ? p.sinks : 0, e.klo) + kTile - 1) / kTile;
  return (nst >= first || i < nst) ? i : i + first - nst;
}
__device__ __forceinline__ int sinks_of(const mla_plan& p) { return plan_has_sinks(p) ? p.sinks : 0; }

// The tiles of this pair, in the order every role walks them.
struct Walk {
  const int *start, *len;  // [nb + 1], [nb]
  int idx, end, step, i;
  Entry e;
  __device__ __forceinline__ Walk(const KeyWeightParams& prm, const uint8_t* smem, bool groups) {
    start = reinterpret_cast<const int*>(smem + kStartOff);
    len = reinterpret_cast<const int*>(smem + kLenOff);
    const int64_t total = start[prm.nb];
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    idx = groups ? pair : (int)(total * pair / pairs);
    end = groups ? (int)total : (int)(total * (pair + 1) / pairs);
    step = groups ? pairs : 1;
    i = -1;
  }
  __device__ __forceinline__ bool more() const { return idx < end; }
  // moves to the entry of idx; true if it is another one than before
  __device__ __forceinline__ bool seek(const KeyWeightParams& prm) {
    if (i >= 0 && idx < start[i + 1]) return false;
    do ++i;
    while (idx >= start[i + 1]);
    e = make_entry(prm, i, len[i], false);
    return true;
  }
  __device__ __forceinline__ int tile(const mla_plan& p) const { return entry_tile(p, e, idx - start[i]); }
  // whether this is the last tile of its entry in this pair's run
  __device__ __forceinline__ bool last_of_entry() const { return idx + 1 >= end || idx + 1 >= start[i + 1]; }
};

// Row groups of the entry that see a key of the tile at key0.
__device__ __forceinline__ void tile_groups(const KeyWeightParams& prm, const Entry& e, int key0, int& g0, int& g1) {
  const mla_plan& p = prm.k.a.plan;
  const int H = p.num_heads, N = prm.n_cols, nq = e.n - e.qlen;
  const int t0 = min(max(key0 - nq, 0), e.qlen - 1);  // first token that sees key0
  int64_t t1 = e.qlen;                                // past the last token whose window reaches the tile
  if (p.window > 0 && key0 >= sinks_of(p)) t1 = min(t1, (int64_t)key0 + kTile + p.window - 1 - nq);
  g0 = t0 * H / N;
  g1 = ((int)t1 * H + N - 1) / N;
}

// A tile's column chunks of 128 bytes, kPer of them to a ring slot (one wait,
// one commit). Larger slots cost the single issuing threads less per byte,
// smaller ones keep a short ring finer.
template <int E, int kPer, int kForm>
struct Cut {
  static constexpr int kChunks = E == 2 ? 9 : 5;
  static constexpr int kSlots = (kChunks + kPer - 1) / kPer;
  static constexpr int kDims = 128 / E;  // dims of a full chunk
  static constexpr uint32_t kRowsAt = kForm == kBothStream ? kPer * kChunkBytes : 0;  // Q's chunks in a ring slot
  static constexpr uint32_t kSlotBytes = kRowsAt + kPer * kChunkBytes;
  static __host__ __device__ constexpr bool rope(int c) { return E == 1 && c == 4; }  // 64 bytes wide
  static __host__ __device__ constexpr int first(int s) { return s * kPer; }
  static __host__ __device__ constexpr int last(int s) { return (s + 1) * kPer < kChunks ? (s + 1) * kPer : kChunks; }
  // bytes per row of slot s
  static __host__ __device__ constexpr uint32_t row_bytes(int s) {
    return (uint32_t)(last(s) - first(s)) * 128u - (rope(last(s) - 1) ? 64u : 0u);
  }
};

template <class C>
__device__ __forceinline__ void load_keys(const KeyWeightParams& prm, uint32_t dst, int c, int pg0, int pg1,
                                          uint32_t full, uint64_t pol) {
  const CUtensorMap* tm = C::rope(c) ? &prm.tm_k_rope : &prm.tm_k;
  tma_load_2d_pair(dst, tm, C::kDims * c, pg0 * kTileKeys, full, pol);
  tma_load_2d_pair(dst + (C::rope(c) ? 4096 : 8192), tm, C::kDims * c, pg1 * kTileKeys, full, pol);
}
template <class C>
__device__ __forceinline__ void load_rows(const KeyWeightParams& prm, uint32_t dst, int c, int row, uint32_t full,
                                          uint64_t pol) {
  tma_load_2d_pair(dst, C::rope(c) ? &prm.tm_q_rope : &prm.tm_q, C::kDims * c, row, full, pol);
}

// The table entry of the 64 keys at `key` where some row sees them, else page
// 0. Read a tile ahead of its use.
__device__ __forceinline__ int key_entry(const DecodeArgs& a, const Entry& e, int key) {
  if (!page_seen(key, e.klo, e.n, sinks_of(a.plan))) return 0;
  if (!in_bounds(a, e.b, a.plan.batch) || !in_bounds(a, key / kTileKeys, a.max_pages_per_seq)) return 0;
  return ld_nc_ordered(a.block_tables + (int64_t)e.b * a.max_pages_per_seq + key / kTileKeys);
}
// Whether key `key` of entry b has a place among the weights (the checking
// build; both arrays have [batch] rows of `cols`).
__device__ __forceinline__ bool weight_in_bounds(const KeyWeightArgs& k, int b, int64_t key) {
  return in_bounds(k.a, b, k.a.plan.batch) && in_bounds(k.a, key, k.cols);
}
__device__ __forceinline__ bool page_valid(const DecodeArgs& a, int pg) { return pg >= 0 && (int64_t)pg < a.num_pages; }
// an entry outside the cache reads page 0 (the sums leave its keys out)
__device__ __forceinline__ int page_or_0(const DecodeArgs& a, int pg) { return page_valid(a, pg) ? pg : 0; }

template <int E, int kForm, int kPer>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    tc_key_weights_kernel(const __grid_constant__ KeyWeightParams prm) {
  using C = Cut<E, kPer, kForm>;
  constexpr bool kGroups = kForm != kRowsStay;    // an entry may have several row groups
  constexpr bool kStays = kForm != kBothStream;   // one operand is resident
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const DecodeArgs& a = prm.k.a;
  const mla_plan& p = a.plan;
  auto bar = [&](int i) -> uint32_t { return sb + kBarOff + 8u * (uint32_t)i; };
  auto lead = [&](int i) -> uint32_t { return mapa(bar(i), 0); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kMiscOff + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMiscOff);
  int* issued = reinterpret_cast<int*>(smem + kMiscOff + 8);  // [ring slots, resident rounds]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0 = leader
  const int N = prm.n_cols, NB = N / 2, NS = prm.stages;
  // whether the two sum groups share every tile (alternate columns)
  const bool halves = kGroups || N > 128;
  // rows of a chunk, both operands' CTA halves: what stays, what a slot takes
  const int res_rows = kForm == kKeysStay ? kHalf : NB;
  const int ring_rows = kForm == kRowsStay ? kHalf : kForm == kKeysStay ? NB : kHalf + NB;
  const uint32_t res0 = sb + kDataOff;
  const uint32_t res_slot = kStays ? (uint32_t)res_rows * 128u : 0u;  // bytes of a resident chunk's place
  const uint32_t ring0 = (res0 + C::kChunks * res_slot + 1023u) & ~1023u;

  if (threadIdx.x < kNumBars) {
    const int i = threadIdx.x;
    // S_EMPTY: the sum warps of a tile in both CTAs; from LSE on a group's warps
    mbar_init(bar(i), (i >= B_S_EMPTY && i < B_S_EMPTY + 2) ? (halves ? 16u : 8u) : i >= B_LSE ? 4u : 1u);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) *abort_flag = issued[0] = issued[1] = 0;
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&prm.tm_q);
    prefetch_tmap(&prm.tm_k);
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  // a programmatic dependent of the kernel before it in the stream: nothing
  // above touches global memory
  grid_dep_wait();

  // first tile of every entry: thread runs, a scan over the block
  {
    int* start = reinterpret_cast<int*>(smem + kStartOff);
    int* len = reinterpret_cast<int*>(smem + kLenOff);
    int* scan = reinterpret_cast<int*>(smem + kScanOff);
    const int per = (prm.nb + kThreads - 1) / kThreads;
    const int i0 = min(prm.nb, (int)threadIdx.x * per), i1 = min(prm.nb, i0 + per);
    int run = 0;
    for (int i = i0; i < i1; ++i) {
      const int n = effective_seq_len(a, prm.b0 + i, blockIdx.x == 0);
      start[i] = run;
      len[i] = n;
      run += entry_tiles(p, make_entry(prm, i, n, blockIdx.x == 0));
    }
    const int incl = warp_incl_scan(run);
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int base = incl - run, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      const int x = scan[w];
      if (w < warp) base += x;
      total += x;
    }
    for (int i = i0; i < i1; ++i) start[i] += base;
    if (threadIdx.x == 0) start[prm.nb] = total;
    __syncthreads();
  }
  const uint32_t tmem = *tmem_slot;
  const bool spread = E == 2 && kForm == kRowsStay && prm.parts > 1;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      const uint64_t pol_once = policy_evict_first(), pol_again = policy_evict_last();
      int filled = 0, round = 0, st = 0;
      uint32_t ph = 1;  // parity to wait for: the ring starts empty
      bool ok = true;
      Walk w(prm, smem, kGroups);
      const uint32_t full0 = lead(B_FULL), res_full0 = lead(B_RES_FULL);
      // one inner step: the resident operand's slots too where `fresh`
      auto step = [&](bool fresh, int row, int pg0, int pg1) {
#pragma unroll
        for (int s = 0; s < C::kSlots; ++s) {
          if (kStays && fresh) {
            if (!(ok = bounded_wait_cta(bar(B_RES_EMPTY + s), (round & 1) ^ 1, abort_flag, a.status))) return;
            if (rank == 0) mbar_arrive_expect_tx(bar(B_RES_FULL + s), 2u * (uint32_t)res_rows * C::row_bytes(s));
#pragma unroll
            for (int c = C::first(s); c < C::last(s); ++c) {
              if (kForm == kKeysStay)
                load_keys<C>(prm, res0 + c * res_slot, c, pg0, pg1, res_full0 + 8u * s, pol_once);
              else
                load_rows<C>(prm, res0 + c * res_slot, c, row, res_full0 + 8u * s, pol_again);
            }
          }
          if (!(ok = bounded_wait_cta(bar(B_EMPTY + st), ph, abort_flag, a.status))) return;
          // failure-detection test mode (FP8 plans): the pair's first slot is never
          // loaded, so the MMA issuer's wait for it runs out
          if (!(E == 1 && p.fault_test == 1 && filled == 0)) {
            if (rank == 0) mbar_arrive_expect_tx(bar(B_FULL + st), 2u * (uint32_t)ring_rows * C::row_bytes(s));
            const uint32_t sd = ring0 + st * C::kSlotBytes, full = full0 + 8u * st;
#pragma unroll
            for (int c = C::first(s); c < C::last(s); ++c) {
              const uint32_t cd = sd + (c - C::first(s)) * kChunkBytes;
              if (kForm != kKeysStay)
                load_keys<C>(prm, cd, c, pg0, pg1, full, kForm == kRowsStay ? pol_once : pol_again);
              if (kForm != kRowsStay) load_rows<C>(prm, cd + C::kRowsAt, c, row, full, pol_again);
            }
          }
          ++filled;
          if (++st == NS) st = 0, ph ^= 1;
        }
        if (fresh) ++round;
      };
      bool other = w.more() && w.seek(prm);
      int e0 = 0, e1 = 0;
      auto entries = [&]() {
        const int key0 = kTile * w.tile(p) + kHalf * (int)rank;
        e0 = key_entry(a, w.e, key0);
        e1 = key_entry(a, w.e, key0 + kTileKeys);
      };
      if (w.more()) entries();
      while (ok && w.more()) {
        const int pg0 = page_or_0(a, e0), pg1 = page_or_0(a, e1);
        const int row0 = (int)(w.e.q0 * p.num_heads) + NB * (int)rank;
        const bool fresh = other;
        int g0 = 0, g1 = 1;
        if (kGroups) tile_groups(prm, w.e, kTile * w.tile(p), g0, g1);
        // the next tile's entries are on their way while this one's chunks are issued
        w.idx += w.step;
        if (w.more()) {
          other = w.seek(prm);
          entries();
        }
        if (kGroups) {
          for (int g = g0; ok && g < g1; ++g) step(g == g0, row0 + g * N, pg0, pg1);
        } else {
          step(fresh, row0, pg0, pg1);
        }
      }
      issued[0] = filled;
      issued[1] = round;
      // the leader's barriers count both CTAs' bytes: nothing is in flight
      // when the pair leaves, after an abort either
      if (rank == 0) {
        drain_loads(bar(B_FULL), NS, filled);
        if (kStays && round > 0)
          for (int s = 0; s < C::kSlots; ++s) drain_phase(bar(B_RES_FULL + s), (uint32_t)(round - 1) & 1);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs (leader)
    if (rank == 0) {
      int round = 0, jt = 0, st = 0;
      uint32_t ph = 0;
      bool ok = true;
      Walk w(prm, smem, kGroups);
      // operand descriptors: chunk c is c * res_slot further in the resident
      // part, (c % kPer) * 16 KB in a ring slot (in 16-byte units); the FP8 rope
      // chunk has the 64-byte swizzle and half the row stride
      const uint64_t res_desc = smem_desc(res0, 16, 1024, kSw128), ring_desc = smem_desc(ring0, 16, 1024, kSw128);
      const uint64_t rope_bits = smem_desc(0, 16, 512, kSw64) - smem_desc(0, 16, 1024, kSw128);
      auto step = [&](bool fresh, bool last) {
        const int buf = jt & 1;
        if (!(ok = warp_wait(bar(B_S_EMPTY + buf), ((jt >> 1) & 1) ^ 1, abort_flag, a.status))) return;
        const uint32_t d = tmem + 256u * buf;
#pragma unroll
        for (int s = 0; s < C::kSlots; ++s) {
          if (kStays && fresh && !(ok = warp_wait(bar(B_RES_FULL + s), round & 1, abort_flag, a.status))) return;
          if (!(ok = warp_wait(bar(B_FULL + st), ph, abort_flag, a.status))) return;
          tc_fence_after();
          const uint64_t slot_desc = ring_desc + (uint64_t)(st * (C::kSlotBytes >> 4));
#pragma unroll
          for (int c = C::first(s); c < C::last(s); ++c) {
            const uint64_t more = C::rope(c) ? rope_bits : 0ull;
            const uint64_t dr = res_desc + (uint64_t)(c * (res_slot >> 4)) + more;
            const uint64_t ds = slot_desc + (uint64_t)((c - C::first(s)) * (kChunkBytes >> 4)) + more;
            // (the part of chunk c, and whether it begins there)
            const int part = c * kParts / C::kChunks;
            const bool begins = c == 0 || part != (c - 1) * kParts / C::kChunks;
            const uint32_t dp = d + (spread ? (uint32_t)(kPartCols * part) : 0u);
            const uint32_t first = spread ? !begins : c > 0;
            const uint64_t dk = kForm == kKeysStay ? dr : ds;
            const uint64_t dq = kForm == kRowsStay ? dr : ds + (C::kRowsAt >> 4);
#pragma unroll
            for (int kk = 0; kk < (C::rope(c) ? 2 : 4); ++kk) {  // 32 bytes of the dims per MMA
              if constexpr (E == 2)
                mma_f16_ss_pair_e(dp, dk + (uint64_t)(2 * kk), dq + (uint64_t)(2 * kk), prm.idesc, kk ? 1u : first);
              else
                mma_f8_ss_pair_e(dp, dk + (uint64_t)(2 * kk), dq + (uint64_t)(2 * kk), prm.idesc, kk ? 1u : first);
            }
          }
          mma_commit_pair_mc_e(bar(B_EMPTY + st), 3);
          if (kStays && last) mma_commit_pair_mc_e(bar(B_RES_EMPTY + s), 3);
          if (++st == NS) st = 0, ph ^= 1;
        }
        mma_commit_pair_mc_e(bar(B_S_FULL + buf), 3);
        if (fresh) ++round;
        ++jt;
      };
      for (; ok && w.more(); w.idx += w.step) {
        const bool other = w.seek(prm);
        if (kGroups) {
          int g0, g1;
          tile_groups(prm, w.e, kTile * w.tile(p), g0, g1);
          for (int g = g0; ok && g < g1; ++g) step(g == g0, g == g1 - 1);
        } else {
          step(other, w.last_of_entry());
        }
      }
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ keys that no row sees
    // (between sinks and window, and all keys of an entry without new tokens):
    // the old weight, decayed
    if ((p.window > 0 || p.varlen) && !(prm.k.w_in == prm.k.w_out && prm.k.decay == 1.f)) {
      const int* lens = reinterpret_cast<const int*>(smem + kLenOff);
      const int w_all = 2 * (int)gridDim.x, w_id = 2 * (int)blockIdx.x + (warp - 2);
      const int parts = max(1, w_all / prm.nb);
      for (int i = w_id / parts; i < prm.nb; i += w_all / parts) {
        if (w_id / parts >= w_all / parts) break;
        const Entry e = make_entry(prm, i, lens[i], false);
        const int n = (int)min((int64_t)e.n, prm.k.cols);
        int k0 = 0, k1 = n;
        if (entry_tiles(p, e) > 0) {
          const int nst = (min(sinks_of(p), e.klo) + kTile - 1) / kTile;
          k0 = min(n, nst * kTile);
          k1 = min(n, e.klo / kTile * kTile);
        }
        const float* in = prm.k.w_in ? prm.k.w_in + (int64_t)e.b * prm.k.in_stride : nullptr;
        float* out = prm.k.w_out + (int64_t)e.b * prm.k.out_stride;
        for (int64_t j = k0 + 32 * (w_id % parts) + lane; j < k1; j += 32 * parts)
          if (weight_in_bounds(prm.k, e.b, j)) out[j] = in ? prm.k.decay * in[j] : 0.f;
      }
    }
  } else {
    // ------------------------------------------------------------ sums
    const int grp = (warp - 4) >> 2, q = warp & 3;
    const int tid = threadIdx.x & 127;
    const int kl = 32 * q + lane;  // this thread's key among the CTA's 128 (its TMEM lane)
    const uint32_t tl = (uint32_t)(32 * q) << 16;
    float* lse_st = reinterpret_cast<float*>(smem + kLseOff) + grp * 512;  // [2][256]
    int* last_st = reinterpret_cast<int*>(smem + kLastOff) + grp * 512;
    float* sums = reinterpret_cast<float*>(smem + kSumOff);
    const float sl2 = a.score_scale_log2;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    const int H = p.num_heads, sinks = sinks_of(p);
    const int W = p.window > 0 ? p.window : 1 << 30;
    int jt = 0, staged = 0, outer = 0;
    bool ok = true;
    Walk w(prm, smem, kGroups);

    // This thread's rows of a row group [r0, r0 + nr): two of all 256 columns, or
    // one of the half that its sum group takes (columns 32 cb .. 32 cb + 31 with
    // cb of the group's parity).
    auto own_row = [&](int u) -> int { return halves ? 64 * (tid >> 5) + 32 * grp + lane : tid + 128 * u; };
    struct RowLse {
      float l[2];
    };
    auto load_lse = [&](const Entry& e, int r0, int nr) -> RowLse {
      RowLse x;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = own_row(u);
        const int64_t row = e.q0 * H + r0 + r;
        x.l[u] = (u == 0 || !halves) && r < nr && in_bounds(a, row, out_rows(a)) ? prm.k.lse[row] : -INFINITY;
      }
      return x;
    };
    // their constants into shared memory: -lse * log2(e), and where a batch of 32
    // columns has masked pairs or ends the group the newest key each row sees (-1
    // past the group, and for a row whose lse is -inf)
    auto stage = [&](const Entry& e, int r0, int nr, const RowLse& x, bool masks) {
      const int at = (staged & 1) * 256;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (u == 1 && halves) break;
        const int r = own_row(u);
        const float l = x.l[u];
        // (rounded once: an error here weighs on every key of the row; a row without keys adds 0)
        lse_st[at + r] = l == -INFINITY ? -INFINITY : (float)((double)l * -1.4426950408889634);
        if (masks) last_st[at + r] = r < nr && l != -INFINITY ? e.n - e.qlen + (r0 + r) / H : -1;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_LSE + grp));
      ok = warp_wait_cta(bar(B_LSE + grp), staged & 1, abort_flag, a.status);
      ++staged;
    };
    // whether every row of the group sees every key of this CTA's half tile
    auto open_tile = [&](const Entry& e, int r0, int nr, int key0) -> bool {
      const int last_a = e.n - e.qlen + r0 / H, last_b = e.n - e.qlen + (r0 + nr - 1) / H;
      return key0 + kHalf - 1 <= last_a && (key0 > last_b - W || key0 + kHalf <= sinks);
    };
    // sum over the group's rows of item t's scores (buffer t & 1)
    auto sum_rows = [&](int nr, int key0, int t, bool open) -> float {
      const int at = ((staged - 1) & 1) * 256;
      const int buf = t & 1, key = key0 + kl;
      if (!(ok = warp_wait_cta(bar(B_S_FULL + buf), (t >> 1) & 1, abort_flag, a.status))) return 0.f;
      tc_fence_after();
      // A row whose lse is -inf adds 0 even where its q holds anything: where its
      // scores made the sum a NaN, a second pass leaves it out. (The question costs
      // 121.8 -> 122.9 us on 16..32 tokens x 64 heads over FP16 keys; a flag beside
      // the staged constants 202 -> 217 on 8 tokens x 64 heads over FP8 keys.)
      auto add_up = [&](auto leave_out) -> float {
        uint64_t s2[2] = {0ull, 0ull};
        float s1 = 0.f;
        for (int cb = halves ? grp : 0; 32 * cb < nr; cb += halves ? 2 : 1) {
          uint32_t sv[32];
          tmem_ld32(tmem + tl + 256u * buf + 32u * cb, sv);
          tmem_wait_ld();
          if (spread) {
#pragma unroll 1
            for (int part = 1; part < kParts; ++part) {
              uint32_t more[32];
              tmem_ld32(tmem + tl + 256u * buf + (uint32_t)(kPartCols * part) + 32u * cb, more);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) sv[i] = __float_as_uint(__uint_as_float(sv[i]) + __uint_as_float(more[i]));
            }
          }
          const float* lr = lse_st + at + 32 * cb;
          if (open && 32 * cb + 32 <= nr) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 l = *reinterpret_cast<const float4*>(lr + i);
              float x0, x1, x2, x3;
              f2_unpack(
                  fma_f32x2(f2_pack(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])), sl2x2, f2_pack(l.x, l.y)), x0,
                  x1);
              f2_unpack(
                  fma_f32x2(f2_pack(__uint_as_float(sv[i + 2]), __uint_as_float(sv[i + 3])), sl2x2, f2_pack(l.z, l.w)),
                  x2, x3);
              if constexpr (decltype(leave_out)::value) {
                x0 = l.x == -INFINITY ? -INFINITY : x0;
                x1 = l.y == -INFINITY ? -INFINITY : x1;
                x2 = l.z == -INFINITY ? -INFINITY : x2;
                x3 = l.w == -INFINITY ? -INFINITY : x3;
              }
              s2[0] = add_f32x2(s2[0], f2_pack(ex2_approx(x0), ex2_approx(x1)));
              s2[1] = add_f32x2(s2[1], f2_pack(ex2_approx(x2), ex2_approx(x3)));
            }
          } else {
            const int* la = last_st + at + 32 * cb;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int last = la[i];
              const bool sees = key <= last && (key > last - W || key < sinks);
              const float x = ex2_approx(fmaf(__uint_as_float(sv[i]), sl2, lr[i]));
              s1 += sees ? x : 0.f;
            }
          }
        }
        float y0, y1, y2, y3;
        f2_unpack(s2[0], y0, y1);
        f2_unpack(s2[1], y2, y3);
        return ((y0 + y1) + (y2 + y3)) + s1;
      };
      float sum = add_up(std::false_type{});
      if (__any_sync(0xffffffffu, sum != sum)) sum = add_up(std::true_type{});
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive(bar(B_S_EMPTY + buf)); else mbar_arrive_remote_relaxed(lead(B_S_EMPTY + buf));
      }
      return sum;
    };
    // this thread's key of a tile: its old weight and its page's table entry,
    // read one tile ahead
    struct Ahead {
      float old;
      int entry;
    };
    auto ahead = [&](const Entry& e, int key0) -> Ahead {
      Ahead h;
      const int key = key0 + kl;
      h.old = prm.k.w_in && key < e.n && key < prm.k.cols && weight_in_bounds(prm.k, e.b, key)
                  ? prm.k.w_in[(int64_t)e.b * prm.k.in_stride + key] : 0.f;
      h.entry = key_entry(a, e, key0 + (kl & ~(kTileKeys - 1)));
      return h;
    };
    auto check_page = [&](int entry) -> bool {
      if (page_valid(a, entry)) return true;
      if ((kl & (kTileKeys - 1)) == 0) atomicOr(a.status, MLA_DEV_BAD_PAGE);
      return false;
    };
    auto write = [&](const Entry& e, int key, float old, float sum) {
      if (key >= e.n || key >= prm.k.cols) return;
      // (test mode 2 of the checking build: every store past its row, where the check skips it)
      const int64_t at = key + (MLA_BOUNDS_CHECK && p.fault_test == 2 ? prm.k.cols : 0);
      if (weight_in_bounds(prm.k, e.b, at)) prm.k.w_out[(int64_t)e.b * prm.k.out_stride + at] = prm.k.decay * old + sum;
    };
    auto tile_key = [&]() -> int { return kTile * w.tile(p) + kHalf * (int)rank; };

    if (halves) {
      Ahead next{0.f, 0};
      RowLse next_l{};
      int ng0 = 0, ng1 = 1;
      bool next_other = true;
      auto look_ahead = [&]() {  // the next tile's constants, on their way while this one is summed
        next_other = w.seek(prm);
        next = ahead(w.e, tile_key());
        if (kGroups) tile_groups(prm, w.e, kTile * w.tile(p), ng0, ng1);
        if (kGroups || next_other) next_l = load_lse(w.e, ng0 * N, min(N, w.e.rows - ng0 * N));
      };
      if (w.more()) look_ahead();
      while (ok && w.more()) {
        const Entry e = w.e;
        const int key0 = tile_key(), key = key0 + kl, g0 = ng0, g1 = ng1;
        const Ahead cur = next;
        const bool other = next_other;
        RowLse cur_l = next_l;
        w.idx += w.step;
        if (w.more()) look_ahead();
        float sum = 0.f;
        for (int g = g0; ok && g < g1; ++g, ++jt) {
          const int nr = min(N, e.rows - g * N);
          const bool open = open_tile(e, g * N, nr, key0);
          // (one group: its rows stay staged, with their newest keys, for the entry's next tiles)
          if (kGroups || other) stage(e, g * N, nr, cur_l, !kGroups || !open || (nr & 31));
          if (g + 1 < g1) cur_l = load_lse(e, (g + 1) * N, min(N, e.rows - (g + 1) * N));
          if (ok) sum += sum_rows(nr, key0, jt, open);
        }
        if (!ok) break;
        // group 1's part through shared memory, then the sum in a fixed order
        if (grp == 1) {
          if (outer > 0 && !(ok = warp_wait_cta(bar(B_SUM_READ), (outer - 1) & 1, abort_flag, a.status))) break;
          sums[kl] = sum;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_SUM));
        } else {
          if (!(ok = warp_wait_cta(bar(B_SUM), outer & 1, abort_flag, a.status))) break;
          sum += sums[kl];
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_SUM_READ));
          write(e, key, cur.old, check_page(cur.entry) ? sum : 0.f);
        }
        ++outer;
      }
    } else {
      // the group's tiles are every other one of the pair's run; an entry's
      // constants are staged by both groups when the run reaches it
      int staged_for = -1;
      auto to_own = [&]() {  // to the group's next tile; the entries passed on the way
        while (ok && w.more()) {
          w.seek(prm);
          if ((jt & 1) == grp) return;
          ++w.idx, ++jt;
        }
      };
      to_own();
      Ahead next{0.f, 0};
      if (w.more()) next = ahead(w.e, tile_key());
      while (ok && w.more()) {
        const Entry e = w.e;
        const int key0 = tile_key(), key = key0 + kl, t = jt;
        const Ahead cur = next;
        if (staged_for != e.b) {
          stage(e, 0, e.rows, load_lse(e, 0, e.rows), true);
          staged_for = e.b;
          if (!ok) break;
        }
        ++w.idx, ++jt;
        to_own();
        if (w.more()) next = ahead(w.e, tile_key());
        const float sum = sum_rows(e.rows, key0, t, open_tile(e, 0, e.rows, key0));
        if (!ok) break;
        write(e, key, cur.old, check_page(cur.entry) ? sum : 0.f);
      }
    }
    tc_fence_before();
  }

  // ---------------------------------------------------------------- teardown
  // The leader's commits arrive in both CTAs; each waits for the last phase of
  // every barrier they arrive on before it may leave (S_FULL was waited for).
  __syncthreads();
  if (warp == 2 && !*abort_flag) {
    const int t = issued[0] - 1 - lane;
    if (lane < NS && t >= 0) drain_phase(bar(B_EMPTY + t % NS), (uint32_t)(t / NS) & 1);
    const int s = lane - kMaxStages;
    if (kStays && s >= 0 && s < C::kSlots && issued[1] > 0) drain_phase(bar(B_RES_EMPTY + s), (uint32_t)(issued[1] - 1) & 1);
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if (*abort_flag) spin_ns(1000000ull);  // let any MMA still in flight finish
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int E, int kForm, int kPer>
cudaError_t launch(KeyWeightParams& prm, cudaStream_t stream) {
  using C = Cut<E, kPer, kForm>;
  const uint32_t res = kForm == kBothStream ? 0u
                       : C::kChunks * (kForm == kKeysStay ? (uint32_t)kHalf : (uint32_t)prm.n_cols / 2) * 128u;
  const uint32_t data = kDataOff + ((res + 1023u) & ~1023u);
  const int stages = (int)((kSmemMax - data) / C::kSlotBytes);
  prm.stages = stages < kMaxStages ? stages : kMaxStages;
  const uint32_t smem = data + (uint32_t)prm.stages * C::kSlotBytes + 1024u;
  auto* const kernel = tc_key_weights_kernel<E, kForm, kPer>;
  static std::atomic<uint64_t> smem_set{0};
  if (cudaError_t e = set_max_dynamic_smem((const void*)kernel, (int)(kSmemMax + 1024), smem_set); e != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)kNumSMs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, prm);
}

}  // namespace

cudaError_t launch_key_weights_tc(const KeyWeightArgs& k, cudaStream_t stream) {
  const mla_plan& p = k.a.plan;
  const int E = p.dtype == MLA_FP8_E4M3 ? 1 : 2;
  const int64_t rows_max = (int64_t)p.q_len * p.num_heads;
  // N: the entry's rows in as few groups of at most 256 as hold them, evenly
  const int64_t groups = (rows_max + 255) / 256;
  const int N = (int)(((rows_max + groups - 1) / groups + 31) / 32 * 32);
  const uint64_t q_rows = (uint64_t)k.a.total_q * p.num_heads;
  const uint64_t kv_rows = (uint64_t)k.a.num_pages * kTileKeys;
  KeyWeightParams prm;
  prm.k = k;
  prm.n_cols = N;
  prm.parts = E == 2 && N <= kPartCols ? kParts : 1;
  const uint32_t fmt = p.dtype == MLA_BF16 ? 1u : 0u;  // BF16 = 1, FP16 = 0; E4M3 = 0 in its own kind
  prm.idesc = instr_desc(fmt, fmt, 0, 256, (uint32_t)N);
  // without a query token no tile is ever loaded; the maps still need an array
  const void* q = q_rows > 0 ? k.a.q : k.a.kv_cache;
  const uint64_t qr = q_rows > 0 ? q_rows : kv_rows;
  const uint32_t dims = (uint32_t)(128 / E), box_q = (uint32_t)(N / 2);
  if (!encode_rows_576(&prm.tm_q, q, E, qr, dims, box_q, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_rows_576(&prm.tm_k, k.a.kv_cache, E, kv_rows, dims, kTileKeys, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if (E == 1) {
    if (!encode_rows_576(&prm.tm_q_rope, q, E, qr, 64, box_q, CU_TENSOR_MAP_SWIZZLE_64B) ||
        !encode_rows_576(&prm.tm_k_rope, k.a.kv_cache, E, kv_rows, 64, kTileKeys, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  } else {
    prm.tm_q_rope = prm.tm_q;
    prm.tm_k_rope = prm.tm_k;
  }
  // entries per launch: their tile counts fit shared memory, and their sum an int
  const int64_t tiles = (int64_t)p.max_seq_len / kTile + 2;
  const int64_t fit = INT32_MAX / tiles;
  const int per = (int)(fit < kMaxEntries ? fit : kMaxEntries);
  for (int b0 = 0; b0 < p.batch; b0 += per) {
    prm.b0 = b0;
    prm.nb = p.batch - b0 < per ? p.batch - b0 : per;
    cudaError_t e;
    if (E == 1)
      e = groups > 1 ? launch<1, kKeysStay, 2>(prm, stream) : launch<1, kRowsStay, 2>(prm, stream);
    else
      e = N > 128 ? launch<2, kBothStream, 1>(prm, stream) : launch<2, kRowsStay, 2>(prm, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mla
