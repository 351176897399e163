// The planner of the packed prefill (prefill_ragged.cu and, for head_dim 256,
// prefill_wide.cu).
#include "bia_internal.h"
#include "ptx.cuh"

namespace bia {

namespace {

// ---------------------------------------------------------------- plan
// One CTA turns the index arrays into per-request records and the units
// (request, group of q tiles, split; one per CTA of a cluster), checks each
// request and clears the status word and the item counter.  Requests and
// their groups are taken in chunks of the block: one scan gives the requests'
// first groups, partial rows and merge rows; then the chunk's units are
// sorted by their key blocks, the most first, into bins of 1/8 octave, as the
// CTAs take units off the list one by one and short ones fill the end best
// (one prompt of 8192 tokens, 8 heads over 2: 163 -> 156 us).  Units of a bin
// come in any order: they are computed alike wherever they stand.  Nothing is
// written past the capacities of the launch; a plan that differs from the
// host's retires every unit and fills the outputs with NaN.  (The general
// planner, plan.cu, takes five scans and looks its groups up in global
// memory: 8 us a call of a few requests, this one 6.)
constexpr int kPlanThreadsR = 512;
constexpr int kPlanWarpsR = kPlanThreadsR / 32;
constexpr int kBinsR = 192; // bin_of(2^23 blocks of 128 keys) is 175

__device__ __forceinline__ int bin_of(int32_t blocks) {
  if (blocks < 8) return max(blocks, 0);
  const int k = 31 - __clz(blocks);
  return 8 + (k - 3) * 8 + ((blocks >> (k - 3)) & 7);
}

struct RaggedRequest {
  int32_t q_start, q_len, kv_begin, kv_len, groups, nsp;
  int64_t rows;
  int32_t merge;
  bool ok;
};

__device__ __forceinline__ RaggedRequest ragged_request(const PlanArgs &p, int b, int32_t gt) {
  RaggedRequest r;
  r.q_start = p.qo_indptr[b];
  r.kv_begin = p.kv_indptr[b];
  const int32_t q_end = p.qo_indptr[b + 1], kv_end = p.kv_indptr[b + 1];
  const int64_t ql = static_cast<int64_t>(q_end) - r.q_start;
  const int64_t kl = static_cast<int64_t>(kv_end) - r.kv_begin;
  r.ok = ql >= 0 && kl >= 0 && kl <= INT32_MAX / 2 && ql <= INT32_MAX / 2 &&
         (!p.causal || ql <= kl) && r.q_start >= 0 && q_end <= p.max_total_q && r.kv_begin >= 0 &&
         kv_end <= p.max_kv_len;
  r.q_len = r.ok ? static_cast<int32_t>(ql) : 0;
  r.kv_len = r.ok ? static_cast<int32_t>(kl) : 0;
  const int32_t tiles = (r.q_len + p.tile_tokens - 1) / p.tile_tokens;
  r.groups = (tiles + gt - 1) / gt;
  r.nsp = tiles > 0
              ? tile_splits(r.q_len, r.kv_len, tiles - 1, p.tile_tokens, p.causal, p.split) : 1;
  r.rows = r.nsp > 1 ? static_cast<int64_t>(r.q_len) * r.nsp : 0;
  r.merge = r.nsp > 1 ? r.q_len - merge_first_token(r.q_len, r.kv_len, p.tile_tokens, p.causal,
                                                    p.split) : 0;
  return r;
}

// Exclusive scan of one value per thread across the block, and its total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *s_warp, int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  __syncthreads(); // the last scan's sums are read
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarpsR; ++w) {
    before += w < warp ? s_warp[w] : 0;
    total += s_warp[w];
  }
  return before + incl - v;
}

__global__ void __launch_bounds__(kPlanThreadsR) plan_ragged_kernel(const PlanArgs p) {
  __shared__ int64_t s_warp[kPlanWarpsR], s_rows[kPlanWarpsR];
  __shared__ int32_t s_group[kPlanThreadsR + 1]; // first group of each request of the chunk
  __shared__ int32_t s_q[kPlanThreadsR], s_kv[kPlanThreadsR];
  __shared__ int32_t s_bin[kBinsR]; // units of each bin, then the next one's place
  const int tid = threadIdx.x;
  grid_dep_launch(); // the attention kernel may set itself up meanwhile
  grid_dep_wait();   // this kernel rewrites the workspace
  const int32_t gt = group_tiles(p.tiles_per_unit, p.ctas);
  if (tid == 0) {
    p.status[0] = 0;
    p.status[kStatusWorkCounter] = 0;
  }
  // the ends too: the rows of the buffers are counted from the host's arrays
  bool bad = tid == 0 && (p.kv_indptr[0] < 0 || p.qo_indptr[0] != 0 ||
                          p.qo_indptr[p.batch] != p.max_total_q ||
                          p.kv_indptr[p.batch] != p.max_kv_len);
  int64_t groups = 0, rows = 0, merges = 0, units = 0; // of the chunks before
  for (int b0 = 0; b0 < p.batch; b0 += kPlanThreadsR) {
    const int b = b0 + tid;
    RaggedRequest r{};
    r.ok = true;
    if (b < p.batch) r = ragged_request(p, b, gt);
    // a chunk whose requests follow one another within the host's totals has no
    // more groups and splits than fit those: the loops below end in time,
    // whatever the arrays hold
    bad = __syncthreads_or(bad || !r.ok) != 0;
    if (bad) break;
    // groups in the low half, merge rows in the high half (each below 2^31)
    int64_t n_gm, n_rows;
    const int64_t gm = block_scan(r.groups + (static_cast<int64_t>(r.merge) << 32), s_warp, n_gm);
    const int64_t row = block_scan(r.rows, s_rows, n_rows);
    const int32_t n_groups = static_cast<int32_t>(n_gm & 0xffffffff);
    if (b < p.batch) {
      ReqInfo x;
      x.q_start = r.q_start;
      x.q_len = r.q_len;
      x.kv_len = r.kv_len;
      x.nsp = r.nsp;
      x.rowbase = r.rows > 0 ? rows + row : -1;
      x.page_base = r.kv_begin;
      x.mbase = static_cast<int32_t>(merges + (gm >> 32));
      p.reqs[b] = x;
    }
    s_group[tid] = static_cast<int32_t>(gm & 0xffffffff);
    if (tid == 0) s_group[kPlanThreadsR] = n_groups;
    s_q[tid] = r.q_len;
    s_kv[tid] = r.kv_len;
    __syncthreads();
    const int nb = min(kPlanThreadsR, p.batch - b0);
    for (int32_t g0 = 0; g0 < n_groups; g0 += kPlanThreadsR) {
      const int32_t g = g0 + tid;
      int lo = 0, n = 0;
      int32_t t0 = 0, tiles = 0;
      if (g < n_groups) {
        int hi = nb - 1; // largest request with s_group <= g
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_group[mid] <= g) lo = mid;
          else hi = mid - 1;
        }
        tiles = (s_q[lo] + p.tile_tokens - 1) / p.tile_tokens;
        t0 = ((tiles + gt - 1) / gt - 1 - (g - s_group[lo])) * gt;
        n = tile_splits(s_q[lo], s_kv[lo], min(t0 + gt, tiles) - 1, p.tile_tokens, p.causal,
                        p.split);
      }
      const int32_t keys =
          n > 0 ? tile_last_key(s_q[lo], s_kv[lo], min(t0 + gt, tiles) - 1, p.tile_tokens,
                                p.causal) + 1 : 0;
      auto bin = [&](int32_t s) {
        const int64_t left = keys - static_cast<int64_t>(s) * p.split;
        return bin_of((static_cast<int32_t>(min(left, static_cast<int64_t>(p.split))) +
                       kKvBlock - 1) / kKvBlock);
      };
      if (tid < kBinsR) s_bin[tid] = 0;
      __syncthreads();
      for (int32_t s = 0; s < n; ++s) atomicAdd(&s_bin[bin(s)], 1);
      __syncthreads();
      int64_t total;
      const int64_t place =
          block_scan(tid < kBinsR ? s_bin[kBinsR - 1 - tid] : 0, s_warp, total);
      if (tid < kBinsR) s_bin[kBinsR - 1 - tid] = static_cast<int32_t>(place);
      __syncthreads();
      for (int32_t s = 0; s < n; ++s) {
        const int64_t u = units + static_cast<int64_t>(atomicAdd(&s_bin[bin(s)], 1)) * p.ctas;
        for (int32_t c = 0; c < p.ctas; ++c) {
          const int32_t tile = t0 + c * p.tiles_per_unit;
          if (u + c < p.n_units_expected)
            p.units[u + c] = Unit{b0 + lo, tile, s, max(0, min(p.tiles_per_unit, tiles - tile))};
        }
      }
      __syncthreads(); // the bins are read
      total *= p.ctas;
      units += total;
    }
    groups += n_groups;
    merges += n_gm >> 32;
    rows += n_rows;
  }
  const bool ok = !bad && groups == p.n_groups_expected &&
                  rows == p.part_rows_expected && units == p.n_units_expected;
  if (tid == 0) p.status[kStatusMergeRows] = ok ? static_cast<int32_t>(merges) : 0;
  if (ok) return;
  if (tid == 0) atomicOr(p.status, kStatusPlanMismatch);
  for (int64_t i = tid; i < p.n_units_expected; i += kPlanThreadsR) p.units[i] = Unit{-1, 0, 0, 0};
  // nothing will be computed: the outputs read NaN instead of stale values
  for (int64_t i = tid; i < p.out_elems; i += kPlanThreadsR) p.out[i] = 0x7fc0u; // bf16 NaN
  for (int64_t i = tid; p.lse && i < p.lse_elems; i += kPlanThreadsR)
    p.lse[i] = __int_as_float(0x7fc00000);
}

} // namespace

cudaError_t launch_plan_ragged(const PlanArgs &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreadsR);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_ragged_kernel, p);
}

} // namespace bia
