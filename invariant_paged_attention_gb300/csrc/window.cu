// Around the kernels of the attention with a window and sinks: the extend's
// plan, and what joins the states that split tiles left, in order (fold.cuh),
// and the status words of a decode's CTAs.
#include "bia_internal.h"
#include "fold.cuh"
#include "ptx.cuh"

namespace bia {

namespace {

constexpr int kJoinWarps = 4;

// Folds the n states of one row, D/32 (rounded up to a multiple of 4) columns
// a lane, and stores it.
template <int V>
__device__ __forceinline__ void fold_row(const float *part_o, const float *part_lse, int n,
                                         int64_t step, int D, int lane, uint16_t *out,
                                         float *lse) {
  float L = -INFINITY, o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  for (int s = 0; s < n; ++s) {
    float v[V];
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const int e = k * 32 + lane * 4;
      const float4 x = e < D ? __ldg(reinterpret_cast<const float4 *>(part_o + s * step * D + e))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
      v[k] = x.x, v[k + 1] = x.y, v[k + 2] = x.z, v[k + 3] = x.w;
    }
    fold_state<V>(L, o, __ldg(part_lse + s * step), v);
  }
#pragma unroll
  for (int k = 0; k < V; k += 4) {
    const int e = k * 32 + lane * 4;
    if (e < D)
      *reinterpret_cast<uint2 *>(out + e) =
          make_uint2(pack_bf16(o[k], o[k + 1]), pack_bf16(o[k + 2], o[k + 3]));
  }
  if (lse && lane == 0) *lse = L;
}

// One warp a (request, q head); the first CTA also joins the status words.
__global__ void __launch_bounds__(kJoinWarps * 32)
    merge_window_decode_kernel(const __grid_constant__ AttnArgs a, const int n_slots) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0) {
    int32_t st = 0;
    for (int i = threadIdx.x; i < n_slots; i += kJoinWarps * 32) st |= a.slots[i];
#pragma unroll
    for (int bit = 1; bit <= kStatusTimeout; bit <<= 1) // every status bit of a decode
      st |= __syncthreads_or(st & bit) ? bit : 0;
    if (threadIdx.x == 0) a.status[0] = st;
  }
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.batch) * a.Hq) return;
  const int b = static_cast<int>(row / a.Hq), h = static_cast<int>(row - static_cast<int64_t>(b) * a.Hq);
  const WindowKeys k = window_keys(a, b);
  const int n = window_tiles(k, a.split);
  if (n <= 1) return; // stored by its only tile, or NaN
  const int64_t first = static_cast<int64_t>(b) * a.parts * a.Hq + h;
  const float *po = a.part_o + first * a.D, *pl = a.part_lse + first;
  uint16_t *out = a.out + row * a.D;
  float *lse = a.lse ? a.lse + row : nullptr;
  if (a.D <= 128) fold_row<4>(po, pl, n, a.Hq, a.D, lane, out, lse);
  else fold_row<8>(po, pl, n, a.Hq, a.D, lane, out, lse);
}

constexpr int kPlanThreadsW = 256;

// The record of every request and the q tile pairs before it.  Arrays that
// break a rule or that the launch was not sized for: no pair at all, status
// bit 1 and NaN in the outputs.
__global__ void __launch_bounds__(kPlanThreadsW) plan_window_kernel(const PlanArgs p) {
  __shared__ int64_t s_warp[kPlanThreadsW / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait(); // this kernel rewrites the workspace
  grid_dep_launch();
  bool ok = true;
  int64_t before = 0; // pairs of the requests before this chunk's
  for (int b0 = 0; b0 < p.batch && ok; b0 += kPlanThreadsW) {
    const int b = b0 + tid;
    int64_t pairs = 0;
    bool good = true;
    ReqInfo r{};
    if (b < p.batch) {
      const int32_t q0 = p.qo_indptr[b], q1 = p.qo_indptr[b + 1];
      const int32_t p0 = p.kv_indptr[b], p1 = p.kv_indptr[b + 1];
      const int32_t last = p.kv_last_page_len[b];
      const int64_t ql = static_cast<int64_t>(q1) - q0, pages = static_cast<int64_t>(p1) - p0;
      const int64_t kl = pages > 0 ? (pages - 1) * p.page_size + last : 0;
      good = q0 >= 0 && ql >= 0 && q1 <= p.max_total_q && p0 >= 0 && pages >= 0 &&
             (pages == 0 || (last >= 1 && last <= p.page_size)) && kl <= p.max_kv_len &&
             ql <= kl && (b > 0 || q0 == 0) && (b < p.batch - 1 || q1 == p.max_total_q);
      r.q_start = q0;
      r.q_len = static_cast<int32_t>(ql);
      r.kv_len = static_cast<int32_t>(kl);
      r.page_base = p0;
      if (good) {
        const int64_t tiles = (ql + p.tile_tokens - 1) / p.tile_tokens;
        pairs = (tiles + p.tiles_per_unit - 1) / p.tiles_per_unit;
      }
    }
    ok = __syncthreads_and(good) != 0;
    int64_t incl = pairs;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += x;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int64_t excl = before + incl - pairs;
#pragma unroll
    for (int w = 0; w < kPlanThreadsW / 32; ++w) {
      excl += w < warp ? s_warp[w] : 0;
      before += s_warp[w];
    }
    ok = ok && before <= p.n_groups_expected;
    if (ok && b < p.batch) {
      p.reqs[b] = r;
      p.group_off[b] = static_cast<int32_t>(excl);
    }
    __syncthreads(); // the warps' sums are read
  }
  ok = ok && before == p.n_groups_expected;
  if (tid == 0) {
    p.status[0] = ok ? 0 : kStatusPlanMismatch;
    p.status[kStatusWorkCounter] = 0;
    p.status[kStatusMergeRows] = ok ? static_cast<int32_t>(before) : 0;
  }
  if (ok) return;
  for (int64_t i = tid; i < p.out_elems; i += kPlanThreadsW) p.out[i] = 0x7fc0u; // bf16 NaN
  for (int64_t i = tid; p.lse && i < p.lse_elems; i += kPlanThreadsW)
    p.lse[i] = __int_as_float(0x7fc00000);
}

// A CTA a token: folds the states of its heads' split tiles.
__global__ void __launch_bounds__(kJoinWarps * 32)
    merge_window_kernel(const __grid_constant__ AttnArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  if (a.status[kStatusMergeRows] == 0) return; // the plan failed its checks
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t token = blockIdx.x;
  int lo = 0, n = a.batch; // its request: the largest b with q_start <= token
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool le = lane * step < n && a.reqs[lo + lane * step].q_start <= token;
    const int k = max(0, 31 - __clz(__ballot_sync(0xffffffffu, le)));
    lo += k * step;
    n = min(step, n - k * step);
  }
  const ReqInfo r = a.reqs[lo];
  const TileKeys t = tile_keys(r.q_len, r.kv_len, static_cast<int32_t>(token - r.q_start) / a.tile_tokens,
                               a.tile_tokens, a.window, a.sinks, a.split, window_key_block(a.D));
  const int parts = t.s1 - t.s0 + 1;
  if (parts <= 1) return; // stored by its only tile
  for (int h = warp; h < a.Hq; h += kJoinWarps) {
    const int64_t first = token * a.parts * a.Hq + h, row = token * a.Hq + h;
    const float *po = a.part_o + first * a.D, *pl = a.part_lse + first;
    uint16_t *out = a.out + row * a.D;
    float *lse = a.lse ? a.lse + row : nullptr;
    if (a.D <= 128) fold_row<4>(po, pl, parts, a.Hq, a.D, lane, out, lse);
    else fold_row<8>(po, pl, parts, a.Hq, a.D, lane, out, lse);
  }
}

cudaError_t launch_chained(const void *fn, unsigned grid, unsigned block, void **args,
                           cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

} // namespace

cudaError_t launch_plan_window(const PlanArgs &p, cudaStream_t s) {
  void *args[] = {const_cast<PlanArgs *>(&p)};
  return launch_chained(reinterpret_cast<const void *>(plan_window_kernel), 1, kPlanThreadsW, args,
                        s);
}

cudaError_t launch_merge_window(const AttnArgs &a, cudaStream_t s) {
  void *args[] = {const_cast<AttnArgs *>(&a)};
  return launch_chained(reinterpret_cast<const void *>(merge_window_kernel),
                        static_cast<unsigned>(a.total_rows), kJoinWarps * 32, args, s);
}

cudaError_t launch_merge_window_decode(const AttnArgs &a, int n_slots, cudaStream_t s) {
  // without a second tile there are only the status words
  const int64_t rows = a.parts > 1 ? static_cast<int64_t>(a.batch) * a.Hq : 1;
  void *args[] = {const_cast<AttnArgs *>(&a), &n_slots};
  return launch_chained(reinterpret_cast<const void *>(merge_window_decode_kernel),
                        static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps),
                        kJoinWarps * 32, args, s);
}

} // namespace bia
