// The planner, the merge and the dispatch of the 8-bit decode (decode_fp8.cuh).
#include <algorithm>

#include "bia_internal.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace bia {

namespace {

// ---------------------------------------------------------------- plan
// One CTA turns the index arrays into per-request records and the units
// (request, split), checks each request (and the bounds of a bounded call),
// and clears the status word and the item counter.  A plan that does not fit
// the launch retires every unit and fills the outputs with NaN.  The general
// planner (plan.cu) does the same for every kind of call with four scans and
// three passes over the units; a decode needs one scan.
constexpr int kPlanThreads8 = 512;

__device__ __forceinline__ bool keys_of(const PlanArgs &p, int b, int32_t &kv_len) {
  const int64_t pages = static_cast<int64_t>(p.kv_indptr[b + 1]) - p.kv_indptr[b];
  const int32_t last = p.kv_last_page_len[b];
  const int64_t kl = pages > 0 ? (pages - 1) * p.page_size + last : 0;
  const bool ok = pages > 0 && last >= 1 && last <= p.page_size && kl <= INT32_MAX / 2 &&
                  (!p.bounded || kl <= p.max_kv_len);
  kv_len = ok ? static_cast<int32_t>(kl) : 0;
  return ok;
}

__global__ void __launch_bounds__(kPlanThreads8)
    plan_decode_fp8_kernel(const PlanArgs p, UnitFp8 *units_out) {
  __shared__ int64_t s_warp[kPlanThreads8 / 32];
  __shared__ int32_t s_off[kPlanThreads8 + 1]; // first unit of each request of the chunk
  __shared__ int32_t s_keys[kPlanThreads8], s_page[kPlanThreads8];
  __shared__ int64_t s_row[kPlanThreads8]; // its first partial row, -1: one split
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_launch(); // the decode may set itself up meanwhile
  grid_dep_wait();   // this kernel rewrites the workspace
  // every request's check and the totals first: nothing is written past the
  // capacities of the launch
  bool bad = tid == 0 && p.kv_indptr[0] < 0;
  int64_t units = 0, rows = 0; // unit and partial-row totals of this thread's requests
  for (int b = tid; b < p.batch; b += kPlanThreads8) {
    int32_t kv_len;
    bad = !keys_of(p, b, kv_len) || bad;
    const int32_t nsp = (kv_len + p.split - 1) / p.split;
    units += nsp;
    rows += nsp > 1 ? nsp : 0;
  }
  if (tid == 0) {
    p.status[0] = 0;
    p.status[kStatusWorkCounter] = 0;
  }
  auto block_sum = [&](int64_t v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    __syncthreads();
    if (lane == 0) s_warp[warp] = v;
    __syncthreads();
    int64_t t = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads8 / 32; ++w) t += s_warp[w];
    return t;
  };
  const bool any_bad = __syncthreads_or(bad) != 0;
  const int64_t n_units = block_sum(units), n_rows = block_sum(rows);
  const bool ok = !any_bad && (p.bounded ? n_units <= p.n_units_expected && n_rows <= p.part_rows_expected
                                         : n_units == p.n_units_expected && n_rows == p.part_rows_expected);
  if (!ok) {
    if (tid == 0) atomicOr(p.status, kStatusPlanMismatch);
    for (int64_t i = tid; i < p.n_units_expected; i += kPlanThreads8) units_out[i].b = -1;
    for (int64_t i = tid; i < p.out_elems; i += kPlanThreads8) p.out[i] = 0x7fc0u; // bf16 NaN
    for (int64_t i = tid; p.lse && i < p.lse_elems; i += kPlanThreads8)
      p.lse[i] = __int_as_float(0x7fc00000);
    return;
  }
  int64_t unit0 = 0, row0 = 0; // of the chunk of kPlanThreads8 requests
  for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads8) {
    const int b = b0 + tid;
    int32_t kv_len = 0;
    if (b < p.batch) keys_of(p, b, kv_len);
    const int32_t nsp = (kv_len + p.split - 1) / p.split;
    // units in the low half, partial rows in the high half (each below 2^31)
    const int64_t mine = nsp + (static_cast<int64_t>(nsp > 1 ? nsp : 0) << 32);
    int64_t incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += x;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads8 / 32; ++w) {
      before += w < warp ? s_warp[w] : 0;
      total += s_warp[w];
    }
    const int64_t excl = before + incl - mine;
    s_off[tid] = static_cast<int32_t>(excl & 0xffffffff);
    if (tid == 0) s_off[kPlanThreads8] = static_cast<int32_t>(total & 0xffffffff);
    if (b < p.batch) {
      ReqInfo r;
      r.q_start = b;
      r.q_len = 1;
      r.kv_len = kv_len;
      r.nsp = nsp;
      r.rowbase = nsp > 1 ? row0 + (excl >> 32) : -1;
      r.page_base = p.kv_indptr[b];
      r.mbase = 0;
      p.reqs[b] = r;
      s_keys[tid] = kv_len;
      s_page[tid] = r.page_base;
      s_row[tid] = r.rowbase;
    }
    __syncthreads();
    const int32_t n = s_off[kPlanThreads8], nb = min(kPlanThreads8, p.batch - b0);
    for (int32_t i = tid; i < n; i += kPlanThreads8) {
      int lo = 0, hi = nb - 1; // largest request with s_off <= i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_off[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      const int32_t split = i - s_off[lo];
      UnitFp8 u;
      u.b = b0 + lo;
      u.key_begin = split * p.split;
      u.key_end = min(u.key_begin + p.split, s_keys[lo]);
      u.page_base = s_page[lo];
      u.prow = s_row[lo] < 0 ? -1 : s_row[lo] + split;
      u.pad = 0;
      units_out[unit0 + i] = u;
    }
    unit0 += n;
    row0 += total >> 32;
  }
  for (int64_t i = unit0 + tid; i < p.n_units_expected; i += kPlanThreads8)
    units_out[i].b = -1; // a bounded launch has room for more
}

// ---------------------------------------------------------------- merge
// Joins a row's split states: with L = max lse_s and w_s = e^(lse_s - L),
// o = sum w_s o_s / sum w_s in ascending split order.  A warp per (request, q
// head); the weights of 32 splits come from their lanes at once and eight
// states' loads are in flight, so a row costs a few memory latencies whatever
// its number of splits (the streamed merge of the bf16 calls walks a token's
// heads and splits one after the other in one CTA: 17 us for 8 requests).
constexpr int kMergeWarps8 = 8;

template <int V>
__global__ void __launch_bounds__(kMergeWarps8 * 32) merge_decode_fp8_kernel(const DecodeGeometry a) {
  constexpr int kChunk = V == 4 ? 8 : 4; // states in flight
  const int lane = threadIdx.x & 31;
  grid_dep_wait(); // the partials are complete
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeWarps8 + (threadIdx.x >> 5);
  const int b = static_cast<int>(row / a.Hq), h = static_cast<int>(row - static_cast<int64_t>(b) * a.Hq);
  ReqInfo r{};
  if (a.slots) { // the decode planned itself: so does the merge, and joins the status
    int32_t noted = 0;
    for (int i = lane; i < a.n_slots; i += 32) noted |= a.slots[i];
    LaneRequest mine;
    const bool ok = lane_requests(a, lane, mine);
    noted = __reduce_or_sync(0xffffffffu, noted);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.status[0] = noted;
    if (!ok || (noted & kStatusPlanMismatch)) return; // the outputs already hold NaN
    r.nsp = __shfl_sync(0xffffffffu, mine.nsp, b & 31);
    r.rowbase = __shfl_sync(0xffffffffu, mine.rows_end, b & 31) - r.nsp;
  } else if (a.status[0] & kStatusPlanMismatch) {
    return; // the outputs already hold NaN
  }
  if (row >= static_cast<int64_t>(a.batch) * a.Hq) return;
  if (!a.slots) r = a.reqs[b];
  if (r.nsp <= 1) return; // the decode wrote the final row
  const float *lse = a.part_lse + r.rowbase * a.Hq + h;
  const float *part = a.part_o + (r.rowbase * a.Hq + h) * a.D + lane * 4;
  const int64_t step = static_cast<int64_t>(a.Hq) * a.D;
  float L = -INFINITY, sum = 0.f, o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  for (int s0 = 0; s0 < r.nsp; s0 += 32) {
    const int n = min(32, r.nsp - s0);
    const float mine = lane < n ? __ldg(lse + static_cast<int64_t>(s0 + lane) * a.Hq) : -INFINITY;
    const float top = fmaxf(L, warp_max(mine));
    const float base = top == -INFINITY ? 0.f : top;
    const float down = ex2((L - base) * kLog2e); // 0 for the first chunk
    const float w = ex2((mine - base) * kLog2e); // 0 for a state without keys
    float wsum = w;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, off);
    sum = __fadd_rn(__fmul_rn(sum, down), wsum);
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = __fmul_rn(o[i], down);
    L = top;
    for (int k0 = 0; k0 < n; k0 += kChunk) {
      float4 v[kChunk][V / 4];
#pragma unroll
      for (int c = 0; c < kChunk; ++c)
#pragma unroll
        for (int e = 0; e < V / 4; ++e) {
          v[c][e] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k0 + c < n && e * 128 + lane * 4 < a.D)
            v[c][e] = __ldg(reinterpret_cast<const float4 *>(part + (s0 + k0 + c) * step + e * 128));
        }
#pragma unroll
      for (int c = 0; c < kChunk; ++c) {
        const float wc = __shfl_sync(0xffffffffu, w, (k0 + c) & 31); // 0 past the last state
        if (k0 + c < n) {
#pragma unroll
          for (int e = 0; e < V / 4; ++e) {
            o[4 * e] = __fmaf_rn(wc, v[c][e].x, o[4 * e]);
            o[4 * e + 1] = __fmaf_rn(wc, v[c][e].y, o[4 * e + 1]);
            o[4 * e + 2] = __fmaf_rn(wc, v[c][e].z, o[4 * e + 2]);
            o[4 * e + 3] = __fmaf_rn(wc, v[c][e].w, o[4 * e + 3]);
          }
        }
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : __frcp_rn(sum);
#pragma unroll
  for (int e = 0; e < V / 4; ++e)
    if (e * 128 + lane * 4 < a.D) {
      uint2 x;
      x.x = pack_bf16(__fmul_rn(o[4 * e], inv), __fmul_rn(o[4 * e + 1], inv));
      x.y = pack_bf16(__fmul_rn(o[4 * e + 2], inv), __fmul_rn(o[4 * e + 3], inv));
      *reinterpret_cast<uint2 *>(a.out + row * a.D + e * 128 + lane * 4) = x;
    }
  if (a.lse && lane == 0)
    a.lse[row] = sum == 0.f ? -INFINITY : __fadd_rn(L, __fmul_rn(lg2(sum), kLn2));
}

template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*fn)(Params...), unsigned grid, unsigned block, cudaStream_t s,
                           const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, args...);
}

} // namespace

cudaError_t launch_plan_decode_fp8(const PlanArgs &p, UnitFp8 *units, cudaStream_t s) {
  return launch_chained(plan_decode_fp8_kernel, 1, kPlanThreads8, s, p, units);
}

cudaError_t launch_merge_decode_fp8(const DecodeGeometry &a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.batch) * a.Hq;
  const int64_t grid = (rows + kMergeWarps8 - 1) / kMergeWarps8;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return a.D <= 128 ? launch_chained(merge_decode_fp8_kernel<4>, static_cast<unsigned>(grid),
                                     kMergeWarps8 * 32, s, a)
                    : launch_chained(merge_decode_fp8_kernel<8>, static_cast<unsigned>(grid),
                                     kMergeWarps8 * 32, s, a);
}

cudaError_t decode_plans_itself(int batch, int64_t items, int64_t part_rows, bool *itself) {
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  *itself = batch <= 32 && part_rows > 0 && items <= std::min<int64_t>(sms, kDecodeSlots);
  return e;
}

cudaError_t launch_decode_fp8(const DecodeFp8Args &f, cudaStream_t s) {
  if (f.a.n_units == 0) return cudaSuccess;
  switch (f.a.G) {
  case 1: return launch_decode_fp8_g1(f, s);
  case 2: return launch_decode_fp8_g2(f, s);
  case 4: return launch_decode_fp8_g4(f, s);
  case 8: return launch_decode_fp8_g8(f, s);
  default: return cudaErrorInvalidValue;
  }
}

} // namespace bia
