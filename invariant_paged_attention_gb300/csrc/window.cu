// Joins what the split tiles of an attention with a window and sinks left: the
// states of a row, in order (fold.cuh), and the status words of the CTAs.
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
  const int n = (k.len + a.split - 1) / a.split;
  if (n <= 1) return; // stored by its only tile, or NaN
  const int64_t first = static_cast<int64_t>(b) * a.parts * a.Hq + h;
  const float *po = a.part_o + first * a.D, *pl = a.part_lse + first;
  uint16_t *out = a.out + row * a.D;
  float *lse = a.lse ? a.lse + row : nullptr;
  if (a.D <= 128) fold_row<4>(po, pl, n, a.Hq, a.D, lane, out, lse);
  else fold_row<8>(po, pl, n, a.Hq, a.D, lane, out, lse);
}

} // namespace

cudaError_t launch_merge_window_decode(const AttnArgs &a, int n_slots, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  // without a second tile there are only the status words
  const int64_t rows = a.parts > 1 ? static_cast<int64_t>(a.batch) * a.Hq : 1;
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_window_decode_kernel, a, n_slots);
}

} // namespace bia
