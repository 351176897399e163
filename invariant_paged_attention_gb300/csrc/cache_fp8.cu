// The 8-bit paged cache (fp8.cuh states the format): append quantises new
// tokens' key and value rows into their pages, gather reads rows back as
// bf16, packed one request after the other.
//
// A row is one (token, kv head) of K or of V; LPR lanes (a power of two) take
// one row, 16 elements a lane: two 16-byte loads, the lanes' largest
// magnitudes meet in log2(LPR) shuffles, one 16-byte store of codes (gather:
// the reverse).  A warp takes a token at a time, its K rows and then its V
// rows, four steps' loads in flight; it finds the token's request with 32
// probes at once and its page by one more load, and for append the first rows
// are already on their way by then.  Nothing is read or written twice: 2*D
// bytes in and D + 1 out per row, HBM bound.  (With a group of lanes per row,
// each finding its slot by binary search and 64-bit divisions, the index work
// bound it: 123 us where the bytes take 40, for 44213 tokens of 8 heads x 128.)
#include <algorithm>

#include "bia_internal.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace bia {

namespace {

constexpr int kCacheThreads = 256;
constexpr int kInFlight = 4; // steps whose loads are issued together

// Largest b with indptr[b] <= t, on every lane: 32 probes a step.
__device__ __forceinline__ int warp_owner(const int32_t *indptr, int batch, int64_t t, int lane) {
  int lo = 0, n = batch;
  while (true) {
    const int step = (n + 31) / 32;
    const int b = lo + lane * step;
    const bool below = lane * step < n && __ldg(indptr + b) <= t; // lane 0 always
    lo += (__popc(__ballot_sync(0xffffffffu, below)) - 1) * step;
    if (step == 1) return lo;
    n = min(step, batch - lo);
  }
}

// Flat cache slot of row `token` of the call (page * page_size + offset), or
// -1 when its page is out of range (status bit 0).  append: the request's
// rows are the last of its keys; gather: the first.
template <bool APPEND>
__device__ __forceinline__ int64_t token_slot(const CacheFp8Args &a, int64_t token, int lane) {
  const int b = warp_owner(a.row_indptr, a.batch, token, lane);
  const int32_t first = __ldg(a.row_indptr + b), next = __ldg(a.row_indptr + b + 1);
  const int32_t p0 = __ldg(a.kv_indptr + b), p1 = __ldg(a.kv_indptr + b + 1);
  const int32_t last = __ldg(a.kv_last_page_len + b);
  const int32_t kv_len = p1 > p0 ? ((p1 - p0 - 1) << a.page_shift) + last : 0;
  const int32_t pos = static_cast<int32_t>(token - first) + (APPEND ? kv_len - (next - first) : 0);
  if (pos >= 0 && pos < kv_len) { // the host checks the row counts
    const int32_t page = __ldg(a.kv_indices + p0 + (pos >> a.page_shift));
    if (page >= 0 && page < a.num_pages)
      return (static_cast<int64_t>(page) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
  }
  if (a.status && lane == 0) atomicOr(a.status, kStatusBadPage);
  return -1;
}

// Row r of a token (K heads, then V heads): its head, and whether it is V.
struct RowOf {
  bool is_v;
  int h;
  __device__ __forceinline__ RowOf(int r, int Hkv) : is_v(r >= Hkv), h(r >= Hkv ? r - Hkv : r) {}
};

// 16 elements of a row quantised; big: the row's largest |x| bits.
__device__ __forceinline__ uint4 quantise16(const uint4 (&x)[2], float inv) {
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i] = e4m3x2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv);
  return make_uint4(c[0] | (c[1] << 16), c[2] | (c[3] << 16), c[4] | (c[5] << 16),
                    c[6] | (c[7] << 16));
}

template <int LPR>
__global__ void __launch_bounds__(kCacheThreads) append_fp8_kernel(const CacheFp8Args a) {
  constexpr int RPS = 32 / LPR; // rows a step
  const int lane = threadIdx.x & 31, c = lane % LPR, rl = lane / LPR;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kCacheThreads / 32);
  const bool in_row = c * 16 < a.D;
  const int rows = 2 * a.Hkv;
  for (int64_t token = static_cast<int64_t>(blockIdx.x) * (kCacheThreads / 32) + (threadIdx.x >> 5);
       token < a.total; token += warps) {
    const uint16_t *k = static_cast<const uint16_t *>(a.k_rows) + token * a.k_stride + c * 16;
    const uint16_t *v = static_cast<const uint16_t *>(a.v_rows) + token * a.v_stride + c * 16;
    int64_t slot = 0;
    for (int r0 = 0; r0 < rows; r0 += kInFlight * RPS) {
      uint4 x[kInFlight][2];
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int r = r0 + i * RPS + rl;
        x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
        if (r < rows && in_row) {
          const RowOf row(r, a.Hkv);
          const uint4 *src = reinterpret_cast<const uint4 *>((row.is_v ? v : k) + row.h * a.D);
          x[i][0] = __ldg(src);
          x[i][1] = __ldg(src + 1);
        }
      }
      if (r0 == 0) slot = token_slot<true>(a, token, lane);
      if (slot < 0) break;
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int r = r0 + i * RPS + rl;
        const uint32_t w[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w,
                               x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
        uint32_t m2 = 0; // largest |x| bits of the low and of the high halves
#pragma unroll
        for (int e = 0; e < 8; ++e) m2 = __vmaxu2(m2, w[e] & 0x7fff7fffu);
        uint32_t big = max(m2 & 0xffffu, m2 >> 16);
        const bool odd = big >= kBf16Inf; // an infinity or NaN among them: rare
        if (odd) {                        // the largest finite one
          big = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
            big = max(big, max(lo < kBf16Inf ? lo : 0u, hi < kBf16Inf ? hi : 0u));
          }
        }
#pragma unroll
        for (int off = LPR / 2; off >= 1; off >>= 1)
          big = max(big, __shfl_xor_sync(0xffffffffu, big, off));
        const int e = row_exponent(__uint_as_float(big << 16));
        uint4 codes = quantise16(x[i], exp2_int(-e));
        if (odd) { // stored as NaN (the conversion keeps NaN, but not infinities)
          uint32_t q[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            if ((w[n] & 0x7fffu) >= kBf16Inf) q[n >> 1] |= 0x7fu << (16 * (n & 1));
            if (((w[n] >> 16) & 0x7fffu) >= kBf16Inf) q[n >> 1] |= 0x7f00u << (16 * (n & 1));
          }
          codes = make_uint4(q[0], q[1], q[2], q[3]);
        }
        if (r < rows && in_row) {
          const RowOf row(r, a.Hkv);
          const int64_t dst = slot * a.Hkv + row.h;
          *reinterpret_cast<uint4 *>((row.is_v ? a.v_codes : a.k_codes) + dst * a.D + c * 16) = codes;
          if (c == 0) (row.is_v ? a.v_scale : a.k_scale)[dst] = static_cast<uint8_t>(e + 127);
        }
      }
    }
  }
}

template <int LPR>
__global__ void __launch_bounds__(kCacheThreads) gather_fp8_kernel(const CacheFp8Args a) {
  constexpr int RPS = 32 / LPR; // rows a step
  const int lane = threadIdx.x & 31, c = lane % LPR, rl = lane / LPR;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kCacheThreads / 32);
  const bool in_row = c * 16 < a.D;
  const int rows = 2 * a.Hkv;
  for (int64_t token = static_cast<int64_t>(blockIdx.x) * (kCacheThreads / 32) + (threadIdx.x >> 5);
       token < a.total; token += warps) {
    const int64_t slot = token_slot<false>(a, token, lane);
    for (int r0 = 0; r0 < rows; r0 += kInFlight * RPS) {
      uint4 x[kInFlight];
      uint32_t sb[kInFlight];
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int r = r0 + i * RPS + rl;
        x[i] = make_uint4(0, 0, 0, 0); // a bad page reads as zeros
        sb[i] = 127;
        if (slot >= 0 && r < rows && in_row) {
          const RowOf row(r, a.Hkv);
          const int64_t at = slot * a.Hkv + row.h;
          x[i] = __ldg(reinterpret_cast<const uint4 *>((row.is_v ? a.v_codes : a.k_codes) +
                                                       at * a.D + c * 16));
          sb[i] = __ldg((row.is_v ? a.v_scale : a.k_scale) + at);
        }
      }
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int r = r0 + i * RPS + rl;
        if (r >= rows || !in_row) continue;
        const RowOf row(r, a.Hkv);
        const float scale = e8m0_value(sb[i]);
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t o[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          float lo, hi;
          e4m3x2_values((w[n >> 1] >> (16 * (n & 1))) & 0xffffu, lo, hi);
          o[n] = pack_bf16(lo * scale, hi * scale);
        }
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(row.is_v ? a.v_out : a.k_out) +
                                               (token * a.Hkv + row.h) * a.D + c * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

template <int LPR>
cudaError_t launch_tokens(const CacheFp8Args &a, bool append, cudaStream_t s) {
  const int64_t grid = (a.total + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
  const unsigned g = static_cast<unsigned>(std::min<int64_t>(grid, 1 << 20));
  if (append)
    append_fp8_kernel<LPR><<<g, kCacheThreads, 0, s>>>(a);
  else
    gather_fp8_kernel<LPR><<<g, kCacheThreads, 0, s>>>(a);
  return cudaGetLastError();
}

} // namespace

cudaError_t launch_cache_fp8(const CacheFp8Args &a, bool append, cudaStream_t s) {
  if (a.total == 0) return cudaSuccess;
  if (a.D == 64) return launch_tokens<4>(a, append, s);
  if (a.D <= 128) return launch_tokens<8>(a, append, s);
  return launch_tokens<16>(a, append, s);
}

} // namespace bia
