// The 8-bit paged cache (fp8.cuh states the format): append quantises new
// tokens' key and value rows into their pages, gather reads rows back as
// bf16, packed one request after the other.
//
// A row is one (token, kv head) of K or of V; LPR lanes (a power of two) take
// one row, 16 elements a lane: two 16-byte loads, the lanes' largest
// magnitudes meet in log2(LPR) shuffles, one 16-byte store of codes (gather:
// the reverse).  A warp takes up to 32 consecutive tokens: each lane finds the
// cache slot of one (its request by a search over the lanes' copy of the index
// arrays, then one load of its page), and the warp runs through their rows,
// the K heads and then the V heads of each token, two steps' loads in flight.
// Nothing is read or written twice: 2*D bytes in and D + 1 out per row, HBM
// bound.  44213 tokens of 8 heads x 128 (272 MB, 40 us at the copy rate): 45
// us for the append, 47 for the gather.  With a group of lanes per row, each
// finding its slot by binary search and 64-bit divisions, the index work bound
// them: 123 and 94 us; with a warp a token, a slot's three dependent loads did
// where tokens are short: 29 us for the append of one 64-wide head (17 MB),
// 11 now.
#include <algorithm>

#include "bia_internal.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace bia {

namespace {

constexpr int kCacheThreads = 256;
constexpr int kInFlight = 2; // steps whose loads are issued together
constexpr int kRounds = 2;   // of such loads a warp

// Flat cache slot (page * page_size + offset) of row `token` of the call, each
// lane its own, or -1 when its page is out of range (status bit 0).  append:
// the request's rows are the last of its keys; gather: the first.  The whole
// warp calls it; lanes without a token pass live = false.
template <bool APPEND>
__device__ __forceinline__ int64_t token_slot(const CacheFp8Args &a, int64_t token, bool live,
                                              int lane) {
  int b = 0; // largest b with row_indptr[b] <= token
  int32_t first, next, p0, p1, last;
  if (a.batch <= 32) { // lane i holds request i
    const int r = min(lane, a.batch - 1);
    const int32_t rf = __ldg(a.row_indptr + r), rn = __ldg(a.row_indptr + r + 1);
    const int32_t k0 = __ldg(a.kv_indptr + r), k1 = __ldg(a.kv_indptr + r + 1);
    const int32_t kl = __ldg(a.kv_last_page_len + r);
#pragma unroll
    for (int s = 16; s >= 1; s /= 2) {
      const int32_t v = __shfl_sync(0xffffffffu, rf, (b + s) & 31);
      if (b + s < a.batch && v <= token) b += s;
    }
    first = __shfl_sync(0xffffffffu, rf, b);
    next = __shfl_sync(0xffffffffu, rn, b);
    p0 = __shfl_sync(0xffffffffu, k0, b);
    p1 = __shfl_sync(0xffffffffu, k1, b);
    last = __shfl_sync(0xffffffffu, kl, b);
  } else {
    int hi = a.batch - 1;
    while (b < hi) {
      const int mid = (b + hi + 1) >> 1;
      if (__ldg(a.row_indptr + mid) <= token) b = mid;
      else hi = mid - 1;
    }
    first = __ldg(a.row_indptr + b);
    next = __ldg(a.row_indptr + b + 1);
    p0 = __ldg(a.kv_indptr + b);
    p1 = __ldg(a.kv_indptr + b + 1);
    last = __ldg(a.kv_last_page_len + b);
  }
  if (!live) return -1;
  const int32_t kv_len = p1 > p0 ? ((p1 - p0 - 1) << a.page_shift) + last : 0;
  const int32_t pos = static_cast<int32_t>(token - first) + (APPEND ? kv_len - (next - first) : 0);
  if (pos >= 0 && pos < kv_len) { // the host checks the row counts
    const int32_t page = __ldg(a.kv_indices + p0 + (pos >> a.page_shift));
    if (page >= 0 && page < a.num_pages)
      return (static_cast<int64_t>(page) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
  }
  if (a.status) atomicOr(a.status, kStatusBadPage);
  return -1;
}

// The row a lane is at: token t of the warp's, row r of it (K heads, then V
// heads); advanced by the rows of a step.
struct RowAt {
  int t, r;
  __device__ __forceinline__ RowAt(int start, int rows) : t(start / rows), r(start - t * rows) {}
  __device__ __forceinline__ void step(int by, int rows) {
    r += by;
    while (r >= rows) {
      r -= rows;
      ++t;
    }
  }
};

// 16 elements of a row as codes; inv: 2^-e of the row.
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
__global__ void __launch_bounds__(kCacheThreads, 6) append_fp8_kernel(const CacheFp8Args a, int per) {
  constexpr int RPS = 32 / LPR; // rows a step
  const int lane = threadIdx.x & 31, c = lane % LPR, rl = lane / LPR;
  const bool in_row = c * 16 < a.D;
  const int rows = 2 * a.Hkv;
  const int64_t token0 =
      (static_cast<int64_t>(blockIdx.x) * (kCacheThreads / 32) + (threadIdx.x >> 5)) * per;
  const int n = static_cast<int>(min(static_cast<int64_t>(per), a.total - token0));
  if (n <= 0) return;
  int64_t slot_l = 0; // of token token0 + lane
  RowAt at(rl, rows);
  for (int q0 = 0; q0 < n * rows; q0 += kInFlight * RPS) {
    uint4 x[kInFlight][2];
    RowAt ahead = at;
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
      if (ahead.t < n && in_row) {
        const bool is_v = ahead.r >= a.Hkv;
        const int h = is_v ? ahead.r - a.Hkv : ahead.r;
        const int64_t token = token0 + ahead.t;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            static_cast<const uint16_t *>(is_v ? a.v_rows : a.k_rows) +
            token * (is_v ? a.v_stride : a.k_stride) + h * a.D + c * 16);
        x[i][0] = __ldg(src);
        x[i][1] = __ldg(src + 1);
      }
      ahead.step(RPS, rows);
    }
    // found while the first rows are on their way
    if (q0 == 0) slot_l = token_slot<true>(a, token0 + lane, lane < n, lane);
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
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
      const int64_t slot = __shfl_sync(0xffffffffu, slot_l, at.t & 31);
      if (at.t < n && in_row && slot >= 0) {
        const bool is_v = at.r >= a.Hkv;
        const int64_t dst = slot * a.Hkv + (is_v ? at.r - a.Hkv : at.r);
        *reinterpret_cast<uint4 *>((is_v ? a.v_codes : a.k_codes) + dst * a.D + c * 16) = codes;
        if (c == 0) (is_v ? a.v_scale : a.k_scale)[dst] = static_cast<uint8_t>(e + 127);
      }
      at.step(RPS, rows);
    }
  }
}

template <int LPR>
__global__ void __launch_bounds__(kCacheThreads, 8) gather_fp8_kernel(const CacheFp8Args a, int per) {
  constexpr int RPS = 32 / LPR; // rows a step
  const int lane = threadIdx.x & 31, c = lane % LPR, rl = lane / LPR;
  const bool in_row = c * 16 < a.D;
  const int rows = 2 * a.Hkv;
  const int64_t token0 =
      (static_cast<int64_t>(blockIdx.x) * (kCacheThreads / 32) + (threadIdx.x >> 5)) * per;
  const int n = static_cast<int>(min(static_cast<int64_t>(per), a.total - token0));
  if (n <= 0) return;
  const int64_t slot_l = token_slot<false>(a, token0 + lane, lane < n, lane);
  RowAt at(rl, rows);
  for (int q0 = 0; q0 < n * rows; q0 += kInFlight * RPS) {
    uint4 x[kInFlight];
    uint32_t sb[kInFlight];
    RowAt ahead = at;
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      x[i] = make_uint4(0, 0, 0, 0); // a bad page reads as zeros
      sb[i] = 127;
      const int64_t slot = __shfl_sync(0xffffffffu, slot_l, ahead.t & 31);
      if (ahead.t < n && in_row && slot >= 0) {
        const bool is_v = ahead.r >= a.Hkv;
        const int64_t src = slot * a.Hkv + (is_v ? ahead.r - a.Hkv : ahead.r);
        x[i] = __ldg(reinterpret_cast<const uint4 *>((is_v ? a.v_codes : a.k_codes) + src * a.D +
                                                     c * 16));
        sb[i] = __ldg((is_v ? a.v_scale : a.k_scale) + src);
      }
      ahead.step(RPS, rows);
    }
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      if (at.t < n && in_row) {
        const bool is_v = at.r >= a.Hkv;
        const float scale = e8m0_value(sb[i]);
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float lo, hi;
          e4m3x2_values((w[e >> 1] >> (16 * (e & 1))) & 0xffffu, lo, hi);
          o[e] = pack_bf16(lo * scale, hi * scale);
        }
        uint4 *dst = reinterpret_cast<uint4 *>(
            static_cast<uint16_t *>(is_v ? a.v_out : a.k_out) +
            ((token0 + at.t) * a.Hkv + (is_v ? at.r - a.Hkv : at.r)) * a.D + c * 16);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
      at.step(RPS, rows);
    }
  }
}

template <int LPR>
cudaError_t launch_tokens(const CacheFp8Args &a, bool append, cudaStream_t s) {
  // Tokens a warp: kRounds rounds of loads, as far as the call still has a
  // warp for each of the SMs' schedulers; one for small calls, where latency
  // counts.
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const int64_t round = std::max<int64_t>(1, kRounds * kInFlight * (32 / LPR) / (2 * a.Hkv));
  const int per = static_cast<int>(
      std::clamp<int64_t>(std::min<int64_t>(round, a.total / (8 * sms)), 1, 32));
  const int64_t block = static_cast<int64_t>(per) * (kCacheThreads / 32);
  const unsigned g = static_cast<unsigned>((a.total + block - 1) / block); // below 2^31 / 16 rows
  if (append)
    append_fp8_kernel<LPR><<<g, kCacheThreads, 0, s>>>(a, per);
  else
    gather_fp8_kernel<LPR><<<g, kCacheThreads, 0, s>>>(a, per);
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
