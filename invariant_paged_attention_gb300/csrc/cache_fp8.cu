// The 8-bit paged cache (fp8.cuh states the format): append quantises new
// tokens' key and value rows into their pages, gather reads rows back as
// bf16, packed one request after the other.
//
// A row is one (token, kv head) of K or of V; a group of LPR lanes (a power
// of two, 8 elements a lane) takes one row.  append: the lanes' largest
// magnitudes meet in log2(LPR) shuffles, then every lane scales and rounds
// its 8 elements.  Nothing is read or written twice: 2*D bytes in and D + 1
// out per row (gather: the reverse), HBM bound.
#include "bia_internal.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace bia {

namespace {

constexpr int kCacheThreads = 256;

// Largest b with indptr[b] <= t.
__device__ __forceinline__ int row_owner(const int32_t *indptr, int batch, int64_t t) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (indptr[mid] <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Flat cache slot of row `token` of the call (page * page_size + offset), or
// -1 when its page is out of range (status bit 0).  append: the request's
// rows are the last of its keys; gather: the first.
template <bool APPEND>
__device__ __forceinline__ int64_t token_slot(const CacheFp8Args &a, int64_t token) {
  const int b = row_owner(a.row_indptr, a.batch, token);
  const int32_t first = a.row_indptr[b], n = a.row_indptr[b + 1] - first;
  const int32_t p0 = a.kv_indptr[b], pages = a.kv_indptr[b + 1] - p0;
  const int32_t kv_len = pages > 0 ? (pages - 1) * a.page_size + a.kv_last_page_len[b] : 0;
  const int32_t pos = static_cast<int32_t>(token - first) + (APPEND ? kv_len - n : 0);
  if (pos >= 0 && pos < kv_len) { // the host checks n <= kv_len
    const int32_t page = a.kv_indices[p0 + pos / a.page_size];
    if (page >= 0 && page < a.num_pages)
      return static_cast<int64_t>(page) * a.page_size + pos % a.page_size;
  }
  if (a.status) atomicOr(a.status, kStatusBadPage);
  return -1;
}

template <int LPR>
__global__ void __launch_bounds__(kCacheThreads) append_fp8_kernel(const CacheFp8Args a) {
  const int lane = threadIdx.x % LPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kCacheThreads / LPR) + threadIdx.x / LPR;
  const int64_t rows = a.total * a.Hkv * 2;
  // the K rows of every token's heads, then its V rows
  const bool live = row < rows;
  const int64_t token = live ? row / (2 * a.Hkv) : 0;
  const int h2 = static_cast<int>((live ? row : 0) - token * (2 * a.Hkv));
  const bool is_v = h2 >= a.Hkv;
  const int h = is_v ? h2 - a.Hkv : h2;
  const int64_t slot = live ? token_slot<true>(a, token) : -1;
  const bool mine = slot >= 0 && lane * 8 < a.D;
  const uint16_t *src = is_v ? static_cast<const uint16_t *>(a.v_rows) + token * a.v_stride
                             : static_cast<const uint16_t *>(a.k_rows) + token * a.k_stride;
  uint32_t w[4] = {0, 0, 0, 0};
  if (mine) {
    const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src + h * a.D + lane * 8));
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
  }
  uint32_t big = 0; // largest finite |x|, as bf16 bits
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
    big = max(big, max(lo < kBf16Inf ? lo : 0u, hi < kBf16Inf ? hi : 0u));
  }
#pragma unroll
  for (int off = LPR / 2; off >= 1; off >>= 1)
    big = max(big, __shfl_xor_sync(0xffffffffu, big, off));
  const int e = row_exponent(__uint_as_float(big << 16));
  if (!mine) return;
  const float inv = exp2_int(-e);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // an infinity is stored as NaN, like NaN itself
    const uint32_t lo = w[i] & 0xffffu, hi = w[i] >> 16;
    const float xl = (lo & 0x7fffu) < kBf16Inf ? __uint_as_float(lo << 16) * inv : NAN;
    const float xh = (hi & 0x7fffu) < kBf16Inf ? __uint_as_float(hi << 16) * inv : NAN;
    c[i] = e4m3x2(xl, xh);
  }
  const int64_t dst = slot * a.Hkv + h;
  uint8_t *codes = is_v ? a.v_codes : a.k_codes;
  *reinterpret_cast<uint2 *>(codes + dst * a.D + lane * 8) =
      make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  if (lane == 0) (is_v ? a.v_scale : a.k_scale)[dst] = static_cast<uint8_t>(e + 127);
}

template <int LPR>
__global__ void __launch_bounds__(kCacheThreads) gather_fp8_kernel(const CacheFp8Args a) {
  const int lane = threadIdx.x % LPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kCacheThreads / LPR) + threadIdx.x / LPR;
  if (row >= a.total * a.Hkv * 2 || lane * 8 >= a.D) return;
  const int64_t token = row / (2 * a.Hkv);
  const int h2 = static_cast<int>(row - token * (2 * a.Hkv));
  const bool is_v = h2 >= a.Hkv;
  const int h = is_v ? h2 - a.Hkv : h2;
  const int64_t slot = token_slot<false>(a, token);
  uint4 out = make_uint4(0, 0, 0, 0); // a bad page reads as zeros
  if (slot >= 0) {
    const int64_t at = slot * a.Hkv + h;
    const uint2 x = __ldg(reinterpret_cast<const uint2 *>((is_v ? a.v_codes : a.k_codes) +
                                                          at * a.D + lane * 8));
    const float scale = e8m0_value(__ldg((is_v ? a.v_scale : a.k_scale) + at));
    float f[8];
    e4m3x2_values(x.x & 0xffffu, f[0], f[1]);
    e4m3x2_values(x.x >> 16, f[2], f[3]);
    e4m3x2_values(x.y & 0xffffu, f[4], f[5]);
    e4m3x2_values(x.y >> 16, f[6], f[7]);
    out.x = pack_bf16(f[0] * scale, f[1] * scale);
    out.y = pack_bf16(f[2] * scale, f[3] * scale);
    out.z = pack_bf16(f[4] * scale, f[5] * scale);
    out.w = pack_bf16(f[6] * scale, f[7] * scale);
  }
  uint16_t *dst = static_cast<uint16_t *>(is_v ? a.v_out : a.k_out);
  *reinterpret_cast<uint4 *>(dst + (token * a.Hkv + h) * a.D + lane * 8) = out;
}

template <int LPR>
cudaError_t launch_rows(const CacheFp8Args &a, bool append, cudaStream_t s) {
  const int64_t rows = a.total * a.Hkv * 2;
  const int per = kCacheThreads / LPR;
  const int64_t grid = (rows + per - 1) / per;
  if (grid > INT32_MAX) return cudaErrorInvalidValue; // refused on the host before
  if (append)
    append_fp8_kernel<LPR><<<static_cast<unsigned>(grid), kCacheThreads, 0, s>>>(a);
  else
    gather_fp8_kernel<LPR><<<static_cast<unsigned>(grid), kCacheThreads, 0, s>>>(a);
  return cudaGetLastError();
}

} // namespace

cudaError_t launch_cache_fp8(const CacheFp8Args &a, bool append, cudaStream_t s) {
  if (a.total == 0) return cudaSuccess;
  if (a.D == 64) return launch_rows<8>(a, append, s);
  if (a.D <= 128) return launch_rows<16>(a, append, s);
  return launch_rows<32>(a, append, s);
}

} // namespace bia
