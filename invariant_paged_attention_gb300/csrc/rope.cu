// Norm and position rotation of query and key heads, to rows (bia_norm_rope)
// or on the way into the paged cache (bia_append_paged_kv_rope, bf16;
// bia_append_paged_kv_fp8_rope, the format of fp8.cuh):
//
//   y = x * w / sqrt(mean(x^2) + eps)     per head of D columns (w given)
//   (a, b) -> (a c - b s, b c + a s)      for the column pair of frequency f,
//                                         c, s = table[position(axis of f)]
//
// in fp32 from the loaded bf16 to the one rounding at the store (bf16, or
// codes: the 8-bit row is quantised from the fp32 values, not from their bf16
// rounding, so nothing is rounded twice).
//
// A head is a row of D/16 lanes, 16 columns a lane as two 16-byte pieces that
// hold both columns of each of its pairs: lane c has frequencies 8c .. 8c+7,
// columns 8c .. and rot/2 + 8c .. (halves) or 16c .. 16c+15 (interleaved); the
// lanes behind the rotating columns, and values, just 16 columns.  So a pair
// never crosses lanes, the norm is one shuffle sum, and a lane's eight (cos,
// sin) serve every head of its token.  A warp runs through the heads of one
// token (queries, keys, values) with kInFlight steps' loads under way; the
// token's slot and position are found meanwhile.  A call with few tokens
// splits a token's heads over several warps, down to a step a warp.
#include <algorithm>

#include "bia_internal.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace bia {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kInFlight = 4; // steps whose loads are issued together
enum RopeDest { kToRows, kToPages, kToPagesFp8 };

// 16 bytes that nobody else reads (also through q_out == q: a row is loaded
// and stored by the same lanes, so no .nc).
__device__ __forceinline__ uint4 ld_once(const uint16_t *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}
// (a, b) turned; explicit roundings, so that every destination has the same bits.
__device__ __forceinline__ void turn(float a, float b, float c, float s, float &x, float &y) {
  x = __fmaf_rn(a, c, -__fmul_rn(b, s));
  y = __fmaf_rn(b, c, __fmul_rn(a, s));
}
// Eight fp32 as codes under the scale 2^-e = inv; non-finite ones as NaN.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if ((__float_as_uint(x[i]) & 0x7fffffffu) >= 0x7f800000u) c[i >> 1] |= 0x7fu << (8 * (i & 1));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The request of a token: the largest b with indptr[b] <= token, by the whole
// warp, 32 probes a round.
__device__ __forceinline__ int find_request(const int32_t *indptr, int batch, int64_t token,
                                            int lane) {
  int lo = 0, n = batch; // it is one of lo .. lo+n-1
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool le = lane * step < n && __ldg(indptr + at) <= token;
    const int k = max(0, 31 - __clz(__ballot_sync(0xffffffffu, le))); // the last that is
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

template <int LPH, int DEST>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeArgs a, const int parts) {
  constexpr int HPS = 32 / LPH; // heads a step
  constexpr bool kPaged = DEST != kToRows;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, c = lane % LPH, hl = lane / LPH;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kRopeWarps + (threadIdx.x >> 5);
  const int64_t token = w / parts;
  if (token >= a.total) return;
  const int part = static_cast<int>(w - token * parts);
  const int D = a.D, half = a.rot >> 1;
  const bool in_row = c * 16 < D;
  const bool turns = c * 16 < a.rot;
  const int n_turned = a.Hq + a.Hk;               // q heads (0: none), then k heads
  const int heads = n_turned + (kPaged ? a.Hk : 0); // then v heads
  // the lane's two pieces of a head that rotates (or not), and of a value
  const int col0 = turns && !a.interleaved ? 8 * c : 16 * c;
  const int col1 = turns && !a.interleaved ? half + 8 * c : 16 * c + 8;

  auto source = [&](int h, int &at0, int &at1) -> const uint16_t * {
    at0 = h < n_turned ? col0 : 16 * c;
    at1 = h < n_turned ? col1 : 16 * c + 8;
    if (h < a.Hq) return a.q + token * a.q_stride + h * D;
    if (h < n_turned) return a.k + token * a.k_stride + (h - a.Hq) * D;
    return a.v + token * a.v_stride + (h - n_turned) * D;
  };

  int64_t slot = -1; // of the token in the cache
  float cs[8], sn[8];
  float wt[16];
  int wt_of = -1; // whose weights wt holds: 0 q, 1 k
  bool found = false;
  for (int s0 = part; s0 * HPS < heads; s0 += kInFlight * parts) {
    uint4 x[kInFlight][2];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int h = (s0 + i * parts) * HPS + hl;
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
      if (h < heads && in_row) {
        int at0, at1;
        const uint16_t *src = source(h, at0, at1);
        x[i][0] = ld_once(src + at0);
        x[i][1] = ld_once(src + at1);
      }
    }
    if (!found) { // while the first heads are on their way
      found = true;
      int32_t pos = 0;
      if constexpr (kPaged) {
        const int b = find_request(a.row_indptr, a.batch, token, lane);
        const int32_t first = __ldg(a.row_indptr + b), next = __ldg(a.row_indptr + b + 1);
        const int32_t p0 = __ldg(a.kv_indptr + b), p1 = __ldg(a.kv_indptr + b + 1);
        const int32_t kv_len =
            p1 > p0 ? ((p1 - p0 - 1) << a.page_shift) + __ldg(a.kv_last_page_len + b) : 0;
        pos = kv_len - (next - first) + static_cast<int32_t>(token - first);
        bool ok = pos >= 0 && pos < kv_len; // the host checks the row counts
        if (ok) {
          const int32_t page = __ldg(a.kv_indices + p0 + (pos >> a.page_shift));
          ok = page >= 0 && page < a.num_pages;
          if (ok)
            slot = (static_cast<int64_t>(page) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
        }
        if (!ok && lane == 0 && a.status) atomicOr(a.status, kStatusBadPage);
      }
      // the lane's (cos, sin); a position outside the table: NaN
#pragma unroll
      for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __int_as_float(0x7fc00000);
      for (int ax = 0; ax < a.axes; ++ax) {
        const int32_t p = a.positions ? __ldg(a.positions + ax * a.total + token) : pos;
        const bool ok = p >= 0 && p < a.num_positions;
        if (!ok) {
          if (lane == 0 && a.status) atomicOr(a.status, kStatusBadPosition);
          continue;
        }
        if (!turns) continue;
        // which of the lane's frequencies follow this axis (two bits each)
        uint32_t mine = 0;
        const uint32_t who = a.freq_axis[c >> 1] >> (16 * (c & 1));
#pragma unroll
        for (int i = 0; i < 8; ++i) mine |= static_cast<uint32_t>(((who >> (2 * i)) & 3u) == ax) << i;
        if (mine == 0) continue;
        const float4 *row =
            reinterpret_cast<const float4 *>(a.table + static_cast<int64_t>(p) * a.rot + 8 * c);
        const float4 *row_s = reinterpret_cast<const float4 *>(
            a.table + static_cast<int64_t>(p) * a.rot + half + 8 * c);
        const float4 t[4] = {__ldg(row), __ldg(row + 1), __ldg(row_s), __ldg(row_s + 1)};
        const float tc[8] = {t[0].x, t[0].y, t[0].z, t[0].w, t[1].x, t[1].y, t[1].z, t[1].w};
        const float ts[8] = {t[2].x, t[2].y, t[2].z, t[2].w, t[3].x, t[3].y, t[3].z, t[3].w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((mine >> i) & 1u) {
            cs[i] = tc[i];
            sn[i] = ts[i];
          }
      }
    }
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int h = (s0 + i * parts) * HPS + hl;
      const bool is_q = h < a.Hq, is_v = kPaged && h >= n_turned;
      if (is_v && DEST == kToPages) { // as they are
        if (h < heads && in_row && slot >= 0) {
          uint16_t *dst = a.v_cache + (slot * a.Hk + (h - n_turned)) * D + 16 * c;
          *reinterpret_cast<uint4 *>(dst) = x[i][0];
          *reinterpret_cast<uint4 *>(dst + 8) = x[i][1];
        }
      }
      float y0[8], y1[8];
      unpack8(x[i][0], y0);
      unpack8(x[i][1], y1);
      const float *weight = is_q ? a.q_weight : a.k_weight;
      if (a.q_weight || a.k_weight) { // uniform; the lanes of a head meet
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y0[e], y0[e], fmaf(y1[e], y1[e], ss));
#pragma unroll
        for (int off = LPH / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        if (!is_v && weight && in_row) {
          const int want = is_q ? 0 : 1;
          if (wt_of != want) { // once, and again where the keys begin
            wt_of = want;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
              const float4 u = __ldg(reinterpret_cast<const float4 *>(weight + col0 + e));
              const float4 v = __ldg(reinterpret_cast<const float4 *>(weight + col1 + e));
              wt[e] = u.x, wt[e + 1] = u.y, wt[e + 2] = u.z, wt[e + 3] = u.w;
              wt[8 + e] = v.x, wt[9 + e] = v.y, wt[10 + e] = v.z, wt[11 + e] = v.w;
            }
          }
          const float r = rsqrtf(__fmaf_rn(ss, a.inv_D, a.eps));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y0[e] = __fmul_rn(__fmul_rn(y0[e], r), wt[e]);
            y1[e] = __fmul_rn(__fmul_rn(y1[e], r), wt[8 + e]);
          }
        }
      }
      if (turns && !is_v) {
        if (a.interleaved) { // pairs inside each piece
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p0 = y0[2 * e], p1 = y0[2 * e + 1], q0 = y1[2 * e], q1 = y1[2 * e + 1];
            turn(p0, p1, cs[e], sn[e], y0[2 * e], y0[2 * e + 1]);
            turn(q0, q1, cs[4 + e], sn[4 + e], y1[2 * e], y1[2 * e + 1]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float p0 = y0[e], p1 = y1[e];
            turn(p0, p1, cs[e], sn[e], y0[e], y1[e]);
          }
        }
      }
      if constexpr (DEST == kToPagesFp8) {
        // the row's largest finite magnitude gives its scale
        uint32_t big = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t b0 = __float_as_uint(y0[e]) & 0x7fffffffu;
          const uint32_t b1 = __float_as_uint(y1[e]) & 0x7fffffffu;
          big = max(big, max(b0 < 0x7f800000u ? b0 : 0u, b1 < 0x7f800000u ? b1 : 0u));
        }
#pragma unroll
        for (int off = LPH / 2; off >= 1; off >>= 1)
          big = max(big, __shfl_xor_sync(0xffffffffu, big, off));
        if (!is_q && h < heads && in_row && slot >= 0) {
          const int e = row_exponent(__uint_as_float(big));
          const float inv = exp2_int(-e);
          const int64_t row = slot * a.Hk + (is_v ? h - n_turned : h - a.Hq);
          uint8_t *dst = (is_v ? a.v_codes : a.k_codes) + row * D;
          const uint2 r0 = codes8(y0, inv), r1 = codes8(y1, inv);
          if (is_v) {
            *reinterpret_cast<uint4 *>(dst + 16 * c) = make_uint4(r0.x, r0.y, r1.x, r1.y);
          } else {
            *reinterpret_cast<uint2 *>(dst + col0) = r0;
            *reinterpret_cast<uint2 *>(dst + col1) = r1;
          }
          if (c == 0) (is_v ? a.v_scale : a.k_scale)[row] = static_cast<uint8_t>(e + 127);
        }
      }
      if (h < n_turned && in_row) { // a bf16 row of q, or of k (rows, or the cache's)
        uint16_t *dst = nullptr;
        if (is_q) dst = a.q_out + token * a.q_out_stride + h * D;
        else if (DEST != kToPages)
          dst = a.k_out ? a.k_out + token * a.k_out_stride + (h - a.Hq) * D : nullptr;
        else if (slot >= 0)
          dst = a.k_cache + (slot * a.Hk + (h - a.Hq)) * D;
        if (dst) {
          *reinterpret_cast<uint4 *>(dst + col0) = pack8(y0);
          *reinterpret_cast<uint4 *>(dst + col1) = pack8(y1);
        }
      }
    }
  }
}

template <int LPH, int DEST>
cudaError_t launch_rope_ld(const RopeArgs &a, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const int heads = a.Hq + a.Hk + (DEST != kToRows ? a.Hk : 0);
  const int64_t steps = (heads + 32 / LPH - 1) / (32 / LPH);
  // warps a token: while the call has fewer than 8 warps an SM
  const int parts = static_cast<int>(std::clamp<int64_t>(8 * sms / a.total, 1, steps));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.total * parts + kRopeWarps - 1) / kRopeWarps));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<LPH, DEST>, a, parts);
}

template <int DEST>
cudaError_t launch_rope_d(const RopeArgs &a, cudaStream_t s) {
  if (a.D == 64) return launch_rope_ld<4, DEST>(a, s);
  return a.D <= 128 ? launch_rope_ld<8, DEST>(a, s) : launch_rope_ld<16, DEST>(a, s);
}

} // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t s) {
  if (a.total == 0 || a.Hq + a.Hk == 0) return cudaSuccess;
  if (a.k_codes) return launch_rope_d<kToPagesFp8>(a, s);
  return a.k_cache ? launch_rope_d<kToPages>(a, s) : launch_rope_d<kToRows>(a, s);
}

} // namespace bia
