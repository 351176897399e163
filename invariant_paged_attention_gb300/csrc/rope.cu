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
// hold both columns of each of its eight pairs: lane c has frequencies 8c ..
// 8c+7, columns 8c .. and rot/2 + 8c .. (halves) or 16c .. 16c+15
// (interleaved; with rot = D columns 8c .. and D/2 + 8c ..); the lanes behind the rotating columns, and values, just 16
// columns.  So a pair never crosses lanes, the norm is one shuffle sum, and a
// lane's factors (cos and sin times the weights of their columns) serve every
// head of its token; the arithmetic runs on fp32 pairs.  A warp runs through
// the heads of one token (queries, keys, values) with kRing steps' loads
// under way; the token's slot and position are found meanwhile.  A call with
// few tokens splits a token's heads over several warps, down to a step a warp.
//
// Bound by the copy rate and, close behind, by its instructions (three in four
// cycles issue one): 17868 tokens of 32/8 heads x 128 68 us (5.4 TB/s, 80 % of a
// plain copy), 44213 tokens into bf16 pages 186 us (5.85 TB/s, 86 %), into 8-bit
// pages 210 us (5.2 TB/s, 77 %; the scales' maxima and the codes come on top).
// 10693 tokens of 16/2 heads, half of the columns turning on three axes, take 27.5
// us (3.6 TB/s): a token waits for a position and then for its table row axis by
// axis, and has five steps to pay for it.
#include <algorithm>

#include "bia_internal.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace bia {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;
// Steps of a warp whose loads are under way (1 KB of shared memory each): with 4
// the four calls above take 70, 188, 214 and 30 us, with 8 (fewer CTAs an SM)
// 76, 203, 229 and 31.
constexpr int kRing = 2;
constexpr float kTinyVar = 0x1p-80f; // mean squares below it are taken again, scaled
enum RopeDest { kToRows, kToPages, kToPagesFp8 };

// The lane's sixteen columns as a[8], b[8]: pair f is (a[f], b[f]).
template <bool INTER>
__device__ __forceinline__ void unpack(const uint4 (&x)[2], float (&a)[8], float (&b)[8]) {
  const uint32_t u[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  if constexpr (INTER) {
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      a[f] = __uint_as_float(u[f] << 16);
      b[f] = __uint_as_float(u[f] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[2 * i] = __uint_as_float(u[i] << 16);
      a[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      b[2 * i] = __uint_as_float(u[4 + i] << 16);
      b[2 * i + 1] = __uint_as_float(u[4 + i] & 0xffff0000u);
    }
  }
}
template <bool INTER>
__device__ __forceinline__ void pack(const float (&a)[8], const float (&b)[8], uint4 (&x)[2]) {
  if constexpr (INTER) {
    x[0] = make_uint4(pack_bf16(a[0], b[0]), pack_bf16(a[1], b[1]), pack_bf16(a[2], b[2]),
                      pack_bf16(a[3], b[3]));
    x[1] = make_uint4(pack_bf16(a[4], b[4]), pack_bf16(a[5], b[5]), pack_bf16(a[6], b[6]),
                      pack_bf16(a[7], b[7]));
  } else {
    x[0] = make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]),
                      pack_bf16(a[6], a[7]));
    x[1] = make_uint4(pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3]), pack_bf16(b[4], b[5]),
                      pack_bf16(b[6], b[7]));
  }
}
// max(m, |x|, |y|); a NaN among them is kept.
__device__ __forceinline__ float max_abs(float m, float x, float y) {
  float r;
  asm("{\n\t.reg .f32 p, q;\n\tabs.f32 p, %2;\n\tabs.f32 q, %3;\n\t"
      "max.NaN.f32 %0, %1, p, q;\n\t}"
      : "=f"(r) : "f"(m), "f"(x), "f"(y));
  return r;
}
// Four fp32 times inv as four codes.
__device__ __forceinline__ uint32_t codes4(float x0, float x1, float x2, float x3, float inv) {
  return e4m3x2(x0 * inv, x1 * inv) | e4m3x2(x2 * inv, x3 * inv) << 16;
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

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

template <int LPH, int DEST, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 6)
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
  const bool in_row = c * 16 < D, turns = c * 16 < a.rot;
  // the lane's two pieces of a head that rotates (or not); of a value 16c, 16c +
  // 8.  Interleaved pairs of a whole row lie half a row apart too, four a piece
  // (44213 tokens into bf16 pages 191 us, with one run of eight pairs 224: two
  // copies touched each sector).
  const bool apart = turns && (!INTER || a.rot == D), split = INTER && apart;
  const int col0 = apart ? 8 * c : 16 * c, col1 = apart ? half + 8 * c : 16 * c + 8;
  const int freq0 = split ? 4 * c : 8 * c, freq1 = split ? half / 2 + 4 * c : 8 * c + 4;
  // steps: of queries, then of keys, then of values; a step is of one kind
  const int steps_q = (a.Hq + HPS - 1) / HPS, steps_k = (a.Hk + HPS - 1) / HPS;
  const int steps = steps_q + (kPaged ? 2 : 1) * steps_k;
  auto kind_of = [&](int s) { return s < steps_q ? 0 : s < steps_q + steps_k ? 1 : 2; };
  auto head_of = [&](int s, int kind) {
    return (s - (kind == 0 ? 0 : kind == 1 ? steps_q : steps_q + steps_k)) * HPS + hl;
  };

  // the token's rows at the lane's first head of a step
  const uint16_t *src[3] = {a.q + token * a.q_stride, a.k + token * a.k_stride,
                            kPaged ? a.v + token * a.v_stride : nullptr};
  uint16_t *q_dst = a.q_out + token * a.q_out_stride;
  uint16_t *k_dst = !a.k_out || DEST == kToPages ? nullptr : a.k_out + token * a.k_out_stride;

  // The lane copies its pieces of a step (and reads only those: no warp meets)
  // into a ring, so that what is under way holds no registers (four steps in
  // registers: 16 warps an SM, 76 us for 17868 tokens of 32/8 heads x 128).
  // Also with q_out == q: a row is loaded and stored by the same lanes.
  extern __shared__ uint4 ring[];
  uint4 *mine = ring + (threadIdx.x >> 5) * (kRing * 64) + lane; // step: 64 pieces
  int n_issued = 0;
  auto issue = [&](int s) {
    const int kind = kind_of(s), h = head_of(s, kind);
    const bool live = s < steps && h < (kind == 0 ? a.Hq : a.Hk) && in_row;
    const uint16_t *row = (kind == 0 ? src[0] : kind == 1 ? src[1] : src[2]) + (live ? h * D : 0);
    const uint32_t dst = smem_u32(mine + (n_issued % kRing) * 64);
    if (live) {
      cp_async16(dst, row + (kPaged && kind == 2 ? 16 * c : col0), true);
      cp_async16(dst + 512, row + (kPaged && kind == 2 ? 16 * c + 8 : col1), true);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++n_issued;
  };
#pragma unroll 1
  for (int i = 0; i < kRing; ++i) issue(part + i * parts);

  // while the first heads are on their way: the token's place
  int64_t slot = -1; // in the cache
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
    if (DEST == kToPages && ok) k_dst = a.k_cache + slot * a.Hk * D;
  }
  // factors of a and b: cos and sin, times the weights of the kind they hold;
  // from a position outside the table: NaN
  float ac[8], as[8], bc[8], bs[8];
  const float *have = nullptr; // whose weights
  bool found = false;
  auto factors = [&](const float *weight) {
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __int_as_float(0x7fc00000);
    for (int ax = 0; ax < a.axes; ++ax) {
      const int32_t p = a.positions ? __ldg(a.positions + ax * a.total + token) : pos;
      if (p < 0 || p >= a.num_positions) {
        if (lane == 0 && a.status) atomicOr(a.status, kStatusBadPosition);
        continue;
      }
      if (!turns) continue;
      // which of the lane's frequencies follow this axis (two bits each)
      const uint32_t who = (a.freq_axis[freq0 >> 4] >> (2 * (freq0 & 15)) & 0xffu) |
                           (a.freq_axis[freq1 >> 4] >> (2 * (freq1 & 15)) & 0xffu) << 8;
      const uint32_t off = who ^ (0x5555u * ax); // zero pairs follow it
      const float *row = a.table + static_cast<int64_t>(p) * a.rot;
      auto four = [&](int f) { return __ldg(reinterpret_cast<const float4 *>(row + f)); };
      const float4 t[4] = {four(freq0), four(freq1), four(half + freq0), four(half + freq1)};
      const float tc[8] = {t[0].x, t[0].y, t[0].z, t[0].w, t[1].x, t[1].y, t[1].z, t[1].w};
      const float ts[8] = {t[2].x, t[2].y, t[2].z, t[2].w, t[3].x, t[3].y, t[3].z, t[3].w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((off >> (2 * i) & 3u) == 0) {
          cs[i] = tc[i];
          sn[i] = ts[i];
        }
    }
    float wa[8], wb[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) wa[e] = wb[e] = 1.f;
    if (weight && in_row) {
      float v[16];
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 u0 = __ldg(reinterpret_cast<const float4 *>(weight + col0 + e));
        const float4 u1 = __ldg(reinterpret_cast<const float4 *>(weight + col1 + e));
        v[e] = u0.x, v[e + 1] = u0.y, v[e + 2] = u0.z, v[e + 3] = u0.w;
        v[8 + e] = u1.x, v[9 + e] = u1.y, v[10 + e] = u1.z, v[11 + e] = u1.w;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        wa[e] = INTER ? v[2 * e] : v[e];
        wb[e] = INTER ? v[2 * e + 1] : v[8 + e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ac[e] = turns ? wa[e] * cs[e] : wa[e];
      as[e] = wa[e] * sn[e];
      bc[e] = turns ? wb[e] * cs[e] : wb[e];
      bs[e] = -(wb[e] * sn[e]);
    }
  };
#pragma unroll 1
  for (int s = part, i = 0; s < steps; s += parts, ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    uint4 x[2] = {mine[(i % kRing) * 64], mine[(i % kRing) * 64 + 32]};
    const int kind = kind_of(s), h = head_of(s, kind); // the same kind on the warp
    const bool live = h < (kind == 0 ? a.Hq : a.Hk) && in_row;
    if (!live) x[0] = x[1] = make_uint4(0, 0, 0, 0);
    issue(s + kRing * parts);
    if (kind == 2 && DEST == kToPages) { // as they are
      if (live && slot >= 0) {
        uint16_t *dst = a.v_cache + slot * a.Hk * D + h * D + 16 * c;
        *reinterpret_cast<uint4 *>(dst) = x[0];
        *reinterpret_cast<uint4 *>(dst + 8) = x[1];
      }
      continue;
    }
    float ya[8], yb[8];
    if (INTER && kind == 2) unpack<false>(x, ya, yb);
    else unpack<INTER>(x, ya, yb);
    if (kind != 2) {
      const float *weight = kind == 0 ? a.q_weight : a.k_weight;
      if (!found || have != weight) { // once, and again where the keys begin
        found = true;
        have = weight;
        factors(weight);
      }
      float r = 1.f;
      if (weight) { // the lanes of a head meet
        uint64_t ss2 = 0;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          ffma2(ss2, f32x2(ya[e], ya[e + 1]), f32x2(ya[e], ya[e + 1]));
          ffma2(ss2, f32x2(yb[e], yb[e + 1]), f32x2(yb[e], yb[e + 1]));
        }
        float s_lo, s_hi;
        f32x2_split(ss2, s_lo, s_hi);
        float ss = s_lo + s_hi;
#pragma unroll
        for (int off = LPH / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        float var = __fmaf_rn(ss, a.inv_D, a.eps);
        if (a.eps < kTinyVar) { // uniform over the call
          // A head whose squares leave fp32 (with a larger eps they do not count) is
          // taken 2^90 times as large, exactly: its elements of 2^-133 to 2^-36 are
          // 2^-43 to 2^54 then.
          const bool tiny = var < kTinyVar;
          const float up = tiny ? 0x1p90f : 1.f;
          ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ya[e] *= up, yb[e] *= up;
            ss = __fmaf_rn(ya[e], ya[e], __fmaf_rn(yb[e], yb[e], ss));
          }
#pragma unroll
          for (int off = LPH / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          if (tiny) var = __fmaf_rn(ss, a.inv_D, a.eps * up * up);
        }
        r = rsqrtf(var);
      }
      // explicit roundings: every destination has the same bits
      const uint64_t r2 = f32x2(r, r);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const uint64_t a2 = f32x2(ya[e], ya[e + 1]), b2 = f32x2(yb[e], yb[e + 1]);
        uint64_t na = fmul2(a2, f32x2(ac[e], ac[e + 1]));
        uint64_t nb = fmul2(b2, f32x2(bc[e], bc[e + 1]));
        if (turns) {
          ffma2(na, b2, f32x2(bs[e], bs[e + 1]));
          ffma2(nb, a2, f32x2(as[e], as[e + 1]));
        }
        if (weight) {
          na = fmul2(na, r2);
          nb = fmul2(nb, r2);
        }
        f32x2_split(na, ya[e], ya[e + 1]);
        f32x2_split(nb, yb[e], yb[e + 1]);
      }
    }
    if (kind != 2 && live) { // a bf16 row of q, or of k (rows, or the cache's)
      uint16_t *dst = kind == 0 ? q_dst : k_dst;
      if (dst) {
        uint4 o[2];
        pack<INTER>(ya, yb, o);
        *reinterpret_cast<uint4 *>(dst + h * D + col0) = o[0];
        *reinterpret_cast<uint4 *>(dst + h * D + col1) = o[1];
      }
    }
    if (DEST == kToPagesFp8 && kind != 0) {
      // the row's largest finite magnitude gives its scale
      float big = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) big = max_abs(big, ya[e], yb[e]);
      const bool odd = !finite(big); // an infinity or NaN among them: rare
      if (odd) {
        big = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          big = fmaxf(big, fmaxf(finite(ya[e]) ? fabsf(ya[e]) : 0.f,
                                 finite(yb[e]) ? fabsf(yb[e]) : 0.f));
      }
#pragma unroll
      for (int off = LPH / 2; off >= 1; off >>= 1)
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
      if (live && slot >= 0) {
        const int ex = row_exponent(big);
        const float inv = exp2_int(-ex);
        if (odd) { // stored as NaN (the conversion keeps NaN, but not infinities)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (!finite(ya[e])) ya[e] = __int_as_float(0x7fc00000);
            if (!finite(yb[e])) yb[e] = __int_as_float(0x7fc00000);
          }
        }
        const int64_t row = slot * a.Hk + h;
        uint8_t *dst = (kind == 2 ? a.v_codes : a.k_codes) + row * D;
        uint2 r0, r1;
        if (INTER && kind != 2) {
          r0 = make_uint2(codes4(ya[0], yb[0], ya[1], yb[1], inv),
                          codes4(ya[2], yb[2], ya[3], yb[3], inv));
          r1 = make_uint2(codes4(ya[4], yb[4], ya[5], yb[5], inv),
                          codes4(ya[6], yb[6], ya[7], yb[7], inv));
        } else {
          r0 = make_uint2(codes4(ya[0], ya[1], ya[2], ya[3], inv),
                          codes4(ya[4], ya[5], ya[6], ya[7], inv));
          r1 = make_uint2(codes4(yb[0], yb[1], yb[2], yb[3], inv),
                          codes4(yb[4], yb[5], yb[6], yb[7], inv));
        }
        if (kind == 2) {
          *reinterpret_cast<uint4 *>(dst + 16 * c) = make_uint4(r0.x, r0.y, r1.x, r1.y);
        } else {
          *reinterpret_cast<uint2 *>(dst + col0) = r0;
          *reinterpret_cast<uint2 *>(dst + col1) = r1;
        }
        if (c == 0) (kind == 2 ? a.v_scale : a.k_scale)[row] = static_cast<uint8_t>(ex + 127);
      }
    }
  }
  cp_async_wait_all(); // no copy outlives the CTA
}

template <int LPH, int DEST, bool INTER>
cudaError_t launch_rope_ldi(const RopeArgs &a, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const int hps = 32 / LPH;
  const int64_t steps =
      (a.Hq + hps - 1) / hps + (DEST != kToRows ? 2 : 1) * ((a.Hk + hps - 1) / hps);
  // warps a token: while the call has fewer than 8 warps an SM
  const int parts = static_cast<int>(std::clamp<int64_t>(8 * sms / a.total, 1, steps));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.total * parts + kRopeWarps - 1) / kRopeWarps));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.dynamicSmemBytes = kRopeWarps * kRing * 1024;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<LPH, DEST, INTER>, a, parts);
}

template <int LPH, int DEST>
cudaError_t launch_rope_ld(const RopeArgs &a, cudaStream_t s) {
  return a.interleaved ? launch_rope_ldi<LPH, DEST, true>(a, s)
                       : launch_rope_ldi<LPH, DEST, false>(a, s);
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
