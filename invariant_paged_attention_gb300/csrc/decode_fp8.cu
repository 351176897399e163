// Split-KV decode of one query token per request over the 8-bit paged cache
// (fp8.cuh states the format), with the fixed split-KV tiles and ascending
// merge of the bf16 decode ("sglang PR #10417 [POC] Support deterministic
// inference", Modifications):
//   s_j = sm_scale * 2^ek_j * <q, ck_j>,   o = sum_j softmax(s)_j 2^ev_j cv_j
//
// One CTA per (request, split tile, kv head).  Warp w takes keys w, w + 8,
// ... of the split; its lanes hold D/32 dims of each of the G query heads and
// of their running O, a score is a butterfly over the warp, and every lane
// keeps the same running max and sum.  The warps' states are folded in index
// order at the end.
#include "bia_internal.h"
#include "fold.cuh"
#include "fp8.cuh"
#include "ptx.cuh"

namespace bia {

namespace {

constexpr int kWarpsF8 = 8;

template <int VPT, int G>
__global__ void __launch_bounds__(kWarpsF8 * 32) decode_fp8_kernel(const DecodeFp8Args f) {
  const AttnArgs &a = f.a;
  constexpr int D = VPT * 32;
  __shared__ float s_l[kWarpsF8][G];
  extern __shared__ float s_o[]; // [warp][G][D]
  grid_dep_wait();
  grid_dep_launch();
  const int64_t unit = blockIdx.x / a.Hkv;
  const int kvh = static_cast<int>(blockIdx.x - unit * a.Hkv);
  const Unit u = a.units[unit];
  if (u.b < 0) return;
  const ReqInfo r = a.reqs[u.b];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t key_begin = u.split * a.split, key_end = min(key_begin + a.split, r.kv_len);
  float q[G][VPT], o[G][VPT], m[G], l[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const uint32_t w =
          a.q[(static_cast<int64_t>(r.q_start) * a.Hq + kvh * G + h) * D + lane * VPT + i];
      q[h][i] = __uint_as_float(w << 16);
      o[h][i] = 0.f;
    }
  }
  for (int32_t key = key_begin + warp; key < key_end; key += kWarpsF8) {
    const int32_t page = a.kv_indices[r.page_base + (key >> a.page_shift)];
    float k[VPT], v[VPT], ks = 1.f, vs = 1.f;
    const bool good = page >= 0 && page < a.num_pages;
    if (!good && lane == 0) atomicOr(a.status, kStatusBadPage);
    const int64_t slot = (static_cast<int64_t>(good ? page : 0) << a.page_shift) +
                         (key & ((1 << a.page_shift) - 1));
    const int64_t row = slot * a.Hkv + kvh;
    if (good) {
      ks = e8m0_value(f.k_scale[row]);
      vs = e8m0_value(f.v_scale[row]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float unused;
      k[i] = v[i] = 0.f; // a bad page reads as zeros
      if (good) {
        e4m3x2_values(f.k_codes[row * D + lane * VPT + i], k[i], unused);
        e4m3x2_values(f.v_codes[row * D + lane * VPT + i], v[i], unused);
      }
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) s = fmaf(q[h][i], k[i], s);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s *= a.scale_log2 * ks;
      const float mn = fmaxf(m[h], s);
      const float alpha = mn == -INFINITY ? 1.f : ex2(m[h] - mn);
      const float p = mn == -INFINITY ? 0.f : ex2(s - mn);
      m[h] = mn;
      l[h] = fmaf(l[h], alpha, p);
#pragma unroll
      for (int i = 0; i < VPT; ++i) o[h][i] = fmaf(o[h][i], alpha, p * vs * v[i]);
    }
  }
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const float inv = l[h] == 0.f ? 0.f : __frcp_rn(l[h]);
#pragma unroll
    for (int i = 0; i < VPT; ++i) s_o[(warp * G + h) * D + lane * VPT + i] = o[h][i] * inv;
    if (lane == 0) s_l[warp][h] = l[h] == 0.f ? -INFINITY : (m[h] + lg2(l[h])) * kLn2;
  }
  __syncthreads();
  const bool single = (r.kv_len - 1) / a.split == 0;
  const int64_t row0 =
      single ? static_cast<int64_t>(r.q_start) * a.Hq + kvh * G
             : (r.rowbase + u.split) * static_cast<int64_t>(a.Hq) + kvh * G;
  for (int h = warp; h < G; h += kWarpsF8) {
    float L = -INFINITY, acc[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) acc[i] = 0.f;
    for (int w = 0; w < kWarpsF8; ++w) {
      float x[VPT];
#pragma unroll
      for (int i = 0; i < VPT; ++i) x[i] = s_o[(w * G + h) * D + lane * VPT + i];
      fold_state<VPT>(L, acc, s_l[w][h], x);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (single)
        a.out[(row0 + h) * D + lane * VPT + i] = to_bf16(acc[i]);
      else
        a.part_o[(row0 + h) * D + lane * VPT + i] = acc[i];
    }
    if (lane == 0) {
      if (single) {
        if (a.lse) a.lse[row0 + h] = L;
      } else {
        a.part_lse[row0 + h] = L;
      }
    }
  }
}

template <int VPT, int G>
cudaError_t launch_f8(const DecodeFp8Args &f, cudaStream_t s) {
  constexpr size_t bytes = sizeof(float) * kWarpsF8 * G * VPT * 32;
  const cudaError_t e = cudaFuncSetAttribute(decode_fp8_kernel<VPT, G>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(f.a.n_units * f.a.Hkv));
  cfg.blockDim = dim3(kWarpsF8 * 32);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_fp8_kernel<VPT, G>, f);
}

template <int VPT>
cudaError_t launch_f8_d(const DecodeFp8Args &f, cudaStream_t s) {
  switch (f.a.G) {
  case 1: return launch_f8<VPT, 1>(f, s);
  case 2: return launch_f8<VPT, 2>(f, s);
  case 4: return launch_f8<VPT, 4>(f, s);
  case 8: return launch_f8<VPT, 8>(f, s);
  default: return cudaErrorInvalidValue;
  }
}

} // namespace

cudaError_t launch_decode_fp8(const DecodeFp8Args &f, cudaStream_t s) {
  if (f.a.n_units == 0) return cudaSuccess;
  switch (f.a.D) {
  case 64: return launch_f8_d<2>(f, s);
  case 96: return launch_f8_d<3>(f, s);
  case 128: return launch_f8_d<4>(f, s);
  case 256: return launch_f8_d<8>(f, s);
  default: return cudaErrorInvalidValue;
  }
}

} // namespace bia
