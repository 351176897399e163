// Attention of packed sequences over contiguous keys and values on the tensor
// cores (tcgen05 + TMEM): the extend of prefill.cu (128-row q tiles of 128/G
// tokens x G heads, "sglang PR #43612", Summary; fixed split-KV tiles merged
// in order, "sglang PR #10417 [POC] Support deterministic inference",
// Modifications; every reduction boundary anchored at absolute key 0) for
// k, v [total_kv, Hkv, D] instead of pages.
//
// A CTA computes one unit: up to two consecutive q tiles of one request and
// one kv head against one split.  A 128-key block of K or V is D/64 tiled TMA
// boxes (64 columns x 1 head x 128 tokens) straight into the 128-byte-swizzled
// operand tile, two stages deep.  Rows past the request's last key belong to
// the next request: their S columns are masked, and their V rows are
// overwritten with zeros before the block's P.V (0 * NaN would reach the
// row).  Warp roles (10 warps): 0-3 and 4-7 softmax + epilogue of the two
// tiles, 8 issues the MMAs and owns TMEM, 9 loads.
//
// Invariance: as for prefill.cu; single-token tiles run here too, so a row's
// bits do not depend on where a chunk boundary falls at all.
#include "bia_internal.h"
#include "ptx.cuh"
#include "softmax_rows.cuh"

namespace bia {

namespace {

constexpr int kMmaWarpR = 8;
constexpr int kProdWarpR = 9;
constexpr int kThreadsR = 320;
constexpr int kAtomR = kTileRows * 128; // one SW128 column block: 128 rows x 64 bf16
constexpr float kRescaleR = 8.0f;       // log2 units

template <int D>
struct SmemR {
  static constexpr int kTile = kTileRows * D * 2; // one Q, K or V tile
  static constexpr int kQ = 0;
  static constexpr int kKV = 2 * kTile; // stage s: K at kKV + 2s*kTile, V after it
  static constexpr int kBar = 6 * kTile;
  static constexpr int kQFull = 0, kKFull = 1, kVFull = 3, kKEmpty = 5, kVEmpty = 7, kSFull = 9,
                       kPFull = 11, kODone = 13, kVTail = 15, kNumBars = 16;
  static constexpr int kSlot = kBar + kNumBars * 8;
  static constexpr int kAlloc = kSlot + 16 + 1024;
};

struct TileR {
  int32_t tile, n_splits, n_blocks;
  bool has;
};

template <int D>
__global__ void __launch_bounds__(kThreadsR, 1)
    prefill_ragged_kernel(const __grid_constant__ AttnArgs a) {
  using L = SmemR<D>;
  constexpr uint32_t kIdescS = idesc_bf16(128, kKvBlock, false);
  constexpr uint32_t kIdescPV = idesc_bf16(128, D, true);
  constexpr uint32_t kTmemCols = 512;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + L::kBar + 8u * static_cast<uint32_t>(i); };
  auto sQ = [&](int t) { return sbase + L::kQ + t * L::kTile; };
  auto sK = [&](int st) { return sbase + L::kKV + (2 * st) * L::kTile; };
  auto sV = [&](int st) { return sbase + L::kKV + (2 * st + 1) * L::kTile; };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kSlot);

  grid_dep_wait();   // the plan is complete
  grid_dep_launch(); // the next kernel of the call may start launching
  const Unit u = a.units[blockIdx.x];
  if (u.b < 0) return; // plan mismatch: every unit of the launch is disabled
  const ReqInfo r = a.reqs[u.b];
  const int kvh = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.G, T = a.tile_tokens;
  const int32_t key_begin = u.split * a.split;

  auto tile_info = [&](int t) {
    TileR x;
    x.tile = u.tile + t;
    const bool exists = t < u.ntiles;
    x.n_splits = exists ? tile_splits(r.q_len, r.kv_len, x.tile, T, a.causal, a.split) : 0;
    x.has = exists && u.split < x.n_splits;
    const int32_t last = tile_last_key(r.q_len, r.kv_len, x.tile, T, a.causal);
    const int32_t end = min(key_begin + a.split, last + 1);
    x.n_blocks = (x.has && end > key_begin) ? (end - key_begin + kKvBlock - 1) / kKvBlock : 0;
    return x;
  };
  const TileR ti0 = tile_info(0), ti1 = tile_info(1);
  const int n_blocks = max(ti0.n_blocks, ti1.n_blocks);
  // the unit's last block holds rows of the next request: only then is its V
  // completed by the producer warp
  const int32_t tail = r.kv_len - (key_begin + (n_blocks - 1) * kKvBlock); // its real rows
  const bool v_tail = n_blocks > 0 && tail < kKvBlock;

  if (warp == kMmaWarpR) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  if (tid == 0) {
    mbar_init(bar(L::kQFull), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(L::kKFull + s), 1);
      mbar_init(bar(L::kVFull + s), 1);
      mbar_init(bar(L::kKEmpty + s), 1);
      mbar_init(bar(L::kVEmpty + s), 1);
      mbar_init(bar(L::kSFull + s), 1);
      mbar_init(bar(L::kPFull + s), 4);
      mbar_init(bar(L::kODone + s), 1);
    }
    mbar_init(bar(L::kVTail), 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // TMEM columns: S_A [0,128) S_B [128,256) O_A [256,256+D) O_B [256+D,256+2D)
  auto tS = [&](int t) { return tmem + 128u * t; };
  auto tO = [&](int t) { return tmem + 256u + static_cast<uint32_t>(D) * t; };

  if (warp == kProdWarpR) {
    // ------------------------------------------------------------ loads
    bool ok = true;
    if (lane == 0 && n_blocks > 0) {
      mbar_expect_tx(bar(L::kQFull), static_cast<uint32_t>(ti0.has + ti1.has) * L::kTile);
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (t ? ti1.has : ti0.has)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(sQ(t) + h * kAtomR, &a.tm_q, 64 * h, kvh * G,
                        r.q_start + (u.tile + t) * T, bar(L::kQFull));
      for (int j = 0; j < n_blocks && ok; ++j) {
        const int st = j & 1;
        const int32_t row = r.page_base + key_begin + j * kKvBlock;
        ok = j < 2 || mbar_wait(bar(L::kKEmpty + st), ((j >> 1) - 1) & 1, a.status);
        if (!ok) break;
        mbar_expect_tx(bar(L::kKFull + st), L::kTile);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tma_load_3d(sK(st) + h * kAtomR, &a.tm_k, 64 * h, kvh, row, bar(L::kKFull + st));
        ok = j < 2 || mbar_wait(bar(L::kVEmpty + st), ((j >> 1) - 1) & 1, a.status);
        if (!ok) break;
        mbar_expect_tx(bar(L::kVFull + st), L::kTile);
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          tma_load_3d(sV(st) + h * kAtomR, &a.tm_v, 64 * h, kvh, row, bar(L::kVFull + st));
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (v_tail && ok) { // the rows past the last key become zeros
      const int j = n_blocks - 1;
      if (mbar_wait(bar(L::kVFull + (j & 1)), (j >> 1) & 1, a.status)) {
        uint8_t *v = smem + L::kKV + (2 * (j & 1) + 1) * L::kTile;
        for (int i = max(tail, 0) * 8 + lane; i < kTileRows * 8; i += 32)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            *reinterpret_cast<uint4 *>(v + h * kAtomR + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async(); // the zeros are read by the MMA (async proxy)
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kVTail));
    }
    // no copy outlives the CTA, also when a wait of the MMA warp ran out
    if (lane == 0 && ok && n_blocks > 0) {
      mbar_wait(bar(L::kQFull), 0, a.status);
      for (int j = max(0, n_blocks - 2); j < n_blocks; ++j) {
        mbar_wait(bar(L::kKFull + (j & 1)), (j >> 1) & 1, a.status);
        mbar_wait(bar(L::kVFull + (j & 1)), (j >> 1) & 1, a.status);
      }
    }
  } else if (warp == kMmaWarpR) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && n_blocks > 0) {
      // descriptors built once: a K step only advances the address field
      const uint64_t dQ0 = desc_sw128(sQ(0), 16, 1024), dQ1 = desc_sw128(sQ(1), 16, 1024);
      const uint64_t dK0 = desc_sw128(sK(0), 16, 1024), dK1 = desc_sw128(sK(1), 16, 1024);
      const uint64_t dV0 = desc_sw128(sV(0), kAtomR, 1024), dV1 = desc_sw128(sV(1), kAtomR, 1024);
      const int nb0 = ti0.n_blocks, nb1 = ti1.n_blocks;
      bool ok = mbar_wait(bar(L::kQFull), 0, a.status);
      auto issue_s = [&](int t, int j) {
        if (!ok) return;
        const uint64_t dq = t ? dQ1 : dQ0, dk = (j & 1) ? dK1 : dK0;
        const uint32_t ts = tS(t);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t koff = ((kk >> 2) * kAtomR + (kk & 3) * 32) >> 4;
          mma_bf16_ss(ts, dq + koff, dk + koff, kIdescS, kk > 0);
        }
        mma_commit(bar(L::kSFull + t));
      };
      auto issue_pv = [&](int t, int j, int nb) {
        ok = ok && mbar_wait(bar(L::kPFull + t), j & 1, a.status);
        if (!ok) return;
        tc_fence_after();
        const uint64_t dv = (j & 1) ? dV1 : dV0;
        const uint32_t to = tO(t), ts = tS(t);
#pragma unroll
        for (int kk = 0; kk < kKvBlock / 16; ++kk)
          mma_bf16_ts(to, ts + kk * 8, dv + ((kk * 2048) >> 4), kIdescPV,
                      (j > 0 || kk > 0) ? 1u : 0u);
        if (j == nb - 1) mma_commit(bar(L::kODone + t));
      };
      ok = ok && mbar_wait(bar(L::kKFull + 0), 0, a.status);
      if (ok) tc_fence_after();
      if (nb0 > 0) issue_s(0, 0);
      if (nb1 > 0) issue_s(1, 0);
      if (ok && 2 < n_blocks) mma_commit(bar(L::kKEmpty + 0));
      for (int j = 0; j < n_blocks && ok; ++j) {
        const int st = j & 1, j1 = j + 1;
        ok = mbar_wait(bar(L::kVFull + st), (j >> 1) & 1, a.status);
        if (ok && v_tail && j1 == n_blocks) ok = mbar_wait(bar(L::kVTail), 0, a.status);
        if (!ok) break;
        if (j < nb0) issue_pv(0, j, nb0);
        if (j1 < n_blocks) {
          ok = ok && mbar_wait(bar(L::kKFull + (j1 & 1)), (j1 >> 1) & 1, a.status);
          if (ok) tc_fence_after();
        }
        if (j1 < nb0) issue_s(0, j1);
        if (j < nb1) issue_pv(1, j, nb1);
        if (j1 < nb1) issue_s(1, j1);
        if (!ok) break;
        // a stage is released only when a later block refills it
        if (j + 2 < n_blocks) mma_commit(bar(L::kVEmpty + st));
        if (j + 3 < n_blocks) mma_commit(bar(L::kKEmpty + (j1 & 1)));
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const TileR me = t ? ti1 : ti0;
    const int gs = __ffs(G) - 1; // G is a power of two
    const int32_t t_row = me.tile * T + (row >> gs);
    const bool row_valid = me.has && t_row < r.q_len;
    const int32_t p_row = a.causal ? r.kv_len - r.q_len + t_row : r.kv_len - 1;
    const int32_t vis_last = min(p_row, r.kv_len - 1);
    const uint32_t all[4] = {~0u, ~0u, ~0u, ~0u};
    float m = -INFINITY, l = 0.f; // running max (log2 units) and sum
    bool failed = false;
    for (int j = 0; j < me.n_blocks; ++j) {
      const int32_t n_vis = vis_last - (key_begin + j * kKvBlock) + 1; // visible columns
      if (!mbar_wait(bar(L::kSFull + t), j & 1, a.status)) {
        failed = true;
        break;
      }
      tc_fence_after();
      // blocks every row of the warp sees in full skip the per-column test
      const bool full = __all_sync(0xffffffffu, n_vis >= kKvBlock);
      const uint32_t srow = tS(t) + lane_base;
      float bm = full ? row_block_max<kKvBlock, kFull>(srow, n_vis, all)
                      : row_block_max<kKvBlock, kFirst>(srow, n_vis, all);
      bm = bm == -INFINITY ? -INFINITY : bm * a.scale_log2;
      float m_use = m, alpha = 1.f;
      if (bm > m + kRescaleR || (m == -INFINITY && bm != -INFINITY)) {
        m_use = bm;
        alpha = ex2(m - bm); // 0 when m == -inf
      }
      const float m_sub = m_use == -INFINITY ? 0.f : m_use;
      const float psum =
          full ? row_block_p<kKvBlock, kFull>(srow, n_vis, all, a.scale_log2, m_sub)
               : row_block_p<kKvBlock, kFirst>(srow, n_vis, all, a.scale_log2, m_sub);
      l = fmaf(l, alpha, psum);
      m = m_use;
      // rescale the running O row when the max moved (the previous P.V has
      // completed: S of this block was issued after it)
      if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t v[16];
          tmem_ld16(tO(t) + lane_base + c * 16, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
          tmem_st16(tO(t) + lane_base + c * 16, v);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kPFull + t));
    }
    // epilogue: o_s = O / l, each row stored by its thread: bf16 when the
    // tile has one split, else the fp32 partial
    if (me.has) {
      // warp-uniform (tcgen05.ld is warp-collective): a warp with a failed
      // wait writes zeros
      const bool have_o = __all_sync(0xffffffffu, !failed && me.n_blocks > 0 &&
                                                      mbar_wait(bar(L::kODone + t), 0, a.status));
      tc_fence_after();
      const bool some = have_o && !(l == 0.f); // NaN sums stay NaN
      const float lse = some ? __fmul_rn(__fadd_rn(m, lg2(l)), kLn2) : -INFINITY;
      const float inv_l = some ? __frcp_rn(l) : 0.f; // o_s = O * (1/l)
      const bool final_row = me.n_splits == 1;       // uniform over the tile
      const int h = kvh * G + (row & (G - 1));
      const int64_t out_row = static_cast<int64_t>(r.q_start + t_row) * a.Hq + h;
      const int64_t part_row =
          (r.rowbase + static_cast<int64_t>(t_row) * r.nsp + u.split) * a.Hq + h;
      const int Dr = a.D; // head_dim 96 runs on the 128-wide layout, zero-padded
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        if (have_o) {
          tmem_ld32(tO(t) + lane_base + c * 32, v);
          tmem_wait_ld();
        }
        if (!row_valid || c * 32 >= Dr) continue;
        float o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i)
          o[i] = some ? __fmul_rn(__uint_as_float(v[i]), inv_l) : 0.f;
        if (final_row) {
          uint4 *dst = reinterpret_cast<uint4 *>(a.out + out_row * Dr + c * 32);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            dst[q] = make_uint4(pack_bf16(o[q * 8 + 0], o[q * 8 + 1]),
                                pack_bf16(o[q * 8 + 2], o[q * 8 + 3]),
                                pack_bf16(o[q * 8 + 4], o[q * 8 + 5]),
                                pack_bf16(o[q * 8 + 6], o[q * 8 + 7]));
        } else {
          float4 *dst = reinterpret_cast<float4 *>(a.part_o + part_row * Dr + c * 32);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            dst[q] = make_float4(o[q * 4], o[q * 4 + 1], o[q * 4 + 2], o[q * 4 + 3]);
        }
      }
      if (row_valid) {
        if (final_row) {
          if (a.lse) a.lse[out_row] = lse;
        } else {
          a.part_lse[part_row] = lse;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarpR) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch_ragged_d(const AttnArgs &a, cudaStream_t s) {
  using L = SmemR<D>;
  const cudaError_t e = cudaFuncSetAttribute(prefill_ragged_kernel<D>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             L::kAlloc);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_units), static_cast<unsigned>(a.Hkv));
  cfg.blockDim = dim3(kThreadsR);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_ragged_kernel<D>, a);
}

} // namespace

cudaError_t launch_prefill_ragged(const AttnArgs &a, cudaStream_t s) {
  if (a.n_units == 0) return cudaSuccess;
  // head_dim 96 runs on the 128-wide layout: the tensor maps read columns
  // 96..127 as zeros
  return a.D > 64 ? launch_ragged_d<128>(a, s) : launch_ragged_d<64>(a, s);
}

} // namespace bia
