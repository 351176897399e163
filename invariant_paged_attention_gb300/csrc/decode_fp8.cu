// Split-KV decode of one query token per request over the 8-bit paged cache
// (fp8.cuh states the format) on the tensor cores, with fixed split-KV tiles
// joined in ascending order as the bf16 decode does ("sglang PR #10417 [POC]
// Support deterministic inference", Modifications):
//   s_j = sm_scale * 2^ek_j * <q, ck_j>,   o = sum_j softmax(s)_j 2^ev_j cv_j
//
// The rows go from HBM to the tensor cores as they are: kind::f8f6f4 MMAs
// read the e4m3 codes, and the operands that are not 8-bit are split into two
// e4m3 terms (a = hi + lo/16, each rounded to nearest), which share the
// MMAs' N columns:
//   S^T = K [q_hi; q_lo]^T    M = 128 keys of a block, N = 16, K = D
//   O^T += V^T [p_hi; p_lo]   M = 128 dims, N = 16, K = 128 keys
// q is scaled by a power of two per head, so that q = hi + lo/16 is exact
// down to 2^-11 of the row's largest element and off by at most 2^-22 of it
// below; a weight keeps 8 significant bits (what a bf16 weight keeps) down to
// 2^-14 of the largest.  The key's scale multiplies its score, the value's
// scale its weight, relative to the largest value scale of the tile (a power
// of two: exact).  Products, sums, the maximum and the row sum are fp32.
// Converting the rows instead (8 -> 16 bits through registers and shared
// memory) would cost more issue slots than the copies themselves.
//
// HBM bound: D + 1 bytes per key, head and cache.  At 6.5 TB/s an SM has
// ~1450 cycles for a 128-key block of head_dim 128, half of what the bf16
// decode has, and an online softmax does not fit: per block its chain of
// waits, maximum exchange and rescaling took ~5000 cycles of a warpgroup, 3.8
// TB/s with two of them on alternate blocks.  So a tile (at most 1024 keys)
// takes two passes: all its scores first, kept in TMEM (16 columns a block,
// two tiles' worth), one maximum over the tile, then the weights.  Nothing is
// rescaled, the weights of a tile are at most 1 and fill e4m3's range, and
// the warps meet once a tile.  The key rows of a tile are copied before its
// value rows, through a ring of their own each (one ring for both would let S
// of the next tile wait on a stage two uses ahead, which an mbarrier's parity
// cannot tell from the use before).
//
// Persistent: one CTA per SM takes (unit, kv head) items from a counter.
// Warps 0-3 and 4-7 softmax (even and odd blocks; the epilogue alternates by
// item), 8 issues P.V (owns TMEM), 9 issues S, 10-13 prepare an item: the
// rows and scales of its keys, its q; 14-21 copy (16-byte cp.async into the
// swizzled operand layout), 22 takes the items and posts them through a
// mailbox in shared memory, one ahead of the copies.  An item's result
// depends on its own keys alone, whichever CTA takes it.
#include <algorithm>

#include "bia_internal.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace bia {

namespace {

constexpr int kKeys8 = 128;           // keys per block: the MMAs' M
constexpr int kPiece8 = kKeys8 * 128; // 128 rows x 128 codes, SW128
constexpr int kN8 = 16;               // the MMAs' N: hi and lo of up to 8 heads
constexpr int kBlocks8 = BIA_DECODE_FP8_SPLIT / kKeys8; // blocks of a tile
constexpr int kPVWarp8 = 8;
constexpr int kSWarp8 = 9;
constexpr int kAuxWarp8 = 10;
constexpr int kCopyWarp8 = 14;
constexpr int kCopyWarps8 = 8;
constexpr int kItemWarp8 = kCopyWarp8 + kCopyWarps8;
constexpr int kThreads8 = (kItemWarp8 + 1) * 32;
constexpr int kCopyThreads8 = kCopyWarps8 * 32;
constexpr int kCopyKeys8 = kKeys8 / kCopyWarps8; // keys of a block a copy warp takes
constexpr int kReaders8 = kItemWarp8;            // warps that read the mailbox
constexpr int kBoost8 = 8; // weights <= 1 times 2^8 fill e4m3's range (448)
constexpr uint32_t kNoRow8 = 0xffffffffu; // a key past the end or on a bad page: zeros

// LPR: lanes (16-byte chunks) per row: 4 (head_dim 64), 8 (96, 128), 16 (256)
template <int LPR>
struct Smem8 {
  static constexpr int NP = LPR > 8 ? 2 : 1; // 128-code pieces of a row
  // A ring stage holds SB blocks: two for rows of up to 128 codes, so that a
  // barrier is waited for (~300 cycles even when it is complete) and the
  // async proxy fenced every 256 keys
  static constexpr int SB = NP == 1 ? 2 : 1;
  static constexpr int kTileStages = kBlocks8 / SB;
  static constexpr int kBlock = NP * kPiece8;
  static constexpr int kStage = SB * kBlock;
  static constexpr int NS = 3;  // stages in the key ring and in the value ring
  static constexpr int NPS = 4; // stages of P
  static constexpr int kKRing = 0;
  static constexpr int kVRing = kKRing + NS * kStage;
  static constexpr int kQBuf = NP * kN8 * 128;
  static constexpr int kQ = kVRing + NS * kStage; // [2]
  static constexpr int kPBuf = SB * kKeys8 * kN8;
  static constexpr int kP = kQ + 2 * kQBuf;      // [NPS]
  static constexpr int kTile = kBlocks8 * kKeys8;
  static constexpr int kRows = kP + NPS * kPBuf;      // uint32 [2][tile]: cache rows
  static constexpr int kKe = kRows + 2 * kTile * 4;   // uint8 [2][tile]: key scales
  static constexpr int kVe = kKe + 2 * kTile;         // uint8 [2][tile]: value scales
  static constexpr int kEmax = kVe + 2 * kTile;       // int [2][kBlocks8]
  static constexpr int kQs = kEmax + 2 * kBlocks8 * 4; // float [2][8]
  static constexpr int kRed = kQs + 64;           // float [2][8 warps][8]
  static constexpr int kStat = kRed + 512;        // float [2][8 warps][8]
  static constexpr int kItems = kStat + 512;      // 32-byte records [4]
  static constexpr int kSlot = kItems + 128;
  static constexpr int kBar = kSlot + 16;
  static constexpr int bKFull = 0, bKEmpty = bKFull + NS, bVFull = bKEmpty + NS,
                       bVEmpty = bVFull + NS, bQFull = bVEmpty + NS, bQEmpty = bQFull + 2,
                       bRows = bQEmpty + 2, bRowsFree = bRows + 2, bAux = bRowsFree + 2,
                       bAuxFree = bAux + 2, bMax = bAuxFree + 2, bStat = bMax + 2,
                       bODone = bStat + 2, bOFree = bODone + 2, bSFull = bOFree + 2,
                       bPFull = bSFull + 2 * kTileStages, bPVDone = bPFull + NPS,
                       bItemFull = bPVDone + NPS,
                       bItemEmpty = bItemFull + 4, bGo = bItemEmpty + 4, kNumBars = bGo + 1;
  static constexpr int kAlloc = kBar + kNumBars * 8 + 1024;
  static_assert(kAlloc <= 232448, "shared memory per CTA");
  static_assert(kQ % 1024 == 0 && kQBuf % 1024 == 0 && kBar % 8 == 0, "alignment");
};

// One item: a tile of one request for one kv head.
struct Item8 {
  int32_t nb;  // 128-key blocks; -1: no more items
  int32_t kvh;
  int32_t b;   // request
  int32_t key_begin, key_end, page_base;
  int64_t prow; // row of the partial states, in units of Hq heads; -1: one tile
};
static_assert(sizeof(Item8) == 32, "Item8 layout");

template <int NL>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t (&r)[NL]) {
  if constexpr (NL == 8) tmem_ld8(taddr, r);
  else tmem_ld16(taddr, r);
}

template <int G, int LPR>
__global__ void __launch_bounds__(kThreads8, 1)
    decode_fp8_kernel(const __grid_constant__ DecodeFp8Args f) {
  using L = Smem8<LPR>;
  constexpr int NP = L::NP, NS = L::NS, SB = L::SB, NPS = L::NPS;
  constexpr int kSBars = 2 * L::kTileStages; // S stages in TMEM: two tiles
  constexpr int LO = G <= 4 ? 4 : 8; // column of a head's second term
  constexpr int NL = 2 * LO;         // columns in use
  constexpr uint32_t kIdescS = idesc_e4m3(128, kN8, false, false);
  constexpr uint32_t kIdescPV = idesc_e4m3(128, kN8, true, true);
  constexpr uint32_t kTmemCols = 512;
  const AttnArgs &a = f.a;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + L::kBar + 8u * static_cast<uint32_t>(i); };
  auto kstage = [&](uint32_t s) { return sbase + L::kKRing + s * L::kStage; };
  auto vstage = [&](uint32_t s) { return sbase + L::kVRing + s * L::kStage; };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kSlot);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == kPVWarp8) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  // q rows of heads that do not exist stay zero
  for (int i = tid; i < 2 * L::kQBuf / 16; i += kThreads8)
    reinterpret_cast<uint4 *>(smem + L::kQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar(L::bKFull + s), kCopyThreads8); // one arrival per copy thread
      mbar_init(bar(L::bKEmpty + s), 1);
      mbar_init(bar(L::bVFull + s), kCopyThreads8);
      mbar_init(bar(L::bVEmpty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::bQFull + i), 4);              // the aux warps
      mbar_init(bar(L::bQEmpty + i), 1);             // the S MMAs
      mbar_init(bar(L::bRows + i), 4);
      mbar_init(bar(L::bRowsFree + i), kCopyWarps8);
      mbar_init(bar(L::bAux + i), 4);
      mbar_init(bar(L::bAuxFree + i), 8);            // the softmax warps, past pass 2
      mbar_init(bar(L::bMax + i), 8);
      mbar_init(bar(L::bStat + i), 8);
      mbar_init(bar(L::bODone + i), 1);
      mbar_init(bar(L::bOFree + i), 4);
    }
    for (int i = 0; i < kSBars; ++i) mbar_init(bar(L::bSFull + i), 1);
    for (int i = 0; i < NPS; ++i) {
      mbar_init(bar(L::bPFull + i), 4 * SB); // the warps of the stage's blocks
      mbar_init(bar(L::bPVDone + i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(L::bItemFull + i), 1);
      mbar_init(bar(L::bItemEmpty + i), kReaders8);
    }
    mbar_init(bar(L::bGo), 1);
    fence_mbar_init();
  }
  grid_dep_launch(); // the merge may start launching
  grid_dep_wait();   // the plan is complete (all of the above ran beside it)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // TMEM columns: S^T [item parity][block] (lanes = keys), then O^T [item
  // parity][piece] (lanes = dims), 16 each
  auto tS = [&](uint32_t ig, int j) {
    return tmem + 16u * ((ig & 1u) * kBlocks8 + static_cast<uint32_t>(j));
  };
  auto tO = [&](uint32_t ig, int p) {
    return tmem + 16u * (2 * kBlocks8 + (ig & 1u) * NP + static_cast<uint32_t>(p));
  };
  // the ig-th item of this CTA; nb = -1 also when the wait ran out
  auto read_item = [&](uint32_t ig) {
    const int s = static_cast<int>(ig & 3u);
    Item8 it;
    it.nb = -1;
    if (mbar_wait(bar(L::bItemFull + s), (ig >> 2) & 1u, a.status))
      it = *reinterpret_cast<const Item8 *>(smem + L::kItems + s * 32);
    return it;
  };
  auto item_read = [&](uint32_t ig) { mbar_arrive(bar(L::bItemEmpty + static_cast<int>(ig & 3u))); };
  // The warp-wide forms: the same answer on every lane, so that a wait that
  // ran out takes the whole warp out (the others then run out of theirs).
  auto wait = [&](int b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, a.status)) != 0;
  };
  auto warp_item = [&](uint32_t ig) {
    Item8 it = read_item(ig);
    if (__any_sync(0xffffffffu, it.nb < 0)) it.nb = -1;
    if (lane == 0) item_read(ig);
    return it;
  };

  if (warp == kItemWarp8) {
    // ------------------------------------------------------------ items
    // The first item is the CTA's own index; each next one is taken from the
    // counter when the copies of the current one start.
    if (lane == 0) {
      const int64_t n_work = a.n_units * a.Hkv;
      int64_t w = blockIdx.x;
      for (uint32_t ig = 0;; ++ig) {
        Item8 it;
        it.nb = -1;
        if (w < n_work) {
          const int64_t unit = w / a.Hkv;
          const int4 u0 = __ldg(reinterpret_cast<const int4 *>(f.units + unit));
          const int4 u1 = __ldg(reinterpret_cast<const int4 *>(f.units + unit) + 1);
          if (u0.x >= 0) { // a retired unit: only retired ones follow
            it.kvh = static_cast<int>(w - unit * a.Hkv);
            it.b = u0.x;
            it.key_begin = u0.y;
            it.key_end = u0.z;
            it.page_base = u0.w;
            it.prow = static_cast<int64_t>(static_cast<uint32_t>(u1.x)) |
                      (static_cast<int64_t>(u1.y) << 32);
            it.nb = (it.key_end - it.key_begin + kKeys8 - 1) / kKeys8;
          }
        }
        const int s = static_cast<int>(ig & 3u);
        if (ig >= 4 && !mbar_wait(bar(L::bItemEmpty + s), ((ig >> 2) - 1) & 1u, a.status)) it.nb = -1;
        *reinterpret_cast<Item8 *>(smem + L::kItems + s * 32) = it;
        mbar_arrive(bar(L::bItemFull + s));
        if (it.nb < 0) break;
        if (!mbar_wait(bar(L::bGo), ig & 1u, a.status)) w = n_work;
        else w = static_cast<int64_t>(gridDim.x) + atomicAdd(a.status + kStatusWorkCounter, 1);
      }
    }
    __syncwarp();
  } else if (warp >= kCopyWarp8) {
    // ------------------------------------------------------------ copies
    // A warp copies 16 keys of each block: chunk cc of every (32 / LPR)-th.
    const int cw = warp - kCopyWarp8;
    const int cc = lane % LPR, kb = lane / LPR;
    const bool in_row = cc * 16 < a.D; // head_dim 96: six of eight lanes
    const uint32_t *rows = reinterpret_cast<const uint32_t *>(smem + L::kRows);
    uint32_t sg = 0; // stages so far
    bool ok = true;
    for (uint32_t ig = 0; ok; ++ig) {
      const Item8 it = warp_item(ig);
      if (it.nb < 0) break;
      const int nst = (it.nb + SB - 1) / SB;
      if (cw == 0 && lane == 0) mbar_arrive(bar(L::bGo));
      ok = wait(L::bRows + static_cast<int>(ig & 1), (ig >> 1) & 1);
      for (int kv = 0; kv < 2 && ok; ++kv) {
        const uint8_t *src = (kv == 0 ? f.k_codes : f.v_codes) + cc * 16;
        const uint32_t *row_w = rows + (ig & 1) * L::kTile + cw * kCopyKeys8 + kb;
        for (int st = 0; st < nst; ++st) {
          const uint32_t ss = sg + st, s = ss % NS;
          if (ss >= NS)
            ok = wait((kv == 0 ? L::bKEmpty : L::bVEmpty) + static_cast<int>(s), ((ss / NS) - 1) & 1);
          if (!ok) break;
#pragma unroll
          for (int hb = 0; hb < SB; ++hb) {
            const uint32_t dst = (kv == 0 ? kstage(s) : vstage(s)) + hb * L::kBlock +
                                 static_cast<uint32_t>(cc >> 3) * kPiece8;
#pragma unroll
            for (int i = 0; i < kCopyKeys8 * LPR / 32; ++i) {
              const int k8 = cw * kCopyKeys8 + i * (32 / LPR) + kb;
              const uint32_t row = row_w[(st * SB + hb) * kKeys8 + i * (32 / LPR)];
              if (in_row)
                cp_async16(dst + static_cast<uint32_t>(k8) * 128 +
                               ((static_cast<uint32_t>(cc & 7) ^ static_cast<uint32_t>(k8 & 7)) << 4),
                           src + (row == kNoRow8 ? 0 : static_cast<uint64_t>(row) * a.D),
                           row != kNoRow8);
            }
          }
          cp_async_arrive(bar((kv == 0 ? L::bKFull : L::bVFull) + s));
        }
      }
      sg += nst;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bRowsFree + static_cast<int>(ig & 1)));
    }
    cp_async_wait_all(); // no copy outlives the CTA
  } else if (warp >= kAuxWarp8) {
    // ------------------------------------------------------------ preparation
    // Aux warp w finds the cache rows and the scales of the keys of blocks w
    // and w + 4 (four keys a lane and block), and splits the q rows of heads
    // w and w + 4, up to two items ahead of their use.
    const int aw = warp - kAuxWarp8;
    const int page_mask = (1 << a.page_shift) - 1;
    uint32_t *s_rows = reinterpret_cast<uint32_t *>(smem + L::kRows);
    int32_t *s_emax = reinterpret_cast<int32_t *>(smem + L::kEmax);
    float *s_qs = reinterpret_cast<float *>(smem + L::kQs);
    for (uint32_t ig = 0;; ++ig) {
      const Item8 it = warp_item(ig);
      if (it.nb < 0) break;
      const int par = static_cast<int>(ig & 1);
      int32_t page[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int32_t key = it.key_begin + (aw + 4 * i) * kKeys8 + n * 32 + lane;
          page[i][n] = key < it.key_end
                           ? __ldg(a.kv_indices + it.page_base + (key >> a.page_shift)) : -1;
        }
      // the q rows: 4 elements a lane and 128 columns
      constexpr int NH = G > 4 ? 2 : 1;
      uint2 qv[NH][NP];
#pragma unroll
      for (int i = 0; i < NH; ++i)
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int h = aw + 4 * i, col = p * 128 + lane * 4;
          qv[i][p] = make_uint2(0, 0);
          if (h < G && col < a.D)
            qv[i][p] = __ldg(reinterpret_cast<const uint2 *>(
                a.q + (static_cast<int64_t>(it.b) * a.Hq + it.kvh * G + h) * a.D + col));
        }
      // rows first: the copies wait for them
      if (ig >= 2 && !wait(L::bRowsFree + par, ((ig >> 1) - 1) & 1)) break;
      uint32_t row[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int t = (aw + 4 * i) * kKeys8 + n * 32 + lane;
          const bool real = it.key_begin + t < it.key_end;
          const bool good = real && page[i][n] >= 0 && page[i][n] < a.num_pages;
          if (real && !good) atomicOr(a.status, kStatusBadPage);
          row[i][n] = good ? static_cast<uint32_t>(((static_cast<int64_t>(page[i][n]) << a.page_shift) +
                                                    ((it.key_begin + t) & page_mask)) * a.Hkv + it.kvh)
                           : kNoRow8;
          s_rows[par * L::kTile + t] = row[i][n];
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bRows + par));
      uint32_t kb[2][4], vb[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          kb[i][n] = vb[i][n] = 0; // no row: zeros with a zero weight, outside the maximum
          if (row[i][n] != kNoRow8) {
            kb[i][n] = __ldg(f.k_scale + row[i][n]);
            vb[i][n] = __ldg(f.v_scale + row[i][n]);
          }
        }
      // q: hi + lo/16 of the row scaled by 2^-e
      if (ig >= 2 && !wait(L::bQEmpty + par, ((ig >> 1) - 1) & 1)) break;
      if (ig >= 2 && !wait(L::bAuxFree + par, ((ig >> 1) - 1) & 1)) break;
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        const int h = aw + 4 * i;
        if (h < G) {
          float x[NP][4];
          uint32_t big = 0;
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const uint32_t u[4] = {qv[i][p].x & 0xffffu, qv[i][p].x >> 16, qv[i][p].y & 0xffffu,
                                   qv[i][p].y >> 16};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool fin = (u[e] & 0x7fffu) < kBf16Inf;
              big = max(big, fin ? u[e] & 0x7fffu : 0u);
              x[p][e] = fin ? __uint_as_float(u[e] << 16) : NAN; // makes its head NaN
            }
          }
          big = __reduce_max_sync(0xffffffffu, big);
          const int e = row_exponent(__uint_as_float(big << 16));
          const float inv = exp2_int(-e);
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            const int col = lane * 4;
            float v[4], back[4];
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = x[p][c] * inv;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              hi[c] = e4m3x2(v[2 * c], v[2 * c + 1]);
              e4m3x2_values(hi[c], back[2 * c], back[2 * c + 1]);
              lo[c] = e4m3x2((v[2 * c] - back[2 * c]) * 16.f, (v[2 * c + 1] - back[2 * c + 1]) * 16.f);
            }
            if (p * 128 + col < a.D) {
              uint8_t *q0 = smem + L::kQ + par * L::kQBuf + p * (kN8 * 128);
              auto at = [&](int rr) { // row rr, 16-byte chunk col / 16
                return rr * 128 + (((col >> 4) ^ (rr & 7)) << 4) + (col & 15);
              };
              *reinterpret_cast<uint32_t *>(q0 + at(h)) = hi[0] | (hi[1] << 16);
              *reinterpret_cast<uint32_t *>(q0 + at(LO + h)) = lo[0] | (lo[1] << 16);
            }
          }
          if (lane == 0) s_qs[par * 8 + h] = a.scale_log2 * exp2_int(e);
        }
      }
      fence_proxy_async(); // q is read by the MMA (async proxy)
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bQFull + par));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t big = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int t = par * L::kTile + (aw + 4 * i) * kKeys8 + n * 32 + lane;
          smem[L::kKe + t] = static_cast<uint8_t>(kb[i][n]);
          smem[L::kVe + t] = static_cast<uint8_t>(vb[i][n]);
          big = max(big, vb[i][n] == 255u ? 0u : vb[i][n]);
        }
        big = __reduce_max_sync(0xffffffffu, big);
        if (lane == 0) s_emax[par * kBlocks8 + aw + 4 * i] = static_cast<int32_t>(big);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bAux + par));
    }
  } else if (warp == kSWarp8) {
    // ------------------------------------------------------------ S issuer
    if (lane == 0) {
      const int ksteps = a.D / 32 < 4 ? a.D / 32 : 4; // 32-code steps of a piece
      uint32_t sg = 0;
      bool ok = true;
      for (uint32_t ig = 0; ok; ++ig) {
        const Item8 it = read_item(ig);
        item_read(ig);
        if (it.nb < 0) break;
        const uint32_t qb = sbase + L::kQ + (ig & 1) * L::kQBuf;
        ok = mbar_wait(bar(L::bQFull + (ig & 1)), (ig >> 1) & 1, a.status);
        // the item's S columns are free once the softmax is through item ig - 2
        if (ok && ig >= 2) ok = mbar_wait(bar(L::bAuxFree + (ig & 1)), ((ig >> 1) - 1) & 1, a.status);
        for (int j = 0; j < it.nb && ok; ++sg) {
          const uint32_t s = sg % NS;
          ok = mbar_wait(bar(L::bKFull + s), (sg / NS) & 1, a.status);
          if (!ok) break;
          fence_proxy_async(); // the rows were written by cp.async (generic proxy)
          tc_fence_after();
          for (int hb = 0; hb < SB && j < it.nb; ++hb, ++j)
#pragma unroll
            for (int p = 0; p < NP; ++p)
              for (int kk = 0; kk < ksteps; ++kk)
                mma_e4m3_ss(tS(ig, j),
                            desc_sw128(kstage(s) + hb * L::kBlock + p * kPiece8 + kk * 32, 16, 1024),
                            desc_sw128(qb + p * (kN8 * 128) + kk * 32, 16, 1024), kIdescS,
                            (p | kk) != 0 ? 1u : 0u);
          mma_commit(bar(L::bKEmpty + s));
          mma_commit(bar(L::bSFull + sg % kSBars));
        }
        if (!ok) break;
        mma_commit(bar(L::bQEmpty + (ig & 1)));
      }
    }
    __syncwarp();
  } else if (warp == kPVWarp8) {
    // ------------------------------------------------------------ P.V issuer
    if (lane == 0) {
      uint32_t sg = 0;
      bool ok = true;
      for (uint32_t ig = 0; ok; ++ig) {
        const Item8 it = read_item(ig);
        item_read(ig);
        if (it.nb < 0) break;
        // the item's O buffer is free once the epilogue of item ig - 2 read it
        if (ig >= 2) ok = mbar_wait(bar(L::bOFree + (ig & 1)), ((ig >> 1) - 1) & 1, a.status);
        for (int j = 0; j < it.nb && ok; ++sg) {
          const uint32_t s = sg % NS, ps = sg % NPS;
          ok = mbar_wait(bar(L::bVFull + s), (sg / NS) & 1, a.status) &&
               mbar_wait(bar(L::bPFull + ps), (sg / NPS) & 1, a.status);
          if (!ok) break;
          fence_proxy_async();
          tc_fence_after();
          for (int hb = 0; hb < SB && j < it.nb; ++hb, ++j)
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
              for (int kk = 0; kk < kKeys8 / 32; ++kk)
                mma_e4m3_ss(tO(ig, p),
                            desc_sw128(vstage(s) + hb * L::kBlock + p * kPiece8 + kk * 4096, 16384, 1024),
                            desc_plain(sbase + L::kP + ps * L::kPBuf + hb * (kKeys8 * kN8) + kk * 512,
                                       128, 128),
                            kIdescPV, (j > 0 || kk > 0) ? 1u : 0u);
          mma_commit(bar(L::bVEmpty + s));
          if constexpr (NPS < L::kTileStages) mma_commit(bar(L::bPVDone + ps));
        }
        if (!ok) break;
        mma_commit(bar(L::bODone + (ig & 1)));
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int wg = warp >> 2, qd = warp & 3; // TMEM lanes 32qd .. 32qd+31
    const int t = qd * 32 + lane;            // key of the block, dim of the output
    const uint32_t lane_base = static_cast<uint32_t>(qd * 32) << 16;
    float *s_red = reinterpret_cast<float *>(smem + L::kRed);
    float *s_stat = reinterpret_cast<float *>(smem + L::kStat);
    const int32_t *s_emax = reinterpret_cast<const int32_t *>(smem + L::kEmax);
    const float *s_qs = reinterpret_cast<const float *>(smem + L::kQs);
    uint32_t sg = 0;
    for (uint32_t ig = 0;; ++ig) {
      const Item8 it = warp_item(ig);
      if (it.nb < 0) break;
      const int nst = (it.nb + SB - 1) / SB;
      const int par = static_cast<int>(ig & 1);
      if (!wait(L::bAux + par, (ig >> 1) & 1)) break;
      const uint8_t *ke = smem + L::kKe + par * L::kTile + t;
      const uint8_t *ve = smem + L::kVe + par * L::kTile + t;
      float qs[G];
#pragma unroll
      for (int h = 0; h < G; ++h) qs[h] = s_qs[par * 8 + h];
      bool ok = true;
      // ---- pass 1: the tile's largest score of each head
      float m[G];
#pragma unroll
      for (int h = 0; h < G; ++h) m[h] = -INFINITY;
      for (int j = wg; j < it.nb; j += 2) {
        const uint32_t ss = sg + j / SB;
        ok = wait(L::bSFull + static_cast<int>(ss % kSBars), (ss / kSBars) & 1);
        if (!ok) break;
        tc_fence_after();
        uint32_t v[NL];
        tmem_ld_n<NL>(tS(ig, j) + lane_base, v);
        const float ks = e8m0_value(ke[j * kKeys8]);
        const bool valid = it.key_begin + j * kKeys8 + t < it.key_end;
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float raw = fmaf(__uint_as_float(v[LO + h]), 0.0625f, __uint_as_float(v[h]));
          m[h] = fmaxf(m[h], valid ? raw * (ks * qs[h]) : -INFINITY);
        }
      }
      if (!ok) break;
      float mine = -INFINITY;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float wm = warp_max(m[h]);
        mine = lane == h ? wm : mine;
      }
      if (lane < 8) s_red[(par * 8 + warp) * 8 + lane] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bMax + par));
      int32_t eref = 0; // the tile's largest value scale
#pragma unroll
      for (int j = 0; j < kBlocks8; ++j) eref = max(eref, s_emax[par * kBlocks8 + j]);
      if (!wait(L::bMax + par, (ig >> 1) & 1)) break;
#pragma unroll
      for (int h = 0; h < G; ++h) m[h] = s_red[par * 64 + h];
#pragma unroll
      for (int w = 1; w < 8; ++w)
#pragma unroll
        for (int h = 0; h < G; ++h) m[h] = fmaxf(m[h], s_red[(par * 8 + w) * 8 + h]);
      // ---- pass 2: the weights 2^(s - m), times 2^(ev - eref + 8) in two
      // e4m3 terms
      float l[G];
#pragma unroll
      for (int h = 0; h < G; ++h) l[h] = 0.f;
      // P of item ig - 1 has been read (its slots are the tile's, or fewer)
      if (ig >= 1 && !wait(L::bODone + (par ^ 1), ((ig - 1) >> 1) & 1)) break;
      for (int j = wg; j < it.nb; j += 2) {
        const int st = j / SB;
        const uint32_t ss = sg + st, ps = ss % NPS;
        uint32_t v[NL];
        tmem_ld_n<NL>(tS(ig, j) + lane_base, v);
        const float ks = e8m0_value(ke[j * kKeys8]);
        const uint32_t vb = ve[j * kKeys8];
        const int32_t de = static_cast<int32_t>(vb) - eref + kBoost8 + 127;
        const float vf = vb == 255u ? NAN : de > 0 ? __uint_as_float(de << 23) : 0.f;
        const bool valid = it.key_begin + j * kKeys8 + t < it.key_end;
        tmem_wait_ld();
        float w[G];
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float raw = fmaf(__uint_as_float(v[LO + h]), 0.0625f, __uint_as_float(v[h]));
          const float p = valid ? ex2(fmaf(raw, ks * qs[h], -m[h])) : 0.f;
          l[h] += p;
          w[h] = p * vf;
        }
        uint32_t pk[4] = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < G; h += 2) {
          const float w0 = w[h], w1 = h + 1 < G ? w[h + 1 < G ? h + 1 : h] : 0.f;
          const uint32_t hi = e4m3x2(w0, w1);
          float b0, b1;
          e4m3x2_values(hi, b0, b1);
          const uint32_t lo = e4m3x2((w0 - b0) * 16.f, (w1 - b1) * 16.f);
          pk[h >> 2] |= hi << (8 * (h & 3));
          pk[(LO + h) >> 2] |= lo << (8 * (h & 3));
        }
        // more stages than P slots: the slot's last P.V of this item is done
        if (NPS < L::kTileStages && st >= NPS) {
          ok = wait(L::bPVDone + static_cast<int>(ps), ((ss / NPS) - 1) & 1);
          if (!ok) break;
        }
        *reinterpret_cast<uint4 *>(smem + L::kP + ps * L::kPBuf + (j % SB) * (kKeys8 * kN8) + t * 16) =
            make_uint4(pk[0], pk[1], pk[2], pk[3]);
        fence_proxy_async(); // P is read by the MMA (async proxy)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bPFull + static_cast<int>(ps)));
      }
      if (SB == 2 && wg == 1 && (it.nb & 1) && lane == 0) // no block in the last stage
        mbar_arrive(bar(L::bPFull + static_cast<int>((sg + nst - 1) % NPS)));
      if (!ok) break;
      // ---- row sums: warp butterfly, then the eight warps in order
#pragma unroll
      for (int h = 0; h < G; ++h)
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
      float lw = 0.f;
#pragma unroll
      for (int h = 0; h < G; ++h) lw = lane == h ? l[h] : lw;
      if (lane < 8) s_stat[(par * 8 + warp) * 8 + lane] = lw;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(L::bAuxFree + par));
        mbar_arrive(bar(L::bStat + par));
      }
      if (par == wg) {
        // ---- epilogue: o = O^T / l
        if (!wait(L::bStat + par, (ig >> 1) & 1) || !wait(L::bODone + par, (ig >> 1) & 1)) break;
        tc_fence_after();
        const float e_val = e8m0_value(static_cast<uint32_t>(eref));
        const bool single = it.prow < 0; // one tile: the final row
        const int64_t head0 = static_cast<int64_t>(single ? it.b : it.prow) * a.Hq + it.kvh * G;
        float inv[G], lse_mine = 0.f;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          float ls = s_stat[par * 64 + h];
#pragma unroll
          for (int w = 1; w < 8; ++w) ls = __fadd_rn(ls, s_stat[(par * 8 + w) * 8 + h]);
          inv[h] = ls == 0.f ? 0.f : __frcp_rn(ls);
          const float lse = ls == 0.f ? -INFINITY : __fmul_rn(__fadd_rn(m[h], lg2(ls)), kLn2);
          lse_mine = t == h ? lse : lse_mine;
        }
#pragma unroll
        for (int pp = 0; pp < NP; ++pp) {
          uint32_t o[NL];
          tmem_ld_n<NL>(tO(ig, pp) + lane_base, o);
          tmem_wait_ld();
          if (pp == NP - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::bOFree + par)); // O read
          }
          const int dim = pp * 128 + t;
          if (dim < a.D) {
#pragma unroll
            for (int h = 0; h < G; ++h) {
              const float x = fmaf(__uint_as_float(o[LO + h]), 0.0625f, __uint_as_float(o[h]));
              const float val =
                  __fmul_rn(__fmul_rn(__fmul_rn(x, inv[h]), 1.f / (1 << kBoost8)), e_val);
              if (single)
                a.out[(head0 + h) * a.D + dim] = to_bf16(val);
              else
                a.part_o[(head0 + h) * a.D + dim] = val;
            }
          }
        }
        if (t < G) {
          if (!single) a.part_lse[head0 + t] = lse_mine;
          else if (a.lse) a.lse[head0 + t] = lse_mine;
        }
      }
      sg += nst;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kPVWarp8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

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
__global__ void __launch_bounds__(kMergeWarps8 * 32) merge_decode_fp8_kernel(const AttnArgs a) {
  constexpr int kChunk = V == 4 ? 8 : 4; // states in flight
  const int lane = threadIdx.x & 31;
  grid_dep_wait(); // the partials are complete
  if (a.status[0] & kStatusPlanMismatch) return; // the outputs already hold NaN
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kMergeWarps8 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(a.batch) * a.Hq) return;
  const int b = static_cast<int>(row / a.Hq), h = static_cast<int>(row - static_cast<int64_t>(b) * a.Hq);
  const ReqInfo r = a.reqs[b];
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

template <int G, int LPR>
cudaError_t launch_f8(const DecodeFp8Args &f, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(decode_fp8_kernel<G, LPR>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Smem8<LPR>::kAlloc);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(f.a.n_units * f.a.Hkv, sms)));
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = Smem8<LPR>::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_fp8_kernel<G, LPR>, f);
}

template <int LPR>
cudaError_t launch_f8_g(const DecodeFp8Args &f, cudaStream_t s) {
  switch (f.a.G) {
  case 1: return launch_f8<1, LPR>(f, s);
  case 2: return launch_f8<2, LPR>(f, s);
  case 4: return launch_f8<4, LPR>(f, s);
  case 8: return launch_f8<8, LPR>(f, s);
  default: return cudaErrorInvalidValue;
  }
}

} // namespace

cudaError_t launch_plan_decode_fp8(const PlanArgs &p, UnitFp8 *units, cudaStream_t s) {
  return launch_chained(plan_decode_fp8_kernel, 1, kPlanThreads8, s, p, units);
}

cudaError_t launch_merge_decode_fp8(const AttnArgs &a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.batch) * a.Hq;
  const int64_t grid = (rows + kMergeWarps8 - 1) / kMergeWarps8;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return a.D <= 128 ? launch_chained(merge_decode_fp8_kernel<4>, static_cast<unsigned>(grid),
                                     kMergeWarps8 * 32, s, a)
                    : launch_chained(merge_decode_fp8_kernel<8>, static_cast<unsigned>(grid),
                                     kMergeWarps8 * 32, s, a);
}

cudaError_t launch_decode_fp8(const DecodeFp8Args &f, cudaStream_t s) {
  if (f.a.n_units == 0) return cudaSuccess;
  if (f.a.D == 64) return launch_f8_g<4>(f, s);
  if (f.a.D <= 128) return launch_f8_g<8>(f, s);
  return launch_f8_g<16>(f, s);
}

} // namespace bia
