// Split-KV decode of one query token per request over the 8-bit paged cache
// (fp8.cuh states the format) on the tensor cores, with the fixed split-KV
// tiles and ascending merge of the bf16 decode ("sglang PR #10417 [POC]
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
// 2^-10 of the largest.  The key's scale multiplies its score, the value's
// scale its weight, relative to the block maximum of the value scales (a
// power of two: exact).  Products, sums, the running maximum and the row sum
// are fp32.  Converting the rows instead (8 -> 16 bits through registers and
// shared memory) would cost more issue slots than the copies themselves.
//
// HBM bound: D + 1 bytes per key, head and cache.  At 6.5 TB/s an SM has
// ~1450 cycles for a 128-key block of head_dim 128, half of what the bf16
// decode has, so a block's latency chain (S, maximum, weights, P.V) does not
// fit one after the other: two softmax warpgroups take alternate blocks, each
// with its own running state and accumulator, joined in the item's epilogue
// (the assignment goes by the block's index in its split, so the bits depend
// on the split alone).
//
// Persistent: one CTA per SM takes (unit, kv head) items from a counter and
// posts them to its roles through a mailbox, as the bf16 decode does.  Roles:
// warps 0-3 and 4-7 softmax + epilogue (WG 0 even blocks, WG 1 odd blocks;
// the epilogue alternates by item), 8 issues P.V (owns TMEM), 9 issues S, 10-13
// hand over the scales of a block's keys and the q rows, 14.. copy (16-byte
// cp.async into the swizzled operand layout, page indices a block ahead).  S
// and P.V come from two threads because each waits for its own inputs: from
// one, S of a later block waited in front of a P.V that was ready (head_dim
// 256, whose rings hold three blocks: 2.8 TB/s).  S also runs ahead into the
// next item.
#include <algorithm>

#include "bia_internal.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace bia {

namespace {

constexpr int kKeys8 = 128;            // keys per block: the MMAs' M
constexpr int kPiece8 = kKeys8 * 128;  // 128 rows x 128 codes, SW128
constexpr int kN8 = 16;                // the MMAs' N: hi and lo of up to 8 heads
constexpr int kPVWarp8 = 8;
constexpr int kSWarp8 = 9;
constexpr int kAuxWarp8 = 10;          // four warps: thread t is key t
constexpr int kCopyWarp8 = 14;
constexpr int kCopyWarps8 = 8;
constexpr int kThreads8 = (kCopyWarp8 + kCopyWarps8) * 32;
constexpr int kCopyThreads8 = kCopyWarps8 * 32;
constexpr int kReaders8 = kThreads8 / 32;         // warps that read the mailbox
constexpr int kCopyKeys8 = kKeys8 / kCopyWarps8;  // keys of a block a copy warp takes
constexpr int kScaleSlots8 = 8;
// The running maximum moves when a block exceeds it by 2^4: weights stay
// below 2^4, and 2^4 more fills e4m3's range (448).
constexpr float kLazy8 = 4.0f;
constexpr int kBoost8 = 4;

// LPR: lanes (16-byte chunks) per row: 4 (head_dim 64), 8 (96, 128), 16 (256)
template <int LPR>
struct Smem8 {
  static constexpr int NP = LPR > 8 ? 2 : 1; // 128-code pieces of a row
  static constexpr int kStage = NP * kPiece8;
  static constexpr int NS = NP == 1 ? 6 : 3; // blocks in the key ring and in the value ring
  static constexpr int kKRing = 0;
  static constexpr int kVRing = kKRing + NS * kStage;
  static constexpr int kQBuf = NP * kN8 * 128;
  static constexpr int kQ = kVRing + NS * kStage; // 2 q buffers
  static constexpr int kPBuf = kKeys8 * kN8;
  static constexpr int kP = kQ + 2 * kQBuf;       // [WG][2]
  static constexpr int kKs = kP + 4 * kPBuf;      // float [slot][128]
  static constexpr int kVe = kKs + kScaleSlots8 * 512; // uint8 [slot][128]
  static constexpr int kEmax = kVe + kScaleSlots8 * 128; // int [slot][4]
  static constexpr int kQs = kEmax + kScaleSlots8 * 16;  // float [2][8]
  static constexpr int kRed = kQs + 64;           // float [WG][2][4][8]
  static constexpr int kLred = kRed + 512;        // float [WG][4][8]
  static constexpr int kStat = kLred + 256;       // float [2][WG][2][8] m, l; then int [2][WG] E
  static constexpr int kStatE = kStat + 256;
  static constexpr int kItems = kStatE + 16;      // int64 [4]
  static constexpr int kSlot = kItems + 32;
  static constexpr int kBar = kSlot + 16;
  static constexpr int bKFull = 0, bKEmpty = bKFull + NS, bVFull = bKEmpty + NS,
                       bVEmpty = bVFull + NS, bQFull = bVEmpty + NS, bQEmpty = bQFull + 2,
                       bSFull = bQEmpty + 2, bPFull = bSFull + 4, bPVDone = bPFull + 4,
                       bODone = bPVDone + 4, bOFree = bODone + 2, bStat = bOFree + 2,
                       bScFull = bStat + 2, bScEmpty = bScFull + kScaleSlots8,
                       bItemFull = bScEmpty + kScaleSlots8, bItemEmpty = bItemFull + 4,
                       kNumBars = bItemEmpty + 4;
  static constexpr int kAlloc = kBar + kNumBars * 8 + 1024;
  static_assert(kAlloc <= 232448, "shared memory per CTA");
  static_assert(kQ % 1024 == 0 && kQBuf % 1024 == 0, "q on the swizzle period");
};

// Work item w: unit w / Hkv, kv head w % Hkv.
struct Item8 {
  bool live;
  int kvh;
  Unit u;
  ReqInfo r;
  int32_t key_begin, key_end;
  int nb; // 128-key blocks
};

__device__ __forceinline__ Item8 item8(const AttnArgs &a, int64_t w) {
  Item8 it;
  const int64_t unit = w / a.Hkv;
  it.kvh = static_cast<int>(w - unit * a.Hkv);
  it.u = a.units[unit];
  it.live = it.u.b >= 0;
  it.nb = 0;
  if (!it.live) return it;
  it.r = a.reqs[it.u.b];
  it.key_begin = it.u.split * a.split;
  it.key_end = min(it.key_begin + a.split, it.r.kv_len);
  it.nb = (it.key_end - it.key_begin + kKeys8 - 1) / kKeys8;
  return it;
}

template <int NL>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t (&r)[NL]) {
  if constexpr (NL == 8) tmem_ld8(taddr, r);
  else tmem_ld16(taddr, r);
}
template <int NL>
__device__ __forceinline__ void tmem_st_n(uint32_t taddr, const uint32_t (&r)[NL]) {
  if constexpr (NL == 8) tmem_st8(taddr, r);
  else tmem_st16(taddr, r);
}

template <int G, int LPR>
__global__ void __launch_bounds__(kThreads8, 1)
    decode_fp8_kernel(const __grid_constant__ DecodeFp8Args f) {
  using L = Smem8<LPR>;
  constexpr int NP = L::NP, NS = L::NS;
  constexpr int LO = G <= 4 ? 4 : 8; // column of a head's second term
  constexpr int NL = 2 * LO;         // columns in use
  constexpr uint32_t kIdescS = idesc_e4m3(128, kN8, false, false);
  constexpr uint32_t kIdescPV = idesc_e4m3(128, kN8, true, true);
  constexpr uint32_t kTmemCols = NP == 1 ? 128 : 256;
  const AttnArgs &a = f.a;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + L::kBar + 8u * static_cast<uint32_t>(i); };
  auto kstage = [&](int s) { return sbase + L::kKRing + static_cast<uint32_t>(s) * L::kStage; };
  auto vstage = [&](int s) { return sbase + L::kVRing + static_cast<uint32_t>(s) * L::kStage; };
  auto qbuf = [&](int i) { return sbase + L::kQ + static_cast<uint32_t>(i) * L::kQBuf; };
  auto pbuf = [&](int w, uint32_t c) {
    return sbase + L::kP + (2u * static_cast<uint32_t>(w) + (c & 1u)) * L::kPBuf;
  };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kSlot);

  const int64_t n_work = a.n_units * a.Hkv;
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
      mbar_init(bar(L::bQFull + i), 4);      // the aux warps
      mbar_init(bar(L::bQEmpty + i), 1 + 8); // the S MMAs, the softmax warps
      mbar_init(bar(L::bODone + i), 1);
      mbar_init(bar(L::bOFree + i), 4);
      mbar_init(bar(L::bStat + i), 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(L::bSFull + i), 1);
      mbar_init(bar(L::bPFull + i), 4);
      mbar_init(bar(L::bPVDone + i), 1);
      mbar_init(bar(L::bItemFull + i), 1);
      mbar_init(bar(L::bItemEmpty + i), kReaders8);
    }
    for (int i = 0; i < kScaleSlots8; ++i) {
      mbar_init(bar(L::bScFull + i), 4);
      mbar_init(bar(L::bScEmpty + i), 4);
    }
    fence_mbar_init();
  }
  grid_dep_launch(); // the merge may start launching
  grid_dep_wait();   // the plan is complete (all of the above ran beside it)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // TMEM columns: S^T buffers [WG][2] (lanes = keys) at 0..63, O^T buffers
  // [item parity][WG][piece] (lanes = dims) from 64
  auto tS = [&](int w, uint32_t c) {
    return tmem + 16u * (2u * static_cast<uint32_t>(w) + (c & 1u));
  };
  auto tO = [&](uint32_t ig, int w, int p) {
    return tmem + 64u + 16u * (((ig & 1u) * 2u + static_cast<uint32_t>(w)) * NP + p);
  };
  volatile int64_t *items = reinterpret_cast<volatile int64_t *>(smem + L::kItems);
  // the k-th item of this CTA (-1: no more, or a wait that ran out); read by a
  // whole warp, or by one thread (single)
  auto read_item = [&](uint32_t k, bool single) -> int64_t {
    const int s = static_cast<int>(k & 3u);
    int64_t w = -1;
    if (mbar_wait(bar(L::bItemFull + s), (k >> 2) & 1u, a.status)) w = items[s];
    if (!single) __syncwarp();
    if (single || lane == 0) mbar_arrive(bar(L::bItemEmpty + s));
    return w;
  };

  if (warp >= kCopyWarp8) {
    // ------------------------------------------------------------ copies
    // A warp takes 16 keys of a block; lane l < 16 finds the row of one (its
    // page index a block ahead) and hands it round, then the lanes copy chunk
    // cc of every (32 / LPR)-th key.
    const int pt = tid - kCopyWarp8 * 32;
    const int cc = lane % LPR, kb = lane / LPR;
    const int key_w = (pt >> 5) * kCopyKeys8; // the warp's first key of a block
    const int page_mask = (1 << a.page_shift) - 1;
    const bool in_row = cc * 16 < a.D; // head_dim 96: six of eight lanes
    const uint32_t piece_off = static_cast<uint32_t>(cc >> 3) * kPiece8;
    uint32_t jg = 0;
    bool ok = true;
    // copy thread 0 fetches the items: the first is the CTA's own index, each
    // next one is taken from the counter when the current item starts and
    // posted once the item's first block of copies is issued
    const bool fetcher = pt == 0;
    if (fetcher) {
      items[0] = blockIdx.x < n_work ? static_cast<int64_t>(blockIdx.x) : -1;
      mbar_arrive(bar(L::bItemFull + 0));
    }
    int32_t taken = 0;
    bool posted = false;
    auto post_next = [&](uint32_t k) { // item k + 1
      if (!fetcher || posted) return;
      posted = true;
      int64_t nw = static_cast<int64_t>(gridDim.x) + taken;
      if (nw >= n_work) nw = -1;
      const uint32_t kn = k + 1;
      if (kn >= 4 && !mbar_wait(bar(L::bItemEmpty + (kn & 3u)), ((kn >> 2) - 1) & 1u, a.status))
        nw = -1;
      items[kn & 3u] = nw;
      mbar_arrive(bar(L::bItemFull + (kn & 3u)));
    };
    for (uint32_t k = 0; ok; ++k) {
      const int64_t w = read_item(k, false);
      if (w < 0) break;
      if (fetcher) taken = atomicAdd(a.status + kStatusWorkCounter, 1);
      posted = false;
      const Item8 it = item8(a, w);
      if (!it.live) {
        post_next(k);
        continue;
      }
      const int32_t key_l = lane < kCopyKeys8 ? it.key_begin + key_w + lane : INT32_MAX / 2;
      auto page_of = [&](int32_t key) { // -1: no such key
        return key < it.key_end ? __ldg(a.kv_indices + it.r.page_base + (key >> a.page_shift)) : -1;
      };
      int32_t page = page_of(key_l);
      for (int j = 0; j < it.nb; ++j, ++jg) {
        const int32_t key = key_l + j * kKeys8;
        const bool good = page >= 0 && page < a.num_pages;
        if (key < it.key_end && !good) atomicOr(a.status, kStatusBadPage);
        // the lane's row (-1: zeros)
        const int64_t row = good ? ((static_cast<int64_t>(page) << a.page_shift) +
                                    (key & page_mask)) * a.Hkv + it.kvh
                                 : -1;
        page = page_of(key + kKeys8); // in flight while this block's copies are issued
        const int s = static_cast<int>(jg % NS);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (jg >= static_cast<uint32_t>(NS) &&
              !mbar_wait(bar((kv == 0 ? L::bKEmpty : L::bVEmpty) + s), ((jg / NS) - 1) & 1,
                         a.status)) {
            ok = false;
            break;
          }
          const uint32_t base = (kv == 0 ? kstage(s) : vstage(s)) + piece_off;
          const uint8_t *src = (kv == 0 ? f.k_codes : f.v_codes) + cc * 16;
#pragma unroll
          for (int i = 0; i < kCopyKeys8 * LPR / 32; ++i) {
            const int kk = i * (32 / LPR) + kb; // key of the warp's 16
            const int64_t r = __shfl_sync(0xffffffffu, row, kk);
            const int k8 = key_w + kk;
            if (in_row)
              cp_async16(base + static_cast<uint32_t>(k8) * 128 +
                             ((static_cast<uint32_t>(cc & 7) ^ static_cast<uint32_t>(k8 & 7)) << 4),
                         src + (r < 0 ? 0 : r * a.D), r >= 0);
          }
          cp_async_arrive(bar((kv == 0 ? L::bKFull : L::bVFull) + s));
        }
        if (!ok) break;
        post_next(k); // after the first block
      }
      post_next(k);
    }
    cp_async_wait_all(); // no copy outlives the CTA
  } else if (warp >= kAuxWarp8) {
    // ------------------------------------------------------------ scales and q
    // Thread t hands key t's scales of each block to the softmax, up to
    // kScaleSlots8 blocks ahead (the page index two blocks ahead, the bytes
    // one); aux warp w also splits the q rows of heads w, w + 4.
    const int aw = warp - kAuxWarp8, t = aw * 32 + lane;
    const int page_mask = (1 << a.page_shift) - 1;
    float *s_ks = reinterpret_cast<float *>(smem + L::kKs);
    uint8_t *s_ve = smem + L::kVe;
    int32_t *s_emax = reinterpret_cast<int32_t *>(smem + L::kEmax);
    float *s_qs = reinterpret_cast<float *>(smem + L::kQs);
    uint32_t jg = 0, ig = 0;
    bool ok = true;
    for (uint32_t k = 0; ok; ++k) {
      const int64_t w = read_item(k, false);
      if (w < 0) break;
      const Item8 it = item8(a, w);
      if (!it.live) continue;
      auto page_of = [&](int j) {
        const int32_t key = it.key_begin + j * kKeys8 + t;
        return key < it.key_end ? __ldg(a.kv_indices + it.r.page_base + (key >> a.page_shift)) : -1;
      };
      // scale bytes of block j's key (past the end or on a bad page: zeros
      // with a zero weight, outside the block's maximum)
      auto bytes_of = [&](int j, int32_t page, uint32_t &kb, uint32_t &vb) {
        kb = vb = 0;
        if (page >= 0 && page < a.num_pages) {
          const int32_t key = it.key_begin + j * kKeys8 + t;
          const int64_t row =
              ((static_cast<int64_t>(page) << a.page_shift) + (key & page_mask)) * a.Hkv + it.kvh;
          kb = __ldg(f.k_scale + row);
          vb = __ldg(f.v_scale + row);
        }
      };
      int32_t pg1 = page_of(0), pg2 = page_of(1);
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
                a.q + (static_cast<int64_t>(it.r.q_start) * a.Hq + it.kvh * G + h) * a.D + col));
        }
      uint32_t kb, vb;
      bytes_of(0, pg1, kb, vb);
      if (ig >= 2 && !mbar_wait(bar(L::bQEmpty + (ig & 1)), ((ig >> 1) - 1) & 1, a.status)) break;
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
            float v[4], b[4];
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = x[p][c] * inv;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              hi[c] = e4m3x2(v[2 * c], v[2 * c + 1]);
              e4m3x2_values(hi[c], b[2 * c], b[2 * c + 1]);
              lo[c] = e4m3x2((v[2 * c] - b[2 * c]) * 16.f, (v[2 * c + 1] - b[2 * c + 1]) * 16.f);
            }
            if (p * 128 + col < a.D) {
              uint8_t *q0 = smem + L::kQ + (ig & 1) * L::kQBuf + p * (kN8 * 128);
              auto at = [&](int rr) { // row rr, 16-byte chunk col / 16
                return rr * 128 + (((col >> 4) ^ (rr & 7)) << 4) + (col & 15);
              };
              *reinterpret_cast<uint32_t *>(q0 + at(h)) = hi[0] | (hi[1] << 16);
              *reinterpret_cast<uint32_t *>(q0 + at(LO + h)) = lo[0] | (lo[1] << 16);
            }
          }
          if (lane == 0) s_qs[(ig & 1) * 8 + h] = a.scale_log2 * exp2_int(e);
        }
      }
      fence_proxy_async(); // q is read by the MMA (async proxy)
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bQFull + (ig & 1)));
      ++ig;
      for (int j = 0; j < it.nb; ++j, ++jg) {
        const int s = static_cast<int>(jg % kScaleSlots8);
        pg1 = pg2;
        pg2 = page_of(j + 2);
        uint32_t kb1, vb1;
        bytes_of(j + 1, pg1, kb1, vb1);
        if (jg >= kScaleSlots8 &&
            !mbar_wait(bar(L::bScEmpty + s), ((jg / kScaleSlots8) - 1) & 1, a.status)) {
          ok = false;
          break;
        }
        s_ks[s * 128 + t] = e8m0_value(kb);
        s_ve[s * 128 + t] = static_cast<uint8_t>(vb);
        const uint32_t big = __reduce_max_sync(0xffffffffu, vb == 255u ? 0u : vb);
        if (lane == 0) s_emax[s * 4 + aw] = static_cast<int32_t>(big);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bScFull + s));
        kb = kb1;
        vb = vb1;
      }
    }
  } else if (warp == kSWarp8) {
    // ------------------------------------------------------------ S issuer
    if (lane == 0) {
      const int ksteps = a.D / 32 < 4 ? a.D / 32 : 4; // 32-code steps of a piece
      uint32_t jg = 0, ig = 0, cnt[2] = {0, 0};
      bool ok = true;
      for (uint32_t k = 0; ok; ++k) {
        const int64_t w = read_item(k, true);
        if (w < 0) break;
        const Item8 it = item8(a, w);
        if (!it.live) continue;
        const uint32_t qb = qbuf(ig & 1);
        ok = mbar_wait(bar(L::bQFull + (ig & 1)), (ig >> 1) & 1, a.status);
        for (int j = 0; j < it.nb && ok; ++j, ++jg) {
          const int s = static_cast<int>(jg % NS), wg = j & 1;
          const uint32_t c = wg ? cnt[1]++ : cnt[0]++;
          // S buffer c % 2 is free once the softmax has read S(c - 2)
          if (c >= 2)
            ok = mbar_wait(bar(L::bPFull + 2 * wg + (c & 1)), ((c >> 1) - 1) & 1, a.status);
          ok = ok && mbar_wait(bar(L::bKFull + s), (jg / NS) & 1, a.status);
          if (!ok) break;
          fence_proxy_async(); // the rows were written by cp.async (generic proxy)
          tc_fence_after();
#pragma unroll
          for (int p = 0; p < NP; ++p)
            for (int kk = 0; kk < ksteps; ++kk)
              mma_e4m3_ss(tS(wg, c), desc_sw128(kstage(s) + p * kPiece8 + kk * 32, 16, 1024),
                          desc_sw128(qb + p * (kN8 * 128) + kk * 32, 16, 1024), kIdescS,
                          (p | kk) != 0 ? 1u : 0u);
          mma_commit(bar(L::bKEmpty + s));
          mma_commit(bar(L::bSFull + 2 * wg + (c & 1)));
        }
        if (!ok) break;
        mma_commit(bar(L::bQEmpty + (ig & 1)));
        ++ig;
      }
    }
    __syncwarp();
  } else if (warp == kPVWarp8) {
    // ------------------------------------------------------------ P.V issuer
    if (lane == 0) {
      uint32_t jg = 0, ig = 0, cnt[2] = {0, 0};
      bool ok = true;
      for (uint32_t k = 0; ok; ++k) {
        const int64_t w = read_item(k, true);
        if (w < 0) break;
        const Item8 it = item8(a, w);
        if (!it.live) continue;
        // the item's O buffers are free once the epilogue of item ig - 2 read them
        if (ig >= 2) ok = mbar_wait(bar(L::bOFree + (ig & 1)), ((ig >> 1) - 1) & 1, a.status);
        for (int j = 0; j < it.nb && ok; ++j, ++jg) {
          const int s = static_cast<int>(jg % NS), wg = j & 1;
          const uint32_t c = wg ? cnt[1]++ : cnt[0]++;
          ok = mbar_wait(bar(L::bVFull + s), (jg / NS) & 1, a.status) &&
               mbar_wait(bar(L::bPFull + 2 * wg + (c & 1)), (c >> 1) & 1, a.status);
          if (!ok) break;
          fence_proxy_async();
          tc_fence_after();
#pragma unroll
          for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int kk = 0; kk < kKeys8 / 32; ++kk)
              mma_e4m3_ss(tO(ig, wg, p), desc_sw128(vstage(s) + p * kPiece8 + kk * 4096, 16384, 1024),
                          desc_plain(pbuf(wg, c) + kk * 512, 128, 128), kIdescPV,
                          (j > 1 || kk > 0) ? 1u : 0u);
          mma_commit(bar(L::bVEmpty + s));
          mma_commit(bar(L::bPVDone + 2 * wg + (c & 1)));
        }
        if (!ok) break;
        mma_commit(bar(L::bODone + (ig & 1)));
        ++ig;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    // A wait that runs out marks its thread; the warpgroup's named barriers
    // reduce the marks, so its four warps leave at the same barrier.
    const int wg = warp >> 2, qd = warp & 3; // TMEM lanes 32qd .. 32qd+31
    const int t = qd * 32 + lane;            // key of the block, dim of the output
    const uint32_t lane_base = static_cast<uint32_t>(qd * 32) << 16;
    const uint32_t nbar = 1 + wg;
    float *red = reinterpret_cast<float *>(smem + L::kRed) + wg * 64;
    float *lr = reinterpret_cast<float *>(smem + L::kLred) + wg * 32;
    float *stat = reinterpret_cast<float *>(smem + L::kStat); // [parity][WG][m, l][8]
    int32_t *stat_e = reinterpret_cast<int32_t *>(smem + L::kStatE);
    const float *s_ks = reinterpret_cast<const float *>(smem + L::kKs);
    const uint8_t *s_ve = smem + L::kVe;
    const int4 *s_emax = reinterpret_cast<const int4 *>(smem + L::kEmax);
    const float *s_qs = reinterpret_cast<const float *>(smem + L::kQs);
    uint32_t jg = 0, ig = 0, c = 0; // c: blocks this warpgroup has taken
    bool failed = false;            // the same on every thread of the warpgroup
    for (uint32_t k = 0; !failed; ++k) {
      const int64_t w = read_item(k, false);
      if (bar_any_named(nbar, 128, w < 0)) break;
      const Item8 it = item8(a, w);
      if (!it.live) continue;
      bool bad = !mbar_wait(bar(L::bQFull + (ig & 1)), (ig >> 1) & 1, a.status);
      float m[G], l[G], qs[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
        qs[h] = s_qs[(ig & 1) * 8 + h];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::bQEmpty + (ig & 1)));
      int32_t eref = -1; // value-scale byte the accumulator is relative to
      for (int j = wg; j < it.nb; j += 2, ++c) {
        const uint32_t jj = jg + j;
        const int ss = static_cast<int>(jj % kScaleSlots8);
        bad = bad || !mbar_wait(bar(L::bScFull + ss), (jj / kScaleSlots8) & 1, a.status);
        const float ks = s_ks[ss * 128 + t];
        const uint32_t ve = s_ve[ss * 128 + t];
        const int4 em = s_emax[ss];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bScEmpty + ss));
        bad = bad || !mbar_wait(bar(L::bSFull + 2 * wg + (c & 1)), (c >> 1) & 1, a.status);
        tc_fence_after();
        uint32_t v[NL];
        if (__any_sync(0xffffffffu, bad)) {
          bad = true;
#pragma unroll
          for (int i = 0; i < NL; ++i) v[i] = 0;
        } else {
          tmem_ld_n<NL>(tS(wg, c) + lane_base, v);
          tmem_wait_ld();
        }
        const bool valid = it.key_begin + j * kKeys8 + t < it.key_end;
        float s[G], p[G];
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float raw = fmaf(__uint_as_float(v[LO + h]), 0.0625f, __uint_as_float(v[h]));
          s[h] = valid ? raw * (ks * qs[h]) : -INFINITY;
        }
        // weights against the running max while the block max is exchanged
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float ms = m[h] == -INFINITY ? 0.f : m[h];
          p[h] = s[h] == -INFINITY ? 0.f : ex2(s[h] - ms);
        }
        float *rd = red + (c & 1) * 32;
        float mine = -INFINITY;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float wm = warp_max(s[h]);
          mine = lane == h ? wm : mine;
        }
        if (lane < G) rd[qd * 8 + lane] = mine;
        if (bar_any_named(nbar, 128, bad)) {
          failed = true;
          break;
        }
        uint32_t up = 0; // heads whose running max moves (the same on every thread)
        float bmv[G], alpha[G];
#pragma unroll
        for (int h = 0; h < G; ++h) {
          bmv[h] = fmaxf(fmaxf(rd[h], rd[8 + h]), fmaxf(rd[16 + h], rd[24 + h]));
          alpha[h] = 1.f;
          if (bmv[h] > m[h] + kLazy8 || (m[h] == -INFINITY && bmv[h] != -INFINITY)) up |= 1u << h;
        }
        if (up != 0) {
#pragma unroll
          for (int h = 0; h < G; ++h) {
            if ((up >> h) & 1u) {
              alpha[h] = ex2(m[h] - bmv[h]); // 0 when m == -inf
              m[h] = bmv[h];
              p[h] = s[h] == -INFINITY ? 0.f : ex2(s[h] - m[h]);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < G; ++h) l[h] = fmaf(l[h], alpha[h], p[h]);
        const int32_t eb = max(max(em.x, em.y), max(em.z, em.w));
        const bool e_up = eb > eref;
        const float e_down = e_up && eref >= 0 ? exp2_int(max(eref - eb, -126)) : 1.f;
        if (e_up) eref = eb;
        // P buffer c % 2 is free once P.V(c - 2) is done; O may be rescaled
        // once P.V(c - 1) is done
        if (c >= 2)
          bad = bad ||
                !mbar_wait(bar(L::bPVDone + 2 * wg + (c & 1)), ((c >> 1) - 1) & 1, a.status);
        if (j > wg && (up != 0 || e_down != 1.f)) {
          bad = bad || !mbar_wait(bar(L::bPVDone + 2 * wg + ((c - 1) & 1)), ((c - 1) >> 1) & 1,
                                  a.status);
          tc_fence_after();
          if (!__any_sync(0xffffffffu, bad)) {
#pragma unroll
            for (int pp = 0; pp < NP; ++pp) {
              uint32_t o[NL];
              tmem_ld_n<NL>(tO(ig, wg, pp) + lane_base, o);
              tmem_wait_ld();
#pragma unroll
              for (int h = 0; h < G; ++h) {
                const float x = alpha[h] * e_down;
                o[h] = __float_as_uint(__uint_as_float(o[h]) * x);
                o[LO + h] = __float_as_uint(__uint_as_float(o[LO + h]) * x);
              }
              tmem_st_n<NL>(tO(ig, wg, pp) + lane_base, o);
            }
            tmem_wait_st();
          }
        }
        if (bad) continue; // the next barrier takes everyone out
        // weight times 2^(ev - eref + 6), in two e4m3 terms
        const int32_t de = static_cast<int32_t>(ve) - eref + kBoost8 + 127;
        const float vf = ve == 255u ? NAN : de > 0 ? __uint_as_float(de << 23) : 0.f;
        uint32_t pk[4] = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < G; h += 2) {
          const float w0 = p[h] * vf, w1 = h + 1 < G ? p[h + 1 < G ? h + 1 : h] * vf : 0.f;
          const uint32_t hi = e4m3x2(w0, w1);
          float b0, b1;
          e4m3x2_values(hi, b0, b1);
          const uint32_t lo = e4m3x2((w0 - b0) * 16.f, (w1 - b1) * 16.f);
          pk[h >> 2] |= hi << (8 * (h & 3));
          pk[(LO + h) >> 2] |= lo << (8 * (h & 3));
        }
        *reinterpret_cast<uint4 *>(smem + L::kP + (2 * wg + (c & 1)) * L::kPBuf + t * 16) =
            make_uint4(pk[0], pk[1], pk[2], pk[3]);
        fence_proxy_async(); // P is read by the MMA (async proxy)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bPFull + 2 * wg + (c & 1)));
      }
      if (failed) break;

      // ---- the warpgroup's state: row sums over its threads (warp butterfly,
      // then the four warps in order), its maxima and its scale reference
#pragma unroll
      for (int h = 0; h < G; ++h)
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
      float lw = 0.f, mw = 0.f;
#pragma unroll
      for (int h = 0; h < G; ++h) {
        lw = lane == h ? l[h] : lw;
        mw = lane == h ? m[h] : mw;
      }
      // the epilogue of item ig - 2 (the other reader of this slot) is done:
      // its OFree preceded this item's first MMA
      if (bar_any_named(nbar, 128, bad)) {
        failed = true;
        break;
      }
      if (lane < G) lr[qd * 8 + lane] = lw;
      bar_sync_named(nbar, 128);
      float *st = stat + ((ig & 1) * 2 + wg) * 16;
      if (t < G) {
        st[t] = mw;
        st[8 + t] = __fadd_rn(__fadd_rn(__fadd_rn(lr[t], lr[8 + t]), lr[16 + t]), lr[24 + t]);
      }
      if (t == 0) stat_e[(ig & 1) * 2 + wg] = eref;
      if (qd == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bStat + (ig & 1)));
      }
      if (static_cast<int>(ig & 1) == wg) {
        // ---- epilogue of this item: the two states joined, o = O^T / l
        bad = !mbar_wait(bar(L::bStat + (ig & 1)), (ig >> 1) & 1, a.status) ||
              !mbar_wait(bar(L::bODone + (ig & 1)), (ig >> 1) & 1, a.status);
        if (bar_any_named(nbar, 128, bad)) {
          failed = true;
          break;
        }
        tc_fence_after();
        const float *s0 = stat + (ig & 1) * 32, *s1 = s0 + 16;
        const int32_t e0 = stat_e[(ig & 1) * 2], e1 = stat_e[(ig & 1) * 2 + 1];
        const bool two = it.nb > 1; // the odd blocks' state exists
        const int32_t em = two ? max(e0, e1) : e0;
        const float g0 = exp2_int(max(e0 - em, -126));
        const float g1 = two ? exp2_int(max(e1 - em, -126)) : 0.f;
        const float e_val = __fmul_rn(e8m0_value(static_cast<uint32_t>(em)), 1.f);
        float f0[G], f1[G], lse_mine = 0.f;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float m0 = s0[h], m1 = two ? s1[h] : -INFINITY;
          const float M = fmaxf(m0, m1);
          const float a0 = m0 == M ? 1.f : ex2(m0 - M);
          const float a1 = !two ? 0.f : m1 == M ? 1.f : ex2(m1 - M);
          const float ls = two ? __fadd_rn(__fmul_rn(a0, s0[8 + h]), __fmul_rn(a1, s1[8 + h]))
                               : s0[8 + h];
          const float inv = ls == 0.f ? 0.f : __frcp_rn(ls);
          f0[h] = __fmul_rn(__fmul_rn(a0, g0), inv);
          f1[h] = __fmul_rn(__fmul_rn(a1, g1), inv);
          const float lse = ls == 0.f ? -INFINITY : __fmul_rn(__fadd_rn(M, lg2(ls)), kLn2);
          lse_mine = t == h ? lse : lse_mine;
        }
        const bool single = (it.r.kv_len - 1) / a.split == 0; // one split: the final row
        const int64_t head0 = static_cast<int64_t>(it.r.q_start) * a.Hq + it.kvh * G;
        const int64_t prow0 = (it.r.rowbase + it.u.split) * static_cast<int64_t>(a.Hq) + it.kvh * G;
#pragma unroll
        for (int pp = 0; pp < NP; ++pp) {
          uint32_t o0[NL], o1[NL];
          tmem_ld_n<NL>(tO(ig, 0, pp) + lane_base, o0);
          if (two) tmem_ld_n<NL>(tO(ig, 1, pp) + lane_base, o1);
          tmem_wait_ld();
          if (pp == NP - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::bOFree + (ig & 1))); // O read
          }
          const int dim = pp * 128 + t;
          if (dim < a.D) {
#pragma unroll
            for (int h = 0; h < G; ++h) {
              const float x0 =
                  fmaf(__uint_as_float(o0[LO + h]), 0.0625f, __uint_as_float(o0[h]));
              float val = __fmul_rn(x0, f0[h]);
              if (two) {
                const float x1 =
                    fmaf(__uint_as_float(o1[LO + h]), 0.0625f, __uint_as_float(o1[h]));
                val = __fmaf_rn(x1, f1[h], val);
              }
              val = __fmul_rn(__fmul_rn(val, 1.f / (1 << kBoost8)), e_val);
              if (single)
                a.out[(head0 + h) * a.D + dim] = to_bf16(val);
              else
                a.part_o[(prow0 + h) * a.D + dim] = val;
            }
          }
        }
        if (t < G) {
          if (single) {
            if (a.lse) a.lse[head0 + t] = lse_mine;
          } else {
            a.part_lse[prow0 + t] = lse_mine;
          }
        }
      }
      jg += it.nb;
      ++ig;
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

__global__ void __launch_bounds__(kPlanThreads8) plan_decode_fp8_kernel(const PlanArgs p) {
  __shared__ int64_t s_warp[kPlanThreads8 / 32];
  __shared__ int32_t s_off[kPlanThreads8 + 1]; // first unit of each request of the chunk
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
    for (int64_t i = tid; i < p.n_units_expected; i += kPlanThreads8) p.units[i] = Unit{-1, 0, 0, 0};
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
      p.units[unit0 + i] = Unit{b0 + lo, 0, i - s_off[lo], 1};
    }
    unit0 += n;
    row0 += total >> 32;
  }
  for (int64_t i = unit0 + tid; i < p.n_units_expected; i += kPlanThreads8)
    p.units[i] = Unit{-1, 0, 0, 0}; // a bounded launch has room for more
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

cudaError_t launch_plan_decode_fp8(const PlanArgs &p, cudaStream_t s) {
  return launch_chained(plan_decode_fp8_kernel, 1, kPlanThreads8, s, p);
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
