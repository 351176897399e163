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
// below.  The key's scale multiplies its score.  The value's scale 2^ev
// multiplies its weight: P holds p_j * 2^(ev_j - c + 8), with c the integer
// nearest to the largest of (score + ev) less the largest score, each over the
// part's keys, so that a head's largest entry lies about 2^8 (2^7.5 .. 2^8.5;
// e4m3 ends at 2^8.8).  An entry keeps 8 significant bits (what a bf16 weight
// keeps) down to 2^-6 and is off by at most 2^-14, 2^-21 of the largest, below:
// only what adds little to the result is held coarsely.  (Scaled by the part's largest value scale instead,
// a row 2^22 times the others in magnitude took every bit from them, attended
// or not.)  Products, sums, the maxima and the row sum are fp32.
// Converting the rows instead (8 -> 16 bits through registers and shared
// memory) would cost more issue slots than the copies themselves.
//
// HBM bound at 128 and 256 columns with up to 4 heads a group: D + 1 bytes per
// key, head and cache (64 requests of 1024 to 32768 keys, 8 kv heads x 128, page
// 16: 6.1 TB/s with 2 heads a group, 5.8 with 4).  Narrower heads and 8 heads a
// group are bound by the softmax warps, whose time for a part hardly depends on
// its bytes: 64 columns 344 us where 128 take 390 (3.3 TB/s), 96 378 us (4.5),
// 8 heads a group 456 us (5.0).  At 6.5 TB/s an SM has
// ~1450 cycles for a 128-key block of one 128-wide head, half of what the bf16
// decode has, and an online softmax does not fit: per block its chain of
// waits, maximum exchange and rescaling took ~5000 cycles of a warpgroup, 3.8
// TB/s with two of them on alternate blocks.  So a tile (at most 1024 keys)
// is taken in parts of 512 keys, and a part in two passes: all its scores
// first, kept in TMEM, the maxima over the part, then the weights.  Nothing
// is rescaled, the entries of P fill e4m3's range, and
// the warps meet once a part; the parts' states (each with its own O columns)
// are joined in the epilogue.  Key and value rows are copied by warps of their
// own through a ring of their own each (one ring for both would let S of the
// next part wait on a stage two uses ahead, which an mbarrier's parity cannot
// tell from the use before).
//
// HB = 2: an item takes two neighbouring kv heads (an even number of kv heads,
// head_dim up to 128).  Their rows lie side by side, and a page-1 cache read
// in random token order gives 5.0 TB/s in segments of 128 bytes but 6.5 in
// segments of 256 (a plain copy loop of the same pattern); a key's row and
// scales are looked up once for both.  Each softmax warpgroup then has a head
// of its own; with HB = 1 the two take even and odd blocks.
//
// Persistent: one CTA per SM takes (tile, kv heads) items from a counter.
// Warps 0-3 and 4-7 softmax + epilogue, 8 issues P.V (owns TMEM), 9 issues S,
// 10-13 prepare: the rows and scales of a part's keys, the item's q; 14-21 and
// 22-29 copy keys and values (16-byte cp.async into the swizzled operand
// layout), 30 takes the items and posts them through a mailbox in shared
// memory, one ahead of the copies.
// An item's result depends on its own keys alone, whichever CTA takes it.
// Up to 32 requests with splits to merge and an SM for every item have no plan:
// each CTA's item warp works its only item out of the index arrays, and notes
// errors in a status word of its own (one request of 4097 keys: 21 -> 19 us, 4
// us less on the host).
#pragma once

#include <algorithm>

#include "bia_internal.h"
#include "fp8.cuh"
#include "ptx.cuh"

namespace bia {

namespace {

constexpr int kKeys8 = 128;           // keys per block: the MMAs' M
constexpr int kPiece8 = kKeys8 * 128; // 128 rows x 128 codes, SW128
constexpr int kN8 = 16;               // the MMAs' N: hi and lo of up to 8 heads
constexpr int kPart8 = 512;           // keys of a part
constexpr int kPartBlocks8 = kPart8 / kKeys8;
constexpr int kParts8 = BIA_DECODE_FP8_SPLIT / kPart8; // parts of a tile
static_assert(kParts8 == 2, "the epilogue joins two parts");
constexpr int kPVWarp8 = 8;
constexpr int kSWarp8 = 9;
constexpr int kAuxWarp8 = 10;
constexpr int kCopyWarp8 = 14;
constexpr int kCopyWarps8 = 8;                           // for keys, and as many for values
constexpr int kItemWarp8 = kCopyWarp8 + 2 * kCopyWarps8;
constexpr int kThreads8 = 1024; // the last warp idles
constexpr int kCopyThreads8 = kCopyWarps8 * 32;
// Registers of the softmax warps and of the others: 8 * 112 + 24 * 48 = 32 * 64,
// what the launch has
constexpr int kSoftRegs8 = 112, kOtherRegs8 = 48;
static_assert(8 * kSoftRegs8 + (kThreads8 / 32 - 8) * kOtherRegs8 <= 65536 / 32, "register split");
static_assert(kItemWarp8 < kThreads8 / 32, "warps");
constexpr int kCopyKeys8 = kKeys8 / kCopyWarps8; // keys of a block a copy warp takes
constexpr int kReaders8 = kItemWarp8;            // warps that read the mailbox
constexpr int kMaxima8 = 20; // 8 heads' scores, 8 score + ev, the ev, up to 16 bytes
constexpr int kBoost8 = 8; // entries of P are at most 2^8.5: e4m3 ends at 448
constexpr uint32_t kNoRow8 = 0xffffffffu; // a key past the end or on a bad page: zeros

// DW: 64, 128 (head_dim 96 too) or 256; HB: kv heads of an item.
template <int DW, int HB>
struct Smem8 {
  static constexpr int NP = DW * HB > 128 ? 2 : 1; // 128-code pieces of a key's rows
  static constexpr int PH = DW == 256 ? 2 : 1;     // pieces of a head
  static constexpr int LPR = DW * HB / 16;         // lanes (16-byte chunks) per key
  // A ring stage holds SB blocks: two for rows of up to 128 codes, so that a
  // barrier is waited for (~300 cycles even when it is complete) and the
  // async proxy fenced every 32 KB
  static constexpr int SB = NP == 1 ? 2 : 1;
  static constexpr int kStages = kPartBlocks8 / SB; // of a part
  static constexpr int kBlock = NP * kPiece8;
  static constexpr int kStage = SB * kBlock;
  static constexpr int NS = 3; // stages in the key ring and in the value ring
  static constexpr int kKRing = 0;
  static constexpr int kVRing = kKRing + NS * kStage;
  static constexpr int kQBuf = NP * kN8 * 128;
  static constexpr int kQ = kVRing + NS * kStage; // [2]
  static constexpr int kPBlock = kKeys8 * kN8;    // P of one head and block
  static constexpr int kP = kQ + 2 * kQBuf;       // [block][HB]
  static constexpr int kRows = kP + kPartBlocks8 * HB * kPBlock; // uint32 [2][part]: cache rows
  static constexpr int kKe = kRows + 2 * kPart8 * 4;   // uint8 [2][HB][part]: key scales
  static constexpr int kVe = kKe + 2 * HB * kPart8;    // uint8 [2][HB][part]: value scales
  static constexpr int kQs = kVe + 2 * HB * kPart8; // float [2][HB][8]
  static constexpr int kMax = kQs + 2 * HB * 32;  // int [3][HB][kMaxima8]: a part's maxima
  static constexpr int kStat = kMax + 3 * HB * kMaxima8 * 4; // float [2][8 warps][8]
  static constexpr int kStatM = kStat + 512;      // float [2][HB][8] maximum, then as many c
  static constexpr int kItems = (kStatM + 4 * HB * 32 + 31) / 32 * 32; // 32-byte records [4]
  static constexpr int kSlot = kItems + 128;
  static constexpr int kBar = kSlot + 16;
  static constexpr int bKFull = 0, bKEmpty = bKFull + NS, bVFull = bKEmpty + NS,
                       bVEmpty = bVFull + NS, bQFull = bVEmpty + NS, bQEmpty = bQFull + 2,
                       bRows = bQEmpty + 2, bRowsFree = bRows + 2, bAux = bRowsFree + 2,
                       bAuxFree = bAux + 2, bMax = bAuxFree + 2, bStat = bMax + 2 * HB,
                       bPart = bStat + 2 * HB, bOFree = bPart + 2, bSFull = bOFree + 2,
                       bPFull = bSFull + 2, bItemFull = bPFull + kStages,
                       bItemEmpty = bItemFull + 4, bGo = bItemEmpty + 4, kNumBars = bGo + 1;
  static constexpr int kAlloc = kBar + kNumBars * 8 + 1024;
  static_assert(kAlloc <= 232448, "shared memory per CTA");
  static_assert(kQ % 1024 == 0 && kQBuf % 1024 == 0 && kMax % 16 == 0 && kBar % 8 == 0,
                "alignment");
};

// One item: a tile of one request for HB kv heads.
struct Item8 {
  int32_t nb;  // 128-key blocks; -1: no more items
  int32_t kvh; // first kv head
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

// Sums of G values over the 32 lanes of a warp: lane h < G gets the sum of
// v[h].  Each step halves the values a lane carries (it sends the others to
// its partner), so it takes G - 1 + log2(32 / G) shuffles instead of 5 G; the
// order of the additions is fixed.
template <int G>
__device__ __forceinline__ float warp_sums(const float (&v)[G], int lane) {
  float x[G];
#pragma unroll
  for (int h = 0; h < G; ++h) x[h] = v[h];
#pragma unroll
  for (int n = G / 2; n >= 1; n /= 2) { // partner: lane bit n; keep the half it names
    const bool up = (lane & n) != 0;
#pragma unroll
    for (int h = 0; h < n; ++h) {
      const float give = up ? x[h] : x[h + n], keep = up ? x[h + n] : x[h];
      x[h] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, n));
    }
  }
#pragma unroll
  for (int off = G; off < 32; off *= 2)
    x[0] = __fadd_rn(x[0], __shfl_xor_sync(0xffffffffu, x[0], off));
  return x[0];
}

// fp32 as int32 in the same order (for atomicMax), and back.
__device__ __forceinline__ int32_t ordered(float x) {
  const int32_t b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_ordered(int32_t b) {
  return __int_as_float(b ^ ((b >> 31) & 0x7fffffff));
}
constexpr int32_t kNoMax8 = static_cast<int32_t>(0xff800000u ^ 0x7fffffffu); // ordered(-inf)

// Element-wise on the G heads' values of a key, two an instruction.
template <int G>
__device__ __forceinline__ void add_heads(const float (&x)[G], const float (&y)[G], float (&z)[G]) {
  if constexpr (G == 1) {
    z[0] = x[0] + y[0];
  } else {
#pragma unroll
    for (int h = 0; h < G; h += 2)
      f32x2_split(fadd2(f32x2(x[h], x[h + 1]), f32x2(y[h], y[h + 1])), z[h], z[h + 1]);
  }
}
template <int G>
__device__ __forceinline__ void add_heads(const float (&x)[G], float y, float (&z)[G]) {
  float all[G];
#pragma unroll
  for (int h = 0; h < G; ++h) all[h] = y;
  add_heads(x, all, z);
}

template <int G, int DW, int HB>
__global__ void __launch_bounds__(kThreads8, 1)
    decode_fp8_kernel(const __grid_constant__ DecodeFp8Args f) {
  using L = Smem8<DW, HB>;
  constexpr int NP = L::NP, PH = L::PH, NS = L::NS, SB = L::SB, LPR = L::LPR, ST = L::kStages;
  constexpr int LO = G <= 4 ? 4 : 8; // column of a head's second term
  constexpr int NL = 2 * LO;         // columns in use
  constexpr int WH = 8 / HB;         // softmax warps that share a kv head
  constexpr int NB = kPartBlocks8 * HB / 2; // blocks of a part a softmax warp takes
  constexpr bool kKeep = NB * G <= 16;      // their scores stay in registers
  constexpr uint32_t kIdescS = idesc_e4m3(128, kN8, false, false);
  constexpr uint32_t kIdescPV = idesc_e4m3(128, kN8, true, true);
  constexpr uint32_t kTmemCols = 512;
  const DecodeGeometry &a = f.a;

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
  if (tid < 3 * HB * kMaxima8) reinterpret_cast<int32_t *>(smem + L::kMax)[tid] = kNoMax8;
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
      mbar_init(bar(L::bRowsFree + i), 2 * kCopyWarps8);
      mbar_init(bar(L::bAux + i), 4);
      mbar_init(bar(L::bAuxFree + i), 8);            // the softmax warps, past pass 2
      mbar_init(bar(L::bSFull + i), 1);              // a part's S
      mbar_init(bar(L::bPart + i), 1);               // a part's P.V
      mbar_init(bar(L::bOFree + i), 4 * HB);
    }
    for (int i = 0; i < 2 * HB; ++i) {
      mbar_init(bar(L::bMax + i), WH);
      mbar_init(bar(L::bStat + i), WH);
    }
    for (int i = 0; i < ST; ++i)
      mbar_init(bar(L::bPFull + i), HB == 2 ? 8 : 4 * SB); // the warps of the stage's P
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
  int32_t *const status = HB == 1 && a.slots ? a.slots + blockIdx.x : a.status;
  // TMEM columns, 16 each: S^T [part parity][block][head] (lanes = keys), then
  // O^T [item parity][part][head][piece] (lanes = dims)
  auto tS = [&](uint32_t ug, int j, int hh) {
    return tmem + 16u * (((ug & 1u) * kPartBlocks8 + static_cast<uint32_t>(j)) * HB + hh);
  };
  auto tO = [&](uint32_t ig, int part, int hh, int p) {
    return tmem + 16u * (2 * kPartBlocks8 * HB +
                         ((((ig & 1u) * kParts8 + static_cast<uint32_t>(part)) * HB + hh) * PH + p));
  };
  // the ig-th item of this CTA; nb = -1 also when the wait ran out
  auto read_item = [&](uint32_t ig) {
    const int s = static_cast<int>(ig & 3u);
    Item8 it;
    it.nb = -1;
    if (mbar_wait(bar(L::bItemFull + s), (ig >> 2) & 1u, status))
      it = *reinterpret_cast<const Item8 *>(smem + L::kItems + s * 32);
    return it;
  };
  auto item_read = [&](uint32_t ig) { mbar_arrive(bar(L::bItemEmpty + static_cast<int>(ig & 3u))); };
  // The warp-wide forms: the same answer on every lane, so that a wait that
  // ran out takes the whole warp out (the others then run out of theirs).
  auto wait = [&](int b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar(b), parity, status)) != 0;
  };
  auto warp_item = [&](uint32_t ig) {
    Item8 it = read_item(ig);
    if (__any_sync(0xffffffffu, it.nb < 0)) it.nb = -1;
    if (lane == 0) item_read(ig);
    return it;
  };
  // parts of an item and blocks of its part
  auto parts_of = [&](const Item8 &it) { return (it.nb + kPartBlocks8 - 1) / kPartBlocks8; };
  auto blocks_of = [&](const Item8 &it, int part) {
    return min(kPartBlocks8, it.nb - part * kPartBlocks8);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs8));
  if (warp == kItemWarp8) {
    // ------------------------------------------------------------ items
    // The first item is the CTA's own index; each next one is taken from the
    // counter when the copies of the current one start.
    const int groups = a.Hkv / HB; // of kv heads
    Item8 own; // of a CTA that plans itself (one head an item)
    own.nb = -1;
    if (HB == 1 && a.slots) {
      LaneRequest r;
      const bool ok = lane_requests(a, lane, r);
      if (lane == 0) *status = ok ? 0 : kStatusPlanMismatch;
      const int unit = static_cast<int>(blockIdx.x) / groups;
      // the first request whose units end past this one
      const int b = __popc(__ballot_sync(0xffffffffu, r.units_end <= unit));
      const int32_t split = unit - __shfl_sync(0xffffffffu, r.units_end - r.nsp, b & 31);
      const int32_t nsp = __shfl_sync(0xffffffffu, r.nsp, b & 31);
      const int32_t row = __shfl_sync(0xffffffffu, r.rows_end, b & 31) - nsp + split;
      const int32_t keys = __shfl_sync(0xffffffffu, r.kv_len, b & 31);
      own.page_base = __shfl_sync(0xffffffffu, r.page_base, b & 31);
      if (ok && b < a.batch) {
        own.kvh = static_cast<int>(blockIdx.x) % groups;
        own.b = b;
        own.key_begin = split * a.split;
        own.key_end = min(own.key_begin + a.split, keys);
        own.prow = nsp > 1 ? row : -1;
        own.nb = (own.key_end - own.key_begin + kKeys8 - 1) / kKeys8;
      } else if (!ok) { // as the planner: NaN instead of stale values
        const int64_t step = static_cast<int64_t>(gridDim.x) * 32;
        const int64_t rows = static_cast<int64_t>(a.batch) * a.Hq;
        for (int64_t e = blockIdx.x * 32 + lane; e < rows * a.D; e += step)
          a.out[e] = 0x7fc0u; // bf16 NaN
        for (int64_t e = blockIdx.x * 32 + lane; a.lse && e < rows; e += step)
          a.lse[e] = __int_as_float(0x7fc00000);
      }
    }
    if (lane == 0) {
      const int64_t n_work = HB == 1 && a.slots ? 0 : a.n_units * groups;
      int64_t w = blockIdx.x;
      for (uint32_t ig = 0;; ++ig) {
        Item8 it;
        it.nb = -1;
        if (ig == 0) it = own;
        if (w < n_work) {
          const int64_t unit = w / groups;
          const int4 u0 = __ldg(reinterpret_cast<const int4 *>(f.units + unit));
          const int4 u1 = __ldg(reinterpret_cast<const int4 *>(f.units + unit) + 1);
          if (u0.x >= 0) { // a retired unit: only retired ones follow
            it.kvh = static_cast<int>(w - unit * groups) * HB;
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
        if (ig >= 4 && !mbar_wait(bar(L::bItemEmpty + s), ((ig >> 2) - 1) & 1u, status)) it.nb = -1;
        *reinterpret_cast<Item8 *>(smem + L::kItems + s * 32) = it;
        mbar_arrive(bar(L::bItemFull + s));
        if (it.nb < 0) break;
        // a CTA that plans itself has one item (and no cleared counter)
        if (!mbar_wait(bar(L::bGo), ig & 1u, status) || n_work == 0) w = n_work;
        else w = static_cast<int64_t>(gridDim.x) + atomicAdd(a.status + kStatusWorkCounter, 1);
      }
    }
    __syncwarp();
  } else if (warp >= kCopyWarp8 && warp < kItemWarp8) {
    // ------------------------------------------------------------ copies
    // Eight warps copy key rows, eight value rows, at their own pace.  A warp
    // copies 16 keys of each block: chunk cc of every (32 / LPR)-th.  A chunk
    // goes to its head's piece (head_dim 64: both heads in one).
    const int kv = (warp - kCopyWarp8) / kCopyWarps8, cw = (warp - kCopyWarp8) % kCopyWarps8;
    const int cc = lane % LPR, kb = lane / LPR;
    const int chunks = a.D / 16; // of a head
    const bool in_row = cc < HB * chunks; // head_dim 96: 6 of 8 lanes a head
    const int piece = DW == 64 ? 0 : DW == 256 ? cc >> 3 : cc / chunks;
    const uint32_t pc = static_cast<uint32_t>(DW == 128 ? cc - piece * chunks : cc & 7); // in the piece
    const uint32_t *rows = reinterpret_cast<const uint32_t *>(smem + L::kRows);
    // Copies one part's key or value rows; sg counts the stages of each ring.
    const uint64_t once = policy_evict_first();
    const int b_full = kv == 0 ? L::bKFull : L::bVFull, b_empty = kv == 0 ? L::bKEmpty : L::bVEmpty;
    const uint32_t ring = (kv == 0 ? kstage(0) : vstage(0)) + static_cast<uint32_t>(piece) * kPiece8;
    const uint8_t *src = (kv == 0 ? f.k_codes : f.v_codes) + cc * 16;
    uint32_t sg = 0, ug = 0; // stages and parts so far
    bool ok = true;
    for (uint32_t ig = 0; ok; ++ig) {
      const Item8 it = warp_item(ig);
      if (it.nb < 0) break;
      if (warp == kCopyWarp8 && lane == 0) mbar_arrive(bar(L::bGo));
      const int n_parts = parts_of(it);
      for (int part = 0; part < n_parts && ok; ++part, ++ug) {
        const int par = static_cast<int>(ug & 1), nst = (blocks_of(it, part) + SB - 1) / SB;
        ok = wait(L::bRows + par, (ug >> 1) & 1);
        const uint32_t *row_w = rows + par * kPart8 + cw * kCopyKeys8 + kb;
        for (int st = 0; st < nst && ok; ++st, ++sg) {
          const uint32_t s = sg % NS;
          if (sg >= NS) ok = wait(b_empty + static_cast<int>(s), ((sg / NS) - 1) & 1);
          if (!ok) break;
#pragma unroll
          for (int hb = 0; hb < SB; ++hb) {
            const uint32_t dst = ring + s * L::kStage + hb * L::kBlock;
#pragma unroll
            for (int i = 0; i < kCopyKeys8 * LPR / 32; ++i) {
              const int k8 = cw * kCopyKeys8 + i * (32 / LPR) + kb;
              const uint32_t row = row_w[(st * SB + hb) * kKeys8 + i * (32 / LPR)];
              if (in_row)
                cp_async16_hint(dst + static_cast<uint32_t>(k8) * 128 +
                                    ((pc ^ static_cast<uint32_t>(k8 & 7)) << 4),
                                src + (row == kNoRow8 ? 0 : static_cast<uint64_t>(row) * a.D),
                                row != kNoRow8, once);
            }
          }
          cp_async_arrive(bar(b_full + static_cast<int>(s)));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bRowsFree + par)); // the part's rows have been read
      }
    }
    cp_async_wait_all(); // no copy outlives the CTA
  } else if (warp >= kAuxWarp8 && warp < kCopyWarp8) {
    // ------------------------------------------------------------ preparation
    // Aux warp w finds the cache rows and the scales of the keys of block w of
    // a part (four a lane) and splits q heads w, w + 4, ... of an item, up to
    // two parts ahead of their use.
    const int aw = warp - kAuxWarp8;
    const int page_mask = (1 << a.page_shift) - 1;
    uint32_t *s_rows = reinterpret_cast<uint32_t *>(smem + L::kRows);
    float *s_qs = reinterpret_cast<float *>(smem + L::kQs);
    const uint64_t keep = policy_evict_last();
    uint32_t ug = 0;
    bool ok = true;
    for (uint32_t ig = 0; ok; ++ig) {
      const Item8 it = warp_item(ig);
      if (it.nb < 0) break;
      for (int part = 0; part < parts_of(it) && ok; ++part, ++ug) {
        const int par = static_cast<int>(ug & 1);
        const int32_t key0 = it.key_begin + part * kPart8 + aw * kKeys8 + lane;
        int32_t page[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
          page[n] = key0 + n * 32 < it.key_end
                        ? __ldg(a.kv_indices + it.page_base + ((key0 + n * 32) >> a.page_shift)) : -1;
        // rows first: the copies wait for them
        if (ug >= 2) ok = wait(L::bRowsFree + par, ((ug >> 1) - 1) & 1);
        if (!ok) break;
        uint32_t row[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int32_t key = key0 + n * 32;
          const bool good = key < it.key_end && page[n] >= 0 && page[n] < a.num_pages;
          if (key < it.key_end && !good) atomicOr(status, kStatusBadPage);
          row[n] = good ? static_cast<uint32_t>(((static_cast<int64_t>(page[n]) << a.page_shift) +
                                                 (key & page_mask)) * a.Hkv + it.kvh)
                        : kNoRow8;
          s_rows[par * kPart8 + aw * kKeys8 + n * 32 + lane] = row[n];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bRows + par));
        // scale bytes of the HB heads; no row: zeros
        uint32_t ke[4], ve[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          ke[n] = ve[n] = 0;
          if (row[n] != kNoRow8) {
            if constexpr (HB == 2) { // an even row (the host checks the arrays' alignment)
              ke[n] = ld_scale_u16(f.k_scale + row[n], keep);
              ve[n] = ld_scale_u16(f.v_scale + row[n], keep);
            } else {
              ke[n] = ld_scale_u8(f.k_scale + row[n], keep);
              ve[n] = ld_scale_u8(f.v_scale + row[n], keep);
            }
          }
        }
        if (ug >= 2) ok = wait(L::bAuxFree + par, ((ug >> 1) - 1) & 1);
        if (!ok) break;
        if (part == 0) {
          // q: hi + lo/16 of the row scaled by 2^-e, 4 elements a lane and
          // 128 columns
          const int qp = static_cast<int>(ig & 1);
          if (ig >= 2) ok = wait(L::bQEmpty + qp, ((ig >> 1) - 1) & 1);
          if (!ok) break;
          constexpr int NH = (HB * G + 3) / 4;
          uint2 qv[NH][PH];
#pragma unroll
          for (int i = 0; i < NH; ++i)
#pragma unroll
            for (int p = 0; p < PH; ++p) {
              const int h = aw + 4 * i, col = p * 128 + lane * 4;
              qv[i][p] = make_uint2(0, 0);
              if (h < HB * G && col < a.D)
                qv[i][p] = __ldg(reinterpret_cast<const uint2 *>(
                    a.q + (static_cast<int64_t>(it.b) * a.Hq + it.kvh * G + h) * a.D + col));
            }
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            const int h = aw + 4 * i;
            if (h < HB * G) {
              float x[PH][4];
              uint32_t big = 0;
#pragma unroll
              for (int p = 0; p < PH; ++p) {
                const uint32_t u[4] = {qv[i][p].x & 0xffffu, qv[i][p].x >> 16,
                                       qv[i][p].y & 0xffffu, qv[i][p].y >> 16};
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
              const int hh = h / G, r = h - hh * G; // kv head of the item, row
#pragma unroll
              for (int p = 0; p < PH; ++p) {
                float v[4], back[4];
                uint32_t hi[2], lo[2];
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = x[p][c] * inv;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  hi[c] = e4m3x2(v[2 * c], v[2 * c + 1]);
                  e4m3x2_values(hi[c], back[2 * c], back[2 * c + 1]);
                  lo[c] = e4m3x2((v[2 * c] - back[2 * c]) * 16.f,
                                 (v[2 * c + 1] - back[2 * c + 1]) * 16.f);
                }
                if (p * 128 + lane * 4 < a.D) {
                  // the columns of the head's codes in the key rows
                  const int col = lane * 4 + (DW == 64 ? 64 * hh : 0);
                  uint8_t *q0 = smem + L::kQ + qp * L::kQBuf +
                                (DW == 64 ? 0 : DW == 256 ? p : hh) * (kN8 * 128);
                  auto at = [&](int rr) { // row rr, 16-byte chunk col / 16
                    return rr * 128 + (((col >> 4) ^ (rr & 7)) << 4) + (col & 15);
                  };
                  *reinterpret_cast<uint32_t *>(q0 + at(r)) = hi[0] | (hi[1] << 16);
                  *reinterpret_cast<uint32_t *>(q0 + at(LO + r)) = lo[0] | (lo[1] << 16);
                }
              }
              if (lane == 0) s_qs[(qp * HB + hh) * 8 + r] = a.scale_log2 * exp2_int(e);
            }
          }
          fence_proxy_async(); // q is read by the MMA (async proxy)
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::bQFull + qp));
        }
#pragma unroll
        for (int hh = 0; hh < HB; ++hh)
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const int t = (par * HB + hh) * kPart8 + aw * kKeys8 + n * 32 + lane;
            smem[L::kKe + t] = static_cast<uint8_t>(ke[n] >> (8 * hh));
            smem[L::kVe + t] = static_cast<uint8_t>(ve[n] >> (8 * hh));
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bAux + par));
      }
    }
  } else if (warp == kSWarp8) {
    // ------------------------------------------------------------ S issuer
    if (lane == 0) {
      // 32-code steps of a head's piece.  The descriptors are built once: a
      // step only adds to the start-address field (16-byte units; every
      // address is below 2^18, so the field never carries), since the thread
      // executes an instruction only about every ten cycles and building each
      // descriptor anew took longer than the MMAs.
      constexpr int KS = DW == 64 ? 2 : 4;
      const bool all_steps = a.D != 96;
      const uint64_t dk0 = desc_sw128(kstage(0), 16, 1024);
      const uint64_t dq0 = desc_sw128(sbase + L::kQ, 16, 1024);
      uint32_t sg = 0, ug = 0;
      bool ok = true;
      for (uint32_t ig = 0; ok; ++ig) {
        const Item8 it = read_item(ig);
        item_read(ig);
        if (it.nb < 0) break;
        const uint64_t dq = dq0 + ((ig & 1) * L::kQBuf >> 4);
        ok = mbar_wait(bar(L::bQFull + (ig & 1)), (ig >> 1) & 1, status);
        for (int part = 0; part < parts_of(it) && ok; ++part, ++ug) {
          const int nb = blocks_of(it, part);
          // the S columns are free once the softmax is through part ug - 2
          if (ug >= 2) ok = mbar_wait(bar(L::bAuxFree + (ug & 1)), ((ug >> 1) - 1) & 1, status);
          for (int j = 0; j < nb && ok; ++sg) {
            const uint32_t s = sg % NS;
            ok = mbar_wait(bar(L::bKFull + s), (sg / NS) & 1, status);
            if (!ok) break;
            fence_proxy_async(); // the rows were written by cp.async (generic proxy)
            tc_fence_after();
            const uint64_t dk = dk0 + (s * L::kStage >> 4);
#pragma unroll
            for (int hb = 0; hb < SB; ++hb, ++j) {
              if (j >= nb) break;
              const uint32_t ts = tS(ug, j, 0);
#pragma unroll
              for (int hh = 0; hh < HB; ++hh)
#pragma unroll
                for (int p = 0; p < PH; ++p)
#pragma unroll
                  for (int kk = 0; kk < KS; ++kk) {
                    const uint32_t pc = DW == 64 ? 0 : DW == 256 ? p : hh;  // piece
                    const uint32_t co = (DW == 64 ? hh * 64 : 0) + kk * 32; // column
                    if (kk < 3 || all_steps)
                      mma_e4m3_ss(ts + 16 * hh, dk + ((hb * L::kBlock + pc * kPiece8 + co) >> 4),
                                  dq + ((pc * (kN8 * 128) + co) >> 4), kIdescS, p + kk > 0);
                  }
            }
            mma_commit(bar(L::bKEmpty + s));
          }
          if (ok) mma_commit(bar(L::bSFull + (ug & 1)));
        }
        if (!ok) break;
        mma_commit(bar(L::bQEmpty + (ig & 1)));
      }
    }
    __syncwarp();
  } else if (warp == kPVWarp8) {
    // ------------------------------------------------------------ P.V issuer
    if (lane == 0) {
      const uint64_t dv0 = desc_sw128(vstage(0), 16384, 1024);
      const uint64_t dp0 = desc_plain(sbase + L::kP, 128, 128);
      uint32_t sg = 0, ug = 0;
      bool ok = true;
      for (uint32_t ig = 0; ok; ++ig) {
        const Item8 it = read_item(ig);
        item_read(ig);
        if (it.nb < 0) break;
        // the item's O buffers are free once the epilogue of item ig - 2 read them
        if (ig >= 2) ok = mbar_wait(bar(L::bOFree + (ig & 1)), ((ig >> 1) - 1) & 1, status);
        for (int part = 0; part < parts_of(it) && ok; ++part, ++ug) {
          const int nb = blocks_of(it, part);
          for (int j = 0; j < nb && ok; ++sg) {
            const uint32_t s = sg % NS, ps = sg % ST;
            ok = mbar_wait(bar(L::bVFull + s), (sg / NS) & 1, status) &&
                 mbar_wait(bar(L::bPFull + ps), (sg / ST) & 1, status);
            if (!ok) break;
            fence_proxy_async();
            tc_fence_after();
            const uint64_t dv = dv0 + (s * L::kStage >> 4);
            const uint64_t dp = dp0 + (ps * (SB * HB * L::kPBlock) >> 4);
            const uint32_t to = tO(ig, part, 0, 0);
#pragma unroll
            for (int hb = 0; hb < SB; ++hb, ++j) {
              if (j >= nb) break;
#pragma unroll
              for (int hh = 0; hh < HB; ++hh)
#pragma unroll
                for (int p = 0; p < PH; ++p)
#pragma unroll
                  for (int kk = 0; kk < kKeys8 / 32; ++kk) {
                    const uint32_t pc = DW == 64 ? 0 : DW == 256 ? p : hh; // piece
                    mma_e4m3_ss(to + 16 * (hh * PH + p),
                                dv + ((hb * L::kBlock + pc * kPiece8 + kk * 4096) >> 4),
                                dp + (((hb * HB + hh) * L::kPBlock + kk * 512) >> 4), kIdescPV,
                                (j > 0 || kk > 0) ? 1u : 0u);
                  }
            }
            mma_commit(bar(L::bVEmpty + s));
          }
          if (ok) mma_commit(bar(L::bPart + (ug & 1)));
        }
      }
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs8));
    // ------------------------------------------------------------ softmax
    // Thread t is key t of a block and dim t of the output.  HB = 2:
    // warpgroup w has head w and every block; HB = 1: both have the one head,
    // warpgroup w the blocks j with j % 2 == w, and the epilogues in turn.
    const int wg = warp >> 2, qd = warp & 3; // TMEM lanes 32qd .. 32qd+31
    const int t = qd * 32 + lane;
    const int hh = HB == 2 ? wg : 0;
    const int wf = HB == 2 ? 4 * wg : 0; // first warp of the head's
    const uint32_t lane_base = static_cast<uint32_t>(qd * 32) << 16;
    int32_t *s_max = reinterpret_cast<int32_t *>(smem + L::kMax) + hh * kMaxima8;
    float *s_stat = reinterpret_cast<float *>(smem + L::kStat);
    float *s_m = reinterpret_cast<float *>(smem + L::kStatM);
    float *s_c = s_m + 2 * HB * 8;
    const float *s_qs = reinterpret_cast<const float *>(smem + L::kQs);
    uint32_t sg = 0, ug = 0;
    int max_at = 0; // ug % 3, times a part's maxima
    bool ok = true;
    for (uint32_t ig = 0; ok; ++ig) {
      const Item8 it = warp_item(ig);
      if (it.nb < 0) break;
      const int n_parts = parts_of(it);
      for (int part = 0; part < n_parts; ++part, ++ug) {
        const int nb = blocks_of(it, part), nst = (nb + SB - 1) / SB;
        const int par = static_cast<int>(ug & 1);
        const int32_t key0 = it.key_begin + part * kPart8 + t;
        ok = wait(L::bAux + par, (ug >> 1) & 1);
        if (!ok) break;
        const uint8_t *ke = smem + L::kKe + (par * HB + hh) * kPart8 + t;
        const uint8_t *ve = smem + L::kVe + (par * HB + hh) * kPart8 + t;
        float qs[G];
#pragma unroll
        for (int h = 0; h < G; ++h) qs[h] = s_qs[(static_cast<int>(ig & 1) * HB + hh) * 8 + h];
        // ---- pass 1: the scores, and of each head the part's largest score
        // and largest score + ev.  The scores stay in registers where 16 hold
        // them, else pass 2 reads S again.
        ok = wait(L::bSFull + par, (ug >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        auto block = [&](int i) { return HB == 2 ? i : 2 * i + wg; };
        auto scores = [&](int j, const uint32_t (&v)[NL], float (&sc)[G]) {
          const float ks = e8m0_value(ke[j * kKeys8]);
          const bool valid = key0 + j * kKeys8 < it.key_end; // false past the part's blocks
          if constexpr (G == 1) {
            const float raw = fmaf(__uint_as_float(v[LO]), 0.0625f, __uint_as_float(v[0]));
            sc[0] = raw * (ks * qs[0]);
          } else {
#pragma unroll
            for (int h = 0; h < G; h += 2) {
              const uint64_t raw =
                  ffma2r(f32x2(__uint_as_float(v[LO + h]), __uint_as_float(v[LO + h + 1])),
                         f32x2(0.0625f, 0.0625f),
                         f32x2(__uint_as_float(v[h]), __uint_as_float(v[h + 1])));
              f32x2_split(fmul2(raw, fmul2(f32x2(ks, ks), f32x2(qs[h], qs[h + 1]))), sc[h], sc[h + 1]);
            }
          }
#pragma unroll
          for (int h = 0; h < G; ++h) sc[h] = valid ? sc[h] : -INFINITY;
        };
        float m[G], r[G], sc[NB][G];
        uint32_t ev_most = 0;
#pragma unroll
        for (int h = 0; h < G; ++h) m[h] = r[h] = -INFINITY;
        auto maxima = [&](int j, const float (&x)[G]) {
          const uint32_t vb = ve[j * kKeys8];
          const float ev = vb == 255u ? -INFINITY : static_cast<float>(vb); // a NaN scale: nowhere
          ev_most = max(ev_most, vb == 255u ? 0u : vb);
          float y[G];
          add_heads(x, ev, y);
#pragma unroll
          for (int h = 0; h < G; ++h) {
            m[h] = fmaxf(m[h], x[h]);
            r[h] = fmaxf(r[h], y[h]);
          }
        };
        if constexpr (kKeep) {
          uint32_t v[NB][NL];
#pragma unroll
          for (int i = 0; i < NB; ++i)
            if (block(i) < nb) tmem_ld_n<NL>(tS(ug, block(i), hh) + lane_base, v[i]);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            scores(block(i), v[i], sc[i]);
            maxima(block(i), sc[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            if (block(i) >= nb) break;
            uint32_t v[NL];
            tmem_ld_n<NL>(tS(ug, block(i), hh) + lane_base, v);
            tmem_wait_ld();
            scores(block(i), v, sc[0]);
            maxima(block(i), sc[0]);
          }
        }
        // The warps' maxima meet in shared memory, lane h < G that of head h,
        // lane 8 + h its score + ev, lane 16 the ev.  Three sets in turn: the
        // next part's is cleared before this part's barrier, behind the barrier
        // of the last part (past which nobody reads it) and before any warp can
        // add to it.
        int32_t mine = static_cast<int32_t>(__reduce_max_sync(0xffffffffu, ev_most));
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float wm = warp_max(m[h]), wr = warp_max(r[h]);
          mine = lane == h ? ordered(wm) : lane == 8 + h ? ordered(wr) : mine;
        }
        if (lane <= 16 && (lane & 7) < G) atomicMax(s_max + max_at + lane, mine);
        const int max_next = max_at == 2 * HB * kMaxima8 ? 0 : max_at + HB * kMaxima8;
        if (warp == wf && lane <= 16) s_max[max_next + lane] = kNoMax8;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::bMax + par * HB + hh));
        ok = wait(L::bMax + par * HB + hh, (ug >> 1) & 1);
        if (!ok) break;
        // c: at least 0, as the key of the largest score has an ev of 0 or more
        // (0 too where an infinite score makes it NaN).  (score + ev) was
        // rounded, by at most 2^-24 of it: c makes up for that, so that no entry
        // passes 2^8.5 however large the scores are, and is at most the part's
        // largest ev, with which no entry passes 2^8.
        const float c_top = static_cast<float>(s_max[max_at + 16]);
        auto c_of = [&](float most, float top) {
          const float c = ceilf(fmaf(fabsf(most), 0x1p-23f, most - top) - 0.5f);
          return fminf(fmaxf(c, 0.f), c_top);
        };
        // lane h (and 8 + h, ...) works out head h's
        const float m_mine = from_ordered(s_max[max_at + (lane & 7)]);
        const float c_mine = c_of(from_ordered(s_max[max_at + 8 + (lane & 7)]), m_mine);
        if (warp == wf && lane < G) { // of the part's state
          s_m[(par * HB + hh) * 8 + lane] = m_mine;
          s_c[(par * HB + hh) * 8 + lane] = c_mine;
        }
        float m_neg[G], c_neg[G];
#pragma unroll
        for (int h = 0; h < G; ++h) {
          if constexpr (G == 8) { // shuffles take ptxas past its registers
            m_neg[h] = -from_ordered(s_max[max_at + h]);
            c_neg[h] = -c_of(from_ordered(s_max[max_at + 8 + h]), -m_neg[h]);
          } else {
            m_neg[h] = -__shfl_sync(0xffffffffu, m_mine, h);
            c_neg[h] = -__shfl_sync(0xffffffffu, c_mine, h);
          }
        }
        max_at = max_next;
        // ---- pass 2: the weights 2^(s - m), and 2^(s - m + ev - c + 8) in two
        // e4m3 terms (an exponential of its own: the weight alone may underflow)
        // row sums: even blocks, odd blocks (HB = 1 with two warpgroups on
        // them adds in the same order: both forms give the same bits)
        float l[2][G];
#pragma unroll
        for (int h = 0; h < G; ++h) l[0][h] = l[1][h] = 0.f;
        // P of part ug - 1 has been read
        if (ug >= 1) ok = wait(L::bPart + (par ^ 1), ((ug - 1) >> 1) & 1);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int j = block(i);
          if (j >= nb) break;
          const uint32_t ps = (sg + j / SB) % ST;
          if constexpr (!kKeep) {
            uint32_t v[NL];
            tmem_ld_n<NL>(tS(ug, j, hh) + lane_base, v);
            tmem_wait_ld();
            scores(j, v, sc[0]);
          }
          const uint32_t vb = ve[j * kKeys8];
          const float ev = vb == 255u ? NAN : static_cast<float>(static_cast<int>(vb) + kBoost8);
          float x[G], y[G], w[G];
          add_heads(sc[kKeep ? i : 0], m_neg, x); // -inf for a key that is not there
          add_heads(c_neg, ev, w);
          add_heads(x, w, y);
#pragma unroll
          for (int h = 0; h < G; ++h) {
            x[h] = ex2(x[h]);
            w[h] = ex2(y[h]);
          }
          add_heads(l[i & (HB - 1)], x, l[i & (HB - 1)]);
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
          *reinterpret_cast<uint4 *>(smem + L::kP + ((ps * SB + j % SB) * HB + hh) * L::kPBlock +
                                     t * 16) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          // a warp's last block of the stage: hand P over
          if (HB == 1 || SB == 1 || j % SB == SB - 1 || j == nb - 1) {
            fence_proxy_async(); // P is read by the MMA (async proxy)
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::bPFull + static_cast<int>(ps)));
          }
        }
        // HB = 1: the odd warpgroup has no block in a last stage of one
        if (HB == 1 && SB == 2 && wg == 1 && (nb & 1) && lane == 0)
          mbar_arrive(bar(L::bPFull + static_cast<int>((sg + nst - 1) % ST)));
        sg += nst;
        // ---- the part's state: the row sums of the warps
        float lw = warp_sums<G>(l[0], lane); // lane h < G: head h
        if (HB == 2) lw = __fadd_rn(lw, warp_sums<G>(l[1], lane));
        if (lane < 8) s_stat[(par * 8 + warp) * 8 + lane] = lw;
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(L::bAuxFree + par));
          mbar_arrive(bar(L::bStat + par * HB + hh));
        }
      }
      if (!ok) break;
      if (HB == 2 || static_cast<int>(ig & 1) == wg) {
        // ---- epilogue: the parts' states joined, o = O^T / l
        const uint32_t u1 = ug - 1, u0 = ug - n_parts; // the last and first part
        ok = wait(L::bStat + static_cast<int>(u0 & 1) * HB + hh, (u0 >> 1) & 1) &&
             wait(L::bStat + static_cast<int>(u1 & 1) * HB + hh, (u1 >> 1) & 1) &&
             wait(L::bPart + static_cast<int>(u1 & 1), (u1 >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        const bool two = n_parts == 2;
        const int p0 = static_cast<int>(u0 & 1), p1 = static_cast<int>(u1 & 1);
        // lane h < G: the join of head h (lanes past G repeat one)
        const int hl = lane & (G - 1);
        const float m0 = s_m[(p0 * HB + hh) * 8 + hl], m1 = s_m[(p1 * HB + hh) * 8 + hl];
        const float M = fmaxf(m0, m1);
        const float d0 = m0 == M ? 0.f : m0 - M, d1 = m1 == M ? 0.f : m1 - M;
        const float a0 = ex2(d0), a1 = ex2(d1);
        // O of a part counts 2^(d + c): that much over the larger of the two
        const float x0 = d0 + s_c[(p0 * HB + hh) * 8 + hl], x1 = d1 + s_c[(p1 * HB + hh) * 8 + hl];
        const float top = fminf(ceilf(fmaxf(x0, x1)), 254.f); // >= 0: that of the larger maximum
        const float e_mine = e8m0_value(static_cast<uint32_t>(top));
        float l0 = 0.f, l1 = 0.f; // the quadrants in order, each even + odd blocks
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          float x0 = s_stat[(p0 * 8 + wf + w) * 8 + hl], x1 = s_stat[(p1 * 8 + wf + w) * 8 + hl];
          if (HB == 1) {
            x0 = __fadd_rn(x0, s_stat[(p0 * 8 + 4 + w) * 8 + hl]);
            x1 = __fadd_rn(x1, s_stat[(p1 * 8 + 4 + w) * 8 + hl]);
          }
          l0 = __fadd_rn(l0, x0);
          l1 = __fadd_rn(l1, x1);
        }
        const float ls = two ? __fadd_rn(__fmul_rn(a0, l0), __fmul_rn(a1, l1)) : l0;
        const float inv = ls == 0.f ? 0.f : __frcp_rn(ls);
        const float f0_mine = __fmul_rn(ex2(x0 - top), inv); // one part: 2^0
        const float f1_mine = __fmul_rn(ex2(x1 - top), inv);
        const float lse_mine = ls == 0.f ? -INFINITY : __fmul_rn(__fadd_rn(M, lg2(ls)), kLn2);
        const bool single = it.prow < 0; // one tile: the final row
        const int64_t head0 =
            static_cast<int64_t>(single ? it.b : it.prow) * a.Hq + (it.kvh + hh) * G;
#pragma unroll
        for (int p = 0; p < PH; ++p) {
          uint32_t o0[NL], o1[NL];
          tmem_ld_n<NL>(tO(ig, 0, hh, p) + lane_base, o0);
          if (two) tmem_ld_n<NL>(tO(ig, 1, hh, p) + lane_base, o1);
          tmem_wait_ld();
          if (p == PH - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::bOFree + static_cast<int>(ig & 1))); // O read
          }
          const int dim = p * 128 + t - (DW == 64 ? 64 * hh : 0);
          const bool real = dim >= 0 && dim < a.D;
#pragma unroll
          for (int h = 0; h < G; ++h) {
            const float f0 = __shfl_sync(0xffffffffu, f0_mine, h);
            const float f1 = __shfl_sync(0xffffffffu, f1_mine, h);
            const float e_val = __shfl_sync(0xffffffffu, e_mine, h);
            float val =
                __fmul_rn(fmaf(__uint_as_float(o0[LO + h]), 0.0625f, __uint_as_float(o0[h])), f0);
            if (two)
              val = __fmaf_rn(fmaf(__uint_as_float(o1[LO + h]), 0.0625f, __uint_as_float(o1[h])), f1,
                              val);
            val = __fmul_rn(__fmul_rn(val, 1.f / (1 << kBoost8)), e_val);
            if (real && single) a.out[(head0 + h) * a.D + dim] = to_bf16(val);
            if (real && !single) a.part_o[(head0 + h) * a.D + dim] = val;
          }
        }
        if (t < G) {
          if (!single) a.part_lse[head0 + t] = lse_mine;
          else if (a.lse) a.lse[head0 + t] = lse_mine;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kPVWarp8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int G, int DW, int HB>
cudaError_t launch_f8(const DecodeFp8Args &f, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  int sms = 0;
  const cudaError_t e =
      prepare_launch(reinterpret_cast<const void *>(decode_fp8_kernel<G, DW, HB>),
                     Smem8<DW, HB>::kAlloc, ready, &sms);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(f.a.n_units * (f.a.Hkv / HB), sms)));
  cfg.blockDim = dim3(kThreads8);
  cfg.dynamicSmemBytes = Smem8<DW, HB>::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_fp8_kernel<G, DW, HB>, f);
}

// Two kv heads an item where they pair up, unless one head an item still gives
// every item an SM of its own (one request of 4097 keys, 8 kv heads: 16.4
// instead of 20.5 us on twice the SMs; one of 32768: 24.6 instead of 22.5 us).
// Both forms give the same bits.
template <int G>
cudaError_t launch_f8_g(const DecodeFp8Args &f, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const bool pairs = f.a.Hkv % 2 == 0 && f.a.n_units * f.a.Hkv > sms;
  if (f.a.D == 64) return pairs ? launch_f8<G, 64, 2>(f, s) : launch_f8<G, 64, 1>(f, s);
  if (f.a.D <= 128) return pairs ? launch_f8<G, 128, 2>(f, s) : launch_f8<G, 128, 1>(f, s);
  return launch_f8<G, 256, 1>(f, s);
}

} // namespace

} // namespace bia
