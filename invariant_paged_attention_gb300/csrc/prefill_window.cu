// Causal extend with a window and sinks over the paged cache on the tensor
// cores (tcgen05 + TMEM): a row at position p sees key j <= p if j > p - window
// or j < sinks.  The tiles, the softmax and the fold are those of
// prefill_ragged.cu (128-row q tiles of 128/G tokens x G heads, "sglang PR
// #43612", Summary; fixed split-KV tiles anchored at key 0 and merged in order,
// "sglang PR #10417 [POC] Support deterministic inference", Modifications); a
// q tile visits only the key blocks (of 128 keys; 64 at head_dim 256) that one
// of its rows sees: the sinks' blocks, then the window's, each anchored at key 0.
//
// A persistent CTA per SM takes items: two consecutive q tiles of one request
// (one at head_dim 256, whose O fills half of TMEM) against one kv head.  Its
// roles walk the same items through a ring of records and each runs ahead as
// far as its buffers allow: warps 0-3 and 4-7 softmax + epilogue of the two
// tiles, 8 issues the MMAs and owns TMEM, 9 loads q and K, 11 V, 10 makes the
// items.  The two tiles share every block that either needs; a tile leaves out
// the blocks that only the other one sees, and the copies the 16-key steps of the
// blocks at the window's and the sinks' ends that no row sees.
//
// A block of K or V comes as runs of 16 keys of one page (3-D TMA boxes) where
// pages hold 16 keys and more, else, and where a run is not wholly needed, as
// gathers of four rows; rows past the sequence, behind the window of the item's
// first row or on a bad page come from outside the tensor map and read as
// zeros, so what the call does not see is never read.
//
// Split tiles: with few items each split of a pair is an item, its fp32 states
// go to the workspace and a merge folds them; with many an item is the whole
// pair and the CTA folds each state into the running one as the merge would
// (fold.cuh).  The sinks go with a q tile's first split.  The bits are the same
// either way, whatever the batch.
//
// Measured with 32/8 heads x 128 on prompts of 512 to 8192 tokens: window 1024
// 657 us (1028 TFLOP/s of the scores seen), 8192 1700 us (1343), 16/8 heads x
// 256 750 us (880); pages of one key 765 and 1220 us.  A pair of tiles takes a
// 128-key block in ~2950 cycles, 2050 of them MMAs back to back; the rest is the
// chain P -> P.V -> S -> P (a wait answered in 100 to 150 cycles, commits of 60)
// and, at the power that this draws, a clock of 1.6 to 1.75 GHz.  Exponentials
// left out, it took as long.  A short window adds its two ends (a block that is
// not whole costs up to twice its time) and an epilogue of ~4500 cycles every
// ten blocks; 256-wide heads, one tile an item, read twice the bytes a flop and
// wait for values; pages of fewer than 16 keys for the gathers (four rows of
// 128 bytes about every 29 cycles an SM; 256-wide heads spill 50 bytes there).
//
// P is rounded to bf16 for the tensor cores; scores, sums and states are fp32.
#include "bia_internal.h"
#include "fold.cuh"
#include "ptx.cuh"

#include <algorithm>

namespace bia {

namespace {

constexpr int kSoftWarpsW = 8;
constexpr int kMmaWarpW = 8;
constexpr int kKeyWarpW = 9; // loads q and K
constexpr int kItemWarpW = 10;
constexpr int kValueWarpW = 11; // loads V
constexpr int kLoad2W = 12; // with row gathers 12 and 13 are second warps of K and of V
constexpr int kItemsW = 3;               // items in flight
constexpr int kAtomQW = kTileRows * 128; // one SW128 column block of a q tile
constexpr float kRescaleW = 16.0f;       // log2 units the running max may lag a block's

struct WindowPrefillArgs {
  int32_t Hq, Hkv, D, G, split, tile_tokens, batch, page_shift, window, sinks, parts, folds;
  int32_t kv_rows, slots; // row extent of the gather maps, slot extent of the run maps
  float scale_log2;
  int64_t num_pages;
  const ReqInfo *reqs;
  const int32_t *group_off; // first pair of each request
  const int32_t *kv_indices;
  float *part_o, *part_lse;
  uint16_t *out;
  float *lse;
  int32_t *status;
  CUtensorMap tm_q, tm_k, tm_v, tm_k3, tm_v3;
};

// What the roles need of an item.  kvh < 0 ends the list.
struct alignas(16) ItemW {
  int32_t kvh, tile, q_start, q_len;
  int32_t kv_len, page_base, lo, nb; // keys >= lo are loaded (and the sinks); blocks in all
  int32_t n_sink, w0;                // the first n_sink blocks are 0 ..; then w0 ..
  int32_t sink[2];                   // whether the tile uses the sinks' blocks
  int32_t j0[2], j1[2];              // window blocks of the tile, counted in the item
  int32_t steps;                     // of the blocks that are not whole
  int32_t w_begin[2], w_end[2];      // blocks that every row of the tile sees in full
  int32_t part[2], n_parts[2];       // which of the tile's states; n_parts 0: not here
};

// The 16-key steps u .. v - 1 of block j of an item that a tile's rows see,
// which are copied.  Only the sinks' last block and the ends of the window are
// not whole.
// An item holds four bits for each: the first step of the tile's block j0 and
// the end of its block j1 - 1 (8 bits a tile), the end of block n_sink - 1.
template <int KB>
struct Steps {
  int n_sink, j0, j1, bits;
  __device__ __forceinline__ int u(int j) const { return j == j0 ? bits & 15 : 0; }
  __device__ __forceinline__ int v(int j) const {
    return j == j1 - 1 ? (bits >> 4) & 15 : j == n_sink - 1 ? (bits >> 16) & 15 : KB / 16;
  }
};

// ROWS: pages of fewer than 16 keys, whose rows are gathered four at a time.  A
// warp issues its lanes' gathers one after the other, so K and V have two warps
// each (window 1024, page 1: 962 us with one, 765 with two; 256-wide heads 1602
// and 1220); runs of 16 keys need one.
template <int D, bool ROWS>
struct SmemW {
  static constexpr int kThreads = ROWS ? 512 : 384, kLoaders = ROWS ? 4 : 2;
  static constexpr int NT = D == 256 ? 1 : 2;    // q tiles an item
  static constexpr int KB = D == 256 ? 64 : 128; // keys a block
  static constexpr int kQTile = kTileRows * D * 2;
  static constexpr int kAtom = KB * 128; // one column block of a K or V block
  static constexpr int kKV = KB * D * 2;
  static constexpr int kRing = NT * kQTile; // stage s: K at kRing + 2s*kKV, V after it
  static constexpr int kItem = kRing + 4 * kKV;
  static constexpr int kBar = kItem + kItemsW * static_cast<int>(sizeof(ItemW));
  static constexpr int kQFull = 0, kQEmpty = 1, kKFull = 2, kVFull = 4, kKEmpty = 6, kVEmpty = 8,
                       kSFull = 10, kPFull = 12, kODone = 14, kIAsk = 16, kIFull = 17,
                       kIEmpty = kIFull + kItemsW, kNumBars = kIEmpty + kItemsW;
  // registers: the softmax warps hold a whole S row
  static constexpr int kSoftRegs = D == 256 && !ROWS ? 200 : 208;
  static constexpr int kOtherRegs = ROWS ? 48 : 504 - 2 * kSoftRegs;
  static_assert(8 * kSoftRegs + (kThreads / 32 - 8) * kOtherRegs <=
                    kThreads / 32 * (ROWS ? 128 : 168), "registers of the launch");
  static constexpr int kSlot = kBar + kNumBars * 8;
  static constexpr int kAlloc = kSlot + 16 + 1024;
  static_assert(kAlloc <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ void gather4(uint32_t dst, const void *tmap, int32_t x,
                                        const int32_t (&y)[4], uint32_t bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::"
               "complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
               "l"(tmap), "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(bar)
               : "memory");
}

// One lane of a warp that runs together.  The MMAs behind a branch on it take
// their operands from uniform registers without a step more: 64 cycles an MMA
// of 128 x 128 x 16, where a predicate on a lane's own flag took 79 whatever N
// (window 8192: 1870 -> 1700 us), and a branch on the lane's number as long.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r));
  return r != 0;
}

// N words of a thread's row, 32 bytes a store where out allows it
template <int N>
__device__ __forceinline__ void store_words(void *p, const uint32_t (&w)[N]) {
  uint32_t *d = static_cast<uint32_t *>(p);
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d + i),
                   "r"(w[i]), "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]),
                   "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<uint4 *>(d + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

// The first n of 32 columns, as bits.
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
}

template <int D, bool ROWS>
__global__ void __launch_bounds__((SmemW<D, ROWS>::kThreads), 1)
    prefill_window_kernel(const __grid_constant__ WindowPrefillArgs a) {
  using L = SmemW<D, ROWS>;
  constexpr int NT = L::NT, KB = L::KB;
  constexpr uint32_t kIdescS = idesc_bf16(128, KB, false);
  constexpr uint32_t kIdescPV = idesc_bf16(128, D, true);
  constexpr uint32_t kTmemCols = 512;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + L::kBar + 8u * static_cast<uint32_t>(i); };
  auto sQ = [&](int t) { return sbase + t * L::kQTile; };
  auto sK = [&](int st) { return sbase + L::kRing + (2 * st) * L::kKV; };
  auto sV = [&](int st) { return sbase + L::kRing + (2 * st + 1) * L::kKV; };
  ItemW *items = reinterpret_cast<ItemW *>(smem + L::kItem);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kSlot);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);

  if (warp == kMmaWarpW) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  if (tid == 0) {
    mbar_init(bar(L::kQFull), 1);
    mbar_init(bar(L::kQEmpty), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(L::kKFull + s), 1);
      mbar_init(bar(L::kVFull + s), 1);
      mbar_init(bar(L::kKEmpty + s), 1);
      mbar_init(bar(L::kVEmpty + s), 1);
      mbar_init(bar(L::kSFull + s), 1);
      mbar_init(bar(L::kPFull + s), 4);
      mbar_init(bar(L::kODone + s), 1);
    }
    mbar_init(bar(L::kIAsk), 1);
    for (int s = 0; s < kItemsW; ++s) {
      mbar_init(bar(L::kIFull + s), 1);
      mbar_init(bar(L::kIEmpty + s), kSoftWarpsW + 1 + L::kLoaders);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // TMEM columns: S buffers (one a tile; two of the one tile) from 0, O from 256
  auto tS = [&](int i) { return tmem + static_cast<uint32_t>(KB) * i; };
  auto tO = [&](int t) { return tmem + 256u + static_cast<uint32_t>(D) * t; };
  grid_dep_wait();   // the plan is complete
  grid_dep_launch(); // the next kernel of the call may start launching
  const int G = a.G, T = a.tile_tokens;

  // A role's walk over the CTA's items; a warp walks together (single: one
  // thread of it).
  int it = -1;
  auto next = [&](bool single) -> const ItemW * {
    ++it;
    const int sl = it % kItemsW;
    bool ok = mbar_wait(bar(L::kIFull + sl), (it / kItemsW) & 1, a.status);
    if (!single) ok = __all_sync(0xffffffffu, ok);
    return ok && items[sl].kvh >= 0 ? items + sl : nullptr;
  };
  auto release = [&]() { mbar_arrive(bar(L::kIEmpty + it % kItemsW)); };
  // whether a tile uses block j of the item
  auto uses = [](int j, int n_sink, bool sink, int j0, int j1) {
    return j < n_sink ? sink : j >= j0 && j < j1;
  };

  if (warp >= kSoftWarpsW) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kOtherRegs));
    if (warp == kItemWarpW) {
      // ------------------------------------------------------------ items
      const int32_t n_pairs = a.status[kStatusMergeRows]; // 0: the plan failed its checks
      const int32_t per = a.folds ? 1 : a.parts;          // units a pair
      const int64_t n_items = static_cast<int64_t>(n_pairs) * per * a.Hkv;
      int64_t w = blockIdx.x; // the CTA's first item is its own, the others come from a counter
      auto take = [&]() {
        if (gridDim.x >= n_items) {
          w = n_items;
          return;
        }
        int k = 0;
        if (lane == 0) k = atomicAdd(a.status + kStatusWorkCounter, 1);
        w = gridDim.x + static_cast<int64_t>(__shfl_sync(0xffffffffu, k, 0));
      };
      ItemW x{};
      x.kvh = -1;
      TileKeys tk[2] = {};
      bool has[2] = {false, false};
      int32_t s = 0, s_end = 0; // split of the item, and the one after the pair's last
      bool more = false;        // the folded pair has another split
      for (int i = 0;; ++i) {
        if (more) {
          ++s;
        } else {
          x.kvh = -1;
          while (w < n_items) {
            const int64_t u = w / a.Hkv;
            const int32_t pair = static_cast<int32_t>(u / per);
            // the request of the pair: the largest b with group_off[b] <= pair
            int lo = 0, n = a.batch;
            while (n > 1) {
              const int step = (n + 31) / 32;
              const bool le = lane * step < n && __ldg(a.group_off + lo + lane * step) <= pair;
              const int k = max(0, 31 - __clz(__ballot_sync(0xffffffffu, le)));
              lo += k * step;
              n = min(step, n - k * step);
            }
            const ReqInfo r = a.reqs[lo];
            const int32_t tiles = (r.q_len + T - 1) / T;
            x.tile = NT * (pair - __ldg(a.group_off + lo));
            has[0] = true;
            has[1] = NT == 2 && x.tile + 1 < tiles;
#pragma unroll
            for (int t = 0; t < NT; ++t)
              if (has[t])
                tk[t] = tile_keys(r.q_len, r.kv_len, x.tile + t, T, a.window, a.sinks, a.split, KB);
            s_end = (has[1] ? tk[1].s1 : tk[0].s1) + 1;
            s = tk[0].s0 + static_cast<int32_t>(u - static_cast<int64_t>(pair) * per);
            if (s < s_end) {
              x.kvh = static_cast<int32_t>(w % a.Hkv);
              x.q_start = r.q_start;
              x.q_len = r.q_len;
              x.kv_len = r.kv_len;
              x.page_base = r.page_base;
              x.lo = max(0, r.kv_len - r.q_len + x.tile * T - a.window + 1);
              break;
            }
            take(); // this pair has fewer splits
          }
        }
        if (x.kvh >= 0) {
          const int32_t b0 = s * (a.split / KB), b1 = b0 + a.split / KB; // blocks of the split
          int32_t f[2], e[2], w1 = 0;
          x.n_sink = 0;
          x.w0 = INT32_MAX;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const bool in = has[t] && s >= tk[t].s0 && s <= tk[t].s1;
            x.n_parts[t] = in ? tk[t].s1 - tk[t].s0 + 1 : 0;
            x.part[t] = in ? s - tk[t].s0 : 0;
            x.sink[t] = in && s == tk[t].s0 && tk[t].n_sink > 0;
            f[t] = in ? max(tk[t].first, b0) : INT32_MAX;
            e[t] = in ? min(tk[t].last + 1, b1) : 0;
            if (x.sink[t]) x.n_sink = tk[t].n_sink;
            x.w0 = min(x.w0, f[t]);
            w1 = max(w1, e[t]);
          }
          x.nb = x.n_sink + w1 - x.w0;
          x.steps = x.n_sink > 0 ? (a.sinks - (x.n_sink - 1) * KB + 15) / 16 << 16 : 0;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            x.j0[t] = x.n_parts[t] ? x.n_sink + f[t] - x.w0 : 0;
            x.j1[t] = x.n_parts[t] ? x.n_sink + e[t] - x.w0 : 0;
            // a split's first block starts it, or holds the window's first key
            const int first = tk[t].first >= b0 ? (tk[t].k0 % KB) / 16 : 0;
            const int end = tk[t].last < b1 ? (tk[t].k1 - tk[t].last * KB + 15) / 16 : KB / 16;
            if (x.n_parts[t]) x.steps |= (first | end << 4) << (8 * t);
            // from the last row's window on, up to the first row's position
            const int32_t p0 = x.kv_len - x.q_len + (x.tile + t) * T;
            const int32_t from = max(0, tk[t].k1 - a.window);
            x.w_begin[t] = max(x.j0[t], x.n_sink + (from + KB - 1) / KB - x.w0);
            x.w_end[t] = min(x.j1[t], x.n_sink + (p0 + 1) / KB - x.w0);
          }
        }
        more = x.kvh >= 0 && a.folds && s + 1 < s_end;
        const int sl = i % kItemsW;
        if (i >= kItemsW &&
            !__all_sync(0xffffffffu,
                        mbar_wait(bar(L::kIEmpty + sl), (i / kItemsW - 1) & 1, a.status)))
          break;
        if (lane == 0) {
          items[sl] = x;
          mbar_arrive(bar(L::kIFull + sl));
        }
        if (x.kvh < 0) break;
        // the loads ask three blocks before they end
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kIAsk), i & 1, a.status))) break;
        if (!more) take();
      }
    } else if (warp == kKeyWarpW || warp == kValueWarpW ||
               (ROWS && (warp == kLoad2W || warp == kLoad2W + 1))) {
      // ------------------------------------------------------------ loads
      // lane: the four rows 4*grp .. of a block, column blocks hh, hh + LPG ..
      constexpr int kGroups = KB / 4, LPG = 32 / kGroups;
      const int grp = lane % kGroups, hh = lane / kGroups;
      const int page_mask = (1 << a.page_shift) - 1;
      constexpr bool runs = !ROWS; // a run of 16 keys lies in one page
      const bool second = ROWS && warp >= kLoad2W;
      const bool keys = warp == kKeyWarpW || warp == kLoad2W;
      const void *rows_map = keys ? &a.tm_k : &a.tm_v, *runs_map = keys ? &a.tm_k3 : &a.tm_v3;
      const uint32_t full0 = bar(keys ? L::kKFull : L::kVFull);
      const uint32_t empty0 = bar(keys ? L::kKEmpty : L::kVEmpty);
      bool ok = true;
      int g = 0, n = 0, nq = 0; // blocks, those whose copies were issued, q tile pairs
      while (const ItemW *xp = next(false)) {
        const int nb = xp->nb, n_sink = xp->n_sink, w0 = xp->w0, kvh = xp->kvh;
        const int kv_len = xp->kv_len, lo = xp->lo;
        // steps of block j that either tile needs
        auto steps = [&](int j, int &u, int &v) {
          u = KB / 16;
          v = 0;
#pragma unroll
          for (int t = 0; t < NT; ++t)
            if (uses(j, n_sink, xp->sink[t] != 0, xp->j0[t], xp->j1[t])) {
              const Steps<KB> s{n_sink, xp->j0[t], xp->j1[t],
                                (xp->steps >> (8 * t) & 255) | (xp->steps & 15 << 16)};
              u = min(u, s.u(j));
              v = max(v, s.v(j));
            }
        };
        const int32_t *pages = a.kv_indices + xp->page_base;
        auto wanted = [&](int32_t key) { return key < kv_len && (key >= lo || key < a.sinks); };
        auto key_of = [&](int j) { // the lane's first key of block j
          return (j < n_sink ? j : w0 + j - n_sink) * KB + 4 * grp;
        };
        // page of each of the lane's keys of block j (-1: not wanted)
        auto fetch = [&](int j, int32_t (&pg)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) pg[i] = -1;
          if (j >= nb) return;
          const int32_t key = key_of(j);
          if (runs) { // of the run, if any key of it is wanted
            const int32_t r0 = key - 4 * (grp & 3);
            if ((r0 + 15 >= lo || r0 < a.sinks) && r0 < kv_len)
              pg[0] = __ldg(pages + (r0 >> a.page_shift));
            pg[1] = pg[2] = pg[3] = pg[0];
          } else if (a.page_shift >= 2) { // one page
            if (wanted(key) || wanted(key + 1) || wanted(key + 2) || wanted(key + 3))
              pg[0] = __ldg(pages + (key >> a.page_shift));
            pg[1] = pg[2] = pg[3] = pg[0];
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (wanted(key + i)) pg[i] = __ldg(pages + ((key + i) >> a.page_shift));
          }
        };
        int32_t pg[4];
        fetch(0, pg);
        for (int j = 0; j < nb; ++j, ++g) {
          if (keys && !second && lane == 0 && j == max(0, nb - 3)) mbar_arrive(bar(L::kIAsk));
          const int st = g & 1;
          const int32_t key = key_of(j), run0 = key - 4 * (grp & 3);
          int32_t rows[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            rows[i] = a.kv_rows; // outside the map: zeros
            if (wanted(key + i)) {
              if (pg[i] >= 0 && pg[i] < a.num_pages)
                rows[i] = ((pg[i] << a.page_shift) + ((key + i) & page_mask)) * a.Hkv + kvh;
              else
                atomicOr(a.status, kStatusBadPage);
            }
          }
          // A run of 16 keys of one page is one copy a column block.  Keys of it
          // that are not wanted only cost their column of S, which no row
          // sees; as values they must be zeros (0 * NaN), so such a run of V
          // is gathered row by row.
          const int32_t page = pg[0];
          const bool whole = run0 + 15 < kv_len && (run0 >= lo || run0 + 15 < a.sinks);
          const bool run = runs && page >= 0 && page < a.num_pages && (keys || whole);
          const int32_t slot = run ? (page << a.page_shift) + (run0 & page_mask) : 0;
          int u, v;
          steps(j, u, v);
          const bool needed = (grp >> 2) >= u && (grp >> 2) < v;
          // The MMAs take a whole block: K columns that no row sees may hold
          // anything, V rows must be zeros.
          const bool zeros = !keys && !needed;
          const int copied = keys ? v - u : KB / 16;
          fetch(j + 1, pg); // in flight while this block's copies are issued
          ok = __all_sync(0xffffffffu,
                          g < 2 || mbar_wait(empty0 + 8 * st, ((g >> 1) - 1) & 1, a.status));
          if (!ok) break;
          const uint32_t b = full0 + 8 * st, dst = keys ? sK(st) : sV(st);
          if (lane == 0 && !second) mbar_expect_tx(b, static_cast<uint32_t>(copied) * (16 * D * 2));
          __syncwarp();
          if ((needed && run) || zeros) {
            if (hh == 0 && !second && (grp & 3) < D / 64)
              tma_load_3d(dst + (grp & 3) * L::kAtom + (grp & ~3) * 512, runs_map, 64 * (grp & 3),
                          kvh, zeros ? a.slots : slot, b);
          } else if (needed) {
#pragma unroll
            for (int h = 0; h < D / 64; h += LPG)
              if (h + hh < D / 64 && (!ROWS || (D == 64 ? !second : second == (h / LPG & 1))))
                gather4(dst + (h + hh) * L::kAtom + grp * 512, rows_map, 64 * (h + hh), rows, b);
          }
          n = g + 1;
          if (keys && !second && j == 0) {
            // q of this item while the previous one is still in its last P.V
            ok = __all_sync(0xffffffffu,
                            nq == 0 || mbar_wait(bar(L::kQEmpty), (nq - 1) & 1, a.status));
            if (!ok) break;
            ++nq;
            if (lane == 0) {
              mbar_expect_tx(bar(L::kQFull),
                             ((xp->n_parts[0] > 0) + (xp->n_parts[1] > 0)) * L::kQTile);
#pragma unroll
              for (int t = 0; t < NT; ++t)
                if (xp->n_parts[t] > 0)
#pragma unroll
                  for (int h = 0; h < D / 64; ++h)
                    tma_load_3d(sQ(t) + h * kAtomQW, &a.tm_q, 64 * h, kvh * G,
                                xp->q_start + (xp->tile + t) * T, bar(L::kQFull));
            }
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) release();
      }
      // no copy and no commit outlives the CTA, also when a wait ran out (the
      // block that was begun then is copied in full all the same)
      __syncwarp();
      if (nq > 0) mbar_wait(bar(L::kQFull), (nq - 1) & 1, a.status);
      if (nq > 0 && ok) mbar_wait(bar(L::kQEmpty), (nq - 1) & 1, a.status);
      for (int b = max(0, n - 2); b < n; ++b) {
        mbar_wait(full0 + 8 * (b & 1), (b >> 1) & 1, a.status);
        if (ok) mbar_wait(empty0 + 8 * (b & 1), (b >> 1) & 1, a.status);
      }
    } else if (warp == kMmaWarpW) {
      // ------------------------------------------------------------ MMA issuer
      // The warp runs together, one lane issues: what the MMAs take is uniform.
      // Every block is taken whole: N and the steps of P.V held to what a
      // block's rows see would be operands that follow data, each MMA's from
      // vector registers.
      auto commit = [&](int b) {
        if (elect_one()) mma_commit(bar(b));
        __syncwarp();
      };
      auto all_wait = [&](uint32_t b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(b, parity, a.status)) != 0;
      };
      auto all_test = [&](uint32_t b, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_test(b, parity)) != 0;
      };
      auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      // a K step only advances the address field of a descriptor
      const uint64_t dQ0 = desc_sw128(sQ(0), 16, 1024), dQ1 = desc_sw128(sQ(NT - 1), 16, 1024);
      const uint64_t dK0 = desc_sw128(sK(0), 16, 1024), dK1 = desc_sw128(sK(1), 16, 1024);
      const uint64_t dV0 = desc_sw128(sV(0), L::kAtom, 1024);
      const uint64_t dV1 = desc_sw128(sV(1), L::kAtom, 1024);
      int g = 0, nq = 0;    // blocks and q tile pairs so far
      int ns = 0;           // S blocks so far (one tile)
      int np0 = 0, np1 = 0; // P blocks of each tile so far
      bool ok = true;
      auto issue_s = [&](int t, int buf, int st) {
        const uint64_t dq = t ? dQ1 : dQ0, dk = st ? dK1 : dK0;
        const uint32_t ts = tS(buf);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t qoff = ((kk >> 2) * kAtomQW + (kk & 3) * 32) >> 4;
            const uint32_t koff = ((kk >> 2) * L::kAtom + (kk & 3) * 32) >> 4;
            mma_bf16_ss(ts, dq + qoff, dk + koff, kIdescS, kk > 0);
          }
          mma_commit(bar(L::kSFull + buf));
        }
        __syncwarp();
      };
      auto issue_pv = [&](int t, int buf, int st, bool first) {
        tc_fence_after();
        const uint64_t dv = st ? dV1 : dV0;
        const uint32_t to = tO(t), ts = tS(buf);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < KB / 16; ++kk)
            mma_bf16_ts(to, ts + kk * 8, dv + ((kk * 2048) >> 4), kIdescPV,
                        (!first || kk > 0) ? 1u : 0u);
        }
        __syncwarp();
      };
      while (ok) {
        const ItemW *xp = next(false);
        if (!xp) break;
        const int nb = same(xp->nb), nsk = same(xp->n_sink);
        const bool sk0 = same(xp->sink[0]) != 0, sk1 = same(xp->sink[1]) != 0;
        const int j00 = same(xp->j0[0]), j01 = same(xp->j1[0]);
        const int j10 = same(xp->j0[1]), j11 = same(xp->j1[1]);
        __syncwarp();
        if (lane == 0) release();
        ok = all_wait(bar(L::kQFull), nq & 1);
        ++nq;
        ok = ok && all_wait(bar(L::kKFull + (g & 1)), (g >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if constexpr (NT == 2) {
          // S of this item follows the last P.V of the one before in the pipe;
          // its first P.V waits for P, and so for the epilogue that reads O
          const int first0 = sk0 ? 0 : j00, first1 = sk1 ? 0 : j10;
          if (uses(0, nsk, sk0, j00, j01)) issue_s(0, 0, g & 1);
          if (uses(0, nsk, sk1, j10, j11)) issue_s(1, 1, g & 1);
          commit(L::kKEmpty + (g & 1));
          if (nb == 1) commit(L::kQEmpty);
          // The pipe holds some 8 MMAs: what the next ones wait for is asked
          // for while it has work (asked for at the head of a block, it ran dry
          // for 600 cycles of 2990).  A test, as a wait for a phase that is not
          // complete would hold the warp.
          bool v_rdy = false, k_rdy = false;
          for (int j = 0; j < nb && ok; ++j, ++g) {
            const int st = g & 1, s1 = st ^ 1, j1 = j + 1;
            const bool u0 = uses(j, nsk, sk0, j00, j01), u1 = uses(j, nsk, sk1, j10, j11);
            ok = v_rdy || all_wait(bar(L::kVFull + st), (g >> 1) & 1);
            if (!ok) break;
            if (u0) {
              ok = all_wait(bar(L::kPFull + 0), np0 & 1);
              ++np0;
              if (!ok) break;
              issue_pv(0, 0, st, j == first0);
              if (j1 == j01) commit(L::kODone + 0);
            }
            if (j1 < nb) {
              ok = k_rdy || all_wait(bar(L::kKFull + s1), ((g + 1) >> 1) & 1);
              if (!ok) break;
              tc_fence_after();
              if (uses(j1, nsk, sk0, j00, j01)) issue_s(0, 0, s1);
            }
            if (u1) {
              ok = all_wait(bar(L::kPFull + 1), np1 & 1);
              ++np1;
              if (!ok) break;
              issue_pv(1, 1, st, j == first1);
              if (j1 == j11) commit(L::kODone + 1);
            }
            v_rdy = j1 < nb && all_test(bar(L::kVFull + s1), ((g + 1) >> 1) & 1);
            k_rdy = j1 + 1 < nb && all_test(bar(L::kKFull + st), ((g + 2) >> 1) & 1);
            if (j1 < nb && uses(j1, nsk, sk1, j10, j11)) issue_s(1, 1, s1);
            if (elect_one()) {
              mma_commit(bar(L::kVEmpty + st));
              if (j1 < nb) mma_commit(bar(L::kKEmpty + s1));
              if (j1 == nb - 1) mma_commit(bar(L::kQEmpty));
            }
            __syncwarp();
          }
        } else {
          // one tile, two S buffers: the next block's S runs while this one's
          // softmax does
          issue_s(0, ns & 1, g & 1);
          ++ns;
          commit(L::kKEmpty + (g & 1));
          if (nb == 1) commit(L::kQEmpty);
          for (int j = 0; j < nb && ok; ++j, ++g) {
            const int st = g & 1, s1 = st ^ 1;
            if (j + 1 < nb) {
              ok = all_wait(bar(L::kKFull + s1), ((g + 1) >> 1) & 1);
              if (!ok) break;
              tc_fence_after();
              issue_s(0, ns & 1, s1);
              ++ns;
              commit(L::kKEmpty + s1);
              if (j + 2 == nb) commit(L::kQEmpty);
            }
            ok = all_wait(bar(L::kVFull + st), (g >> 1) & 1) &&
                 all_wait(bar(L::kPFull + (np0 & 1)), (np0 >> 1) & 1);
            if (!ok) break;
            issue_pv(0, np0 & 1, st, j == 0);
            commit(L::kODone + (np0 & 1));
            ++np0;
            commit(L::kVEmpty + st);
          }
        }
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kSoftRegs));
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int gs = __ffs(G) - 1; // G is a power of two
    int ns = 0, no = 0;        // S blocks and O tiles of this q tile so far
    float run_lse = -INFINITY; // of the splits folded so far
    while (const ItemW *xp = next(false)) {
      // read again where they are used: the scores need the registers
      const volatile ItemW *vx = xp;
      float m = -INFINITY, l = 0.f; // running max (log2 units) and sum
      bool failed = false;
      bool begun = false; // O holds an earlier block's
      for (int j = vx->sink[t] ? 0 : vx->j0[t]; j < vx->j1[t]; ++j) {
        if (j == vx->n_sink && vx->sink[t]) j = vx->j0[t]; // past what only the other tile sees
        const bool whole = j >= vx->w_begin[t] && j < vx->w_end[t];
        const int buf = NT == 2 ? t : ns & 1;
        failed = __any_sync(
            0xffffffffu, !mbar_wait(bar(L::kSFull + buf), (NT == 2 ? ns : ns >> 1) & 1, a.status));
        if (failed) break;
        tc_fence_after();
        const uint32_t srow = tS(buf) + lane_base;
        float alpha = 1.f, m_sub = 0.f;
        auto move_max = [&](float bm) { // bm: the block's largest score
          bm = bm == -INFINITY ? -INFINITY : bm * a.scale_log2;
          if (bm > m + kRescaleW || (m == -INFINITY && bm != -INFINITY)) {
            alpha = ex2(m - bm); // 0 when m == -inf
            m = bm;
          }
          m_sub = m == -INFINITY ? 0.f : m;
        };
        // P = 2^(s * scale - m) of 32 columns as bf16 pairs over 16 of S's
        uint64_t psum2 = 0;
        auto weights = [&](int c, const uint32_t (&v)[32]) {
          const uint64_t scale2 = f32x2(a.scale_log2, a.scale_log2);
          const uint64_t neg2 = f32x2(-m_sub, -m_sub);
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float x0, x1;
            f32x2_split(
                ffma2r(f32x2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), scale2, neg2), x0,
                x1);
            const float q0 = ex2(x0), q1 = ex2(x1);
            psum2 = fadd2(psum2, f32x2(q0, q1));
            pk[i / 2] = pack_bf16(q0, q1);
          }
          tmem_st16(srow + c * 16, pk);
        };
        if (whole) {
          uint32_t v[KB / 32][32]; // the row's scores, in registers from here on
          float b4[KB / 32];       // the loads give the maximum of their 32 columns
#pragma unroll
          for (int c = 0; c < KB / 32; ++c) tmem_ld32_max(srow + c * 32, v[c], b4[c]);
          tmem_wait_ld();
          float bm = b4[0];
#pragma unroll
          for (int c = 1; c < KB / 32; ++c) bm = fmaxf(bm, b4[c]);
          move_max(bm);
#pragma unroll
          for (int c = 0; c < KB / 32; ++c) weights(c, v[c]);
        } else {
          // The row sees keys < p1, of them those >= p1 - window or < sinks; what
          // the warp's rows see of 32 columns may be all of them, none (no
          // exponentials), or not the same (a test a column): the first row's
          // limits are `span` below the last one's.
          uint32_t v[KB / 32][32];
          float b4[KB / 32];
          uint32_t none = 0; // bit c: none of columns 32c ..
#pragma unroll
          for (int c = 0; c < KB / 32; ++c) tmem_ld32_max(srow + c * 32, v[c], b4[c]);
          const int key0 = (j < vx->n_sink ? j : vx->w0 + j - vx->n_sink) * KB;
          const int span = 31 >> gs, snk = a.sinks - key0;
          const int vis_0 = vx->kv_len - vx->q_len + (vx->tile + t) * T +
                            (((warp & 3) * 32) >> gs) + 1 - key0;
          const int lo_0 = vis_0 - a.window, n_vis = vis_0 + (lane >> gs);
          tmem_wait_ld();
          float bm = -INFINITY;
#pragma unroll
          for (int c = 0; c < KB / 32; ++c) {
            if (vis_0 + span <= 32 * c || (lo_0 >= 32 * c + 32 && snk <= 32 * c)) {
              none |= 1u << c;
              continue;
            }
            if (vis_0 < 32 * c + 32 || (lo_0 + span > 32 * c && snk < 32 * c + 32)) {
              const uint32_t vis = first_bits(n_vis - 32 * c) &
                                   (~first_bits(n_vis - a.window - 32 * c) | first_bits(snk - 32 * c));
              b4[c] = -INFINITY;
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                if (!((vis >> i) & 1u)) v[c][i] = 0xff800000u; // -inf: a weight of zero
                if (!((vis >> i) & 2u)) v[c][i + 1] = 0xff800000u;
                b4[c] = fmax3(b4[c], __uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1]));
              }
            }
            bm = fmaxf(bm, b4[c]);
          }
          move_max(bm);
#pragma unroll
          for (int c = 0; c < KB / 32; ++c) {
            if (none >> c & 1u) {
              const uint32_t zero[16] = {};
              tmem_st16(srow + c * 16, zero);
            } else {
              weights(c, v[c]);
            }
          }
        }
        float ps0, ps1;
        f32x2_split(psum2, ps0, ps1);
        l = fmaf(l, alpha, ps0 + ps1);
        // rescale the running O row when the max moved, once the previous P.V
        // has completed (two tiles: S of this block was issued after it)
        if (begun && __any_sync(0xffffffffu, alpha != 1.f)) {
          if constexpr (NT == 1) {
            failed = __any_sync(0xffffffffu, !mbar_wait(bar(L::kODone + ((ns - 1) & 1)),
                                                        ((ns - 1) >> 1) & 1, a.status));
            if (failed) break;
            tc_fence_after();
          }
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(tO(t) + lane_base + c * 16, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16(tO(t) + lane_base + c * 16, o);
          }
        }
        begun = true;
        ++ns;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kPFull + buf));
      }
      // epilogue: o_s = O / l; bf16 when the tile has one state or this is the
      // last of the folded ones, else the fp32 state; a thread stores its own row
      const ItemW &x = *xp;
      const int n_parts = x.n_parts[t];
      int ln = lane; // opaque: what follows from it is not kept over the blocks
      asm volatile("" : "+r"(ln));
      if (n_parts > 0) {
        // warp-uniform (tcgen05.ld is warp-collective): a warp with a failed
        // wait writes zeros
        // one tile: a barrier for every other P.V, as the last but one may still run
        const int which = NT == 2 ? t : (ns - 1) & 1, phase = NT == 2 ? no : (ns - 1) >> 1;
        const bool have_o = __all_sync(
            0xffffffffu, !failed && mbar_wait(bar(L::kODone + which), phase & 1, a.status));
        ++no;
        tc_fence_after();
        const bool some = have_o && !(l == 0.f); // NaN sums stay NaN
        const float inv_l = some ? __frcp_rn(l) : 0.f; // o_s = O * (1/l)
        float lse = some ? __fmul_rn(__fadd_rn(m, lg2(l)), kLn2) : -INFINITY;
        const int part = x.part[t];
        const bool folds = a.folds && n_parts > 1; // uniform over the tile, as the next two
        const bool add = folds && part > 0;
        const bool last = folds ? part == n_parts - 1 : n_parts == 1;
        float wa = 1.f, wb = 0.f;
        int how = kFoldTake;
        if (add) {
          how = fold_weights(run_lse, lse, wa, wb);
          lse = run_lse;
        } else {
          run_lse = lse;
        }
        const int Dr = a.D; // head_dim 96 runs on the 128-wide layout, zero-padded
        // rows of out, or of the states for the merge: token, part, head
        const int tok0 = (x.tile + t) * T;
        const int64_t token = static_cast<int64_t>(x.q_start) + tok0 + (row >> gs);
        const int64_t dst_row = (last ? token : token * a.parts + part) * a.Hq + x.kvh * G +
                                (((warp & 3) * 32 + ln) & (G - 1));
        const bool store = tok0 + (row >> gs) < x.q_len;
        // the running state, this CTA's own: float4 column x tile row
        float4 *run = reinterpret_cast<float4 *>(a.part_o) +
                      static_cast<int64_t>(blockIdx.x) * (NT * kTileRows * D / 4) +
                      t * (kTileRows * D / 4) + (warp & 3) * 32 + ln;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          if (have_o) {
            tmem_ld32(tO(t) + lane_base + c * 32, v);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = some ? __float_as_uint(__fmul_rn(__uint_as_float(v[i]), inv_l)) : 0u;
          if (add) {
            float4 prev[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) // all eight in flight
              asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(prev[q].x), "=f"(prev[q].y), "=f"(prev[q].z), "=f"(prev[q].w)
                           : "l"(run + (c * 8 + q) * kTileRows)
                           : "memory");
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float o[4] = {prev[q].x, prev[q].y, prev[q].z, prev[q].w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                v[q * 4 + i] = __float_as_uint(
                    fold_value(how, wa, wb, o[i], __uint_as_float(v[q * 4 + i])));
            }
          }
          if (last) {
            if (store && c * 32 < Dr) {
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 16; ++i)
                w[i] = pack_bf16(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
              store_words(a.out + dst_row * Dr + c * 32, w);
            }
          } else if (folds) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              run[(c * 8 + q) * kTileRows] =
                  make_float4(__uint_as_float(v[q * 4]), __uint_as_float(v[q * 4 + 1]),
                              __uint_as_float(v[q * 4 + 2]), __uint_as_float(v[q * 4 + 3]));
          } else if (store && c * 32 < Dr) {
            store_words(a.part_o + dst_row * Dr + c * 32, v);
          }
        }
        if (store && (last || !folds)) {
          if (!last) a.part_lse[dst_row] = lse;
          else if (a.lse) a.lse[dst_row] = lse;
        }
      }
      __syncwarp();
      if (lane == 0) release();
      if (failed) break;
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarpW) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool ROWS>
cudaError_t launch_window_dr(const WindowPrefillArgs &a, int64_t items, cudaStream_t s) {
  using L = SmemW<D, ROWS>;
  static std::atomic<uint64_t> ready{0};
  int sms = 0;
  const cudaError_t e = prepare_launch(reinterpret_cast<const void *>(prefill_window_kernel<D, ROWS>),
                                       L::kAlloc, ready, &sms);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // (the running states of folded pairs are kept for kFoldCtas CTAs)
  cfg.gridDim = dim3(static_cast<unsigned>(std::min({static_cast<int64_t>(sms), kFoldCtas, items})));
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_window_kernel<D, ROWS>, a);
}

template <int D>
cudaError_t launch_window_d(const WindowPrefillArgs &a, int64_t items, cudaStream_t s) {
  return a.page_shift >= 4 ? launch_window_dr<D, false>(a, items, s)
                           : launch_window_dr<D, true>(a, items, s);
}

} // namespace

cudaError_t launch_prefill_window(const AttnArgs &a, const int32_t *group_off, int folds,
                                  cudaStream_t s) {
  WindowPrefillArgs w{};
  w.Hq = a.Hq;
  w.Hkv = a.Hkv;
  w.D = a.D;
  w.G = a.G;
  w.split = a.split;
  w.tile_tokens = a.tile_tokens;
  w.batch = a.batch;
  w.page_shift = a.page_shift;
  w.window = a.window;
  w.sinks = a.sinks;
  w.parts = a.parts;
  w.folds = folds;
  w.kv_rows = a.kv_rows;
  w.slots = a.kv_rows / a.Hkv;
  w.scale_log2 = a.scale_log2;
  w.num_pages = a.num_pages;
  w.reqs = a.reqs;
  w.group_off = group_off;
  w.kv_indices = a.kv_indices;
  w.part_o = a.part_o;
  w.part_lse = a.part_lse;
  w.out = a.out;
  w.lse = a.lse;
  w.status = a.status;
  w.tm_q = a.tm_q;
  w.tm_k = a.tm_k;
  w.tm_v = a.tm_v;
  w.tm_k3 = a.tm_k3;
  w.tm_v3 = a.tm_v3;
  const int64_t items = a.n_units * a.Hkv;
  // head_dim 96 runs on the 128-wide layout: the tensor maps read columns
  // 96..127 as zeros
  if (a.D == 256) return launch_window_d<256>(w, items, s);
  return a.D > 64 ? launch_window_d<128>(w, items, s) : launch_window_d<64>(w, items, s);
}

} // namespace bia
