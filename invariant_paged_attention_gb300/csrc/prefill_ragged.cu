// Attention of packed sequences over contiguous keys and values on the tensor
// cores (tcgen05 + TMEM): the extend of prefill.cu (128-row q tiles of 128/G
// tokens x G heads, "sglang PR #43612", Summary; fixed split-KV tiles merged
// in order, "sglang PR #10417 [POC] Support deterministic inference",
// Modifications; every reduction boundary anchored at absolute key 0) for
// k, v [total_kv, Hkv, D] instead of pages.
//
// A persistent CTA per SM takes items: two consecutive q tiles of one request
// against one split and kv head.  Its roles (12 warps) walk the same items
// through a ring of records and each runs ahead as far as its buffers allow,
// so the next item's q, K, V and first S overlap this one's last softmax,
// P.V and stores: 0-3 and 4-7 softmax + epilogue of the two tiles, 8 issues
// the MMAs and owns TMEM, 9 loads, 10 fetches items, 11 completes V tiles.
// A 128-key block of K or V is D/64 tiled TMA boxes (64 columns x 1 head x
// 128 tokens) straight into the 128-byte-swizzled operand tile, two stages
// deep.  Rows past the request's last key belong to the next request: their S
// columns are masked, and their V rows are overwritten with zeros before the
// block's P.V (0 * NaN would reach the row).
//
// With few items (chunks over a long prefix) the splits of a q tile are items
// of their own, their fp32 states go to the workspace and a merge kernel
// folds them.  With many, none of them longer than a CTA's share of the call,
// an item of the plan is the whole q tile pair: the CTA runs through its splits and folds each state into the running one as
// the merge would (fold.cuh), which saves a state per row and split in memory
// and the merge (one 16384-token prompt, 32 heads x 128: 1.81 -> 1.64 ms, the
// workspace 1.1 GB -> 20 MB).  The bits are the same either way.
//
// Bound by the chain of a q tile: S, softmax (1350 cycles), P.V and the waits
// between them take ~3400 cycles a block where the two tiles' MMAs take 2048
// alone (2800 with the S operands' shared-memory reads at their limit).  16384
// tokens, 32/8 heads x 128: 1662 us a call, 1320 TFLOP/s, 77 % of the sustained
// cuBLAS rate; three prompts of 4096 to 8192 tokens 1250 (950 at 96 columns, 760
// at 64, where a block's MMAs halve and its softmax does not);
// 6 prompts of 100 to 2048 tokens (4 to 5 blocks an item) 61 us, 730 TFLOP/s.
//
// A call of up to 32 requests without splits to merge and with an SM for
// every item has no plan: each CTA's item warp works its unit out of the index
// arrays (a prompt of 256 tokens: 18 -> 14 us).
//
// Invariance: as for prefill.cu; single-token tiles run here too, so a row's
// bits do not depend on where a chunk boundary falls at all.
#include "bia_internal.h"
#include "fold.cuh"
#include "ptx.cuh"

#include <algorithm>

namespace bia {

namespace {

constexpr int kSoftWarpsR = 8; // 0-3 and 4-7: one warp per 32 rows of each q tile
constexpr int kMmaWarpR = 8;
constexpr int kProdWarpR = 9;
constexpr int kItemWarpR = 10;
constexpr int kTailWarpR = 11;
constexpr int kThreadsR = 384;
// Registers: the softmax warps hold a whole S row (at 168 they spill, and so
// do the MMA issuer's descriptors below 72: 1.88 -> 1.67 ms for 16384 tokens)
constexpr int kSoftRegsR = 216, kOtherRegsR = 72;
static_assert(8 * kSoftRegsR + 4 * kOtherRegsR <= 12 * 168, "registers of the launch");
constexpr int kItemsR = 3;              // items in flight: loads run ahead of the stores
constexpr int kAtomR = kTileRows * 128; // one SW128 column block: 128 rows x 64 bf16
// log2 units the running max may lag a block's: weights reach 2^16 (bf16 and
// fp32 sums keep their relative precision), and fewer blocks rescale O than at
// 8 (16384 tokens: 1.65 -> 1.62 ms; nothing more at 40)
constexpr float kRescaleR = 16.0f;

// What the kernel needs of AttnArgs, without the tensor maps it does not use.
struct RaggedArgs {
  int32_t Hq, Hkv, D, G, causal, split, tile_tokens, batch, kv_rows;
  float scale_log2;
  int64_t n_units;
  const ReqInfo *reqs;
  const Unit *units;
  const int32_t *qo_indptr, *kv_indptr; // of a call that plans itself, else kv_indptr NULL
  int64_t total_q;
  float *part_o, *part_lse;
  uint16_t *out;
  float *lse;
  int32_t *status;
  CUtensorMap tm_q, tm_k, tm_v;
};

// One (unit, kv head): what the roles need of it.  kvh < 0 ends the list.
struct alignas(16) ItemR {
  int32_t kvh, tile, split, pad;
  int32_t q_start, q_len, kv_len, row0; // row0: k, v row of the split's first key
  int64_t rowbase; // -1: the splits are folded here
  int32_t nsp, key_begin;
  int32_t n_blocks[2], n_splits[2]; // per q tile; n_splits 0: no such tile
};

template <int D>
struct SmemR {
  static constexpr int kTile = kTileRows * D * 2; // one Q, K or V tile
  static constexpr int kQ = 0;
  static constexpr int kKV = 2 * kTile; // stage s: K at kKV + 2s*kTile, V after it
  static constexpr int kItem = 6 * kTile;
  static constexpr int kBar = kItem + kItemsR * static_cast<int>(sizeof(ItemR));
  static constexpr int kQFull = 0, kQEmpty = 1, kKFull = 2, kVFull = 4, kKEmpty = 6, kVEmpty = 8,
                       kSFull = 10, kPFull = 12, kODone = 14, kVGo = 16, kVTail = 18,
                       kIAsk = 20, kIFull = 21, kIEmpty = kIFull + kItemsR,
                       kNumBars = kIEmpty + kItemsR;
  static constexpr int kSlot = kBar + kNumBars * 8;
  static constexpr int kAlloc = kSlot + 16 + 1024;
};

// N words of a thread's row, 32 bytes a store where out allows it
template <int N>
__device__ __forceinline__ void store_row(void *p, const uint32_t (&w)[N]) {
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

template <int D>
__global__ void __launch_bounds__(kThreadsR, 1)
    prefill_ragged_kernel(const __grid_constant__ RaggedArgs a) {
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
  ItemR *items = reinterpret_cast<ItemR *>(smem + L::kItem);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kSlot);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == kMmaWarpR) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
  if (warp == kProdWarpR && lane < (a.kv_rows > 0 ? 3 : 1)) // without keys there is only q's
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0   ? &a.tm_q
                                                  : lane == 1 ? &a.tm_k
                                                              : &a.tm_v)
                 : "memory");
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
      mbar_init(bar(L::kVGo + s), 1);
      mbar_init(bar(L::kVTail + s), 1);
    }
    mbar_init(bar(L::kIAsk), 1);
    for (int s = 0; s < kItemsR; ++s) {
      mbar_init(bar(L::kIFull + s), 1);
      mbar_init(bar(L::kIEmpty + s), kSoftWarpsR + 3);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // TMEM columns: S_A [0,128) S_B [128,256) O_A [256,256+D) O_B [256+D,256+2D)
  auto tS = [&](int t) { return tmem + 128u * t; };
  auto tO = [&](int t) { return tmem + 256u + static_cast<uint32_t>(D) * t; };
  grid_dep_wait();   // the plan is complete
  grid_dep_launch(); // the next kernel of the call may start launching
  const int G = a.G, T = a.tile_tokens;

  // A role's walk over the CTA's items: next() gives the item or null at the
  // end, release() hands its slot back (one arrival per role or warp).
  int it = -1; // items taken by this warp
  auto next = [&]() -> const ItemR * {
    ++it;
    const int sl = it % kItemsR;
    if (!mbar_wait(bar(L::kIFull + sl), (it / kItemsR) & 1, a.status)) return nullptr;
    return items[sl].kvh < 0 ? nullptr : items + sl;
  };
  auto release = [&]() { mbar_arrive(bar(L::kIEmpty + it % kItemsR)); };
  // the last block of the item holds rows of the next request: the tail warp
  // completes its V
  auto v_tail_rows = [&](const ItemR &x, int nb) { // real rows of the last block
    return x.kv_len - (x.key_begin + (nb - 1) * kKvBlock);
  };

  if (warp >= kSoftWarpsR) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegsR));
    if (warp == kItemWarpR) {
      // ------------------------------------------------------------ items
      const int64_t n_items = a.n_units * a.Hkv;
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
      // up to 32 requests' records stay in the lanes: an item is then one
      // memory latency away, not two
      ReqInfo mine{};
      Unit own{-1, 0, 0, 0}; // the only unit of a CTA that plans itself
      if (a.kv_indptr) {
        const bool live = lane < a.batch;
        const int r = live ? lane : a.batch;
        const int32_t q0 = a.qo_indptr[r], k0 = a.kv_indptr[r];
        const int64_t ql = static_cast<int64_t>(a.qo_indptr[live ? r + 1 : r]) - q0;
        const int64_t kl = static_cast<int64_t>(a.kv_indptr[live ? r + 1 : r]) - k0;
        bool ok = ql >= 0 && kl >= 0 && kl <= INT32_MAX / 2 && ql <= INT32_MAX / 2 &&
                  (!a.causal || ql <= kl) && (lane > 0 || (q0 == 0 && k0 >= 0)) &&
                  (lane != a.batch - 1 || (q0 + ql == a.total_q && k0 + kl == a.kv_rows));
        mine.q_start = q0;
        mine.q_len = ok ? static_cast<int32_t>(ql) : 0;
        mine.kv_len = ok ? static_cast<int32_t>(kl) : 0;
        mine.nsp = 1;
        mine.rowbase = -1;
        mine.page_base = k0;
        const int32_t tiles = (mine.q_len + T - 1) / T, groups = (tiles + 1) / 2;
        ok = ok && (tiles == 0 ||
                    tile_splits(mine.q_len, mine.kv_len, tiles - 1, T, a.causal, a.split) == 1);
        int64_t end = groups; // of the request's groups
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int64_t x = __shfl_up_sync(0xffffffffu, end, off);
          if (lane >= off) end += x;
        }
        ok = __all_sync(0xffffffffu, ok) && __shfl_sync(0xffffffffu, end, 31) == a.n_units;
        // no other error can be noted before: the kernel's waits last seconds
        if (blockIdx.x == 0 && lane == 0) a.status[0] = ok ? 0 : kStatusPlanMismatch;
        if (ok) {
          const int64_t g = w / a.Hkv;
          const int b = __popc(__ballot_sync(0xffffffffu, end <= g)); // the first that ends past g
          own.b = b;
          own.tile = 2 * static_cast<int32_t>(g - __shfl_sync(0xffffffffu, end - groups, b));
          own.ntiles = min(2, __shfl_sync(0xffffffffu, tiles, b) - own.tile);
        } else { // as the planner: NaN instead of stale values
          w = n_items;
          const int64_t step = static_cast<int64_t>(gridDim.x) * 32, rows = a.total_q * a.Hq;
          for (int64_t e = blockIdx.x * 32 + lane; e < rows * a.D; e += step)
            a.out[e] = 0x7fc0u; // bf16 NaN
          for (int64_t e = blockIdx.x * 32 + lane; a.lse && e < rows; e += step)
            a.lse[e] = __int_as_float(0x7fc00000);
        }
      } else if (a.batch <= 32 && lane < a.batch) {
        mine = a.reqs[lane];
      }
      auto request = [&](int b) {
        if (a.batch > 32) return a.reqs[b];
        ReqInfo r;
        r.q_start = __shfl_sync(0xffffffffu, mine.q_start, b);
        r.q_len = __shfl_sync(0xffffffffu, mine.q_len, b);
        r.kv_len = __shfl_sync(0xffffffffu, mine.kv_len, b);
        r.nsp = __shfl_sync(0xffffffffu, mine.nsp, b);
        r.rowbase = __shfl_sync(0xffffffffu, mine.rowbase, b);
        r.page_base = __shfl_sync(0xffffffffu, mine.page_base, b);
        return r;
      };
      ItemR x{};
      x.kvh = -1;
      int ns[2] = {0, 0}; // splits of the two tiles
      bool more = false;  // the folded item has another split
      for (int i = 0;; ++i) {
        if (more) {
          ++x.split;
          x.key_begin += a.split;
          x.row0 += a.split;
        } else {
          x.kvh = -1;
          while (w < n_items) {
            const Unit u = a.kv_indptr ? own : a.units[w / a.Hkv];
            if (u.b >= 0) { // not retired by the plan
              const ReqInfo r = request(u.b);
              x.kvh = static_cast<int32_t>(w % a.Hkv);
              x.tile = u.tile;
              x.split = u.split;
              x.q_start = r.q_start;
              x.q_len = r.q_len;
              x.kv_len = r.kv_len;
              x.key_begin = u.split * a.split;
              x.row0 = r.page_base + x.key_begin;
              x.rowbase = r.rowbase;
              x.nsp = r.nsp;
#pragma unroll
              for (int t = 0; t < 2; ++t)
                ns[t] = t < u.ntiles ? tile_splits(r.q_len, r.kv_len, u.tile + t, T, a.causal,
                                                   a.split) : 0;
              break;
            }
            take();
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const bool has = x.split < ns[t];
          const int32_t last = tile_last_key(x.q_len, x.kv_len, x.tile + t, T, a.causal);
          const int32_t end = min(x.key_begin + a.split, last + 1);
          x.n_splits[t] = has ? ns[t] : 0;
          x.n_blocks[t] =
              has && end > x.key_begin ? (end - x.key_begin + kKvBlock - 1) / kKvBlock : 0;
        }
        more = x.kvh >= 0 && x.rowbase < 0 && x.split + 1 < max(ns[0], ns[1]);
        const int sl = i % kItemsR;
        if (i >= kItemsR &&
            !__all_sync(0xffffffffu,
                        mbar_wait(bar(L::kIEmpty + sl), (i / kItemsR - 1) & 1, a.status)))
          break;
        if (lane == 0) {
          items[sl] = x;
          mbar_arrive(bar(L::kIFull + sl));
        }
        if (x.kvh < 0) break;
        // the loads ask three blocks before they end: late enough for the
        // counter to balance the CTAs, early enough to hide the fetch
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kIAsk), i & 1, a.status))) break;
        if (!more) take();
      }
    } else if (warp == kProdWarpR) {
      // ------------------------------------------------------------ loads
      if (lane == 0) {
        bool ok = true;
        int g = 0, nk = 0, nq = 0; // blocks, K blocks and q tile pairs loaded
        while (const ItemR *xp = next()) {
          const ItemR x = *xp;
          release();
          const int nb = max(x.n_blocks[0], x.n_blocks[1]);
          if (nb == 0) mbar_arrive(bar(L::kIAsk));
          for (int j = 0; j < nb && ok; ++j, ++g) {
            if (j == max(0, nb - 3)) mbar_arrive(bar(L::kIAsk));
            const int st = g & 1;
            const int32_t row = x.row0 + j * kKvBlock;
            ok = g < 2 || mbar_wait(bar(L::kKEmpty + st), ((g >> 1) - 1) & 1, a.status);
            if (!ok) break;
            mbar_expect_tx(bar(L::kKFull + st), L::kTile);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(sK(st) + h * kAtomR, &a.tm_k, 64 * h, x.kvh, row, bar(L::kKFull + st));
            nk = g + 1;
            if (j == 0) {
              // q of this item while the previous one is still in its last P.V
              ok = nq == 0 || mbar_wait(bar(L::kQEmpty), (nq - 1) & 1, a.status);
              if (!ok) break;
              ++nq;
              mbar_expect_tx(bar(L::kQFull),
                             ((x.n_splits[0] > 0) + (x.n_splits[1] > 0)) * L::kTile);
#pragma unroll
              for (int t = 0; t < 2; ++t)
                if (x.n_splits[t] > 0)
#pragma unroll
                  for (int h = 0; h < D / 64; ++h)
                    tma_load_3d(sQ(t) + h * kAtomR, &a.tm_q, 64 * h, x.kvh * G,
                                x.q_start + (x.tile + t) * T, bar(L::kQFull));
            }
            ok = g < 2 || mbar_wait(bar(L::kVEmpty + st), ((g >> 1) - 1) & 1, a.status);
            if (!ok) break;
            mbar_expect_tx(bar(L::kVFull + st), L::kTile);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_3d(sV(st) + h * kAtomR, &a.tm_v, 64 * h, x.kvh, row, bar(L::kVFull + st));
            if (j == nb - 1 && v_tail_rows(x, nb) < kKvBlock) mbar_arrive(bar(L::kVGo + st));
          }
          if (!ok) break;
        }
        // no copy and no commit outlives the CTA, also when a wait ran out
        if (nq > 0) mbar_wait(bar(L::kQFull), (nq - 1) & 1, a.status);
        if (nq > 0 && ok) mbar_wait(bar(L::kQEmpty), (nq - 1) & 1, a.status);
        for (int b = max(0, nk - 2); b < nk; ++b) {
          mbar_wait(bar(L::kKFull + (b & 1)), (b >> 1) & 1, a.status);
          if (ok) mbar_wait(bar(L::kKEmpty + (b & 1)), (b >> 1) & 1, a.status);
        }
        for (int b = max(0, g - 2); b < g; ++b) {
          mbar_wait(bar(L::kVFull + (b & 1)), (b >> 1) & 1, a.status);
          if (ok) mbar_wait(bar(L::kVEmpty + (b & 1)), (b >> 1) & 1, a.status);
        }
      }
    } else if (warp == kTailWarpR) {
      // ------------------------------------------------------------ zeros behind the last key
      // Asked by the loads, per stage: when a request arrives, the stage's
      // current phase is that block's (a parity cannot tell a phase further on),
      // and the stage's next request follows the P.V of this one.
      int g = 0;
      uint32_t asked = 0; // parity of the requests of each stage
      while (const ItemR *xp = next()) {
        const int nb = max(xp->n_blocks[0], xp->n_blocks[1]);
        const int tail = v_tail_rows(*xp, nb);
        __syncwarp();
        if (lane == 0) release();
        g += nb;
        if (nb == 0 || tail >= kKvBlock) continue;
        const int b = g - 1, st = b & 1;
        if (!__all_sync(0xffffffffu,
                        mbar_wait(bar(L::kVGo + st), (asked >> st) & 1, a.status) &&
                            mbar_wait(bar(L::kVFull + st), (b >> 1) & 1, a.status)))
          break;
        asked ^= 1u << st;
        uint8_t *v = smem + L::kKV + (2 * st + 1) * L::kTile;
        for (int i = tail * 8 + lane; i < kTileRows * 8; i += 32)
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            *reinterpret_cast<uint4 *>(v + h * kAtomR + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async(); // the zeros are read by the MMA (async proxy)
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kVTail + st));
      }
    } else if (warp == kMmaWarpR) {
      // ------------------------------------------------------------ MMA issuer
      if (lane == 0) {
        // descriptors built once: a K step only advances the address field
        const uint64_t dQ0 = desc_sw128(sQ(0), 16, 1024), dQ1 = desc_sw128(sQ(1), 16, 1024);
        const uint64_t dK0 = desc_sw128(sK(0), 16, 1024), dK1 = desc_sw128(sK(1), 16, 1024);
        const uint64_t dV0 = desc_sw128(sV(0), kAtomR, 1024), dV1 = desc_sw128(sV(1), kAtomR, 1024);
        int g = 0, nq = 0;      // blocks and q tile pairs so far
        uint32_t tails = 0;        // parity of each stage's completed V tails
        int np0 = 0, np1 = 0;      // P blocks of each tile so far
        bool ok = true;
        auto issue_s = [&](int t, int st) {
          uint64_t dq = t ? dQ1 : dQ0, dk = st ? dK1 : dK0;
          asm volatile("" : "+l"(dq), "+l"(dk)); // kept from hoisting: 32 registers
          const uint32_t ts = tS(t);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t koff = ((kk >> 2) * kAtomR + (kk & 3) * 32) >> 4;
            mma_bf16_ss(ts, dq + koff, dk + koff, kIdescS, kk > 0);
          }
          mma_commit(bar(L::kSFull + t));
        };
        auto issue_pv = [&](int t, int st, int &np, bool first, bool last, bool rdy) {
          ok = ok && (rdy || mbar_wait(bar(L::kPFull + t), np & 1, a.status));
          if (!ok) return;
          ++np;
          tc_fence_after();
          uint64_t dv = st ? dV1 : dV0;
          asm volatile("" : "+l"(dv));
          const uint32_t to = tO(t), ts = tS(t);
#pragma unroll
          for (int kk = 0; kk < kKvBlock / 16; ++kk)
            mma_bf16_ts(to, ts + kk * 8, dv + ((kk * 2048) >> 4), kIdescPV,
                        (!first || kk > 0) ? 1u : 0u);
          if (last) mma_commit(bar(L::kODone + t));
        };
        while (ok) {
          const ItemR *xp = next();
          if (!xp) break;
          const int nb0 = xp->n_blocks[0], nb1 = xp->n_blocks[1];
          const int nb = max(nb0, nb1);
          const bool v_tail = v_tail_rows(*xp, nb) < kKvBlock;
          release();
          if (nb == 0) continue;
          ok = mbar_wait(bar(L::kQFull), nq & 1, a.status);
          ++nq;
          ok = ok && mbar_wait(bar(L::kKFull + (g & 1)), (g >> 1) & 1, a.status);
          if (!ok) break;
          tc_fence_after();
          // S of this item follows the last P.V of the one before in the pipe;
          // its first P.V waits for P, and so for the epilogue that reads O
          if (nb0 > 0) issue_s(0, g & 1);
          if (nb1 > 0) issue_s(1, g & 1);
          mma_commit(bar(L::kKEmpty + (g & 1)));
          if (nb == 1) mma_commit(bar(L::kQEmpty));
          for (int j = 0; j < nb && ok; ++j, ++g) {
            const int st = g & 1, s1 = st ^ 1, j1 = j + 1;
            // a barrier's answer takes ~170 cycles even when its phase is complete:
            // ask for the three at once (16384 tokens: 1.68 -> 1.65 ms)
            const bool v_rdy = mbar_try(bar(L::kVFull + st), (g >> 1) & 1);
            const bool pa_rdy = j < nb0 && mbar_try(bar(L::kPFull + 0), np0 & 1);
            const bool k_rdy = j1 < nb && mbar_try(bar(L::kKFull + s1), ((g + 1) >> 1) & 1);
            ok = v_rdy || mbar_wait(bar(L::kVFull + st), (g >> 1) & 1, a.status);
            if (ok && v_tail && j1 == nb) {
              ok = mbar_wait(bar(L::kVTail + st), (tails >> st) & 1, a.status);
              tails ^= 1u << st;
            }
            if (!ok) break;
            if (j < nb0) issue_pv(0, st, np0, j == 0, j1 == nb0, pa_rdy);
            if (ok && j1 < nb) {
              ok = k_rdy || mbar_wait(bar(L::kKFull + s1), ((g + 1) >> 1) & 1, a.status);
              if (ok) tc_fence_after();
            }
            if (ok && j1 < nb0) issue_s(0, s1);
            if (j < nb1) issue_pv(1, st, np1, j == 0, j1 == nb1, false);
            if (!ok) break;
            if (j1 < nb1) issue_s(1, s1);
            mma_commit(bar(L::kVEmpty + st));
            if (j1 < nb) mma_commit(bar(L::kKEmpty + s1));
            if (j1 == nb - 1) mma_commit(bar(L::kQEmpty));
          }
        }
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegsR));
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int gs = __ffs(G) - 1; // G is a power of two
    int ns = 0, no = 0;        // S blocks and O tiles of this q tile so far
    float run_lse = -INFINITY; // of the splits folded so far
    while (const ItemR *xp = next()) {
      const int nb = xp->n_blocks[t];
      // the row's visible keys, counted from the split's first
      const int32_t t_row = (xp->tile + t) * T + (row >> gs);
      const int32_t kv_len = xp->kv_len;
      const int32_t n_seen =
          (a.causal ? min(kv_len - xp->q_len + t_row + 1, kv_len) : kv_len) - xp->key_begin;
      float m = -INFINITY, l = 0.f; // running max (log2 units) and sum
      bool failed = false;
      for (int j = 0; j < nb; ++j, ++ns) {
        const int32_t n_vis = n_seen - j * kKvBlock; // visible columns
        failed = __any_sync(0xffffffffu, !mbar_wait(bar(L::kSFull + t), ns & 1, a.status));
        if (failed) break;
        tc_fence_after();
        // blocks every row of the warp sees in full skip the per-column test
        const bool full = __all_sync(0xffffffffu, n_vis >= kKvBlock);
        const uint32_t srow = tS(t) + lane_base;
        // the row's 128 scores, in registers from here on
        uint32_t v[4][32];
        float bm;
        if (full) { // the loads give the maximum of their 32 columns
          float b4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_max(srow + c * 32, v[c], b4[c]);
          tmem_wait_ld();
          bm = fmax3(fmaxf(b4[0], b4[1]), b4[2], b4[3]);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(srow + c * 32, v[c]);
          tmem_wait_ld();
          bm = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (c * 32 + i >= n_vis) v[c][i] = 0xff800000u; // -inf: a weight of zero
              bm = fmaxf(bm, __uint_as_float(v[c][i]));
            }
        }
        bm = bm == -INFINITY ? -INFINITY : bm * a.scale_log2;
        float m_use = m, alpha = 1.f;
        if (bm > m + kRescaleR || (m == -INFINITY && bm != -INFINITY)) {
          m_use = bm;
          alpha = ex2(m - bm); // 0 when m == -inf
        }
        const float m_sub = m_use == -INFINITY ? 0.f : m_use;
        // P = 2^(s * scale - m) as bf16 pairs over the row's first 64 columns
        const uint64_t scale2 = f32x2(a.scale_log2, a.scale_log2);
        const uint64_t neg2 = f32x2(-m_sub, -m_sub);
        uint64_t psum2 = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float x0, x1;
            f32x2_split(ffma2r(f32x2(__uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1])), scale2,
                               neg2),
                        x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            psum2 = fadd2(psum2, f32x2(p0, p1));
            pk[i / 2] = pack_bf16(p0, p1);
          }
          tmem_st16(srow + c * 16, pk);
        }
        float ps0, ps1;
        f32x2_split(psum2, ps0, ps1);
        const float psum = ps0 + ps1;
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
      // epilogue: o_s = O / l; bf16 when the tile has one split or this is the
      // last of the folded ones, else the fp32 state.  A thread stores its own
      // row: a store instruction costs the SM an L1 cycle per row, so 32 bytes
      // of it each (6 prompts of 100 to 2048 tokens: 70 us with 16-byte stores
      // through shared memory, 68)
      const ItemR &x = *xp;
      int ln = lane; // opaque: what follows from it is not kept over the blocks
      asm volatile("" : "+r"(ln));
      const int n_splits = x.n_splits[t];
      if (n_splits > 0) {
        // warp-uniform (tcgen05.ld is warp-collective): a warp with a failed
        // wait writes zeros
        const bool have_o = __all_sync(
            0xffffffffu, !failed && nb > 0 && mbar_wait(bar(L::kODone + t), no & 1, a.status));
        no += nb > 0;
        tc_fence_after();
        const bool some = have_o && !(l == 0.f); // NaN sums stay NaN
        const float inv_l = some ? __frcp_rn(l) : 0.f; // o_s = O * (1/l)
        float lse = some ? __fmul_rn(__fadd_rn(m, lg2(l)), kLn2) : -INFINITY;
        const bool folds = x.rowbase < 0 && n_splits > 1; // uniform over the tile, as the next two
        const bool add = folds && x.split > 0;
        const bool last = folds ? x.split == n_splits - 1 : n_splits == 1;
        float wa = 1.f, wb = 0.f;
        int how = kFoldTake;
        if (add) {
          how = fold_weights(run_lse, lse, wa, wb);
          lse = run_lse;
        } else {
          run_lse = lse;
        }
        const int Dr = a.D; // head_dim 96 runs on the 128-wide layout, zero-padded
        // rows of out, or of the states for the merge: token, split, head
        const int64_t row_base =
            (last ? static_cast<int64_t>(x.q_start) : x.rowbase + x.split) * a.Hq + x.kvh * G;
        const int64_t row_step = last ? a.Hq : static_cast<int64_t>(x.nsp) * a.Hq;
        const int tok0 = (x.tile + t) * T, q_len = x.q_len;
        const int64_t dst = (row_base + (tok0 + (row >> gs)) * row_step + (row & (G - 1))) * Dr;
        const bool store = tok0 + (row >> gs) < q_len;
        // the running state, this CTA's own: float4 column x tile row
        float4 *run = reinterpret_cast<float4 *>(a.part_o) +
                      static_cast<int64_t>(blockIdx.x) * (2 * kTileRows * D / 4) +
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
          float4 prev[8];
          if (add) {
#pragma unroll
            for (int q = 0; q < 8; ++q) // all eight in flight (the compiler takes them one by one)
              asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(prev[q].x), "=f"(prev[q].y), "=f"(prev[q].z), "=f"(prev[q].w)
                           : "l"(run + (c * 8 + q) * kTileRows)
                           : "memory");
          }
          if (add) {
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
              store_row(a.out + dst + c * 32, w);
            }
          } else if (folds) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              run[(c * 8 + q) * kTileRows] =
                  make_float4(__uint_as_float(v[q * 4]), __uint_as_float(v[q * 4 + 1]),
                              __uint_as_float(v[q * 4 + 2]), __uint_as_float(v[q * 4 + 3]));
          } else if (store && c * 32 < Dr) {
            store_row(a.part_o + dst + c * 32, v);
          }
        }
        if (t_row < q_len && (last || !folds)) {
          const int64_t lse_row = row_base + t_row * row_step + (((warp & 3) * 32 + ln) & (G - 1));
          if (!last) a.part_lse[lse_row] = lse;
          else if (a.lse) a.lse[lse_row] = lse;
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
  if (warp == kMmaWarpR) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch_ragged_d(const RaggedArgs &a, cudaStream_t s) {
  using L = SmemR<D>;
  static std::atomic<uint64_t> ready{0};
  int sms = 0;
  const cudaError_t e = prepare_launch(reinterpret_cast<const void *>(prefill_ragged_kernel<D>),
                                       L::kAlloc, ready, &sms);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min({static_cast<int64_t>(sms), kFoldCtas, a.n_units * a.Hkv})));
  cfg.blockDim = dim3(kThreadsR);
  cfg.dynamicSmemBytes = L::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {chained_launch_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_ragged_kernel<D>, a);
}

} // namespace

cudaError_t ragged_plans_itself(int head_dim, int batch, int64_t items, int64_t part_rows,
                                bool *itself) {
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  *itself = head_dim != 256 && batch <= 32 && part_rows == 0 &&
            items <= std::min<int64_t>(sms, kFoldCtas);
  return e;
}

cudaError_t launch_prefill_ragged(const AttnArgs &a, const int32_t *kv_indptr, cudaStream_t s) {
  if (a.n_units == 0) return cudaSuccess;
  RaggedArgs r{};
  r.Hq = a.Hq;
  r.Hkv = a.Hkv;
  r.D = a.D;
  r.G = a.G;
  r.causal = a.causal;
  r.split = a.split;
  r.tile_tokens = a.tile_tokens;
  r.batch = a.batch;
  r.kv_rows = a.kv_rows;
  r.scale_log2 = a.scale_log2;
  r.n_units = a.n_units;
  r.reqs = a.reqs;
  r.units = a.units;
  r.qo_indptr = a.qo_indptr;
  r.kv_indptr = kv_indptr;
  r.total_q = a.total_rows;
  r.part_o = a.part_o;
  r.part_lse = a.part_lse;
  r.out = a.out;
  r.lse = a.lse;
  r.status = a.status;
  r.tm_q = a.tm_q;
  r.tm_k = a.tm_k;
  r.tm_v = a.tm_v;
  // head_dim 96 runs on the 128-wide layout: the tensor maps read columns
  // 96..127 as zeros
  return r.D > 64 ? launch_ragged_d<128>(r, s) : launch_ragged_d<64>(r, s);
}

} // namespace bia
