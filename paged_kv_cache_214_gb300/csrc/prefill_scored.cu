// prefill_scored.cu — paged (chunked) prefill attention whose scores are capped
// or biased by distance and whose rows see an interval of keys
// (pkv_score_options: a window, documents, a two-way prefix), on the sm_103a
// tensor cores (tcgen05, tensor memory, TMA).
//
// Mathematics.  Row r of a chunk lies at position i = Lk - Lq + r and sees the
// keys [lo, hi]; s = scale <q, K_j>, capped to c tanh(s / c), less slope |i - j|.
// One pass over the key tiles with a running maximum and sum in log2 units:
// O = sum 2^(s - m) V_j, l = sum 2^(s - m), out = O / l, lse = m + log2 l.
//
// Work item: 128 rows of one sequence and query head, and the 128-key tiles from
// the lowest lo to the highest hi of those rows, so that a window or a document
// costs its own tiles.  The grid has a block for every item; a block that is done
// with its own takes over blocks that have not started (cluster launch control),
// so that barriers and tensor memory are set up once per SM and uneven items even
// out (two sequences of five documents, 4000 rows, 32 heads: 99 us with a fixed
// walk over the items, 83 us so, 78 now).  16 warps:
//   warp 12 (TMA)  finds the next item, publishes it to the other warps through
//                  a ring of descriptors, loads its K tiles (3 stages) and Q (2).
//   warp 13 (TMA)  V tiles (2 stages).
//   warp 14 (MMA)  S_t = Q K_t^T into one of three S buffers in tensor memory.
//   warp 15 (MMA)  O += P_t V_t, A = P_t from tensor memory, B = V_t MN-major.
//   warps 0-11     softmax, in three groups of four: group t % 3 takes tile t of
//                  the block's running count, thread t of a group row t of the
//                  tile (32 consecutive TMEM lanes a warp).
// The softmax of a tile is a long chain (load S, maximum, 2^x, store P), some 8
// to 14 instructions a pair of scores, and with every warp on every tile the
// chain's latency is the time of a tile: two warps a scheduler on half a row
// each ran at 45% of the issue rate (b16 below: 249 us), four on a quarter at
// 50% (268 us).  Three tiles in flight overlap the chains.  What the groups hand
// on from tile t to t + 1, row by row through shared memory: the running maximum
// m(t), as soon as the tile's maximum is known and before its 2^x, and the
// running sum l(t), after them.  m moves only when a tile exceeds it by 2^60, so
// that O is hardly ever rescaled; scores capped by at most 52 need no m at all
// (kFixed), and one pass over S instead of two.  The group of an item's last tile
// writes its output, while the others work on the next item's first tiles; that
// item's first PV waits until O has been read.
// Measured (b16: 16 sequences, 32 / 8 heads, 512 new rows behind 1024, 172 GFLOP;
// the kernel, warm L2): capped by 50 150 us (1.15 PFLOP/s, 60% of the measured bf16
// rate), by 200 165, no options 140, biased 177; 8192 rows in a window of 1024 66 us.
// With inputs that are not in L2 capped by 50 takes 160 us (56%), the window 68.
// Bound by the chains of the softmax warps: the tensor pipe is 54% busy, issue 51%.
// What the last steps gave: maxima reduced by the TMEM load itself 162 -> 160 (by
// 200: 184 -> 172), the output written by the group that has just finished the item
// and not by the one that starts the next 160 -> 152.  Caps past 1000 keep an error
// relative to the score (cap_relative) and take 312.  Without gain: P handed over in
// halves so that PV starts earlier, O read out whole (64 packed registers) before it
// is written, the first pass in loads of 64 columns.
// TMEM (512 columns): S_0 | S_1 | S_2 | O; P overlays the first 64 columns of its
// S, in 32-key chunks behind the chunk being read.
// Rounding: P goes to the second product as bf16, as both operands of a tcgen05
// product have one type and V is bf16.  That is at most 2^-8 of each weight, of
// either sign: the whole output is 0.0022 off against 64 bits, of which 0.0017 is its
// own rounding to bf16; a second product with the weights' remainders would cost as
// much tensor time again.  Scores, maxima, sums and O are fp32.
// Every wait is bounded: a wait that runs out records an error, the block drains
// what it started, frees its tensor memory and exits.

#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "pipeline.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

// A bounded wait with every lane of the warp; the result is the same for all
// lanes.  What follows a first unsuccessful try is out of line: the instruction
// fetch is a limit of the softmax loops, and with every wait's loop inline around
// them they ran 1 to 5% slower.
__device__ __noinline__ bool slow_wait(uint32_t bar, uint32_t parity) {
  return mbar_wait(bar, parity);
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
  bool ok = mbar_try_wait(bar, parity);
  if (!ok) ok = slow_wait(bar, parity);
  return __all_sync(kFull, ok);
}

constexpr int kM = 128;   // query rows per tile
constexpr int kN = 128;   // keys per tile
constexpr int kGroups = 3;                 // softmax groups of four warps
constexpr int kSoftmaxWarps = 4 * kGroups;
constexpr int kQKWarp = kSoftmaxWarps;
constexpr int kVWarp = kQKWarp + 1;
constexpr int kSWarp = kQKWarp + 2;
constexpr int kThreads = (kSoftmaxWarps + 4) * 32;
constexpr int kHalf = 128 * 128;           // 128 rows x 64 bf16 (one 128-byte swizzled box)
constexpr int kTile = 2 * kHalf;           // 128 rows x 128 bf16
constexpr int kQStages = 2;
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kSBufs = 3;
static_assert(kGroups == kSBufs, "a group has an S buffer of its own");
constexpr int kRing = 4;                   // item descriptors
constexpr int kOffQ = 0;                              // kQStages buffers
constexpr int kOffK = kOffQ + kQStages * kTile;       // kKStages stages
constexpr int kOffV = kOffK + kKStages * kTile;       // kVStages stages
constexpr int kOffM = kOffV + kVStages * kTile;       // m(t): [t & 1][row] fp32
constexpr int kOffL = kOffM + 2 * kM * 4;             // l(t): [t & 1][row] fp32
constexpr int kOffItems = kOffL + 2 * kM * 4;         // kRing descriptors
constexpr int kItemBytes = 48;
constexpr int kOffAnswer = kOffItems + kRing * kItemBytes;
constexpr int kOffBars = kOffAnswer + 16;
static_assert(kOffAnswer % 16 == 0, "answer alignment");
// barriers
constexpr int kBarQFull = 0;                       // [Q buffer]
constexpr int kBarQEmpty = kBarQFull + kQStages;
constexpr int kBarKFull = kBarQEmpty + kQStages;   // [K stage]
constexpr int kBarKEmpty = kBarKFull + kKStages;
constexpr int kBarVFull = kBarKEmpty + kKStages;   // [V stage]
constexpr int kBarVEmpty = kBarVFull + kVStages;
constexpr int kBarSFull = kBarVEmpty + kVStages;   // [S buffer]
constexpr int kBarPFull = kBarSFull + kSBufs;      // [S buffer], its group's warps
constexpr int kBarPVDone = kBarPFull + kSBufs;     // [S buffer]: the PV that read P has completed
constexpr int kBarOFree = kBarPVDone + kSBufs;     // O of an item has been read, a group's warps
constexpr int kBarDrainS = kBarOFree + 1;
constexpr int kBarDrainPV = kBarDrainS + 1;
constexpr int kBarItemFull = kBarDrainPV + 1;      // [descriptor]
constexpr int kBarItemEmpty = kBarItemFull + kRing;   // [descriptor], every other warp
constexpr int kBarM = kBarItemEmpty + kRing;       // m(t) is there: [t & 1][row / 32]
constexpr int kBarL = kBarM + 8;                   // l(t) is there: [t & 1][row / 32]
constexpr int kBarNext = kBarL + 8;                // the next item's answer is there
constexpr int kNumBars = kBarNext + 1;
constexpr int kOffTmem = kOffBars + kNumBars * 8;
constexpr int kOffFlags = kOffTmem + 8;
constexpr int kSmemBytes = kOffFlags + 16;
static_assert(kSmemBytes <= 227 * 1024, "one block per SM must fit in shared memory");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;      // + 128 * buffer
constexpr uint32_t kColO = 384;
// The running maximum moves when a tile's exceeds it by 2^60: weights up to 2^60
// and their sums and products stay far inside fp32's range, at the same relative
// precision, and moving it means waiting for the previous tile's PV.
constexpr float kLazyRescale = 60.f;   // log2 units
constexpr float kLn2 = 0.69314718055994530942f;
// Caps up to this (log2 units; 52) need no maximum: with m = 0 every weight lies in
// 2^+-75, and sums of 2^20 weights times values up to 2^32 in fp32's range (the
// range that the call documents; a maximum for these rows too would cost 10%, the
// difference of caps 50 and 200 above).
constexpr float kFixedCap = 75.f;

struct Params {
  __nv_bfloat16* out;
  float* lse;
  const int32_t* block_tables;
  const int32_t* cu_q;
  const int32_t* cu_k;
  const float* slopes;         // per head, or null
  const int32_t* first_keys;   // per row, or null
  const int32_t* prefix_lens;  // per sequence, or null
  unsigned* err;
  int B, Hq, Hkv, maxblk, max_q, max_k, window;
  int n_qt;          // ceil(max_q / 128)
  int sweep;         // sequences of a sweep (get_item)
  int64_t num_blocks, total_q;
  bool out32;        // out is 32-byte aligned: rows are written a sector at a time
  float scale_log2;  // raw product -> log2 units; capped, not kWide: -> 2 log2(e) s / c
  float cap_log2;    // the cap in log2 units
  float cap_x;       // raw product -> s / c, infinity where the near form is not sound
  float cap_inv;     // 1 / cap_log2 (kWide)
  float poly[4];     // c tanh(s / c) in log2 units = raw (poly[0] + poly[1] raw^2 + ...)
};

// One query tile and its keys.
struct Item {
  int n;          // key tiles (0: no more items)
  int kt0;        // first key tile
  int rows;       // valid query rows of the tile
  int diag;       // position of the tile's first row
  int kvh, h;     // kv head, query head
  int row0;       // row of q / out of the tile's first row
  int b;          // sequence
  int prefix;     // tokens that every row sees
  int vlo, vhi;   // keys outside [vlo, vhi] are hidden from every row and may hold
                  // anything (vlo > vhi: no row has a key)
};
static_assert(sizeof(Item) <= kItemBytes, "descriptor");

// Item idx, by a whole warp (the row bounds are reduced across it).
__device__ __forceinline__ Item get_item(const Params& p, int idx, int lane) {
  Item it = {};
  // a sweep of sequences after another; in a sweep, heavier (later) row tiles first
  const int per_sweep = p.sweep * p.n_qt * p.Hq;
  const int sweep = idx / per_sweep;
  int rem = idx - sweep * per_sweep;
  const int per_lvl = min(p.sweep, p.B - sweep * p.sweep) * p.Hq;
  const int lvl = rem / per_lvl;
  rem -= lvl * per_lvl;
  it.b = sweep * p.sweep + rem / p.Hq;
  it.h = rem % p.Hq;
  it.kvh = it.h / (p.Hq / p.Hkv);
  const int q_begin = p.cu_q[it.b];
  const int Lq = p.cu_q[it.b + 1] - q_begin;
  const int Lk = p.cu_k[it.b + 1] - p.cu_k[it.b];
  it.prefix = p.prefix_lens ? p.prefix_lens[it.b] : 0;
  if (q_begin < 0 || Lq < 0 || q_begin + static_cast<int64_t>(Lq) > p.total_q || Lk < Lq ||
      Lq > p.max_q || Lk > p.max_k ||
      static_cast<int64_t>(Lk) > static_cast<int64_t>(p.maxblk) * kBlockSize || it.prefix < 0 ||
      it.prefix > Lk) {
    if (lane == 0) record_error(p.err, kErrIndex);
    return it;
  }
  const int q0 = (p.n_qt - 1 - lvl) * kM;
  if (q0 >= Lq) return it;
  it.rows = min(kM, Lq - q0);
  it.row0 = q_begin + q0;
  it.diag = Lk - Lq + q0;
  int klo = p.window > 0 ? max(0, it.diag - p.window + 1) : 0;
  int khi = max(it.diag + it.rows - 1, it.prefix - 1);
  it.vlo = p.window > 0 ? max(0, Lk - Lq - p.window + 1) : 0;
  it.vhi = Lk - 1;
  if (p.first_keys) {
    klo = INT32_MAX;
    khi = -1;
    for (int r = lane; r < it.rows; r += 32) {
      const int i = it.diag + r;
      const int lo = max(p.window > 0 ? max(0, i - p.window + 1) : 0,
                         __ldg(p.first_keys + it.row0 + r));
      const int hi = max(i, it.prefix - 1);
      if (lo <= hi) {
        klo = min(klo, lo);
        khi = max(khi, hi);
      }
    }
    klo = __reduce_min_sync(kFull, klo);
    khi = __reduce_max_sync(kFull, khi);
    it.vlo = klo;
    it.vhi = khi;
    if (klo > khi) klo = khi = 0;   // no row has a key: one tile, all of it hidden
  }
  it.kt0 = klo / kN;
  it.n = khi / kN - it.kt0 + 1;
  return it;
}

// The grid has one block for each item, and as many run as there are SMs: a
// running block takes the place of one that has not started yet (a cluster launch
// control request, answered in 16 bytes of shared memory) until none is left.
__device__ __forceinline__ void request_block(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
      ::"r"(answer), "r"(bar) : "memory");
}
// Index of the block whose place the answer gives, -1 if none was left.
__device__ __forceinline__ int taken_block(uint32_t answer) {
  int idx;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t.reg .b32 x, y, z, w;\n\t"
      "ld.shared.b128 a, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "mov.b32 x, -1;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {x, y, z, w}, a;\n\t"
      "mov.b32 %0, x;\n\t}"
      : "=r"(idx)
      : "r"(answer)
      : "memory");
  return idx;
}

// kCap: capped scores; kBias: biased ones; kFixed: capped by at most kFixedCap and
// not biased, so that m = 0 throughout and one pass over a tile's scores is enough;
// kWide: a cap so wide that the form of its far scores is cap_relative (a branch on
// it at run time took capped and biased b16 from 231 to 266 us).
template <bool kCap, bool kBias, bool kFixed, bool kWide>
__global__ void __launch_bounds__(kThreads, 1)
scored_prefill_kernel(const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const Params p) {
  // (no room for a realignment: the tiles' 128-byte swizzle wants 1024 bytes)
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_addr(smem);
  if (sbase & 1023u) {
    if (threadIdx.x == 0) record_error(p.err, kErrTimeout);
    return;
  }
  const uint32_t bars = sbase + kOffBars;
  auto bar = [&](int i) { return bars + 8u * i; };
  volatile int* flags = reinterpret_cast<volatile int*>(smem + kOffFlags);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kOffTmem);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kNumBars; ++i) {
      uint32_t count = 1;
      if ((i >= kBarPFull && i < kBarPFull + kSBufs) || i == kBarOFree) count = 4;
      if (i >= kBarItemEmpty && i < kBarItemEmpty + kRing) count = kSoftmaxWarps + 3;
      mbar_init(bar(i), count);
    }
    flags[0] = 0;  // abort
    flags[1] = 0;  // K tiles issued
    flags[2] = 0;  // V tiles issued
    flags[3] = 0;  // Q tiles issued
    fence_barrier_init();
  }
  if (warp == kSWarp) {
    tmem_alloc(sbase + kOffTmem, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kQKWarp && lane == 0) {
    tma_prefetch_map(&qmap);
    tma_prefetch_map(&kmap);
  }
  if (warp == kVWarp && lane == 0) tma_prefetch_map(&vmap);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // The block's gi-th item, for every warp but the one that publishes them;
  // false: a wait ran out.
  auto take_item = [&](int gi, Item& it) -> bool {
    const int slot = gi % kRing;
    if (!wait(bar(kBarItemFull + slot), (gi / kRing) & 1)) return false;
    it = *reinterpret_cast<const Item*>(smem + kOffItems + slot * kItemBytes);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarItemEmpty + slot));
    return true;
  };

  if (warp >= kSoftmaxWarps) {
    bool ok = true, timeout = false;
    if (warp == kQKWarp) {
      // ---------------------------------------------------------- items, K and Q
      // An item's Q goes into its buffer right after its first K tile has been
      // issued, once the S MMAs of the item before the previous one are done.
      int gk = 0, idx = static_cast<int>(blockIdx.x);
      uint32_t next_ph = 0;
      bool asked = false;   // a request is on its way
      BlockIds ids;
      Ring<kKStages> rk;
      const int withhold = withheld_tile();   // test hook: K tiles from here on are never copied
      auto ask = [&]() {
        if (lane == 0) {
          // (the last answer has been read before it is written over)
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(bar(kBarNext), 16);
          request_block(sbase + kOffAnswer, bar(kBarNext));
        }
        __syncwarp();
        asked = true;
      };
      // The next item's index, -1 if there is none; false: the wait ran out.
      auto answer = [&](int& next) -> bool {
        asked = false;
        if (!wait(bar(kBarNext), next_ph)) return false;
        next_ph ^= 1u;
        next = taken_block(sbase + kOffAnswer);
        __syncwarp();
        return true;
      };
      ask();
      for (int gi = 0; ok; ++gi) {
        Item it = {};
        while (idx >= 0) {   // items without rows are passed over
          it = get_item(p, idx, lane);
          if (it.n) break;
          if (!answer(idx)) {
            ok = false;
            timeout = true;
            break;
          }
          if (idx >= 0) ask();
        }
        if (!ok) break;
        const int slot = gi % kRing;
        if (gi >= kRing && !wait(bar(kBarItemEmpty + slot), (gi / kRing - 1) & 1)) {
          ok = false;
          timeout = true;
          break;
        }
        if (lane == 0) {
          *reinterpret_cast<Item*>(smem + kOffItems + slot * kItemBytes) = it;
          mbar_arrive(bar(kBarItemFull + slot));
        }
        __syncwarp();
        if (it.n == 0) break;
        const int32_t* table = p.block_tables + static_cast<int64_t>(it.b) * p.maxblk;
        ids.chunk = -1;
        bool stopped = false;
        for (int kt = 0; kt < it.n; ++kt, ++gk, rk.next()) {
          if (__any_sync(kFull, flags[0] != 0)) { ok = false; break; }
          if (gk >= withhold) { stopped = true; break; }
          const int gkt = it.kt0 + kt;
          // (an item without keys reads no table entry)
          const int id = it.vlo > it.vhi
                             ? 0 : ids.get(table, p.maxblk, gkt >> 1, lane, p.num_blocks, p.err);
          const int at = id * kBlockSize + (gkt & 1) * kN;
          if (gk >= kKStages && !wait(bar(kBarKEmpty + rk.idx), rk.ph ^ 1u)) {
            ok = false;
            timeout = true;
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(kBarKFull + rk.idx), kTile);
            flags[1] = gk + 1;
          }
          __syncwarp();
          // lanes 2s, 2s+1 load stage s: a lane's next copy never queues behind
          // its previous one
          if ((lane >> 1) == rk.idx)
            tma_load_3d(sbase + kOffK + rk.idx * kTile + (lane & 1) * kHalf, &kmap,
                        bar(kBarKFull + rk.idx), (lane & 1) * 64, it.kvh, at);
          __syncwarp();
          if (kt == 0) {
            const int qb = gi % kQStages;
            if (gi >= kQStages && !wait(bar(kBarQEmpty + qb), (gi / kQStages - 1) & 1)) {
              ok = false;
              timeout = true;
              break;
            }
            if (lane == 0) {
              // rows past the sequence are its neighbour's, or zeros past total_q
              mbar_arrive_expect_tx(bar(kBarQFull + qb), kTile);
              flags[3] = gi + 1;
            }
            __syncwarp();
            if (lane >= 2 * kKStages && lane < 2 * kKStages + 2)   // lanes of their own
              tma_load_3d(sbase + kOffQ + qb * kTile + (lane & 1) * kHalf, &qmap,
                          bar(kBarQFull + qb), (lane & 1) * 64, it.h, it.row0);
            __syncwarp();
          }
        }
        if (stopped || !ok) break;
        if (!answer(idx)) {
          ok = false;
          timeout = true;
        } else if (idx >= 0) {
          ask();
        }
      }
      // no answer may be on its way when the block ends
      if (asked) (void)wait(bar(kBarNext), next_ph);
    } else if (warp == kVWarp) {
      // ---------------------------------------------------------- V
      int gk = 0;
      BlockIds ids;
      Ring<kVStages> rv;
      for (int gi = 0; ok; ++gi) {
        Item it;
        if (!take_item(gi, it)) { ok = false; timeout = true; break; }
        if (it.n == 0) break;
        const int32_t* table = p.block_tables + static_cast<int64_t>(it.b) * p.maxblk;
        ids.chunk = -1;
        for (int kt = 0; kt < it.n; ++kt, ++gk, rv.next()) {
          if (__any_sync(kFull, flags[0] != 0)) { ok = false; break; }
          const int gkt = it.kt0 + kt;
          const int id = it.vlo > it.vhi
                             ? 0 : ids.get(table, p.maxblk, gkt >> 1, lane, p.num_blocks, p.err);
          const int at = id * kBlockSize + (gkt & 1) * kN;
          if (gk >= kVStages && !wait(bar(kBarVEmpty + rv.idx), rv.ph ^ 1u)) {
            ok = false;
            timeout = true;
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(kBarVFull + rv.idx), kTile);
            flags[2] = gk + 1;
          }
          __syncwarp();
          if ((lane >> 1) == rv.idx)
            tma_load_3d(sbase + kOffV + rv.idx * kTile + (lane & 1) * kHalf, &vmap,
                        bar(kBarVFull + rv.idx), (lane & 1) * 64, it.kvh, at);
          __syncwarp();
        }
      }
    } else if (warp == kSWarp) {
      // ---------------------------------------------------------- MMA: S = Q K^T
      // (the whole warp runs the loop and waits; an elected lane issues)
      constexpr uint32_t idesc_s = idesc_bf16_f32(kM, kN, 0);   // B = K, K-major
      int gk = 0;
      Ring<kSBufs> sb;
      Ring<kKStages> rk;
      for (int gi = 0; ok; ++gi) {
        Item it;
        if (!take_item(gi, it)) { ok = false; timeout = true; break; }
        if (it.n == 0) break;
        const int qb = gi % kQStages;
        if (!wait(bar(kBarQFull + qb), (gi / kQStages) & 1)) { ok = false; timeout = true; break; }
        const uint32_t q_s = sbase + kOffQ + qb * kTile;
        for (int kt = 0; kt < it.n; ++kt, ++gk, sb.next(), rk.next()) {
          if (__any_sync(kFull, flags[0] != 0)) { ok = false; break; }
          // K here, and the S buffer free: the PV that read P from it (three
          // tiles back) is done
          if (!wait(bar(kBarKFull + rk.idx), rk.ph) ||
              (gk >= kSBufs && !wait(bar(kBarPVDone + sb.idx), sb.ph ^ 1u))) {
            ok = false;
            timeout = true;
            break;
          }
          tc_fence_after();
          const uint32_t k_s = sbase + kOffK + rk.idx * kTile;
          const uint32_t d_s = tmem + kColS + sb.idx * kN;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint32_t off = (ks >> 2) * kHalf + (ks & 3) * 32;
            umma_bf16_warp(d_s, smem_desc_sw128(q_s + off, 16, 1024),
                           smem_desc_sw128(k_s + off, 16, 1024), idesc_s, ks > 0);
          }
          umma_commit_warp(bar(kBarSFull + sb.idx));
          umma_commit_warp(bar(kBarKEmpty + rk.idx));
        }
        if (!ok) break;
        umma_commit_warp(bar(kBarQEmpty + qb));
      }
      // every MMA this warp issued has completed once this arrives
      umma_commit_warp(bar(kBarDrainS));
      (void)wait(bar(kBarDrainS), 0);
    } else {
      // ---------------------------------------------------------- MMA: O += P V
      constexpr uint32_t idesc_o = idesc_bf16_f32(kM, kHeadDim, 1);  // B = V, MN-major
      Ring<kSBufs> sb;
      Ring<kVStages> rv;
      const uint32_t d_o = tmem + kColO;
      for (int gi = 0; ok; ++gi) {
        Item it;
        if (!take_item(gi, it)) { ok = false; timeout = true; break; }
        if (it.n == 0) break;
        for (int kt = 0; kt < it.n; ++kt, sb.next(), rv.next()) {
          if (__any_sync(kFull, flags[0] != 0)) { ok = false; break; }
          if (!wait(bar(kBarVFull + rv.idx), rv.ph) ||
              !wait(bar(kBarPFull + sb.idx), sb.ph) ||
              (kt == 0 && gi > 0 && !wait(bar(kBarOFree), (gi - 1) & 1))) {
            ok = false;
            timeout = true;
            break;
          }
          tc_fence_after();
          const uint32_t v_s = sbase + kOffV + rv.idx * kTile;
          const uint32_t p_t = tmem + kColS + sb.idx * kN;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            // A = P: 16 keys = 8 packed columns per step.  B = V: 64-dim boxes
            // kHalf apart (LBO), 8-key swizzle atoms 1024 bytes apart (SBO).
            umma_bf16_tmem_a_warp(d_o, p_t + ks * 8, smem_desc_sw128(v_s + ks * 2048, kHalf, 1024),
                                  idesc_o, (kt > 0 || ks > 0) ? 1u : 0u);
          }
          umma_commit_warp(bar(kBarVEmpty + rv.idx));
          umma_commit_warp(bar(kBarPVDone + sb.idx));
        }
      }
      umma_commit_warp(bar(kBarDrainPV));
      (void)wait(bar(kBarDrainPV), 0);
    }
    if (timeout && lane == 0) record_error(p.err, kErrTimeout);
    if (!ok && lane == 0) flags[0] = 1;
  } else {
    // ------------------------------------------------------------ softmax
    const int group = warp >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;   // this thread's row of every tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_col = lane_base + kColS + group * kN;
    const uint32_t o_col = lane_base + kColO;
    float* const m_slot = reinterpret_cast<float*>(smem + kOffM) + row;
    float* const l_slot = reinterpret_cast<float*>(smem + kOffL) + row;
    bool ok = true, timeout = false;
    const f32x2 sc2 = pack2(p.scale_log2, p.scale_log2);

    // m(t) and l(t) pass through two slots each: the writer of t + 2 has read the
    // value of t + 1, whose writer had read that of t.
    auto hand_on = [&](int first_bar, float* slot, int t, float v) {
      slot[(t & 1) * kM] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(first_bar + (t & 1) * 4 + quarter));
    };
    auto receive = [&](int first_bar, const float* slot, int t, float& v) -> bool {
      if (!wait(bar(first_bar + (t & 1) * 4 + quarter), (t >> 1) & 1)) return false;
      v = *const_cast<const volatile float*>(slot + (t & 1) * kM);
      return true;
    };
    // Output of an item (its m and l) by the group of its last tile, whose PV is the
    // S buffer's phase ph: O / l, row by row.  O is then free for the
    // next item's PV.  A row that sees one key divides by that key's weight as P holds
    // it, so that its output is the key's value, bit for bit.
    auto epilogue = [&](const Item& e, uint32_t ph, float m, float l, bool one_key) -> bool {
      if (!wait(bar(kBarPVDone + group), ph)) return false;
      tc_fence_after();
      const float held = one_key ? __bfloat162float(__float2bfloat16_rn(l)) : l;
      const float inv = l > 0.f ? 1.f / held : 0.f;   // a row without keys: 0 and -inf
      const bool valid = row < e.rows;
      const int64_t at = static_cast<int64_t>(e.row0 + row) * p.Hq + e.h;
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * kHeadDim);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tmem_ld32x32_x32(o_col + 32 * c, o);
        tmem_wait_ld(o);
        if (valid) {
          auto two = [&](int k) {
            return pack_bf16x2(__uint_as_float(o[k]) * inv, __uint_as_float(o[k + 1]) * inv);
          };
#pragma unroll
          for (int k = 0; k < 32; k += 16) {   // 16 dims: one 32-byte sector
            uint32_t* to = dst + 16 * c + k / 2;
            if (p.out32) {
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to),
                           "r"(two(k)), "r"(two(k + 2)), "r"(two(k + 4)), "r"(two(k + 6)),
                           "r"(two(k + 8)), "r"(two(k + 10)), "r"(two(k + 12)), "r"(two(k + 14))
                           : "memory");
            } else {
              reinterpret_cast<uint4*>(to)[0] =
                  make_uint4(two(k), two(k + 2), two(k + 4), two(k + 6));
              reinterpret_cast<uint4*>(to)[1] =
                  make_uint4(two(k + 8), two(k + 10), two(k + 12), two(k + 14));
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarOFree));
      if (p.lse && valid) p.lse[at] = l > 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;
      return true;
    };

    uint32_t ph = 0;          // phase of the group's S buffer
    int gi = 0, t_item = 0;   // items, and the running count of the item's first tile
    for (; ok; ++gi) {
      Item it;
      if (!take_item(gi, it)) { ok = false; timeout = true; break; }
      if (it.n == 0) break;
      // position of the row, the keys [lo, hi] it sees, the head's slope in log2 units
      const int pos = it.diag + row;
      int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
      if (p.first_keys && row < it.rows) lo = max(lo, __ldg(p.first_keys + it.row0 + row));
      const int hi = max(pos, it.prefix - 1);
      float slope = 0.f;
      if constexpr (kBias) slope = __ldg(p.slopes + it.h) * 1.4426950408889634f;
      const f32x2 slope2 = pack2(slope, slope);

      int kt = group - t_item % kGroups;
      if (kt < 0) kt += kGroups;
      const unsigned span = lo > hi ? 0u : static_cast<unsigned>(hi - lo);
      for (; kt < it.n; kt += kGroups, ph ^= 1u) {
        const int t = t_item + kt;
        if (!(ok = wait(bar(kBarSFull + group), ph))) { timeout = true; break; }
        tc_fence_after();
        const int tile = (it.kt0 + kt) * kN;
        // the row's keys within the tile: c with c - c_lo <= span, unsigned
        const int c_lo = lo > hi ? 1 << 30 : lo - tile;
        const bool edge = __any_sync(kFull, c_lo > 0 || hi - tile < kN - 1);
        auto hidden = [&](int c) { return static_cast<unsigned>(c - c_lo) > span; };
        // How the warp's rows see 32 keys from c0 on: -1 not at all, 0 wholly, 1 in
        // part.  (Of a tile on the diagonal or at a window's end a warp sees about
        // one chunk in part, and need not look at those it does not see.)
        const int c_hi = lo > hi ? -1 : min(hi - tile, kN);
        auto view = [&](auto is_edge, int c0) -> int {
          if constexpr (is_edge) {
            if (!__any_sync(kFull, c_lo < c0 + 32 && c_hi >= c0)) return -1;
            return __any_sync(kFull, c_lo > c0 || c_hi < c0 + 31) ? 1 : 0;
          }
          return 0;
        };
        auto by_edge = [&](auto body) {
          if (edge)
            body(std::true_type{});
          else
            body(std::false_type{});
        };
        // Biased: -slope |pos - j| = slope c + slope (tile - pos) for key j = tile + c
        // up to the row's own position; the second part is a constant of row and
        // tile, off.  Past that position (a two-way prefix) it is 2 slope (c - past)
        // less, past = pos - tile.
        const float past = static_cast<float>(pos - tile);
        const float off = kBias ? -slope * past : 0.f;
        const bool two_way =
            kBias && it.prefix > 0 && __any_sync(kFull, hi > pos && tile + kN - 1 > pos);
        auto bias = [&](auto both, f32x2 c, f32x2 add) {
          f32x2 b = fma2(c, slope2, add);
          if constexpr (both)
            b = fma2(pack2(fmaxf(lo2(c) - past, 0.f), fmaxf(hi2(c) - past, 0.f)),
                     pack2(-2.f * slope, -2.f * slope), b);
          return b;
        };
        // Capped: c tanh(s / c), s / c = x.  While |x| <= 0.45 for all products at hand
        // of the warp: tanh_ratio on the FMA pipe, x's factor in the coefficients (five
        // terms up to 0.6 took 171 us instead of 163).  Else c - 2c / (1 + e^2x), with
        // two special-function operations, which are scarcer.
        auto near_cap = [&](f32x2 v, f32x2 add) {
          const f32x2 u = mul2(v, v);
          f32x2 y = fma2(pack2(p.poly[3], p.poly[3]), u, pack2(p.poly[2], p.poly[2]));
          y = fma2(y, u, pack2(p.poly[1], p.poly[1]));
          y = fma2(y, u, pack2(p.poly[0], p.poly[0]));
          return kFixed ? mul2(v, y) : fma2(v, y, add);
        };
        // Under a wide cap that form's error, a few 2^-24 of the cap, would be large
        // next to small scores: those take cap_relative.
        auto far_cap = [&](f32x2 raw, f32x2 add) {
          f32x2 v = mul2(raw, sc2);
          if constexpr (kWide) {
            v = pack2(cap_relative(lo2(v), p.cap_log2, p.cap_inv),
                      cap_relative(hi2(v), p.cap_log2, p.cap_inv));
            return add2(v, add);
          }
          v = add2(pack2(ex2(lo2(v)), ex2(hi2(v))), pack2(1.f, 1.f));
          v = fma2(pack2(rcp_approx(lo2(v)), rcp_approx(hi2(v))),
                   pack2(-2.f * p.cap_log2, -2.f * p.cap_log2), pack2(p.cap_log2, p.cap_log2));
          return kFixed ? v : add2(v, add);
        };
        auto plain = [&](f32x2 v, f32x2 add) { return fma2(v, sc2, add); };

        uint32_t r0[32];
        float m = 0.f, alpha = 1.f, m_before = 0.f;
        bool far = false;
        if constexpr (!kFixed) {
        // First pass: the row's maximum.  Unbiased: of the products, as the cap is
        // increasing.  Biased: per 32 keys that of the products, modified as the
        // key of the greatest bias would be.  That is at most 31 slopes too high,
        // which the sums bear as they do a late maximum; steeper slopes take the
        // maximum of the scores themselves (b16 with slopes up to 0.1: 177 us, with
        // the scores' own maximum 198).
        float mx = -INFINITY;
        auto chunk_max = [&](float& mx, const uint32_t (&r)[32], int c0, int seen) {
          if (seen == 1) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!hidden(c0 + c)) mx = fmaxf(mx, __uint_as_float(r[c]));
          } else {
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              mx = max3(mx, __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
          }
        };
        auto capped_max = [&](float v) {
          if constexpr (kWide)   // (the other form may be off by more than the sums bear)
            return v == -INFINITY ? v : cap_relative(v * p.scale_log2, p.cap_log2, p.cap_inv);
          else if constexpr (kCap)
            return v == -INFINITY ? v
                                  : fmaf(-2.f * p.cap_log2,
                                         rcp_approx(1.f + ex2(v * p.scale_log2)), p.cap_log2);
          else
            return v * p.scale_log2;
        };
        const bool loose = kBias && 31.f * fabsf(slope) <= kLazyRescale;
        if (kCap || !kBias || loose) {
          float big = 0.f, red;
          by_edge([&](auto is_edge) {
#pragma unroll 1
            for (int c0 = 0; c0 < kN; c0 += 32) {
              const int seen = view(is_edge, c0);
              if (seen < 0) continue;
              if constexpr (kCap) {
                tmem_ld32x32_x32_absmax(s_col + c0, r0, red);
                tmem_wait_ld(r0, red);
                big = fmaxf(big, red);
              }
              if (!kBias || loose) {
                tmem_ld32x32_x32_max(s_col + c0, r0, red);
                tmem_wait_ld(r0, red);
                if (is_edge && seen) {
                  red = -INFINITY;
                  chunk_max(red, r0, c0, seen);
                }
                if constexpr (kBias) {
                  const float c_first = static_cast<float>(c0), c_last = c_first + 31.f;
                  auto biased = [&](float c) {   // (as the second pass does: the same `off`)
                    return fmaf(-2.f * slope, fmaxf(c - past, 0.f), fmaf(slope, c, off));
                  };
                  red = capped_max(red) +
                        (slope >= 0.f ? biased(fminf(fmaxf(past, c_first), c_last))
                                      : fmaxf(biased(c_first), biased(c_last)));
                }
                mx = fmaxf(mx, red);
              }
            }
          });
          if constexpr (kCap) far = __any_sync(kFull, !(big * p.cap_x <= kTanhPoly));
        }
        if constexpr (!kBias) {
          mx = capped_max(mx);
        } else if (__builtin_expect(!loose, 0)) {
          auto scan = [&](auto both, auto score) {
#pragma unroll 1
            for (int c0 = 0; c0 < kN; c0 += 32) {
              const int seen = edge ? view(std::true_type{}, c0) : 0;
              if (seen < 0) continue;
              f32x2 c2 = pack2(static_cast<float>(c0), static_cast<float>(c0 + 1));
              tmem_ld32x32_x32(s_col + c0, r0);
              tmem_wait_ld(r0);
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const f32x2 v = score(pack2(__uint_as_float(r0[c]), __uint_as_float(r0[c + 1])),
                                      bias(both, c2, pack2(0.f, 0.f)));
                c2 = add2(c2, pack2(2.f, 2.f));
                r0[c] = __float_as_uint(lo2(v));
                r0[c + 1] = __float_as_uint(hi2(v));
              }
              chunk_max(mx, r0, c0, seen);
            }
          };
          auto scan_with = [&](auto both) {
            if (!kCap)
              scan(both, plain);
            else if (__builtin_expect(far, 0))
              scan(both, far_cap);
            else
              scan(both, near_cap);
          };
          if (two_way)
            scan_with(std::true_type{});
          else
            scan_with(std::false_type{});
          mx += off;
        }

        // The running maximum.  (Received for an item's first tile as well, like the
        // sum: whoever writes t + 1 may then take the slot of t - 1.)
        if (t > 0 && !(ok = receive(kBarM, m_slot, t - 1, m_before))) { timeout = true; break; }
        const bool need = kt > 0 && mx > m_before + kLazyRescale;
        m = kt > 0 && !need ? m_before : mx;
        hand_on(kBarM, m_slot, t, m);   // before the rescaling, which waits
        if (need) alpha = ex2(m_before - mx);
        if (kt > 0) {
          // (a row without keys so far has O = 0 at any m)
          if (__any_sync(kFull, need && m_before > -INFINITY)) {
            // the previous tile's PV must have finished accumulating into O
            if (!(ok = wait(bar(kBarPVDone + (t - 1) % kSBufs), ((t - 1) / kSBufs) & 1))) {
              timeout = true;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              tmem_ld32x32_x32(o_col + 32 * c, r0);
              tmem_wait_ld(r0);
#pragma unroll
              for (int k = 0; k < 32; ++k) r0[k] = __float_as_uint(__uint_as_float(r0[k]) * alpha);
              tmem_st32x32_x32(o_col + 32 * c, r0);
            }
          }
        }
        }   // !kFixed

        // Second pass: P = 2^(s - m) as bf16 pairs, column c / 2 for keys c, c + 1.  A
        // hidden key gets weight 0; a row that has seen no key yet has m = -inf and
        // hidden keys only.
        const float base = m == -INFINITY ? 0.f : off - m;
        const f32x2 base2 = pack2(base, base);
        f32x2 sum2 = pack2(0.f, 0.f);
        auto chunk = [&](auto is_edge, auto both, auto score, int c0) {
          uint32_t pk[16];
          // (biased) the pair's keys within the tile
          f32x2 c2 = pack2(static_cast<float>(c0), static_cast<float>(c0 + 1));
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            f32x2 add = base2;
            if constexpr (kBias) {
              add = bias(both, c2, base2);
              c2 = add2(c2, pack2(2.f, 2.f));
            }
            const f32x2 x = score(pack2(__uint_as_float(r0[c]), __uint_as_float(r0[c + 1])), add);
            float w0 = ex2(lo2(x)), w1 = ex2(hi2(x));
            if constexpr (is_edge) {
              if (hidden(c0 + c)) w0 = 0.f;
              if (hidden(c0 + c + 1)) w1 = 0.f;
            }
            pk[c / 2] = pack_bf16x2(w0, w1);
            sum2 = add2(sum2, pack2(w0, w1));
          }
          tmem_st32x32_x16(s_col + c0 / 2, pk);
        };
        auto chunk_as = [&](auto is_edge, int seen, auto both, auto score, int c0) {
          if (is_edge && seen)
            chunk(std::true_type{}, both, score, c0);
          else
            chunk(std::false_type{}, both, score, c0);
        };
        by_edge([&](auto is_edge) {
#pragma unroll 1
          for (int c0 = 0; c0 < kN; c0 += 32) {
            const int seen = view(is_edge, c0);
            if (seen < 0) {
              uint32_t none[16] = {};
              tmem_st32x32_x16(s_col + c0 / 2, none);
              continue;
            }
            constexpr std::false_type one_way{};
            if constexpr (kFixed) {
              float big;
              tmem_ld32x32_x32_absmax(s_col + c0, r0, big);
              tmem_wait_ld(r0, big);
              far = __any_sync(kFull, !(big * p.cap_x <= kTanhPoly));
            } else {
              tmem_ld32x32_x32(s_col + c0, r0);
              tmem_wait_ld(r0);
            }
            if (two_way) {
              constexpr std::integral_constant<bool, kBias> both{};
              if (!kCap)
                chunk(std::true_type{}, both, plain, c0);
              else if (__builtin_expect(far, 0))
                chunk(std::true_type{}, both, far_cap, c0);
              else
                chunk(std::true_type{}, both, near_cap, c0);
            } else if (!kCap) {
              chunk_as(is_edge, seen, one_way, plain, c0);
            } else if (__builtin_expect(far, 0)) {
              chunk_as(is_edge, seen, one_way, far_cap, c0);
            } else {
              chunk_as(is_edge, seen, one_way, near_cap, c0);
            }
          }
        });

        // keys outside [vlo, vhi]: zero their V rows so that 0 * (stale data)
        // cannot put a NaN into O (the group's thread s clears row s)
        if ((kt == 0 && tile < it.vlo) || (kt == it.n - 1 && tile + kN - 1 > it.vhi)) {
          const int vs = t % kVStages;
          if (!(ok = wait(bar(kBarVFull + vs), (t / kVStages) & 1))) { timeout = true; break; }
          if (tile + row < it.vlo || tile + row > it.vhi) {
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const uint32_t vrow = sbase + kOffV + vs * kTile + row * 128;
#pragma unroll
            for (int cc = 0; cc < 8; ++cc) {
              sts128(vrow + cc * 16, zero);
              sts128(vrow + kHalf + cc * 16, zero);
            }
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        float l = lo2(sum2) + hi2(sum2), l_before = 0.f;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPFull + group));
        if (t > 0 && !(ok = receive(kBarL, l_slot, t - 1, l_before))) { timeout = true; break; }
        if (kt > 0) l = fmaf(l_before, alpha, l);
        hand_on(kBarL, l_slot, t, l);
        if (kt == it.n - 1 && !(ok = epilogue(it, ph, m, l, lo == hi))) { timeout = true; break; }
      }
      if (!ok) break;
      t_item += it.n;
    }
    if (timeout && lane == 0) record_error(p.err, kErrTimeout);
    if (!ok && lane == 0) flags[0] = 1;
  }

  tc_fence_before();
  __syncthreads();
  // After an abort, wait (bounded) for TMA copies that may still be landing:
  // the last issued tiles of each ring.
  if (flags[0] && tid == kQKWarp * 32) {
    const int kin = flags[1], qin = flags[3];
    for (int x = max(0, kin - kKStages); x < kin; ++x)
      (void)slow_wait(bar(kBarKFull + x % kKStages), (x / kKStages) & 1);
    for (int x = max(0, qin - kQStages); x < qin; ++x)
      (void)slow_wait(bar(kBarQFull + x % kQStages), (x / kQStages) & 1);
  }
  if (flags[0] && tid == kVWarp * 32) {
    const int vin = flags[2];
    for (int x = max(0, vin - kVStages); x < vin; ++x)
      (void)slow_wait(bar(kBarVFull + x % kVStages), (x / kVStages) & 1);
  }
  __syncthreads();
  if (warp == kSWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool kCap, bool kBias, bool kFixed = false, bool kWide = false>
int launch_form(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
                const Params& prm, unsigned blocks, cudaStream_t stream) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !attr_set[dev]) {
    if (cudaFuncSetAttribute(scored_prefill_kernel<kCap, kBias, kFixed, kWide>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemBytes) != cudaSuccess)
      return PKV_ERR_LAUNCH;
    attr_set[dev] = true;
  }
  scored_prefill_kernel<kCap, kBias, kFixed, kWide>
      <<<blocks, kThreads, kSmemBytes, stream>>>(qm, km, vm, prm);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

}  // namespace

int set_wait_hook_prefill_scored(unsigned long long limit_ns, int withhold_plus1) {
  const WaitHook h{limit_ns, withhold_plus1, 0};
  return cudaMemcpyToSymbol(g_wait_hook, &h, sizeof h) == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

int launch_prefill_scored(const PrefillArgs& a, int64_t total_q, const pkv_score_options& opt,
                          unsigned* err, cudaStream_t stream) {
  if (a.B == 0 || a.max_seqlen_q == 0 || total_q == 0) return PKV_OK;
  CUtensorMap qm, km, vm;
  const int64_t slots = a.num_blocks * kBlockSize;
  if (!encode_pool_map(&qm, a.q, total_q, a.Hq, kM) ||
      !encode_pool_map(&km, a.k_cache, slots, a.Hkv, kN) ||
      !encode_pool_map(&vm, a.v_cache, slots, a.Hkv, kN))
    return PKV_ERR_ARG;
  Params prm = {};
  prm.out = static_cast<__nv_bfloat16*>(a.out);
  prm.lse = a.lse;
  prm.block_tables = a.block_tables;
  prm.cu_q = a.cu_seqlens_q;
  prm.cu_k = a.cu_seqlens_k;
  prm.slopes = opt.alibi_slopes;
  prm.first_keys = opt.first_keys;
  prm.prefix_lens = opt.prefix_lens;
  prm.err = err;
  prm.B = a.B;
  prm.Hq = a.Hq;
  prm.Hkv = a.Hkv;
  prm.maxblk = a.max_blocks_per_seq;
  prm.max_q = a.max_seqlen_q;
  prm.max_k = a.max_seqlen_k;
  prm.window = opt.window;
  if (!prefill_items_fit(a.max_seqlen_q, a.B, a.Hq)) return PKV_ERR_SHAPE;
  prm.n_qt = prefill_row_tiles(a.max_seqlen_q);
  const unsigned blocks = static_cast<unsigned>(prm.n_qt) * a.B * a.Hq;
  // Every row tile of a sequence reads its keys again.  A sweep is as many sequences
  // as have their K and V in a quarter of L2 (32 MB), at least one: with all 16 of
  // b16 in one (100 MB) 177 us instead of 170 with a cold L2, 412 MB read from HBM.
  // One sequence a sweep is as fast there, but two small ones that could mix their
  // tiles take 78.5 us instead of 77.6.
  const int64_t seq_bytes =
      std::max<int64_t>(1, static_cast<int64_t>(a.max_seqlen_k) * a.Hkv * 2 * kHeadDim * 2);
  prm.sweep = static_cast<int>(std::clamp<int64_t>((int64_t(32) << 20) / seq_bytes, 1, a.B));
  prm.num_blocks = a.num_blocks;
  prm.total_q = total_q;
  prm.out32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
  const bool cap = opt.softcap > 0.f, bias = opt.alibi_slopes != nullptr;
  if (!cap) {
    prm.scale_log2 = a.scale * 1.4426950408889634f;
    return bias ? launch_form<false, true>(qm, km, vm, prm, blocks, stream)
                : launch_form<false, false>(qm, km, vm, prm, blocks, stream);
  }
  prm.scale_log2 = a.scale * 2.8853900817779268f / opt.softcap;
  prm.cap_log2 = opt.softcap * 1.4426950408889634f;
  prm.cap_x = a.scale / opt.softcap;
  // tanh(x) / x of x = raw * cap_x: the powers of cap_x are folded into the
  // coefficients, unless they would leave fp32's range
  const double t[4] = {kTanhT0, kTanhT1, kTanhT2, kTanhT3};
  double f = static_cast<double>(prm.cap_log2) * prm.cap_x;
  for (int k = 0; k < 4; ++k, f *= static_cast<double>(prm.cap_x) * prm.cap_x)
    prm.poly[k] = static_cast<float>(t[k] * f);
  // (above 1000 the far form's error, a few 2^-24 of the cap, would reach 1e-4 of a
  // score's unit, for rows that share a warp with scores past 0.45 of the cap)
  bool wide = opt.softcap > 1000.f;
  if (!(prm.cap_x > 1e-4f && prm.cap_x < 1e3f && f > 1e-36 && f < 1e36)) {
    prm.cap_x = INFINITY;
    wide = true;
  }
  if (!bias && prm.cap_log2 <= kFixedCap)   // (an error of 2^-24 of such a cap is no matter)
    return launch_form<true, false, true>(qm, km, vm, prm, blocks, stream);
  if (!wide)
    return bias ? launch_form<true, true>(qm, km, vm, prm, blocks, stream)
                : launch_form<true, false>(qm, km, vm, prm, blocks, stream);
  prm.scale_log2 = a.scale * 1.4426950408889634f;
  prm.cap_inv = 1.f / prm.cap_log2;
  return bias ? launch_form<true, true, false, true>(qm, km, vm, prm, blocks, stream)
              : launch_form<true, false, false, true>(qm, km, vm, prm, blocks, stream);
}

}  // namespace pkv
