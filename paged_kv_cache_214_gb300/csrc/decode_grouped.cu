// decode_grouped.cu — paged decode attention for requests with several sequences each
// (beams, samples of one prompt) whose block tables share blocks
// (paged_decode_attention_grouped).
//
// The operation is the decode's (decode_kernel.cuh): for every sequence and query head
// softmax(scale q K^T) V over the sequence's own table.  A block that several sequences of
// a request hold is read once for all of them, so the bytes are those of the request's
// distinct blocks.
//
// Two kernels.  The plan (a thread block for every group of sequences) finds a request's
// distinct blocks: a column of the tables whose entries are all the same is one block for
// everybody (a thread a column); in any other column a warp compares the entries
// (match.any) and each distinct id becomes a block with the set of sequences that hold
// it.  It lists them as tiles of 64 tokens.
//
// Work decomposition of the attention
//   grid (as many thread blocks as the GPU holds at a time, kv heads x head groups).  A
//   thread block serves all sequences of a request (up to 64 query rows: sequences x heads
//   of one kv head; larger requests are cut into groups of sequences) over a range of
//   their tiles, and goes on with the next request's where its share of all tiles reaches
//   that far: shares are equal, whatever the lengths (16 requests of 512 to 4700 tokens
//   51 us; with ranges that end with their request 55).  Every thread block works out its
//   share for itself from the lists' lengths.
//   A producer warp copies the tiles (TMA, 64 tokens of K and V, 128-byte swizzle) into a
//   ring; four consumer warps share a tile as MT groups of 16 rows by 4 / MT shares of its
//   tokens (MT = 1, 2, 4 for up to 16, 32, 64 rows), so that a warp always holds the
//   output and the queries of 16 rows in registers and K and V leave shared memory MT
//   times.  Both products run on the warp-level MMA (m16n8k16, fp32 accumulation),
//   operands by ldmatrix; E4M3 codes are converted to f16, exactly.  With at most 64 rows
//   a byte of bf16 K carries at most 64 operations and one of V 128 (weights in two parts), a
//   sixth of the warp-level MMA's rate at the copy bandwidth.  Up to 32 bf16 rows HBM is the
//   bound while tiles stream, beyond, and over E4M3 codes, the products, the softmax and the
//   conversions between them are, as below.
//   Rows that do not hold a tile, and positions behind a row's length, score -inf.
//   The shares are merged through shared memory, the ranges through the workspace by the
//   last block to arrive, as in the decode, many of them in two steps.
//
// Measured (one call of a graph of many, inputs in memory; floor: the distinct blocks' bytes
// at the copy bandwidth).  4 x 8 sequences of 16k to 40k tokens, 32 / 8 heads, 415 MB: 84
// us (floor 62), 4.9 TB/s; 16 x 4 of 512 to 4700, 238 MB: 52 us (36), 7.7 TB/s inside the
// loop over tiles, with 20 us around it: the plan (5), lengths and the first copy (5), both
// merges (8).  4 x 12 of 8k to 20k, 48 rows in a tile of 64: 104 us (47), 1 x 16 of 30000, 64 / 8
// heads, 128 rows: 102 (22).  24 x 5 E4M3, 35 rows a kv head, 78 MB: 58 us (12): 2.0 us a tile
// of 64 tokens that all rows see and 1.5 us one of a single sequence, of code conversion,
// products and softmax in a chain of dependent instructions (issue 28%, tensor pipe 24%), three
// warps of four with rows.  One sequence after the other (paged_decode_attention) the same calls
// take 276, 85, 254, 213 and 243 us.

#include <cmath>

#include "decode_kernel.cuh"

namespace pkv {

int set_wait_hook_decode_grouped(unsigned long long limit_ns, int withhold_plus1) {
  const WaitHook h{limit_ns, withhold_plus1, 0};
  return cudaMemcpyToSymbol(g_wait_hook, &h, sizeof h) == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

namespace {

constexpr int kMaxRanges = 1024;     // of a sequence group
// What starting on a group costs (its queries, an empty ring, its merge), in tiles, and the
// least that a thread block is given where there are few tiles (it costs more than a few
// itself).  Measured with 1 / 3 / 5 / 8 for the first: 16 x 4 sequences 53.6, 50.7, 50.7, 50.7
// us, 8 x 4 of 3000 tokens (E4M3) 22.4, 21.4, 21.3, 23.2.  With 1 / 4 / 6 / 8 / 11 for the
// second: 4 x 8 of 700 tokens 34, 29, 27, 28, 33; one of 4000 tokens 22.8, 20.4, 21.2, 22.5,
// 23.5; a single sequence of 1000 tokens 11.3, 12.5, 13.0, 14.6, 16.5.
constexpr int kSegment = 3;
constexpr int kMinShare = 6;
// Ranges that are merged at a time where there are more than twice as many: one block would
// read all of a long request's partial results (1 x 8 sequences of 40000 tokens, 5 / 1 heads:
// 72 us; eight at a time 34, 32 at a time 41.  Up to 16 ranges one step is as good).
constexpr int kMergeGroup = 8;
constexpr int kMaxColumns = 16384;   // of a block table
constexpr int kTilesPerBlock = kBlockSize / kTile;

// What the plan leaves in the workspace.
struct PlanArrays {
  int* tiles;        // [units]: of a group of sequences
  uint32_t* word;    // [units, most]: block id << 9 | tile of the block << 7 | tokens
  uint32_t* mask;    // [units, most]: sequences that hold it
  uint16_t* column;  // [units, most]
  int64_t most;      // tiles of a group at most
};

// Sequences that one thread block serves: `seqs` consecutive ones of a request.
struct Units {
  int count, width, seqs, groups;   // groups of a request
  __device__ __forceinline__ void get(int unit, int& first_row, int& n) const {
    const int seq0 = unit % groups * seqs;
    n = min(seqs, width - seq0);
    first_row = unit / groups * width + seq0;
  }
};

struct GroupedParams {
  __nv_bfloat16* out;
  float* lse;
  const __nv_bfloat16* q;
  const void* k_cache;
  const void* v_cache;
  uint32_t num_blocks;
  const int32_t* context_lens;
  float* ws_o;         // [2 x thread blocks, rows, 128] normalised partial outputs
  float* ws_lse;       // [2 x thread blocks, rows] log2-sum-exps
  unsigned* ws_count;  // [units, kv heads x head groups] arrival counters
  unsigned* group_count;   // [partial results] of kMergeGroup ranges, or null: no room
  unsigned* err;
  PlanArrays plan;
  Units units;
  int Hq, Hkv, max_len;
  int split;               // ranges of every group, or 0: by their tiles
  int heads, head_groups;  // query heads of a kv head that a thread block serves, groups
  float scale_log2, k_scale, v_scale;
};

// ---------------------------------------------------------------- the plan

struct PlanParams {
  const int32_t* block_tables;
  const int32_t* context_lens;
  PlanArrays out;
  Units units;
  int maxblk, num_blocks;
  unsigned* err;
};

// Inclusive sum over the lanes.
__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

constexpr int kPlanThreads = 256;
constexpr int kPlanWarps = kPlanThreads / 32;

__global__ void __launch_bounds__(kPlanThreads) grouped_plan_kernel(const PlanParams p) {
  __shared__ int staged[kMaxWidth * kPlanThreads];   // entries of a chunk of columns
  __shared__ int lens[kMaxWidth], buf[kPlanWarps], n_divided;
  __shared__ uint16_t tiles_in[kPlanThreads], divided_columns[kPlanThreads];
  __shared__ int first_in[kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // May start while the kernel in front of it ends, and lets the attention start (which
  // waits for it); see decode_kernel.cuh.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int unit = blockIdx.x;
  int first_row, n_seqs;
  p.units.get(unit, first_row, n_seqs);
  const int32_t* tables = p.block_tables + static_cast<int64_t>(first_row) * p.maxblk;
  // entries behind a row's length hold anything and are not looked at
  auto stage = [&](int c) {
#pragma unroll 8
    for (int w = 0; w < n_seqs; ++w)
      if (c < p.maxblk)
        staged[w * kPlanThreads + tid] = tables[static_cast<int64_t>(w) * p.maxblk + c];
  };
  stage(tid);   // with the lengths
  if (tid < kMaxWidth) {
    int n = 0;
    if (tid < n_seqs) {
      n = p.context_lens[first_row + tid];
      if (n < 0 || n > p.maxblk * kBlockSize) {
        record_error(p.err, kErrIndex);
        n = n < 0 ? 0 : p.maxblk * kBlockSize;
      }
    }
    lens[tid] = n;
  }
  if (tid == 0) n_divided = 0;
  __syncthreads();
  int most = 0;
  for (int w = 0; w < n_seqs; ++w) most = max(most, lens[w]);
  const int columns = (most + kBlockSize - 1) / kBlockSize;
  const int64_t list = static_cast<int64_t>(unit) * p.out.most;
  // 64-token tiles of a block in column c for a sequence of n tokens
  auto tiles_of = [](int n, int c) {
    return min(kTilesPerBlock, (n - c * kBlockSize + kTile - 1) / kTile);
  };
  auto put = [&](int at, int col, unsigned who, int id, int longest) {
    if (id < 0 || id >= p.num_blocks) {
      record_error(p.err, kErrIndex);
      id = 0;
    }
    const int tiles = tiles_of(longest, col);
    for (int k = 0; k < tiles; ++k) {
      const int tokens = min(kTile, longest - col * kBlockSize - k * kTile);
      p.out.word[list + at + k] = static_cast<uint32_t>(id) << 9 | k << 7 | tokens;
      p.out.mask[list + at + k] = who;
      p.out.column[list + at + k] = static_cast<uint16_t>(col);
    }
  };

  int total = 0;   // tiles of the columns before c0
  for (int c0 = 0; c0 < columns; c0 += kPlanThreads) {
    if (c0 > 0) {
      stage(c0 + tid);
      __syncthreads();
    }
    // Column c as one block, if its sequences agree: who holds it, its id, the longest.
    const int c = c0 + tid;
    bool same = true;
    unsigned who = 0;
    int id = -1, longest = 0, n = 0;
    if (c < columns) {
      for (int w0 = 0; w0 < n_seqs; w0 += 8) {
        int x[8], len[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {   // (eight rows in flight)
          const int w = min(w0 + k, n_seqs - 1);
          x[k] = staged[w * kPlanThreads + tid];
          len[k] = lens[w];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (w0 + k >= n_seqs || c * kBlockSize >= len[k]) continue;
          if (!who) id = x[k];
          same = same && x[k] == id;
          who |= 1u << (w0 + k);
          longest = max(longest, len[k]);
        }
      }
      if (same) n = tiles_of(longest, c);
      else divided_columns[atomicAdd(&n_divided, 1)] = static_cast<uint16_t>(tid);
      tiles_in[tid] = static_cast<uint16_t>(n);
    }
    __syncthreads();
    // The others by a whole warp each, lane w looking at sequence w: the first of the
    // sequences that share a block leads them.  Once for their tiles, once for the list.
    auto divided = [&](int at, unsigned& set, int& block, int& len) {
      const int mine = lane < n_seqs ? lens[lane] : 0;
      const bool in = (c0 + at) * kBlockSize < mine;
      block = in ? staged[lane * kPlanThreads + at] : 0;
      set = __match_any_sync(0xffffffffu,
                             in ? static_cast<long long>(static_cast<uint32_t>(block)) : -1ll - lane);
      len = 0;
      for (unsigned left = set; in && left; left &= left - 1)
        len = max(len, lens[__ffs(left) - 1]);
      return in && lane == __ffs(set) - 1;
    };
    for (int k = warp; k < n_divided; k += kPlanWarps) {
      unsigned set;
      int block, len;
      const int at = divided_columns[k];
      const bool leads = divided(at, set, block, len);
      const int all = __reduce_add_sync(0xffffffffu, leads ? tiles_of(len, c0 + at) : 0);
      if (lane == 0) tiles_in[at] = static_cast<uint16_t>(all);
    }
    __syncthreads();
    const int mine = c < columns ? tiles_in[tid] : 0;
    const int upto = warp_scan(mine, lane);
    if (lane == 31) buf[warp] = upto;
    __syncthreads();
    int at = total + upto - mine;
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
      if (w < warp) at += buf[w];
      total += buf[w];
    }
    first_in[tid] = at;
    if (c < columns && same) put(at, c, who, id, longest);
    __syncthreads();
    for (int k = warp; k < n_divided; k += kPlanWarps) {
      unsigned set;
      int block, len;
      const int col = divided_columns[k];
      const bool leads = divided(col, set, block, len);
      const int own = leads ? tiles_of(len, c0 + col) : 0;
      const int ends = warp_scan(own, lane);
      if (leads) put(first_in[col] + ends - own, c0 + col, set, block, len);
    }
    __syncthreads();
    if (tid == 0) n_divided = 0;
  }

  if (tid == 0) p.out.tiles[unit] = total;
}

// How the tiles are dealt out.  A group of T tiles is a stretch of kSegment + T on a line
// of all groups, and thread block b takes what lies in [b share, (b + 1) share): the first
// kSegment places of a group stand for what starting on a group costs beside its tiles.
struct Stretch {
  int unit;          // sequence group of the first place, -1: nothing is left for this block
  int tiles;         // of that group
  int start;         // where the group begins on the line
  int from, to;      // the block's places
  int share;
};
__device__ __forceinline__ int tiles_of(const PlanArrays& plan, int unit) {
  // (a workspace that holds no plan of these sizes leads to wrong results, not out of the list)
  return static_cast<int>(min(static_cast<int64_t>(max(__ldcg(plan.tiles + unit), 0)), plan.most));
}
__device__ __forceinline__ Stretch find_stretch(const PlanArrays& plan, int units, int blocks,
                                                int which, int lane) {
  constexpr int kHeld = 4;   // groups whose tiles a lane keeps
  int held[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    held[k] = lane + 32 * k < units ? tiles_of(plan, lane + 32 * k) : 0;
  int all = 0;   // (the host has checked that places fit 31 bits)
#pragma unroll
  for (int k = 0; k < kHeld; ++k) all += held[k];
#pragma unroll 4
  for (int z = lane + 32 * kHeld; z < units; z += 32) all += tiles_of(plan, z);
  all = __reduce_add_sync(0xffffffffu, all) + units * kSegment;
  Stretch r;
  r.unit = -1;
  r.share = max((all + blocks - 1) / blocks, kMinShare);
  r.from = which * r.share;
  r.to = min(all, r.from + r.share);
  int before = 0;
  auto look = [&](int z, int T) {   // 32 groups, the lane's z
    const int upto = before + warp_scan(z < units ? T + kSegment : 0, lane);
    const unsigned past = __ballot_sync(0xffffffffu, r.from < upto);
    before = __shfl_sync(0xffffffffu, upto, 31);
    if (!past) return false;
    const int at = __ffs(past) - 1;
    r.unit = __shfl_sync(0xffffffffu, z, at);
    r.tiles = __shfl_sync(0xffffffffu, T, at);
    r.start = __shfl_sync(0xffffffffu, upto, at) - r.tiles - kSegment;
    return true;
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (32 * k < units && look(lane + 32 * k, held[k])) return r;
  for (int z0 = 32 * kHeld; z0 < units; z0 += 32 * kHeld) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      held[k] = z0 + 32 * k + lane < units ? tiles_of(plan, z0 + 32 * k + lane) : 0;
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (z0 + 32 * k < units && look(z0 + 32 * k + lane, held[k])) return r;
  }
  return r;
}

template <bool kFp8>
struct GroupedLayout {
  static constexpr int kConsumers = 4;
  static constexpr int kThreads = (kConsumers + 1) * 32;
  static constexpr int kOpBytes = kTile * (kFp8 ? 128 : 256);
  static constexpr int kStageBytes = 2 * kOpBytes;
  static constexpr int kStages = 96 * 1024 / kStageBytes;
  static constexpr int kRing = kStages * kStageBytes;
  // over the ring after the last copy: the warps' outputs, [4][16] rows of 128 f32
  static_assert(64 * kHeadDim * 4 <= kRing, "over the ring");
  static constexpr int kTiles = kRing;                 // uint4 a stage: word, mask, column
  static constexpr int kMergeM = kTiles + kStages * 16;   // [4][16]
  static constexpr int kMergeL = kMergeM + 64 * 4;
  static constexpr int kBars = kMergeL + 64 * 4;
  static constexpr int kFlags = kBars + 2 * kStages * 8;   // abort, last, issued, again; partly [4]
  static constexpr int kBytes = kFlags + 32 + 1024;             // + alignment slack
  static_assert(kBytes <= 113 * 1024, "two blocks per SM");
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// The running softmax of one warp: 16 rows (this lane's are gq and gq + 8) over its
// share of the tiles.
struct Stream {
  float o[16][4];   // o[n][0..1] row gq, o[n][2..3] row gq + 8; columns: see out_dim
  float m[2], l[2];   // reference of the weights (near the maximum), sum
};

// Dim of output column 2c + e of n-tile n.  E4M3 codes come in pairs, so a pair of
// n-tiles holds the even and the odd dims of 16.
template <bool kFp8>
__device__ __forceinline__ int out_dim(int n, int c, int e) {
  return kFp8 ? 16 * (n >> 1) + 4 * c + 2 * e + (n & 1) : 8 * n + 2 * c + e;
}

// 16 J tokens of a tile from t0 on: kb, vb the tile's K and V.  lim: tokens of the tile
// that rows gq and gq + 8 see; valid: tokens that any row sees (those behind hold
// anything).  kAll: the rows see all of them.
//
// Weights for the second product.  bf16 pools: the value and its rounded remainder, 16
// significant bits, as the decode does, for any number of rows.  (The value alone, off by 2^-8 at
// most, would take 85 us in place of 84 for 4 x 8 of 16k to 40k tokens, 32 rows, but 81 in place
// of 101 for 4 x 12 of 8k to 20k, 48 rows, and for 1 x 16 of 30000, 128: the second set of
// products holds up the copies there.)  E4M3 pools: f16, rounded once, off by 2^-11 at most; the
// codes themselves are off by up to 2^-4 of what was stored, and the remainder (22 bits) would take
// 74 us in place of 58 for 24 x 5 and 120 in place of 91 for 4 x 12.  f16
// ends at 2^-25 (half its smallest step), so the largest weight is kept between 2^11 and 2^15:
// a weight below 2^-25 of it has fewer bits and one below 2^-36 is lost (all of them together
// 2^-14 of the sum in the longest table; with a largest weight of 1 four million keys of 2^-25.4
// lost 8% of it).
template <int J, bool kFp8, bool kAll>
__device__ __forceinline__ void consume_tokens(uint32_t kb, uint32_t vb, int t0, int lane,
                                               const uint32_t (&qa)[8][4], const float (&qmul)[2],
                                               const int (&lim)[2], int valid, Stream& st) {
  constexpr int NT = 2 * J;   // groups of 8 tokens
  // log2 of the weight that a new maximum gets, and of the largest
  constexpr float kTopWeight = kFp8 ? 11.f : 0.f, kMostWeight = kFp8 ? 15.f : 8.f;
  const int c = lane & 3;
  const int mi = lane >> 3, mr = lane & 7;   // ldmatrix: this lane gives row mr of matrix mi
  float sc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
  // an ldmatrix of 8 tokens gives the B operands of two k-steps (E4M3: of four)
  constexpr int kSteps = kFp8 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < 8 / kSteps; ++i) {
    uint32_t r[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint32_t row = kb + (t0 + 8 * n + mr) * 128;
      if constexpr (kFp8)
        ldmatrix4(row + (((4 * i + mi) ^ mr) << 4), r[n]);
      else
        ldmatrix4(row + (i >> 1) * kHalfBytes + (((4 * (i & 1) + mi) ^ mr) << 4), r[n]);
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const uint32_t (&a)[4] = qa[kSteps * i + k];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (kFp8)
          mma_16x8x16<true>(sc[n], a[0], a[1], a[2], a[3], e4m3x2_lo_to_f16x2(r[n][k]),
                            e4m3x2_hi_to_f16x2(r[n][k]));
        else
          mma_16x8x16<false>(sc[n], a[0], a[1], a[2], a[3], r[n][2 * k], r[n][2 * k + 1]);
      }
    }
  }
  // sc[n][2 r + e]: row r of the lane, token t0 + 8 n + 2 c + e; scores, then weights
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float top = -INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float& x = sc[n][2 * r + e];
        x = kAll || t0 + 8 * n + 2 * c + e < lim[r] ? x * qmul[r] : -INFINITY;
        top = fmaxf(top, x);
      }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // as in the decode, the reference moves only when the maximum rises far above it
    if (top > st.m[r] + kMostWeight) {
      const float m = top - kTopWeight, alpha = rescale(st.m[r], m);
      st.l[r] *= alpha;
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        st.o[n][2 * r] *= alpha;
        st.o[n][2 * r + 1] *= alpha;
      }
      st.m[r] = m;
    }
    const float ref = st.m[r] == -INFINITY ? 0.f : st.m[r];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float& x = sc[n][2 * r + e];
        x = ex2(x - ref);
        st.l[r] += x;
      }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {   // 16 tokens a time
    uint32_t ph[4], pl[4];
    const float (&x)[4] = sc[2 * j], (&y)[4] = sc[2 * j + 1];
    if constexpr (kFp8) {
      ph[0] = pack_f16x2(x[0], x[1]);
      ph[1] = pack_f16x2(x[2], x[3]);
      ph[2] = pack_f16x2(y[0], y[1]);
      ph[3] = pack_f16x2(y[2], y[3]);
    } else {
      split_pair<false>(x[0], x[1], ph[0], pl[0]);
      split_pair<false>(x[2], x[3], ph[1], pl[1]);
      split_pair<false>(y[0], y[1], ph[2], pl[2]);
      split_pair<false>(y[2], y[3], ph[3], pl[3]);
    }
    // tokens behind the last one that any row sees are zeroed: they may hold NaN patterns
    const int tj = t0 + 16 * j;
    const bool ragged = !kAll && valid < tj + 16;
    uint32_t keep[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = tj + 8 * h + 2 * c;
      keep[h] = (t < valid ? 0xffffu : 0u) | (t + 1 < valid ? 0xffff0000u : 0u);
    }
    const int vt = tj + 8 * (mi & 1) + mr;
#pragma unroll
    for (int i = 0; i < (kFp8 ? 4 : 8); ++i) {
      uint32_t r[4];   // tokens tj.. and tj + 8.. of 16-byte chunk 2i, then of chunk 2i + 1
      if constexpr (kFp8)
        ldmatrix4_trans(vb + vt * 128 + (((2 * i + (mi >> 1)) ^ mr) << 4), r);
      else
        ldmatrix4_trans(vb + (i >> 2) * kHalfBytes + vt * 128 +
                            (((2 * (i & 3) + (mi >> 1)) ^ mr) << 4), r);
      if (ragged) {
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] &= keep[k & 1];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (kFp8) {
          // bytes (token a: even dim, odd dim; token b: even, odd) to pairs of one dim
          const uint32_t w0 = __byte_perm(r[2 * h], 0u, 0x3120);
          const uint32_t w1 = __byte_perm(r[2 * h + 1], 0u, 0x3120);
          const int n = 2 * (2 * i + h);
          mma_16x8x16<true>(st.o[n], ph[0], ph[1], ph[2], ph[3], e4m3x2_lo_to_f16x2(w0),
                            e4m3x2_lo_to_f16x2(w1));
          mma_16x8x16<true>(st.o[n + 1], ph[0], ph[1], ph[2], ph[3], e4m3x2_hi_to_f16x2(w0),
                            e4m3x2_hi_to_f16x2(w1));
        } else {
          const int n = 2 * i + h;
          mma_16x8x16<false>(st.o[n], ph[0], ph[1], ph[2], ph[3], r[2 * h], r[2 * h + 1]);
          mma_16x8x16<false>(st.o[n], pl[0], pl[1], pl[2], pl[3], r[2 * h], r[2 * h + 1]);
        }
      }
    }
  }
}

// Row r of the lane (gq, gq + 8) as the A operand of the score product: qa[kk][r] and
// qa[kk][2 + r] are the two halves of k-step kk, two dims of q each (null: zeros).
template <bool kFp8>
__device__ __forceinline__ void load_q(const __nv_bfloat16* q, int c, int r, uint32_t (&qa)[8][4]) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d = 16 * kk + (kFp8 ? 4 * c + 2 * h : 8 * h + 2 * c);
      qa[kk][2 * h + r] = q ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
    }
}
// E4M3: to f16, scaled by the power of two that brings the row's maximum into [2^14, 2^15),
// as in the decode; returns what turns a product into a score in log2 units.
__device__ __forceinline__ float f16_q(uint32_t (&qa)[8][4], int r, float scale_log2, float k_scale) {
  float amax = 0.f;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      amax = fmaxf(amax, fmaxf(fabsf(bf16lo(qa[kk][2 * h + r])), fabsf(bf16hi(qa[kk][2 * h + r]))));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int e = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFFu) - 126;
  const int sh = min(15 - e, 100);
  const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t& x = qa[kk][2 * h + r];
      x = pack_f16x2(bf16lo(x) * up, bf16hi(x) * up);
    }
  return scale_log2 * k_scale * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
}

// By one warp: a row alone over the tiles of a segment's list, from global memory (see serve()).
// q: the row; w: its sequence in the group; len: its length; lane: dims 4 lane and on.  Leaves
// the output against the reference m and the sum l.
template <bool kFp8>
__device__ __forceinline__ void attend_alone(const GroupedParams& p, int64_t list, int count, int kvh,
                                             const __nv_bfloat16* q, int w, int len, float4& o,
                                             float& m, float& l) {
  const int lane = threadIdx.x & 31;
  auto four = [&](const void* pool, int64_t slot) {
    const int64_t at = (slot * p.Hkv + kvh) * kHeadDim + 4 * lane;
    if constexpr (kFp8) {
      const uint32_t x = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(pool) + at);
      float4 v;
      f16x2_unpack(e4m3x2_lo_to_f16x2(x), v.x, v.y);
      f16x2_unpack(e4m3x2_hi_to_f16x2(x), v.z, v.w);
      return v;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(pool) + at);
      return make_float4(bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y));
    }
  };
  const uint2 qw = *reinterpret_cast<const uint2*>(q + 4 * lane);
  const float mul = p.scale_log2 * (kFp8 ? p.k_scale : 1.f);
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  m = -INFINITY;
  l = 0.f;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const uint32_t word = p.plan.word[list + i];
    // (no block of this pool: not a plan of these arguments, see tiles_of())
    if (!(p.plan.mask[list + i] >> w & 1u) || word >> 9 >= p.num_blocks) continue;
    const int k = word >> 7 & 3;
    const int n = min(kTile, len - (p.plan.column[list + i] * kBlockSize + k * kTile));
    const int64_t slot = static_cast<int64_t>(word >> 9) * kBlockSize + k * kTile;
#pragma unroll 1
    for (int t0 = 0; t0 < n; t0 += 32) {
      float s = -INFINITY;   // of token t0 + lane
      const int tokens = min(32, n - t0);
      float4 x[8];   // (on their way at a time; those behind the last one are the last again)
      auto eight = [&](const void* pool, int t) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = four(pool, slot + t0 + min(t + j, tokens - 1));
      };
#pragma unroll 1
      for (int t = 0; t < tokens; t += 8) {
        eight(p.k_cache, t);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float d = bf16lo(qw.x) * x[j].x + bf16hi(qw.x) * x[j].y + bf16lo(qw.y) * x[j].z +
                    bf16hi(qw.y) * x[j].w;
#pragma unroll
          for (int sh = 16; sh; sh >>= 1) d += __shfl_xor_sync(0xffffffffu, d, sh);
          if (lane == t + j && lane < tokens) s = d * mul;
        }
      }
      float top = s;
#pragma unroll
      for (int sh = 16; sh; sh >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
      if (top > m) {
        const float alpha = rescale(m, top);
        l *= alpha;
        o.x *= alpha;
        o.y *= alpha;
        o.z *= alpha;
        o.w *= alpha;
        m = top;
      }
      const float e = lane < tokens ? ex2(s - (m == -INFINITY ? 0.f : m)) : 0.f;
      l += e;
#pragma unroll 1
      for (int t = 0; t < tokens; t += 8) {
        eight(p.v_cache, t);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float weight = __shfl_sync(0xffffffffu, e, (t + j) & 31);
          o.x = fmaf(weight, x[j].x, o.x);
          o.y = fmaf(weight, x[j].y, o.y);
          o.z = fmaf(weight, x[j].z, o.z);
          o.w = fmaf(weight, x[j].w, o.w);
        }
      }
    }
  }
#pragma unroll
  for (int sh = 16; sh; sh >>= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
}

// By one warp: the output of a row without keys.
__device__ __forceinline__ void write_empty(__nv_bfloat16* out, float* lse, int lane) {
  *reinterpret_cast<uint2*>(out + 4 * lane) = make_uint2(0u, 0u);
  if (lse && lane == 0) *lse = -INFINITY;
}

// Partial results, of `rows` rows each.  A thread block has two at most: that of a group that
// it goes on with (not the group's first range), and that of one whose first range ends it.
// In a group's first thread block the latter is the odd one; range s of the group is then
// the group's
__device__ __forceinline__ int64_t partial_of(int s) { return s == 0 ? 1 : 2 * s; }

// By the thread block: the log-sum-exp merge of rows' n partial results, `stride` rows each,
// in os ([.., 128]) and lses.  A chain of dependent loads for each row would take 2 us a
// row and warp (measured: 17 us for 32 rows), so all log-sum-exps are loaded at once, four
// threads a row turn them into weights in shared memory, and the outputs of two rows are
// on their way at a time.
constexpr int kMergeWeights = 16384;
template <class Row>
__device__ __forceinline__ void merge_ranges(float* lses, float* os, int from, int by, int n, int stride,
                                             bool final, int n_rows, const Row& row_of,
                                             __nv_bfloat16* out, float* lse, float* weights) {
  auto part = [&](int s) { return partial_of(from + by * s) * stride; };   // its first row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int warps = blockDim.x >> 5;
  const int group = min(n_rows, max(1, kMergeWeights / n));
  for (int g0 = 0; g0 < n_rows; g0 += group) {
    const int rows = min(group, n_rows - g0);
    for (int i = tid; i < rows * n; i += blockDim.x) {
      const int s = i / rows, r = i - s * rows;
      weights[r * n + s] = __ldcg(lses + part(s) + g0 + r);
    }
    __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += blockDim.x / 4) {
      const int r = r0 + tid / 4;
      float* w = weights + min(r, rows - 1) * n;
      float mx = -INFINITY, sum = 0.f;
      for (int s = tid % 4; s < n; s += 4) mx = fmaxf(mx, w[s]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // (no keys: -inf everywhere; a NaN in some partial stays one)
      const float ref = mx == -INFINITY ? 0.f : mx;
      for (int s = tid % 4; s < n; s += 4) sum += ex2(w[s] - ref);
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (r < rows) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        for (int s = tid % 4; s < n; s += 4) w[s] = ex2(w[s] - ref) * inv;
        if (tid % 4 == 0) {
          const float lse2 = mx + __log2f(sum);
          if (!final) __stcg(lses + part(0) + g0 + r, lse2);
          else if (lse) lse[row_of(g0 + r)] = lse2 * kLn2;
        }
      }
    }
    __syncthreads();
    for (int r = 2 * warp; r < rows; r += 2 * warps) {
      const int second = min(r + 1, rows - 1);
      float4 acc[2] = {};
      const int row[2] = {g0 + r, g0 + second};
      const float* w[2] = {weights + r * n, weights + second * n};
      for (int s0 = 0; s0 < n; s0 += 8) {
        float4 v[2][8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            v[j][k] = __ldcg(reinterpret_cast<const float4*>(
                                 os + (part(min(s0 + k, n - 1)) + row[j]) * kHeadDim) +
                             lane);
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float x = s0 + k < n ? w[j][s0 + k] : 0.f;
            acc[j].x = fmaf(x, v[j][k].x, acc[j].x);
            acc[j].y = fmaf(x, v[j][k].y, acc[j].y);
            acc[j].z = fmaf(x, v[j][k].z, acc[j].z);
            acc[j].w = fmaf(x, v[j][k].w, acc[j].w);
          }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (r + j >= rows) break;
        if (final) {
          uint2 packed;
          packed.x = pack_bf16x2(acc[j].x, acc[j].y);
          packed.y = pack_bf16x2(acc[j].z, acc[j].w);
          *reinterpret_cast<uint2*>(out + row_of(row[j]) * kHeadDim + 4 * lane) = packed;
        } else {
          __stcg(reinterpret_cast<float4*>(os + (part(0) + row[j]) * kHeadDim) + lane, acc[j]);
        }
      }
    }
    __syncthreads();
  }
}

// Some of a group's tiles: [begin, begin + count) of its list, the range-th of its `ranges`
// ranges, which are those of the thread blocks from first_block on.
struct Segment {
  int unit, begin, count, range, ranges, first_block;
  int before;   // tiles that the thread block has had already
};

template <int MT, bool kFp8>
__device__ __forceinline__ void serve(const CUtensorMap* kmap, const CUtensorMap* vmap,
                                      const GroupedParams& p, const Segment& seg, uint8_t* smem) {
  using L = GroupedLayout<kFp8>;
  constexpr int kWarpsN = L::kThreads / 32;
  float* merge_o = reinterpret_cast<float*>(smem);
  uint4* tile_of = reinterpret_cast<uint4*>(smem + L::kTiles);
  float* merge_m = reinterpret_cast<float*>(smem + L::kMergeM);
  float* merge_l = reinterpret_cast<float*>(smem + L::kMergeL);
  volatile int* flags = reinterpret_cast<volatile int*>(smem + L::kFlags);
  const uint32_t bars = smem_addr(smem + L::kBars);
  auto full_bar = [&](int s) { return bars + 8u * s; };
  auto empty_bar = [&](int s) { return bars + 8u * (L::kStages + s); };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kvh = blockIdx.y / p.head_groups, head0 = blockIdx.y % p.head_groups * p.heads;
  const int g = p.Hq / p.Hkv;
  const int n_heads = min(p.heads, g - head0);
  int first_row, n_seqs;
  p.units.get(seg.unit, first_row, n_seqs);
  const int n_rows = n_seqs * n_heads;
  auto out_row = [&](int r) {   // row of q / out / lse of the block's row r
    return static_cast<int64_t>(first_row + r / n_heads) * p.Hq + kvh * g + head0 + r % n_heads;
  };
  if (seg.ranges == 0) {   // a group without keys
    for (int r = warp; r < n_rows; r += kWarpsN)
      write_empty(p.out + out_row(r) * kHeadDim, p.lse ? p.lse + out_row(r) : nullptr, lane);
    return;
  }
  const int gq = lane >> 2, c4 = lane & 3;
  const int mt = warp % MT, t0 = warp / MT * (16 * MT);   // a consumer's rows and tokens
  const bool consumer = warp < L::kConsumers;
  Stream st;
  if (!consumer) {
    // ------------------------------------------------------------ producer
    // It holds the next 32 tiles of the list, one a lane, and loads the 32 after them early.
    const uint64_t policy = l2_policy_evict_first();
    const int withhold = withheld_tile();   // test hook
    const int64_t list = static_cast<int64_t>(seg.unit) * p.plan.most + seg.begin;
    uint32_t word = 0, who = 0, col = 0, word2 = 0, who2 = 0, col2 = 0;
    auto fetch = [&](int i, uint32_t& a, uint32_t& b, uint32_t& c) {
      if (i < seg.count) {
        a = p.plan.word[list + i];
        b = p.plan.mask[list + i];
        c = p.plan.column[list + i];
      }
    };
    fetch(lane, word2, who2, col2);
    for (int i = 0; i < seg.count; ++i) {
      const int it = seg.before + i;
      if (i % 32 == 0) {
        word = word2;
        who = who2;
        col = col2;
        fetch(i + 32 + lane, word2, who2, col2);
      }
      const int s = it % L::kStages;
      if (__any_sync(0xffffffffu, flags[0] != 0)) break;
      if (it >= L::kStages) {
        if (!__all_sync(0xffffffffu, mbar_wait(empty_bar(s), (it / L::kStages - 1) & 1))) {
          if (lane == 0) {
            record_error(p.err, kErrTimeout);
            flags[0] = 1;
          }
          break;
        }
      }
      const uint32_t w = __shfl_sync(0xffffffffu, word, i % 32);
      if (it >= withhold) continue;
      if (lane == i % 32) tile_of[s] = make_uint4(word, who, col, 0u);
      __syncwarp();
      const int slot = static_cast<int>(w >> 9) * kBlockSize + (w >> 7 & 3) * kTile;
      const uint32_t dst = smem_addr(smem + s * L::kStageBytes);
      mbar_arrive_expect_tx_warp(full_bar(s), L::kStageBytes);
      tma_load_3d_hint_warp(dst, kmap, full_bar(s), 0, kvh, slot, policy);
      if constexpr (!kFp8)
        tma_load_3d_hint_warp(dst + kHalfBytes, kmap, full_bar(s), 64, kvh, slot, policy);
      tma_load_3d_hint_warp(dst + L::kOpBytes, vmap, full_bar(s), 0, kvh, slot, policy);
      if constexpr (!kFp8)
        tma_load_3d_hint_warp(dst + L::kOpBytes + kHalfBytes, vmap, full_bar(s), 64, kvh, slot,
                              policy);
      if (lane == 0) flags[2] = it + 1;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ consumers
    // (the queries' latency is hidden by that of the first tile)
    uint32_t qa[8][4];
    float qmul[2] = {p.scale_log2, p.scale_log2};
    int len[2];
    unsigned bit[2], rows_of = 0;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 16 * mt + 8 * r + gq;
      const bool real = row < n_rows;
      load_q<kFp8>(real ? p.q + out_row(row) * kHeadDim : nullptr, c4, r, qa);
      const int w = real ? row / n_heads : 0;
      len[r] = real ? min(max(p.context_lens[first_row + w], 0), p.max_len) : INT32_MAX;
      bit[r] = real ? 1u << w : ~0u;
      rows_of |= real ? bit[r] : 0u;
    }
    if constexpr (kFp8) {
#pragma unroll
      for (int r = 0; r < 2; ++r) qmul[r] = f16_q(qa, r, p.scale_log2, p.k_scale);
    }
    rows_of = __reduce_or_sync(0xffffffffu, rows_of);
#pragma unroll
    for (int n = 0; n < 16; ++n) st.o[n][0] = st.o[n][1] = st.o[n][2] = st.o[n][3] = 0.f;
    st.m[0] = st.m[1] = -INFINITY;
    st.l[0] = st.l[1] = 0.f;
    volatile int& partly = flags[4 + warp];   // some row did not see all of some tile
    if (lane == 0) partly = 0;
    for (int i = 0; i < seg.count; ++i) {
      const int it = seg.before + i, s = it % L::kStages;
      if (flags[0]) break;
      if (!mbar_wait(full_bar(s), (it / L::kStages) & 1)) {
        record_error(p.err, kErrTimeout);
        flags[0] = 1;
        break;
      }
      const uint4 tile = tile_of[s];
      const int pos = tile.z * kBlockSize + static_cast<int>(tile.x >> 7 & 3) * kTile;
      const int valid = static_cast<int>(tile.x & 127u);
      // rows of other sequences, and shares behind the last token, have nothing to do
      if (tile.y & rows_of) {
        // (rows that are not there: no limit, so that they do not count; nobody reads them)
        const int lim[2] = {tile.y & bit[0] ? len[0] - pos : 0, tile.y & bit[1] ? len[1] - pos : 0};
        const uint32_t kb = smem_addr(smem + s * L::kStageBytes);
        // Up to 32 tokens at a time (64 would not leave the registers for the scores), 16 with 32
        // bf16 rows (4 x 8 sequences of 16k to 40k tokens 84 us, 32 at a time 90; with 64 rows 4 x
        // 12 of 8k to 20k 107 and 101).  Most tiles are of a prompt, which every row sees whole:
        // without the comparisons and the zeroing of what lies behind a length, 16 rows of 8 heads
        // over 30000 tokens take a tenth less, 24 x 5 E4M3 rows 59.6 us, not 61.1; narrow groups the
        // same
        constexpr int J = MT == 1 || (MT == 2 && !kFp8) ? 1 : 2;
        if (__all_sync(0xffffffffu, min(lim[0], lim[1]) >= kTile)) {
#pragma unroll 1
          for (int t = t0; t < t0 + 16 * MT; t += 16 * J)
            consume_tokens<J, kFp8, true>(kb, kb + L::kOpBytes, t, lane, qa, qmul, lim, kTile, st);
        } else {
          if (lane == 0) partly = 1;
#pragma unroll 1
          for (int t = t0; t < t0 + 16 * MT && t < valid; t += 16 * J)
            consume_tokens<J, kFp8, false>(kb, kb + L::kOpBytes, t, lane, qa, qmul, lim, valid, st);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(s));
    }
    // The weight 0 of a token that a row does not see, times a value that is not finite, is NaN.
    // That is rare, and testing the values in the loop cost 4 x 8 of 16k to 40k tokens 13 us
    // and 24 x 5 E4M3 21, so the outputs are tested here; with a NaN among them the segment's
    // rows are worked out again, each by itself (one NaN in a beam's page: 16 x 4 0.5 ms, 4 x 8 of
    // 16k to 40k 1.9 ms).
    float z[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e >> 1] = fmaf(st.o[n][e], 0.f, z[e >> 1]);
    __syncwarp();
    if (partly && ((16 * mt + gq < n_rows && z[0] != 0.f) || (16 * mt + 8 + gq < n_rows && z[1] != 0.f)))
      flags[3] = 1;
    __syncwarp();
  }
  __syncthreads();   // every warp is done with the ring, and every copy was waited for,
  // unless a wait ran out: then (bounded) for those in flight, before it is written
  if (flags[0]) {
    if (tid == 0) {
      const int issued = flags[2];
      for (int s = 0; s < L::kStages; ++s) {
        int last = -1;
        for (int it = s; it < issued; it += L::kStages) last = it;
        if (last >= 0) (void)mbar_wait(full_bar(s), (last / L::kStages) & 1);
      }
    }
    __syncthreads();
  }

  // ---------------------------------------------------------------- epilogue
  const bool again = flags[3] && !flags[0];
  if (again) {   // (each row in the place of its first share, the others empty)
    const int64_t list = static_cast<int64_t>(seg.unit) * p.plan.most + seg.begin;
    for (int r = warp; r < n_rows; r += kWarpsN) {
      const int w = r / n_heads, len = min(max(p.context_lens[first_row + w], 0), p.max_len);
      float4 o;
      float m, l;
      attend_alone<kFp8>(p, list, seg.count, kvh, p.q + out_row(r) * kHeadDim, w, len, o, m, l);
      for (int k = 0; k < 4 / MT; ++k) {
        const int row = 16 * (k * MT + r / 16) + r % 16;
        reinterpret_cast<float4*>(merge_o + row * kHeadDim)[lane] =
            k ? make_float4(0.f, 0.f, 0.f, 0.f) : o;
        merge_m[row] = k ? -INFINITY : m;
        merge_l[row] = k ? 0.f : l;
      }
    }
  } else if (consumer) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 1);
      st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 2);
      const int row = 16 * warp + 8 * r + gq;
      float* dst = merge_o + row * kHeadDim;
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        if constexpr (kFp8) {
          dst[out_dim<true>(n, c4, 0)] = st.o[n][2 * r];
          dst[out_dim<true>(n, c4, 1)] = st.o[n][2 * r + 1];
        } else {
          *reinterpret_cast<float2*>(dst + out_dim<false>(n, c4, 0)) =
              make_float2(st.o[n][2 * r], st.o[n][2 * r + 1]);
        }
      }
      if (c4 == 0) {
        merge_m[row] = st.m[r];
        merge_l[row] = st.l[r];
      }
    }
  }
  __syncthreads();
  if (tid == 0) flags[3] = 0;   // (before the next segment's first barrier)
  // a warp a row, a lane four dims
  const int stride_rows = p.units.seqs * p.heads;   // rows of a partial result
  const int64_t part0 =
      2 * (static_cast<int64_t>(blockIdx.y) * gridDim.x + seg.first_block) * stride_rows;
  for (int r = warp; r < n_rows; r += kWarpsN) {
    // the row in the k-th share's warp, k MT + r / 16
    auto at = [&](int k) { return 16 * (k * MT + r / 16) + r % 16; };
    float M = -INFINITY;
#pragma unroll
    for (int k = 0; k < 4 / MT; ++k) M = fmaxf(M, merge_m[at(k)]);
    float sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 4 / MT; ++k) {
      const float f = rescale(merge_m[at(k)], M);
      const float4 x = reinterpret_cast<const float4*>(merge_o + at(k) * kHeadDim)[lane];
      sum += merge_l[at(k)] * f;
      o.x += x.x * f;
      o.y += x.y * f;
      o.z += x.z * f;
      o.w += x.w * f;
    }
    // (a row may hold none of the range's blocks: 0, -inf)
    const float inv = sum > 0.f ? (kFp8 ? p.v_scale : 1.f) / sum : sum * 0.f;
    o.x *= inv;
    o.y *= inv;
    o.z *= inv;
    o.w *= inv;
    const float lse2 = M + __log2f(sum);
    if (seg.ranges > 1) {
      const int64_t at_row = part0 + partial_of(seg.range) * stride_rows + r;
      __stcg(reinterpret_cast<float4*>(p.ws_o + at_row * kHeadDim) + lane, o);
      if (lane == 0) __stcg(p.ws_lse + at_row, lse2);
    } else {
      const int64_t row = out_row(r);
      uint2 packed;
      packed.x = pack_bf16x2(o.x, o.y);
      packed.y = pack_bf16x2(o.z, o.w);
      *reinterpret_cast<uint2*>(p.out + row * kHeadDim + 4 * lane) = packed;
      if (p.lse && lane == 0) p.lse[row] = lse2 * kLn2;
    }
  }
  if (seg.ranges <= 1) return;

  // ---------------------------------------------------------------- merge of the ranges
  // By the last block to arrive; many ranges kMergeGroup at a time first, by the last block of
  // each, into the first one's place.
  const bool two = p.group_count && seg.ranges > 2 * kMergeGroup;
  const int groups = (seg.ranges + kMergeGroup - 1) / kMergeGroup;
  const int group = two ? seg.range / kMergeGroup : 0;
  for (int step = two ? 0 : 1; step < 2; ++step) {
    const bool final = step == 1;
    const int from = final ? 0 : group * kMergeGroup, by = final && two ? kMergeGroup : 1;
    const int n = !final ? min(kMergeGroup, seg.ranges - from) : two ? groups : seg.ranges;
    __syncthreads();
    if (tid == 0) {
      unsigned* counter =
          final ? p.ws_count + static_cast<int64_t>(seg.unit) * gridDim.y + blockIdx.y
                : p.group_count +
                      2 * (static_cast<int64_t>(blockIdx.y) * gridDim.x + seg.first_block) +
                      partial_of(from);
      __threadfence();
      const bool last = atomicAdd(counter, 1u) == static_cast<unsigned>(n - 1);
      if (last) {
        __threadfence();
        *counter = 0u;   // ready for the next call
      }
      flags[1] = last ? 1 : 0;
    }
    __syncthreads();
    if (!flags[1]) return;
    merge_ranges(p.ws_lse + part0, p.ws_o + part0 * kHeadDim, from, by, n, stride_rows, final, n_rows,
                 out_row, p.out, p.lse, reinterpret_cast<float*>(smem));
  }
}

// Calls serve(segment) for each of this thread block's (every warp works them out by itself;
// one call in the code, as a second copy of it would not stay in the instruction cache).
template <class Serve>
__device__ __forceinline__ void each_segment(const GroupedParams& p, int lane, const Serve& serve) {
  const bool dealt = p.split == 0;   // or: a range of one group, as the caller asked
  Stretch mine;
  if (dealt) {
    mine = find_stretch(p.plan, p.units.count, gridDim.x, blockIdx.x, lane);
    if (mine.unit < 0) return;
  } else {
    mine.unit = blockIdx.x / p.split;
    mine.tiles = tiles_of(p.plan, mine.unit);
    mine.share = max(1, (mine.tiles + p.split - 1) / p.split);
    mine.start = -kSegment;
    mine.from = blockIdx.x % p.split * mine.share;
    mine.to = min(mine.tiles, mine.from + mine.share);
    // (a group without keys is its first block's)
    if (mine.from >= max(mine.tiles, 1)) return;
    if (mine.tiles == 0) mine.from = mine.start;
  }
  Segment seg;
  seg.before = 0;
  int T = mine.tiles, start = mine.start;
  for (seg.unit = mine.unit;; ++seg.unit) {
    const int next = dealt && seg.unit + 1 < p.units.count ? tiles_of(p.plan, seg.unit + 1) : 0;
    const int first = start + kSegment, last = first + T;   // the tiles' places
    const int from = max(mine.from, first), to = min(mine.to, last);
    seg.begin = from - first;
    seg.count = to - from;
    const int block0 = first / mine.share;   // of the dealt ones, or of the group's
    seg.ranges = T > 0 ? (last - 1) / mine.share - block0 + 1 : 0;
    seg.first_block = dealt ? block0 : seg.unit * p.split;
    seg.range = static_cast<int>(blockIdx.x) - seg.first_block;
    if (seg.count > 0 || (T == 0 && mine.from <= start)) {
      serve(seg);
      seg.before += max(seg.count, 0);
    }
    start = last;
    if (start >= mine.to) break;
    T = next;
    // what the last group left in the ring is read and written before copies come again
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
}

template <int MT, bool kFp8>
__global__ void __launch_bounds__(GroupedLayout<kFp8>::kThreads, 2)
grouped_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const GroupedParams p) {
  using L = GroupedLayout<kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (threadIdx.x == 0) {
    const uint32_t bars = smem_addr(smem + L::kBars);
    volatile int* flags = reinterpret_cast<volatile int*>(smem + L::kFlags);
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bars + 8u * s, 1);
      mbar_init(bars + 8u * (L::kStages + s), L::kConsumers);
    }
    flags[0] = flags[1] = flags[2] = flags[3] = 0;
    fence_barrier_init();
  }
  // May start while the plan is being made, and lets the next kernel start (see
  // decode_kernel.cuh): nothing is read before the wait, and nothing through the
  // read-only path.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();   // (the barriers are set up)

  each_segment(p, threadIdx.x & 31,
               [&](const Segment& seg) { serve<MT, kFp8>(&kmap, &vmap, p, seg, smem); });
}

struct GroupedPlan {
  int m_tiles;             // MT
  int heads, head_groups;
  Units units;
  int split, ranges;       // ranges: of all sequence groups, per kv head and head group
  int64_t most;            // tiles of a group, if its sequences share nothing
  size_t part_rows;        // rows of all partial results
  size_t list_at, part_at; // in the workspace: the plan's arrays, the partial results
  size_t workspace_bytes;
};

int plan_grouped(int B, int width, int Hq, int Hkv, int maxblk, int num_splits, int sm_count,
                 GroupedPlan* plan) {
  if (B < 0 || width < 1 || Hq < 1 || Hkv < 1 || maxblk < 0 || num_splits < 0) return PKV_ERR_ARG;
  if (Hq % Hkv || B % width || width > kMaxWidth || maxblk > kMaxColumns) return PKV_ERR_SHAPE;
  const int g = Hq / Hkv;
  // at most 64 rows a thread block: whole sequences, in groups of about equal size
  plan->head_groups = (g + 63) / 64;
  plan->heads = (g + plan->head_groups - 1) / plan->head_groups;
  const int fit = 64 / plan->heads;
  Units& u = plan->units;
  u.width = width;
  u.groups = (width + fit - 1) / fit;
  u.seqs = (width + u.groups - 1) / u.groups;
  const int rows = plan->heads * u.seqs;
  plan->m_tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  const int64_t y = static_cast<int64_t>(Hkv) * plan->head_groups;
  const int64_t units = static_cast<int64_t>(B / width) * u.groups;
  if (y > 65535 || y * units > kWorkspaceCounters) return PKV_ERR_SHAPE;
  u.count = static_cast<int>(units);
  plan->split = static_cast<int>(num_splits < kMaxRanges ? num_splits : kMaxRanges);
  int64_t ranges = units * plan->split;
  if (plan->split == 0 && units > 0) {
    // as many thread blocks as the SMs hold at a time, two each
    const int64_t slots = 2 * static_cast<int64_t>(sm_count > 0 ? sm_count : 148);
    ranges = slots > y ? slots / y : 1;
  }
  plan->ranges = static_cast<int>(ranges);
  plan->most = static_cast<int64_t>(u.seqs) * maxblk * kTilesPerBlock;
  // places on the line of all tiles are 32-bit (groups of a request hold less than twice its
  // sequences)
  if (static_cast<int64_t>(B) * maxblk > 1 << 27) return PKV_ERR_SHAPE;
  plan->list_at = kWorkspaceCounterBytes;
  const size_t tiles = static_cast<size_t>(units) * plan->most;
  plan->part_at = plan->list_at + align_up(units * 4, 256) + 2 * align_up(tiles * 4, 256) +
                  align_up(tiles * 2, 256);
  plan->part_rows = 2 * static_cast<size_t>(ranges) * y * rows;
  plan->workspace_bytes = plan->part_at + align_up(plan->part_rows * kHeadDim * 4, 256) +
                          align_up(plan->part_rows * 4, 256);
  return PKV_OK;
}

PlanArrays plan_arrays(const GroupedPlan& plan, void* workspace) {
  uint8_t* at = static_cast<uint8_t*>(workspace) + plan.list_at;
  const size_t tiles = static_cast<size_t>(plan.units.count) * plan.most;
  PlanArrays a;
  a.tiles = reinterpret_cast<int*>(at);
  at += align_up(static_cast<size_t>(plan.units.count) * 4, 256);
  a.word = reinterpret_cast<uint32_t*>(at);
  at += align_up(tiles * 4, 256);
  a.mask = reinterpret_cast<uint32_t*>(at);
  at += align_up(tiles * 4, 256);
  a.column = reinterpret_cast<uint16_t*>(at);
  a.most = plan.most;
  return a;
}

// Both kernels are launched with programmatic stream serialization.
cudaLaunchConfig_t dependent_launch(dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                    cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int MT, bool kFp8>
int launch_form(const GroupedPlan& plan, const GroupedParams& prm, const CUtensorMap& km,
                const CUtensorMap& vm, cudaStream_t stream) {
  using L = GroupedLayout<kFp8>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    if (cudaFuncSetAttribute(grouped_decode_kernel<MT, kFp8>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             L::kBytes) != cudaSuccess)
      return PKV_ERR_LAUNCH;
    if (dev < 64) attr_set[dev] = true;
  }
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = dependent_launch(dim3(plan.ranges, prm.Hkv * plan.head_groups),
                                                  L::kThreads, L::kBytes, stream, &attr);
  if (cudaLaunchKernelEx(&cfg, grouped_decode_kernel<MT, kFp8>, km, vm, prm) != cudaSuccess)
    return PKV_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

int grouped_entry(const DecodeArgs& a, int width, int D, int block_size, int planned,
                  pkv_stream_t stream) {
  int st = check_decode_args(a, D, block_size);
  if (st) return st;
  if (!std::isfinite(a.scale)) return PKV_ERR_ARG;
  GroupedPlan plan;
  st = plan_grouped(a.B, width, a.Hq, a.Hkv, a.max_blocks_per_seq, a.num_splits,
                    device_sm_count(), &plan);
  if (st || a.B == 0) return st;
  if (!workspace_fits(a.workspace, a.workspace_bytes, plan.workspace_bytes))
    return PKV_ERR_WORKSPACE;
  unsigned* err = device_error_word();
  if (!err) return PKV_ERR_LAUNCH;
  CUtensorMap km, vm;
  if (!decode_maps(a, &km, &vm)) return PKV_ERR_ARG;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  PlanParams pp = {};
  pp.block_tables = a.block_tables;
  pp.context_lens = a.context_lens;
  pp.out = plan_arrays(plan, ws);
  pp.units = plan.units;
  pp.maxblk = a.max_blocks_per_seq;
  pp.num_blocks = static_cast<int>(a.num_blocks);
  pp.err = err;
  if (!planned) {
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg =
        dependent_launch(dim3(plan.units.count), kPlanThreads, 0, cs, &attr);
    if (cudaLaunchKernelEx(&cfg, grouped_plan_kernel, pp) != cudaSuccess) return PKV_ERR_LAUNCH;
  }

  GroupedParams prm = {};
  prm.out = static_cast<__nv_bfloat16*>(a.out);
  prm.lse = a.lse;
  prm.q = static_cast<const __nv_bfloat16*>(a.q);
  prm.k_cache = a.k_cache;
  prm.v_cache = a.v_cache;
  prm.num_blocks = static_cast<uint32_t>(a.num_blocks);
  prm.context_lens = a.context_lens;
  prm.ws_count = reinterpret_cast<unsigned*>(ws);
  const int64_t y = static_cast<int64_t>(a.Hkv) * plan.head_groups;
  if (y * (plan.units.count + 2 * static_cast<int64_t>(plan.ranges)) <= kWorkspaceCounters)
    prm.group_count = prm.ws_count + y * plan.units.count;
  prm.ws_o = reinterpret_cast<float*>(ws + plan.part_at);
  prm.ws_lse = reinterpret_cast<float*>(ws + plan.part_at +
                                        align_up(plan.part_rows * kHeadDim * 4, 256));
  prm.err = err;
  prm.plan = pp.out;
  prm.units = plan.units;
  prm.Hq = a.Hq;
  prm.Hkv = a.Hkv;
  prm.max_len = a.max_blocks_per_seq * kBlockSize;
  prm.split = plan.split;
  prm.heads = plan.heads;
  prm.head_groups = plan.head_groups;
  prm.scale_log2 = a.scale * 1.4426950408889634f;
  prm.k_scale = a.k_scale;
  prm.v_scale = a.v_scale;
  if (a.fp8) {
    if (plan.m_tiles == 1) return launch_form<1, true>(plan, prm, km, vm, cs);
    if (plan.m_tiles == 2) return launch_form<2, true>(plan, prm, km, vm, cs);
    return launch_form<4, true>(plan, prm, km, vm, cs);
  }
  if (plan.m_tiles == 1) return launch_form<1, false>(plan, prm, km, vm, cs);
  if (plan.m_tiles == 2) return launch_form<2, false>(plan, prm, km, vm, cs);
  return launch_form<4, false>(plan, prm, km, vm, cs);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t paged_decode_grouped_workspace_bytes(int B, int width, int Hq, int Hkv, int D,
                                                       int max_blocks_per_seq, int block_size,
                                                       int fp8, int num_splits) {
  if (D != kHeadDim || block_size != kBlockSize) return 0;
  GroupedPlan plan;
  (void)fp8;   // (the plan does not depend on it)
  if (plan_grouped(B, width, Hq, Hkv, max_blocks_per_seq, num_splits, device_sm_count(), &plan))
    return 0;
  return plan.workspace_bytes;
}

extern "C" int paged_decode_attention_grouped(
    void* out, float* lse, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens, int B,
    int width, int Hq, int Hkv, int D, int block_size, int64_t num_blocks, float scale,
    void* workspace, size_t workspace_bytes, int num_splits, int planned,
    pkv_stream_t stream) {
  const DecodeArgs a{out, lse, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                     context_lens, B, Hq, Hkv, num_blocks, scale, workspace, workspace_bytes,
                     num_splits, 0};
  return grouped_entry(a, width, D, block_size, planned, stream);
}

extern "C" int paged_decode_attention_grouped_fp8(
    void* out, float* lse, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens, int B,
    int width, int Hq, int Hkv, int D, int block_size, int64_t num_blocks, float scale,
    float k_scale, float v_scale, void* workspace, size_t workspace_bytes, int num_splits,
    int planned, pkv_stream_t stream) {
  const DecodeArgs a{out, lse, q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                     context_lens, B, Hq, Hkv, num_blocks, scale, workspace, workspace_bytes,
                     num_splits, 0, 1, 1, k_scale, v_scale};
  return grouped_entry(a, width, D, block_size, planned, stream);
}
