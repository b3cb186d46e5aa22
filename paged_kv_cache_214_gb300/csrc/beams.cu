// beams.cu — block tables of sequences that grow and fork, on the device: room for new
// tokens (paged_append_tokens), the tables after a selection of beams
// (paged_reorder_beams) and the copies that it asks for (kv_cache_copy_rows).
//
// The first two move a few hundred kilobytes at most and are bound by latency: a chain of
// dependent loads (lengths, prefix sums, table entries) and one launch each.  So every
// thread block works out the prefix sums that it needs for itself, and what depends on all
// blocks (lengths written in place, the stack of free blocks) is left to the last one
// to arrive: one launch, nothing spins, and the order of the stack follows from the
// inputs alone.  A call of a graph of many: appending a token to 256 sequences 3.9 us, up to
// 1500 tokens to 48 sequences 5.8; reordering 1 x 4 / 64 x 4 / 20 x 12 rows 5.5, 7.8 and 9.5
// us (tables, lengths and stack are under 1 MB).  The copies are bound by memory where there
// are many: 55 MB read and 55 written in 11.5 us (the writes stay in L2).

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kMaxRows = 8192;   // rows whose prefix sums a thread block keeps

// Exclusive prefix sums of two values over the block's threads, and their totals.
// `buf`: 2 * 32 values.
template <typename T>
__device__ __forceinline__ void block_scan2(T a, T b, T* buf, T& ea, T& eb, T& ta, T& tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  T ia = a, ib = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T xa = __shfl_up_sync(0xffffffffu, ia, d), xb = __shfl_up_sync(0xffffffffu, ib, d);
    if (lane >= d) {
      ia += xa;
      ib += xb;
    }
  }
  __syncthreads();   // the buffer may still be read from a scan before
  if (lane == 31) {
    buf[warp] = ia;
    buf[32 + warp] = ib;
  }
  __syncthreads();
  ea = ia - a;
  eb = ib - b;
  ta = tb = 0;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) {
      ea += buf[w];
      eb += buf[32 + w];
    }
    ta += buf[w];
    tb += buf[32 + w];
  }
}

// Whether this block is the last of `blocks` to get here; everything that the others
// wrote before is then visible to it.  The counter is left zero.
__device__ __forceinline__ bool last_block(unsigned* counter, unsigned blocks, int* flag) {
  if (blocks == 1) {
    __syncthreads();
    return true;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const bool last = atomicAdd(counter, 1u) == blocks - 1;
    if (last) {
      __threadfence();
      *counter = 0u;
    }
    *flag = last ? 1 : 0;
  }
  __syncthreads();
  return *flag != 0;
}

// Last index i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_not_above(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ append

struct AppendParams {
  int32_t* slots;
  int32_t* positions;
  int32_t* cu_q;
  int32_t* cu_k;
  int32_t* out_lens;
  int32_t* out_num_free;
  int32_t* tables;
  const int32_t* lens;
  const int32_t* new_lens;   // null: a decode step
  const int32_t* free_blocks;
  const int32_t* num_free;
  int R, maxblk;
  int tokens;     // entries of slots and positions
  int num_blocks;
  unsigned* counter;
  unsigned* err;
};

constexpr int kAppendThreads = 256;

// cu_tok[r], cu_need[r]: tokens and blocks of the rows before r that are served, and
// old[r], kept in shared memory by every block.  A token finds its row by bisection.
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
  extern __shared__ int smem[];
  __shared__ long long buf[64];
  __shared__ int flag;
  const int R = p.R, tid = threadIdx.x;
  int* cu_tok = smem;              // [R + 1]
  int* cu_need = smem + R + 1;     // [R + 1]
  int* old = smem + 2 * (R + 1);   // [R]
  // a thread's rows in the prefix sums: an odd number, which lie in different banks
  const int per = (R + kAppendThreads - 1) / kAppendThreads | 1;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  const bool packed = p.new_lens != nullptr, reports = blockIdx.x == 0;
  int nf = *p.num_free;
  if (nf < 0 || nf > p.num_blocks) {
    if (reports && tid == 0) record_error(p.err, kErrIndex);
    nf = nf < 0 ? 0 : p.num_blocks;
  }
  const long long cap = static_cast<long long>(p.maxblk) * kBlockSize;

  // what the rows ask for
#pragma unroll 4
  for (int r = tid; r < R; r += kAppendThreads) {
    const int o = p.lens[r];
    int n = packed ? p.new_lens[r] : (o > 0 ? 1 : 0), blocks = 0;
    if (o < 0 || n < 0 || static_cast<long long>(o) + n > cap) {
      if (reports) record_error(p.err, kErrIndex);
      n = 0;
    } else if (n > 0) {
      blocks = (o + n - 1) / kBlockSize - (o - 1 + kBlockSize) / kBlockSize + 1;
    }
    old[r] = o;
    cu_tok[r] = n;
    cu_need[r] = blocks;
  }
  __syncthreads();
  long long tok = 0, need = 0;
  for (int r = r0; r < r1; ++r) {
    tok += cu_tok[r];
    need += cu_need[r];
  }
  long long tok0, need0, tok_all, need_all;
  block_scan2(tok, need, buf, tok0, need0, tok_all, need_all);
  // what they get; the blocks of a row that is served come behind those that all rows
  // before it asked for, which were served too (the needs only grow)
  long long got = 0, keys = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = cu_tok[r], blocks = cu_need[r];
    tok0 += n;
    need0 += blocks;
    const bool served =
        n > 0 && (blocks == 0 || need0 <= nf) && (!packed || tok0 <= p.tokens);
    cu_tok[r] = served ? n : 0;
    cu_need[r] = served ? blocks : 0;
    got += cu_tok[r];
    keys += max(old[r], 0) + static_cast<long long>(cu_tok[r]);
  }
  long long got0, keys0, got_all, keys_all;
  block_scan2(got, keys, buf, got0, keys0, got_all, keys_all);
  long long have = 0, spare = 0, have0, spare0, have_all, spare_all;
  for (int r = r0; r < r1; ++r) have += cu_need[r];
  block_scan2(have, spare, buf, have0, spare0, have_all, spare_all);
  const bool writes_cu = reports && packed;
  if (writes_cu && keys_all > INT32_MAX && tid == 0) record_error(p.err, kErrIndex);
  for (int r = r0; r < r1; ++r) {
    const int n = cu_tok[r], blocks = cu_need[r];
    cu_tok[r] = static_cast<int>(got0);
    cu_need[r] = static_cast<int>(have0);
    if (writes_cu) {
      p.cu_q[r] = static_cast<int>(got0);
      p.cu_k[r] = static_cast<int>(min(keys0, static_cast<long long>(INT32_MAX)));
    }
    got0 += n;
    have0 += blocks;
    keys0 += max(old[r], 0) + static_cast<long long>(n);
  }
  const int total = static_cast<int>(got_all), taken = static_cast<int>(have_all);
  if (tid == 0) {
    cu_tok[R] = total;
    cu_need[R] = taken;
    if (writes_cu) {
      p.cu_q[R] = total;
      p.cu_k[R] = static_cast<int>(min(keys_all, static_cast<long long>(INT32_MAX)));
    }
  }
  __syncthreads();

  const int step = gridDim.x * kAppendThreads, first = blockIdx.x * kAppendThreads + tid;
  // a free block's id, or -1 for one outside the pool
  auto popped = [&](int i) {
    const int id = p.free_blocks[nf - 1 - i];
    if (id >= 0 && id < p.num_blocks) return id;
    record_error(p.err, kErrIndex);
    return -1;
  };
  for (int t = first; t < p.tokens; t += step) {
    int r = -1, pos = 0, slot = -1;
    if (packed) {
      if (t < total) {
        r = last_not_above(cu_tok, R, t);
        pos = old[r] + t - cu_tok[r];
      }
    } else if (cu_tok[t + 1] > cu_tok[t]) {
      r = t;
      pos = old[t];
    }
    if (r >= 0) {
      const int column = pos / kBlockSize;
      const int fresh = column - (old[r] + kBlockSize - 1) / kBlockSize;
      int id;
      if (fresh >= 0) {
        id = popped(cu_need[r] + fresh);
      } else {
        id = p.tables[static_cast<int64_t>(r) * p.maxblk + column];
        if (id < 0 || id >= p.num_blocks) {
          record_error(p.err, kErrIndex);
          id = -1;
        }
      }
      if (id >= 0) slot = id * kBlockSize + pos % kBlockSize;
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
  for (int i = first; i < taken; i += step) {
    const int r = last_not_above(cu_need, R, i);
    const int column = (old[r] + kBlockSize - 1) / kBlockSize + i - cu_need[r];
    p.tables[static_cast<int64_t>(r) * p.maxblk + column] = popped(i);
  }
  // lengths and the stack's height may be written over the inputs: once every block
  // has read them
  if (!last_block(p.counter, gridDim.x, &flag)) return;
  for (int r = tid; r < R; r += kAppendThreads) p.out_lens[r] = old[r] + cu_tok[r + 1] - cu_tok[r];
  if (tid == 0) *p.out_num_free = nf - taken;
}

constexpr int kAppendBlocks = 304;
int append_blocks(int R, int64_t tokens) {
  const int64_t work = tokens > R ? tokens : R;
  // a token a thread, although every block repeats the prefix sums: 48 rows of up to 1500
  // new tokens take 5.5 us, with eight tokens a thread 7.9
  const int64_t blocks = (work + kAppendThreads - 1) / kAppendThreads;
  return static_cast<int>(blocks < 1 ? 1 : blocks > kAppendBlocks ? kAppendBlocks : blocks);
}

// ------------------------------------------------------------------ reorder

struct ReorderParams {
  int32_t* out_tables;
  int32_t* out_lens;
  int32_t* copies;        // [3, R]
  int32_t* out_num_free;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* parents;
  const int32_t* kept;    // or null
  int32_t* free_blocks;
  const int32_t* num_free;
  int B, W, maxblk, num_blocks;
  int* freed;             // [B, W * maxblk] blocks that each request gives back
  int* n_freed;           // [B]
  unsigned* wants;        // [B] rows that need a block of their own
  unsigned* counter;
  unsigned* err;
};

constexpr int kReorderThreads = 256;

// One thread block a request, which walks over the columns in chunks of kColumns.  A chunk's
// entries of all rows go to shared memory before any is written, so that the tables may
// be reordered in place; a thread then looks after one (row, column): what the row's
// child table holds there, and whether the block is given back (no row with a child and
// no earlier row holds it).
constexpr int kColumns = 64;
__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(const ReorderParams p) {
  extern __shared__ int smem[];              // [W][kColumns] entries of the chunk, -1: none
  __shared__ int par[kMaxWidth], len[kMaxWidth], buf[64], flag;
  __shared__ unsigned freed_rows[kColumns], sourceless;   // (rows whose copy has no source)
  const int W = p.W, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x, R = p.B * W;
  const int row0 = b * W;
  const int kept = p.kept ? p.kept[b] : 0;
  if (tid < W) {
    int q = p.parents[row0 + tid], n = p.lens[row0 + tid];
    if (q < -1 || q >= W) {
      record_error(p.err, kErrIndex);
      q = -1;
    }
    if (n < 0 || n > static_cast<int64_t>(p.maxblk) * kBlockSize) {
      record_error(p.err, kErrIndex);
      n = 0;
    }
    par[tid] = q;
    len[tid] = n;
  }
  if (tid == 0) sourceless = 0;
  __syncthreads();
  // every thread: rows that have a child, and rows that are not their parent's first
  unsigned has_child = 0, later = 0;
  int most = 0;
  for (int i = 0; i < W; ++i) {
    most = max(most, len[i]);
    if (par[i] >= 0) {
      if (has_child >> par[i] & 1u) later |= 1u << i;
      has_child |= 1u << par[i];
    }
  }
  const int held_columns = (most + kBlockSize - 1) / kBlockSize;

  int count = 0;   // blocks given back so far
  for (int c0 = 0; c0 < held_columns; c0 += kColumns) {
    const int columns = min(kColumns, p.maxblk - c0), items = W * columns;
    if (tid < kColumns) freed_rows[tid] = 0;
#pragma unroll 4
    for (int i = tid; i < items; i += kReorderThreads) {
      const int w = i / columns, c = i - w * columns;
      const bool held = (c0 + c) * kBlockSize < len[w];
      int id = held ? p.tables[static_cast<int64_t>(row0 + w) * p.maxblk + c0 + c] : -1;
      if (held && (id < 0 || id >= p.num_blocks)) {
        record_error(p.err, kErrIndex);
        id = -1;
      }
      smem[w * kColumns + c] = id;
    }
    __syncthreads();
    for (int i = tid; i < items; i += kReorderThreads) {
      const int w = i / columns, c = i - w * columns, column = c0 + c;
      const int from = par[w];
      int next = from < 0 ? -1 : smem[from * kColumns + c];
      // the block that the parent is filling stays with its first child
      if ((later >> w & 1u) && len[from] / kBlockSize == column && len[from] % kBlockSize) {
        p.copies[row0 + w] = next;
        p.copies[2 * R + row0 + w] = next < 0 ? 0 : len[from] % kBlockSize;
        if (next < 0) atomicOr(&sourceless, 1u << w);
        next = -1;
      }
      p.out_tables[static_cast<int64_t>(row0 + w) * p.maxblk + column] = next;
      const int id = smem[w * kColumns + c];
      if (id >= 0 && column >= kept) {
        bool gone = !(has_child >> w & 1u);
        for (int u = 0; u < W && gone; ++u)
          gone = smem[u * kColumns + c] != id || (u >= w && !(has_child >> u & 1u));
        if (gone) atomicOr(&freed_rows[c], 1u << w);
      }
    }
    __syncthreads();
    // in the order of columns, then rows
    int at, unused0, all, unused1;
    const unsigned mine = tid < kColumns ? freed_rows[tid] : 0u;
    block_scan2(__popc(mine), 0, buf, at, unused0, all, unused1);
    int* out = p.freed + static_cast<int64_t>(row0) * p.maxblk + count + at;
    for (unsigned left = mine; left; left &= left - 1)
      *out++ = smem[(__ffs(left) - 1) * kColumns + tid];
    count += all;
    __syncthreads();
  }
  // columns that no row holds
  const int done = min(p.maxblk, (held_columns + kColumns - 1) / kColumns * kColumns);
  for (int w = 0; w < W; ++w)
    for (int c = done + tid; c < p.maxblk; c += kReorderThreads)
      p.out_tables[static_cast<int64_t>(row0 + w) * p.maxblk + c] = -1;
  // a row that would copy a block which is none becomes empty (the chunks' entries are written),
  // and takes no block off the stack
  const unsigned gone_rows = sourceless;
  for (unsigned left = gone_rows; left; left &= left - 1)
    for (int c = tid; c < done; c += kReorderThreads)
      p.out_tables[static_cast<int64_t>(row0 + __ffs(left) - 1) * p.maxblk + c] = -1;
  if (tid < W) {
    const bool gone = gone_rows >> tid & 1u;
    const int row = row0 + tid, n = par[tid] < 0 || gone ? 0 : len[par[tid]];
    p.out_lens[row] = n;
    if (!(later >> tid & 1u) || n % kBlockSize == 0) {
      p.copies[row] = -1;
      p.copies[2 * R + row] = 0;
      later &= ~(1u << tid);
    }
    p.copies[R + row] = -1;
  }
  if (warp == 0) {
    const unsigned wants = __ballot_sync(0xffffffffu, lane < W && (later >> lane & 1u));
    if (lane == 0) {
      p.n_freed[b] = count;
      p.wants[b] = wants;
    }
  }
  if (!last_block(p.counter, gridDim.x, &flag)) return;

  // The last block: all requests' blocks onto the stack, in order, then the rows' own
  // ones off it; a thread a block or row, its request found by bisection.
  __shared__ int base[kReorderThreads];
  __shared__ unsigned want[kReorderThreads];
  int nf = *p.num_free;
  if (nf < 0 || nf > p.num_blocks) {
    if (tid == 0) record_error(p.err, kErrIndex);
    nf = nf < 0 ? 0 : p.num_blocks;
  }
  long long top = nf;
  for (int b0 = 0; b0 < p.B; b0 += kReorderThreads) {
    const int n = min(kReorderThreads, p.B - b0);
    int at, unused0, all, unused1;
    block_scan2(tid < n ? __ldcg(p.n_freed + b0 + tid) : 0, 0, buf, at, unused0, all, unused1);
    base[tid] = at;
    __syncthreads();
    for (int i = tid; i < all; i += kReorderThreads) {
      const int k = last_not_above(base, n, i);
      const int id = __ldcg(p.freed + static_cast<int64_t>(b0 + k) * W * p.maxblk + i - base[k]);
      if (top + i < p.num_blocks) p.free_blocks[top + i] = id;
      else record_error(p.err, kErrIndex);   // more blocks than the pool has
    }
    top = min(top + all, static_cast<long long>(p.num_blocks));
    __syncthreads();
  }
  for (int b0 = 0; b0 < p.B; b0 += kReorderThreads) {
    const int n = min(kReorderThreads, p.B - b0);
    want[tid] = tid < n ? __ldcg(p.wants + b0 + tid) : 0u;
    int at, unused0, all, unused1;
    block_scan2(__popc(want[tid]), 0, buf, at, unused0, all, unused1);
    base[tid] = at;
    __syncthreads();
    for (int e = tid; e < all; e += kReorderThreads) {
      const int k = last_not_above(base, n, e);
      unsigned rows = want[k];
      for (int skip = e - base[k]; skip > 0; --skip) rows &= rows - 1;
      const int row = (b0 + k) * W + __ffs(rows) - 1;
      const long long i = top - 1 - e;
      int32_t* entries = p.out_tables + static_cast<int64_t>(row) * p.maxblk;
      const int column = __ldcg(p.out_lens + row) / kBlockSize;
      const int id = i >= 0 ? __ldcg(p.free_blocks + i) : -1;
      if (id >= 0 && id < p.num_blocks) {
        entries[column] = id;
        p.copies[R + row] = id;
      } else {   // none left: the row cannot go on
        record_error(p.err, kErrIndex);
        for (int c = 0; c < column; ++c) entries[c] = -1;
        p.out_lens[row] = 0;
        p.copies[row] = -1;
        p.copies[2 * R + row] = 0;
      }
    }
    top = max(0ll, top - all);
    __syncthreads();
  }
  if (tid == 0) *p.out_num_free = static_cast<int>(top);
}

size_t reorder_workspace(int B, int W, int maxblk) {
  return kWorkspaceCounterBytes + 2 * align_up(static_cast<size_t>(B) * 4, 256) +
         align_up(static_cast<size_t>(B) * W * maxblk * 4, 256);
}

// ------------------------------------------------------------------ row copies

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;                                  // 16-byte words a thread
constexpr int kPieceVecs = kCopyThreads * kCopyVecs;          // 16 KB

// The copied rows of a block are contiguous ([token, Hkv, D]): pieces of 16 KB of all
// copies, K's then V's, are dealt out to the thread blocks, which find a piece's copy by
// bisection over prefix sums that each works out for itself.
__global__ void __launch_bounds__(kCopyThreads)
copy_rows_kernel(uint4* k_cache, uint4* v_cache, const int32_t* copies, int R, int row_vecs,
                 int num_blocks, unsigned* err) {
  extern __shared__ int cu[];   // [R + 1] pieces of the rows before r, in one pool
  __shared__ int buf[64];
  const int tid = threadIdx.x;
  const int per = (R + kCopyThreads - 1) / kCopyThreads;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  int mine = 0;
  for (int r = r0; r < r1; ++r) {
    const int src = copies[r], dst = copies[R + r], n = copies[2 * R + r];
    int pieces = 0;
    if (src >= 0) {
      if (src >= num_blocks || dst < 0 || dst >= num_blocks || n < 0 || n > kBlockSize) {
        if (blockIdx.x == 0) record_error(err, kErrIndex);
      } else {
        pieces = (n * row_vecs + kPieceVecs - 1) / kPieceVecs;
      }
    }
    cu[r] = pieces;
    mine += pieces;
  }
  int at, unused0, total, unused1;
  block_scan2(mine, 0, buf, at, unused0, total, unused1);
  for (int r = r0; r < r1; ++r) {
    const int pieces = cu[r];
    cu[r] = at;
    at += pieces;
  }
  __syncthreads();
  for (int64_t i = blockIdx.x; i < 2 * static_cast<int64_t>(total); i += gridDim.x) {
    const bool second = i >= total;
    const int piece = static_cast<int>(second ? i - total : i);
    const int r = last_not_above(cu, R, piece);
    const int64_t block_vecs = static_cast<int64_t>(kBlockSize) * row_vecs;
    uint4* pool = second ? v_cache : k_cache;
    const uint4* from = pool + copies[r] * block_vecs;
    uint4* to = pool + copies[R + r] * block_vecs;
    const int n = copies[2 * R + r] * row_vecs;
    const int v0 = (piece - cu[r]) * kPieceVecs + tid;
    uint4 x[kCopyVecs];
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j)
      if (v0 + j * kCopyThreads < n) x[j] = from[v0 + j * kCopyThreads];
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j)
      if (v0 + j * kCopyThreads < n) to[v0 + j * kCopyThreads] = x[j];
  }
}

int launched() { return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH; }

// Pool and table sizes of the calls that see neither heads nor values.
int check_tables(int rows, int maxblk, int block_size, int64_t num_blocks) {
  if (rows < 0 || maxblk < 0) return PKV_ERR_ARG;
  const int st = check_pool(1, kHeadDim, block_size, num_blocks);
  if (st) return st;
  return rows > kMaxRows ? PKV_ERR_SHAPE : PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t paged_append_tokens_workspace_bytes(int R, int64_t max_tokens) {
  if (R < 0 || R > kMaxRows || max_tokens < 0 || max_tokens > INT32_MAX) return 0;
  return append_blocks(R, max_tokens) > 1 ? kWorkspaceCounterBytes : 0;
}

extern "C" int paged_append_tokens(int32_t* slot_mapping, int32_t* positions,
                                   int32_t* cu_seqlens_q, int32_t* cu_seqlens_k,
                                   int32_t* out_lens, int32_t* out_num_free,
                                   int32_t* block_tables, int max_blocks_per_seq,
                                   const int32_t* context_lens, const int32_t* new_lens,
                                   const int32_t* free_blocks, const int32_t* num_free, int R,
                                   int64_t max_tokens, int block_size, int64_t num_blocks,
                                   void* workspace, size_t workspace_bytes,
                                   pkv_stream_t stream) {
  const int st = check_tables(R, max_blocks_per_seq, block_size, num_blocks);
  if (st) return st;
  if (max_tokens < 0 || (!new_lens && max_tokens != R)) return PKV_ERR_ARG;
  // a thread's walk over the tokens ends a grid's threads behind the last one at most
  if (max_tokens > INT32_MAX - kAppendBlocks * kAppendThreads) return PKV_ERR_SHAPE;
  // token positions are 32-bit
  if (max_blocks_per_seq > INT32_MAX / kBlockSize) return PKV_ERR_SHAPE;
  if (!num_free || !out_num_free) return PKV_ERR_ARG;
  if (R > 0 && (!out_lens || !context_lens)) return PKV_ERR_ARG;
  if (R > 0 && max_blocks_per_seq > 0 && !block_tables) return PKV_ERR_ARG;
  if (num_blocks > 0 && !free_blocks) return PKV_ERR_ARG;
  if (max_tokens > 0 && (!slot_mapping || !positions)) return PKV_ERR_ARG;
  if (new_lens && (!cu_seqlens_q || !cu_seqlens_k)) return PKV_ERR_ARG;
  const int blocks = append_blocks(R, max_tokens);
  if (!workspace_fits(workspace, workspace_bytes, blocks > 1 ? kWorkspaceCounterBytes : 0))
    return PKV_ERR_WORKSPACE;
  unsigned* err = device_error_word();
  if (!err) return PKV_ERR_LAUNCH;
  const AppendParams p{slot_mapping, positions, cu_seqlens_q, cu_seqlens_k, out_lens,
                       out_num_free, block_tables, context_lens, new_lens, free_blocks, num_free,
                       R, max_blocks_per_seq, static_cast<int>(max_tokens),
                       static_cast<int>(num_blocks), static_cast<unsigned*>(workspace), err};
  auto smem_of = [](size_t rows) { return (3 * rows + 2) * sizeof(int); };
  const size_t smem = smem_of(R);
  // Without the attribute 48 KB hold the kernel's static shared memory (half a KB) too.  (Always
  // to the most that a call can need: another thread may be about to launch.)
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(append_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem_of(kMaxRows))) != cudaSuccess)
    return PKV_ERR_LAUNCH;
  append_kernel<<<blocks, kAppendThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return launched();
}

extern "C" size_t paged_reorder_beams_workspace_bytes(int B, int width, int max_blocks_per_seq) {
  if (B < 0 || width < 1 || width > kMaxWidth || max_blocks_per_seq < 0 ||
      static_cast<int64_t>(B) * width > kMaxRows)
    return 0;
  return reorder_workspace(B, width, max_blocks_per_seq);
}

extern "C" int paged_reorder_beams(int32_t* out_tables, int32_t* out_lens, int32_t* copies,
                                   int32_t* out_num_free, const int32_t* block_tables,
                                   int max_blocks_per_seq, const int32_t* context_lens,
                                   const int32_t* parents, const int32_t* kept_blocks,
                                   int32_t* free_blocks, const int32_t* num_free, int B,
                                   int width, int block_size, int64_t num_blocks,
                                   void* workspace, size_t workspace_bytes,
                                   pkv_stream_t stream) {
  if (B < 0 || width < 1) return PKV_ERR_ARG;
  if (width > kMaxWidth || B > kMaxRows) return PKV_ERR_SHAPE;
  const int st = check_tables(B * width, max_blocks_per_seq, block_size, num_blocks);
  if (st) return st;
  if (max_blocks_per_seq > INT32_MAX / kBlockSize) return PKV_ERR_SHAPE;
  if (!num_free || !out_num_free) return PKV_ERR_ARG;
  if (num_blocks > 0 && !free_blocks) return PKV_ERR_ARG;
  if (B > 0 && (!out_lens || !copies || !context_lens || !parents)) return PKV_ERR_ARG;
  if (B > 0 && max_blocks_per_seq > 0 && (!out_tables || !block_tables)) return PKV_ERR_ARG;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0) {
    if (num_free == out_num_free) return PKV_OK;
    return cudaMemcpyAsync(out_num_free, num_free, sizeof(int32_t), cudaMemcpyDeviceToDevice,
                           cs) == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
  }
  if (!workspace_fits(workspace, workspace_bytes, reorder_workspace(B, width, max_blocks_per_seq)))
    return PKV_ERR_WORKSPACE;
  unsigned* err = device_error_word();
  if (!err) return PKV_ERR_LAUNCH;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t list = align_up(static_cast<size_t>(B) * 4, 256);
  const ReorderParams p{out_tables, out_lens, copies, out_num_free, block_tables, context_lens,
                        parents, kept_blocks, free_blocks, num_free, B, width,
                        max_blocks_per_seq, static_cast<int>(num_blocks),
                        reinterpret_cast<int*>(ws + kWorkspaceCounterBytes + 2 * list),
                        reinterpret_cast<int*>(ws + kWorkspaceCounterBytes),
                        reinterpret_cast<unsigned*>(ws + kWorkspaceCounterBytes + list),
                        reinterpret_cast<unsigned*>(ws), err};
  const size_t smem = static_cast<size_t>(width) * kColumns * sizeof(int);
  reorder_kernel<<<B, kReorderThreads, smem, cs>>>(p);
  return launched();
}

extern "C" int kv_cache_copy_rows(void* k_cache, void* v_cache, const int32_t* copies, int R,
                                  int Hkv, int D, int elem_bytes, int block_size,
                                  int64_t num_blocks, pkv_stream_t stream) {
  if (R < 0 || (elem_bytes != 1 && elem_bytes != 2)) return PKV_ERR_ARG;
  const int st = check_pool(Hkv, D, block_size, num_blocks);
  if (st) return st;
  if (R > kMaxRows) return PKV_ERR_SHAPE;
  const int64_t row_vecs = static_cast<int64_t>(Hkv) * D * elem_bytes / 16;
  // a block's words and the pieces of all copies are counted in 32 bits
  const int64_t block_pieces = (kBlockSize * row_vecs + kPieceVecs - 1) / kPieceVecs;
  if (kBlockSize * row_vecs > INT32_MAX - kPieceVecs || block_pieces * R > INT32_MAX)
    return PKV_ERR_SHAPE;
  if (R == 0) return PKV_OK;
  if (!k_cache || !v_cache || !copies) return PKV_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 15u)
    return PKV_ERR_ARG;
  unsigned* err = device_error_word();
  if (!err) return PKV_ERR_LAUNCH;
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  // no more blocks than pieces, if every row had a copy
  const int64_t pieces = 2 * R * block_pieces;
  const int64_t grid = pieces < 4 * static_cast<int64_t>(sms) ? pieces : 4 * static_cast<int64_t>(sms);
  const size_t smem = (static_cast<size_t>(R) + 1) * sizeof(int);
  copy_rows_kernel<<<static_cast<unsigned>(grid), kCopyThreads, smem,
                     reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), copies, R,
      static_cast<int>(row_vecs), static_cast<int>(num_blocks), err);
  return launched();
}
