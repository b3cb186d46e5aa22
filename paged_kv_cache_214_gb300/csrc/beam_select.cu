// beam_select.cu — the best continuations of each request's beams (beam_select).
//
//   s[w, v] = c[w] + x[w, v] - ln(sum_u exp(x[w, u])),   the num_out best of a request
//
// One pass over the logits, which is all the traffic there is.  A row is cut into segments
// of 512 logits; the pass keeps a running maximum and sum of exponentials and one number
// a segment, its maximum.  That is enough to find the candidates afterwards, so the
// streaming loop carries no lists: the last thread block of a request to finish takes
// the K-th largest of its threads' largest maxima as a bound (K continuations reach it),
// reads the segments that reach it again (K or a few more, K KB and mostly from L2) and
// ranks the logits that do.  Bounds are compared in fp32 with a margin for its rounding,
// candidates ranked by their score in 64 bits.
// 64 x 8 rows of 150001 bf16 logits, 154 MB, 16 best: 41 us a call of a graph (floor 23), 29 of
// them the pass (5.3 TB/s; issue 55%, 2^x 25%), the rest the last block's work, in which
// the other SMs idle.  4 rows of 32000: 10.2 us, a chain of dependent steps.  Two, four or
// five thread blocks an SM took 51, 43 and 43 us where three took 40.
// Work a logit: widening, maximum (three at a time), two multiply-adds (two at a time), one
// 2^x, one addition (two at a time).
//
// Sums.  Scores of different beams are compared, so a row's sum has to be right to better
// than a score's own rounding.  2^(x log2(e) - C) with C = fl(m log2(e)) and log2(e) as a sum
// of two fp32 numbers leaves the roundings of single terms (2^-22 and less) and of the additions
// in fp32 (16 terms in two chains, a segment a step, five steps over the lanes); C itself cancels
// exactly, as the merge adds it back in 64 bits, in which the warps' sums are joined too.
// Measured against 64 bits, rows of 1000 to 150001 logits, flat, ordinary and with one token
// that has half of the mass, around 0 and around 8000: off by 1e-7 (root of the mean square up
// to 1.9e-7), 3.2e-7 at most.

#include <cuda_bf16.h>
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSegment = 512;     // logits; 16 a lane
constexpr int kPerSm = 3;         // thread blocks
constexpr int kMaxOut = 64;
constexpr int kHeld = 10;         // maxima of a request that a thread keeps
constexpr int kMostFound = kThreads;   // segments read again, candidates ranked
constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596299e-8f;
constexpr double kLn2d = 0.69314718055994530942;
// Largest maximum whose C = fl(m log2(e)) is used: C's own rounding is at most 2^-11 there,
// so 2^(x log2(e) - C) stays near 1 for x = m.
constexpr float kFar = 8192.f;

struct SelectParams {
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  float* out_end;
  const void* logits;
  int64_t row_stride;
  const float* scores;
  int B, W, V, K, eos;
  int segments;         // of a row
  int share;            // segments that a thread block reads, of the request's rows in order
  int pieces;           // that a row is cut into at most
  float2* stats;        // [R][pieces * kWarps] (maximum, sum against it) of a warp's logits
  float* maxima;        // [R][segments]
  unsigned* counters;   // [B]
};

// fp32 or bf16 logits of one lane in a segment, 16 in two (bf16) or four vectors.
template <bool kF32>
struct Row {
  static constexpr int kVec = kF32 ? 4 : 8;   // logits of a 16-byte word
  const uint8_t* base;   // 16-byte aligned address at or below the row's first logit
  int skew;              // logits between
  int V;
  __device__ Row(const void* logits, int64_t at, int n) : V(n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(logits) + at * (kF32 ? 4 : 2);
    base = reinterpret_cast<const uint8_t*>(a & ~uintptr_t(15));
    skew = static_cast<int>((a & 15) / (kF32 ? 4 : 2));
  }
  // The segments lie on 16-byte boundaries of memory: place u is logit u - skew.
  __device__ int first(int seg, int lane, int j) const {
    return seg * kSegment + (j * 32 + lane) * kVec - skew;
  }
  // word j of the lane; places outside the row read as -inf
  __device__ __forceinline__ uint4 load(int seg, int lane, int j) const {
    const int v = first(seg, lane, j);
    const uint4* at = reinterpret_cast<const uint4*>(base) +
                      (static_cast<int64_t>(seg) * kSegment / kVec + j * 32 + lane);
    if (v >= 0 && v + kVec <= V) return __ldg(at);
    uint32_t w[4];
    const uint32_t none = kF32 ? 0xff800000u : 0xff80u;
    if constexpr (kF32) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = v + i >= 0 && v + i < V ? reinterpret_cast<const uint32_t*>(at)[i] : none;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(at) + 2 * i;
        const uint32_t lo = v + 2 * i >= 0 && v + 2 * i < V ? h[0] : none;
        const uint32_t hi = v + 2 * i + 1 >= 0 && v + 2 * i + 1 < V ? h[1] : none;
        w[i] = lo | hi << 16;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static constexpr int kWords = 16 / kVec;
  __device__ __forceinline__ void load_segment(int seg, int lane, uint4 (&u)[kWords]) const {
    const int from = seg * kSegment - skew;
    if (from >= 0 && from + kSegment <= V) {   // all of it
      const uint4* at = reinterpret_cast<const uint4*>(base) + static_cast<int64_t>(seg) * (kSegment / kVec) + lane;
#pragma unroll
      for (int j = 0; j < kWords; ++j) u[j] = __ldg(at + 32 * j);
    } else {
#pragma unroll
      for (int j = 0; j < kWords; ++j) u[j] = load(seg, lane, j);
    }
  }
  __device__ __forceinline__ static void widen(const uint4 (&u)[kWords], float (&x)[16]) {
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kF32) {
          x[4 * j + i] = __uint_as_float(w[i]);
        } else {
          x[8 * j + 2 * i] = bf16lo(w[i]);
          x[8 * j + 2 * i + 1] = bf16hi(w[i]);
        }
      }
    }
  }
};

__device__ __forceinline__ float max16(const float (&x)[16]) {
  float a = max3(x[0], x[1], x[2]), b = max3(x[3], x[4], x[5]), c = max3(x[6], x[7], x[8]);
  float d = max3(x[9], x[10], x[11]), e = max3(x[12], x[13], x[14]);
  return fmaxf(max3(a, b, c), max3(d, e, x[15]));
}

// Largest of the lanes' values (one instruction on sm_100 and later; a NaN is ignored
// unless all are).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// A running sum of e^(x - m) is kept against C = fl(m log2(e)) of the maximum m, that of
// rows with larger logits (masks of the type's lowest value) against m itself.  (The rounded
// product wherever it is used: a subtraction that took it into an FMA would be off by its
// rounding, 2^-24 of the logit.)
__device__ __forceinline__ float reference(float m) { return __fmul_rn(m, kLog2eHi); }

__device__ __forceinline__ float sum16(const float (&x)[16], float m) {
  float s;
  if (fabsf(m) <= kFar) {
    const f32x2 hi = pack2(kLog2eHi, kLog2eHi), lo = pack2(kLog2eLo, kLog2eLo);
    const float C = reference(m);
    const f32x2 c = pack2(-C, -C);
    f32x2 total = 0;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const f32x2 v = pack2(x[i], x[i + 1]);
      const f32x2 t = fma2(v, lo, fma2(v, hi, c));
      total = add2(total, pack2(ex2(lo2(t)), ex2(hi2(t))));
    }
    s = lo2(total) + hi2(total);
  } else {   // large logits, infinities, NaN
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      s += m == -INFINITY ? (x[i] == x[i] ? 0.f : x[i]) : ex2((x[i] - m) * kLog2eHi);
  }
  return s;
}

// Factor that takes a sum against m to one against the larger maximum n.  Each is kept as its own
// maximum says: with one beyond kFar and one not, the near one's C is taken as it is and the far
// one's logarithm worked out to its difference from C (its rounding alone would leave 2^-11).
__device__ __forceinline__ float shift(float m, float n) {
  if (m == -INFINITY) return 0.f;
  const bool near_m = fabsf(m) <= kFar, near_n = fabsf(n) <= kFar;
  if (near_m && near_n) return ex2(reference(m) - reference(n));
  if (near_m) return ex2(fmaf(-n, kLog2eLo, fmaf(-n, kLog2eHi, reference(m))));
  if (near_n) return ex2(fmaf(m, kLog2eLo, fmaf(m, kLog2eHi, -reference(n))));
  return m == n ? 1.f : ex2((m - n) * kLog2eHi);
}

// A score as an integer of the same order (compared at the integer rate, an eighth of a
// 64-bit float's cost and less): larger is better.  Below every score: kNone.
constexpr long long kNone = INT64_MIN;
__device__ __forceinline__ long long key_of(double s) {
  const long long b = __double_as_longlong(s + 0.0);   // (-0 is 0)
  return b < 0 ? b ^ INT64_MAX : b;
}
__device__ __forceinline__ double score_of(long long k) {
  return __longlong_as_double(k < 0 ? k ^ INT64_MAX : k);
}

// A candidate's place in the order: by score, equal ones by index.
__device__ __forceinline__ bool before(long long s, int i, long long t, int j) {
  return s > t || (s == t && i < j);
}

constexpr int kFinders = kThreads - 32;   // threads that look for candidates

struct alignas(16) MergeSmem {
  // ln p(v) = (x[v] - ref) - log_sum: in this order, rows of large logits keep the second
  double ref[kMaxWidth], log_sum[kMaxWidth], cum[kMaxWidth], sum[kMaxWidth];
  float max[kMaxWidth], at_eos[kMaxWidth];
  float ref_f[kMaxWidth], off_f[kMaxWidth];   // scores in fp32: (x - ref_f) + off_f (NaN: none)
  int tops[kFinders / 2];
  int segment[kMostFound];       // w * segments + s
  long long found_s[kMostFound];
  float found_x[kMostFound];
  int found_i[kMostFound];       // w * V + v
  long long next_s[kMaxWidth];   // a beam's next continuation, where there are many equal ones
  float next_x[kMaxWidth], best_x[kWarps];
  int next_i[kMaxWidth], best_v[kWarps];
  int kth, margin, n_segments, n_found, last;
};

// fp32 as an integer of the same order.
__device__ __forceinline__ int order_of(float x) {
  const int b = __float_as_int(x);
  return b < 0 ? b ^ 0x7fffffff : b;
}
__device__ __forceinline__ float float_of(int k) {
  return __int_as_float(k < 0 ? k ^ 0x7fffffff : k);
}

// The K-th largest of the values that pairs of finders hold at most (-inf where fewer have
// any): K of all values reach it.
__device__ __forceinline__ float kth_largest(float mine, int K, MergeSmem& sm) {
  const int tid = threadIdx.x;
  const float pair = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, 1));
  if (tid % 2 == 0) sm.tops[tid / 2] = order_of(pair);
  if (tid == 0) sm.kth = order_of(-INFINITY);
  named_barrier(1, kFinders);
  if (tid < kFinders / 2) {
    const int own = sm.tops[tid];
    int not_less = 0;
#pragma unroll 4
    for (int j = 0; j < kFinders / 8; ++j) {
      const int4 v = reinterpret_cast<const int4*>(sm.tops)[j];
      not_less += (v.x >= own) + (v.y >= own) + (v.z >= own) + (v.w >= own);
    }
    if (not_less >= K) atomicMax(&sm.kth, own);
  }
  named_barrier(1, kFinders);
  return float_of(sm.kth);
}

// A beam's score of logit x in fp32 (NaN: no continuations).  With its terms rounded it is off
// by 2^-24 of 2 |ref| + 2 |off| + 2 |score| and of twice the logarithm (22 at most).
__device__ __forceinline__ float rough(const MergeSmem& sm, int w, float x) {
  return (x - sm.ref_f[w]) + sm.off_f[w];
}
// A bound on scores as one on rough scores: lower by more than twice their error.
__device__ __forceinline__ float lowered(float bound, const MergeSmem& sm) {
  return bound - (__int_as_float(sm.margin) + fabsf(bound) + 22.f) * 4e-7f;   // (-inf stays)
}

// f(w, logit, token, rough score) for the continuations in the listed segments (in all, where
// there was no room for the list because of equal scores) that reach the bound, a segment a
// warp; the next one is on its way while one is looked at.
template <bool kF32, class F>
__device__ __forceinline__ void each_logit(const SelectParams& p, int b, const MergeSmem& sm,
                                           int warp, int warps, float bound, const F& f) {
  const int lane = threadIdx.x & 31, S = p.segments;
  const bool listed = sm.n_segments <= kMostFound;
  const int n = listed ? sm.n_segments : p.W * S;
  constexpr int kWords = Row<kF32>::kWords;
  uint4 u[kWords], ahead[kWords];
  auto row_of = [&](int w) {
    return Row<kF32>(p.logits, (static_cast<int64_t>(b) * p.W + w) * p.row_stride, p.V);
  };
  auto fetch = [&](int k) {
    if (k >= n) return;
    const int at = listed ? sm.segment[k] : k;
    const Row<kF32> in = row_of(at / S);
    in.load_segment(at % S, lane, ahead);
  };
  fetch(warp);
#pragma unroll 1
  for (int k = warp; k < n; k += warps) {
    const int at = listed ? sm.segment[k] : k;
    const int w = at / S;
    const float ref = sm.ref_f[w], off = sm.off_f[w];
#pragma unroll
    for (int j = 0; j < kWords; ++j) u[j] = ahead[j];
    fetch(k + warps);
    const Row<kF32> in = row_of(w);
    float x[16];
    Row<kF32>::widen(u, x);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float r = (x[e] - ref) + off;   // rough()
      if (!(r >= bound && r > -INFINITY)) continue;
      const int v = in.first(at % S, lane, e / Row<kF32>::kVec) + e % Row<kF32>::kVec;
      if (v != p.eos) f(w, x[e], v, r);
    }
  }
}

// The logits that may be among the K best, into sm.found (and their number, which may be more
// than fit).  By kFinders threads.
template <bool kF32>
__device__ __forceinline__ void find_candidates(const SelectParams& p, int b,
                                                const float (&held)[kHeld], MergeSmem& sm) {
  const int tid = threadIdx.x, warp = tid >> 5;
  const int W = p.W, K = p.K, S = p.segments;
  const float* maxima = p.maxima + static_cast<int64_t>(b) * W * S;
  // f(place, rough score) for the thread's maxima
  const int w0 = tid / S, rest0 = tid % S, dw = kFinders / S, dr = kFinders % S;
  auto each_maximum = [&](auto f) {
    int w = w0, rest = rest0;
    auto step = [&] {
      const bool carry = rest + dr >= S;
      w += dw + (carry ? 1 : 0);
      rest += dr - (carry ? S : 0);
    };
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      if (tid + e * kFinders < W * S) f(tid + e * kFinders, rough(sm, w, held[e]));
      step();
    }
    for (int i = tid + kHeld * kFinders; i < W * S; i += kFinders, step()) f(i, rough(sm, w, __ldcg(maxima + i)));
  };
  float top = -INFINITY;
  each_maximum([&](int, float r) { top = r > top ? r : top; });
  float bound = lowered(kth_largest(top, K, sm), sm);
  each_maximum([&](int i, float r) {
    if (r >= bound && r > -INFINITY) {
      const int at = atomicAdd(&sm.n_segments, 1);
      if (at < kMostFound) sm.segment[at] = i;
    }
  });
  named_barrier(1, kFinders);
  auto collect = [&] {
    each_logit<kF32>(p, b, sm, warp, kFinders / 32, bound, [&](int w, float x, int v, float) {
      // (once there are too many it is enough to know that)
      if (*const_cast<volatile int*>(&sm.n_found) > kMostFound) return;
      const int at = atomicAdd(&sm.n_found, 1);
      if (at < kMostFound) {
        sm.found_x[at] = x;
        sm.found_i[at] = w * p.V + v;
      }
    });
    named_barrier(1, kFinders);
  };
  // (no bound: fewer segments than places)
  const bool none = bound == -INFINITY && p.V > kMostFound;
  if (!none) collect();
  if (none || sm.n_found > kMostFound) {
    // A weak bound (or long rows of equal logits): a better one from the logits themselves.
    top = -INFINITY;
    each_logit<kF32>(p, b, sm, warp, kFinders / 32, bound,
                     [&](int, float, int, float r) { top = fmaxf(top, r); });
    bound = lowered(kth_largest(top, K, sm), sm);
    if (tid == 0) sm.n_found = 0;
    named_barrier(1, kFinders);
    collect();
  }
}

// The last thread block of request b.  64-bit arithmetic is slow: the sums' logarithms are
// taken by a warp of its own (all beams at once) while the others look for candidates by
// fp32 scores, and candidates are scored one a lane.  The code is kept short because it
// runs once, from a cold instruction cache.
template <bool kF32>
__device__ __forceinline__ void merge_request(const SelectParams& p, int b, MergeSmem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int W = p.W, K = p.K, S = p.segments;
  const double nan = __longlong_as_double(0x7ff8000000000000ll);

  // The maxima that this finder looks after, every kFinders-th of the request's.
  const float* maxima = p.maxima + static_cast<int64_t>(b) * W * S;
  float held[kHeld];
#pragma unroll
  for (int e = 0; e < kHeld; ++e)
    held[e] = tid + e * kFinders < W * S ? __ldcg(maxima + tid + e * kFinders) : -INFINITY;

  // a warp a beam: its sum (what a beam that has not begun left here counts for nothing)
#pragma unroll 1
  for (int w = warp; w < W; w += kWarps) {
    const int64_t row = static_cast<int64_t>(b) * W + w;
    const float2* st = p.stats + row * p.pieces * kWarps;
    const int parts = (((w + 1) * S - 1) / p.share - w * S / p.share + 1) * kWarps;
    const float2 first = lane < parts ? __ldcg(st + lane) : make_float2(-INFINITY, 0.f);
    const float cum = p.scores[row];
    float at_eos = 0.f;
    if (p.eos >= 0 && lane == 0 && isfinite(cum))
      at_eos = kF32 ? static_cast<const float*>(p.logits)[row * p.row_stride + p.eos]
                    : __bfloat162float(static_cast<const __nv_bfloat16*>(
                          p.logits)[row * p.row_stride + p.eos]);
    float m = first.x;
    for (int i = lane + 32; i < parts; i += 32) m = fmaxf(m, __ldcg(st + i).x);
    m = warp_max(m);
    // (a NaN stays one, and an infinite maximum leaves one)
    double sum = first.y * shift(first.x, m);
    for (int i = lane + 32; i < parts; i += 32) {
      const float2 v = __ldcg(st + i);
      sum += static_cast<double>(v.y * shift(v.x, m));
    }
#pragma unroll 1
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) {
      sm.cum[w] = cum;
      sm.sum[w] = isfinite(cum) ? sum : 0.;
      sm.max[w] = m;
      sm.at_eos[w] = at_eos;
    }
  }
  if (tid == 0) sm.margin = sm.n_segments = sm.n_found = 0;
  __syncthreads();
  const bool finder = tid < kFinders;
  // all logits -inf: a sum of 0
  auto alive = [&](int w) { return sm.sum[w] > 0 && isfinite(sm.sum[w]) && isfinite(sm.max[w]); };
  if (!finder) {
    if (lane < W) {
      const float m = sm.max[lane];
      const double ref = fabsf(m) <= kFar ? static_cast<double>(reference(m)) * kLn2d
                                          : static_cast<double>(m);
      const double log_sum = alive(lane) ? log(sm.sum[lane]) : nan;
      sm.ref[lane] = ref;
      sm.log_sum[lane] = log_sum;
      if (p.eos >= 0)
        p.out_end[static_cast<int64_t>(b) * W + lane] =
            alive(lane) ? static_cast<float>(sm.cum[lane] + ((sm.at_eos[lane] - ref) - log_sum))
                        : -INFINITY;
    }
  } else {
    if (tid < W) {
      const float m = sm.max[tid];
      const float ref = fabsf(m) <= kFar ? reference(m) * static_cast<float>(kLn2d) : m;
      const float off = static_cast<float>(sm.cum[tid]) - logf(static_cast<float>(sm.sum[tid]));
      sm.ref_f[tid] = ref;
      sm.off_f[tid] = alive(tid) ? off : __int_as_float(0x7fffffff);   // NaN
      if (alive(tid)) atomicMax(&sm.margin, __float_as_int(fabsf(ref) + fabsf(off)));
    }
    named_barrier(1, kFinders);
    find_candidates<kF32>(p, b, held, sm);
  }
  __syncthreads();
  const int n_found = sm.n_found;
  float* out_s = p.out_scores + static_cast<int64_t>(b) * K;
  int32_t* out_w = p.out_parents + static_cast<int64_t>(b) * K;
  int32_t* out_v = p.out_tokens + static_cast<int64_t>(b) * K;
  auto write = [&](int k, long long s, int i) {
    out_s[k] = i < 0 ? -INFINITY : static_cast<float>(score_of(s));
    out_w[k] = i < 0 ? -1 : i / p.V;
    out_v[k] = i < 0 ? -1 : i % p.V;
  };
  auto exact = [&](int w, float x) { return key_of(sm.cum[w] + ((x - sm.ref[w]) - sm.log_sum[w])); };
  if (n_found <= kMostFound) {
    if (tid < n_found) sm.found_s[tid] = exact(sm.found_i[tid] / p.V, sm.found_x[tid]);
    __syncthreads();
    if (tid < n_found) {
      const long long s = sm.found_s[tid];
      const int i = sm.found_i[tid];
      int rank = 0;
#pragma unroll 4
      for (int c = 0; c < n_found; ++c) rank += before(sm.found_s[c], sm.found_i[c], s, i) ? 1 : 0;
      if (rank < K) write(rank, s, i);
    }
    for (int k = n_found + tid; k < K; k += kThreads) write(k, kNone, -1);
    return;
  }
  // More candidates than room still: many equal logits (masks of the type's lowest value are
  // some).  In a beam the order is that of (logit, token), whatever the rounding, so each
  // beam's next continuation is kept; the best of them is taken and the beam's next one
  // looked for, K passes over a beam's logits.  (8 x 4 rows of 50001 with ten tokens that are
  // not masked, 8 best: 330 us, 150 where all logits are equal; a pass over all beams for each
  // continuation took 2600 and 700.)
  auto next = [&](int w, float last_x, int last_v) {   // behind (last_x, last_v), into sm
    if (!alive(w)) {   // (its logits are not read)
      if (tid == 0) {
        sm.next_i[w] = -1;
        sm.next_s[w] = kNone;
      }
      __syncthreads();
      return;
    }
    const Row<kF32> in(p.logits, (static_cast<int64_t>(b) * W + w) * p.row_stride, p.V);
    constexpr int kWords = Row<kF32>::kWords;
    float x = -INFINITY;
    int v = INT32_MAX;
#pragma unroll 2
    for (int g = warp; g < S; g += kWarps) {
      uint4 u[kWords];
      in.load_segment(g, lane, u);
      float y[16];
      Row<kF32>::widen(u, y);
#pragma unroll
      for (int e = 0; e < 16; ++e) {   // (tokens of a lane come in order)
        const int t = in.first(g, lane, e / Row<kF32>::kVec) + e % Row<kF32>::kVec;
        if (y[e] > x && t != p.eos && (y[e] < last_x || (y[e] == last_x && t > last_v))) {
          x = y[e];
          v = t;
        }
      }
    }
    auto take = [&](float ox, int ov) {
      if (ox > x || (ox == x && ov < v)) {
        x = ox;
        v = ov;
      }
    };
#pragma unroll 1
    for (int d = 16; d; d >>= 1) {
      const float ox = __shfl_xor_sync(0xffffffffu, x, d);
      take(ox, __shfl_xor_sync(0xffffffffu, v, d));
    }
    if (lane == 0) {
      sm.best_x[warp] = x;
      sm.best_v[warp] = v;
    }
    __syncthreads();
    for (int c = 0; c < kWarps; ++c) take(sm.best_x[c], sm.best_v[c]);
    if (tid == 0) {
      const bool any = x > -INFINITY && rough(sm, w, x) > -INFINITY;
      sm.next_x[w] = x;
      sm.next_i[w] = any ? w * p.V + v : -1;
      sm.next_s[w] = any ? exact(w, x) : kNone;
    }
    __syncthreads();
  };
#pragma unroll 1
  for (int k = -W; k < K; ++k) {
    int w = k + W;   // the beams' first ones, in turn
    float x = INFINITY;
    int v = -1;
    if (k >= 0) {
      w = -1;
      for (int c = 0; c < W; ++c)
        if (sm.next_i[c] >= 0 && (w < 0 || before(sm.next_s[c], sm.next_i[c], sm.next_s[w], sm.next_i[w])))
          w = c;
      if (tid == 0) write(k, w < 0 ? kNone : sm.next_s[w], w < 0 ? -1 : sm.next_i[w]);
      if (w < 0) continue;
      x = sm.next_x[w];
      v = sm.next_i[w] % p.V;
      __syncthreads();   // (read by all before it is replaced)
    }
    next(w, x, v);
  }
}

// grid (shares of a request, requests).  Equal shares of a request's segments, whatever rows
// they belong to.
template <bool kF32>
__global__ void __launch_bounds__(kThreads, kPerSm) select_kernel(const SelectParams p) {
  __shared__ MergeSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = p.segments, b = blockIdx.y;
  constexpr int kWords = Row<kF32>::kWords;
  const int g0 = blockIdx.x * p.share, g1 = min(p.W * S, g0 + p.share);
  for (int w = g0 / S; w <= (g1 - 1) / S; ++w) {
    const int64_t row = static_cast<int64_t>(b) * p.W + w, row_at = row * S;
    const int begin = max(g0 - w * S, 0), end = min(g1 - w * S, S);
    float m = -INFINITY, sum = 0.f;   // m: the warp's, sum: the lane's
    if (isfinite(p.scores[row])) {
      const Row<kF32> in(p.logits, row * p.row_stride, p.V);
      const int eos_seg = p.eos < 0 ? -1 : (p.eos + in.skew) / kSegment;
      float* maxima = p.maxima + row_at;
      // the warp's next segments are on their way while one is worked on (rows begin with
      // another warp each, for rows of a few segments)
      constexpr int kAhead = kF32 ? 1 : 2;
      uint4 ahead[kAhead][kWords];
      auto fetch = [&](int seg, uint4 (&to)[kWords]) {
        if (seg < end) in.load_segment(seg, lane, to);
      };
      const int first = begin + (warp + w) % kWarps;
#pragma unroll
      for (int h = 0; h < kAhead; ++h) fetch(first + h * kWarps, ahead[h]);
      for (int at = first; at < end; at += kAhead * kWarps) {
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
          const int s = at + h * kWarps;
          if (h > 0 && s >= end) break;
          float x[16];
          Row<kF32>::widen(ahead[h], x);
          fetch(s + kAhead * kWarps, ahead[h]);
          const float top = warp_max(max16(x));
          float of_segment = top;
          if (s == eos_seg) {   // the ending token is no candidate
            float y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              y[e] = in.first(s, lane, e / Row<kF32>::kVec) + e % Row<kF32>::kVec == p.eos
                         ? -INFINITY
                         : x[e];
            of_segment = warp_max(max16(y));
          }
          if (lane == 0) __stcg(maxima + s, of_segment);
          if (top > m) {
            sum *= shift(m, top);
            m = top;
          }
          sum += sum16(x, m);
        }
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) {
      const int piece = blockIdx.x - w * S / p.share;
      __stcg(p.stats + (row * p.pieces + piece) * kWarps + warp, make_float2(m, sum));
    }
  }
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    const bool last = atomicAdd(p.counters + b, 1u) == gridDim.x - 1;
    if (last) {
      __threadfence();
      p.counters[b] = 0u;
    }
    sm.last = last ? 1 : 0;
  }
  __syncthreads();
  if (sm.last) merge_request<kF32>(p, b, sm);
}

struct SelectPlan {
  int segments, share, pieces, blocks;   // blocks: of a request
  size_t stats_bytes, workspace_bytes;
};

// Segments of a row (it may begin up to 15 bytes behind a 16-byte boundary), and the shares of
// a request, a segment for each warp at least: one wave of thread blocks where that fills
// the SMs, else three and more.  (Measured with shares of one row's 32 to 160 segments,
// 512 rows of 150001: 51 to 43 us.)
SelectPlan plan_select(int B, int W, int V, bool f32, int sm_count) {
  SelectPlan plan;
  const int skew = f32 ? 3 : 7;
  plan.segments = static_cast<int>((static_cast<int64_t>(V) + skew + kSegment - 1) / kSegment);
  const int64_t rows = static_cast<int64_t>(B) * W;
  const int segments = W * plan.segments;   // of a request
  const int slots = kPerSm * (sm_count > 0 ? sm_count : 148);
  int n = B > 0 ? slots / B : 1;
  if (n * B < slots * 7 / 8) n = (3 * slots + B - 1) / B;
  const int most = (segments + kWarps - 1) / kWarps;
  if (n > most) n = most;
  plan.share = (segments + n - 1) / n;
  plan.blocks = (segments + plan.share - 1) / plan.share;
  plan.pieces = (plan.segments - 1) / plan.share + 2;
  plan.stats_bytes = align_up(static_cast<size_t>(rows) * plan.pieces * kWarps * 8, 256);
  plan.workspace_bytes = kWorkspaceCounterBytes + plan.stats_bytes +
                         align_up(static_cast<size_t>(rows) * plan.segments * 4, 256);
  return plan;
}

int check_select(int B, int W, int V, int K) {
  if (B < 0 || W < 1 || V < 1 || K < 1) return PKV_ERR_ARG;
  if (W > kMaxWidth || K > kMaxOut) return PKV_ERR_SHAPE;
  // (a place in the row's last segment, or one segment on, is a 32-bit number too)
  if (static_cast<int64_t>(W) * V > INT32_MAX - 2 * kSegment) return PKV_ERR_SHAPE;
  if (static_cast<int64_t>(B) * W > 65535) return PKV_ERR_SHAPE;
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" size_t beam_select_workspace_bytes(int B, int width, int V, int logits_fp32) {
  if (check_select(B, width, V, 1) != PKV_OK || B == 0) return 0;
  return plan_select(B, width, V, logits_fp32 != 0, device_sm_count()).workspace_bytes;
}

extern "C" int beam_select(float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                           float* out_end, const void* logits, int logits_fp32,
                           int64_t row_stride, const float* scores, int B, int width, int V,
                           int num_out, int eos_token, void* workspace, size_t workspace_bytes,
                           pkv_stream_t stream) {
  const int st = check_select(B, width, V, num_out);
  if (st) return st;
  if (eos_token < -1 || eos_token >= V || row_stride < V) return PKV_ERR_ARG;
  if (B == 0) return PKV_OK;
  if (!out_scores || !out_parents || !out_tokens || !logits || !scores) return PKV_ERR_ARG;
  if (eos_token >= 0 && !out_end) return PKV_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % (logits_fp32 ? 4 : 2)) return PKV_ERR_ARG;
  const SelectPlan plan = plan_select(B, width, V, logits_fp32 != 0, device_sm_count());
  if (!workspace_fits(workspace, workspace_bytes, plan.workspace_bytes)) return PKV_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const SelectParams p{out_scores, out_parents, out_tokens, out_end, logits, row_stride, scores,
                       B, width, V, num_out, eos_token, plan.segments, plan.share,
                       plan.pieces, reinterpret_cast<float2*>(ws + kWorkspaceCounterBytes),
                       reinterpret_cast<float*>(ws + kWorkspaceCounterBytes + plan.stats_bytes),
                       reinterpret_cast<unsigned*>(ws)};
  const dim3 grid(plan.blocks, B);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (logits_fp32)
    select_kernel<true><<<grid, kThreads, 0, cs>>>(p);
  else
    select_kernel<false><<<grid, kThreads, 0, cs>>>(p);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}
