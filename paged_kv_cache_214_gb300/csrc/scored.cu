// scored.cu — paged attention whose scores are capped, biased by distance or
// restricted (pkv_score_options), in its plainest form: one warp per (query
// row, query head) walks its visible keys through the block table with an
// online softmax, each lane holding four of the 128 dims.

#include <cuda_bf16.h>
#include <math.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ void load4(const void* base, int64_t row, int lane, bool fp8,
                                      float (&x)[4]) {
  if (fp8) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(base) + row * 32 + lane);
    f16x2_unpack(e4m3x2_lo_to_f16x2(w), x[0], x[1]);
    f16x2_unpack(e4m3x2_hi_to_f16x2(w), x[2], x[3]);
  } else {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(base) + row * 32 + lane);
    x[0] = bf16lo(w.x);
    x[1] = bf16hi(w.x);
    x[2] = bf16lo(w.y);
    x[3] = bf16hi(w.y);
  }
}

__global__ void __launch_bounds__(kWarps * 32) scored_rows_kernel(const ScoredRowsArgs a,
                                                                  unsigned* err) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  // (sequence, row of the chunk, head); rows past a chunk's length have nothing to do
  const int h = static_cast<int>(unit % a.Hq);
  const int64_t br = unit / a.Hq;
  const int r = static_cast<int>(br % a.max_q);
  const int64_t b = br / a.max_q;
  if (b >= a.B) return;
  const int64_t cap = static_cast<int64_t>(a.max_blocks_per_seq) * kBlockSize;
  int64_t row;   // row of q and out
  int i, last;   // position of the query, last visible key
  if (a.context_lens) {
    int ctx = a.context_lens[b];
    if (ctx < 0 || ctx > cap) {
      if (h == 0 && lane == 0) record_error(err, kErrIndex);
      ctx = static_cast<int>(cap);
    }
    row = b;
    i = last = ctx - 1;
  } else {
    const int q0 = a.cu_seqlens_q[b];
    const int Lq = a.cu_seqlens_q[b + 1] - q0;
    const int Lk = a.cu_seqlens_k[b + 1] - a.cu_seqlens_k[b];
    const int prefix = a.opt.prefix_lens ? a.opt.prefix_lens[b] : 0;
    if (q0 < 0 || Lq < 0 || q0 + static_cast<int64_t>(Lq) > a.total_q || Lk < Lq || Lq > a.max_q || Lk > a.max_k || Lk > cap || prefix < 0 ||
        prefix > Lk) {
      if (h == 0 && r == 0 && lane == 0) record_error(err, kErrIndex);
      return;
    }
    if (r >= Lq) return;
    row = static_cast<int64_t>(q0) + r;
    i = Lk - Lq + r;
    last = max(i, prefix - 1);
  }
  int first = a.opt.window > 0 ? max(0, i - a.opt.window + 1) : 0;
  if (a.opt.first_keys) first = max(first, a.opt.first_keys[row]);

  const int64_t at = row * a.Hq + h;
  const int kvh = h / (a.Hq / a.Hkv);
  const float slope = a.opt.alibi_slopes ? a.opt.alibi_slopes[h] : 0.f;
  float q[4], o[4] = {0.f, 0.f, 0.f, 0.f};
  load4(a.q, at, lane, false, q);
  float m = -INFINITY, l = 0.f;
  for (int j = first; j <= last; ++j) {
    int id = __ldg(a.block_tables + b * a.max_blocks_per_seq + j / kBlockSize);
    if (id < 0 || id >= a.num_blocks) {
      if (lane == 0) record_error(err, kErrIndex);
      id = 0;
    }
    const int64_t kv = (static_cast<int64_t>(id) * kBlockSize + j % kBlockSize) * a.Hkv + kvh;
    float k[4], v[4];
    load4(a.k_cache, kv, lane, a.fp8, k);
    load4(a.v_cache, kv, lane, a.fp8, v);
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int sh = 16; sh >= 1; sh >>= 1) s += __shfl_xor_sync(0xffffffffu, s, sh);
    s *= a.scale * a.k_scale;
    if (a.opt.softcap > 0.f) s = a.opt.softcap * tanhf(s / a.opt.softcap);
    s -= slope * fabsf(static_cast<float>(i - j));
    const float mn = fmaxf(m, s);
    const float alpha = m == -INFINITY ? 0.f : expf(m - mn);
    const float p = expf(s - mn);
    l = l * alpha + p;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = o[d] * alpha + p * v[d];
    m = mn;
  }
  const float inv = l > 0.f ? a.v_scale / l : 0.f;
  uint2 w;
  w.x = pack_bf16x2(o[0] * inv, o[1] * inv);
  w.y = pack_bf16x2(o[2] * inv, o[3] * inv);
  reinterpret_cast<uint2*>(a.out)[at * 32 + lane] = w;
  if (a.lse && lane == 0) a.lse[at] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

int launch_scored_rows(const ScoredRowsArgs& a, unsigned* err, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(a.B) * a.max_q * a.Hq;
  if (units == 0) return PKV_OK;
  const int64_t blocks = (units + kWarps - 1) / kWarps;
  if (blocks > INT32_MAX) return PKV_ERR_SHAPE;
  scored_rows_kernel<<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(a, err);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

}  // namespace pkv
