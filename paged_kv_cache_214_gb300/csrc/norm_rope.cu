// norm_rope.cu — kv_cache_store_norm_rope and its E4M3 form for sm_103a: the
// norm of every query and key head, the rotation by position, and the store of
// K and V into their pages, in one pass.
//
// Mathematics, for one 128-dim head row x of a token at position t:
//   y   = x * rsqrt(mean(x^2) + eps) * w        (skipped without a weight)
//   y'  = y with its first R dims rotated: for the pair (a, b) number i
//         (a, b) = (y[i], y[i + R/2]), or (y[2i], y[2i+1]) interleaved,
//         a' = a cos - b sin,  b' = b cos + a sin,  cos / sin = row t of the table
//   q row: bf16(y').  K row: bf16(y') or the E4M3 code of fp32(y' / k_scale).
//   V row: its bits, or the E4M3 code of fp32(v / v_scale).
// Everything up to the last rounding is fp32; each output is rounded once (an
// E4M3 key is rounded from fp32, not from its bf16 value, which would round
// twice).
//
// Bound: HBM for prompts (each row is read and written once, the table row
// once per token), launch latency for a decode step.  A row of 128 dims is
// sixteen lanes of eight dims (16-byte accesses); the sum of squares is four
// shuffles, and the partner of a half-split pair is one shuffle per dim.  A
// half-warp takes kRows rows of one token, so that the token's cos / sin stay
// in registers and kRows loads are in flight per lane.

#include <cuda_bf16.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16;                  // lanes of a row
constexpr int kUnits = kThreads / kLanes;   // half-warps of a block

struct Params {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;   // elements between tokens
  uint4* q_out;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int32_t* slots;
  const int32_t* positions;
  const float* cos_sin;     // [max_positions, R]
  const float* q_weight;
  const float* k_weight;
  unsigned* err;
  int64_t T, num_slots, units;   // units: half-warp tasks, T * groups
  int Hq, Hkv, groups, R, max_positions, interleaved;
  float eps, k_inv, v_inv;
};

// Eight consecutive bf16 of a row.
template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
  if constexpr (kVec) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | (static_cast<uint32_t>(p[2 * i + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void load8f(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8], float inv) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = e4m3x2_from_f32(x[2 * i] * inv, x[2 * i + 1] * inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <int kRows, bool kVec, bool kFp8>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const Params p) {
  const int sub = threadIdx.x / kLanes;
  const int l = threadIdx.x % kLanes;
  const int rows = p.Hq + 2 * p.Hkv;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kUnits;
  // every lane of a warp makes the same number of rounds (the shuffles need
  // both halves); a half without a unit of its own repeats the last one and
  // stores nothing
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kUnits + (sub & ~1); base < p.units;
       base += stride) {
    const int64_t mine = base + (sub & 1);
    const bool live = mine < p.units;
    const int64_t unit = live ? mine : p.units - 1;
    int64_t t;
    if (p.units <= INT32_MAX)
      t = static_cast<unsigned>(unit) / static_cast<unsigned>(p.groups);
    else
      t = unit / p.groups;
    const int row0 = static_cast<int>(unit - t * p.groups) * kRows;

    uint4 raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = min(row0 + i, rows - 1);
      const uint16_t* src = r < p.Hq ? p.q + t * p.q_stride + r * kHeadDim
                            : r < p.Hq + p.Hkv
                                ? p.k + t * p.k_stride + (r - p.Hq) * kHeadDim
                                : p.v + t * p.v_stride + (r - p.Hq - p.Hkv) * kHeadDim;
      raw[i] = load8<kVec>(src + 8 * l);
    }
    const int64_t slot = __ldg(p.slots + t);
    // the lane's factors: y' = y * c + partner * s
    float c[8], s[8];
    bool ok = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = 1.f;
      s[e] = 0.f;
    }
    const int hl = p.R / 16;   // lanes of half the rotated dims
    if (p.R > 0) {
      const int pos = __ldg(p.positions + t);
      ok = pos >= 0 && pos < p.max_positions;
      if (ok && l < 2 * hl) {
        const float* row = p.cos_sin + static_cast<int64_t>(pos) * p.R;
        if (p.interleaved) {   // pairs 4l .. 4l+3 lie within the lane
          const float4 cc = __ldg(reinterpret_cast<const float4*>(row) + l);
          const float4 ss = __ldg(reinterpret_cast<const float4*>(row + p.R / 2) + l);
          c[0] = c[1] = cc.x; c[2] = c[3] = cc.y; c[4] = c[5] = cc.z; c[6] = c[7] = cc.w;
          s[1] = ss.x; s[3] = ss.y; s[5] = ss.z; s[7] = ss.w;
          s[0] = -ss.x; s[2] = -ss.y; s[4] = -ss.z; s[6] = -ss.w;
        } else {               // pair i: dims i (lane i/8) and i + R/2 (lane i/8 + hl)
          const int i = 8 * (l < hl ? l : l - hl);
          load8f(row + i, c);
          load8f(row + p.R / 2 + i, s);
          if (l < hl) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = -s[e];
          }
        }
      }
    }
    if (live && row0 == 0 && l == 0 && (!ok || slot >= p.num_slots)) record_error(p.err, kErrIndex);
    const int partner = l < hl ? l + hl : (l < 2 * hl ? l - hl : l);

#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = row0 + i;
      const bool is_q = r < p.Hq;
      const bool is_v = r >= p.Hq + p.Hkv;
      float x[8];
      const uint32_t w4[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16lo(w4[e]);
        x[2 * e + 1] = bf16hi(w4[e]);
      }
      const float* weight = is_q ? p.q_weight : p.k_weight;
      float y[8];
      {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int sh = 8; sh >= 1; sh >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, sh);
        if (weight) {
          const float inv = rsqrtf(ss * (1.f / kHeadDim) + p.eps);
          float w[8];
          load8f(weight + 8 * l, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e] * inv * w[e];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e];
        }
      }
      float z[8];
      if (p.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = fmaf(y[e ^ 1], s[e], y[e] * c[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          z[e] = fmaf(__shfl_sync(0xffffffffu, y[e], partner, kLanes), s[e], y[e] * c[e]);
      }
      if (!live || !ok || r >= rows) continue;
      if (is_q) {
        p.q_out[(t * p.Hq + r) * (kHeadDim / 8) + l] =
            make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]), pack_bf16x2(z[4], z[5]),
                       pack_bf16x2(z[6], z[7]));
      } else if (slot >= 0 && slot < p.num_slots) {
        const int kv = is_v ? r - p.Hq - p.Hkv : r - p.Hq;
        const int64_t at = (slot * p.Hkv + kv) * kLanes + l;
        uint8_t* pool = is_v ? p.v_cache : p.k_cache;
        if constexpr (kFp8) {
          reinterpret_cast<uint2*>(pool)[at] = is_v ? e4m3x8(x, p.v_inv) : e4m3x8(z, p.k_inv);
        } else {
          reinterpret_cast<uint4*>(pool)[at] =
              is_v ? raw[i]
                   : make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]),
                                pack_bf16x2(z[4], z[5]), pack_bf16x2(z[6], z[7]));
        }
      }
    }
  }
}

template <int kRows, bool kVec, bool kFp8>
int launch(Params p, cudaStream_t stream) {
  p.groups = (p.Hq + 2 * p.Hkv + kRows - 1) / kRows;
  p.units = p.T * p.groups;
  int64_t blocks = (p.units + kUnits - 1) / kUnits;
  if (blocks > (1 << 30)) blocks = 1 << 30;
  norm_rope_kernel<kRows, kVec, kFp8>
      <<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

bool rows16(const void* p, int64_t stride) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0;
}

}  // namespace

int launch_norm_rope(const NormRopeArgs& a, unsigned* err, cudaStream_t stream) {
  if (a.T == 0) return PKV_OK;
  Params p = {};
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = static_cast<const uint16_t*>(a.k);
  p.v = static_cast<const uint16_t*>(a.v);
  p.q_stride = a.q_tok_stride;
  p.k_stride = a.k_tok_stride;
  p.v_stride = a.v_tok_stride;
  p.q_out = static_cast<uint4*>(a.q_out);
  p.k_cache = static_cast<uint8_t*>(a.k_cache);
  p.v_cache = static_cast<uint8_t*>(a.v_cache);
  p.slots = a.slot_mapping;
  p.positions = a.positions;
  p.cos_sin = a.cos_sin;
  p.q_weight = a.q_weight;
  p.k_weight = a.k_weight;
  p.err = err;
  p.T = a.T;
  p.num_slots = a.num_slots;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.R = a.rotary_dim;
  p.max_positions = a.max_positions;
  p.interleaved = a.interleaved;
  p.eps = a.eps;
  p.k_inv = a.k_inv;
  p.v_inv = a.v_inv;
  const bool vec = rows16(a.q, a.q_tok_stride) && rows16(a.k, a.k_tok_stride) &&
                   rows16(a.v, a.v_tok_stride);
  if (a.fp8) return vec ? launch<4, true, true>(p, stream) : launch<4, false, true>(p, stream);
  return vec ? launch<4, true, false>(p, stream) : launch<4, false, false>(p, stream);
}

}  // namespace pkv
