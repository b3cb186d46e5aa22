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
// once per token), launch latency for a decode step.
//
// A row is sixteen lanes of eight dims; a lane holds both dims of its four pairs
// (two 8-byte pieces R/2 apart, or 16 contiguous bytes interleaved), so that the
// rotation needs no exchange and the sum of squares is the only one.  A warp takes
// 2 kRows rows of one token and of one tensor, kRows to a half, with the weight
// folded into the token's cos / sin once for its rows; the norm's factor, common
// to the row, multiplies last.  Four rows' sums of squares are reduced together
// (lanes trade rows while they add: nine shuffles and one rsqrt instead of sixteen
// and four).  A warp keeps its rows' place and walks over tokens, so that indexes
// and weights are worked out once.  Values are a plain copy.
// Instructions were the limit on the way here (8192 tokens of 32 / 8 heads, 206
// MB): 60 us with rows of contiguous dims, partners exchanged by shuffles and all
// three tensors in one warp (93 instructions a row), 45 us in this layout with one
// task a warp and each row reduced by itself, 38 us now (5.4 TB/s, 80% of the
// measured copy; 36 to 37 in the kernel alone).  Loading the next token's rows ahead
// (more registers) took 42.  Into E4M3 pages (189 MB) 38 us too.

#include <cuda_bf16.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16;   // lanes of a row

struct Params {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;   // elements between tokens
  uint16_t* q_out;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int32_t* slots;
  const int32_t* positions;
  const float* cos_sin;     // [max_positions, R]
  const float* q_weight;
  const float* k_weight;
  unsigned* err;
  int64_t num_slots, T;
  int Hq, Hkv, R, max_positions;
  int q_groups, kv_groups, groups;   // warps of a token: of its queries, keys (values), all
  float eps, k_inv, v_inv;
};

// Four consecutive bf16 of a row.
template <bool kVec>
__device__ __forceinline__ uint2 load4(const uint16_t* p) {
  if constexpr (kVec) return *reinterpret_cast<const uint2*>(p);
  return make_uint2(p[0] | (static_cast<uint32_t>(p[1]) << 16),
                    p[2] | (static_cast<uint32_t>(p[3]) << 16));
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2_from_f32(a, b) | (static_cast<uint32_t>(e4m3x2_from_f32(c, d)) << 16);
}

// kInter: interleaved pairs.  A lane's eight dims are pieces A and B of four; a
// pair is (A[i], B[i]), or, interleaved, two neighbours of A or of B.
template <int kRows, bool kVec, bool kFp8, bool kInter>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_kernel(const Params p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int half = (threadIdx.x >> 4) & 1;
  const int l = threadIdx.x % kLanes;
  // warps of the grid in sets of p.groups; a warp's place in its set is its rows
  const int warp = static_cast<int>(blockIdx.x) * (kThreads / 32) + static_cast<int>(threadIdx.x >> 5);
  const int sets = static_cast<int>(gridDim.x) * (kThreads / 32) / p.groups;
  const int set = warp / p.groups;
  if (set >= sets) return;
  int grp = warp - set * p.groups;
  const bool first = grp == 0;
  // the warp's tensor: 0 queries, 1 keys, 2 values
  const int which = grp < p.q_groups ? 0 : grp < p.q_groups + p.kv_groups ? 1 : 2;
  grp -= which == 0 ? 0 : which == 1 ? p.q_groups : p.q_groups + p.kv_groups;
  const int heads = which == 0 ? p.Hq : p.Hkv;
  const int row0 = grp * 2 * kRows + half;   // this half's rows: row0, row0 + 2, ...
  // The lane's pieces.  Lanes below R/8 hold the rotated dims, the others two
  // pieces of the dims past R (half-split) or eight of them (interleaved).
  const bool turns = 8 * l < p.R;
  int oa = 8 * l, ob = oa + 4;
  if (!kInter && which != 2) {
    oa = turns ? 4 * l : p.R + 4 * (l - p.R / 8);
    ob = oa + (turns ? p.R / 2 : (kHeadDim - p.R) / 2);
  }
  const float* weight = which == 0 ? p.q_weight : p.k_weight;
  float4 wa = make_float4(1.f, 1.f, 1.f, 1.f), wb = wa;
  if (weight && which != 2) {
    wa = *reinterpret_cast<const float4*>(weight + oa);
    wb = *reinterpret_cast<const float4*>(weight + ob);
  }
  const uint16_t* const base = (which == 0 ? p.q : which == 1 ? p.k : p.v) +
                               static_cast<int64_t>(row0) * kHeadDim;
  const int64_t tok_stride = which == 0 ? p.q_stride : which == 1 ? p.k_stride : p.v_stride;
  for (int64_t t = set; t < p.T; t += sets) {
    // Everything that depends on nothing but the task is loaded first, so that
    // one latency covers the rows, the slot and the position.
    const int64_t slot = p.slots[t];
    int pos = 0;
    if (p.R > 0) pos = p.positions[t];
    const uint16_t* src = base + t * tok_stride;
    uint2 a[kRows], b[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      a[i] = b[i] = make_uint2(0u, 0u);
      if (row0 + 2 * i >= heads) continue;
      const uint16_t* row = src + 2 * i * kHeadDim;
      if (kVec && (kInter || which == 2)) {
        const uint4 x = *reinterpret_cast<const uint4*>(row + oa);
        a[i] = make_uint2(x.x, x.y);
        b[i] = make_uint2(x.z, x.w);
      } else {
        a[i] = load4<kVec>(row + oa);
        b[i] = load4<kVec>(row + ob);
      }
    }
    const bool stored = slot >= 0 && slot < p.num_slots;
    const bool placed = p.R == 0 || (pos >= 0 && pos < p.max_positions);
    if (first && threadIdx.x % 32 == 0 && (!placed || slot >= p.num_slots))
      record_error(p.err, kErrIndex);
    if (!placed || (which != 0 && !stored)) continue;   // (the same for the whole warp)

    if (which == 2) {   // values: a copy, 16 bytes a lane
      const int64_t at = (slot * p.Hkv + row0) * kLanes + l;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (row0 + 2 * i >= heads) continue;
        if constexpr (kFp8) {
          const float s = p.v_inv;
          reinterpret_cast<uint2*>(p.v_cache)[at + 2 * i * kLanes] =
              make_uint2(e4m3x4(bf16lo(a[i].x) * s, bf16hi(a[i].x) * s, bf16lo(a[i].y) * s,
                                bf16hi(a[i].y) * s),
                         e4m3x4(bf16lo(b[i].x) * s, bf16hi(b[i].x) * s, bf16lo(b[i].y) * s,
                                bf16hi(b[i].y) * s));
        } else {
          reinterpret_cast<uint4*>(p.v_cache)[at + 2 * i * kLanes] =
              make_uint4(a[i].x, a[i].y, b[i].x, b[i].y);
        }
      }
      continue;
    }
    // the lane's place in its first output row
    uint16_t* const dst =
        which == 0 ? p.q_out + (t * p.Hq + row0) * kHeadDim
                   : reinterpret_cast<uint16_t*>(p.k_cache) + (slot * p.Hkv + row0) * kHeadDim;
    uint8_t* const dst8 = p.k_cache + (slot * p.Hkv + row0) * kHeadDim;
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turns) {   // pairs 4l .. 4l + 3
      const float4* row = reinterpret_cast<const float4*>(p.cos_sin + static_cast<int64_t>(pos) * p.R);
      c = row[l];
      s = row[p.R / 8 + l];
    }
    // A' = A fa + B' ga, B' = B fb + A ga' as pairs of floats: own factor f, the
    // partner's factor g (weight of the partner, signed sine)
    f32x2 fa[2], fb[2], ga[2], gb[2];
    if constexpr (kInter) {   // dims (A0 A1) (A2 A3) (B0 B1) (B2 B3) are the pairs
      fa[0] = pack2(wa.x * c.x, wa.y * c.x);
      fa[1] = pack2(wa.z * c.y, wa.w * c.y);
      fb[0] = pack2(wb.x * c.z, wb.y * c.z);
      fb[1] = pack2(wb.z * c.w, wb.w * c.w);
      ga[0] = pack2(-wa.y * s.x, wa.x * s.x);
      ga[1] = pack2(-wa.w * s.y, wa.z * s.y);
      gb[0] = pack2(-wb.y * s.z, wb.x * s.z);
      gb[1] = pack2(-wb.w * s.w, wb.z * s.w);
    } else {
      fa[0] = pack2(wa.x * c.x, wa.y * c.y);
      fa[1] = pack2(wa.z * c.z, wa.w * c.w);
      fb[0] = pack2(wb.x * c.x, wb.y * c.y);
      fb[1] = pack2(wb.z * c.z, wb.w * c.w);
      ga[0] = pack2(-wb.x * s.x, -wb.y * s.y);
      ga[1] = pack2(-wb.z * s.z, -wb.w * s.w);
      gb[0] = pack2(wa.x * s.x, wa.y * s.y);
      gb[1] = pack2(wa.z * s.z, wa.w * s.w);
    }
    // the norm's factor of each row
    float inv[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) inv[i] = 1.f;
    if (weight) {
      float ss[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const f32x2 a0 = pack2(bf16lo(a[i].x), bf16hi(a[i].x)), a1 = pack2(bf16lo(a[i].y), bf16hi(a[i].y));
        const f32x2 b0 = pack2(bf16lo(b[i].x), bf16hi(b[i].x)), b1 = pack2(bf16lo(b[i].y), bf16hi(b[i].y));
        const f32x2 ss2 = add2(fma2(a0, a0, mul2(b0, b0)), fma2(a1, a1, mul2(b1, b1)));
        ss[i] = lo2(ss2) + hi2(ss2);
      }
      auto from = [](float v, int mask) { return __shfl_xor_sync(0xffffffffu, v, mask); };
      if constexpr (kRows == 4) {
        // lanes with bit 3 go on with rows 2 and 3, then lanes with bit 2 with the
        // second of two: lane group (l >> 2) ends with the sum of row l >> 2
        const bool h8 = l & 8, h4 = l & 4;
        const float s0 = (h8 ? ss[2] : ss[0]) + from(h8 ? ss[0] : ss[2], 8);
        const float s1 = (h8 ? ss[3] : ss[1]) + from(h8 ? ss[1] : ss[3], 8);
        float s = (h4 ? s1 : s0) + from(h4 ? s0 : s1, 4);
        s += from(s, 2);
        s += from(s, 1);
        s = rsqrtf(s * (1.f / kHeadDim) + p.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i) inv[i] = __shfl_sync(0xffffffffu, s, 4 * i, kLanes);
      } else {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          float s = ss[i];
#pragma unroll
          for (int sh = 8; sh >= 1; sh >>= 1) s += from(s, sh);
          inv[i] = rsqrtf(s * (1.f / kHeadDim) + p.eps);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const f32x2 a0 = pack2(bf16lo(a[i].x), bf16hi(a[i].x)), a1 = pack2(bf16lo(a[i].y), bf16hi(a[i].y));
      const f32x2 b0 = pack2(bf16lo(b[i].x), bf16hi(b[i].x)), b1 = pack2(bf16lo(b[i].y), bf16hi(b[i].y));
      const f32x2 inv2 = pack2(inv[i], inv[i]);
      f32x2 za0, za1, zb0, zb1;
      if constexpr (kInter) {
        za0 = fma2(pack2(hi2(a0), lo2(a0)), ga[0], mul2(a0, fa[0]));
        za1 = fma2(pack2(hi2(a1), lo2(a1)), ga[1], mul2(a1, fa[1]));
        zb0 = fma2(pack2(hi2(b0), lo2(b0)), gb[0], mul2(b0, fb[0]));
        zb1 = fma2(pack2(hi2(b1), lo2(b1)), gb[1], mul2(b1, fb[1]));
      } else {
        za0 = fma2(b0, ga[0], mul2(a0, fa[0]));
        za1 = fma2(b1, ga[1], mul2(a1, fa[1]));
        zb0 = fma2(a0, gb[0], mul2(b0, fb[0]));
        zb1 = fma2(a1, gb[1], mul2(b1, fb[1]));
      }
      if (p.R < kHeadDim && !turns) {   // 0 * partner would pass its infinities on
        za0 = mul2(a0, fa[0]);
        za1 = mul2(a1, fa[1]);
        zb0 = mul2(b0, fb[0]);
        zb1 = mul2(b1, fb[1]);
      }
      za0 = mul2(za0, inv2);
      za1 = mul2(za1, inv2);
      zb0 = mul2(zb0, inv2);
      zb1 = mul2(zb1, inv2);
      if (row0 + 2 * i >= heads) continue;
      if (kFp8 && which == 1) {
        const float k = p.k_inv;
        uint8_t* const to = dst8 + 2 * i * kHeadDim;
        const uint32_t ca = e4m3x4(lo2(za0) * k, hi2(za0) * k, lo2(za1) * k, hi2(za1) * k);
        const uint32_t cb = e4m3x4(lo2(zb0) * k, hi2(zb0) * k, lo2(zb1) * k, hi2(zb1) * k);
        if constexpr (kInter) {
          *reinterpret_cast<uint2*>(to + oa) = make_uint2(ca, cb);
        } else {
          *reinterpret_cast<uint32_t*>(to + oa) = ca;
          *reinterpret_cast<uint32_t*>(to + ob) = cb;
        }
      } else {
        uint16_t* const to = dst + 2 * i * kHeadDim;
        const uint2 ya = make_uint2(pack_bf16x2(lo2(za0), hi2(za0)), pack_bf16x2(lo2(za1), hi2(za1)));
        const uint2 yb = make_uint2(pack_bf16x2(lo2(zb0), hi2(zb0)), pack_bf16x2(lo2(zb1), hi2(zb1)));
        if constexpr (kInter) {
          *reinterpret_cast<uint4*>(to + oa) = make_uint4(ya.x, ya.y, yb.x, yb.y);
        } else {
          *reinterpret_cast<uint2*>(to + oa) = ya;
          *reinterpret_cast<uint2*>(to + ob) = yb;
        }
      }
    }
  }
}

template <int kRows, bool kVec, bool kFp8, bool kInter>
int launch(Params p, int64_t T, cudaStream_t stream) {
  p.q_groups = (p.Hq + 2 * kRows - 1) / (2 * kRows);
  p.kv_groups = (p.Hkv + 2 * kRows - 1) / (2 * kRows);
  p.groups = p.q_groups + 2 * p.kv_groups;
  p.T = T;
  // at most 24 warps an SM (three blocks, up to 85 registers a thread; four blocks of
  // 64 registers measured the same), at least one set
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  constexpr int kWarps = kThreads / 32;
  const int64_t most = static_cast<int64_t>(sms) * 3;
  int64_t blocks = T < most * kWarps ? (T * p.groups + kWarps - 1) / kWarps : most;
  if (blocks > most) blocks = most;
  const int64_t least = (p.groups + kWarps - 1) / kWarps;
  if (blocks < least) blocks = least;
  // may be scheduled while the stream's previous kernel finishes; it waits
  // (griddepcontrol.wait) before its first global read
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, norm_rope_kernel<kRows, kVec, kFp8, kInter>, p) != cudaSuccess)
    return PKV_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

template <int kRows, bool kVec, bool kFp8>
int launch_pairs(const Params& p, int64_t T, bool interleaved, cudaStream_t stream) {
  return interleaved ? launch<kRows, kVec, kFp8, true>(p, T, stream)
                     : launch<kRows, kVec, kFp8, false>(p, T, stream);
}

template <int kRows>
int launch_rows(const Params& p, const NormRopeArgs& a, bool vec, cudaStream_t stream) {
  const bool inter = a.interleaved != 0;
  if (a.fp8)
    return vec ? launch_pairs<kRows, true, true>(p, a.T, inter, stream)
               : launch_pairs<kRows, false, true>(p, a.T, inter, stream);
  return vec ? launch_pairs<kRows, true, false>(p, a.T, inter, stream)
             : launch_pairs<kRows, false, false>(p, a.T, inter, stream);
}

bool rows16(const void* p, int64_t stride) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0;
}

// Row slots of a token when a warp takes 2 k rows of one tensor.
int64_t row_slots(int Hq, int Hkv, int k) {
  const auto up = [&](int h) { return static_cast<int64_t>((h + 2 * k - 1) / (2 * k)) * 2 * k; };
  return up(Hq) + 2 * up(Hkv);
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
  p.q_out = static_cast<uint16_t*>(a.q_out);
  p.k_cache = static_cast<uint8_t*>(a.k_cache);
  p.v_cache = static_cast<uint8_t*>(a.v_cache);
  p.slots = a.slot_mapping;
  p.positions = a.positions;
  p.cos_sin = a.cos_sin;
  p.q_weight = a.q_weight;
  p.k_weight = a.k_weight;
  p.err = err;
  p.num_slots = a.num_slots;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.R = a.rotary_dim;
  p.max_positions = a.max_positions;
  p.eps = a.eps;
  p.k_inv = a.k_inv;
  p.v_inv = a.v_inv;
  const bool vec = rows16(a.q, a.q_tok_stride) && rows16(a.k, a.k_tok_stride) &&
                   rows16(a.v, a.v_tok_stride);
  // Rows a half-warp takes: as many as share the token's factors without leaving
  // more than an eighth of the row slots empty, but one while the warps of all
  // tokens would not fill the SMs four times over.
  const int64_t rows = static_cast<int64_t>(a.Hq) + 2 * a.Hkv;
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  int k = 1;
  if (a.T * rows >= static_cast<int64_t>(sms) * 4 * 16) {
    k = 4;
    while (k > 1 && row_slots(a.Hq, a.Hkv, k) * 8 > rows * 9) k /= 2;
  }
  if (k == 4) return launch_rows<4>(p, a, vec, stream);
  if (k == 2) return launch_rows<2>(p, a, vec, stream);
  return launch_rows<1>(p, a, vec, stream);
}

}  // namespace pkv
