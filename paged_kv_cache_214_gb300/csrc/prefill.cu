// prefill.cu — launches of the tensor-core attention kernel (prefill_kernel.cuh)
// for causal and chunked prefill, the shared-prefix pass of a decode batch and
// the verify step of speculative decoding.

#include "prefill_kernel.cuh"

namespace pkv {

int set_wait_hook_prefill(unsigned long long limit_ns, int withhold_plus1) {
  const WaitHook h{limit_ns, withhold_plus1, 0};
  return cudaMemcpyToSymbol(g_wait_hook, &h, sizeof h) == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

int prefix_rows_per_tile(int g) { return (g >= 1 && g <= kM) ? (kM / g) * g : 0; }

int launch_prefill(const PrefillArgs& a, unsigned* err, cudaStream_t stream) {
  if (a.B == 0 || a.max_seqlen_q == 0) return PKV_OK;
  // The query map spans B * max_seqlen_q rows, at least the real sum of Lq.
  // Only full 128-row tiles go through it, and a full tile never leaves its
  // sequence, so every row it reads exists.
  const int64_t q_rows = static_cast<int64_t>(a.B) * a.max_seqlen_q;
  if (q_rows > INT32_MAX) return PKV_ERR_SHAPE;
  CUtensorMap qm, km, vm;
  const int64_t slots = a.num_blocks * kBlockSize;
  if (!encode_pool_map(&qm, a.q, q_rows, a.Hq, kM) ||
      !encode_pool_map(&km, a.k_cache, slots, a.Hkv, kN) ||
      !encode_pool_map(&vm, a.v_cache, slots, a.Hkv, kN))
    return PKV_ERR_ARG;
  PrefillParams prm = {};
  prm.out = static_cast<__nv_bfloat16*>(a.out);
  prm.lse = a.lse;
  prm.q = static_cast<const __nv_bfloat16*>(a.q);
  prm.block_tables = a.block_tables;
  prm.cu_q = a.cu_seqlens_q;
  prm.cu_k = a.cu_seqlens_k;
  prm.err = err;
  prm.B = a.B;
  prm.Hq = a.Hq;
  prm.Hkv = a.Hkv;
  prm.maxblk = a.max_blocks_per_seq;
  prm.max_q = a.max_seqlen_q;
  prm.max_k = a.max_seqlen_k;
  prm.n_qt = (a.max_seqlen_q + kM - 1) / kM;
  prm.num_blocks = a.num_blocks;
  prm.scale_log2 = a.scale * 1.4426950408889634f;
  const int64_t items = static_cast<int64_t>(prm.n_qt) * a.B * a.Hq;
  if (items > INT32_MAX) return PKV_ERR_SHAPE;
  prm.n_items = static_cast<int>(items);
  if (!set_smem_attr<kCausal>()) return PKV_ERR_LAUNCH;
  paged_prefill_kernel<kCausal><<<grid_for(prm.n_items), kThreads, kSmemBytes, stream>>>(
      qm, km, vm, prm);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

int launch_prefix_attention(const PrefixArgs& a, unsigned* err, cudaStream_t stream) {
  if (a.B == 0 || a.prefix_tokens == 0) return PKV_OK;
  const int g = a.Hq / a.Hkv;
  const int rpt = prefix_rows_per_tile(g);
  if (rpt == 0) return PKV_ERR_SHAPE;
  CUtensorMap qm, km, vm;
  const int64_t slots = a.num_blocks * kBlockSize;
  // q [B, Hq, 128]: a box is 64 dims x the g heads of one kv head x rpt/g tokens
  if (!encode_pool_map(&qm, a.q, a.B, a.Hq, rpt / g, g) ||
      !encode_pool_map(&km, a.k_cache, slots, a.Hkv, kN) ||
      !encode_pool_map(&vm, a.v_cache, slots, a.Hkv, kN))
    return PKV_ERR_ARG;
  PrefillParams prm = {};
  prm.part_o = a.part_o;
  prm.part_lse = a.part_lse;
  prm.prefix_tokens = a.prefix_tokens;
  prm.prefix_kt_per = a.kt_per;
  prm.splits = a.splits;
  prm.rows_per_tile = rpt;
  prm.n_rt = (a.B * g + rpt - 1) / rpt;
  prm.q = static_cast<const __nv_bfloat16*>(a.q);
  prm.block_tables = a.block_tables;
  prm.err = err;
  prm.B = a.B;
  prm.Hq = a.Hq;
  prm.Hkv = a.Hkv;
  prm.num_blocks = a.num_blocks;
  prm.scale_log2 = a.scale * 1.4426950408889634f;
  const int64_t items = static_cast<int64_t>(prm.n_rt) * a.Hkv * a.splits;
  if (items > INT32_MAX) return PKV_ERR_SHAPE;
  prm.n_items = static_cast<int>(items);
  if (!set_smem_attr<kPrefixPass>()) return PKV_ERR_LAUNCH;
  paged_prefill_kernel<kPrefixPass><<<grid_for(prm.n_items), kThreads, kSmemBytes, stream>>>(
      qm, km, vm, prm);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

int verify_rows_fit(int g, int q_len) { return g >= 1 && q_len >= 1 && g * q_len <= kM; }

int launch_verify(const VerifyArgs& a, unsigned* err, cudaStream_t stream) {
  if (a.B == 0) return PKV_OK;
  const int g = a.Hq / a.Hkv;
  if (!verify_rows_fit(g, a.q_len)) return PKV_ERR_SHAPE;
  const int64_t q_rows = static_cast<int64_t>(a.B) * a.q_len;
  if (q_rows > INT32_MAX) return PKV_ERR_SHAPE;
  CUtensorMap qm, km, vm;
  const int64_t slots = a.num_blocks * kBlockSize;
  // q [B*q_len, Hq, 128]: a box is 64 dims x the g heads of one kv head x q_len positions
  if (!encode_pool_map(&qm, a.q, q_rows, a.Hq, a.q_len, g) ||
      !encode_pool_map(&km, a.k_cache, slots, a.Hkv, kN) ||
      !encode_pool_map(&vm, a.v_cache, slots, a.Hkv, kN))
    return PKV_ERR_ARG;
  PrefillParams prm = {};
  prm.out = static_cast<__nv_bfloat16*>(a.out);
  prm.lse = a.lse;
  prm.q = static_cast<const __nv_bfloat16*>(a.q);
  prm.block_tables = a.block_tables;
  prm.ctx = a.context_lens;
  prm.err = err;
  prm.B = a.B;
  prm.Hq = a.Hq;
  prm.Hkv = a.Hkv;
  prm.maxblk = a.max_blocks_per_seq;
  prm.q_len = a.q_len;
  prm.rows_per_tile = g * a.q_len;
  prm.num_blocks = a.num_blocks;
  prm.scale_log2 = a.scale * 1.4426950408889634f;
  const int64_t items = static_cast<int64_t>(a.B) * a.Hkv;
  if (items > INT32_MAX) return PKV_ERR_SHAPE;
  prm.n_items = static_cast<int>(items);
  if (!set_smem_attr<kVerify>()) return PKV_ERR_LAUNCH;
  paged_prefill_kernel<kVerify><<<grid_for(prm.n_items), kThreads, kSmemBytes, stream>>>(
      qm, km, vm, prm);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

}  // namespace pkv
