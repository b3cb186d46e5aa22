// prefill_scored.cu — paged (chunked) prefill whose scores are capped or biased
// by distance and whose rows see an interval of keys (pkv_score_options: a
// window, documents, a two-way prefix), on the tensor-core kernel of
// prefill_kernel.cuh.

#include "prefill_kernel.cuh"

namespace pkv {

int set_wait_hook_prefill_scored(unsigned long long limit_ns, int withhold_plus1) {
  const WaitHook h{limit_ns, withhold_plus1, 0};
  return cudaMemcpyToSymbol(g_wait_hook, &h, sizeof h) == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

namespace {

template <bool kCap, bool kBias>
int launch_form(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
                const PrefillParams& prm, cudaStream_t stream) {
  if (!set_smem_attr<kScored, kCap, kBias>()) return PKV_ERR_LAUNCH;
  paged_prefill_kernel<kScored, kCap, kBias>
      <<<grid_for(prm.n_items), kThreads, kSmemBytes, stream>>>(qm, km, vm, prm);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

}  // namespace

int launch_prefill_scored(const PrefillArgs& a, int64_t total_q, const pkv_score_options& opt,
                          unsigned* err, cudaStream_t stream) {
  if (a.B == 0 || a.max_seqlen_q == 0 || total_q == 0) return PKV_OK;
  CUtensorMap qm, km, vm;
  const int64_t slots = a.num_blocks * kBlockSize;
  // q holds exactly total_q rows: a ragged tile reads its neighbour's rows, or
  // zeros past the end, and stores none of them
  if (!encode_pool_map(&qm, a.q, total_q, a.Hq, kM) ||
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
  prm.total_q = total_q;
  prm.window = opt.window;
  prm.slopes = opt.alibi_slopes;
  prm.first_keys = opt.first_keys;
  prm.prefix_lens = opt.prefix_lens;
  if (opt.softcap > 0.f) {
    prm.cap_log2 = opt.softcap * 1.4426950408889634f;
    prm.cap_x = a.scale / opt.softcap;
    prm.scale_log2 = a.scale * 2.8853900817779268f / opt.softcap;
  }
  const int64_t items = static_cast<int64_t>(prm.n_qt) * a.B * a.Hq;
  if (items > INT32_MAX) return PKV_ERR_SHAPE;
  prm.n_items = static_cast<int>(items);
  const bool cap = opt.softcap > 0.f, bias = opt.alibi_slopes != nullptr;
  if (cap)
    return bias ? launch_form<true, true>(qm, km, vm, prm, stream)
                : launch_form<true, false>(qm, km, vm, prm, stream);
  return bias ? launch_form<false, true>(qm, km, vm, prm, stream)
              : launch_form<false, false>(qm, km, vm, prm, stream);
}

}  // namespace pkv
