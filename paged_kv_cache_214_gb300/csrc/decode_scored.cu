// decode_scored.cu — paged decode attention whose scores are capped or biased by
// distance and whose keys may start at a window's or a document's first one
// (pkv_score_options), on the split-K kernel of decode_kernel.cuh.
//
// What the options add to that kernel.  Per score: the cap, two special-function
// operations (modify_scores), and one multiply-add of the distance; both work
// in log2 units.  Per block: the first key comes from the context length, so
// with a window or documents a block's page ids are read after it (one more
// dependent load).  Ranges start at the first key's block and the ring at its
// 64-token tile, so a window costs the bytes of the window, and pages behind it
// are never read.  The grid covers the blocks a window can touch, not the
// table's.  Bound by HBM as the plain decode is; a capped score's arithmetic hides
// under the copies.  Measured on 64 sequences of 512 to 4096 tokens, 16 / 8 heads: a
// batch of 524 MB capped 84.9 us against 84.4 plain (91% of the measured copy rate),
// one of 594 MB capped 96.4 (91%).  A window of 1000, 64 sequences, 32 / 8 heads: 45
// us (259 MB, 85%).  E4M3, 8 sequences of 32768 to 131072 tokens, capped: 198 us
// (1147 MB, 85%).

#include "decode_kernel.cuh"

namespace pkv {

int set_wait_hook_decode_scored(unsigned long long limit_ns, int withhold_plus1) {
  const WaitHook h{limit_ns, withhold_plus1, 0};
  return cudaMemcpyToSymbol(g_wait_hook, &h, sizeof h) == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

int plan_decode_scored(int B, int Hq, int Hkv, int max_blocks_per_seq, int window, int num_splits,
                       int fp8, int sm_count, DecodePlan* plan) {
  if (B < 0 || window < 0 || max_blocks_per_seq < 0) return PKV_ERR_ARG;
  // token positions are 32-bit in the kernel, those of empty ranges past the last too
  if (max_blocks_per_seq > INT32_MAX / kBlockSize - kMaxSplits * kMaxSplitBlocks)
    return PKV_ERR_SHAPE;
  int blocks = max_blocks_per_seq;
  const bool bounded = window > 0 && window <= static_cast<int64_t>(blocks) * kBlockSize;
  if (bounded) {
    // the window's tokens and up to a block before them
    const int touched = (window + 2 * kBlockSize - 2) / kBlockSize;
    if (touched < blocks) blocks = touched;
  }
  const int st = plan_decode(B, Hq, Hkv, blocks, num_splits, sm_count, 0, plan);
  if (st) return st;
  const int64_t row_units = static_cast<int64_t>(Hkv) * plan->head_groups;   // of a sequence
  // the launch grid: (splits, kv heads x head groups, sequences)
  if (B > 65535 || row_units > 65535) return PKV_ERR_SHAPE;
  if (!bounded || num_splits > 0 || B == 0) return PKV_OK;

  // Every context has about the window's tokens, so that equal ranges of 64-token
  // tiles are balanced, and few of them do: ranges to merge cost about 8 us more
  // than one (partials written, a ticket, partials read), which is a chain of 11
  // tiles (0.7 us a tile and block, half that with two consumer groups) unless the
  // copy bandwidth is the limit (5 ns a tile of every block, E4M3 3 ns).  One range
  // while that chain is the shorter, else ranges for one wave of two blocks an SM.
  // Measured, one range against three: 64 sequences of 8 kv heads and a window of
  // 1000 tokens 50 and 62 us; 16 sequences and 4096 tokens over E4M3 46 and 34 us.
  const int64_t units = row_units * B;
  const int64_t sms = sm_count > 0 ? sm_count : 148;
  const int64_t tiles = (window - 1) / kTile + 2;   // that the window can touch
  const bool two_groups = !fp8 && units <= sms;
  const int64_t chain_ns = two_groups ? 350 : 700, copy_ns = fp8 ? 3 : 5;
  int64_t S = 1;
  if (units < 2 * sms && tiles * (chain_ns - copy_ns * units) > 8000)
    S = (2 * sms + units - 1) / units;
  if (S > tiles) S = tiles;
  constexpr int kMostTiles = (kMaxSplitBlocks - 2) * (kBlockSize / kTile);   // block ids of a range
  int per = static_cast<int>((tiles + S - 1) / S);
  if (per > kMostTiles) per = kMostTiles;
  // (a range of whole blocks would begin at a block, not at the window's tile)
  if (per % (kBlockSize / kTile) == 0) per = per < kMostTiles ? per + 1 : per - 1;
  S = (tiles + per - 1) / per;
  if (S > kMaxSplits) return PKV_OK;   // plan_decode's ranges are longer
  if (S > 1 && units > kMaxCounters) return PKV_ERR_SHAPE;
  plan->split_tokens = per * kTile;
  plan->num_splits = static_cast<int>(S);
  plan->consumer_groups = S == 1 && two_groups ? 2 : 1;
  plan->workspace_bytes = S > 1 ? decode_partials_bytes(B, Hq, plan->num_splits) : 0;
  return PKV_OK;
}

namespace {

template <int G>
int launch_form(const DecodeArgs& a, const DecodePlan& plan, const DecodeParams& prm,
                const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t stream) {
  // the forms and the rules between them are the plain decode's (launch_decode)
  if (a.fp8)
    return plan.split_tokens >= 8 * kBlockSize
               ? launch_g<G, false, true, true, 1, true>(a, plan, prm, km, vm, stream)
               : launch_g<G, false, true, false, 1, true>(a, plan, prm, km, vm, stream);
  if (plan.consumer_groups == 2)
    return launch_g<G, false, false, true, 2, true>(a, plan, prm, km, vm, stream);
  if (plan.split_tokens < kBlockSize)
    return launch_g<G, false, false, false, 1, true>(a, plan, prm, km, vm, stream);
  return launch_g<G, false, false, true, 1, true>(a, plan, prm, km, vm, stream);
}

}  // namespace

int launch_decode_scored(const DecodeArgs& a, const pkv_score_options& opt, const DecodePlan& plan,
                         unsigned* err, cudaStream_t stream) {
  CUtensorMap km, vm;
  if (!decode_maps(a, &km, &vm)) return PKV_ERR_ARG;
  DecodeParams prm = decode_params(a, plan, err);
  if (opt.softcap > 0.f) {
    prm.cap_log2 = opt.softcap * 1.4426950408889634f;
    if (prm.cap_log2 <= kWideCap) prm.scale_log2 = a.scale * 2.8853900817779268f / opt.softcap;
  }
  prm.window = opt.window;
  prm.slopes = opt.alibi_slopes;
  prm.first_keys = opt.first_keys;
  switch (plan.heads_per_cta) {
    case 8: return launch_form<8>(a, plan, prm, km, vm, stream);
    case 4: return launch_form<4>(a, plan, prm, km, vm, stream);
    case 2: return launch_form<2>(a, plan, prm, km, vm, stream);
    default: return launch_form<1>(a, plan, prm, km, vm, stream);
  }
}

}  // namespace pkv
