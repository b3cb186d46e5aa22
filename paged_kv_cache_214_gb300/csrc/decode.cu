// decode.cu — paged decode attention (split-K flash-decoding) for sm_103a: the
// split plan, and the choice of the kernel form (decode_kernel.cuh) for plain,
// multi-query and shared-prefix decode.

#include "decode_kernel.cuh"

namespace pkv {

int set_wait_hook_decode(unsigned long long limit_ns, int withhold_plus1) {
  const WaitHook h{limit_ns, withhold_plus1, 0};
  return cudaMemcpyToSymbol(g_wait_hook, &h, sizeof h) == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

size_t decode_partials_bytes(int B, int Hq, int num_splits) {
  const size_t rows = static_cast<size_t>(B) * Hq * num_splits;
  return kCounterRegion + align_up(rows * kHeadDim * sizeof(float), 256) +
         align_up(rows * sizeof(float), 256);
}

int plan_decode(int B, int Hq, int Hkv, int max_blocks_per_seq, int num_splits,
                int sm_count, int prefix_blocks, DecodePlan* plan) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || max_blocks_per_seq < 0 || prefix_blocks < 0 ||
      prefix_blocks > max_blocks_per_seq)
    return PKV_ERR_ARG;
  if (Hq % Hkv) return PKV_ERR_SHAPE;
  const int g = Hq / Hkv;
  const int G = (g % 8 == 0) ? 8 : (g % 4 == 0) ? 4 : (g % 2 == 0) ? 2 : 1;
  plan->heads_per_cta = G;
  plan->head_groups = g / G;
  plan->consumer_groups = 1;
  // One kv head per block.  (Reading two kv heads per block as 512-byte
  // chunks per token measured 2% slower on GB300 on the batch-64 decode and
  // slower on short contexts.)
  const int kv_groups = Hkv;
  const int rest = max_blocks_per_seq - prefix_blocks;
  const int maxblk = rest > 0 ? rest : 1;
  const int sms = sm_count > 0 ? sm_count : 148;
  const int64_t seq_units = static_cast<int64_t>(B) * kv_groups * plan->head_groups;
  int split_blocks;
  bool small = false;
  if (num_splits > 0) {
    split_blocks = (maxblk + num_splits - 1) / num_splits;
  } else {
    // Enough (sequence, head group, split) units for about eight waves of two
    // blocks per SM if every context were full length; whole blocks per split.
    const int64_t units = seq_units * maxblk;
    const int64_t target = static_cast<int64_t>(sms) * 2 * 8;
    split_blocks = static_cast<int>((units + target - 1) / target);
    // A batch whose one-block splits would not even fill one wave of one
    // block per SM splits into 64-token tiles instead (a launch-latency
    // bound step: more blocks, each with a shorter chain of copies).
    small = units < sms;
    if (split_blocks < 2) split_blocks = maxblk < 2 ? maxblk : 2;
  }
  if (split_blocks < 1) split_blocks = 1;
  if (split_blocks > kMaxSplitBlocks) split_blocks = kMaxSplitBlocks;
  int S = (maxblk + split_blocks - 1) / split_blocks;
  if (S > kMaxSplits) return PKV_ERR_SHAPE;
  // re-balance so that the splits are as even as possible
  split_blocks = (maxblk + S - 1) / S;
  plan->split_tokens = split_blocks * kBlockSize;
  if (small && maxblk <= 3) {
    // Contexts of at most three blocks: one split per sequence, no merge.  The
    // merge of split partials (store, ticket, reads) costs about as much as
    // eight or nine 64-token tiles of one block's chain (measured: 4 sequences
    // of up to 513 tokens, 6.74 us per call under graph replay against 7.34
    // us with 64-token splits; 13.3 against 14.3 us per call).
    S = 1;
    plan->split_tokens = maxblk * kBlockSize;
    // The grid (one block per sequence and kv head group) is under one wave,
    // so each block may take a whole SM: two groups of consumer warps take
    // alternate tiles, which halves the chain of tiles of the longest context.
    plan->consumer_groups = 2;
  } else if (small) {
    constexpr int kTilesPerBlock = kBlockSize / kTile;
    const int64_t tiles = static_cast<int64_t>(maxblk) * kTilesPerBlock;
    const int64_t want = static_cast<int64_t>(sms) * 4;   // about one tile per block
    int split_tiles = static_cast<int>((seq_units * tiles + want - 1) / want);
    if (split_tiles < 1) split_tiles = 1;
    if (split_tiles < kTilesPerBlock) {
      S = static_cast<int>((tiles + split_tiles - 1) / split_tiles);
      plan->split_tokens = split_tiles * kTile;
    }
  }
  plan->num_splits = S;
  plan->prefix_offset = 0;
  plan->prefix_splits = 0;
  plan->prefix_kt_per = 0;
  if (prefix_blocks > 0) {
    // Key ranges of the shared-prefix pass: enough blocks for about one wave.
    const int kt = prefix_blocks * (kBlockSize / 128);
    const int rpt = prefix_rows_per_tile(g);
    if (rpt == 0) return PKV_ERR_SHAPE;
    const int base = (B * g + rpt - 1) / rpt * Hkv;   // query tiles of the pass
    const int sms = sm_count > 0 ? sm_count : 148;
    int ps = base >= sms ? 1 : sms / base;
    if (ps > kt) ps = kt;
    if (ps < 1) ps = 1;
    plan->prefix_kt_per = (kt + ps - 1) / ps;
    plan->prefix_splits = (kt + plan->prefix_kt_per - 1) / plan->prefix_kt_per;
  }
  if (S == 1 && prefix_blocks == 0) {
    plan->workspace_bytes = 0;
  } else {
    if (static_cast<int64_t>(B) * kv_groups * plan->head_groups > kMaxCounters)
      return PKV_ERR_SHAPE;
    size_t bytes = decode_partials_bytes(B, Hq, S);
    if (prefix_blocks > 0) {
      plan->prefix_offset = bytes;
      const size_t prow = static_cast<size_t>(B) * Hq * plan->prefix_splits;
      bytes += align_up(prow * kHeadDim * sizeof(float), 256);
      bytes += align_up(prow * sizeof(float), 256);
    }
    plan->workspace_bytes = bytes;
  }
  return PKV_OK;
}

int launch_decode(const DecodeArgs& a, const DecodePlan& plan, unsigned* err,
                  cudaStream_t stream) {
  if (a.B == 0) return PKV_OK;
  CUtensorMap km, vm;
  if (!decode_maps(a, &km, &vm)) return PKV_ERR_ARG;
  const DecodeParams prm = decode_params(a, plan, err);
  // bf16 pools: the producer-warp form (two blocks per SM either way).  E4M3
  // pools: three blocks per SM of the consumer-issued form, or two of the
  // producer-warp form with a deeper ring; the latter wins once a split is
  // long enough (measured on GB300: 8-block splits of the 32K-128K-token
  // contexts 6% faster, 4-block splits of 512-4096-token contexts 1.5% slower).
  if (a.fp8) {
    const bool prod = plan.split_tokens >= 8 * kBlockSize;
    switch (plan.heads_per_cta) {
      case 8:
        return prod ? launch_g<8, false, true, true>(a, plan, prm, km, vm, stream)
                    : launch_g<8, false, true, false>(a, plan, prm, km, vm, stream);
      case 4:
        return prod ? launch_g<4, false, true, true>(a, plan, prm, km, vm, stream)
                    : launch_g<4, false, true, false>(a, plan, prm, km, vm, stream);
      case 2:
        return prod ? launch_g<2, false, true, true>(a, plan, prm, km, vm, stream)
                    : launch_g<2, false, true, false>(a, plan, prm, km, vm, stream);
      default:
        return prod ? launch_g<1, false, true, true>(a, plan, prm, km, vm, stream)
                    : launch_g<1, false, true, false>(a, plan, prm, km, vm, stream);
    }
  }
  // bf16 single-token batches of one split per sequence under one wave: the
  // producer-warp form with two consumer groups (one block per SM)
  if (plan.consumer_groups == 2 && a.q_len == 1) {
    switch (plan.heads_per_cta) {
      case 8: return launch_g<8, false, false, true, 2>(a, plan, prm, km, vm, stream);
      case 4: return launch_g<4, false, false, true, 2>(a, plan, prm, km, vm, stream);
      case 2: return launch_g<2, false, false, true, 2>(a, plan, prm, km, vm, stream);
      default: return launch_g<1, false, false, true, 2>(a, plan, prm, km, vm, stream);
    }
  }
  // bf16 batches split into 64-token tiles: the 2-stage consumer-issued form
  // (three blocks per SM)
  if (plan.split_tokens < kBlockSize) {
    switch (plan.heads_per_cta) {
      case 8:
        return a.q_len > 1 ? launch_g<8, true, false, false>(a, plan, prm, km, vm, stream)
                           : launch_g<8, false, false, false>(a, plan, prm, km, vm, stream);
      case 4:
        return a.q_len > 1 ? launch_g<4, true, false, false>(a, plan, prm, km, vm, stream)
                           : launch_g<4, false, false, false>(a, plan, prm, km, vm, stream);
      case 2:
        return a.q_len > 1 ? launch_g<2, true, false, false>(a, plan, prm, km, vm, stream)
                           : launch_g<2, false, false, false>(a, plan, prm, km, vm, stream);
      default:
        return a.q_len > 1 ? launch_g<1, true, false, false>(a, plan, prm, km, vm, stream)
                           : launch_g<1, false, false, false>(a, plan, prm, km, vm, stream);
    }
  }
  switch (plan.heads_per_cta) {
    case 8:
      return a.q_len > 1 ? launch_g<8, true, false, true>(a, plan, prm, km, vm, stream)
                         : launch_g<8, false, false, true>(a, plan, prm, km, vm, stream);
    case 4:
      return a.q_len > 1 ? launch_g<4, true, false, true>(a, plan, prm, km, vm, stream)
                         : launch_g<4, false, false, true>(a, plan, prm, km, vm, stream);
    case 2:
      return a.q_len > 1 ? launch_g<2, true, false, true>(a, plan, prm, km, vm, stream)
                         : launch_g<2, false, false, true>(a, plan, prm, km, vm, stream);
    default:
      return a.q_len > 1 ? launch_g<1, true, false, true>(a, plan, prm, km, vm, stream)
                         : launch_g<1, false, false, true>(a, plan, prm, km, vm, stream);
  }
}

}  // namespace pkv
