"""Grouped decode over bf16 pools: the softmax weights carry 16 bits whatever the number of rows,
as the per-sequence decode's do."""
import math

import pytest
import torch

from paged_kv_cache_214_gb300 import pkv

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("width,Hq", [(1, 8), (2, 8), (3, 8), (4, 8), (5, 8), (8, 8), (16, 8), (32, 8),
                                      (3, 33)])
def test_weights_that_round_in_one_direction(width, Hq):
    """The first key of each 16 of the first 64 has score 0, the others ln(2^-5 (1 + 2^-8 - 2^-12)),
    whose weight rounds down to 2^-5 in 8 bits: all but 3% of a row's sum, 2^-8 too low.  V is 1, so
    is the output: 1 - 2^-9 and above round to it.  (Weights of 16 bits: off by 2^-16; sums of n
    weights and n / 16 steps of an accumulator, 2^-24 and 2^-23 each: 2^-12 for n = 4096.)"""
    n, columns = 4096, 16
    score = math.log(2.0 ** -5 * (1 + 2.0 ** -8 - 2.0 ** -12))
    high = torch.tensor(score).to(torch.bfloat16)
    k = torch.zeros(2, 256, 1, 128)
    k[..., 0] = high.float()
    k[..., 1] = torch.tensor(score - high.double().item()).to(torch.bfloat16).float()
    k[1, 0:64:16, 0, :2] = 0
    k = k.to(torch.bfloat16).cuda()
    v = torch.ones(2, 256, 1, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(width, Hq, 128, dtype=torch.bfloat16, device="cuda")
    q[..., :2] = 1
    table = torch.zeros(width, columns, dtype=torch.int32, device="cuda")
    table[:, 0] = 1
    lens = torch.full((width,), n, dtype=torch.int32, device="cuda")
    want = math.log(4 + (n - 4) * math.exp(score))
    for splits in (1, 0):
        out, lse = pkv.paged_decode_attention_grouped(q, k, v, table, lens, width, 1.0, num_splits=splits)
        assert (out == 1).all(), f"{splits}: {out.unique().tolist()}"
        # (the key's second part is off by 2^-9 of it, 2^-18; a score 2^-22; the sums as above)
        assert (lse.double() - want).abs().max() <= 2.0 ** -17 + 2.0 ** -12
    each, _ = pkv.paged_decode_attention(q, k, v, table, lens, 1.0)
    assert torch.equal(each, out)
    assert pkv.get_device_error() == pkv.PKV_OK
