"""Grouped decode over E4M3 pools where most of the output comes from keys whose weights are
far below the largest: one key above a long row of others, values of one sign.

Bound.  A weight is rounded to f16, 2^-11 of itself; the largest is at least 2^11 and f16's
smallest step 2^-24, so a small one is off by 2^-36 of the largest.  The output is rounded to
bf16, 2^-8.  Sums are fp32: with one range of n keys a lane adds n / 4 weights (16 rows to a
warp, four lanes a row) and an accumulator takes 16 products at a time, n / 16 steps, each
addition off by 2^-24 of the sum and each step by 2^-23."""
import math

import pytest
import torch

from paged_kv_cache_214_gb300 import pkv

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("width,Hq", [(1, 1), (2, 8), (3, 8), (5, 8)])
@pytest.mark.parametrize("where", [0, 3, -1])
@pytest.mark.parametrize("bits", [20.0, 25.4, 28.0])
def test_one_key_above_many(bits, where, width, Hq):
    """Block 0: keys of score 0.  Block 1: the same with one key 2^bits above.  A row names them
    in 2000 columns."""
    columns = 2000
    n = 256 * columns
    k = torch.zeros(2, 256, 1, 128, device="cuda")
    k[1, 77, 0, 0] = 8.0
    v = torch.full((2, 256, 1, 128), 1.5, device="cuda")
    v[1, 77] = 0.25
    codes = [x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v)]
    q = torch.zeros(width, Hq, 128, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = bits * math.log(2) / 8
    table = torch.zeros(width, columns, dtype=torch.int32, device="cuda")
    table[:, where] = 1
    lens = torch.full((width,), n, dtype=torch.int32, device="cuda")
    for splits in (0, 1, 7):
        out, lse = pkv.paged_decode_attention_grouped_fp8(q, *codes, table, lens, width, 1.0, 1.0, 1.0,
                                                          num_splits=splits)
        top = math.exp(8.0 * q[0, 0, 0].item())
        total = top + n - 1
        want = (0.25 * top + 1.5 * (n - 1)) / total
        # (the score: 8 q in fp32, times log2(e): 2^-22 of it at most; a weight 2^-22)
        sums = n / 4 * 2.0 ** -24, n / 16 * 2.0 ** -23
        tol = want * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20 * bits + sum(sums)) + 1.5 * n * 2.0 ** -36
        assert (out.double() - want).abs().max() <= tol
        assert (lse.double() - math.log(total)).abs().max() <= 2.0 ** -20 * (bits + 20) + sums[0]
    assert pkv.get_device_error() == pkv.PKV_OK
