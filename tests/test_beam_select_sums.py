"""How well beam_select keeps the sums: scores whose exact value is near 0, so that their own
rounding does not hide the sums', and the order of beams whose scores lie close together.

Bound.  A term is 2^t, t rounded twice (2^-23 |t| ln 2 together) by a function good to 2^-22.
A lane adds 16 terms of a segment in two chains of 8, joins them and adds the segment to its sum:
9 roundings of a segment's terms and one for each of its n segments, 5 more over the lanes.  A
warp's maximum may move with each of the n segments, and moves once more where the warps' sums
meet: a factor good to 2^-22 (its argument, a difference, is rounded by 2^-24 of it) and a
product.  Everything behind is in 64 bits."""
import math

import pytest
import torch

from paged_kv_cache_214_gb300 import pkv

gpu = pytest.mark.gpu


def sums(x):
    """(max, ln(sum of e^(x - max)), bound of its error) of rows, in 64 bits."""
    x = x.double()
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    t = (m - x) / math.log(2)
    n = -(-(x.shape[-1] // 512 + 1) // 8)   # (a thread block may have a whole row)
    terms = (e / total * (2.0 ** -22 + 2.0 ** -23 * math.log(2) * t)).sum(-1)
    moves = (n + 1) * (2.0 ** -22 + 2.0 ** -24 + 2.0 ** -24 * 10)
    return m[..., 0], total.log()[..., 0], terms + 2.0 ** -24 * (9 + n + 5) + moves


def check_rows(x, what=""):
    """x [B, V]: each row a request with one beam, whose score takes away its best logit's."""
    m, log_sum, err = sums(x.cuda())
    scores = log_sum.float()
    best, parents, tokens, _ = pkv.beam_select(x.cuda()[:, None], scores[:, None], 1)
    off = (best[:, 0].double() - (scores.double() - log_sum)).abs()
    assert (parents == 0).all()
    assert torch.equal(x.cuda().gather(1, tokens.long())[:, 0].double(), m), what
    assert (off <= err + 2.0 ** -24 * best[:, 0].abs()).all(), f"{what}: {(off / err).max()} of the bound"
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
@pytest.mark.parametrize("order", ["ascending", "descending", "shuffled", "warps"])
@pytest.mark.parametrize("side", [1.0, -1.0])
def test_maxima_on_both_sides_of_the_limit(side, order):
    """Sums are kept differently below and above 8192: rows with logits on both sides, close
    enough for all of them to count."""
    g = torch.Generator().manual_seed(7)
    for V, width in ((600, 4.0), (5000, 4.0), (20011, 0.2), (150001, 4.0)):
        x = side * 8192.0 + width * (torch.rand(6, V, generator=g) - 0.5)
        if order == "ascending":
            x = x.sort(-1).values
        elif order == "descending":
            x = x.sort(-1, descending=True).values
        elif order == "warps":   # segments of the one side and of the other in turn
            below = (torch.arange(V) // 512) % 2 == 0
            x = torch.where(below, side * 8192.0 - 0.03, side * 8192.0 + 0.03) + 1e-3 * x.frac()
        check_rows(x, f"V {V}")


def one_segment_bound(x):
    """The bound where a warp has one segment of a row at most: nothing moves in the stream."""
    x = x.double()
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    t = (m - x) / math.log(2)
    terms = (e / total * (2.0 ** -22 + 2.0 ** -23 * math.log(2) * t)).sum(-1)
    return m[..., 0], total.log()[..., 0], terms + 2.0 ** -24 * (9 + 1 + 5) + 2.0 ** -22 + 2.0 ** -23


def peaked(x, g):
    """One token a row with about half of the mass."""
    rows = x.shape[0]
    mass = x.double().logsumexp(-1).float()
    at = torch.randint(0, x.shape[-1], (rows,), generator=g)
    x[torch.arange(rows), at] = mass + 0.01 * torch.randn(rows, generator=g)
    return x


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [0.0, 200.0, 1000.0, 8000.0])
@pytest.mark.parametrize("V", [700, 50001, 150001])
def test_sums_of_ordinary_and_peaked_rows(V, offset, dtype):
    """Few requests, whose segments are dealt out to more warps than there are.  (A product with
    log2(e) rounded to fp32 would be off by 1.3e-8 of the offset: 1.3e-5 at 1000.)"""
    g = torch.Generator().manual_seed(V)
    for x in (3 * torch.randn(4, V, generator=g), 0.1 * torch.randn(4, V, generator=g),
              peaked(torch.randn(4, V, generator=g), g)):
        x = (x + offset).to(dtype).cuda()
        m, log_sum, err = one_segment_bound(x)
        scores = log_sum.float()
        best, _, tokens, _ = pkv.beam_select(x[:, None], scores[:, None], 1)
        assert torch.equal(x.gather(1, tokens[:, 0].long()[:, None])[:, 0].double(), m)
        off = (best[:, 0].double() - (scores.double() - log_sum)).abs()
        assert (off <= err + 2.0 ** -24 * best[:, 0].abs()).all(), f"{(off / err).max()} of the bound"


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [50001, 150001])
def test_order_of_beams_that_lie_close_together(V, dtype):
    """The best tokens of two beams, further apart than both sums' errors by a few steps of a
    score (an fp32 number below 1) at most: the better one comes first, whichever beam has it."""
    g = torch.Generator().manual_seed(V + 1)
    for seed in range(6):
        x = torch.randn(1, 2, V, generator=g)
        x = torch.stack([peaked(x[:, w], g) for w in range(2)], 1).to(dtype).cuda()
        m, log_sum, err = one_segment_bound(x[0])
        log_p = -log_sum                      # of each beam's best token
        for better in (0, 1):
            scores = torch.zeros(1, 2, device="cuda")
            gap = float(err.sum())
            scores[0, 1 - better] = -log_p[1 - better]
            scores[0, better] = (-log_p[better] + gap + 2.0 ** -23).float()
            s = scores[0].double() + log_p
            assert gap < s[better] - s[1 - better] < gap + 2.0 ** -22
            _, parents, tokens, _ = pkv.beam_select(x, scores, 2)
            assert parents.tolist() == [[better, 1 - better]]
