"""Grouped decode: infinities and NaN in the values that one of a request's sequences sees are
nobody else's: pages of its own, pages that some share, positions behind a shorter one's length."""
import pytest
import torch

import scored_ref as R
from paged_kv_cache_214_gb300 import pkv
from test_grouped_decode import Group, mixed, prompt

gpu = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def spoil(g, places):
    """Puts a value that is not finite at (row, position, kv head, dim) of the rows' pages; returns
    which outputs see one."""
    Hq, Hkv = g.q.shape[1], g.kc.shape[2]
    at = {}
    for k, (row, pos, head, dim) in enumerate(places):
        slot = int(g.tables[row, pos // 256]) * 256 + pos % 256
        at[slot, head, dim] = (0x7f, 0xff)[k % 2] if g.fp8 else (NAN, INF, -INF)[k % 3]
    seen = torch.zeros(g.q.shape, dtype=torch.bool)
    for row, n in enumerate(g.lens.tolist()):
        j = torch.arange(n)
        slots = set((g.tables[row].long()[j // 256] * 256 + j % 256).tolist())
        for slot, head, dim in at:
            if slot in slots:
                seen[row, head * (Hq // Hkv):(head + 1) * (Hq // Hkv), dim] = True
    clean = g.vc.clone()
    for (slot, head, dim), value in at.items():
        g.vc.view(-1, *g.vc.shape[2:])[slot, head, dim] = value
        clean.view(-1, *clean.shape[2:])[slot, head, dim] = 0
    spoiled, g.vc = g.vc, clean
    want = g.want()   # (what is not spoiled does not depend on the places that are)
    g.vc = spoiled
    return seen, want


def check(g, places, splits=(0, 1, 2), what=""):
    seen, want = spoil(g, places)
    assert seen.any() and not seen.all()
    for n in splits:
        out, lse = g.run(num_splits=n)
        out = out.cpu()
        assert not torch.isfinite(out[seen]).any(), f"{what} S={n}: a row that sees it is finite"
        R.check(torch.where(seen, want[0], out.double()), lse, want, f"{what} S={n}")
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,width", [(8, 2, 2), (8, 2, 4), (8, 2, 7), (14, 2, 5), (5, 1, 12), (64, 1, 3),
                                          (4, 2, 32)])
def test_pages_of_one_sequence(Hq, Hkv, width, fp8):
    lens = [600 + 7 * w for w in range(width)] + [300 + w for w in range(width)]
    g = Group(lens, width, Hq, Hkv, 10 + width, prompt(1), fp8).poison()
    check(g, [(1, 256, 0, 0), (1, 300, Hkv - 1, 77), (1, 606, 0, 127), (width, 299, 0, 5), (width, 270, 0, 6)])


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("width", [2, 5, 16])
def test_positions_behind_a_shorter_length(width, fp8):
    """All share their pages; the longer ones see what lies behind the shorter ones' ends."""
    for short in (1, 15, 16, 63, 64, 100, 255, 256, 300):
        lens = [short + 3 * w for w in range(width)]
        g = Group(lens, width, 8, 2, 30 + short, prompt(9), fp8).poison()
        last = lens[-1] - 1
        check(g, [(width - 1, last, 0, 3), (width - 1, last, 1, 64), (width - 1, last - 1, 0, 100)],
              what=f"{short}")


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("width", [3, 11])
def test_pages_that_some_share(width, fp8):
    g = Group([900 + 5 * w for w in range(2 * width)], width, 8, 2, 50 + width, mixed(width), fp8).poison()
    check(g, [(0, 10, 0, 1), (1, 500, 1, 2), (2, 800, 0, 50), (width + 1, 64, 1, 9), (width, 63, 0, 9)],
          (0, 1, 3))


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_many_values_of_a_page(fp8):
    """A whole page that is not finite, of one beam."""
    g = Group([700, 700, 700, 512, 512, 512], 3, 8, 2, 70, prompt(2), fp8).poison()
    check(g, [(1, p, h, d) for p in range(512, 700, 9) for h in range(2) for d in range(0, 128, 5)])


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_all_see_it(fp8):
    """In a prompt's page it is everybody's (of that request)."""
    g = Group([700, 690, 700, 512, 511, 400], 3, 8, 2, 71, prompt(2), fp8).poison()
    check(g, [(0, 17, 0, 3), (1, 200, 1, 90)])


@gpu
def test_keys_of_one_sequence():
    g = Group([600, 610, 300, 310], 2, 8, 2, 72, prompt(1)).poison()
    for row, pos in ((1, 300), (2, 299)):
        slot = int(g.tables[row, pos // 256]) * 256 + pos % 256
        g.kc.view(-1, 2, 128)[slot, 0, 5] = NAN
    want = g.want()
    out, lse = g.run()
    bad = torch.zeros(4, 8, dtype=torch.bool)
    bad[1, :4] = bad[2, :4] = True
    assert torch.isnan(out.cpu()[bad]).all() and torch.isnan(lse.cpu()[bad]).all()
    for x in (*want,):
        assert x[~bad].isfinite().all()
    for r, h in (~bad).nonzero().tolist():
        R.check(out[r, h][None, None], lse[r, h][None, None], [x[r, h][None, None] for x in want], f"{r} {h}")
