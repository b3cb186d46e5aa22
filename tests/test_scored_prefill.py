"""paged_prefill_attention_scored against a plain 64-bit computation: caps,
distance biases, windows, documents, two-way prefixes, rows without keys, stale
and poisoned pages; and its refusals."""
import ctypes
import itertools
import time

import pytest
import torch

import scored_ref as R
from paged_kv_cache_214_gb300 import build as B
from paged_kv_cache_214_gb300 import pkv
from paged_kv_cache_214_gb300 import workloads as W

gpu = pytest.mark.gpu


class Batch:
    """Chunks of new rows over cached tokens, everything already in the pool."""

    def __init__(self, old, new, Hq, Hkv, seed, spread=3.0):
        blocks = sum(-(-(a + b) // 256) for a, b in zip(old, new)) + 3
        w = W.make_prefill(old, new, Hq, Hkv, blocks, seed)
        self.q = (w.q.float() * spread).to(torch.bfloat16)
        self.kc, self.vc, self.tables = w.k_cache, w.v_cache, w.block_tables
        self.cu_q, self.cu_k, self.scale, self.Hq = w.cu_seqlens_q, w.cu_seqlens_k, w.scale, Hq
        self.max_q, self.max_k = w.max_seqlen_q, w.max_seqlen_k
        self.old, self.new = old, new

    def run(self, tables=None, **kw):
        args = [x.to("cuda") for x in (self.q, self.kc, self.vc,
                                       self.tables if tables is None else tables, self.cu_q,
                                       self.cu_k)]
        kw = {k: v.to("cuda") if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
        return pkv.paged_prefill_attention_scored(*args, self.max_q, self.max_k, self.scale, **kw)

    def want(self, softcap=0.0, alibi_slopes=None, window=0, first_keys=None, prefix_lens=None):
        return R.prefill(self.q, self.kc, self.vc, self.tables, self.cu_q, self.cu_k, self.scale,
                         softcap, alibi_slopes, window, first_keys, prefix_lens)

    def check(self, what="", **opt):
        out, lse = self.run(**opt)
        R.check(out, lse, self.want(**opt), f"{what} {sorted(opt)}")
        assert pkv.get_device_error() == pkv.PKV_OK


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


@gpu
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (5, 1), (6, 3)])
@pytest.mark.parametrize("name", ["plain", "cap", "alibi", "window", "all"])
def test_options_and_heads(Hq, Hkv, name):
    opt = {"plain": {}, "cap": dict(softcap=30.0), "alibi": dict(alibi_slopes=R.alibi(Hq)),
           "window": dict(window=70),
           "all": dict(softcap=12.0, alibi_slopes=R.alibi(Hq), window=200)}[name]
    Batch([0, 0, 256, 500, 37], [1, 130, 129, 150, 5], Hq, Hkv, 10 + Hq).check(name, **opt)


@gpu
@pytest.mark.parametrize("opt", [dict(softcap=20.0), dict(window=129),
                                 dict(softcap=20.0, window=128)])
def test_tile_and_page_edges(opt):
    new = [127, 128, 129, 255, 256, 257]
    old = [1, 127, 128, 129, 0, 255]
    Batch(old, new, 2, 1, 50).check("edges", **opt)


@gpu
@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 255, 256, 300, 2 ** 31 - 1])
def test_windows(window):
    Batch([0, 700, 300, 255], [400, 1, 140, 258], 2, 1, 60 + window % 1000).check(
        f"window {window}", window=window)


@gpu
@pytest.mark.parametrize("softcap,window", list(itertools.product([0.0, 10.0], [0, 100])))
def test_documents(softcap, window):
    """Five documents of ragged lengths that do not see one another, then rows
    that see all of them; first keys of any value."""
    b = Batch([0, 90], [500, 333], 4, 2, 70)
    first = []
    for n, o in zip(b.new, b.old):
        at = [0, 100, 101, 128, 300]
        first += [o + max(a for a in at if a <= r) if r < n - 60 else 0 for r in range(n)]
    b.check("documents", softcap=softcap, window=window, first_keys=ints(first))


@gpu
def test_rows_without_keys():
    b = Batch([0, 300], [200, 140], 4, 2, 80)
    first = torch.zeros(340, dtype=torch.int32)
    first[5] = 6                      # one past its own position
    first[100:128] = 2 ** 31 - 1      # part of a row tile
    first[130] = -2 ** 31
    first[200:340] = 1000             # every row of a sequence
    out, lse = b.run(first_keys=first, softcap=8.0)
    R.check(out, lse, b.want(first_keys=first, softcap=8.0), "empty rows")
    for rows in (slice(5, 6), slice(100, 128), slice(200, 340)):
        assert not out[rows].any() and (lse[rows] == float("-inf")).all()
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
def test_first_keys_in_any_order():
    b = Batch([40], [300], 4, 2, 90)
    g = torch.Generator().manual_seed(1)
    first = torch.randint(-50, 400, (300,), generator=g, dtype=torch.int32)
    b.check("random", first_keys=first)
    b.check("random", first_keys=first, alibi_slopes=R.alibi(4), window=150)


@gpu
@pytest.mark.parametrize("opt", [{}, dict(softcap=15.0), dict(alibi=True), dict(window=120)])
def test_two_way_prefixes(opt):
    opt = dict(opt)
    if opt.pop("alibi", False):
        opt["alibi_slopes"] = R.alibi(4)
    b = Batch([0, 0, 100, 200, 0, 0], [300, 300, 200, 129, 1, 260], 4, 2, 100)
    b.check("prefix", prefix_lens=ints([0, 300, 180, 329, 1, 129]), **opt)


@gpu
def test_prefix_and_documents_together():
    b = Batch([0], [400], 4, 2, 110)
    first = ints([0 if r < 150 else 150 for r in range(400)])
    b.check("both", first_keys=first, prefix_lens=ints([150]), softcap=30.0)
    b.check("both", first_keys=first, prefix_lens=ints([200]))


@gpu
def test_hidden_keys_may_hold_anything():
    """NaN and infinities in every slot that no row of its sequence sees, and
    freed pages (-1 in the table) behind the window."""
    old, new = [700, 1030, 0], [65, 200, 300]
    b = Batch(old, new, 4, 2, 120)
    window = 100
    want = b.want(window=window, softcap=20.0)
    seen = torch.zeros(b.kc.shape[0] * 256, dtype=torch.bool)
    tables = b.tables.clone()
    for i, (o, n) in enumerate(zip(old, new)):
        lo = max(0, o - window + 1)
        j = torch.arange(lo, o + n)
        seen[b.tables[i].long()[j // 256] * 256 + j % 256] = True
        tables[i, :lo // 256] = -1
    for pool, poison in ((b.kc, ("nan", "inf")), (b.vc, ("inf", "nan"))):
        rows = pool.view(-1, *pool.shape[2:])
        hidden = (~seen).nonzero().flatten()
        rows[hidden[::2]] = float(poison[0])
        rows[hidden[1::2]] = float(poison[1])
    out, lse = b.run(tables=tables, window=window, softcap=20.0)
    R.check(out, lse, want, "poisoned")
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
def test_large_scores():
    b = Batch([0, 100], [150, 40], 4, 2, 130, spread=300.0)
    b.check("capped", softcap=50.0)
    b.check("not capped")


@gpu
@pytest.mark.parametrize("softcap", [1e-3, 0.3, 51.0, 53.0, 90.0, 500.0, 1e4, 1e7])
def test_caps_of_any_size(softcap):
    b = Batch([0, 100], [150, 300], 4, 2, 131, spread=20.0)
    b.check("cap", softcap=softcap)
    b.check("cap", softcap=softcap, alibi_slopes=R.alibi(4), window=200)


@gpu
@pytest.mark.parametrize("softcap", [0.0, 30.0, 51.0, 200.0])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_scores_all_of_one_sign(sign, softcap):
    """Every score far below zero (or above): the whole row at one end of the cap."""
    b = Batch([0, 130], [200, 260], 4, 2, 132)
    b.kc.copy_(b.kc.float().abs())
    b.q.copy_(sign * 4 * b.q.float().abs())
    b.check("one sign", softcap=softcap)


@gpu
@pytest.mark.parametrize("softcap", [1e9, 1e10, 1e12, 1e30, 1e37])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_wide_caps_with_scores_of_hundreds(sign, softcap):
    """Caps that change nothing, with every score near -200 or near 200."""
    b = Batch([0, 130], [200, 260], 4, 2, 134)
    b.kc.copy_(b.kc.float().abs())
    b.q.copy_(sign * 10 * b.q.float().abs())
    b.check("wide cap", softcap=softcap)
    b.check("wide cap", softcap=softcap, alibi_slopes=R.alibi(4), window=100)
    b.check("wide cap", softcap=softcap, alibi_slopes=torch.tensor([6.0, 1.4, -1.4, 0.0]))


@gpu
@pytest.mark.parametrize("opt", [{}, dict(alibi=True)])
def test_small_scores_next_to_saturated_rows(opt):
    """Rows whose scores are a few units, between rows (of the same warp) at the
    ends of a wide cap."""
    b = Batch([0, 130], [200, 260], 2, 1, 135, spread=1.0)
    b.scale = 100.0
    row = torch.arange(len(b.q)) % 2 == 1
    b.q.copy_(b.q.float() * torch.where(row, 900.0, 2.7e-3)[:, None, None])
    if opt:
        opt = dict(alibi_slopes=R.alibi(2))
    b.check("mixed", softcap=5e5, **opt)


@gpu
@pytest.mark.parametrize("softcap", [2e4, 1e33, 1e37])
def test_wide_caps_with_tiny_scales(softcap):
    """A scale of 2^-24 or so over large queries: scale / softcap may lie below the
    smallest normal number."""
    b = Batch([0, 130], [200, 60], 4, 2, 136)
    b.scale *= 2.0 ** -20
    b.q.copy_(b.q.float() * 2.0 ** 20)
    b.check("tiny scale", softcap=softcap)
    b.check("tiny scale", softcap=softcap, alibi_slopes=R.alibi(4))


@gpu
@pytest.mark.parametrize("opt", [{}, dict(softcap=300.0), dict(alibi=True), dict(window=300)])
def test_maximum_that_keeps_rising(opt):
    """Scores that grow by hundreds from tile to tile, so that the running maximum
    moves at every one of them."""
    opt = dict(opt)
    if opt.pop("alibi", False):
        opt["alibi_slopes"] = R.alibi(2)
    b = Batch([0, 130], [700, 400], 2, 1, 133, spread=1.0)
    b.q.copy_(b.q.float().abs())
    for i, n in enumerate((700, 530)):
        j = torch.arange(n)
        slots = b.tables[i].long()[j // 256] * 256 + j % 256
        rows = b.kc.view(-1, 1, 128)
        rows[slots] = (rows[slots].float().abs() * (j[:, None, None] * 0.1)).to(torch.bfloat16)
    b.check("rising", **opt)


@gpu
@pytest.mark.parametrize("softcap", [0.0, 20.0, 50.0, 300.0])
@pytest.mark.parametrize("biased", [False, True])
def test_rows_that_see_one_key_return_its_value(biased, softcap):
    """A window of one token, documents of one token, the first row of a prompt: the
    output is the value itself."""
    b = Batch([0, 130], [200, 260], 8, 2, 138)
    opt = dict(softcap=softcap)
    if biased:
        opt["alibi_slopes"] = torch.tensor([1.3, 1.34, 1.345, 6.0, 0.0, -1.3, -1.36, -0.01])
    v = torch.cat([R.gather(b.vc, b.tables[i], o + n)[o:]
                   for i, (o, n) in enumerate(zip(b.old, b.new))]).repeat_interleave(4, 1)
    own = ints([o + r for o, n in zip(b.old, b.new) for r in range(n)])
    for more in (dict(window=1), dict(first_keys=own), {}):
        out, lse = b.run(**opt, **more)
        R.check(out, lse, b.want(**opt, **more), f"{sorted(more)}")
        rows = slice(None) if more else slice(0, 1)
        assert torch.equal(out.cpu().double()[rows], v[rows])
    # one key of a two-way prefix, behind the row itself and in another tile
    first = torch.full((460,), 299, dtype=torch.int32)
    out, lse = b.run(first_keys=first, prefix_lens=ints([0, 300]), **opt)
    want = R.gather(b.vc, b.tables[1], 390)[299].repeat_interleave(4, 0)
    assert torch.equal(out.cpu().double()[200:370], want.expand(170, 8, 128))
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
@pytest.mark.parametrize("size", [2.0 ** 32, 2.0 ** -40])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("softcap", [0.0, 50.0, 51.9, 300.0])
def test_values_at_the_ends_of_their_range(softcap, sign, size):
    """Every score at one end of the cap (or at +-86), so that weights are as large or
    as small as they get, over values near the ends of the range that the call names."""
    b = Batch([900, 0], [130, 300], 2, 1, 137)
    b.kc.copy_(b.kc.float().abs())
    b.q.copy_(sign * (60.0 if softcap else 4.0) * b.q.float().abs())
    b.vc.copy_(size * (0.5 + torch.rand(b.vc.shape, generator=torch.Generator().manual_seed(2)) / 2))
    b.check("values", softcap=softcap)
    b.check("values", softcap=softcap, alibi_slopes=torch.tensor([1.3, -0.3]))


@gpu
@pytest.mark.parametrize("softcap", [0.0, 10.0, 200.0])
def test_slopes_of_any_size(softcap):
    """Slopes around 1.34, where the maximum is taken another way, steep ones, and
    negative ones (far keys weigh more); with and without a two-way prefix."""
    b = Batch([0, 150, 290], [200, 140, 70], 8, 2, 168)
    slopes = torch.tensor([1.3, 1.34, 1.345, 6.0, 0.0, -1.3, -1.36, -0.01])
    b.check("slopes", softcap=softcap, alibi_slopes=slopes)
    b.check("slopes", softcap=softcap, alibi_slopes=slopes, window=77)
    b.check("slopes", softcap=softcap, alibi_slopes=slopes, prefix_lens=ints([130, 40, 360]))


@gpu
def test_no_options_equal_plain_attention():
    b = Batch([0, 300, 17], [260, 129, 1], 8, 2, 140)
    out, lse = b.run()
    args = [x.to("cuda") for x in (b.q, b.kc, b.vc, b.tables, b.cu_q, b.cu_k)]
    o2, l2 = pkv.paged_prefill_attention(*args, b.max_q, b.max_k, b.scale)
    want = b.want()
    R.check(out, lse, want, "scored")
    R.check(o2, l2, want, "plain")


@gpu
def test_many_items_per_block():
    """More (row tile, sequence, head) items than SMs, heads and lengths mixed;
    a sample of the rows is checked."""
    g = torch.Generator().manual_seed(3)
    new = torch.randint(1, 500, (24,), generator=g).tolist()
    old = torch.randint(0, 700, (24,), generator=g).tolist()
    b = Batch(old, new, 16, 4, 150)
    opt = dict(softcap=25.0, window=300)
    out, lse = b.run(**opt)
    pick = []
    for i, n in enumerate(new):
        pick += [int(b.cu_q[i]) + r for r in {0, n // 2, n - 1}]
    parts = []
    for i, (o, n) in enumerate(zip(old, new)):
        k, v = (R.gather(p, b.tables[i], o + n) for p in (b.kc, b.vc))
        rows = sorted({0, n // 2, n - 1})
        at = [int(b.cu_q[i]) + r for r in rows]
        pos = [o + r for r in rows]
        want = R.attend(b.q[at], k, v, pos, [max(0, x - 299) for x in pos], pos, b.scale, 25.0,
                        None, 2.0 ** -8)
        R.check(out[at], lse[at], want, f"sequence {i}")
    again = b.run(**opt)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
@pytest.mark.parametrize("max_k", [4096, 16384, 65536])
def test_any_stated_longest_sequence(max_k):
    """The order of the work depends on the longest sequence that the call states (all
    five sequences together, two at a time, one at a time); the results do not."""
    b = Batch([0, 300, 20, 0, 129], [260, 140, 1, 513, 128], 6, 2, 175)
    tables = torch.zeros(5, max_k // 256, dtype=torch.int32)
    tables[:, :b.tables.shape[1]] = b.tables
    want = b.want(softcap=15.0, window=200)
    b.max_k = max_k
    out, lse = b.run(tables, softcap=15.0, window=200)
    R.check(out, lse, want, f"at most {max_k}")
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
@pytest.mark.parametrize("max_q", [513, 5130, 2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 1])
def test_any_stated_longest_chunk(max_q):
    """A bound on the rows of a sequence, however loose, changes nothing."""
    b = Batch([0, 300, 20], [260, 1, 513], 6, 2, 176)
    want = b.want(softcap=15.0)
    b.max_q = max_q
    out, lse = b.run(softcap=15.0)
    R.check(out, lse, want, f"at most {max_q}")
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
def test_rows_behind_the_last_sequence_stay():
    b = Batch([0, 40], [100, 30], 4, 2, 160)
    q = torch.cat([b.q, torch.zeros(9, 4, 128, dtype=torch.bfloat16)])
    out = torch.full_like(q, 5.0).to("cuda")
    lse = torch.full((139, 4), 5.0, device="cuda")
    args = [x.to("cuda") for x in (q, b.kc, b.vc, b.tables, b.cu_q, b.cu_k)]
    pkv.paged_prefill_attention_scored(*args, b.max_q, b.max_k, b.scale, softcap=7.0, out=out,
                                       lse=lse)
    R.check(out[:130], lse[:130], b.want(softcap=7.0))
    assert (out[130:] == 5.0).all() and (lse[130:] == 5.0).all()


@gpu
def test_bad_sequences_are_reported_and_left():
    b = Batch([0, 100], [64, 64], 4, 2, 170)
    good = b.want(softcap=9.0)

    def call(cu_q=b.cu_q, cu_k=b.cu_k, tables=b.tables, **kw):
        args = [x.to("cuda") for x in (b.q, b.kc, b.vc, tables, cu_q, cu_k)]
        out = torch.full_like(args[0], 5.0)
        lse = torch.full((128, 4), 5.0, device="cuda")
        assert pkv.get_device_error() == pkv.PKV_OK
        pkv.paged_prefill_attention_scored(*args, b.max_q, b.max_k, b.scale, softcap=9.0, out=out,
                                           lse=lse, **kw)
        assert pkv.get_device_error() == pkv.PKV_ERR_DEVICE_INDEX
        return out, lse

    def first_alone(out, lse):
        R.check(out[:64], lse[:64], [x[:64] for x in good])
        assert (out[64:] == 5.0).all() and (lse[64:] == 5.0).all()

    first_alone(*call(cu_k=ints([0, 64, 74])))               # Lk < Lq
    first_alone(*call(cu_q=ints([0, 64, 129])))              # past total_q, and past max_seqlen_q
    first_alone(*call(cu_q=ints([0, 64, 10])))               # backwards
    for p in ([0, -1], [0, 165]):
        first_alone(*call(prefix_lens=ints(p).to("cuda")))
    out, lse = call(cu_q=ints([-1, 0, 64]))                  # starts before q
    assert (out[64:] == 5.0).all()
    t = b.tables.clone()
    t[1, 0] = -7
    call(tables=t)


@gpu
def test_captured_and_replayed():
    b = Batch([0, 40], [100, 30], 4, 2, 180)
    args = [x.to("cuda") for x in (b.q, b.kc, b.vc, b.tables, b.cu_q, b.cu_k)]
    first = torch.zeros(130, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(args[0]), torch.empty(130, 4, device="cuda")

    def step():
        pkv.paged_prefill_attention_scored(*args, 100, 140, b.scale, softcap=7.0, first_keys=first,
                                           out=out, lse=lse)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    first[50:100] = 50
    args[4].copy_(ints([0, 90, 130]))       # other lengths: 90 and 40 rows
    b.cu_q = ints([0, 90, 130])
    graph.replay()
    torch.cuda.synchronize()
    R.check(out, lse, b.want(softcap=7.0, first_keys=first.cpu()), "replay")
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
def test_two_calls_at_once():
    """Calls of both directions on two streams; outputs made by the call itself."""
    b = Batch([0, 700, 130], [900, 300, 513], 8, 2, 185)
    args = [x.to("cuda") for x in (b.q, b.kc, b.vc, b.tables, b.cu_q, b.cu_k)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [pkv.paged_prefill_attention_scored(*args, b.max_q, b.max_k, b.scale, softcap=9.0,
                                              window=300, stream=s)
           for _ in range(20) for s in streams]
    torch.cuda.synchronize()
    R.check(*got[0], b.want(softcap=9.0, window=300), "two streams")
    for out, lse in got:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
def test_wait_runs_out_then_recovers():
    b = Batch([512, 300, 0], [256, 300, 640], 8, 8, 190)
    assert pkv.get_device_error() == pkv.PKV_OK
    before = b.run(softcap=20.0)
    try:
        pkv.testing_set_wait_fault(1_000_000, 3)
        t0 = time.perf_counter()
        b.run(softcap=20.0)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 10.0
        assert pkv.get_device_error() == pkv.PKV_ERR_TIMEOUT
    finally:
        pkv.testing_set_wait_fault(0, -1)
    after = b.run(softcap=20.0)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
def test_wrapper_refusals():
    b = Batch([0, 40], [100, 30], 4, 2, 200)
    args = [x.to("cuda") for x in (b.q, b.kc, b.vc, b.tables, b.cu_q, b.cu_k)]

    def bad(error, n=None, **kw):
        with pytest.raises(error):
            pkv.paged_prefill_attention_scored(*(n or args), b.max_q, b.max_k, b.scale, **kw)

    bad(pkv.PkvError, out=args[0])
    bad(ValueError, out=torch.empty_like(args[0][:5]))
    bad(ValueError, lse=torch.empty(130, 3, device="cuda"))
    bad(ValueError, first_keys=torch.zeros(129, dtype=torch.int32, device="cuda"))
    bad(TypeError, first_keys=torch.zeros(130, dtype=torch.int64, device="cuda"))
    bad(ValueError, prefix_lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    bad(ValueError, prefix_lens=torch.zeros(2, dtype=torch.int32))
    bad(ValueError, alibi_slopes=torch.zeros(2, device="cuda"))
    bad(ValueError, [args[0].transpose(0, 1), *args[1:]])
    bad(ValueError, [*args[:3], args[3][:1], *args[4:]])
    bad(pkv.PkvError, softcap=-2.0)
    bad(pkv.PkvError, window=-2)


def test_host_refusals():
    B.build()
    lib = pkv.load_library()
    P = 1 << 24   # a stand-in address: the checks below fail before any use

    def prefill(out=P, q=2 * P, kc=P, vc=P, bt=P, maxblk=4, cq=P, ck=P, B=2, total=64, max_q=32,
                max_k=500, Hq=16, Hkv=8, D=128, bs=256, NB=16, scale=0.1, **opt):
        o = pkv.ScoreOptions(**opt)
        return lib.paged_prefill_attention_scored(out, None, q, kc, vc, bt, maxblk, cq, ck, B,
                                                  total, max_q, max_k, Hq, Hkv, D, bs, NB, scale,
                                                  ctypes.byref(o), None)

    nan, inf = float("nan"), float("inf")
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=nan), dict(scale=inf),
               dict(softcap=-1.0), dict(softcap=nan), dict(softcap=inf), dict(softcap=2e37),
               dict(softcap=1e-33), dict(window=-1),
               dict(alibi_slopes=P + 2), dict(first_keys=P + 1), dict(prefix_lens=P + 3),
               dict(B=-1), dict(total=-1), dict(max_q=-1), dict(max_k=-1), dict(Hq=0),
               dict(maxblk=-1), dict(out=None), dict(q=None), dict(kc=None), dict(vc=None),
               dict(cq=None), dict(ck=None), dict(bt=None), dict(out=P + 8), dict(q=2 * P + 2),
               dict(q=P), dict(q=P + 4096), dict(max_k=1025), dict(NB=0)):
        assert prefill(**kw) == pkv.PKV_ERR_ARG, kw
    for kw in (dict(Hq=12), dict(D=64), dict(bs=128), dict(NB=1 << 24), dict(total=1 << 31)):
        assert prefill(**kw) == pkv.PKV_ERR_SHAPE, kw
    for kw in (dict(B=0), dict(total=0), dict(max_q=0)):
        assert prefill(q=None, **kw) == pkv.PKV_OK, kw


def test_host_refuses_more_items_than_indexes():
    """Items are (128-row tile, sequence, head); their number is worked out without
    overflow and refused before anything is launched."""
    B.build()
    lib = pkv.load_library()
    P, far = 1 << 24, 1 << 50

    def prefill(B, total, max_q, Hq):
        return lib.paged_prefill_attention_scored(P, None, far, P, P, P, 4, P, P, B, total, max_q,
                                                  500, Hq, 8, 128, 256, 16, 0.1, None, None)

    big = 2 ** 31 - 1
    for max_q in (big, big - 126, big - 127):
        assert prefill(1, big, max_q, 128) == pkv.PKV_ERR_SHAPE
        assert prefill(2, big, max_q, 128) == pkv.PKV_ERR_SHAPE
        assert prefill(big, big, max_q, 1024) == pkv.PKV_ERR_SHAPE
