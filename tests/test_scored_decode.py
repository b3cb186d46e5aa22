"""paged_decode_attention_scored (bf16 and E4M3 pools) against a plain 64-bit
computation: caps, distance biases, windows, documents, empty rows, stale and
poisoned pages, splits, streams, graphs; and its refusals."""
import ctypes
import time

import pytest
import torch

import scored_ref as R
from paged_kv_cache_214_gb300 import build as B
from paged_kv_cache_214_gb300 import pkv
from paged_kv_cache_214_gb300 import workloads as W

gpu = pytest.mark.gpu
KS, VS = 0.011, 0.014


def codes(x):
    return (x.float() / KS).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


class Batch:
    """A decode batch; scores of a few units (q is `spread` times normal)."""

    def __init__(self, lens, Hq, Hkv, seed, fp8=False, spread=3.0):
        blocks = sum(-(-n // 256) for n in lens) + 3
        w = W.make_decode(lens, Hq, Hkv, blocks, seed, store_new_token=False)
        self.q = (w.q.float() * spread).to(torch.bfloat16)
        self.kc, self.vc = (codes(w.k_cache), codes(w.v_cache)) if fp8 else (w.k_cache, w.v_cache)
        self.tables, self.lens, self.scale, self.fp8, self.Hq = (w.block_tables, w.context_lens,
                                                                 w.scale, fp8, Hq)

    def run(self, tables=None, **kw):
        args = [x.to("cuda") for x in (self.q, self.kc, self.vc,
                                       self.tables if tables is None else tables, self.lens)]
        kw = {k: v.to("cuda") if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
        if self.fp8:
            return pkv.paged_decode_attention_scored_fp8(*args, self.scale, KS, VS, **kw)
        return pkv.paged_decode_attention_scored(*args, self.scale, **kw)

    def want(self, softcap=0.0, alibi_slopes=None, window=0, first_keys=None):
        ks, vs = (KS, VS) if self.fp8 else (1.0, 1.0)
        return R.decode(self.q, self.kc, self.vc, self.tables, self.lens, self.scale, softcap,
                        alibi_slopes, window, first_keys, ks, vs)

    def check(self, what="", splits=(0,), **opt):
        want = self.want(**opt)
        for n in splits:
            out, lse = self.run(num_splits=n, **opt)
            R.check(out, lse, want, f"{what} S={n} {sorted(opt)}")
        assert pkv.get_device_error() == pkv.PKV_OK


OPTIONS = {
    "plain": {},
    "cap": dict(softcap=30.0),
    "cap-small": dict(softcap=2.5),
    "alibi": dict(alibi=True),
    "window": dict(window=100),
    "all": dict(softcap=20.0, alibi=True, window=333),
}


def options(name, Hq):
    o = dict(OPTIONS[name])
    if o.pop("alibi", False):
        o["alibi_slopes"] = R.alibi(Hq)
    return o


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(OPTIONS))
@pytest.mark.parametrize("Hq,Hkv", [(16, 8), (32, 8), (8, 8), (12, 4), (14, 2), (5, 1), (64, 8)])
def test_options_and_heads(Hq, Hkv, name, fp8):
    b = Batch([1, 17, 256, 300, 513, 1100], Hq, Hkv, 100 + Hq, fp8)
    b.check(f"{name} {Hq}/{Hkv}", **options(name, Hq))


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_tile_and_page_edges(fp8):
    lens = [1, 2, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 511, 512, 513]
    b = Batch(lens, 8, 2, 201, fp8)
    b.check("edges", splits=(0, 1, 2), softcap=25.0)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 255, 256, 257, 700, 5000, 2 ** 31 - 1])
def test_windows(window, fp8):
    b = Batch([1, 64, 65, 300, 512, 777, 1500], 8, 4, 300 + window % 1000, fp8)
    b.check(f"window {window}", splits=(0, 1, 3), window=window)


@gpu
@pytest.mark.parametrize("num_splits", [1, 2, 3, 7, 0, 64])
def test_splits(num_splits):
    b = Batch([1, 255, 700, 4097, 2500], 16, 8, 400)
    b.check("splits", splits=(num_splits,), softcap=15.0, alibi_slopes=R.alibi(16))
    b.check("splits", splits=(num_splits,), softcap=15.0, window=2000)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_documents_and_rows_without_keys(fp8):
    lens = [300, 300, 300, 513, 900, 1, 64]
    first = torch.tensor([0, 299, 300, 512, 600, -5, 2 ** 31 - 1], dtype=torch.int32)
    b = Batch(lens, 8, 2, 500, fp8)
    for n in (0, 1, 2):
        out, lse = b.run(first_keys=first, num_splits=n)
        R.check(out, lse, b.want(first_keys=first), f"documents S={n}")
        assert not out[2].any() and not out[6].any()
        assert (lse[2] == float("-inf")).all() and (lse[6] == float("-inf")).all()
    b.check("documents and window", first_keys=first, window=150)
    # a context of no tokens
    b.lens[0] = 0
    out, lse = b.run(softcap=10.0)
    assert not out[0].any() and (lse[0] == float("-inf")).all()
    R.check(out, lse, b.want(softcap=10.0), "ctx 0")
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_hidden_keys_may_hold_anything(fp8):
    """NaN and infinities in every slot that no row sees, and freed pages (-1 in
    the table) behind the window."""
    lens = [700, 900, 65, 1300]
    b = Batch(lens, 8, 2, 600, fp8)
    window = 130
    want = b.want(window=window, softcap=20.0)
    seen = torch.zeros(b.kc.shape[0] * 256, dtype=torch.bool)
    tables = b.tables.clone()
    for i, n in enumerate(lens):
        j = torch.arange(max(0, n - window), n)
        seen[b.tables[i].long()[j // 256] * 256 + j % 256] = True
        tables[i, :max(0, n - window) // 256] = -1
    shape = b.kc.shape
    for pool, poison in ((b.kc, (float("nan"), float("inf"))), (b.vc, (float("inf"), float("nan")))):
        rows = pool.view(-1, *shape[2:])
        hidden = (~seen).nonzero().flatten()
        if fp8:
            rows[hidden] = 0x7F
        else:
            rows[hidden[::2]] = poison[0]
            rows[hidden[1::2]] = poison[1]
    for n in (0, 1, 2):
        out, lse = b.run(tables=tables, window=window, softcap=20.0, num_splits=n)
        R.check(out, lse, want, f"poisoned S={n}")
    first = torch.tensor([n - 130 if n > 130 else 0 for n in lens], dtype=torch.int32)
    out, lse = b.run(tables=tables, first_keys=first, softcap=20.0)
    R.check(out, lse, want, "poisoned documents")
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
def test_large_scores():
    """Scores far past the cap, and hundreds without one."""
    b = Batch([40, 513], 8, 2, 700, spread=300.0)
    b.check("capped", softcap=50.0)
    b.check("not capped")


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("softcap", [1e-3, 0.3, 70.0, 500.0, 1e4, 1e7])
def test_caps_of_any_size(softcap, fp8):
    b = Batch([40, 513, 1100], 8, 2, 710, fp8, spread=20.0)
    b.check("cap", softcap=softcap)
    b.check("cap", softcap=softcap, alibi_slopes=R.alibi(8), window=200)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("spread,scaled", [(20.0, 1.0), (2.0 ** -12, 2.0 ** 14), (2.0 ** 20, 2.0 ** -20)])
@pytest.mark.parametrize("softcap", [1e12, 1e33, 1e37])
def test_wide_caps_keep_every_bit(softcap, spread, scaled, fp8):
    """Caps that change nothing, small and large queries: the multipliers of a raw
    product may lie below the smallest normal number.

    E4M3 pools carry a weight as two f16 numbers.  Both are multiples of 2^-24, the
    step of f16's subnormal numbers, so the weight is off by 2^-25 at most beside
    its relative error.  Weights are taken against a maximum that no score is below
    in all its keys, so that their sum is at least 1: the output is off by another
    2^-25 sum_j |v_j| over the visible keys at most."""
    b = Batch([40, 513, 1100], 8, 2, 720, fp8, spread=spread)
    b.scale *= scaled
    for opt in ({}, dict(alibi_slopes=R.alibi(8), window=200)):
        want = b.want(softcap=softcap, **opt)
        if fp8:
            for i, n in enumerate(b.lens.tolist()):
                v = R.gather(b.vc, b.tables[i], n)[-opt.get("window", n):].abs() * VS
                want[2][i] += 2.0 ** -25 * v.sum(0).repeat_interleave(4, 0)
        out, lse = b.run(softcap=softcap, **opt)
        R.check(out, lse, want, f"cap {softcap} {sorted(opt)}")
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_no_options_equal_plain_attention(fp8):
    b = Batch([1, 300, 1000, 4100], 16, 8, 800, fp8)
    args = [x.to("cuda") for x in (b.q, b.kc, b.vc, b.tables, b.lens)]
    out, lse = b.run()
    if fp8:
        o2, l2 = pkv.paged_decode_attention_fp8(*args, b.scale, KS, VS)
    else:
        o2, l2 = pkv.paged_decode_attention(*args, b.scale)
    want = b.want()
    R.check(out, lse, want, "scored")
    R.check(o2, l2, want, "plain")


@gpu
def test_far_positions_and_small_slopes():
    """A distance past 2^16 with slopes small enough to leave it some weight."""
    b = Batch([70000], 2, 1, 900, spread=1.0)
    b.check("far", splits=(0, 5), alibi_slopes=torch.tensor([1e-4, -1e-5]))


@gpu
def test_bad_entries_are_reported():
    b = Batch([700], 8, 2, 1000)
    t = b.tables.clone()
    t[0, 1] = 999
    b.run(tables=t, softcap=5.0)
    assert pkv.get_device_error() == pkv.PKV_ERR_DEVICE_INDEX
    b.lens[0] = 256 * t.shape[1] + 1
    b.run(softcap=5.0)
    assert pkv.get_device_error() == pkv.PKV_ERR_DEVICE_INDEX
    b.lens[0] = -3
    b.run(softcap=5.0)
    assert pkv.get_device_error() == pkv.PKV_ERR_DEVICE_INDEX
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
def test_streams_do_not_share_a_workspace():
    """Two calls at once, each on a stream of its own, without given workspaces."""
    b = Batch([4000, 3000, 4096, 3500], 16, 8, 1100)
    want = b.want(softcap=30.0)
    args = [x.to("cuda") for x in (b.q, b.kc, b.vc, b.tables, b.lens)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s in streams:
            got.append(pkv.paged_decode_attention_scored(*args, b.scale, softcap=30.0, num_splits=8,
                                                         stream=s))
    torch.cuda.synchronize()
    R.check(*got[0], want, "two streams")
    for out, lse in got:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    assert pkv.get_device_error() == pkv.PKV_OK


def test_kept_workspaces_are_bounded(monkeypatch):
    """A program that makes a stream for every request does not keep a workspace for
    each of them."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(pkv, "_stream_workspaces", {})
    like = torch.zeros(1)
    for handle in range(1000):
        ws = pkv._workspace(None, 512, like, handle)
        assert ws.numel() >= 512 and not ws.any()
        assert pkv._workspace(None, 256, like, handle) is ws
        assert pkv._workspace(None, 1024, like, handle) is not ws
    assert len(pkv._stream_workspaces) <= 64
    assert pkv._workspace(None, 0, like, 1) is None


@gpu
def test_many_streams_one_after_another():
    """More streams than workspaces are kept for, twice over."""
    b = Batch([4000, 3000, 4096, 3500], 16, 8, 1150)
    want = b.want(softcap=30.0)
    args = [x.to("cuda") for x in (b.q, b.kc, b.vc, b.tables, b.lens)]
    streams = [torch.cuda.Stream(priority=p) for p in (0, -1) for _ in range(32)]
    streams += [torch.cuda.default_stream()]
    torch.cuda.synchronize()
    got = [pkv.paged_decode_attention_scored(*args, b.scale, softcap=30.0, num_splits=8, stream=s)
           for _ in range(2) for s in streams]
    torch.cuda.synchronize()
    R.check(*got[0], want, "first stream")
    for out, lse in got:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
def test_captured_and_replayed():
    a = Batch([300, 2500, 17, 4096], 16, 8, 1200)
    b = Batch([4000, 12, 2222, 800], 16, 8, 1201)
    maxblk = 16
    NB = max(a.kc.shape[0], b.kc.shape[0])
    kc = torch.zeros(NB, 256, 8, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    tables = torch.full((4, maxblk), -1, dtype=torch.int32, device="cuda")
    q, lens = a.q.to("cuda"), a.lens.to("cuda")
    slopes = R.alibi(16).to("cuda")
    out = torch.empty_like(q)
    lse = torch.empty(4, 16, device="cuda")
    need = pkv.paged_decode_scored_workspace_bytes(4, 16, 8, 128, maxblk, window=3000)
    ws = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")
    kw = dict(softcap=30.0, alibi_slopes=slopes, window=3000, out=out, lse=lse)

    def fill(x):
        kc[:x.kc.shape[0]].copy_(x.kc)
        vc[:x.vc.shape[0]].copy_(x.vc)
        tables.fill_(-1)
        tables[:, :x.tables.shape[1]].copy_(x.tables)
        q.copy_(x.q)
        lens.copy_(x.lens)

    s = torch.cuda.Stream()
    fill(a)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        pkv.paged_decode_attention_scored(q, kc, vc, tables, lens, a.scale, workspace=ws, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pkv.paged_decode_attention_scored(q, kc, vc, tables, lens, a.scale, workspace=ws, **kw)
        if need:   # without one of its own the call is refused, and capture goes on
            with pytest.raises(ValueError):
                pkv.paged_decode_attention_scored(q, kc, vc, tables, lens, a.scale, **kw)
    for x in (b, a, b):
        fill(x)
        graph.replay()
        torch.cuda.synchronize()
        R.check(out, lse, x.want(softcap=30.0, alibi_slopes=R.alibi(16), window=3000), "replay")
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
def test_given_outputs_and_no_lse():
    b = Batch([300, 900], 8, 2, 1300)
    args = [x.to("cuda") for x in (b.q, b.kc, b.vc, b.tables, b.lens)]
    out = torch.full_like(args[0], 3.0)
    o, lse = pkv.paged_decode_attention_scored(*args, b.scale, softcap=9.0, out=out, want_lse=False)
    assert o is out and lse is None
    R.check(out, b.want(softcap=9.0)[1], b.want(softcap=9.0), "no lse")
    def bad(error, **kw):
        with pytest.raises(error):
            pkv.paged_decode_attention_scored(*args, b.scale, **kw)

    bad(pkv.PkvError, out=args[0])
    bad(ValueError, out=out[:1])
    bad(ValueError, lse=torch.empty(2, 4, device="cuda"))
    bad(ValueError, alibi_slopes=torch.zeros(4, device="cuda"))
    bad(ValueError, alibi_slopes=torch.zeros(8))
    bad(TypeError, first_keys=torch.zeros(2, device="cuda"))
    bad(ValueError, first_keys=torch.zeros(3, dtype=torch.int32, device="cuda"))
    bad(pkv.PkvError, softcap=-1.0)
    bad(pkv.PkvError, window=-1)
    bad(ValueError, stream=None, workspace=torch.zeros(1 << 22, dtype=torch.uint8))


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("num_splits", [1, 4])
def test_wait_runs_out_then_recovers(num_splits, fp8):
    """Every block's range is longer than the withheld tile; the call comes back
    with an error and the next one is right."""
    b = Batch([3000, 1500, 3500], 16, 8, 1400, fp8)
    want = b.want(softcap=30.0)
    assert pkv.get_device_error() == pkv.PKV_OK
    try:
        pkv.testing_set_wait_fault(1_000_000, 2)
        t0 = time.perf_counter()
        b.run(softcap=30.0, num_splits=num_splits)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 10.0
        assert pkv.get_device_error() == pkv.PKV_ERR_TIMEOUT
    finally:
        pkv.testing_set_wait_fault(0, -1)
    R.check(*b.run(softcap=30.0, num_splits=num_splits), want, "after a timeout")
    assert pkv.get_device_error() == pkv.PKV_OK


def test_host_refusals():
    B.build()
    lib = pkv.load_library()
    P = 1 << 24   # a stand-in address: the checks below fail before any use

    def decode(out=P, lse=None, q=2 * P, kc=P, vc=P, bt=P, maxblk=4, cl=P, B=2, Hq=16, Hkv=8,
               D=128, bs=256, NB=16, scale=0.1, scales=None, ws=None, ws_bytes=0, splits=0, **opt):
        o = pkv.ScoreOptions(**opt)
        head = (out, lse, q, kc, vc, bt, maxblk, cl, B, Hq, Hkv, D, bs, NB, scale)
        tail = (ctypes.byref(o), ws, ws_bytes, splits, None)
        if scales is None:
            return lib.paged_decode_attention_scored(*head, *tail)
        return lib.paged_decode_attention_scored_fp8(*head, *scales, *tail)

    nan, inf = float("nan"), float("inf")
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=nan), dict(scale=inf),
               dict(softcap=-1.0), dict(softcap=nan), dict(softcap=inf), dict(softcap=2e37),
               dict(softcap=1e-33), dict(window=-1), dict(prefix_lens=P), dict(alibi_slopes=P + 2), dict(first_keys=P + 1), dict(B=-1),
               dict(Hq=0), dict(maxblk=-1), dict(splits=-1), dict(out=None), dict(q=None),
               dict(kc=None), dict(vc=None), dict(cl=None), dict(bt=None), dict(out=P + 8),
               dict(q=P), dict(q=P + 4096)):
        assert decode(**kw) == pkv.PKV_ERR_ARG, kw
        assert decode(**kw, scales=(1.0, 1.0)) == pkv.PKV_ERR_ARG, kw
    for kw in (dict(Hq=12), dict(D=64), dict(bs=128), dict(NB=1 << 24)):
        assert decode(**kw) == pkv.PKV_ERR_SHAPE, kw
    for s in ((0.0, 1.0), (1.0, -1.0), (nan, 1.0), (1.0, inf)):
        assert decode(scales=s) == pkv.PKV_ERR_ARG
    assert decode(B=0, q=None) == pkv.PKV_OK
    assert decode(B=0, q=None, scale=0.0) == pkv.PKV_ERR_ARG
    # no options at all: a NULL struct
    assert lib.paged_decode_attention_scored(None, None, None, None, None, None, 1, None, 0, 16, 8,
                                             128, 256, 4, 1.0, None, None, 0, 0,
                                             None) == pkv.PKV_OK


def test_numbers_past_32_bits_are_refused():
    """The library takes 32-bit ints; a larger number is not cut to its low bits."""
    B.build()
    ten = [None] * 10   # (refused before any tensor is looked at)
    for n in (2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1):
        for kw in (dict(window=n), dict(num_splits=n)):
            name = next(iter(kw))
            with pytest.raises(ValueError, match=name):
                pkv.paged_decode_attention_scored(*ten[:6], **kw)
            with pytest.raises(ValueError, match=name):
                pkv.paged_decode_attention_scored_fp8(*ten[:8], **kw)
            with pytest.raises(ValueError, match=name):
                pkv.paged_decode_scored_workspace_bytes(4, 16, 8, 128, 16, **kw)
        with pytest.raises(ValueError, match="max_blocks_per_seq"):
            pkv.paged_decode_scored_workspace_bytes(4, 16, 8, 128, n)
        with pytest.raises(ValueError, match="window"):
            pkv.paged_prefill_attention_scored(*ten[:6], 1, 1, 1.0, window=n)
        with pytest.raises(ValueError, match="max_seqlen_q"):
            pkv.paged_prefill_attention_scored(*ten[:6], n, 1, 1.0)
        with pytest.raises(ValueError, match="max_seqlen_k"):
            pkv.paged_prefill_attention_scored(*ten[:6], 1, n, 1.0)


def test_caps_too_small_for_the_arithmetic_are_refused():
    """A cap that 32 bits round to 0 is not no cap; over E4M3 pages the multiplier of a
    raw product, scale * k_scale / softcap, has to stay finite."""
    B.build()
    for softcap in (1e-50, -1e-50, 1e-45):
        with pytest.raises(ValueError, match="softcap"):
            pkv._score_options(softcap, None, 0, None)
    lib, P = pkv.load_library(), 1 << 24

    def decode(softcap, k_scale):
        o = pkv.ScoreOptions(softcap=softcap)
        return lib.paged_decode_attention_scored_fp8(P, None, 2 * P, P, P, P, 4, P, 2, 16, 8, 128,
                                                     256, 16, 0.1, k_scale, 1.0, ctypes.byref(o),
                                                     None, 0, 0, None)

    assert decode(1e-30, 1e9) == pkv.PKV_ERR_ARG
    assert decode(3e-23, 1e9) == pkv.PKV_ERR_ARG
    assert decode(1e-32, 1e-9) == pkv.PKV_ERR_ARG   # (as over bf16 pages)


def test_block_tables_of_two_to_the_31_tokens_are_refused():
    """With a window the table may be far wider than what is read of it; positions
    are 32-bit all the same."""
    B.build()
    lib, P = pkv.load_library(), 1 << 24

    def decode(maxblk, window):
        o = pkv.ScoreOptions(window=window)
        return lib.paged_decode_attention_scored(P, None, 2 * P, P, P, P, maxblk, P, 2, 16, 8, 128,
                                                 256, 16, 0.1, ctypes.byref(o), None, 0, 0, None)

    for maxblk in (2 ** 23, 2 ** 24, 2 ** 31 - 1):
        for window in (1, 1000, 2 ** 31 - 1):
            assert decode(maxblk, window) == pkv.PKV_ERR_SHAPE
    assert decode(2 ** 23 - 1, 2 ** 31 - 300) == pkv.PKV_ERR_SHAPE
