"""kv_cache_store_norm_rope: norm of query / key heads, rotation and store in one
pass, against a plain 64-bit computation (values still zero where nothing is
stored), and its refusals."""
import itertools

import pytest
import torch

import scored_ref as R
from paged_kv_cache_214_gb300 import build as B
from paged_kv_cache_214_gb300 import pkv

gpu = pytest.mark.gpu


def table(places, rotary, gen):
    angle = torch.arange(places, dtype=torch.float64)[:, None] * torch.pow(
        1e4, -torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def make(T, Hq, Hkv, rotary=128, packed=True, norm=True, seed=0, NB=None, pad=0, odd=0):
    """Host inputs; `odd`: elements by which the rows are shifted off 16 bytes."""
    g = torch.Generator().manual_seed(seed)
    D = 128
    NB = NB or max(1, -(-(T + 5) // 256))
    n = (Hq + 2 * Hkv) * D
    if packed:
        row = torch.randn(T, n + odd, generator=g).to(torch.bfloat16)[:, odd:]
        q, k, v = (x.unflatten(1, (-1, D)) for x in row.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        q, k, v = (torch.randn(T, h, D, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    slots = torch.randperm(NB * 256, generator=g)[:T].to(torch.int32)
    if pad:
        slots[T - pad:] = -1
    places = 5000
    return dict(q=q, k=k, v=v, slots=slots,
                positions=torch.randint(0, places, (T,), generator=g, dtype=torch.int32),
                cos_sin=table(places, rotary, g) if rotary else None,
                q_weight=1 + 0.3 * torch.randn(128, generator=g) if norm else None,
                k_weight=1 + 0.3 * torch.randn(128, generator=g) if norm else None,
                NB=NB, Hkv=Hkv)


def on_gpu(m, name):
    """The device copy of a tensor, token stride kept."""
    t = m[name]
    if t is None:
        return None
    if name in "qkv" and not t.is_contiguous():
        base = t._base.to("cuda")
        return base.as_strided(t.shape, t.stride(), t.storage_offset())
    return t.to("cuda")


def call(m, fp8=False, interleaved=False, eps=1e-6, scales=(0.02, 0.015), **more):
    dtype = torch.uint8 if fp8 else torch.bfloat16
    kc = torch.zeros(m["NB"], 256, m["Hkv"], 128, dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    args = [on_gpu(m, "q"), on_gpu(m, "k"), on_gpu(m, "v"), kc, vc, on_gpu(m, "slots"),
            on_gpu(m, "positions"), on_gpu(m, "cos_sin")]
    kw = dict(q_weight=on_gpu(m, "q_weight"), k_weight=on_gpu(m, "k_weight"), eps=eps,
              interleaved=interleaved, **more)
    if fp8:
        q = pkv.kv_cache_store_norm_rope_fp8(*args, *scales, **kw)
    else:
        q = pkv.kv_cache_store_norm_rope(*args, **kw)
    return q, kc, vc


def verify(m, got, fp8=False, interleaved=False, eps=1e-6, scales=(0.02, 0.015)):
    q, kc, vc = (x.cpu() for x in got)
    ref = lambda x, w: R.norm_rope(x, w, eps, m["positions"], m["cos_sin"], interleaved)  # noqa: E731
    R.check_rows(q, ref(m["q"], m["q_weight"]), "q")
    kept = m["slots"] >= 0
    at = m["slots"][kept].long()
    kc, vc = kc.view(-1, m["Hkv"], 128), vc.view(-1, m["Hkv"], 128)
    k = ref(m["k"], m["k_weight"])[kept]
    if fp8:
        R.check_codes(kc[at], k, scales[0], "k")
        R.check_codes(vc[at], m["v"].double()[kept], scales[1], "v")
    else:
        R.check_rows(kc[at], k, "k")
        assert torch.equal(vc[at].view(torch.int16), m["v"][kept].contiguous().view(torch.int16))
    rest = torch.ones(kc.shape[0], dtype=torch.bool)
    rest[at] = False
    assert not kc[rest].float().any() and not vc[rest].float().any()
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 2, 3, 17, 64, 300])
@pytest.mark.parametrize("heads", [(16, 8), (32, 8), (12, 4), (5, 1), (14, 2)])
def test_tokens_and_heads(T, heads, fp8):
    m = make(T, *heads, seed=T)
    verify(m, call(m, fp8=fp8), fp8=fp8)


@gpu
@pytest.mark.parametrize("rotary,interleaved,norm,packed",
                         list(itertools.product([0, 16, 32, 64, 80, 96, 128], [False, True],
                                                [False, True], [False, True])))
def test_forms(rotary, interleaved, norm, packed):
    m = make(23, 6, 2, rotary=rotary, packed=packed, norm=norm, seed=rotary + norm)
    verify(m, call(m, interleaved=interleaved), interleaved=interleaved)


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_off_sixteen_bytes(fp8):
    for odd in (1, 4):
        m = make(9, 5, 1, seed=odd, odd=odd)
        assert on_gpu(m, "q").data_ptr() % 16
        verify(m, call(m, fp8=fp8), fp8=fp8)


@gpu
def test_one_weight_alone():
    for name in ("q_weight", "k_weight"):
        m = make(11, 4, 2, seed=5)
        m[name] = None
        verify(m, call(m))


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_padding_rows_store_nothing(fp8):
    m = make(40, 6, 2, seed=6, pad=13)
    verify(m, call(m, fp8=fp8), fp8=fp8)
    m = make(40, 6, 2, seed=6, pad=40)
    verify(m, call(m, fp8=fp8), fp8=fp8)


@gpu
def test_in_place_equals_out_of_place():
    m = make(70, 16, 8, packed=False, seed=7)
    want = [x.clone() for x in call(m)]
    kc, vc = torch.zeros_like(want[1]), torch.zeros_like(want[2])
    q = on_gpu(m, "q").clone()
    got = pkv.kv_cache_store_norm_rope(q, on_gpu(m, "k"), on_gpu(m, "v"), kc, vc,
                                       on_gpu(m, "slots"), on_gpu(m, "positions"),
                                       on_gpu(m, "cos_sin"), on_gpu(m, "q_weight"),
                                       on_gpu(m, "k_weight"), q_out=q)
    assert got is q
    for a, b in zip((q, kc, vc), want):
        assert torch.equal(a, b)


@gpu
def test_values_are_those_of_the_plain_stores():
    """V lands as kv_cache_store / kv_cache_store_fp8 put it, NaN payloads and
    infinities included."""
    m = make(33, 8, 2, packed=False, seed=8)
    special = torch.tensor([0x7F80, 0xFF80, 0x7FC1, 0x0001, 0x8000, 0x7F7F], dtype=torch.int32)
    m["v"].view(torch.int16).view(-1)[:6] = special.to(torch.int16)
    q, kc, vc = call(m)
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    pkv.kv_cache_store(on_gpu(m, "k"), on_gpu(m, "v"), k2, v2, on_gpu(m, "slots"))
    assert torch.equal(vc.view(torch.int16), v2.view(torch.int16))
    q, kc, vc = call(m, fp8=True)
    k2, v2 = torch.zeros_like(kc), torch.zeros_like(vc)
    pkv.kv_cache_store_fp8(on_gpu(m, "k"), on_gpu(m, "v"), k2, v2, on_gpu(m, "slots"), 0.02, 0.015)
    assert torch.equal(vc, v2)


@gpu
def test_zero_rows_and_tiny_eps():
    m = make(4, 4, 2, packed=False, seed=9)
    m["q"][1], m["k"][2] = 0, 0
    q, kc, vc = call(m)
    assert not q[1].any() and not torch.isnan(q.float()).any()
    verify(m, (q, kc, vc))
    m["q"] = (m["q"].float() * 1e-18).to(torch.bfloat16)   # mean square far below eps
    verify(m, call(m))


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_infinities_stay_in_their_pair(interleaved):
    """Without a norm, an infinity reaches its rotated partner and nothing else."""
    m = make(3, 4, 2, rotary=32, norm=False, packed=False, seed=16)
    m["q"][0, 0, 5], m["q"][1, 1, 100], m["q"][2, 2, 40] = float("inf"), float("nan"), -float("inf")
    q = call(m, interleaved=interleaved)[0].cpu().double()
    want = R.norm_rope(m["q"], None, 0.0, m["positions"], m["cos_sin"], interleaved)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(q), fine)
    assert (~fine).sum().item() == 4
    over = (q - want).abs()[fine] - 2.0 ** -8 * want.abs()[fine] - 2.0 ** -16
    assert over.max().item() <= 0


@gpu
def test_bad_indices_are_reported_and_skipped():
    m = make(20, 6, 2, packed=False, seed=10)
    good = make(20, 6, 2, packed=False, seed=10)
    for place, slot in ((5000, None), (-1, None), (None, 256 * m["NB"]), (None, 2 ** 31 - 1)):
        m["positions"], m["slots"] = good["positions"].clone(), good["slots"].clone()
        if place is not None:
            m["positions"][7] = place
        if slot is not None:
            m["slots"][7] = slot
        out = torch.full((20, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        assert pkv.get_device_error() == pkv.PKV_OK
        q, kc, vc = call(m, q_out=out)
        assert pkv.get_device_error() == pkv.PKV_ERR_DEVICE_INDEX
        rows = kc.view(-1, 2, 128)[good["slots"][7].long()]
        assert not rows.any()
        assert (place is None) or (q[7] == 7.0).all()
        others = [t for t in range(20) if t != 7]
        ref = R.norm_rope(good["q"], good["q_weight"], 1e-6, good["positions"], good["cos_sin"], False)
        R.check_rows(q[others], ref[others])


@gpu
def test_many_units_and_a_side_stream():
    """More half-warp tasks than one wave, launched on a stream of its own."""
    m = make(5000, 12, 4, seed=12)
    s = torch.cuda.Stream()
    args = [on_gpu(m, n) for n in ("q", "k", "v")]
    kc = torch.zeros(m["NB"], 256, 4, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    rest = [on_gpu(m, n) for n in ("slots", "positions", "cos_sin", "q_weight", "k_weight")]
    s.wait_stream(torch.cuda.current_stream())
    q = pkv.kv_cache_store_norm_rope(*args, kc, vc, *rest, stream=s)
    q2 = pkv.kv_cache_store_norm_rope(*args, kc, vc, *rest, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(q, q2)
    pick = torch.arange(0, 5000, 37)
    ref = R.norm_rope(m["q"][pick], m["q_weight"], 1e-6, m["positions"][pick], m["cos_sin"], False)
    R.check_rows(q.cpu()[pick], ref)


def check_store(m, got, fp8, interleaved, scales=(0.02, 0.015), sample=None):
    """Everything that a call over `m` leaves: every stored row and every slot that
    takes none; the queries of the tokens `sample` (all of them).  Tokens whose
    position is outside the table leave their row of q_out (7 before the call) and
    their slot; slots past the pool, and below 0, take nothing."""
    q, kc, vc = (x.cpu() for x in got)
    T = len(m["slots"])
    placed = torch.ones(T, dtype=torch.bool)
    if m["cos_sin"] is not None:
        placed = (m["positions"] >= 0) & (m["positions"] < m["cos_sin"].shape[0])
    t = torch.arange(T) if sample is None else sample
    t = t[placed[t]]
    R.check_rows(q[t], R.norm_rope(m["q"][t], m["q_weight"], 1e-6, m["positions"][t], m["cos_sin"],
                                   interleaved), "q")
    assert (q[~placed] == 7.0).all()
    stored = placed & (m["slots"] >= 0) & (m["slots"] < m["NB"] * 256)
    at = m["slots"][stored].long()
    kc, vc = kc.view(-1, m["Hkv"], 128), vc.view(-1, m["Hkv"], 128)
    k = R.norm_rope(m["k"][stored], m["k_weight"], 1e-6, m["positions"][stored], m["cos_sin"],
                    interleaved)
    if fp8:
        R.check_codes(kc[at], k, scales[0], "k")
        R.check_codes(vc[at], m["v"].double()[stored], scales[1], "v")
    else:
        R.check_rows(kc[at], k, "k")
        assert torch.equal(vc[at].view(torch.int16), m["v"][stored].contiguous().view(torch.int16))
    rest = torch.ones(kc.shape[0], dtype=torch.bool)
    rest[at] = False
    assert not kc[rest].float().any() and not vc[rest].float().any()


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [(32, 8), (12, 4), (5, 1)])
@pytest.mark.parametrize("rotary,interleaved,norm,odd", [
    (128, False, True, 0), (128, True, True, 0), (64, False, True, 0), (96, True, False, 0),
    (0, False, True, 0), (64, True, True, 1), (96, False, True, 4)])
def test_several_rows_and_tokens_a_warp(heads, rotary, interleaved, norm, odd, fp8):
    """Enough tokens that a half-warp takes four rows (32 / 8 heads), two (12 / 4) or
    one (5 / 1) and goes on to a third token, with padding, slots past the pool and
    positions outside the table in between."""
    T = 2000
    m = make(T, *heads, rotary=rotary, norm=norm, seed=40 + rotary, odd=odd)
    bad = torch.arange(3, T, 41)
    m["slots"][bad[0::4]] = -1
    m["slots"][bad[1::4]] = m["NB"] * 256 + torch.arange(len(bad[1::4]), dtype=torch.int32)
    m["slots"][bad[2::4]] = -2 ** 31
    if rotary:
        m["positions"][bad[3::4]] = 5000
        m["positions"][bad[2::4]] = -1
    out = torch.full((T, heads[0], 128), 7.0, dtype=torch.bfloat16, device="cuda")
    assert pkv.get_device_error() == pkv.PKV_OK
    got = call(m, fp8=fp8, interleaved=interleaved, q_out=out)
    assert pkv.get_device_error() == pkv.PKV_ERR_DEVICE_INDEX
    check_store(m, got, fp8, interleaved, sample=torch.cat([bad, torch.arange(0, T, 7)]).unique())


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_every_row_of_a_large_store(fp8):
    """Values, keys and the slots that take none, over 5000 tokens; some queries."""
    m = make(5000, 12, 4, seed=12)
    out = torch.full((5000, 12, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    check_store(m, call(m, fp8=fp8, q_out=out), fp8, False, sample=torch.arange(0, 5000, 37))
    assert pkv.get_device_error() == pkv.PKV_OK


@gpu
def test_captured_and_replayed():
    m = make(50, 8, 2, packed=False, seed=13)
    dev = {n: on_gpu(m, n) for n in ("q", "k", "v", "slots", "positions", "cos_sin", "q_weight",
                                     "k_weight")}
    kc = torch.zeros(m["NB"], 256, 2, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    out = torch.empty_like(dev["q"])

    def step():
        pkv.kv_cache_store_norm_rope(dev["q"], dev["k"], dev["v"], kc, vc, dev["slots"],
                                     dev["positions"], dev["cos_sin"], dev["q_weight"],
                                     dev["k_weight"], q_out=out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    other = make(50, 8, 2, packed=False, seed=14)
    for n in ("q", "k", "v", "positions", "slots"):
        dev[n].copy_(other[n])
    kc.zero_()
    vc.zero_()
    graph.replay()
    torch.cuda.synchronize()
    other.update({n: m[n] for n in ("cos_sin", "q_weight", "k_weight")})
    verify(other, (out, kc, vc))


@gpu
def test_wrapper_refusals():
    m = make(6, 4, 2, packed=False, seed=15)
    a = {n: on_gpu(m, n) for n in ("q", "k", "v", "slots", "positions", "cos_sin", "q_weight")}
    kc = torch.zeros(1, 256, 2, 128, dtype=torch.bfloat16, device="cuda")

    def bad(error, **over):
        x = {**a, **over}
        with pytest.raises(error):
            pkv.kv_cache_store_norm_rope(x["q"], x["k"], x["v"], kc, kc.clone(), x["slots"],
                                         x["positions"], x["cos_sin"], x["q_weight"],
                                         q_out=x.get("q_out"))

    bad(TypeError, q=a["q"].float())
    bad(ValueError, q=a["q"].cpu())
    bad(ValueError, k=a["k"][:5])
    bad(ValueError, v=a["v"][:, :1])
    bad(ValueError, q=a["q"].transpose(0, 1).contiguous().transpose(0, 1))
    bad(TypeError, positions=a["positions"].long())
    bad(TypeError, positions=None)
    bad(ValueError, positions=a["positions"][:3])
    bad(ValueError, slots=a["slots"][:3])
    bad(TypeError, q_weight=a["q_weight"].to(torch.bfloat16))
    bad(ValueError, q_weight=a["q_weight"][:64])
    bad(ValueError, cos_sin=a["cos_sin"].cpu())
    bad(pkv.PkvError, cos_sin=a["cos_sin"][:, :24].contiguous())
    bad(ValueError, q_out=a["q"][:3])
    # a packed projection cannot take its own queries back
    row = torch.zeros(6, 8, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        pkv.kv_cache_store_norm_rope(row[:, :4], row[:, 4:6], row[:, 6:], kc, kc.clone(),
                                     a["slots"], a["positions"], a["cos_sin"], q_out=row[:, :4])
    with pytest.raises(pkv.PkvError):   # memory of the projection
        pkv.kv_cache_store_norm_rope(row[:, :4], row[:, 4:6], row[:, 6:], kc, kc.clone(),
                                     a["slots"], a["positions"], a["cos_sin"],
                                     q_out=row.view(-1)[:6 * 512].view(6, 4, 128))


def test_host_refusals():
    B.build()
    lib = pkv.load_library()
    P = 1 << 20   # a stand-in address: the checks below fail before any use

    def store(q_out=P, q=4 * P, k=8 * P, v=12 * P, qs=512, ks=256, vs=256, kc=16 * P, vc=20 * P,
              slots=P, pos=P, cs=P, places=10, rotary=128, qw=P, kw=P, eps=1e-6, T=4, Hq=4, Hkv=2,
              D=128, bs=256, NB=2, scales=None):
        args = (q_out, q, k, v, qs, ks, vs, kc, vc, slots, pos, cs, places, rotary, 0, qw, kw, eps,
                T, Hq, Hkv, D, bs, NB)
        if scales is None:
            return lib.kv_cache_store_norm_rope(*args, None)
        return lib.kv_cache_store_norm_rope_fp8(*args, *scales, None)

    nan, inf = float("nan"), float("inf")
    for kw in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf),
               dict(q_out=None), dict(q=None), dict(k=None), dict(v=None), dict(kc=None),
               dict(vc=None), dict(slots=None), dict(pos=None), dict(cs=None), dict(places=-1),
               dict(qs=511), dict(ks=255), dict(vs=0), dict(q_out=P + 2), dict(kc=16 * P + 8),
               dict(cs=P + 4), dict(qw=P + 8), dict(kw=P + 4),
               dict(q_out=4 * P, qs=1024), dict(q_out=4 * P + 1024), dict(q_out=8 * P),
               dict(q_out=12 * P + 16), dict(q_out=16 * P), dict(q_out=20 * P + 4096)):
        assert store(**kw) == pkv.PKV_ERR_ARG, kw
        if "scales" not in kw:
            assert store(**kw, scales=(1.0, 1.0)) == pkv.PKV_ERR_ARG, kw
    for kw in (dict(D=64), dict(bs=128), dict(rotary=8), dict(rotary=136), dict(rotary=-16),
               dict(Hq=1 << 20, qs=1 << 27), dict(NB=1 << 24)):
        assert store(**kw) == pkv.PKV_ERR_SHAPE, kw
    for s in ((0.0, 1.0), (1.0, -1.0), (nan, 1.0), (1.0, inf)):
        assert store(scales=s) == pkv.PKV_ERR_ARG
    assert store(T=0, q=None, k=None, v=None, q_out=None) == pkv.PKV_OK
    assert store(T=0, q=None, scales=(1.0, 1.0)) == pkv.PKV_OK
