"""A layer's cache path as an engine runs it: packed projections go through the
norm, rotation and store, a prompt is prefilled in chunks, then decode steps
follow, in a layer with capped scores and a window; every output is compared
with a 64-bit computation over contiguous keys that never saw a page."""
import pytest
import torch

import scored_ref as R
from paged_kv_cache_214_gb300 import pkv
from paged_kv_cache_214_gb300.blocks import BlockManager

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS, NB, MAXBLK = 8, 2, 128, 256, 12, 3
CAP, WINDOW, EPS = 20.0, 150, 1e-6


def table(places, rotary):
    angle = torch.arange(places, dtype=torch.float64)[:, None] * torch.pow(
        1e4, -torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_chunks_then_decode_steps(fp8):
    if fp8:   # prompts over E4M3 pages are attended one position at a time
        chunks = []
    else:
        chunks = [200, 97]
    g = torch.Generator().manual_seed(5)
    cos_sin = table(1024, 64)
    qw, kw = (2 + torch.rand(D, generator=g) for _ in range(2))
    scale, ks, vs = D ** -0.5, 0.02, 0.012
    dtype = torch.uint8 if fp8 else torch.bfloat16
    kc = torch.zeros(NB, BS, HKV, D, dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    dev = {n: t.to("cuda") for n, t in (("cos_sin", cos_sin), ("qw", qw), ("kw", kw))}
    bm = BlockManager(NB, BS)
    seqs = (0, 1)
    tokens = {s: list(range(1000 * s, 1000 * s + sum(chunks))) for s in seqs}
    keys = {s: torch.zeros(0, HKV, D, dtype=torch.float64) for s in seqs}
    vals = {s: torch.zeros(0, HKV, D, dtype=torch.float64) for s in seqs}

    def project(n):
        return torch.randn(n, (HQ + 2 * HKV) * D, generator=g).to(torch.bfloat16)

    def store(row, slots, positions):
        """The library's step on a packed projection; returns q, and the stored
        keys and values as the pool holds them."""
        q, k, v = (x.unflatten(1, (-1, D)) for x in
                   row.to("cuda").split([HQ * D, HKV * D, HKV * D], 1))
        args = (q, k, v, kc, vc, slots.to("cuda"), positions.to("cuda"), dev["cos_sin"])
        more = dict(q_weight=dev["qw"], k_weight=dev["kw"], eps=EPS)
        got = (pkv.kv_cache_store_norm_rope_fp8(*args, ks, vs, **more) if fp8
               else pkv.kv_cache_store_norm_rope(*args, **more))
        hq, hk, hv = (x.unflatten(1, (-1, D)) for x in row.split([HQ * D, HKV * D, HKV * D], 1))
        R.check_rows(got, R.norm_rope(hq, qw, EPS, positions, cos_sin, False), "q")
        rk = R.norm_rope(hk, kw, EPS, positions, cos_sin, False)
        at = slots.long()
        k_rows, v_rows = (p.view(-1, HKV, D).cpu()[at] for p in (kc, vc))
        if fp8:
            R.check_codes(k_rows, rk, ks, "k")
            R.check_codes(v_rows, hv.double(), vs, "v")
            k64 = k_rows.view(torch.float8_e4m3fn).double() * ks
            return got, k64, v_rows.view(torch.float8_e4m3fn).double() * vs
        R.check_rows(k_rows, rk, "k")
        return got, k_rows.double(), v_rows.double()

    def check(s, out, lse, q, rows, p_step):
        n = len(keys[s])
        pos = [n - rows + r for r in range(rows)]
        want = R.attend(q.cpu(), keys[s], vals[s], pos, [max(0, i - WINDOW + 1) for i in pos], pos,
                        scale, CAP, None, p_step)
        R.check(out, lse, want, f"sequence {s} at {n}")

    if chunks:
        for s in seqs:
            assert bm.add_sequence(s, tokens[s]) == 0
        done = 0
        for n in chunks:
            slots = torch.cat([torch.from_numpy(bm.slot_mapping(s, done, done + n)) for s in seqs])
            positions = torch.arange(done, done + n, dtype=torch.int32).repeat(2)
            q, k, v = store(project(2 * n), slots.to(torch.int32), positions)
            for i, s in enumerate(seqs):
                keys[s] = torch.cat([keys[s], k[i * n:(i + 1) * n]])
                vals[s] = torch.cat([vals[s], v[i * n:(i + 1) * n]])
            done += n
            cu = lambda m: torch.tensor([0, m, 2 * m], dtype=torch.int32, device="cuda")  # noqa: E731
            tables = torch.from_numpy(bm.block_tables(seqs, MAXBLK)).to("cuda")
            out, lse = pkv.paged_prefill_attention_scored(q, kc, vc, tables, cu(n), cu(done), n, done,
                                                          scale, softcap=CAP, window=WINDOW)
            for i, s in enumerate(seqs):
                part = slice(i * n, (i + 1) * n)
                check(s, out[part], lse[part], q[part], n, 2.0 ** -8)
    else:
        for s in seqs:
            tokens[s] = [7000 + s]
            assert bm.add_sequence(s, tokens[s]) == 0

    for step in range(180 if fp8 else 4):
        if chunks or step:
            slots = torch.tensor([bm.append_token(s, 5000 + 10 * step + s)[0] for s in seqs],
                                 dtype=torch.int32)
        else:
            slots = torch.tensor([int(bm.slot_mapping(s, 0, 1)[0]) for s in seqs],
                                 dtype=torch.int32)
        n = len(keys[0]) + 1
        q, k, v = store(project(2), slots, torch.full((2,), n - 1, dtype=torch.int32))
        for i, s in enumerate(seqs):
            keys[s], vals[s] = torch.cat([keys[s], k[i:i + 1]]), torch.cat([vals[s], v[i:i + 1]])
        tables = torch.from_numpy(bm.block_tables(seqs, MAXBLK)).to("cuda")
        lens = torch.full((2,), n, dtype=torch.int32, device="cuda")
        if fp8:
            out, lse = pkv.paged_decode_attention_scored_fp8(q, kc, vc, tables, lens, scale, ks, vs,
                                                             softcap=CAP, window=WINDOW)
        else:
            out, lse = pkv.paged_decode_attention_scored(q, kc, vc, tables, lens, scale, softcap=CAP,
                                                         window=WINDOW)
        if not fp8 or step % 20 in (0, 19):
            for i, s in enumerate(seqs):
                check(s, out[i:i + 1], lse[i:i + 1], q[i:i + 1], 1, 2.0 ** -16)
    assert pkv.get_device_error() == pkv.PKV_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_past_32_bits(fp8):
    """The same step over the first pages of a small pool and over the last pages of
    one whose byte offsets pass 2^32 (and elements 2^31): equal results, bit for bit."""
    hkv = 8
    dtype, far = (torch.uint8, 16500) if fp8 else (torch.bfloat16, 8300)   # 2^18 values a page
    g = torch.Generator().manual_seed(6)
    T = 600
    q, k, v = (torch.randn(T, h, D, generator=g).to(torch.bfloat16).cuda()
               for h in (HQ, hkv, hkv))
    place = torch.arange(T, dtype=torch.int32)
    cos_sin = table(T, D).cuda()
    order = torch.tensor([2, 0, 1])
    results = []
    for blocks in (3, far):
        ids = (blocks - 3 + order).to(torch.int32)
        kc, vc = (torch.empty(blocks, BS, hkv, D, dtype=dtype, device="cuda") for _ in range(2))
        kc[-3:] = 0   # (compared whole below)
        vc[-3:] = 0
        slots = (ids[place.long() // BS] * BS + place % BS).cuda()
        args = (q, k, v, kc, vc, slots, place.cuda(), cos_sin)
        rotated = (pkv.kv_cache_store_norm_rope_fp8(*args, 0.02, 0.02) if fp8
                   else pkv.kv_cache_store_norm_rope(*args))
        row, lens = ids[None].cuda(), torch.tensor([T], dtype=torch.int32, device="cuda")
        last = rotated[-1:].contiguous()
        got = [rotated, kc[-3:].clone(), vc[-3:].clone()]
        if fp8:
            got += pkv.paged_decode_attention_scored_fp8(last, kc, vc, row, lens, 0.1, 0.02, 0.02,
                                                         softcap=CAP, window=400)
        else:
            got += pkv.paged_decode_attention_scored(last, kc, vc, row, lens, 0.1, softcap=CAP)
            cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
            got += pkv.paged_prefill_attention_scored(rotated, kc, vc, row, cu, cu, T, T, 0.1,
                                                      softcap=CAP, window=400)
        torch.cuda.synchronize()
        results.append(got)
        del kc, vc
    assert int(slots.max()) * hkv * D > 2 ** 31
    for near, distant in zip(*results):
        assert torch.equal(near, distant)
    assert pkv.get_device_error() == pkv.PKV_OK
