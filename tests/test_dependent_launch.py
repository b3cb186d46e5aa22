"""Kernels that may start before the stream's previous kernel has ended: what they
read is written while they are resident, so none of their loads may take the
read-only path (whose data must not change during the kernel's life), and a step's
decode sees what the store in front of it has just written."""
import os
import re

import pytest
import torch

from paged_kv_cache_214_gb300 import pkv

CSRC = os.path.join(os.path.dirname(os.path.abspath(pkv.__file__)), "csrc")


def test_early_kernels_do_not_read_through_the_read_only_path():
    early = []
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            source = re.sub(r"//[^\n]*", "", f.read())
        if "griddepcontrol.wait" in source:
            early.append(name)
            assert "__ldg(" not in source and "ld.global.nc" not in source, name
    assert {"decode_kernel.cuh", "norm_rope.cu"} <= set(early)


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("call", ["plain", "capped", "window"])
def test_steps_without_a_pause_equal_steps_one_by_one(call, fp8):
    """Sixty steps of store (queries rotated in place) and decode over one query
    buffer, launched without a pause, then again with one after every call."""
    B, Hq, Hkv, D, steps, first = 32, 16, 8, 128, 60, 250
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = torch.randn(steps, B, Hq + 2 * Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randperm(2 * B, generator=g, device="cuda").to(torch.int32).view(B, 2)
    angle = torch.rand(512, 64, generator=g, device="cuda") * 6.28
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1)
    weight = 1 + torch.rand(D, generator=g, device="cuda")
    dtype = torch.uint8 if fp8 else torch.bfloat16

    def run(pause):
        kc = torch.zeros(2 * B, 256, Hkv, D, dtype=dtype, device="cuda")
        vc = torch.zeros_like(kc)
        q = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
        got = []
        for t in range(steps):
            at = first + t
            slots = table[:, at // 256] * 256 + at % 256
            places = torch.full((B,), at, dtype=torch.int32, device="cuda")
            lens = places + 1
            q.copy_(rows[t, :, :Hq])
            args = (q, rows[t, :, Hq:Hq + Hkv], rows[t, :, Hq + Hkv:], kc, vc, slots, places,
                    cos_sin)
            more = dict(q_weight=weight, k_weight=weight, q_out=q)
            pause()
            if fp8:
                pkv.kv_cache_store_norm_rope_fp8(*args, 0.02, 0.02, **more)
            else:
                pkv.kv_cache_store_norm_rope(*args, **more)
            pause()
            args = (q, kc, vc, table, lens, 0.1) + ((0.02, 0.02) if fp8 else ())
            if call == "plain":
                step = (pkv.paged_decode_attention_fp8 if fp8 else pkv.paged_decode_attention)(*args)
            else:
                opt = dict(softcap=20.0) if call == "capped" else dict(window=40)
                step = (pkv.paged_decode_attention_scored_fp8 if fp8
                        else pkv.paged_decode_attention_scored)(*args, **opt)
            pause()
            got.append(step)
        torch.cuda.synchronize()
        return got

    for (a, la), (b, lb) in zip(run(lambda: None), run(torch.cuda.synchronize)):
        assert torch.equal(a, b) and torch.equal(la, lb)
    assert pkv.get_device_error() == pkv.PKV_OK


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_captured_steps_equal_steps_one_by_one(fp8):
    """Four steps of store and decode in one graph, over buffers that change between
    replays."""
    B, Hq, Hkv, D, steps = 24, 16, 8, 128, 4
    g = torch.Generator(device="cuda").manual_seed(4)
    table = torch.randperm(2 * B, generator=g, device="cuda").to(torch.int32).view(B, 2)
    angle = torch.rand(512, 64, generator=g, device="cuda") * 6.28
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1)
    rows = torch.empty(steps, B, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    first = torch.empty(B, dtype=torch.int32, device="cuda")
    dtype = torch.uint8 if fp8 else torch.bfloat16
    kc = torch.zeros(2 * B, 256, Hkv, D, dtype=dtype, device="cuda")
    vc = torch.zeros_like(kc)
    q = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    outs = [torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
    lses = [torch.empty(B, Hq, device="cuda") for _ in range(steps)]
    need = pkv.paged_decode_scored_workspace_bytes(B, Hq, Hkv, D, 2, fp8=fp8, num_splits=2)
    ws = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")

    def run(pause=lambda: None):
        for t in range(steps):
            places = first + t
            page = (places // 256).long()
            slots = table.gather(1, page[:, None])[:, 0] * 256 + places % 256
            lens = places + 1
            pause()
            args = (rows[t, :, :Hq], rows[t, :, Hq:Hq + Hkv], rows[t, :, Hq + Hkv:], kc, vc, slots,
                    places, cos_sin)
            if fp8:
                pkv.kv_cache_store_norm_rope_fp8(*args, 0.02, 0.02, q_out=q)
            else:
                pkv.kv_cache_store_norm_rope(*args, q_out=q)
            pause()
            more = dict(softcap=20.0, out=outs[t], lse=lses[t], workspace=ws, num_splits=2)
            if fp8:
                pkv.paged_decode_attention_scored_fp8(q, kc, vc, table, lens, 0.1, 0.02, 0.02, **more)
            else:
                pkv.paged_decode_attention_scored(q, kc, vc, table, lens, 0.1, **more)
            pause()

    def fill(seed):
        h = torch.Generator(device="cuda").manual_seed(seed)
        rows.copy_(torch.randn(rows.shape, generator=h, device="cuda"))
        first.copy_(torch.randint(200, 500, (B,), generator=h, device="cuda"))
        pool = torch.randn(kc.shape, generator=h, device="cuda")
        kc.copy_((pool * 40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8
                 else pool)
        vc.copy_(kc.flip(0))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    for seed in (1, 2, 3):
        fill(seed)
        run(torch.cuda.synchronize)
        want = [x.clone() for x in (*outs, *lses, kc, vc)]
        fill(seed)
        for x in (*outs, *lses):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*outs, *lses, kc, vc), want):
            assert torch.equal(a, b)
    assert pkv.get_device_error() == pkv.PKV_OK
