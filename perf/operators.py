"""Cases of the cache's layer operators: the fused query/key norm, rotation and
store, and paged attention whose scores are capped, biased by distance or
restricted by a window, documents or a prefix.

A case is a dict of plain values.  `run` computes it either in plain torch
operations (`own` false) or through the library's calls (`own` true)."""

import math
import random

import torch

own = False

D = 128          # head dimension of the pools
BLOCK = 256      # tokens of a page
E4M3_MAX = 448.0


def _heads(case):
    return case["Hq"], case["Hkv"]


def _spread(lo, hi, n, seed):
    """n lengths from [lo, hi], the same for everybody who asks with this seed."""
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(n)]


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # the step of a single stream: one token, its row of the packed projection
        _store("store-1", T=1, Hq=16, Hkv=8, lens_seed=1),
        # a decode step of 64 streams over E4M3 pages
        _store("store-b64-fp8", T=64, Hq=16, Hkv=8, fp8=True, lens_seed=2),
        # the prefill chunk of 16 prompts, 512 new tokens each
        _store("store-chunk-b16", T=8192, Hq=32, Hkv=8, lens_seed=3),
        # half of each head rotated in adjacent pairs, separate projections, padding rows
        _store("store-odd", T=1777, Hq=12, Hkv=4, rotary=64, interleaved=True, packed=False,
               padded=True, fp8=True, lens_seed=4),
        # four short streams of a model with capped scores: latency
        _decode("decode-tiny-cap", lens="17,256,300,513", Hq=16, Hkv=8, softcap=50.0),
        # 64 streams of a model with capped scores
        _decode("decode-b64-cap", B=64, lo=512, hi=4096, Hq=16, Hkv=8, softcap=50.0, lens_seed=5),
        # 64 streams in a layer that looks back 1000 tokens, with a distance bias
        _decode("decode-b64-window", B=64, lo=512, hi=8192, Hq=32, Hkv=8, window=1000, alibi=True,
                lens_seed=6),
        # long contexts over E4M3 pages, capped
        _decode("decode-long-b8-cap-fp8", B=8, lo=32768, hi=131072, Hq=32, Hkv=8, softcap=30.0,
                fp8=True, lens_seed=7),
        # chunked prefill of 16 prompts: 1024 cached tokens, 512 new ones, capped
        _prefill("prefill-b16-cap", B=16, new_lo=512, new_hi=512, old_lo=1024, old_hi=1024, Hq=32,
                 Hkv=8, softcap=50.0, lens_seed=8),
        # one long prompt in a layer that looks back 1024 tokens
        _prefill("prefill-long-window", B=1, new_lo=8192, new_hi=8192, old_lo=0, old_hi=0, Hq=16,
                 Hkv=8, window=1024, lens_seed=9),
        # prompts whose beginning is read in both directions, ragged, with a distance bias
        _prefill("prefill-prefix-ragged", B=6, new_lo=90, new_hi=900, old_lo=0, old_hi=0, Hq=12,
                 Hkv=4, prefix=True, alibi=True, lens_seed=10),
        # documents that do not see one another and a question that sees them all, capped
        _prefill("prefill-documents-cap", B=2, new_lo=1500, new_hi=2500, old_lo=100, old_hi=300,
                 Hq=32, Hkv=8, documents=5, softcap=30.0, lens_seed=11),
    ]


def _store(name, *, T, Hq, Hkv, lens_seed, rotary=128, interleaved=False, packed=True,
           padded=False, fp8=False, norm=True):
    return {"name": name, "op": "store", "T": T, "Hq": Hq, "Hkv": Hkv, "rotary": rotary,
            "interleaved": interleaved, "packed": packed, "padded": padded, "fp8": fp8,
            "norm": norm, "lens_seed": lens_seed}


def _decode(name, *, Hq, Hkv, B=0, lo=0, hi=0, lens="", softcap=0.0, alibi=False, window=0,
            documents=False, fp8=False, lens_seed=0):
    return {"name": name, "op": "decode", "Hq": Hq, "Hkv": Hkv, "B": B, "lo": lo, "hi": hi,
            "lens": lens, "softcap": softcap, "alibi": alibi, "window": window,
            "documents": documents, "fp8": fp8, "lens_seed": lens_seed}


def _prefill(name, *, B, new_lo, new_hi, old_lo, old_hi, Hq, Hkv, softcap=0.0, alibi=False,
             window=0, documents=0, prefix=False, lens_seed=0):
    return {"name": name, "op": "prefill", "B": B, "new_lo": new_lo, "new_hi": new_hi,
            "old_lo": old_lo, "old_hi": old_hi, "Hq": Hq, "Hkv": Hkv, "softcap": softcap,
            "alibi": alibi, "window": window, "documents": documents, "prefix": prefix,
            "lens_seed": lens_seed}


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "decode", "prefill"])
    Hq, Hkv = rng.choice([(16, 8), (32, 8), (12, 4), (14, 2), (5, 1), (64, 8), (6, 6)])
    seed = rng.randrange(1 << 20)
    if op == "store":
        c = _store("", T=_log_int(rng, 1, 12000), Hq=Hq, Hkv=Hkv, rotary=rng.choice([128, 128, 96, 64, 32]),
                   interleaved=rng.random() < 0.4, packed=rng.random() < 0.6,
                   padded=rng.random() < 0.3, fp8=rng.random() < 0.4, norm=rng.random() < 0.8,
                   lens_seed=seed)
    elif op == "decode":
        B = _log_int(rng, 1, 128)
        fp8 = rng.random() < 0.4
        most = 1000000000 // (B * Hkv * D * (2 if fp8 else 4))   # tokens of a stream
        hi = _log_int(rng, 16, min(100000, most))
        c = _decode("", B=B, lo=max(1, hi // rng.choice([1, 2, 8])), hi=hi, Hq=Hq, Hkv=Hkv,
                    softcap=rng.choice([0.0, 20.0, 30.0, 50.0]), alibi=rng.random() < 0.3,
                    window=rng.choice([0, 0, _log_int(rng, 16, 8192)]),
                    documents=rng.random() < 0.25, fp8=fp8, lens_seed=seed)
    else:
        B = _log_int(rng, 1, 16)
        old = rng.choice([0, _log_int(rng, 1, 2048)])
        most = 300000000 // (Hq * B)   # (row, key) pairs of a prompt and head
        new = _log_int(rng, 1, min(4096, int(math.sqrt(most + old * old / 4) - old / 2)))
        documents = rng.choice([0, 0, rng.randint(2, 9)])
        c = _prefill("", B=B, new_lo=max(1, new // rng.choice([1, 2, 8])), new_hi=new,
                     old_lo=old // 2, old_hi=old, Hq=Hq, Hkv=Hkv,
                     softcap=rng.choice([0.0, 20.0, 30.0, 50.0]), alibi=rng.random() < 0.3,
                     window=rng.choice([0, 0, _log_int(rng, 16, 4096)]), documents=documents,
                     prefix=rng.random() < 0.25, lens_seed=seed)
    del c["name"]
    return c


# ------------------------------------------------- lengths, which the case alone sets

def _decode_lens(case):
    if case["lens"]:
        return [int(x) for x in case["lens"].split(",")]
    return _spread(case["lo"], case["hi"], case["B"], case["lens_seed"])


def _decode_first(case, lens):
    """First key of each stream's own document."""
    if not case["documents"]:
        return None
    r = random.Random(case["lens_seed"] + 1)
    return [r.randint(0, n - 1) for n in lens]


def _prefill_lens(case):
    new = _spread(case["new_lo"], case["new_hi"], case["B"], case["lens_seed"])
    old = _spread(case["old_lo"], case["old_hi"], case["B"], case["lens_seed"] + 1)
    return new, old


def _prefill_first(case, new, old):
    """First key of each new row: `documents` documents of the new tokens, each
    blind to the others, and a last tenth of the rows that sees everything."""
    if not case["documents"]:
        return None
    r = random.Random(case["lens_seed"] + 2)
    rows = []
    for n, o in zip(new, old):
        tail = n - n // 10
        cuts = sorted(r.randint(0, max(0, tail - 1)) for _ in range(case["documents"] - 1))
        first, at = [], 0
        for i in range(n):
            while cuts and i >= cuts[0]:
                at = o + cuts.pop(0)
            first.append(at if i < tail else 0)
        rows += first
    return rows


def _prefill_prefix(case, new, old):
    """Tokens at the beginning of each prompt that are read in both directions."""
    if not case["prefix"]:
        return None
    r = random.Random(case["lens_seed"] + 3)
    return [r.randint(0, n + o) for n, o in zip(new, old)]


def _bounds(case, new, old):
    """(first key, last key) of every new row, as two lists."""
    first = _prefill_first(case, new, old)
    prefix = _prefill_prefix(case, new, old)
    lo, hi, row = [], [], 0
    for b, (n, o) in enumerate(zip(new, old)):
        for r in range(n):
            i = o + r
            l = max(0, i - case["window"] + 1) if case["window"] else 0
            lo.append(max(l, first[row]) if first else l)
            hi.append(max(i, prefix[b] - 1) if prefix else i)
            row += 1
    return lo, hi


# ------------------------------------------------------------------------ work

def work(case):
    Hq, Hkv = _heads(case)
    if case["op"] == "store":
        T, e = case["T"], 1 if case["fp8"] else 2
        stored = T - (T // 7 if case["padded"] else 0)
        read = T * (Hq * D * 2 + 8 + 4 * case["rotary"]) + stored * 2 * Hkv * D * 2
        return {"bytes": read + T * Hq * D * 2 + stored * 2 * Hkv * D * e,
                "flops": 8 * T * (Hq + Hkv) * D}
    if case["op"] == "decode":
        lens = _decode_lens(case)
        first = _decode_first(case, lens) or [0] * len(lens)
        keys = sum(n - max(f, n - case["window"] if case["window"] else 0)
                   for n, f in zip(lens, first))
        e = 1 if case["fp8"] else 2
        pages = sum(-(-n // BLOCK) for n in lens)
        return {"bytes": keys * Hkv * D * 2 * e + len(lens) * Hq * (D * 4 + 4) + 4 * pages,
                "flops": 4 * D * Hq * keys}
    new, old = _prefill_lens(case)
    lo, hi = _bounds(case, new, old)
    pairs = sum(max(0, h - l + 1) for l, h in zip(lo, hi))
    tokens, at = 0, 0
    for n, o in zip(new, old):
        tokens += o + n - min(lo[at:at + n])
        at += n
    rows = sum(new)
    return {"bytes": tokens * Hkv * D * 4 + rows * Hq * (D * 4 + 4), "flops": 4 * D * Hq * pairs}


# --------------------------------------------------------------------- prepare

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(lens, gen, spare=3):
    """A page table whose pages are scattered over the pool, and the pool's size."""
    pages = [-(-n // BLOCK) for n in lens]
    total = sum(pages) + spare
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _pool(pages, Hkv, fp8, gen):
    shape = (pages, BLOCK, Hkv, D)
    if not fp8:
        return [torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
                for _ in range(2)]
    codes = []
    for _ in range(2):
        x = torch.empty(shape, dtype=torch.uint8, device="cuda")
        for p in range(0, pages, 512):   # a few pages at a time
            part = torch.randn((min(512, pages - p),) + shape[1:], generator=gen, device="cuda")
            x[p:p + 512] = (part * (E4M3_MAX / 6)).clamp(-E4M3_MAX, E4M3_MAX).to(
                torch.float8_e4m3fn).view(torch.uint8)
        codes.append(x)
    return codes


def _slopes(Hq):
    """One slope for each head, a geometric series that ends at 2^-8."""
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    Hq, Hkv = _heads(case)
    s = dict(case)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    if case["op"] == "store":
        T = case["T"]
        pages = max(1, -(-T * 5 // (4 * BLOCK)))
        if case["packed"]:   # one projection's output holds a token's q, k and v
            row = randn(T, (Hq + 2 * Hkv) * D).to(torch.bfloat16)
            q, k, v = (x.view(T, -1, D) for x in row.split([Hq * D, Hkv * D, Hkv * D], dim=1))
        else:
            q, k, v = (randn(T, h, D).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        slots = torch.randperm(pages * BLOCK, generator=gen, device="cuda")[:T].to(torch.int32)
        if case["padded"]:   # rows behind the last sequence of a padded batch
            slots[T - T // 7:] = -1
        positions = 32768
        R = case["rotary"]
        angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * torch.pow(
            1e6, -torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["positions"] = torch.randint(0, positions, (T,), generator=gen, device="cuda",
                                       dtype=torch.int32)
        s.update(q=q, k=k, v=v, slots=slots, q_weight=None, k_weight=None)
        if case["norm"]:
            s["q_weight"] = 1 + 0.2 * randn(D)
            s["k_weight"] = 1 + 0.2 * randn(D)
        dtype = torch.uint8 if case["fp8"] else torch.bfloat16
        s["k_cache"] = torch.zeros(pages, BLOCK, Hkv, D, dtype=dtype, device="cuda")
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        s["k_scale"] = s["v_scale"] = 6.0 / E4M3_MAX
        s["inverse"] = (1 / torch.tensor(6.0 / E4M3_MAX)).item()   # in 32 bits
        return s
    s["scale"] = D ** -0.5
    s["slopes"] = _slopes(Hq) if case["alibi"] else None
    # scores of a few units, as trained heads have them
    spread = 3.0 if case["softcap"] else 1.5
    if case["op"] == "decode":
        lens = _decode_lens(case)
        first = _decode_first(case, lens)
        s["table"], pages = _tables(lens, gen)
        s["lens"] = _ints(lens)
        s["first"] = _ints(first) if first else None
        s["longest"] = max(lens)
        s["q"] = (spread * randn(len(lens), Hq, D)).to(torch.bfloat16)
        s["k_cache"], s["v_cache"] = _pool(pages, Hkv, case["fp8"], gen)
        s["k_scale"], s["v_scale"] = 6.0 / E4M3_MAX, 5.0 / E4M3_MAX
        return s
    new, old = _prefill_lens(case)
    total = [n + o for n, o in zip(new, old)]
    first, prefix = _prefill_first(case, new, old), _prefill_prefix(case, new, old)
    s["table"], pages = _tables(total, gen)
    s["first"] = _ints(first) if first else None
    s["prefix_lens"] = _ints(prefix) if prefix else None
    cu = lambda v: _ints([sum(v[:i]) for i in range(len(v) + 1)])  # noqa: E731
    s["cu_q"], s["cu_k"] = cu(new), cu(total)
    s["longest_q"], s["longest_k"] = max(new), max(total)
    s["q"] = (spread * randn(sum(new), Hq, D)).to(torch.bfloat16)
    s["k_cache"], s["v_cache"] = _pool(pages, Hkv, False, gen)
    return s


# ------------------------------------------------------------------------- run

def run(s):
    if own:
        return _own(s)
    return {"store": _plain_store, "decode": _plain_decode, "prefill": _plain_prefill}[s["op"]](s)


def _own(s):
    from paged_kv_cache_214_gb300 import pkv

    if s["op"] == "store":
        more = {"q_weight": s["q_weight"], "k_weight": s["k_weight"], "eps": 1e-6,
                "interleaved": s["interleaved"]}
        args = (s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                s["cos_sin"])
        if s["fp8"]:
            q = pkv.kv_cache_store_norm_rope_fp8(*args, s["k_scale"], s["v_scale"], **more)
            return [q, _values(s["k_cache"]), _values(s["v_cache"])]
        return [pkv.kv_cache_store_norm_rope(*args, **more), s["k_cache"], s["v_cache"]]
    more = {"softcap": s["softcap"], "alibi_slopes": s["slopes"], "window": s["window"],
            "first_keys": s["first"]}
    args = (s["q"], s["k_cache"], s["v_cache"], s["table"])
    if s["op"] == "decode":
        if s["fp8"]:
            return pkv.paged_decode_attention_scored_fp8(*args, s["lens"], s["scale"], s["k_scale"],
                                                         s["v_scale"], **more)
        return pkv.paged_decode_attention_scored(*args, s["lens"], s["scale"], **more)
    return pkv.paged_prefill_attention_scored(*args, s["cu_q"], s["cu_k"], s["longest_q"],
                                              s["longest_k"], s["scale"],
                                              prefix_lens=s["prefix_lens"], **more)


def _values(codes):
    return codes.view(torch.float8_e4m3fn)


def _normed(x, weight):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight


def _rotated(x, s):
    R = s["rotary"]
    table = s["cos_sin"][s["positions"].long()]
    c, n = table[:, None, :R // 2], table[:, None, R // 2:]
    if s["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_store(s):
    Hkv = s["Hkv"]
    q = _rotated(_normed(s["q"], s["q_weight"]), s).to(torch.bfloat16)
    k = _rotated(_normed(s["k"], s["k_weight"]), s)
    v = s["v"]
    # padding rows have the slot -1 and come last
    kept = s["slots"] >= 0
    slots = s["slots"][kept].long()
    k, v = k[kept], v[kept]
    if s["fp8"]:
        k, v = ((x.float() * s["inverse"]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
                .view(torch.uint8) for x in (k, v))
    else:
        k = k.to(torch.bfloat16)
    s["k_cache"].view(-1, Hkv, D)[slots] = k
    s["v_cache"].view(-1, Hkv, D)[slots] = v
    if s["fp8"]:
        return [q, _values(s["k_cache"]), _values(s["v_cache"])]
    return [q, s["k_cache"], s["v_cache"]]


def _gathered(cache, table, longest, scale, fp8):
    """Every stream's keys or values in fp32, [B, Hkv, tokens, D]."""
    x = cache[table[:, :-(-longest // BLOCK)].long().clamp(min=0)].flatten(1, 2)[:, :longest]
    x = (_values(x).float() * scale if fp8 else x.float())
    return x.transpose(1, 2)


def _attended(scores, seen, v):
    """(output, log-sum-exp) of scores [..., rows, keys] where `seen`; a row that
    sees nothing gives 0 and -inf."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, torch.ones_like(total))
    return out, (torch.log(total) + top).squeeze(-1)


def _modified(scores, s, distance):
    """Cap and distance bias of scores [B, Hkv, g, rows, keys]."""
    if s["softcap"]:
        scores = s["softcap"] * torch.tanh(scores / s["softcap"])
    if s["slopes"] is not None:
        g = s["Hq"] // s["Hkv"]
        scores = scores - s["slopes"].view(-1, g, 1, 1) * distance[:, None, None]
    return scores


def _plain_decode(s):
    Hq, Hkv = _heads(s)
    B, n = s["q"].shape[0], s["longest"]
    k = _gathered(s["k_cache"], s["table"], n, s["k_scale"], s["fp8"])
    v = _gathered(s["v_cache"], s["table"], n, s["v_scale"], s["fp8"])
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    scores = (q @ k.transpose(2, 3) * s["scale"])[:, :, :, None]     # [B, Hkv, g, 1, n]
    j = torch.arange(n, device="cuda")[None, None]
    i = (s["lens"] - 1)[:, None, None]
    scores = _modified(scores, s, (i - j).abs().float())
    seen = j <= i
    if s["window"]:
        seen = seen & (i - j < s["window"])
    if s["first"] is not None:
        seen = seen & (j >= s["first"][:, None, None])
    out, lse = _attended(scores[:, :, :, 0], seen[:, None], v)
    return out.reshape(B, Hq, D).to(torch.bfloat16), lse.reshape(B, Hq)


def _plain_prefill(s):
    Hq, Hkv = _heads(s)
    nq, nk = s["longest_q"], s["longest_k"]
    k = _gathered(s["k_cache"], s["table"], nk, 1.0, False)
    v = _gathered(s["v_cache"], s["table"], nk, 1.0, False)
    B, rows = k.shape[0], s["q"].shape[0]
    # rows of the packed batch, padded to the longest chunk
    r = torch.arange(nq, device="cuda")
    at = s["cu_q"][:-1, None] + r
    new = (s["cu_q"][1:] - s["cu_q"][:-1])[:, None]
    total = (s["cu_k"][1:] - s["cu_k"][:-1])[:, None]
    at = at.clamp(max=rows - 1).long()
    q = s["q"].float()[at].view(B, nq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    scores = q @ k.transpose(2, 3)[:, :, None] * s["scale"]          # [B, Hkv, g, nq, nk]
    j = torch.arange(nk, device="cuda")
    i = total - new + r
    distance = (i[:, :, None] - j).abs().float()
    scores = _modified(scores, s, distance)
    seen = j <= i[:, :, None]
    if s["prefix_lens"] is not None:
        seen = seen | (j < s["prefix_lens"][:, None, None])
    if s["window"]:
        seen = seen & (i[:, :, None] - j < s["window"])
    if s["first"] is not None:
        seen = seen & (j >= s["first"][at][:, :, None])
    out, lse = _attended(scores, (seen & (j < total[:, :, None]))[:, None, None], v[:, :, None])
    # back to the packed rows
    t = torch.arange(rows, device="cuda")
    b = torch.searchsorted(s["cu_q"][1:].long().contiguous(), t, right=True)
    row = t - s["cu_q"][b].long()
    out = out.permute(0, 3, 1, 2, 4)[b, row].reshape(rows, Hq, D)
    lse = lse.permute(0, 3, 1, 2)[b, row].reshape(rows, Hq)
    return out.to(torch.bfloat16), lse.contiguous()


# ----------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "store":
        return _exact_store(case, s)
    if case["op"] == "decode":
        lens = _decode_lens(case)
        first = _decode_first(case, lens) or [0] * len(lens)
        lo = [max(f, n - case["window"] if case["window"] else 0) for n, f in zip(lens, first)]
        per_stream = [(b, [n - 1], [l], [n - 1]) for b, (n, l) in enumerate(zip(lens, lo))]
    else:
        new, old = _prefill_lens(case)
        lo, hi = _bounds(case, new, old)
        per_stream, at = [], 0
        for b, (n, o) in enumerate(zip(new, old)):
            per_stream.append((b, list(range(o, o + n)), lo[at:at + n], hi[at:at + n]))
            at += n
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    g = case["Hq"] // case["Hkv"]
    row = 0
    for b, where, lo, hi in per_stream:
        for r0 in range(0, len(where), 1024):
            i, l, h = (torch.tensor(x[r0:r0 + 1024], device="cuda") for x in (where, lo, hi))
            begin, end = int(l.min()), int(h.max()) + 1
            j = torch.arange(begin, end, device="cuda")
            slot = s["table"][b].long()[j // BLOCK] * BLOCK + j % BLOCK
            keys, vals = (_wide(s[c].view(-1, case["Hkv"], D)[slot], s, c) for c in
                          ("k_cache", "v_cache"))
            outside = (j < l[:, None]) | (j > h[:, None])
            for head in range(case["Hq"]):
                q = s["q"][row + r0:row + r0 + len(i), head].double()
                z = torch.einsum("rd,jd->rj", q, keys[:, head // g]) * s["scale"]
                if case["softcap"]:
                    z = torch.tanh(z / case["softcap"]) * case["softcap"]
                if case["alibi"]:
                    z = z - (i[:, None] - j).abs() * s["slopes"][head].double()
                z[outside] = -math.inf
                norm = torch.logsumexp(z, 1)
                lse[row + r0:row + r0 + len(i), head] = norm
                w = torch.exp(z - norm.masked_fill(norm == -math.inf, 0.0)[:, None])
                out[row + r0:row + r0 + len(i), head] = w @ vals[:, head // g]
        row += len(where)
    return out, lse


def _wide(x, s, cache):
    if x.dtype == torch.uint8:
        return x.view(torch.float8_e4m3fn).double() * s["k_scale" if cache == "k_cache" else "v_scale"]
    return x.double()


def _exact_store(case, s):
    T, R = case["T"], case["rotary"]
    half = R // 2
    turn = torch.eye(D, dtype=torch.float64, device="cuda").repeat(T, 1, 1)   # [T, to, from]
    table = s["cos_sin"][s["positions"].long()].double()
    for p in range(half):
        a, b = (2 * p, 2 * p + 1) if case["interleaved"] else (p, p + half)
        c, n = table[:, p], table[:, half + p]
        turn[:, a, a], turn[:, a, b], turn[:, b, a], turn[:, b, b] = c, -n, n, c

    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + 1e-6) * weight.double()
        return torch.einsum("tab,thb->tha", turn, x)

    q, k = turned(s["q"], s["q_weight"]), turned(s["k"], s["k_weight"])
    pools = []
    for x, scale in ((k, s["k_scale"]), (s["v"].double(), s["v_scale"])):
        pool = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda")
        if case["fp8"]:
            x = (x / scale).clamp(-E4M3_MAX, E4M3_MAX)
        kept = s["slots"] >= 0
        pool.view(-1, case["Hkv"], D)[s["slots"][kept].long()] = x[kept]
        pools.append(pool)
    return [q, *pools]
