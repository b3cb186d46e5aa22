"""Plain 64-bit definitions of the norm / rotation / store and of scored
attention, with the error that the kernels' arithmetic may leave.

Bounds.  A value rounded to bf16 is off by at most 2^-8 of itself (2^-4 for
E4M3, at least 2^-10, half its smallest step).  A score is a sum of 128 products
in fp32: 128 roundings of at most 2^-23 of the sum of |q k| (tensor cores may
truncate), and a handful more of the score, the cap and the bias (2^-24 each;
the cap is exact to a few 2^-24 of itself or, above 1000, to 2^-19 of the score:
its polynomial's relative error is 1.05e-6).  A score off by d changes a key's
weight by the factor e^d, and so the output by at most sum_j w_j d_j (|v_j| +
|out|) and the log-sum-exp by at most sum_j w_j d_j, to first order.  The
prefill rounds its weights to bf16, which adds 2^-8 sum_j w_j |v_j|; the decode
carries them with 16 bits or more: 2^-16 sum_j w_j |v_j|.  A weight below the
smallest normal fp32 number may be dropped: 2^-126 sum_j |v_j|."""
from __future__ import annotations

import math

import torch

E4M3_MAX = 448.0


def to64(x):
    return x.detach().cpu().double()


def gather(pool, table_row, length):
    """Rows [length, Hkv, D] of one sequence, in 64 bits (bf16 pool, or E4M3 codes)."""
    bs = pool.shape[1]
    j = torch.arange(length)
    slots = table_row.long()[j // bs] * bs + j % bs if length else j
    rows = pool.reshape(-1, *pool.shape[2:])[slots]
    if pool.dtype == torch.uint8:
        rows = rows.view(torch.float8_e4m3fn).float()
    return rows.double()


def attend(q, k, v, pos, first, last, scale, softcap=0.0, slopes=None, p_step=2.0 ** -16):
    """q [R, Hq, D]; k, v [L, Hkv, D]; pos / first / last: ints [R].  Returns
    out [R, Hq, D], lse [R, Hq] and the errors allowed for both."""
    R, Hq, D = q.shape
    g = Hq // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out = torch.zeros(R, Hq, D, dtype=torch.float64)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(R):
        lo, hi = max(0, int(first[r])), int(last[r])
        if lo > hi:
            continue
        kk, vv = k[lo:hi + 1], v[lo:hi + 1]
        dist = (int(pos[r]) - torch.arange(lo, hi + 1)).abs().double()
        for h in range(Hq):
            kh, vh = kk[:, h // g], vv[:, h // g]
            s = kh @ q[r, h] * scale
            err = 2.0 ** -23 * 136 * scale * (kh.abs() @ q[r, h].abs())
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                err = err + 2.0 ** -21 * min(softcap, 1000.0) + 2.0 ** -19 * s.abs()
            if slopes is not None:
                bias = slopes[h].item() * dist
                s = s - bias
                err = err + 2.0 ** -22 * bias
            err = err + 2.0 ** -22 * s.abs() + 2.0 ** -20
            z = torch.logsumexp(s, 0)
            w = torch.exp(s - z)
            o = w @ vh
            off = float(w @ err)
            out[r, h], lse[r, h] = o, z
            tol_o[r, h] = (2.0 ** -8 * o.abs() + p_step * (w @ vh.abs())
                           + (w * err) @ vh.abs() + off * o.abs()) * 1.001
            tol_o[r, h] += 2.0 ** -126 * vh.abs().sum(0)
            tol_l[r, h] = off + 2.0 ** -21 * (1 + abs(float(z)))
    return out, lse, tol_o, tol_l


def check(out, lse, want, what=""):
    o, z, tol_o, tol_l = want
    out, lse = to64(out), to64(lse)
    over = (out - o).abs() - tol_o
    assert not torch.isnan(out).any(), f"{what}: NaN in out"
    assert over.max().item() <= 0, f"{what}: out is {over.max().item()} past its bound"
    fin = torch.isfinite(z)
    assert torch.equal(lse[~fin], z[~fin]), f"{what}: lse of empty rows"
    if fin.any():
        over = ((lse - z).abs() - tol_l)[fin]
        assert over.max().item() <= 0, f"{what}: lse is {over.max().item()} past its bound"


def decode(q, kc, vc, tables, lens, scale, softcap=0.0, slopes=None, window=0, first_keys=None,
           k_scale=1.0, v_scale=1.0):
    """Reference of paged_decode_attention_scored over host tensors."""
    parts = []
    for b in range(q.shape[0]):
        n = int(lens[b])
        k, v = gather(kc, tables[b], n) * k_scale, gather(vc, tables[b], n) * v_scale
        lo = max(0, n - window) if window else 0
        if first_keys is not None:
            lo = max(lo, int(first_keys[b]))
        parts.append(attend(q[b:b + 1], k, v, [n - 1], [lo], [n - 1], scale, softcap, slopes))
    return [torch.cat(x) for x in zip(*parts)]


def prefill(q, kc, vc, tables, cu_q, cu_k, scale, softcap=0.0, slopes=None, window=0,
            first_keys=None, prefix_lens=None):
    """Reference of paged_prefill_attention_scored over host tensors."""
    parts = []
    for b in range(len(cu_q) - 1):
        q0, q1 = int(cu_q[b]), int(cu_q[b + 1])
        Lk = int(cu_k[b + 1] - cu_k[b])
        k, v = gather(kc, tables[b], Lk), gather(vc, tables[b], Lk)
        pos = [Lk - (q1 - q0) + r for r in range(q1 - q0)]
        first = [max(0, i - window + 1) if window else 0 for i in pos]
        if first_keys is not None:
            first = [max(f, int(x)) for f, x in zip(first, first_keys[q0:q1])]
        last = [max(i, int(prefix_lens[b]) - 1) if prefix_lens is not None else i for i in pos]
        parts.append(attend(q[q0:q1], k, v, pos, first, last, scale, softcap, slopes, 2.0 ** -8))
    return [torch.cat(x) for x in zip(*parts)]


def norm_rope(x, weight, eps, positions, cos_sin, interleaved):
    """x [T, H, D] -> the normed and rotated rows in 64 bits."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * weight.double()
    if cos_sin is None:
        return y
    R = cos_sin.shape[1]
    t = cos_sin[positions.long()].double()
    c, s = t[:, None, :R // 2], t[:, None, R // 2:]
    z = y.clone()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        z[..., a] = y[..., a] * c[..., i] - y[..., b] * s[..., i]
        z[..., b] = y[..., b] * c[..., i] + y[..., a] * s[..., i]
    return z


def check_rows(got, want, what=""):
    """bf16 rows of norm_rope: one rounding, and a few fp32 roundings of the row."""
    if not want.numel():
        return
    d = (to64(got) - want).abs() - 2.0 ** -8 * want.abs() - 2.0 ** -19 * want.abs().amax(
        -1, keepdim=True)
    assert d.max().item() <= 0, f"{what}: {d.max().item()} past its bound"


def check_codes(codes, want, scale, what=""):
    """E4M3 codes of `want` / scale, saturated."""
    if not want.numel():
        return
    got = codes.cpu().view(torch.float8_e4m3fn).double()
    x = (want / scale).clamp(-E4M3_MAX, E4M3_MAX)
    row = x.abs().amax(-1, keepdim=True)
    d = (got - x).abs() - torch.clamp(2.0 ** -4 * x.abs(), min=2.0 ** -10) - 2.0 ** -19 * row
    assert d.max().item() <= 0, f"{what}: {d.max().item()} past its bound"


def alibi(Hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)])
