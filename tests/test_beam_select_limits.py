"""beam_select at the largest vocabularies: what is refused (a place behind a row's last word
must fit 32 bits), and the largest that is not."""
import math

import pytest
import torch

from paged_kv_cache_214_gb300 import build as B
from paged_kv_cache_214_gb300 import pkv

MOST = 2 ** 31 - 1 - 2 * 512   # width * V


@pytest.mark.parametrize("width,V", [(1, MOST + 1), (1, 2 ** 31 - 1 - 512), (1, 2 ** 31 - 1),
                                     (2, MOST // 2 + 1), (32, MOST // 32 + 1)])
@pytest.mark.parametrize("fp32", [0, 1])
def test_too_wide_vocabularies_are_refused(width, V, fp32):
    B.build()
    lib, P = pkv.load_library(), 256   # (a stand-in address: refused before any use)
    assert lib.beam_select(P, P, P, P, P, fp32, V, P, 1, width, V, 4, -1, P, 1 << 20,
                           None) == pkv.PKV_ERR_SHAPE
    assert lib.beam_select_workspace_bytes(1, width, V, fp32) == 0


def test_widest_vocabularies_pass_the_checks():
    B.build()
    lib, P = pkv.load_library(), 256
    for width in (1, 2, 32):
        V = MOST // width
        assert lib.beam_select(P, P, P, P, P, 0, V, P, 1, width, V, 4, -1, P, 1 << 20,
                               None) == pkv.PKV_ERR_WORKSPACE   # (the next check)
        assert lib.beam_select_workspace_bytes(1, width, V, 0) > 1 << 20
    assert lib.beam_select(P, P, P, P, P, 0, 9, P, 65535 // 5, 5, 9, 4, -1, P, 0,
                           None) == pkv.PKV_ERR_WORKSPACE
    assert lib.beam_select(P, P, P, P, P, 0, 9, P, 65535 // 5 + 1, 5, 9, 4, -1, P, 0,
                           None) == pkv.PKV_ERR_SHAPE


@pytest.mark.gpu
def test_the_widest_vocabulary():
    V, part = MOST, 1 << 27
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(1, 1, V, dtype=torch.bfloat16, device="cuda")
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for a in range(0, V, part):
        piece = x[0, 0, a:a + part]
        piece.copy_(torch.randn(piece.shape, generator=g, device="cuda").clamp(-3, 3))
        total += piece.float().exp().sum(dtype=torch.float64)
    best = [(V - 1, 9.0), (0, 8.5), (V // 3, 8.5), (V // 2, 8.0)]
    for at, value in best:
        total += math.exp(value) - x[0, 0, at].double().exp()
        x[0, 0, at] = value
    scores, parents, tokens, end = pkv.beam_select(x, torch.zeros(1, 1, device="cuda"), 4,
                                                   eos_token=V - 2)
    assert tokens.tolist() == [[at for at, _ in best]] and (parents == 0).all()
    # (2^-24 of the sum for each of a lane's few thousand additions, in either sum's worst case)
    want = torch.tensor([value for _, value in best], dtype=torch.float64) - total.log().item()
    assert (scores[0].cpu().double() - want).abs().max() <= 2.0 ** -11
    assert (end[0, 0].double() - (x[0, 0, V - 2].double() - total.log())).abs() <= 2.0 ** -11
    assert pkv.get_device_error() == pkv.PKV_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beams_that_have_not_begun_beside_masses_of_equal_logits(dtype):
    """Their logits are not read; whatever they hold, the live beam's come in their order."""
    x = torch.full((2, 5, 5003), torch.finfo(dtype).min, dtype=dtype, device="cuda")
    x[..., 7] = 1.0
    scores = torch.full((2, 5), -math.inf, device="cuda")
    scores[0, 3], scores[1, 0], scores[1, 4] = -1.0, -2.0, -2.5
    x[0, :3], x[0, 4], x[1, 1], x[1, 2], x[1, 3] = math.nan, 50.0, math.inf, -math.inf, 9.0
    best, parents, tokens, end = pkv.beam_select(x, scores, 40, eos_token=2)
    rest = [v for v in range(41) if v not in (2, 7)]
    assert parents[0].tolist() == [3] * 40 and tokens[0].tolist() == [7] + rest[:39]
    assert parents[1].tolist() == [0, 4] + [0] * 38 and tokens[1].tolist() == [7, 7] + rest[:38]
    assert best[0, 0] == -1.0 and best[1, 0] == -2.0 and best[1, 1] == -2.5
    live = torch.isfinite(scores)
    assert (end[~live] == -math.inf).all() and (end[live] < -1e30).all()
    assert pkv.get_device_error() == pkv.PKV_OK
