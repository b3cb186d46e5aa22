"""paged_reorder_beams where a partly filled block with several heirs is none: no block of the
stack is taken for a row that becomes empty."""
import pytest
import torch

from paged_kv_cache_214_gb300 import pkv

gpu = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("bad", [-1, 1000])
def test_rows_without_a_source_take_no_block(bad, in_place):
    # two requests of three rows with two blocks each, the second partly filled; 12 is free
    tables = [[0, 1, -1], [2, 3, -1], [4, bad, -1], [5, 6, -1], [7, 8, -1], [9, 10, -1]]
    lens = [300] * 6
    parents = [[2, 2, 0], [1, 1, 2]]
    free = [11, 12, 13] + [-9] * 11
    t, n, f, height = ints(tables), ints(lens), ints(free), ints([3])
    outs = {} if in_place else dict(out_tables=torch.full_like(t, -3), out_lens=torch.full_like(n, -3),
                                    out_num_free=torch.full_like(height, -3))
    copies = pkv.paged_reorder_beams(t, n, ints(parents), f, height, **outs)
    assert pkv.get_device_error() == pkv.PKV_ERR_DEVICE_INDEX
    assert pkv.get_device_error() == pkv.PKV_OK
    if not in_place:
        t, n, height = outs["out_tables"], outs["out_lens"], outs["out_num_free"]
    # row 1 would have copied the block that is none; row 4 copies block 8 as ever
    assert n.tolist() == [300, 0, 300, 300, 300, 300]
    # given back: column by column rows 1 (2, 3) and, of the second request, row 0 (5, 6)
    stack = [11, 12, 13, 2, 3, 5, 6]
    own = stack.pop()
    assert height.tolist() == [len(stack)] and f[:len(stack)].tolist() == stack
    assert t.tolist() == [[4, -1, -1], [-1, -1, -1], [0, 1, -1], [7, 8, -1], [7, own, -1], [9, 10, -1]]
    assert copies.tolist() == [[-1, -1, -1, -1, 8, -1], [-1, -1, -1, -1, own, -1], [0, 0, 0, 0, 44, 0]]
    # every block is held or on the stack
    held = {x for row in t.tolist() for x in row if x >= 0}
    assert held | set(f[:len(stack)].tolist()) == set(range(14))
