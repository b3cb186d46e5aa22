"""paged_append_tokens with the numbers of rows around 48 KB of shared memory, in a process
that has not called it yet (a call with more rows would raise the kernel's limit for good)."""
import subprocess
import sys
from pathlib import Path

import pytest

CODE = """
import torch
from paged_kv_cache_214_gb300 import pkv
for R in (3400, 4051, 4052, 4060, 4095, 4096, 4097, 8192):
    lens = torch.arange(R, dtype=torch.int32, device="cuda") % 256
    table = torch.zeros(R, 1, dtype=torch.int32, device="cuda")
    free = torch.zeros(1, dtype=torch.int32, device="cuda")
    height = torch.zeros(1, dtype=torch.int32, device="cuda")
    old = lens.clone()
    slots, positions = pkv.paged_append_tokens(table, lens, free, height)
    there = old > 0
    assert torch.equal(lens, old + there), R
    assert torch.equal(slots, torch.where(there, old, -1)), R
    assert torch.equal(positions, old), R
    assert pkv.get_device_error() == pkv.PKV_OK
print("rows ok")
"""


@pytest.mark.gpu
def test_rows_around_48_kb_in_a_fresh_process():
    done = subprocess.run([sys.executable, "-c", CODE], cwd=Path(__file__).parent.parent,
                          capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "rows ok" in done.stdout, done.stdout + done.stderr
