"""Decode calls of every number of splits up to a cache of 40 key tiles, each
the first such call of a process that has made no larger one (a kernel's limit
of dynamic shared memory, once raised, stays raised)."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CHILD = """
import torch
from long_context_compressed_overlapped_b200 import api
from oracle import csahca_oracle as O
from tests.helpers import check_close, npy
g = torch.Generator(device="cuda").manual_seed(1)
normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
for tiles in range(1, 41):
    N = 128 * tiles
    kv, win, q, sinks = normal(1, N, 512), normal(1, 128, 512), normal(1, 64, 512), torch.zeros(64, device="cuda")
    pos = torch.tensor([16 * N], device="cuda", dtype=torch.int32)
    out = api.compressed_attn_decode("hca", q, pos, kv, win, sinks, m=16, rope_dims=64)
    if tiles in (5, 16, 20, 33):
        ref = O.decode_attention("hca", npy(q[0]), 16 * N, npy(kv[0]), npy(win[0]), npy(sinks), m=16, w=128, r=64)
        check_close(npy(out[0]), ref, "bf16", f"{tiles} tiles")
assert api.device_error() == 0
"""


def test_every_number_of_splits_in_a_fresh_process():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", CHILD], cwd=root, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
