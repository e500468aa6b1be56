"""TreeStep.commit: numbers in a path that are no node's end it (nothing is read
past the drafted tokens), and layers that share one pos tensor move it once.
The state is the decode steps', bit for bit."""

import pytest
import torch

from long_context_compressed_overlapped_b200 import api, runtime, synth
from tests import tree_reference as R
from tests.test_gpu_tree_step import DEV, clone, decode_path

pytestmark = pytest.mark.gpu
T = 6


def make(ctx=509, B=3):
    wl = synth.WORKLOADS["decode_1m"]
    layers = synth.tree_inputs(wl, T, DEV, ctx=ctx, B=B, layers=("csa", "hca"), room=2 * T)
    return wl, layers, clone(layers), [R.path_of(row, T - 1) for row in layers[0]["parents"].tolist()]


def check_state(wl, layers, before, paths, pos):
    for li, (L, was) in enumerate(zip(layers, before)):
        for b, path in enumerate(paths):
            if path:
                _, _, one = decode_path(wl, was, b, path, pos)
            else:
                one = {n: was[n][b:b + 1] for n in ("kv", "win", "ring", "iring", "kI", "kI_scale") if was.get(n) is not None}
            for key in ("kv", "win", "ring", "iring", "kI", "kI_scale"):
                if L.get(key) is not None:
                    assert torch.equal(L[key][b], one[key][0]), f"layer {li} {key} of sequence {b}"
            assert int(L["pos"][b]) == pos + len(path)


@pytest.mark.parametrize("cpu", [False, True])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_numbers_that_are_no_nodes_end_a_path(cpu, dtype):
    wl, layers, before, full = make()
    step = runtime.TreeStep(wl, layers, torch.cuda.Stream())
    big = 2**31 - 1
    rows = [full[0][:1] + [T] + full[0][1:], full[1][:2] + [-7] + full[1][2:], [big] + full[2]]      # a hole, then nodes
    n = max(map(len, rows))
    paths = torch.tensor([r + [-1] * (n - len(r)) for r in rows], dtype=dtype, device="cpu" if cpu else DEV)
    step.commit(paths)
    step.stream.synchronize()
    check_state(wl, layers, before, [full[0][:1], full[1][:2], []], 509)
    assert api.device_error() == 0


def test_layers_that_share_their_positions():
    wl, layers, before, full = make()
    for L in layers[1:]:
        L["pos"] = layers[0]["pos"]
    step = runtime.TreeStep(wl, layers, torch.cuda.Stream())
    n = max(map(len, full))
    step.commit(R.ints([p + [-1] * (n - len(p)) for p in full], DEV))
    step.stream.synchronize()
    check_state(wl, layers, before, full, 509)


def test_paths_of_other_shapes_or_types_are_refused():
    wl, layers, before, _ = make()
    step = runtime.TreeStep(wl, layers, torch.cuda.Stream())
    for bad in (torch.zeros(2, 3, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV),
                torch.zeros(3, 2, device=DEV)):
        with pytest.raises(ValueError):
            step.commit(bad)
    step.commit(torch.zeros(3, 0, dtype=torch.int32, device=DEV))                       # nothing accepted
    step.stream.synchronize()
    check_state(wl, layers, before, [[], [], []], 509)
