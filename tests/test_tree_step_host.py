"""Refusals of runtime.TreeStep on the host, before anything is laid out: a step
reads the layers' own tensors, so one that would be converted once, into a copy
that later steps and commits do not write, is refused."""

import pytest
import torch

from long_context_compressed_overlapped_b200 import runtime, synth


@pytest.mark.parametrize("name,change", [
    ("pos", lambda t: t.long()),
    ("parents", lambda t: t.long()),
    ("parents", lambda t: t.t().contiguous().t()),
    ("tw", lambda t: t.bfloat16()),
    ("tw", lambda t: torch.stack([t, t], -1)[..., 0]),
    ("kI_scale", lambda t: t.double()),
])
def test_converted_inputs_are_refused(name, change):
    wl = synth.WORKLOADS["decode_1m"]
    layers = synth.tree_inputs(wl, 5, "cpu", ctx=300, B=2, layers=("hca", "csa"))
    L = layers[1]                                                           # (the CSA layer has all of them)
    L[name] = change(L[name])
    with pytest.raises(TypeError, match=name):
        runtime.TreeStep(wl, layers, None)
