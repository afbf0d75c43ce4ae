"""GPU tests of what the layer runner's inference forward leaves alone, and of its norm's eps."""
import pytest
import torch

from gated_mlp_gemms_amd.moe_runner import MoeRunner, moe_tensors
from gpu_helpers import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_inference_leaves_the_training_forwards_results(kind):
    """An inference forward on another input, between a step and a step's use of its results: loss, loads and statistics are
    the training forward's, and the output is what a runner for inference gives."""
    size = dict(act="swiglu", dtype="bf16", tokens=70, width=64, hidden=40, experts=8)
    announce(f"inference forward of a training runner, {kind}")
    t = moe_tensors(seed=21, norm=kind, **size)
    r = MoeRunner(choices=3, tensors=t, norm=kind, balance=0.5, **size)
    r.step()
    kept = {n: getattr(r, n) for n in ("loss", "counts", "shares", "rstd", "preact") + (("mean",) if kind == "layer" else ())}
    want = {n: v.clone() for n, v in kept.items()}
    first = r.out.clone()
    r.stream.mul_(3.0).add_(0.25)
    other = r.forward_infer().clone()
    assert not torch.equal(other, first)
    for n, v in want.items():
        assert torch.equal(kept[n], v), n
    alone = MoeRunner(choices=3, tensors={**t, "x": r.stream}, norm=kind, train=False, **size)
    assert torch.equal(alone.forward_infer(), other)
