"""GPU tests of what the layer runner's inference forward leaves alone, and of its norm's eps."""
import pytest
import torch

import gated_mlp_gemms_amd as gm
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


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("train", [True, False])
def test_eps_reaches_the_norm(kind, train):
    """A stream so small that eps decides: the layer's input is the norm with the runner's eps, 1e-5 unless given; a step's
    gradients are then those with its statistics (the gradient has no eps of its own)."""
    size = dict(act="swiglu", dtype="f32", tokens=33, width=64, hidden=40, experts=8)
    announce(f"runner's eps, {kind}, train={train}")
    t = moe_tensors(seed=22, norm=kind, **size)
    t["x"].mul_(1e-3)

    def normed(eps):
        y, rstd = torch.empty_like(t["x"]), torch.empty(33, device="cuda")
        gm.norm_fwd(t["x"], y, weight=t["norm_weight"], bias=t.get("norm_bias"), rstd=rstd, kind=kind, eps=eps)
        return y, rstd

    assert not torch.equal(normed(1e-6)[0], normed(1e-5)[0])
    for given, eps in (({}, 1e-5), ({"eps": 1e-6}, 1e-6), ({"eps": 0.5}, 0.5)):
        r = MoeRunner(choices=3, tensors=t, norm=kind, train=train, **given, **size)
        r.step() if train else r.forward_infer()
        y, rstd = normed(eps)
        assert torch.equal(r.x, y)
        if train:
            assert torch.equal(r.rstd, rstd)
            dx = torch.empty_like(y)
            gm.norm_bwd(r.dx, t["x"], rstd, dx, mean=r.mean, weight=t["norm_weight"], dresidual=t["dout"], kind=kind)
            assert torch.equal(r.grads()["dx"], dx)


def test_a_bad_eps_is_refused():
    size = dict(act="swiglu", dtype="f32", tokens=3, width=64, hidden=40, experts=4)
    t = moe_tensors(norm="rms", **size)
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(gm.MlpError, match="eps"):
            MoeRunner(choices=2, tensors=t, norm="rms", eps=eps, train=False, **size).forward_infer()
