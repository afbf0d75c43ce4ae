"""A workspace that a call allocates itself is allocated on the stream that the call runs on: torch's allocator
hands a freed block on in that stream's order, so a block of another stream could be given away while the call's
kernels still use it. On the CPU: the tensors are fake ones of a GPU, whose addresses are NULL, so the library
refuses each call after the workspace has been made and before any HIP call."""
import contextlib

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import gated_mlp_gemms_amd as gm
from gated_mlp_gemms_amd import _lib

CURRENT, OTHER = 0x5550, 0x7770   # stream handles, never used as such


class Handle:
    """What a torch stream passed as `stream` is to a call."""
    cuda_stream = OTHER


@pytest.fixture
def seen(monkeypatch):
    """[(bytes, the stream they were allocated on)] of every allocation of bytes."""
    log, entered = [], [CURRENT]
    make = torch.empty

    @contextlib.contextmanager
    def on(stream):
        entered.append(stream)
        yield
        entered.pop()

    def empty(n, dtype=None, device=None):
        assert dtype == torch.uint8 and torch.device(device) == torch.device("cuda", 0)
        log.append((n, entered[-1]))
        return make(n, dtype=dtype, device=device)

    def external(handle, device=None):
        assert torch.device(device) == torch.device("cuda", 0)
        return handle

    _lib.bind()
    with FakeTensorMode():
        monkeypatch.setattr(torch.cuda, "ExternalStream", external)
        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: CURRENT)
        monkeypatch.setattr(torch, "empty", empty)
        yield log, lambda *s, dtype=torch.bfloat16: make(*s, dtype=dtype, device="cuda")


def calls(t):
    """name, the call as a function of its stream, and the bytes of its workspace"""
    i32 = torch.int32
    ids, off, order = t(5000, dtype=i32), t(9, dtype=i32), [t(5000, dtype=i32) for _ in range(2)]
    d = gm.make_linear_desc(40, 64, 72, act="relu", experts=8)
    x, w, y = t(40, 64), t(8, 72, 64), t(40, 72)
    m = gm.make_desc(40, 64, 72, act="relu")
    w1, w2 = t(72, 64), t(64, 72)
    return [
        ("moe_sort", lambda s: gm.moe_sort(ids, 8, off, *order, stream=s), gm.moe_sort_workspace_bytes(5000, 8)),
        ("linear_fwd", lambda s: gm.linear_fwd(d, x, w, y, offsets=off, stream=s), gm.linear_workspace_bytes(d, "fwd")),
        ("linear_bwd", lambda s: gm.linear_bwd(d, y, x, w, preact=y, offsets=off, dx=x, stream=s),
         gm.linear_workspace_bytes(d, "bwd")),
        ("mlp_fwd", lambda s: gm.mlp_fwd(m, None, None, w1, w2, x, stream=s), gm.workspace_bytes(m, "fwd")),
        ("mlp_fwd_infer", lambda s: gm.mlp_fwd_infer(m, None, None, w1, w2, x, stream=s), gm.workspace_bytes(m, "fwd_infer")),
        ("mlp_bwd", lambda s: gm.mlp_bwd(m, x, None, None, w1, w2, stream=s), gm.workspace_bytes(m, "bwd")),
        ("mlp_quantize_e4m3", lambda s: gm.mlp_quantize_e4m3(x, None, None, stream=s), gm.mlp_quantize_workspace_bytes()),
    ]


@pytest.mark.filterwarnings("ignore::UserWarning")
@pytest.mark.parametrize("which", range(7))
@pytest.mark.parametrize("stream,handle", [(CURRENT, CURRENT), (OTHER, OTHER), (Handle(), OTHER)],
                         ids=["the current one", "another's handle", "another"])
def test_workspace_is_allocated_on_the_calls_stream(seen, which, stream, handle):
    log, t = seen
    name, call, need = calls(t)[which]
    with pytest.raises(gm.MlpError, match=f"{name}: .*(NULL|required)"):
        call(stream)
    assert log == [(need, handle)]


def test_raw_stream_is_torchs_current_one(seen):
    assert _lib.raw_stream(0) == CURRENT
