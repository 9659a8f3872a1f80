"""CPU test of the layer's and swa_fwd's `stream=`: the tensors that a call makes
for itself and its caller come from that stream's pool, because the current
stream's may hand out a block whose last users are still queued there; what the
caller gets is recorded on the current stream, where it may be read.  Streams
are names here and the library's calls are not made."""
import pytest
import torch

import chunk_test_b200 as ct
from chunk_test_b200 import _abi, layer


class OnGpu(torch.Tensor):
    """A host tensor that says it is on a GPU."""
    device = torch.device("cuda", 0)


class Lib:
    """The library's size queries; its launches succeed without one."""

    def __getattr__(self, name):
        if name in ("lact_ttt_fwd_ex", "lact_ttt_bwd_ex", "lact_swa_fwd"):
            return lambda *a: _abi.LACT_OK
        return getattr(real, name)


real = None


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


@pytest.mark.parametrize("name,results", [("ttt_fwd", 4), ("ttt_bwd", 12), ("swa_fwd", 1)])
def test_own_stream_makes_its_tensors_there(name, results, monkeypatch):
    global real
    real = _abi.lib()
    current, made, recorded = ["main"], [], []

    class Stream:
        cuda_stream = 0

        def __enter__(self):
            current.append("side")

        def __exit__(self, *a):
            current.pop()

    def tracked(make):
        def call(*args, **kw):
            kw.pop("device", None)
            t = make(*args, **kw)
            made.append(current[-1])
            return t
        return call

    for n in ("empty", "empty_like"):
        monkeypatch.setattr(torch, n, tracked(getattr(torch, n)))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    monkeypatch.setattr(_abi, "lib", Lib)
    monkeypatch.setattr(layer, "_check_outputs", lambda *a: None)
    monkeypatch.setattr(layer, "_check_workspace", lambda *a: None)

    B, H, T, d, dh = 1, 2, 256, 64, 64
    if name == "swa_fwd":
        x = [zeros(B, H, T, d, dtype=torch.bfloat16) for _ in range(3)]
        got = [ct.swa_fwd(*x, *[zeros(H, d) for _ in range(4)], 128, stream=Stream())]
    else:
        q, k, v = (zeros(B, H, T, d) for _ in range(3))
        args = (q, k, v, zeros(B, H, T, 3), zeros(B, H, T), zeros(H, dh, d), zeros(H, d, dh), zeros(H, dh, d), 64,
                ct.APPLY_THEN_UPDATE, ct.RULE_MOMENTUM)
        if name == "ttt_fwd":
            got = ct.ttt_fwd(*args, stream=Stream())
        else:
            got = ct.ttt_bwd(*args, zeros(B, H, T, d), out_scale=zeros(B, H, T), momentum_grads=True,
                             stream=Stream()).values()
    assert made == ["side"] * (results + 1)      # and the workspace
    assert sorted(t.data_ptr() for t in got) == sorted(p for p, s in recorded if s == "main")
