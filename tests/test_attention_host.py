"""CPU tests of the attention half's operators: the library's argument checks
(found before anything is enqueued, so no GPU is needed), the wrappers' checks,
the frequencies, and the oracle's gradients against differences."""
import ctypes
import math

import pytest
import torch

import chunk_test_b200 as ct
from chunk_test_b200 import _abi
from oracle import attention_oracle as ao

G = 1 << 32


def t4(i, B=2, H=4, T=64, d=64, layout="bhtd", at=0):
    s = (H * T * d, T * d, d) if layout == "bhtd" else (T * H * d, d, H * d)
    return _abi.LactTensor4(G * (i + 1) + at, *s)


def rot_problem(**kw):
    a = dict(B=2, H=4, Hkv=2, T=64, d=64, rot=32, start=0, interleaved=0, dtype=1, amplitude=1.0, reserved=0)
    a.update(kw)
    return _abi.LactRotaryProblem(*a.values())


def swa_problem(**kw):
    a = dict(B=2, H=4, Hkv=2, T=64, Tq=64, d=64, window=16, sinks=4, scale=0.125, dtype=1)
    a.update(kw)
    return _abi.LactSwaSinkProblem(*a.values())


def ref(x):
    return None if x is None else ctypes.byref(x)


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(H=0), dict(Hkv=-1), dict(T=0), dict(d=0), dict(d=60), dict(d=520), dict(rot=0), dict(rot=31),
    dict(rot=66), dict(start=-1), dict(interleaved=2), dict(dtype=2), dict(amplitude=math.nan), dict(B=70000),
    dict(T=(1 << 30) + 1),
])
def test_rotary_problems_refused(bad):
    p = rot_problem(**bad)
    assert ct.lib().lact_rotary_bwd_workspace_bytes(ctypes.byref(p)) == 0
    rc = ct.lib().lact_rotary_fwd(ctypes.byref(p), ref(t4(0)), ref(t4(1, H=2)), 9 * G, None, None, None, None, None,
                                  ref(t4(2)), ref(t4(3, H=2)), None)
    assert rc == ct.LACT_EINVAL


def test_rotary_arguments_refused():
    p = rot_problem()
    lib = ct.lib()

    def call(q=t4(0), k=t4(1, H=2), freqs=9 * G, par=(None,) * 4, qo=t4(2), ko=t4(3, H=2)):
        return lib.lact_rotary_fwd(ctypes.byref(p), ref(q), ref(k), freqs, None, *par, ref(qo), ref(ko), None)

    assert call(q=None) == ct.LACT_EINVAL
    assert call(k=None) == ct.LACT_EINVAL
    assert call(freqs=None) == ct.LACT_EINVAL
    assert call(freqs=9 * G + 8) == ct.LACT_EINVAL
    assert call(q=t4(0, at=8)) == ct.LACT_EINVAL                       # 16-byte alignment
    assert call(par=(5 * G, 6 * G, 7 * G, None)) == ct.LACT_EINVAL     # all parameters or none
    bent = t4(0)
    bent.stride_t = 68                                                 # not a multiple of 16 bytes
    assert call(q=bent) == ct.LACT_EINVAL
    for name in ("stride_b", "stride_h", "stride_t"):
        flat = t4(2)
        setattr(flat, name, 0)                                         # one row for all
        assert call(qo=flat) == ct.LACT_EINVAL
    folded = t4(2)
    folded.stride_h = 64                                               # heads over tokens
    assert call(qo=folded) == ct.LACT_EINVAL
    assert call(qo=t4(0, at=128)) == ct.LACT_EINVAL                    # shifted onto q
    assert call(ko=t4(0)) == ct.LACT_EINVAL                            # k's result onto q
    assert call(ko=t4(2)) == ct.LACT_EINVAL                            # both results in one place
    # the backward with scales wants the workspace
    nul = None
    rc = lib.lact_rotary_bwd(ctypes.byref(p), ref(t4(0)), ref(t4(1, H=2)), 9 * G, nul, ref(t4(2)), ref(t4(3, H=2)),
                             10 * G, 11 * G, ref(t4(4)), ref(t4(5, H=2)), 12 * G, 13 * G, 14 * G, 15 * G, 16 * G,
                             ctypes.c_size_t(8), nul)
    assert rc == ct.LACT_ENOSPC
    rc = lib.lact_rotary_bwd(ctypes.byref(p), ref(t4(0)), ref(t4(1, H=2)), 9 * G, nul, ref(t4(2)), ref(t4(3, H=2)),
                             10 * G, 11 * G, ref(t4(4)), ref(t4(5, H=2)), 12 * G, 12 * G, 14 * G, 15 * G, 16 * G,
                             ctypes.c_size_t(1 << 30), nul)
    assert rc == ct.LACT_EINVAL                                        # two sums in one place


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(H=0), dict(Hkv=0), dict(H=3), dict(T=0), dict(Tq=0), dict(Tq=65), dict(d=0), dict(d=60),
    dict(d=264), dict(window=0), dict(sinks=-1), dict(scale=math.inf), dict(scale=0.0), dict(scale=-1.0), dict(dtype=3), dict(B=20000),
    dict(T=(1 << 24) + 1),
])
def test_attention_problems_refused(bad):
    p = swa_problem(**bad)
    lib = ct.lib()
    assert lib.lact_swa_sink_bwd_workspace_bytes(ctypes.byref(p)) == 0
    k, v = t4(1, H=2), t4(2, H=2)
    assert lib.lact_swa_sink_fwd(ctypes.byref(p), ref(t4(0)), ref(k), ref(v), None, ref(t4(3)), 9 * G, None) == ct.LACT_EINVAL
    assert lib.lact_swa_sink_bwd(ctypes.byref(p), ref(t4(0)), ref(k), ref(v), ref(t4(3)), 9 * G, ref(t4(4)), None,
                                 ref(t4(5)), ref(t4(6, H=2)), ref(t4(7, H=2)), 10 * G, ctypes.c_size_t(1 << 40),
                                 None) == ct.LACT_EINVAL


def test_attention_arguments_refused():
    p, lib = swa_problem(), ct.lib()

    def fwd(q=t4(0), k=t4(1, H=2), v=t4(2, H=2), out=t4(3), lse=9 * G):
        return lib.lact_swa_sink_fwd(ctypes.byref(p), ref(q), ref(k), ref(v), None, ref(out), lse, None)

    for name in ("q", "k", "v", "out", "lse"):
        assert fwd(**{name: None}) == ct.LACT_EINVAL, name
    assert fwd(out=t4(0)) == ct.LACT_EINVAL
    assert fwd(out=t4(1, H=2)) == ct.LACT_EINVAL
    assert fwd(lse=G) == ct.LACT_EINVAL                                # onto q
    assert fwd(k=t4(1, H=2, at=8)) == ct.LACT_EINVAL
    flat = t4(1, H=2)
    flat.stride_b = 0
    assert fwd(k=flat) == ct.LACT_EINVAL

    def bwd(ws=10 * G, n=1 << 40, dq=t4(5), dk=t4(6, H=2), dv=t4(7, H=2)):
        return lib.lact_swa_sink_bwd(ctypes.byref(p), ref(t4(0)), ref(t4(1, H=2)), ref(t4(2, H=2)), ref(t4(3)), 9 * G,
                                     ref(t4(4)), None, ref(dq), ref(dk), ref(dv), ws, ctypes.c_size_t(n), None)

    assert bwd(ws=None) == ct.LACT_EINVAL
    assert bwd(ws=10 * G + 16) == ct.LACT_EINVAL
    assert bwd(n=16) == ct.LACT_ENOSPC
    assert bwd(dq=t4(0)) == ct.LACT_EINVAL
    assert bwd(dk=t4(7, H=2)) == ct.LACT_EINVAL                        # dk onto dv
    assert bwd(dv=t4(1, H=2)) == ct.LACT_EINVAL                        # dv onto k


def test_workspace_grows_with_the_sinks_only():
    """Without sinks the backward keeps one float per query row; a sink tile
    adds its parts, one near and one for each 1024 later query rows."""
    def need(**kw):
        return ct.lib().lact_swa_sink_bwd_workspace_bytes(ctypes.byref(swa_problem(**kw)))

    assert need(T=4096, Tq=4096, sinks=0) == 2 * 4 * 4096 * 4
    far = -(-(4096 - (127 + 16)) // 1024)
    tile = 2 * 128 * 64 * 4
    assert need(T=4096, Tq=4096, sinks=4) == 2 * 4 * 4096 * 4 + 2 * 2 * (1 + far) * tile
    assert need(T=4096, Tq=4096, sinks=129) == 2 * 4 * 4096 * 4 + 2 * 2 * 2 * (1 + far) * tile
    assert need(T=4096, Tq=4096, sinks=4, window=4096) == 2 * 4 * 4096 * 4


@pytest.mark.parametrize("bad", [
    dict(T=2), dict(Tq=2), dict(window=0), dict(sinks=-1), dict(d=100), dict(H=3), dict(dtype=5),
    dict(window=(1 << 30) + 1),
])
def test_decode_problems_refused(bad):
    p = swa_problem(**{**dict(T=1, Tq=1), **bad})
    one = lambda i, H: t4(i, H=H, T=1)  # noqa: E731
    rc = ct.lib().lact_swa_sink_decode(ctypes.byref(p), ref(one(0, 4)), ref(one(1, 2)), ref(one(2, 2)), 4 * G, 5 * G,
                                       6 * G, ref(one(7, 4)), None)
    assert rc == ct.LACT_EINVAL


def test_decode_arguments_refused():
    p = swa_problem(T=1, Tq=1)
    one = lambda i, H: t4(i, H=H, T=1)  # noqa: E731

    def call(q=one(0, 4), k=one(1, 2), v=one(2, 2), kc=4 * G, vc=5 * G, seen=6 * G, out=one(7, 4)):
        return ct.lib().lact_swa_sink_decode(ctypes.byref(p), ref(q), ref(k), ref(v), kc, vc, seen, ref(out), None)

    for name in ("q", "k", "v", "kc", "vc", "seen", "out"):
        assert call(**{name: None}) == ct.LACT_EINVAL, name
    assert call(vc=4 * G) == ct.LACT_EINVAL
    assert call(kc=4 * G + 8) == ct.LACT_EINVAL
    assert call(out=one(0, 4)) == ct.LACT_EINVAL
    assert call(kc=G) == ct.LACT_EINVAL                                # the cache onto q
    p2 = swa_problem()
    assert ct.lib().lact_swa_cache_fill(ctypes.byref(p2), ref(t4(0, H=2)), None, None, 4 * G, 5 * G, None) == ct.LACT_EINVAL
    assert ct.lib().lact_swa_cache_fill(ctypes.byref(p2), ref(t4(0, H=2)), ref(t4(1, H=2)), None, G, 5 * G,
                                        None) == ct.LACT_EINVAL


def test_wrappers_refuse_cpu_tensors_and_wrong_shapes():
    q = torch.zeros(1, 2, 4, 64)
    f = torch.zeros(8, dtype=torch.float64)
    with pytest.raises(ValueError):
        ct.rotary_fwd(q, q, f)
    with pytest.raises(ValueError):
        ct.swa_sink_fwd(q, q, q, 4)
    with pytest.raises(ValueError):
        ct.swa_sink_decode(q, q, q, q, q, f, 4)
    with pytest.raises(ValueError):
        ct.rotary_fwd(q[0], q, f)


def test_frequencies():
    f, a = ct.rotary_frequencies(8, device="cpu")
    want = torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64)
    assert a == 1.0 and torch.allclose(f, want, rtol=1e-14, atol=0)
    assert torch.allclose(ct.rotary_frequencies(8, method="linear", factor=4.0, device="cpu")[0], want / 4, rtol=1e-14, atol=0)
    g = ct.rotary_frequencies(8, method="base", factor=4.0, device="cpu")[0]
    assert abs(float(g[0]) - 1.0) < 1e-14 and abs(float(g[-1]) * 4 - float(want[-1])) < 1e-14
    # 2000 trained positions: the pairs turn 318, 31.8, 3.18 and 0.318 times
    g, a = ct.rotary_frequencies(8, method="by_parts", factor=4.0, context=2000, low=1.0, high=32.0, device="cpu")
    assert abs(a - (1 + 0.1 * math.log(4.0))) < 1e-14
    assert float(g[0]) == float(want[0]) and abs(float(g[3]) * 4 - float(want[3])) < 1e-16
    turns = 0.01 * 2000 / (2 * math.pi)
    keep = (turns - 1) / 31
    assert abs(float(g[2]) - 0.01 * (keep + (1 - keep) / 4)) < 1e-14
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, method="other"), dict(rot=8, factor=0.5),
                dict(rot=8, method="by_parts"), dict(rot=2, method="base")):
        with pytest.raises(ValueError):
            ct.rotary_frequencies(**{**dict(device="cpu"), **bad})


def test_oracle_gradients_match_differences():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    q, k, v, dout = r(2, 4, 9, 8), r(2, 2, 13, 8), r(2, 2, 13, 8), r(2, 4, 9, 8)
    args = dict(window=5, sinks=2, lengths=(13, 8))
    w = ao.attention(q, k, v, dout=dout, **args)
    f = lambda *x: float((ao.attention(*x, **args)["out"] * dout).sum())  # noqa: E731
    for i, n in enumerate(("dq", "dk", "dv")):
        e = r(*(q, k, v)[i].shape)
        up, dn = [q, k, v], [q, k, v]
        up[i], dn[i] = up[i] + 1e-5 * e, dn[i] - 1e-5 * e
        d = (f(*up) - f(*dn)) / 2e-5
        assert abs(d - float((w[n] * e).sum())) < 1e-7 * (1 + abs(d)), n
    freqs = torch.tensor([1.0, 0.3, 0.05], dtype=torch.float64)
    pos = torch.arange(9).expand(2, 9)
    sc, of = r(4, 8), r(4, 8)
    dx, ds, do, _, _ = ao.rotary_vjp(dout, freqs, pos, True, 1.1, q, sc)
    fr = lambda a, b, c: float((ao.rotary(a, freqs, pos, True, 1.1, b, c) * dout).sum())  # noqa: E731
    for i, got in enumerate((dx, ds, do)):
        x = [q, sc, of]
        e = r(*x[i].shape)
        up, dn = list(x), list(x)
        up[i], dn[i] = up[i] + 1e-5 * e, dn[i] - 1e-5 * e
        d = (fr(*up) - fr(*dn)) / 2e-5
        assert abs(d - float((got * e).sum())) < 1e-7 * (1 + abs(d)), i


def test_oracle_is_plain_attention_where_the_window_covers_all():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((1, 2, 12, 8), generator=g, dtype=torch.float64) for _ in range(3))
    s = (q @ k.transpose(-1, -2) / math.sqrt(8)).masked_fill(~torch.ones(12, 12).tril().bool(), -math.inf)
    assert torch.allclose(ao.attention(q, k, v, 12)["out"], s.softmax(-1) @ v, rtol=1e-12, atol=1e-14)
    assert torch.allclose(ao.attention(q, k, v, 3, 12)["out"], s.softmax(-1) @ v, rtol=1e-12, atol=1e-14)


def test_oracle_decode_follows_the_sequence():
    """The rolling cache, token by token, gives the attention over the whole sequence."""
    g = torch.Generator().manual_seed(2)
    T, window, sinks = 20, 6, 2
    q, k, v = (torch.randn((1, n, T, 8), generator=g, dtype=torch.float64) for n in (4, 2, 2))
    want = ao.attention(q, k, v, window, sinks)["out"]
    kc = torch.full((1, 2, window + sinks, 8), math.nan, dtype=torch.float64)
    vc = kc.clone()
    for t in range(T):
        o, _, kc, vc = ao.decode(q[:, :, t:t + 1], k[:, :, t:t + 1], v[:, :, t:t + 1], kc, vc, [t], window, sinks)
        assert torch.allclose(o, want[:, :, t:t + 1], rtol=1e-12, atol=1e-14)


def test_own_stream_makes_its_tensors_there(monkeypatch):
    """With stream= the results and workspaces come from that stream's pool (the
    current stream's may hand out a block whose last users are still queued),
    and the results are recorded on the current stream.  Without a GPU: the
    library is not called, and streams are names."""
    from chunk_test_b200 import attention as at
    current, made, recorded = ["main"], [], []

    class Stream:
        cuda_stream = 0

        def __enter__(self):
            current.append("side")

        def __exit__(self, *a):
            current.pop()

    def tracked(make):
        def call(*args, **kw):
            t = make(*args, **kw)
            made.append((t.data_ptr(), current[-1]))
            return t
        return call

    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((t.data_ptr(), s)))
    monkeypatch.setattr(torch.Tensor, "new_empty", tracked(torch.Tensor.new_empty))
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, tracked(getattr(torch, name)))
    monkeypatch.setattr(at, "_query", lambda q: None)
    monkeypatch.setattr(at, "_dense", lambda name, t, *a: t)
    monkeypatch.setattr(at, "_call", lambda *a: None)
    q, k = torch.zeros(2, 4, 600, 64), torch.zeros(2, 2, 600, 64)
    one, key = q[:, :, :1], k[:, :, :1]
    kc, vc = torch.zeros(2, 2, 8, 64), torch.zeros(2, 2, 8, 64)
    lse, freqs, scale = torch.zeros(2, 4, 600), torch.ones(32, dtype=torch.float64), torch.ones(4, 64)
    side = Stream()
    calls = {
        "rotary_fwd": (2, 0, lambda: ct.rotary_fwd(q, k, freqs, stream=side)),
        "rotary_bwd": (6, 1, lambda: ct.rotary_bwd(q, k, freqs, q=q, k=k, q_scale=scale, k_scale=scale[:2], stream=side)),
        "fwd": (2, 0, lambda: ct.swa_sink_fwd(q, k, k, 8, 2, stream=side)),
        "bwd": (3, 1, lambda: ct.swa_sink_bwd(q, k, k, q, lse, q, 8, 2, stream=side)),
        "decode": (1, 0, lambda: ct.swa_sink_decode(one, key, key, kc, vc, lse, 6, 2, stream=side)),
    }
    for name, (results, workspaces, call) in calls.items():
        made.clear(), recorded.clear()
        kept = call()
        assert len(made) == results + workspaces, name
        assert all(where == "side" for _, where in made), name
        got = [x for x in (kept.values() if isinstance(kept, dict) else kept if isinstance(kept, tuple) else [kept])]
        assert sorted(x.data_ptr() for x in got) == sorted(p for p, s in recorded if s == "main"), name


def slices(B, T, heads, d, layout):
    """The tensors of `heads` heads each that a packed buffer at G holds side by
    side: in each row ("rows", [B, T, all heads, d]), in each sequence ("heads",
    [B, all heads, T, d]) or in each head's row ("channels", [B, H, T, parts d])."""
    n, total = len(heads), sum(heads)
    at = [sum(heads[:i]) for i in range(n)]
    if layout == "rows":
        return [_abi.LactTensor4(G + 2 * a * d, T * total * d, d, total * d) for a in at]
    if layout == "heads":
        return [_abi.LactTensor4(G + 2 * a * T * d, total * T * d, T * d, d) for a in at]
    return [_abi.LactTensor4(G + 2 * i * d, heads[0] * T * n * d, T * n * d, n * d) for i in range(n)]


def rotary_bwd_rc(p, dq_out, dk_out, dq, dk):
    """lact_rotary_bwd with too small a workspace: its layouts are looked at
    before, so LACT_ENOSPC says that they are accepted.  Nothing is launched."""
    far = lambda i, H: t4(i, p.B, H, p.T, p.d)  # noqa: E731
    return ct.lib().lact_rotary_bwd(ref(p), ref(dq_out), ref(dk_out), 9 * G, None, ref(far(20, p.H)),
                                    ref(far(21, p.Hkv)), 10 * G, 11 * G, ref(dq), ref(dk), 12 * G, 13 * G, 14 * G,
                                    15 * G, 16 * G, ctypes.c_size_t(8), None)


@pytest.mark.parametrize("layout", ["rows", "heads", "channels"])
@pytest.mark.parametrize("B,T", [(1, 1), (2, 1), (8, 1), (1, 5), (2, 2), (8, 5)])
def test_packed_slices_are_apart(B, T, layout):
    """q and k of one packed buffer in place, one token per sequence too."""
    heads = (4, 4, 4) if layout == "channels" else (4, 2, 2)
    p = rot_problem(B=B, T=T, Hkv=heads[1])
    q, k, v = slices(B, T, heads, 64, layout)
    assert rotary_bwd_rc(p, q, k, q, k) == ct.LACT_ENOSPC
    assert rotary_bwd_rc(p, k if layout == "channels" else q, v, q, k) == (
        ct.LACT_EINVAL if layout == "channels" else ct.LACT_ENOSPC)
    # one row of 16 bytes too far: into the neighbour
    near = _abi.LactTensor4(k.data - 16, k.stride_b, k.stride_h, k.stride_t)
    assert rotary_bwd_rc(p, q, near, q, near) == ct.LACT_EINVAL
    # the attention's gradients beside one another
    s = swa_problem(B=B, T=T, Tq=T, Hkv=heads[1])
    far = lambda i, H: t4(i, B, H, T, 64)  # noqa: E731
    for dv, want in ((v, ct.LACT_ENOSPC), (k, ct.LACT_EINVAL)):
        rc = ct.lib().lact_swa_sink_bwd(ref(s), ref(far(20, 4)), ref(far(21, heads[1])), ref(far(22, heads[1])),
                                        ref(far(23, 4)), 9 * G, ref(far(24, 4)), None, ref(q), ref(k), ref(dv), 10 * G,
                                        ctypes.c_size_t(8), None)
        assert rc == want


def test_one_token_between_the_rows_of_another():
    """A single row in the gap between another tensor's rows, and on one of them."""
    p = rot_problem(B=1, H=1, Hkv=1, T=1)
    row = t4(0, B=1, H=1, T=1)
    for B, at, want in ((2, 64, ct.LACT_ENOSPC), (2, 128, ct.LACT_EINVAL), (2, 56, ct.LACT_EINVAL)):
        s = swa_problem(B=B, H=1, Hkv=1, T=1, Tq=1)
        far = lambda i: t4(i, B, 1, 1, 64)  # noqa: E731
        dq = _abi.LactTensor4(G, 128, 64, 64)
        dk = _abi.LactTensor4(G + 2 * at, 128, 64, 64)
        rc = ct.lib().lact_swa_sink_bwd(ref(s), ref(far(20)), ref(far(21)), ref(far(22)), ref(far(23)), 9 * G, ref(far(24)),
                                        None, ref(dq), ref(dk), ref(far(25)), 10 * G, ctypes.c_size_t(8), None)
        assert rc == want, at
    assert rotary_bwd_rc(p, row, t4(1, B=1, H=1, T=1), row, t4(0, B=1, H=1, T=1, at=16)) == ct.LACT_EINVAL


@pytest.mark.parametrize("over", [1, 1024])
def test_caches_past_the_kernels_32_bit_slots_refused(over):
    """The last slots' numbers, rounded up, have to fit 32 bits; checked before anything is enqueued."""
    window = (1 << 30) - 1024 + over
    p = swa_problem(B=1, H=1, Hkv=1, T=1, Tq=1, d=8, window=window, sinks=1 << 30)
    one = lambda i: t4(i, 1, 1, 1, 8)  # noqa: E731
    lib, kc, vc = ct.lib(), 100 * G, 200 * G
    assert lib.lact_swa_sink_decode(ref(p), ref(one(0)), ref(one(1)), ref(one(2)), kc, vc, 6 * G, ref(one(7)),
                                    None) == ct.LACT_EINVAL
    assert lib.lact_swa_cache_fill(ref(p), ref(one(0)), ref(one(1)), None, kc, vc, None) == ct.LACT_EINVAL


@pytest.mark.parametrize("sizes", [dict(B=1 << 32, H=1 << 32, Hkv=1 << 32), dict(B=1 << 62, H=4, Hkv=4),
                                   dict(B=4, H=1 << 62, Hkv=1 << 62), dict(B=2, H=1 << 62, Hkv=1 << 62)])
def test_products_past_64_bits_refused(sizes):
    """Batches times heads of 2^63 and more, whose product wraps to a small number."""
    lib = ct.lib()
    for T in (1, 64):
        p, r = swa_problem(T=T, Tq=T, **sizes), rot_problem(T=T, **sizes)
        assert lib.lact_swa_sink_bwd_workspace_bytes(ref(p)) == 0
        assert lib.lact_rotary_bwd_workspace_bytes(ref(r)) == 0
        t = lambda i: t4(i, 2, 1, T)  # noqa: E731
        assert lib.lact_swa_sink_fwd(ref(p), ref(t(0)), ref(t(1)), ref(t(2)), None, ref(t(3)), 9 * G, None) == ct.LACT_EINVAL
        assert lib.lact_rotary_fwd(ref(r), ref(t(0)), ref(t(1)), 9 * G, *[None] * 5, ref(t(2)), ref(t(3)), None) == ct.LACT_EINVAL
    p = swa_problem(T=1, Tq=1, **sizes)
    t = lambda i: t4(i, 2, 1, 1)  # noqa: E731
    assert lib.lact_swa_sink_decode(ref(p), ref(t(0)), ref(t(1)), ref(t(2)), 4 * G, 5 * G, 6 * G, ref(t(7)),
                                    None) == ct.LACT_EINVAL
    assert lib.lact_swa_cache_fill(ref(p), ref(t(0)), ref(t(1)), None, 4 * G, 5 * G, None) == ct.LACT_EINVAL


def test_cache_fill_has_no_use_for_queries():
    """H and Tq may hold anything.  The last check before the launch, the caches'
    overlap, cannot tell (it gives LACT_EINVAL too), so the call is made from a
    child whose device is hidden: past the checks it finds none."""
    import os
    import subprocess
    import sys
    code = ("import ctypes, chunk_test_b200 as ct\n"
            "from tests.test_attention_host import swa_problem, t4, G, ref\n"
            "for H, Tq in ((0, 64), (3, 64), (-1, 0), (1 << 40, 1 << 40)):\n"
            "    p = swa_problem(H=H, Tq=Tq)\n"
            "    rc = ct.lib().lact_swa_cache_fill(ref(p), ref(t4(0, H=2)), ref(t4(1, H=2)), None, 4 * G, 5 * G, None)\n"
            "    assert rc == -3, (H, Tq, rc)\n"
            "assert ct.lib().lact_swa_cache_fill(None, None, None, None, None, None, None) == -1\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                         env={**os.environ, "CUDA_VISIBLE_DEVICES": "", "PYTHONPATH": root})
    assert run.returncode == 0, run.stderr


def test_accepted_layouts_share_no_address():
    """Random strides and offsets of dq and dk in one small buffer: what is
    accepted (LACT_ENOSPC, see rotary_bwd_rc) shares no element, and nothing is
    written twice."""
    import itertools
    import random
    rng = random.Random(0)
    far = {}
    seen = {ct.LACT_ENOSPC: 0, ct.LACT_EINVAL: 0}
    packed = 0

    def elements(at, strides, n):
        return [at + sum(i * s for i, s in zip(ix, strides)) + c
                for ix in itertools.product(*(range(x) for x in n)) for c in range(8)]

    for _ in range(4000):
        B, Hkv, T = (rng.choice([1, 2, 3]) for _ in range(3))
        H = Hkv * rng.choice([1, 2])
        p = swa_problem(B=B, H=H, Hkv=Hkv, T=T, Tq=T, d=8)
        key = (B, H, Hkv, T)
        if key not in far:
            far[key] = [t4(20 + i, B, h, T, 8) for i, h in enumerate((H, Hkv, Hkv, H, H, Hkv))]
        x = far[key]
        if rng.random() < 0.5:    # nested in some order, with gaps
            row, order = 8, rng.sample(range(3), 3)
            one = [0, 0, 0]
            for i in order:
                row *= rng.choice([1, 2, 3])
                one[i] = row
                row *= (B, H, T)[i]
            other = list(one) if rng.random() < 0.7 else [8 * rng.randint(1, 30) for _ in range(3)]
        else:
            one, other = ([8 * rng.randint(1, 30) for _ in range(3)] for _ in range(2))
        at = 8 * rng.randint(0, 40)
        dq, dk = _abi.LactTensor4(G, *one), _abi.LactTensor4(G + 2 * at, *other)
        rc = ct.lib().lact_swa_sink_bwd(ref(p), ref(x[0]), ref(x[1]), ref(x[2]), ref(x[3]), 9 * G, ref(x[4]), None,
                                        ref(dq), ref(dk), ref(x[5]), 10 * G, ctypes.c_size_t(8), None)
        seen[rc] += 1
        if rc != ct.LACT_ENOSPC:
            continue
        a, b = elements(0, one, (B, H, T)), elements(at, other, (B, Hkv, T))
        assert len(set(a)) == len(a) and len(set(b)) == len(b), (key, one, other)
        assert not set(a) & set(b), (key, one, other, at)
        packed += max(a) > min(b) and max(b) > min(a)
    assert packed > 100 and min(seen.values()) > 500, (packed, seen)
