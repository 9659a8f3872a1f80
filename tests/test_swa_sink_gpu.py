"""GPU tests of the window attention with sinks, its backward and its
single-token form against the fp64 definitions (oracle/attention_oracle.py).

Bounds, elementwise, u = 2^-8 for bf16 (half a step), e the 32-bit part.
Forward: the probabilities of the second product are rounded (u), the result
is rounded (u):  |err| <= u (|out| + sum p |v|) + e (...).
Backward: dv like the forward; ds is rounded (u |ds|), and out, which delta is
formed from, was rounded and carries the forward's error, so delta is off by
u sum |dout| (|out| + sum p |v|):  |dk err| <= u (|dk| + sum (|ds| + own) |q|),
own = p scale times that sum without u.
32-bit part: a score is off by 2^-23 d sum |q||k| scale at most (products
exact, a chain of d additions), exp and the sums add a few 2^-23 each per
addition: e = 2^-23 (d qk + n + 32) with qk the largest sum scale |q||k| and n
the longest row or column of a sum.  float32 results have u = 2^-24 and no
rounded factors; their products' terms are bounded by the sums themselves."""
import math

import pytest
import torch

import chunk_test_b200 as ct
from oracle import attention_oracle as ao

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(B, H, Hkv, T, Tq, d, dtype, layout="bhtd", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def one(heads, n):
        if layout == "bthd":
            return torch.randn((B, n, heads, d), generator=g, device="cuda").to(dtype).transpose(1, 2)
        return torch.randn((B, heads, n, d), generator=g, device="cuda").to(dtype)

    return one(H, Tq), one(Hkv, T), one(Hkv, T), one(H, Tq)


def within(name, got, want, bound):
    assert bool(torch.isfinite(got).all()), name
    over = (got.double() - want).abs() / (bound + 1e-30)
    assert float(over.max()) <= 1.0, (name, float(over.max()))


def check_forward(got, lse, w, dtype, d, n):
    e = 2.0 ** -23 * (d * w["qk"] + n + 32)
    u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    p_round = u if dtype == BF16 else 0.0
    within("out", got, w["out"], u * w["out"].abs() + (1 + u) * (p_round + e) * w["pv"])
    empty = torch.isinf(w["lse"])
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert bool((got[empty] == 0).all())
    diff = (lse.double() - w["lse"])[~empty].abs()
    assert diff.numel() == 0 or float((diff - 2.0 ** -23 * w["lse"][~empty].abs()).max()) <= e


def check_backward(res, w, dtype, d, n):
    e = 2.0 ** -23 * (2 * d * max(w["qk"], 1.0) + n + 64)
    u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    r = u if dtype == BF16 else 0.0
    within("dq", res["dq"], w["dq"], u * w["dq"].abs() + (1 + u) * (r * w["adq"] + e * w["ddq"]))
    within("dk", res["dk"], w["dk"], u * w["dk"].abs() + (1 + u) * (r * w["adk"] + e * w["ddk"]))
    within("dv", res["dv"], w["dv"], u * w["dv"].abs() + (1 + u) * (r + e) * w["adv"])


CASES = [
    # B, H, Hkv, T, Tq, d, window, sinks, lengths, layout
    (1, 1, 1, 1, 1, 64, 1, 0, None, "bhtd"),
    (1, 2, 1, 2, 2, 64, 2, 0, None, "bhtd"),
    (1, 2, 2, 77, 77, 64, 32, 1, None, "bhtd"),
    (2, 2, 1, 128, 128, 64, 128, 0, None, "bthd"),
    (1, 2, 1, 129, 129, 128, 64, 4, None, "bthd"),
    (1, 3, 1, 300, 300, 128, 1, 3, None, "bhtd"),           # the token itself and three sinks
    (1, 1, 1, 400, 400, 64, 100, 130, None, "bhtd"),        # sinks over more than one tile
    (1, 2, 2, 511, 511, 80, 1000, 2, None, "bthd"),         # window longer than the sequence
    (1, 2, 1, 640, 640, 256, 256, 0, None, "bhtd"),
    (1, 1, 1, 700, 700, 192, 129, 16, None, "bthd"),
    (1, 2, 1, 513, 200, 96, 130, 5, None, "bthd"),          # the last 200 positions
    (1, 1, 1, 600, 1, 64, 70, 5, None, "bhtd"),             # the last position
    (4, 2, 1, 260, 260, 64, 50, 4, (260, 0, 129, 1), "bhtd"),   # an empty sequence and ragged ends
    (3, 4, 2, 300, 150, 128, 64, 8, (300, 170, 149), "bthd"),   # no query of the last one is left
    (2, 6, 2, 1500, 1500, 64, 200, 4, None, "bhtd"),        # far parts of the sinks' gradients
    (1, 1, 1, 2600, 2600, 8, 40, 200, (2500,), "bhtd"),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hkv,T,Tq,d,window,sinks,lengths,layout", CASES)
def test_forward_and_backward(B, H, Hkv, T, Tq, d, window, sinks, lengths, layout, dtype):
    q, k, v, dout = make(B, H, Hkv, T, Tq, d, dtype, layout, seed=T + d)
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = ct.swa_sink_fwd(q, k, v, window, sinks, lengths=lens)
    assert ct.status() == ct.LACT_OK
    w = ao.attention(q, k, v, window, sinks, lengths, dout=dout)
    check_forward(out, lse, w, dtype, d, min(T, window + sinks))
    res = ct.swa_sink_bwd(q, k, v, out, lse, dout, window, sinks, lengths=lens)
    assert ct.status() == ct.LACT_OK
    check_backward(res, w, dtype, d, T * (H // Hkv))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_padding_is_never_used(dtype):
    """NaN and infinities behind the lengths, in every input: rows there get
    out 0, lse -inf and gradients 0, the others are what they are without."""
    B, H, Hkv, T, d, window, sinks = 3, 2, 1, 300, 64, 90, 4
    lens = [300, 140, 3]
    q, k, v, dout = make(B, H, Hkv, T, T, d, dtype)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean = ct.swa_sink_fwd(q, k, v, window, sinks, lengths=lt)
    g_clean = ct.swa_sink_bwd(q, k, v, *clean, dout, window, sinks, lengths=lt)
    for x, bad in ((q, math.nan), (k, math.inf), (v, math.nan), (dout, -math.inf)):
        for b, n in enumerate(lens):
            x[b, :, n:] = bad
    out, lse = ct.swa_sink_fwd(q, k, v, window, sinks, lengths=lt)
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    for b, n in enumerate(lens):
        assert bool((out[b, :, n:] == 0).all()) and bool((lse[b, :, n:] == -math.inf).all())
        out[b, :, n:] = math.nan
    res = ct.swa_sink_bwd(q, k, v, out, lse, dout, window, sinks, lengths=lt)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(res[n], g_clean[n]), n
        for b, m in enumerate(lens):
            assert bool((res[n][b, :, m:] == 0).all())
    assert ct.status() == ct.LACT_OK


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_scores(dtype):
    """Scores in the hundreds that rise along the keys, so the running maximum grows tile after tile."""
    B, H, T, d, window = 1, 1, 700, 64, 600
    q, k, v, dout = make(B, H, H, T, T, d, dtype)
    q.fill_(1.0)
    k.copy_((torch.arange(T, device="cuda", dtype=torch.float32) / 8).view(1, 1, T, 1).expand_as(k))
    out, lse = ct.swa_sink_fwd(q, k, v, window, 2)
    w = ao.attention(q, k, v, window, 2, dout=dout)
    check_forward(out, lse, w, dtype, d, window)
    check_backward(ct.swa_sink_bwd(q, k, v, out, lse, dout, window, 2), w, dtype, d, T)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scale_outputs_and_repeats(dtype):
    """An own scale, outputs in a [B, T, H, d] layout, a workspace with other
    contents: the same bits each time, nothing written beside the outputs."""
    B, H, Hkv, T, d, window, sinks = 2, 2, 1, 333, 64, 60, 4
    q, k, v, dout = make(B, H, Hkv, T, T, d, dtype, "bthd")
    out, lse = ct.swa_sink_fwd(q, k, v, window, sinks, scale=0.3)
    w = ao.attention(q, k, v, window, sinks, scale=0.3, dout=dout)
    check_forward(out, lse, w, dtype, d, window + sinks)
    first = ct.swa_sink_bwd(q, k, v, out, lse, dout, window, sinks, scale=0.3)
    check_backward(first, w, dtype, d, T * 2)

    def packed(heads):
        whole = torch.full((B, T, heads + 2, d), 7.0, dtype=dtype, device="cuda")
        return whole, whole[:, :, 1:-1].transpose(1, 2)

    (wo, o2), (wq, dq), (wk, dk), (wv, dv) = packed(H), packed(H), packed(Hkv), packed(Hkv)
    ct.swa_sink_fwd(q, k, v, window, sinks, scale=0.3, out=o2)
    ws = torch.full((ct.swa_sink_bwd_workspace_bytes(q, k, window, sinks),), 255, dtype=torch.uint8, device="cuda")
    ct.swa_sink_bwd(q, k, v, o2, lse, dout, window, sinks, scale=0.3, dq=dq, dk=dk, dv=dv, workspace=ws)
    for whole, got, ref in ((wo, o2, out), (wq, dq, first["dq"]), (wk, dk, first["dk"]), (wv, dv, first["dv"])):
        assert torch.equal(got, ref)
        assert bool((whole[:, :, 0] == 7).all()) and bool((whole[:, :, -1] == 7).all())


def test_backward_is_the_forwards_gradient():
    """Differences in 64 bits of the float32 kernel's own forward along a direction."""
    q, k, v, dout = make(1, 2, 1, 150, 150, 64, F32, seed=5)
    out, lse = ct.swa_sink_fwd(q, k, v, 40, 3)
    res = ct.swa_sink_bwd(q, k, v, out, lse, dout, 40, 3)
    h = 2.0 ** -6
    for i, n in enumerate(("dq", "dk", "dv")):
        x = [q, k, v]
        e = torch.randn(x[i].shape, generator=torch.Generator(device="cuda").manual_seed(20 + i), device="cuda")
        up, dn = list(x), list(x)
        up[i], dn[i] = x[i] + h * e, x[i] - h * e
        f = [float((ct.swa_sink_fwd(*y, 40, 3)[0].double() * dout.double()).sum()) for y in (up, dn)]
        diff, want = (f[0] - f[1]) / (2 * h), float((res[n].double() * e.double()).sum())
        # the third derivative's share, h^2 / 6 of terms as large as the gradient's, and 32-bit noise over h
        size = float((res[n].double() * e.double()).abs().sum())
        noise = 2.0 ** -20 * float((out.double() * dout.double()).abs().sum()) / h
        assert abs(diff - want) <= h * h * size + noise, (n, diff, want)


def test_long_sequence_far_sinks():
    """The sinks' gradients over many far parts, bf16, on one head."""
    T, d, window, sinks = 9000, 64, 128, 4
    q, k, v, dout = make(1, 1, 1, T, T, d, BF16)
    out, lse = ct.swa_sink_fwd(q, k, v, window, sinks)
    w = ao.attention(q, k, v, window, sinks, dout=dout)
    check_forward(out, lse, w, BF16, d, window + sinks)
    check_backward(ct.swa_sink_bwd(q, k, v, out, lse, dout, window, sinks), w, BF16, d, T)


def test_captured_and_replayed():
    """A captured forward and backward, replayed on new values in the same
    buffers, twice, while an uncaptured call of the same inputs runs before."""
    q, k, v, dout = make(2, 4, 2, 400, 400, 128, BF16, "bthd")
    lens = torch.tensor([400, 131], dtype=torch.int32, device="cuda")

    def step():
        out, lse = ct.swa_sink_fwd(q, k, v, 100, 4, lengths=lens)
        return [out, lse] + list(ct.swa_sink_bwd(q, k, v, out, lse, dout, 100, 4, lengths=lens).values())

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (5, 6):
        for x, y in zip((q, k, v, dout), make(2, 4, 2, 400, 400, 128, BF16, "bthd", seed=seed)):
            x.copy_(y)
        lens.copy_(torch.tensor([400 - seed, 200 + seed], dtype=torch.int32))
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    assert ct.status() == ct.LACT_OK


def test_two_streams_at_once():
    """Backward passes in flight on two streams, each with its own workspace, give what they give alone."""
    cases = [make(1, 4, 2, 1500, 1500, d, BF16, seed=d) for d in (128, 256)]
    fwd = [ct.swa_sink_fwd(q, k, v, 300, 4) for q, k, v, _ in cases]
    alone = [ct.swa_sink_bwd(q, k, v, *f, g, 300, 4) for (q, k, v, g), f in zip(cases, fwd)]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    res = [[], []]
    for _ in range(3):
        for i, ((q, k, v, g), f) in enumerate(zip(cases, fwd)):
            with torch.cuda.stream(streams[i]):
                res[i].append(ct.swa_sink_bwd(q, k, v, *f, g, 300, 4))
    torch.cuda.synchronize()
    for i in range(2):
        for r in res[i]:
            for n in r:
                assert torch.equal(r[n], alone[i][n]), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hkv,d", [(1, 16, 1, 64), (5, 3, 3, 40), (130, 2, 1, 16)])
def test_many_heads_and_batches(B, H, Hkv, d, dtype):
    T, window, sinks = 140, 33, 2
    q, k, v, dout = make(B, H, Hkv, T, T, d, dtype)
    out, lse = ct.swa_sink_fwd(q, k, v, window, sinks)
    w = ao.attention(q, k, v, window, sinks, dout=dout)
    check_forward(out, lse, w, dtype, d, window + sinks)
    check_backward(ct.swa_sink_bwd(q, k, v, out, lse, dout, window, sinks), w, dtype, d, T * (H // Hkv))


def test_refused_on_the_gpu():
    q, k, v, dout = make(1, 2, 1, 64, 64, 64, BF16)
    out, lse = ct.swa_sink_fwd(q, k, v, 8, 1)
    with pytest.raises(ct.LactError):
        ct.swa_sink_fwd(q, k, v, 0, 1)                           # no window
    with pytest.raises(ct.LactError):
        ct.swa_sink_fwd(q, k, v, 8, -1)
    with pytest.raises(ct.LactError):
        ct.swa_sink_fwd(q, k, v, 8, 1, scale=-1.0)
    with pytest.raises(ct.LactError):
        ct.swa_sink_fwd(q, k, v, 8, 1, out=q)                    # onto an input
    with pytest.raises(ct.LactError):
        ct.swa_sink_bwd(q, k, v, out, lse, dout[:, :1].expand(1, 2, 64, 64)[:, :, :1].expand_as(q), 8, 1)  # stride 0
    with pytest.raises(ValueError):
        ct.swa_sink_fwd(q, k.float(), v, 8, 1)
    with pytest.raises(ValueError):
        ct.swa_sink_fwd(q, k, v[:, :, :-1], 8, 1)
    with pytest.raises(ValueError):
        ct.swa_sink_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, v, 8, 1)   # channels apart
    with pytest.raises(ValueError):
        ct.swa_sink_fwd(q, k, v, 8, 1, lengths=torch.tensor([64], device="cuda"))     # int64
    with pytest.raises(ValueError):
        ct.swa_sink_bwd(q, k, v, out, lse, dout, 8, 1, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        ct.swa_sink_fwd(q.half(), k.half(), v.half(), 8, 1)
    assert torch.equal(ct.swa_sink_fwd(q, k, v, 8, 1)[0], out)   # and the next call is as good as the first


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_statistics_at_any_float_address(dtype):
    """lse as a slice of a larger buffer, 4 bytes past a 16-byte boundary."""
    q, k, v, dout = make(1, 1, 1, 131, 131, 64, dtype)
    out, lse = ct.swa_sink_fwd(q, k, v, 20, 2)
    part = torch.full((133,), 7.0, device="cuda")
    at = part[1:132].view(1, 1, 131)
    out2, _ = ct.swa_sink_fwd(q, k, v, 20, 2, lse=at)
    assert torch.equal(out2, out) and torch.equal(at, lse) and float(part[0]) == 7 and float(part[-1]) == 7
    a, b = (ct.swa_sink_bwd(q, k, v, out, x, dout, 20, 2) for x in (lse, at))
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,window,sinks", [(300, 100, 199), (300, 100, 200), (300, 1, 300), (300, 1, 10 ** 6),
                                            (700, 1, 600), (300, 10 ** 9, 5)])
def test_sinks_and_window_up_to_everything(T, window, sinks, dtype):
    """Sinks over most of the sequence, one hidden key, none: causal attention."""
    q, k, v, dout = make(1, 2, 1, T, T, 64, dtype)
    out, lse = ct.swa_sink_fwd(q, k, v, window, sinks)
    w = ao.attention(q, k, v, window, sinks, dout=dout)
    check_forward(out, lse, w, dtype, 64, T)
    check_backward(ct.swa_sink_bwd(q, k, v, out, lse, dout, window, sinks), w, dtype, 64, 2 * T)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lengths_are_clamped(dtype):
    q, k, v, dout = make(3, 1, 1, 150, 150, 64, dtype)
    wide, tight = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ((10 ** 9, -7, 150), (150, 0, 150)))
    a, b = (ct.swa_sink_fwd(q, k, v, 40, 2, lengths=x) for x in (wide, tight))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = (ct.swa_sink_bwd(q, k, v, *a, dout, 40, 2, lengths=x) for x in (wide, tight))
    for n in ga:
        assert torch.equal(ga[n], gb[n]), n


def test_workspace_stays_bounded_with_many_sinks():
    """Half of a long sequence as sinks: the parts' sums are a few per tile."""
    q = torch.empty((1, 1, 32768, 256), dtype=BF16, device="cuda")
    need = ct.swa_sink_bwd_workspace_bytes(q, q, 64, 16384)
    assert need <= 32768 * 4 + 128 * 6 * 2 * 128 * 256 * 4 + 512, need


def test_own_stream_without_a_workspace():
    """stream= alone: the workspace that the call makes lives until that stream is done with it."""
    q, k, v, dout = make(1, 2, 1, 3000, 3000, 128, BF16)
    out, lse = ct.swa_sink_fwd(q, k, v, 200, 4)
    want = ct.swa_sink_bwd(q, k, v, out, lse, dout, 200, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        got.append(ct.swa_sink_bwd(q, k, v, out, lse, dout, 200, 4, stream=side))
        for _ in range(3):   # what would take the dropped workspace on the current stream
            torch.full((ct.swa_sink_bwd_workspace_bytes(q, k, 200, 4),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for g in got:
        for n in g:
            assert torch.equal(g[n], want[n]), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B", [31, 70])
def test_many_ragged_sequences(B, dtype):
    T, window, sinks = 150, 40, 3
    lengths = [(37 * b) % (T + 1) for b in range(B)]
    q, k, v, dout = make(B, 2, 1, T, T, 64, dtype)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = ct.swa_sink_fwd(q, k, v, window, sinks, lengths=lens)
    w = ao.attention(q, k, v, window, sinks, lengths, dout=dout)
    check_forward(out, lse, w, dtype, 64, window + sinks)
    check_backward(ct.swa_sink_bwd(q, k, v, out, lse, dout, window, sinks, lengths=lens), w, dtype, 64, 2 * T)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_ragged_tiles_whose_last_rows_are_missing(d):
    """Several query tiles per CTA, the last of each head with rows for some of
    its warps only (40 and 8 of 128), and tiles wholly behind their sequence's
    length right after tiles with tokens: every row, several times over."""
    H, Hkv, window, sinks = 12, 4, 100, 4
    for T in (7 * 128 + 40, 7 * 128 + 8):
        lengths = [T if b % 3 == 0 else (97 * b) % T for b in range(14)]     # 1344 tiles
        q, k, v, _ = make(14, H, Hkv, T, T, d, BF16, "bthd", seed=T)
        lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        w = ao.attention(q, k, v, window, sinks, lengths)
        first = ct.swa_sink_fwd(q, k, v, window, sinks, lengths=lens)
        check_forward(*first, w, BF16, d, window + sinks)
        for _ in range(10):
            out = torch.full_like(first[0], 7.0)
            again = ct.swa_sink_fwd(q, k, v, window, sinks, lengths=lens, out=out)
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert ct.status() == ct.LACT_OK


def test_own_stream_takes_no_block_in_use():
    """A backward on the current stream and, at once, one on another stream whose
    inputs are there: the second does not take the first one's workspace, which
    went back to the current stream's pool while the first still runs."""
    cases = [make(1, 4, 2, 6000, 6000, 128, BF16, seed=s) for s in (1, 2)]
    fwd = [ct.swa_sink_fwd(q, k, v, 1000, 4) for q, k, v, _ in cases]
    alone = [ct.swa_sink_bwd(q, k, v, *f, g, 1000, 4) for (q, k, v, g), f in zip(cases, fwd)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for (q, k, v, g), f, s in zip(cases, fwd, (None, side)):
            got.append(ct.swa_sink_bwd(q, k, v, *f, g, 1000, 4, stream=s))
        torch.cuda.synchronize()
        for a, b in zip(got, alone):
            for n in a:
                assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hkv,T,Tq,d,window,sinks,lengths,layout", [
    (2, 2, 1, 900, 900, 256, 256, 4, None, "bhtd"),             # the language model's head dim with sinks
    (2, 3, 3, 1500, 1500, 256, 200, 4, (1500, 1130), "bthd"),   # far parts, a length inside a half tile of values
    (4, 4, 2, 400, 400, 256, 100, 4, (400, 0, 193, 63), "bhtd"),
    (2, 2, 1, 700, 333, 256, 130, 8, (700, 650), "bthd"),       # the last 333 positions
    (1, 2, 2, 600, 1, 256, 70, 5, None, "bhtd"),
    (3, 2, 1, 500, 500, 192, 129, 16, (500, 320, 1), "bthd"),
    (2, 2, 2, 513, 200, 192, 130, 5, (513, 449), "bhtd"),
    (3, 4, 1, 700, 700, 128, 100, 16, (700, 450, 64), "bthd"),
    (2, 4, 2, 640, 257, 128, 64, 130, (640, 511), "bhtd"),
    (1, 2, 1, 1100, 1100, 256, 100, 260, (1037,), "bthd"),      # sinks over three tiles
    (2, 1, 1, 300, 300, 200, 64, 3, (300, 129), "bhtd"),        # a padded head dim above 192
])
def test_lengths_sinks_and_late_queries_at_each_head_dim(B, H, Hkv, T, Tq, d, window, sinks, lengths, layout, dtype):
    """Above d 128 the values come in half tiles and the last product's operand is
    refilled by halves: with sinks, lengths and Tq < T, NaN behind the lengths."""
    q, k, v, dout = make(B, H, Hkv, T, Tq, d, dtype, layout, seed=T + d)
    lens = None
    if lengths is not None:
        lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lengths):
            q[b, :, max(n - (T - Tq), 0):] = math.nan
            dout[b, :, max(n - (T - Tq), 0):] = math.nan
            k[b, :, n:], v[b, :, n:] = math.nan, math.inf
    out, lse = ct.swa_sink_fwd(q, k, v, window, sinks, lengths=lens)
    w = ao.attention(q, k, v, window, sinks, lengths, dout=dout)
    check_forward(out, lse, w, dtype, d, min(T, window + sinks))
    res = ct.swa_sink_bwd(q, k, v, out, lse, dout, window, sinks, lengths=lens)
    check_backward(res, w, dtype, d, T * (H // Hkv))
    assert ct.status() == ct.LACT_OK


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("B,H,T", [(8, 8, 1000), (9, 8, 1000), (3, 24, 2600), (8, 2, 300), (40, 6, 700)])
def test_a_ragged_batch_is_its_sequences(B, H, T, d):
    """On both sides of the rules for the order of the tiles: each sequence of a
    ragged batch gets the same bits as alone."""
    window, sinks = 150, 4
    lengths = [(T if b == 1 else (613 * b + 7) % T) for b in range(B)]
    q, k, v, dout = make(B, H, 2, T, T, d, BF16, "bthd", seed=B)
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = ct.swa_sink_fwd(q, k, v, window, sinks, lengths=lens)
    res = ct.swa_sink_bwd(q, k, v, out, lse, dout, window, sinks, lengths=lens)
    for b in range(B):
        x = [t[b:b + 1] for t in (q, k, v)]
        o, l = ct.swa_sink_fwd(*x, window, sinks, lengths=lens[b:b + 1])
        assert torch.equal(out[b:b + 1], o) and torch.equal(lse[b:b + 1], l), b
        g = ct.swa_sink_bwd(*x, o, l, dout[b:b + 1], window, sinks, lengths=lens[b:b + 1])
        assert torch.equal(res["dq"][b:b + 1], g["dq"]), b   # the sinks' far parts follow the batch
    assert ct.status() == ct.LACT_OK
