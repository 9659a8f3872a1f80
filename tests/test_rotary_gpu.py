"""GPU tests of the rotary positions and their backward against the fp64
definitions (oracle/attention_oracle.py).

Bounds, elementwise.  The angle's turn is formed in 64 bits and handed to
sincospi in 32: at most 2^-24 of a half turn and a few 2^-24 of sincospi, so
cos and sin are within 2^-21; two products and a sum add 3 * 2^-24 of the
operands, the scale and offset 2^-23.  So 32-bit results are within
2^-20 amp (|x'_a| + |x'_b|), and a bf16 result adds its rounding, 2^-8 |y|.
The parameters' gradients are sums in 32 bits through chains of at most 400
additions here: 400 * 2^-24 + 2^-20 of the sum of absolute values."""
import pytest
import torch

import chunk_test_b200 as ct
from oracle import attention_oracle as ao

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def inputs(B, H, Hkv, T, d, dtype, layout="bhtd", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def one(heads):
        if layout == "bthd":
            return torch.randn((B, T, heads, d), generator=g, device="cuda").to(dtype).transpose(1, 2)
        return torch.randn((B, heads, T, d), generator=g, device="cuda").to(dtype)

    return one(H), one(Hkv), g


def params(H, Hkv, d, g):
    return dict(q_scale=1 + 0.2 * torch.randn((H, d), generator=g, device="cuda"),
                q_offset=0.2 * torch.randn((H, d), generator=g, device="cuda"),
                k_scale=1 + 0.2 * torch.randn((Hkv, d), generator=g, device="cuda"),
                k_offset=0.2 * torch.randn((Hkv, d), generator=g, device="cuda"))


def partner_sum(x, rot, interleaved):
    """|x_a| + |x_b| of each channel's pair."""
    a = x.abs()
    y = a.clone()
    if interleaved:
        s = a[..., 0:rot:2] + a[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = s, s
    else:
        s = a[..., :rot // 2] + a[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = s, s
    return y


def check(got, want, pair, amp):
    u = U[got.dtype] if got.dtype == torch.bfloat16 else 0.0
    bound = u * want.abs() + (1 + 2 * u) * 2.0 ** -20 * max(1.0, abs(amp)) * pair + 1e-30
    over = (got.double() - want).abs() / bound
    assert bool(torch.isfinite(got).all())
    assert float(over.max()) <= 1.0, float(over.max())


CASES = [
    # B, H, Hkv, T, d, rot, interleaved, affine, dtype, layout
    (1, 1, 1, 1, 64, 64, False, False, torch.bfloat16, "bhtd"),
    (2, 3, 1, 5, 128, 128, True, True, torch.bfloat16, "bthd"),
    (1, 2, 2, 130, 256, 256, False, True, torch.bfloat16, "bhtd"),
    (1, 2, 1, 77, 96, 48, False, True, torch.bfloat16, "bthd"),       # pairs 24: whole vectors
    (1, 2, 1, 77, 96, 50, False, True, torch.bfloat16, "bthd"),       # pairs 25: single channels
    (2, 2, 2, 33, 80, 2, False, False, torch.bfloat16, "bhtd"),       # one pair, 78 channels pass
    (2, 2, 2, 33, 80, 2, True, True, torch.bfloat16, "bhtd"),
    (1, 1, 1, 65, 8, 6, True, True, torch.bfloat16, "bhtd"),
    (1, 1, 1, 3, 512, 512, False, True, torch.bfloat16, "bhtd"),
    (1, 1, 1, 3, 512, 2, False, True, torch.bfloat16, "bhtd"),        # 511 units of a row
    (1, 3, 1, 200, 96, 96, True, True, torch.float32, "bthd"),
    (1, 2, 2, 64, 64, 24, False, True, torch.float32, "bhtd"),
    (1, 2, 2, 64, 64, 26, False, False, torch.float32, "bhtd"),
    (3, 4, 2, 700, 128, 64, False, True, torch.bfloat16, "bthd"),
]


@pytest.mark.parametrize("B,H,Hkv,T,d,rot,inter,affine,dtype,layout", CASES)
def test_forward_and_backward(B, H, Hkv, T, d, rot, inter, affine, dtype, layout):
    q, k, g = inputs(B, H, Hkv, T, d, dtype, layout, seed=T)
    freqs, _ = ct.rotary_frequencies(rot)
    pos = torch.arange(T, device="cuda").expand(B, T)
    kw = params(H, Hkv, d, g) if affine else {}
    amp = 1.25
    got = ct.rotary_fwd(q, k, freqs, interleaved=inter, amplitude=amp, **kw)
    for x, y, n in ((q, got[0], "q"), (k, got[1], "k")):
        sc, of = kw.get(n + "_scale"), kw.get(n + "_offset")
        want = ao.rotary(x, freqs, pos, inter, amp, sc, of)
        xp = x.double() if sc is None else x.double() * sc.double()[:, None] + of.double()[:, None]
        size = x.double().abs() if sc is None else (x.double() * sc.double()[:, None]).abs() + of.double().abs()[:, None]
        check(y, want, partner_sum(torch.maximum(xp.abs(), size), rot, inter), amp)

    dq, dk, _ = inputs(B, H, Hkv, T, d, dtype, "bhtd", seed=T + 1)
    more = dict(q=q, k=k, **kw) if affine else {}
    res = ct.rotary_bwd(dq, dk, freqs, interleaved=inter, amplitude=amp, **more)
    for dy, x, n in ((dq, q, "q"), (dk, k, "k")):
        sc = kw.get(n + "_scale")
        dx, ds, do, ads, ado = ao.rotary_vjp(dy, freqs, pos, inter, amp, x, sc)
        pair = partner_sum(dy.double(), rot, inter)
        check(res["d" + n], dx, pair if sc is None else pair * sc.double().abs()[:, None], amp)
        if sc is None:
            assert res[f"d{n}_scale"] is None and res[f"d{n}_offset"] is None
            continue
        t = 400 * 2.0 ** -24 + 2.0 ** -20 * amp
        slack = 2.0 ** -20 * amp * (pair * x.double().abs()).sum((0, 2)), 2.0 ** -20 * amp * pair.sum((0, 2))
        assert bool(((res[f"d{n}_scale"].double() - ds).abs() <= t * ads + slack[0]).all())
        assert bool(((res[f"d{n}_offset"].double() - do).abs() <= t * ado + slack[1]).all())
    assert ct.status() == ct.LACT_OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_far_positions(dtype):
    """Positions around 2^30, where a 32-bit angle has no fraction left."""
    B, H, T, d = 2, 2, 9, 64
    q, k, g = inputs(B, H, 1, T, d, dtype)
    freqs, _ = ct.rotary_frequencies(d)
    pos = torch.randint(0, 2 ** 30, (B, T), generator=g, device="cuda").to(torch.int32)
    got = ct.rotary_fwd(q, k, freqs, positions=pos)
    # 64-bit angles up to 2^30 radians leave 2^-23 of a radian
    for x, y in ((q, got[0]), (k, got[1])):
        want = ao.rotary(x, freqs, pos, False)
        check(y, want, partner_sum(x.double(), d, False), 1.0)
    start = ct.rotary_fwd(q, None, freqs, start=2 ** 33 + 5)[0]
    want = ao.rotary(q, freqs, (torch.arange(T, device="cuda", dtype=torch.float64) + 2 ** 33 + 5).expand(B, T), False)
    # 2^33 radians: the product's last bit is 2^-19 of a radian here and in the oracle
    bound = (2.0 ** -8 if dtype == torch.bfloat16 else 0.0) * want.abs() + 2.0 ** -17 * partner_sum(q.double(), d, False)
    assert bool(((start.double() - want).abs() <= bound).all())


def test_in_place_packed_and_repeatable():
    """q and k as slices of one packed projection, rotated in place; the other
    slice stays; the parameters' gradients have the same bits on every run."""
    B, T, H, d = 2, 150, 3, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn((B, T, 3 * H, d), generator=g, device="cuda").bfloat16()
    kept = qkv.clone()
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:2 * H].transpose(1, 2)
    freqs, _ = ct.rotary_frequencies(d)
    want = ct.rotary_fwd(q, k, freqs)
    ct.rotary_fwd(q, k, freqs, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[:, :, 2 * H:], kept[:, :, 2 * H:])
    kw = params(H, H, d, g)
    a, b = (ct.rotary_bwd(want[0], want[1], freqs, q=q, k=k, **kw) for _ in range(2))
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_backward_is_the_forwards_gradient():
    """<dy, f(x + e) - f(x)> against <dx, e> for the linear map in x, in float32."""
    q, k, g = inputs(1, 2, 1, 40, 64, torch.float32)
    freqs, amp = ct.rotary_frequencies(48, method="by_parts", factor=4.0, context=16)
    kw = params(2, 1, 64, g)
    dq, dk, _ = inputs(1, 2, 1, 40, 64, torch.float32, seed=9)
    e, _, _ = inputs(1, 2, 1, 40, 64, torch.float32, seed=10)
    y0 = ct.rotary_fwd(q, k, freqs, amplitude=amp, **kw)[0].double()
    y1 = ct.rotary_fwd(q + e, k, freqs, amplitude=amp, **kw)[0].double()
    res = ct.rotary_bwd(dq, dk, freqs, amplitude=amp, q=q, k=k, **kw)
    lhs, rhs = float((dq.double() * (y1 - y0)).sum()), float((res["dq"].double() * e.double()).sum())
    size = float((dq.abs() * (y0.abs() + y1.abs())).sum())
    assert abs(lhs - rhs) <= 2.0 ** -18 * size, (lhs, rhs)


def test_captured_and_replayed():
    """A captured forward and backward, replayed on new values in the same buffers."""
    q, k, g = inputs(2, 2, 1, 70, 64, torch.bfloat16)
    freqs, _ = ct.rotary_frequencies(64)
    kw = params(2, 1, 64, g)
    ct.rotary_bwd(*ct.rotary_fwd(q, k, freqs, **kw), freqs, q=q, k=k, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ct.rotary_fwd(q, k, freqs, **kw)
        res = ct.rotary_bwd(y[0], y[1], freqs, q=q, k=k, **kw)
    q.copy_(torch.randn(q.shape, generator=g, device="cuda"))
    graph.replay()
    want = ct.rotary_fwd(q, k, freqs, **kw)
    ref = ct.rotary_bwd(want[0], want[1], freqs, q=q, k=k, **kw)
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
    for n in ref:
        assert torch.equal(res[n], ref[n]), n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_queries_alone(dtype):
    """No keys, with the scales' gradients: what q gets beside keys."""
    q, k, g = inputs(2, 3, 2, 50, 64, dtype)
    freqs, _ = ct.rotary_frequencies(32)
    kw = params(3, 2, 64, g)
    mine = {n: x for n, x in kw.items() if n.startswith("q")}
    both, one = ct.rotary_fwd(q, k, freqs, **kw), ct.rotary_fwd(q, None, freqs, **mine)
    assert torch.equal(both[0], one[0]) and one[1] is None
    a = ct.rotary_bwd(q, k, freqs, q=both[0], k=both[1], **kw)
    b = ct.rotary_bwd(q, None, freqs, q=both[0], **mine)
    assert torch.equal(a["dq"], b["dq"]) and b["dk"] is None and b["dk_scale"] is None
    # the tokens are cut differently: two 32-bit sums of 100 terms each, from the same terms
    pos = torch.arange(50, device="cuda").expand(2, 50)
    _, _, _, ads, ado = ao.rotary_vjp(q, freqs, pos, False, 1.0, both[0], kw["q_scale"])
    assert bool(((a["dq_scale"] - b["dq_scale"]).abs() <= 2 * 100 * 2.0 ** -24 * 1.01 * ads).all())
    assert bool(((a["dq_offset"] - b["dq_offset"]).abs() <= 2 * 100 * 2.0 ** -24 * 1.01 * ado).all())


def test_refused_on_the_gpu():
    q, k, g = inputs(1, 2, 1, 8, 64, torch.bfloat16)
    freqs, _ = ct.rotary_frequencies(32)
    kw = params(2, 1, 64, g)
    want = ct.rotary_fwd(q, k, freqs)
    with pytest.raises(ValueError):
        ct.rotary_fwd(q, k, freqs.float())
    with pytest.raises(ValueError):
        ct.rotary_fwd(q, k, freqs, q_scale=kw["q_scale"])                 # all parameters or none
    with pytest.raises(ValueError):
        ct.rotary_fwd(q, None, freqs, **kw)                               # k's without k
    with pytest.raises(ValueError):
        ct.rotary_fwd(q, k, freqs, positions=torch.zeros((1, 8), device="cuda", dtype=torch.int64))
    with pytest.raises(ValueError):
        ct.rotary_bwd(q, k, freqs, q_scale=kw["q_scale"], k_scale=kw["k_scale"])   # the inputs are missing
    with pytest.raises(ct.LactError):
        ct.rotary_fwd(q, k, freqs, out=(k.expand(1, 2, 8, 64), k))        # heads on one place
    with pytest.raises(ct.LactError):
        ct.rotary_fwd(q, k, torch.ones(40, dtype=torch.float64, device="cuda"))    # 80 channels of 64
    with pytest.raises(ct.LactError):
        ct.rotary_fwd(q, k, freqs, start=-1)
    got = ct.rotary_fwd(q, k, freqs)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("layout", ["rows", "heads"])
@pytest.mark.parametrize("B,T", [(1, 1), (5, 1), (3, 7)])
def test_in_place_on_slices_of_one_buffer(B, T, layout):
    """q and k of a packed [B, T, heads, d] or [B, heads, T, d] projection in
    place, the step of one token per sequence among them, and the attention's
    gradients written side by side."""
    H, Hkv, d = 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(B + T)
    shape = (B, T, H + 2 * Hkv, d) if layout == "rows" else (B, H + 2 * Hkv, T, d)
    at = lambda x, i, n: x[:, :, i:i + n].transpose(1, 2) if layout == "rows" else x[:, i:i + n]  # noqa: E731
    qkv = torch.randn(shape, generator=g, device="cuda").bfloat16()
    kept = qkv.clone()
    q, k, v = at(qkv, 0, H), at(qkv, H, Hkv), at(qkv, H + Hkv, Hkv)
    freqs, _ = ct.rotary_frequencies(d)
    want = ct.rotary_fwd(q, k, freqs, start=1000)
    ct.rotary_fwd(q, k, freqs, start=1000, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(v, at(kept, H + Hkv, Hkv))
    back = ct.rotary_bwd(q, k, freqs, start=1000)
    out, lse = ct.swa_sink_fwd(q, k, v, 4, 1)
    ref = ct.swa_sink_bwd(q, k, v, out, lse, out, 4, 1)
    grads = torch.full_like(qkv, 7.0)
    ct.swa_sink_bwd(q, k, v, out, lse, out, 4, 1, dq=at(grads, 0, H), dk=at(grads, H, Hkv), dv=at(grads, H + Hkv, Hkv))
    for i, n, name in ((0, H, "dq"), (H, Hkv, "dk"), (H + Hkv, Hkv, "dv")):
        assert torch.equal(at(grads, i, n), ref[name]), name
    ct.rotary_bwd(q, k, freqs, start=1000, out=(q, k))
    assert torch.equal(q, back["dq"]) and torch.equal(k, back["dk"])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot,bad", [(16, float("nan")), (16, float("inf")), (6, float("nan")), (6, -float("inf"))])
def test_a_frequency_that_is_no_number_shows(rot, bad, inter):
    """Its pair is NaN at every position, in both layouts; the other channels are
    what they are without."""
    q, k, _ = inputs(2, 2, 1, 20, 32, torch.bfloat16)
    freqs, _ = ct.rotary_frequencies(rot)
    want = ct.rotary_fwd(q, k, freqs, interleaved=inter)
    back = ct.rotary_bwd(q, k, freqs, interleaved=inter)
    freqs[1] = bad
    pair = [2, 3] if inter else [1, 1 + rot // 2]
    rest = [c for c in range(32) if c not in pair]
    got, gb = ct.rotary_fwd(q, k, freqs, interleaved=inter), ct.rotary_bwd(q, k, freqs, interleaved=inter)
    for a, b in ((got[0], want[0]), (got[1], want[1]), (gb["dq"], back["dq"]), (gb["dk"], back["dk"])):
        assert bool(torch.isnan(a[..., pair]).all())
        assert torch.equal(a[..., rest], b[..., rest])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hkv,T,d,rot,inter", [
    (13, 3, 37, 256, 256, False),      # 12 heads a block: whole vectors, two blocks of heads
    (40, 8, 21, 128, 64, False),       # pairs and passing channels in one block of several heads
    (30, 5, 33, 96, 50, False),        # single channels: 5 heads a block
    (33, 8, 19, 128, 128, True),
    (1, 1, 700, 8, 8, False),          # one unit a head
])
def test_more_heads_than_a_block_holds(H, Hkv, T, d, rot, inter, dtype):
    q, k, g = inputs(2, H, Hkv, T, d, dtype, "bthd", seed=T)
    dq, dk, _ = inputs(2, H, Hkv, T, d, dtype, seed=T + 1)
    freqs, _ = ct.rotary_frequencies(rot)
    pos = torch.arange(T, device="cuda").expand(2, T)
    kw = params(H, Hkv, d, g)
    got = ct.rotary_fwd(q, k, freqs, interleaved=inter, **kw)
    res = ct.rotary_bwd(dq, dk, freqs, interleaved=inter, q=q, k=k, **kw)
    plain = ct.rotary_bwd(dq, dk, freqs, interleaved=inter)
    for x, y, dy, n in ((q, got[0], dq, "q"), (k, got[1], dk, "k")):
        sc, of = kw[n + "_scale"], kw[n + "_offset"]
        size = (x.double() * sc.double()[:, None]).abs() + of.double().abs()[:, None]
        check(y, ao.rotary(x, freqs, pos, inter, 1.0, sc, of), partner_sum(size, rot, inter), 1.0)
        dx, ds, do, ads, ado = ao.rotary_vjp(dy, freqs, pos, inter, 1.0, x, sc)
        pair = partner_sum(dy.double(), rot, inter)
        check(res["d" + n], dx, pair * sc.double().abs()[:, None], 1.0)
        check(plain["d" + n], ao.rotary_vjp(dy, freqs, pos, inter)[0], pair, 1.0)
        t = 400 * 2.0 ** -24 + 2.0 ** -20
        slack = 2.0 ** -20 * (pair * x.double().abs()).sum((0, 2)), 2.0 ** -20 * pair.sum((0, 2))
        assert bool(((res[f"d{n}_scale"].double() - ds).abs() <= t * ads + slack[0]).all())
        assert bool(((res[f"d{n}_offset"].double() - do).abs() <= t * ado + slack[1]).all())
    assert ct.status() == ct.LACT_OK
