"""GPU tests of the window attention's single-token form over a rolling cache,
of filling the cache from a prompt, and of the attention half's operators run
together.  Bounds: test_swa_sink_gpu.py (forward)."""
import math

import pytest
import torch

import chunk_test_b200 as ct
from oracle import attention_oracle as ao

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def make(B, H, Hkv, C, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    return r(B, H, 1, d), r(B, Hkv, 1, d), r(B, Hkv, 1, d), r(B, Hkv, C, d), r(B, Hkv, C, d)


def check(got, want, pv, dtype, d, n):
    # 32-bit part as in the forward, with |q||k| at most 6 sigma of d terms over sqrt(d)
    e = 2.0 ** -23 * (d * 6 * math.sqrt(d) + n + 32)
    u, r = (2.0 ** -8, 2.0 ** -8) if dtype == BF16 else (2.0 ** -24, 0.0)
    assert bool(torch.isfinite(got).all())
    over = (got.double() - want).abs() / (u * want.abs() + (1 + u) * (r + e) * pv + 1e-30)
    assert float(over.max()) <= 1.0, float(over.max())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hkv,d,window,sinks,seen", [
    (1, 1, 1, 64, 1, 0, (0,)),
    (1, 1, 1, 64, 1, 0, (9,)),
    (3, 2, 1, 64, 5, 2, (0, 2, 100)),
    (2, 6, 6, 256, 300, 4, (303, 304)),            # the cache full, then wrapped
    (2, 12, 4, 128, 1000, 16, (15, 5000)),
    (1, 24, 2, 80, 333, 0, (332,)),                # 12 heads of a group: two blocks of heads
    (4, 3, 1, 192, 129, 1, (-1, 0, 128, 129)),     # an inactive sequence
    (1, 8, 1, 96, 4096, 64, (2 ** 31 - 1,)),       # the last position there is
    (70, 4, 2, 64, 17, 3, tuple(range(70))),
])
def test_decode(B, H, Hkv, d, window, sinks, seen, dtype):
    C = sinks + window
    q, k, v, kc, vc = make(B, H, Hkv, C, d, dtype, seed=window)
    for b, p in enumerate(seen):                   # slots without a token hold anything
        kc[b, :, max(p, 0) + 1:] = math.nan
        vc[b, :, max(p, 0) + 1:] = math.inf
    pos = torch.tensor(seen, dtype=torch.int32, device="cuda")
    want, pv, kw, vw = ao.decode(q, k, v, kc, vc, seen, window, sinks)
    out = ct.swa_sink_decode(q, k, v, kc, vc, pos, window, sinks)
    check(out, want, pv, dtype, d, C)
    assert torch.equal(kc.view(torch.int16 if dtype == BF16 else torch.int32),
                       kw.view(torch.int16 if dtype == BF16 else torch.int32))
    assert torch.equal(vc.view(torch.int16 if dtype == BF16 else torch.int32),
                       vw.view(torch.int16 if dtype == BF16 else torch.int32))
    again = ct.swa_sink_decode(q, k, v, kc, vc, pos, window, sinks)
    assert torch.equal(again, out)
    assert ct.status() == ct.LACT_OK


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,window,sinks", [(5, 8, 2), (10, 8, 2), (11, 8, 2), (100, 8, 0), (100, 1, 3), (7, 16, 9)])
def test_cache_fill(T, window, sinks, dtype):
    B, Hkv, d, C = 3, 2, 64, window + sinks
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn((B, T, Hkv, d), generator=g, device="cuda").to(dtype).transpose(1, 2) for _ in range(2))
    lens = [T, T // 2, 0]
    for lt in (None, lens):
        kc, vc = (torch.full((B, Hkv, C, d), 9.0, dtype=dtype, device="cuda") for _ in range(2))
        ct.swa_cache_fill(k, v, kc, vc, window, sinks,
                          lengths=None if lt is None else torch.tensor(lt, dtype=torch.int32, device="cuda"))
        for x, c in ((k, kc), (v, vc)):
            want = torch.full_like(c, 9.0)
            for b in range(B):
                for p in range(T if lt is None else lt[b]):      # in order: later tokens overwrite
                    want[b, :, p if p < sinks else sinks + (p - sinks) % window] = x[b, :, p]
            assert torch.equal(c, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_then_tokens_is_the_whole_sequence(dtype):
    """A prompt through rotary, attention and the cache, then token by token
    through rotary and the single-token form: the outputs of the attention over
    the whole sequence.  The tokens' steps are one captured graph, replayed."""
    B, H, Hkv, T, P, d, window, sinks = 2, 4, 2, 96, 61, 64, 24, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((B, T, n, d), generator=g, device="cuda").to(dtype).transpose(1, 2) for n in (H, Hkv, Hkv))
    freqs, amp = ct.rotary_frequencies(32, method="linear", factor=2.0)
    qr, kr = ct.rotary_fwd(q, k, freqs, amplitude=amp)
    whole, _ = ct.swa_sink_fwd(qr, kr, v, window, sinks)
    w = ao.attention(qr, kr, v, window, sinks)
    check(whole, w["out"], w["pv"], dtype, d, window + sinks)

    qp, kp = ct.rotary_fwd(q[:, :, :P], k[:, :, :P], freqs, amplitude=amp)
    first, _ = ct.swa_sink_fwd(qp, kp, v[:, :, :P], window, sinks)
    check(first, w["out"][:, :, :P], w["pv"][:, :, :P], dtype, d, window + sinks)
    kc, vc = (torch.empty((B, Hkv, sinks + window, d), dtype=dtype, device="cuda") for _ in range(2))
    ct.swa_cache_fill(kp, v[:, :, :P], kc, vc, window, sinks)
    seen = torch.full((B,), P, dtype=torch.int32, device="cuda")
    token = [x[:, :, P:P + 1].clone() for x in (q, k, v)]

    def step():
        a, b = ct.rotary_fwd(token[0], token[1], freqs, amplitude=amp, positions=seen.view(B, 1))
        o = ct.swa_sink_decode(a, b, token[2], kc, vc, seen, window, sinks)
        seen.add_(1)
        return o

    kept = kc.clone(), vc.clone(), seen.clone()
    step()
    for x, y in zip((kc, vc, seen), kept):
        x.copy_(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step()
    for t in range(P, T):
        for x, y in zip(token, (q, k, v)):
            x.copy_(y[:, :, t:t + 1])
        graph.replay()
        check(o, w["out"][:, :, t:t + 1], w["pv"][:, :, t:t + 1], dtype, d, window + sinks)
    assert int(seen[0]) == T
    assert ct.status() == ct.LACT_OK


def test_on_another_stream():
    """Each call on a stream of its own, ordered by events."""
    q, k, v, kc, vc = make(2, 2, 1, 40, 64, BF16)
    pos = torch.tensor([3, 50], dtype=torch.int32, device="cuda")
    k2, v2 = kc.clone(), vc.clone()
    want = ct.swa_sink_decode(q, k, v, k2, v2, pos, 36, 4)
    side = torch.cuda.Stream()
    out = torch.empty_like(q)
    side.wait_stream(torch.cuda.current_stream())
    ct.swa_sink_decode(q, k, v, kc, vc, pos, 36, 4, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(kc, k2) and torch.equal(vc, v2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_cache_past_32_bit_offsets(dtype):
    """A cache of 2^31 elements and more: the last slots hold the keys that
    matter, the others zeros with scores far below."""
    d, sinks = 256, 4
    window = 2 ** 31 // d + 300
    C = sinks + window
    kc = torch.zeros((1, 1, C, d), dtype=dtype, device="cuda")
    vc = torch.zeros((1, 1, C, d), dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    q, k, v = (torch.randn((1, 1, 1, d), generator=g, device="cuda").to(dtype) for _ in range(3))
    # scores near 40 against 0 for the zero keys: exp(-40) * 2^23 of them leave 2^-34 of the weight
    tail = torch.randn((16, d), generator=g, device="cuda")
    qf = q[0, 0, 0].float()
    tail += (40.0 * 16.0 - tail @ qf)[:, None] * qf / (qf @ qf)
    kc[0, 0, -16:] = tail.to(dtype)
    vc[0, 0, -16:] = torch.randn((16, d), generator=g, device="cuda").to(dtype)
    k.copy_(kc[0, 0, -1])
    pos = torch.tensor([C - 2], dtype=torch.int32, device="cuda")    # the new token takes the slot before the last
    out = ct.swa_sink_decode(q, k, v, kc, vc, pos, window, sinks)
    keys = torch.cat((kc[0, 0, -16:-2], k[0, 0])).double()
    vals = torch.cat((vc[0, 0, -16:-2], v[0, 0])).double()
    p = torch.softmax(keys @ q[0, 0, 0].double() / math.sqrt(d), 0)
    assert torch.equal(kc[0, 0, -2], k[0, 0, 0]) and torch.equal(vc[0, 0, -2], v[0, 0, 0])
    # the zero keys' weight is below 2^-30 of the sum; scores of 40 in 32 bits are off by 2^-18 of them at most
    over = (out[0, 0, 0].double() - p @ vals).abs()
    u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    bound = u * (p @ vals).abs() + ((u if dtype == BF16 else 0) + 2.0 ** -12) * (p @ vals.abs())
    assert float((over / bound).max()) <= 1.0, float((over / bound).max())


def test_refused_on_the_gpu():
    q, k, v, kc, vc = make(2, 2, 1, 40, 64, BF16)
    pos = torch.tensor([3, 50], dtype=torch.int32, device="cuda")
    want = ct.swa_sink_decode(q, k, v, kc, vc, pos, 36, 4)
    with pytest.raises(ValueError):
        ct.swa_sink_decode(q, k, v, kc, vc, pos, 37, 4)          # not the cache's size
    with pytest.raises(ValueError):
        ct.swa_sink_decode(q, k, v, kc[:, :, :39], vc, pos, 36, 4)
    with pytest.raises(ValueError):
        ct.swa_sink_decode(q.expand(2, 2, 3, 64), k, v, kc, vc, pos, 36, 4)
    with pytest.raises(ValueError):
        ct.swa_sink_decode(q, k, v, kc, vc, pos.long(), 36, 4)
    with pytest.raises(ct.LactError):
        ct.swa_sink_decode(q, k, v, kc, kc, pos, 36, 4)          # one buffer for both
    assert torch.equal(ct.swa_sink_decode(q, k, v, kc, vc, pos, 36, 4), want)
