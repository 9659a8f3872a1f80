"""The operators of the LaCT block's attention half, as cases to be measured:
rotary positions (with the per-channel scales and offsets of the block's
queries and keys), sliding-window attention with first tokens that stay
visible (forward and backward), and its single-token form over a rolling
cache.

`own = False` computes each operator in its plain form, from elementary torch
operations in 32 bits (angles of far positions and sums over all tokens in
64); `own = True` makes the calls of chunk_test_b200.  `exact` restates the
definitions in 64 bits.

Layouts: q [B, H, T, d], k and v [B, Hkv, T, d], query head h reads key head
h // (H / Hkv).  "bthd" cases hold the same tensors as projections leave them,
[B, T, H, d] in memory.  Key j is visible to the query at position i when
j <= i and (j > i - window or j < sinks), both below the sequence's length.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the 760M language model's queries and keys, once per step
        dict(name="rotary-fwd-lm760m-32k", op="rotary_fwd", dtype=BF16, B=2, H=6, Hkv=6, T=32768, d=256, rot=256,
             interleaved=False, affine=True, layout="bhtd", far=0),
        # one decode step of a batch: a single token per sequence, far positions, part of the head rotated
        dict(name="rotary-fwd-token-b8", op="rotary_fwd", dtype=BF16, B=8, H=12, Hkv=4, T=1, d=128, rot=64,
             interleaved=True, affine=False, layout="bthd", far=1000000),
        # the gradients of the same, with those of the learned scales and offsets
        dict(name="rotary-bwd-lm760m-8k", op="rotary_bwd", dtype=BF16, B=2, H=6, Hkv=6, T=8192, d=256, rot=256,
             interleaved=False, affine=True, layout="bhtd", far=0),
        # a float32 fine-tuning run at odd sizes, straight from the projections
        dict(name="rotary-bwd-f32-odd", op="rotary_bwd", dtype=F32, B=1, H=12, Hkv=3, T=4097, d=96, rot=48,
             interleaved=True, affine=True, layout="bthd", far=100000),
        # the 760M language model's window attention over 32K tokens
        dict(name="swa-fwd-lm760m-32k", op="swa_fwd", dtype=BF16, B=2, H=6, Hkv=6, T=32768, Tq=32768, d=256,
             window=2048, sinks=4, ragged=False, layout="bhtd"),
        # a padded batch of prompts, shared key heads, odd lengths
        dict(name="swa-fwd-ragged-gqa", op="swa_fwd", dtype=BF16, B=3, H=12, Hkv=4, T=5000, Tq=5000, d=128,
             window=1000, sinks=16, ragged=True, layout="bthd"),
        # a short prompt, where the launch counts
        dict(name="swa-fwd-short", op="swa_fwd", dtype=BF16, B=1, H=2, Hkv=2, T=77, Tq=77, d=64,
             window=32, sinks=1, ragged=False, layout="bhtd"),
        # the 760M model's training step at 8K tokens
        dict(name="swa-bwd-lm760m-8k", op="swa_bwd", dtype=BF16, B=2, H=6, Hkv=6, T=8192, Tq=8192, d=256,
             window=2048, sinks=4, ragged=False, layout="bhtd"),
        # the same with shared key heads, at odd sizes
        dict(name="swa-bwd-gqa-odd", op="swa_bwd", dtype=BF16, B=2, H=12, Hkv=4, T=4001, Tq=4001, d=128,
             window=1000, sinks=8, ragged=False, layout="bthd"),
        # a float32 check run
        dict(name="swa-bwd-f32", op="swa_bwd", dtype=F32, B=1, H=4, Hkv=4, T=1025, Tq=1025, d=64,
             window=256, sinks=4, ragged=False, layout="bhtd"),
        # one sequence answering: latency
        dict(name="decode-one-lm760m", op="decode", dtype=BF16, B=1, H=6, Hkv=6, d=256, window=2048, sinks=4,
             ragged=False),
        # a serving batch with shared key heads and a long window, at different lengths
        dict(name="decode-batch-gqa", op="decode", dtype=BF16, B=64, H=12, Hkv=4, d=128, window=8192, sinks=64,
             ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary_fwd", "rotary_bwd", "swa_fwd", "swa_bwd", "decode"])
    dtype = F32 if rng.random() < 0.25 else BF16
    hkv = rng.choice([1, 2, 3, 4, 6])
    h = hkv * rng.choice([1, 1, 2, 3, 4])
    b = rng.choice([1, 2, 3, 5])
    d = rng.choice([64, 64, 80, 96, 128, 128, 192, 256])
    layout = rng.choice(["bhtd", "bthd"])
    size = 4 if dtype == F32 else 2
    if op.startswith("rotary"):
        most = (3 << 27) // (b * (h + hkv) * d * size)
        return dict(op=op, dtype=dtype, B=b, H=h, Hkv=hkv, T=_log(rng, 1, min(32768, most)), d=d,
                    rot=2 * rng.randint(1, d // 2), interleaved=rng.random() < 0.5, affine=rng.random() < 0.5,
                    layout=layout, far=rng.choice([0, 5000, 1000000]))
    if op == "decode":
        b = rng.choice([1, 2, 7, 16, 33, 64])
        most = (1 << 29) // (b * hkv * d * size)
        return dict(op=op, dtype=dtype, B=b, H=h, Hkv=hkv, d=d, window=_log(rng, 1, min(16384, most)),
                    sinks=rng.choice([0, 1, 4, 64]), ragged=rng.random() < 0.5)
    # the scores' work is bounded to a part of the largest listed case's, in 32 bits to less
    w = _log(rng, 2, 4096)
    most = min((1 << 24 if dtype == F32 else 1 << 28) // (b * h * w), 100000000 // (b * h * d))
    t = _log(rng, 2, max(2, min(32768 if op == "swa_fwd" else 8192, most)))
    tq = t if rng.random() < 0.7 else rng.randint(1, t)
    return dict(op=op, dtype=dtype, B=b, H=h, Hkv=hkv, T=t, Tq=tq, d=d, window=w, sinks=rng.choice([0, 1, 4, 16, 130]),
                ragged=rng.random() < 0.4, layout=layout)


# --------------------------------------------------------------------------- inputs
def _randn(g, shape, dtype, layout="bhtd"):
    """N(0, 1) as [B, H, T, d]; with "bthd" the memory is [B, T, H, d]."""
    if layout == "bthd":
        b, h, t, d = shape
        return torch.randn((b, t, h, d), generator=g, device="cuda").to(dtype).transpose(1, 2)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _frequencies(rot):
    """Radians per position of each rotated pair, base 10000, float64."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    return 10000.0 ** (-2.0 * i / rot)


def _lengths(c):
    """Ragged batches fall from the whole length to about T / B, in even steps."""
    B, T = c["B"], c["T"]
    return [T - (T * b) // B for b in range(B)]


def _seen(c):
    """Decode: tokens already seen by each sequence.  A full batch has wrapped
    around its cache; a ragged one goes from an empty cache to a wrapped one."""
    B, full = c["B"], c["sinks"] + c["window"]
    if not c["ragged"]:
        return [full + full // 3 + b for b in range(B)]
    return [(2 * full * b) // B for b in range(B)]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _DT[c["dtype"]]
    s = dict(case=c)
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["op"] in ("rotary_fwd", "rotary_bwd"):
        T, lay = c["T"], c["layout"]
        s["q"], s["k"] = _randn(g, (B, H, T, d), dt, lay), _randn(g, (B, Hkv, T, d), dt, lay)
        s["freqs"] = _frequencies(c["rot"])
        s["positions"] = None
        if c["far"]:
            first = torch.randint(0, c["far"], (B, 1), generator=g, device="cuda")
            s["positions"] = (first + torch.arange(T, device="cuda")).to(torch.int32)
        s["affine"] = None
        if c["affine"]:
            s["affine"] = [1.0 + 0.1 * torch.randn((H, d), generator=g, device="cuda"),
                           0.1 * torch.randn((H, d), generator=g, device="cuda"),
                           1.0 + 0.1 * torch.randn((Hkv, d), generator=g, device="cuda"),
                           0.1 * torch.randn((Hkv, d), generator=g, device="cuda")]
        if c["op"] == "rotary_bwd":
            s["dq"], s["dk"] = _randn(g, (B, H, T, d), dt), _randn(g, (B, Hkv, T, d), dt)
        return s
    if c["op"] == "decode":
        C = c["sinks"] + c["window"]
        s["q"] = _randn(g, (B, H, 1, d), dt)
        s["k"], s["v"] = _randn(g, (B, Hkv, 1, d), dt), _randn(g, (B, Hkv, 1, d), dt)
        s["k_cache"], s["v_cache"] = _randn(g, (B, Hkv, C, d), dt), _randn(g, (B, Hkv, C, d), dt)
        s["seen"] = torch.tensor(_seen(c), dtype=torch.int32, device="cuda")
        return s
    T, Tq, lay = c["T"], c["Tq"], c["layout"]
    s["q"] = _randn(g, (B, H, Tq, d), dt, lay)
    s["k"], s["v"] = _randn(g, (B, Hkv, T, d), dt, lay), _randn(g, (B, Hkv, T, d), dt, lay)
    s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda") if c["ragged"] else None
    if c["op"] == "swa_bwd":
        out, lse = _plain_forward(s)
        s["out"], s["lse"] = out.to(dt), lse
        s["dout"] = _randn(g, (B, H, Tq, d), dt)
    return s


# --------------------------------------------------------------------------- plain forms
def _angles(s):
    """cos and sin [B or 1, 1, T, rot / 2], the angles in 64 bits."""
    T = s["q"].shape[2]
    pos = s["positions"]
    pos = torch.arange(T, device="cuda")[None] if pos is None else pos
    a = pos.double()[..., None] * s["freqs"]
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(x, cos, sin, rot, interleaved):
    """The rotated pairs are (2i, 2i + 1), or (i, i + rot / 2) in the half layout."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _plain_rotary_fwd(s):
    c = s["case"]
    cos, sin = _angles(s)
    q, k = s["q"].float(), s["k"].float()
    if s["affine"] is not None:
        qs, qo, ks, ko = s["affine"]
        q = q * qs[:, None] + qo[:, None]
        k = k * ks[:, None] + ko[:, None]
    dt = s["q"].dtype
    return [_rotate(q, cos, sin, c["rot"], c["interleaved"]).to(dt),
            _rotate(k, cos, sin, c["rot"], c["interleaved"]).to(dt)]


def _plain_rotary_bwd(s):
    c = s["case"]
    cos, sin = _angles(s)
    dt = s["q"].dtype
    gq = _rotate(s["dq"].float(), cos, -sin, c["rot"], c["interleaved"])
    gk = _rotate(s["dk"].float(), cos, -sin, c["rot"], c["interleaved"])
    if s["affine"] is None:
        return {"dq": gq.to(dt), "dk": gk.to(dt)}
    qs, _, ks, _ = s["affine"]
    total = lambda x: x.sum(dim=(0, 2), dtype=torch.float64).float()  # noqa: E731
    return {"dq": (gq * qs[:, None]).to(dt), "dk": (gk * ks[:, None]).to(dt),
            "dq_scale": total(gq * s["q"].float()), "dq_offset": total(gq),
            "dk_scale": total(gk * s["k"].float()), "dk_offset": total(gk)}


class _Band:
    """The window's scores by blocks of C >= window positions: the queries of
    block n against the keys of blocks n - 1 and n, and every query against
    the first `sinks` keys."""

    def __init__(self, s):
        c = s["case"]
        self.B, self.H, self.Hkv, self.T, self.Tq, self.d = c["B"], c["H"], c["Hkv"], c["T"], c["Tq"], c["d"]
        self.G = self.H // self.Hkv
        self.W, self.S = min(c["window"], self.T), min(c["sinks"], self.T)
        self.C = max(self.W, min(self.T, 64))
        self.N = -(-self.T // self.C)
        self.pad = self.N * self.C - self.T
        dev = s["q"].device
        off = self.T - self.Tq
        length = s["lengths"]
        length = torch.full((self.B,), self.T, device=dev) if length is None else length.long()
        length = length[:, None, None, None]                                   # [B, 1, 1, 1]
        i = torch.arange(self.N * self.C, device=dev).view(self.N, self.C, 1)  # query positions
        j = (i[:, :1] - self.C) + torch.arange(2 * self.C, device=dev)         # [N, 1, 2C] key positions
        seen = (i >= off) & (i < self.T) & (j >= 0) & (j <= i) & (j > i - self.W)
        self.mask = (seen & (i < length) & (j < length))[:, None, None]        # [B, 1, 1, N, C, 2C]
        i1 = torch.arange(self.T, device=dev)[:, None]
        js = torch.arange(self.S, device=dev)
        sink = (i1 >= off) & (js <= i1) & (js <= i1 - self.W)
        self.sink_mask = (sink & (i1 < length[:, 0]) & (js < length[:, 0]))[:, None, None]  # [B, 1, 1, T, S]
        self.scale = 1.0 / math.sqrt(self.d)

    def queries(self, x):
        """[B, H, Tq, d] -> [B, Hkv, G, T, d] in 32 bits, zeros before the first query."""
        x = x.float().reshape(self.B, self.Hkv, self.G, self.Tq, -1)
        return torch.nn.functional.pad(x, (0, 0, self.T - self.Tq, 0))

    def blocks(self, x):
        """[..., T, d] -> [..., N, C, d]"""
        x = torch.nn.functional.pad(x, (0, 0, 0, self.pad))
        return x.unflatten(-2, (self.N, self.C))

    def pairs(self, x):
        """[B, Hkv, T, d] -> [B, Hkv, 1, N, 2C, d]: each block's keys behind those of the block before."""
        x = self.blocks(x)
        before = torch.nn.functional.pad(x, (0, 0, 0, 0, 1, 0))[..., :-1, :, :]
        return torch.cat((before, x), dim=-2)[:, :, None]

    def unpair(self, y):
        """The sum of [B, Hkv, N, 2C, d] over the two blocks that hold each key: [B, Hkv, T, d]"""
        own_, before = y[..., self.C:, :], y[..., :self.C, :]
        before = torch.nn.functional.pad(before, (0, 0, 0, 0, 0, 1))[..., 1:, :, :]
        return (own_ + before).flatten(-3, -2)[..., :self.T, :]

    def unblock(self, x):
        """[B, Hkv, G, N, C, d] -> [B, H, Tq, d]"""
        x = x.flatten(-3, -2)[..., self.T - self.Tq:self.T, :]
        return x.reshape(self.B, self.H, self.Tq, -1)

    def scores(self, q, k):
        """Masked scores [B, Hkv, G, N, C, 2C] and [B, Hkv, G, T, S]; q [B, Hkv, G, T, d], k [B, Hkv, T, d]."""
        band = (self.blocks(q) @ self.pairs(k).transpose(-1, -2)).mul_(self.scale)
        sink = (q @ k[:, :, None, :self.S].transpose(-1, -2)).mul_(self.scale)
        return band.masked_fill_(~self.mask, -math.inf), sink.masked_fill_(~self.sink_mask, -math.inf)


def _plain_forward(s):
    b = _Band(s)
    q, k, v = b.queries(s["q"]), s["k"].float(), s["v"].float()
    band, sink = b.scores(q, k)
    top = band.amax(-1, keepdim=True)                                  # [B, Hkv, G, N, C, 1]
    sink = b.blocks(torch.nn.functional.pad(sink, (0, 1), value=-math.inf))
    if b.pad:
        sink[..., -1, b.C - b.pad:, :] = -math.inf
    top = torch.maximum(top, sink.amax(-1, keepdim=True))
    safe = top.masked_fill(top == -math.inf, 0.0)
    band, sink = band.sub_(safe).exp_(), sink.sub_(safe).exp_()
    total = band.sum(-1, keepdim=True) + sink.sum(-1, keepdim=True)
    out = band @ b.pairs(v) + sink[..., :-1] @ v[:, :, None, None, :b.S]
    out = out / total.clamp_min(1e-38)
    lse = top + total.log()
    return b.unblock(out), b.unblock(lse)[..., 0].contiguous()


def _plain_backward(s):
    b = _Band(s)
    q, k, v = b.queries(s["q"]), s["k"].float(), s["v"].float()
    do = b.queries(s["dout"])
    lse = b.queries(s["lse"][..., None])
    lse = lse.masked_fill(lse == -math.inf, 0.0)
    delta = (do * b.queries(s["out"])).sum(-1, keepdim=True)
    band, sink = b.scores(q, k)
    band, sink = band.sub_(b.blocks(lse)).exp_(), sink.sub_(lse).exp_()   # the probabilities
    dob = b.blocks(do)
    dv = b.unpair((band.transpose(-1, -2) @ dob).sum(2))
    dv[:, :, :b.S] += (sink.transpose(-1, -2) @ do).sum(2)
    band = (dob @ b.pairs(v).transpose(-1, -2)).sub_(b.blocks(delta)).mul_(band).mul_(b.scale)
    sink = (do @ v[:, :, None, :b.S].transpose(-1, -2)).sub_(delta).mul_(sink).mul_(b.scale)
    dk = b.unpair((band.transpose(-1, -2) @ b.blocks(q)).sum(2))
    dk[:, :, :b.S] += (sink.transpose(-1, -2) @ q).sum(2)
    dq = band @ b.pairs(k)
    dq = dq.flatten(-3, -2)[..., :b.T, :] + sink @ k[:, :, None, :b.S]
    dq = dq[..., b.T - b.Tq:, :].reshape(b.B, b.H, b.Tq, b.d)
    dt = s["q"].dtype
    return {"dq": dq.to(dt), "dk": dk.to(dt), "dv": dv.to(dt)}


def _plain_decode(s):
    c = s["case"]
    S, W = c["sinks"], c["window"]
    kc, vc, pos = s["k_cache"], s["v_cache"], s["seen"].long()
    slot = torch.where(pos < S, pos, S + (pos - S) % W)
    row = torch.arange(c["B"], device=pos.device)
    kc[row, :, slot] = s["k"][:, :, 0]
    vc[row, :, slot] = s["v"][:, :, 0]
    at = torch.arange(S + W, device=pos.device)
    held = at <= pos[:, None]                                             # [B, S + W]
    q = s["q"].float().view(c["B"], c["Hkv"], -1, c["d"])
    x = (q @ kc.float().transpose(-1, -2)) / math.sqrt(c["d"])
    x = x.masked_fill(~held[:, None, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp()
    out = (x @ vc.float()) / x.sum(-1, keepdim=True)
    return {"out": out.view(c["B"], c["H"], 1, c["d"]).to(kc.dtype), "k_cache": kc, "v_cache": vc}


# --------------------------------------------------------------------------- the framework's calls
def _own_run(s):
    import chunk_test_b200 as ct
    c = s["case"]
    op = c["op"]
    if op in ("rotary_fwd", "rotary_bwd"):
        kw = dict(positions=s["positions"], interleaved=c["interleaved"])
        if s["affine"] is not None:
            kw.update(zip(("q_scale", "q_offset", "k_scale", "k_offset"), s["affine"]))
        if op == "rotary_fwd":
            return list(ct.rotary_fwd(s["q"], s["k"], s["freqs"], **kw))
        g = ct.rotary_bwd(s["dq"], s["dk"], s["freqs"], q=s["q"], k=s["k"], **kw)
        return {n: x for n, x in g.items() if x is not None}
    if op == "swa_fwd":
        return list(ct.swa_sink_fwd(s["q"], s["k"], s["v"], c["window"], c["sinks"], lengths=s["lengths"]))
    if op == "swa_bwd":
        return ct.swa_sink_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], c["window"], c["sinks"],
                               lengths=s["lengths"])
    out = ct.swa_sink_decode(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["seen"], c["window"], c["sinks"])
    return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "rotary_fwd":
        return _plain_rotary_fwd(state)
    if op == "rotary_bwd":
        return _plain_rotary_bwd(state)
    if op == "swa_fwd":
        out, lse = _plain_forward(state)
        return [out.to(state["q"].dtype), lse]
    if op == "swa_bwd":
        return _plain_backward(state)
    return _plain_decode(state)


# --------------------------------------------------------------------------- work
def _pairs(c):
    """Visible (query, key) pairs of one head, over the batch."""
    def upto(n, lo):          # sum over positions lo <= i < n of the keys that i sees
        total = 0
        W, S = c["window"], c["sinks"]

        def cum(m):           # positions 0 .. m - 1
            full = W + S      # from position W + S - 1 on each sees all of both
            a = min(m, full)
            return a * (a + 1) // 2 + (m - a) * full
        total = cum(n) - cum(min(lo, n))
        return total
    lens = _lengths(c) if c["ragged"] else [c["T"]] * c["B"]
    return sum(upto(n, c["T"] - c["Tq"]) for n in lens)


def work(case):
    c = case
    size = 2 if c["dtype"] == BF16 else 4
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    if c["op"] in ("rotary_fwd", "rotary_bwd"):
        n = B * (H + Hkv) * c["T"] * d
        params = 2 * (H + Hkv) * d * 4 if c["affine"] else 0
        # forward: x in, y out; backward: dy in, dx out, and x and the parameters' gradients where there are any
        moved = 2 * n * size + params
        if c["op"] == "rotary_bwd" and c["affine"]:
            moved += n * size + params // 2
        return {"bytes": moved, "flops": 3 * B * (H + Hkv) * c["T"] * c["rot"]}
    if c["op"] == "decode":
        held = sum(min(p + 1, c["sinks"] + c["window"]) for p in _seen(c))
        # the held keys and values, the new token in and into the cache, q and out
        moved = 2 * Hkv * d * size * (held + 2 * B) + 2 * B * H * d * size
        return {"bytes": moved, "flops": 4 * H * d * held}
    T, Tq, pairs = c["T"], c["Tq"], _pairs(c) * H
    qn, kn = B * H * Tq * d * size, B * Hkv * T * d * size
    if c["op"] == "swa_fwd":
        return {"bytes": 2 * qn + 2 * kn + 4 * B * H * Tq, "flops": 4 * d * pairs}
    return {"bytes": 4 * qn + 4 * kn + 4 * B * H * Tq, "flops": 10 * d * pairs}


# --------------------------------------------------------------------------- 64 bits
def _exact_attention(s, with_grad):
    c = s["case"]
    B, H, Hkv, T, Tq, d, W, S = (c[n] for n in ("B", "H", "Hkv", "T", "Tq", "d", "window", "sinks"))
    G, off = H // Hkv, T - Tq
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    out, lse = torch.zeros_like(q), torch.full((B, H, Tq), -math.inf, dtype=torch.float64, device=q.device)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    lens = _lengths(c) if c["ragged"] else [T] * B
    step = max(64, min(1024, W))
    for b in range(B):
        for lo in range(off, lens[b], step):
            hi = min(lo + step, lens[b])
            first = max(0, lo - W + 1)
            js = torch.cat((torch.arange(min(S, first)), torch.arange(first, hi))).to(q.device)
            i = torch.arange(lo, hi, device=q.device)[:, None]
            ok = (js <= i) & ((js > i - W) | (js < S))
            for h in range(H):
                qh, kh, vh = q[b, h, lo - off:hi - off], k[b, h // G, js], v[b, h // G, js]
                x = (qh @ kh.T / math.sqrt(d)).masked_fill(~ok, -math.inf)
                z = torch.logsumexp(x, dim=1)
                p = torch.exp(x - z[:, None])
                o = p @ vh
                out[b, h, lo - off:hi - off], lse[b, h, lo - off:hi - off] = o, z
                if with_grad:
                    g = s["dout"][b, h, lo - off:hi - off].double()
                    ds = p * (g @ vh.T - (g * o).sum(1, keepdim=True)) / math.sqrt(d)
                    dq[b, h, lo - off:hi - off] = ds @ kh
                    dk[b, h // G].index_add_(0, js, ds.T @ qh)
                    dv[b, h // G].index_add_(0, js, p.T @ g)
    return {"dq": dq, "dk": dk, "dv": dv} if with_grad else [out, lse]


def _exact_rotary(s, backward):
    """Pairs as complex numbers: the forward turns them by the angle, the backward by its negative."""
    c = s["case"]
    rot, T = c["rot"], c["T"]
    pos = torch.arange(T, device="cuda")[None] if s["positions"] is None else s["positions"]
    angle = pos.double()[:, None, :, None] * s["freqs"]
    turn = torch.polar(torch.ones_like(angle), -angle if backward else angle)

    def turned(x):
        y = x.clone()
        if c["interleaved"]:
            z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * turn
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    a = [x.double()[:, None] for x in s["affine"]] if s["affine"] is not None else [1.0, 0.0, 1.0, 0.0]
    q, k = s["q"].double(), s["k"].double()
    if not backward:
        return [turned(q * a[0] + a[1]), turned(k * a[2] + a[3])]
    gq, gk = turned(s["dq"].double()), turned(s["dk"].double())
    if s["affine"] is None:
        return {"dq": gq, "dk": gk}
    return {"dq": gq * a[0], "dk": gk * a[2], "dq_scale": (gq * q).sum((0, 2)), "dq_offset": gq.sum((0, 2)),
            "dk_scale": (gk * k).sum((0, 2)), "dk_offset": gk.sum((0, 2))}


def _exact_decode(s):
    c = s["case"]
    S, W, G = c["sinks"], c["window"], c["H"] // c["Hkv"]
    kc, vc, out = s["k_cache"].double(), s["v_cache"].double(), torch.zeros_like(s["q"], dtype=torch.float64)
    for b, pos in enumerate(_seen(c)):
        slot = pos if pos < S else S + (pos - S) % W
        kc[b, :, slot], vc[b, :, slot] = s["k"][b, :, 0].double(), s["v"][b, :, 0].double()
        n = min(pos + 1, S + W)      # slots are filled in order, then overwritten
        for h in range(c["H"]):
            p = torch.softmax(kc[b, h // G, :n] @ s["q"][b, h, 0].double() / math.sqrt(c["d"]), dim=0)
            out[b, h, 0] = p @ vc[b, h // G, :n]
    return {"out": out, "k_cache": kc, "v_cache": vc}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rotary"):
        return _exact_rotary(s, case["op"] == "rotary_bwd")
    if case["op"] == "decode":
        return _exact_decode(s)
    return _exact_attention(s, case["op"] == "swa_bwd")
