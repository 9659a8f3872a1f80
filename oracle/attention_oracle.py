"""fp64 oracle of the block's attention half -- TEST INFRASTRUCTURE.

Rotary positions with scales and offsets, sliding-window attention with sinks
(forward, backward, single-token form), straight from the definitions on dense
[T, T] masks in torch float64 (CPU or GPU).  Beside each result stand the sums
of absolute values that bound a rounded computation of it:

  one rounding of x to a type is off by at most u |x|, u = finfo.eps / 2;
  a sum of products whose factors are each rounded (relative error e) is off
  by at most e times the sum of the products' absolute values.
"""
from __future__ import annotations

import math

import torch


def rotate(x, angle, rot, interleaved):
    """x [..., T, d], angle [..., T, rot / 2] (float64)."""
    y = x.clone()
    c, s = angle.cos(), angle.sin()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        y[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
    return y


def rotary(x, freqs, positions, interleaved, amplitude=1.0, scale=None, offset=None):
    """x [B, H, T, d] -> y; positions [B, T]."""
    x = x.double()
    if scale is not None:
        x = x * scale.double()[:, None] + offset.double()[:, None]
    rot = 2 * freqs.numel()
    y = rotate(x, positions.double()[:, None, :, None] * freqs, rot, interleaved)
    y[..., :rot] *= amplitude
    return y


def rotary_vjp(dy, freqs, positions, interleaved, amplitude=1.0, x=None, scale=None):
    """(dx, dscale, doffset, sum |g x|, sum |g|); the last four None without scale."""
    rot = 2 * freqs.numel()
    g = rotate(dy.double(), -positions.double()[:, None, :, None] * freqs, rot, interleaved)
    g[..., :rot] *= amplitude
    if scale is None:
        return g, None, None, None, None
    gx = g * x.double()
    return g * scale.double()[:, None], gx.sum((0, 2)), g.sum((0, 2)), gx.abs().sum((0, 2)), g.abs().sum((0, 2))


def visible(T, Tq, window, sinks, length, device):
    """[Tq, T]: which keys each query sees."""
    i = torch.arange(T - Tq, T, device=device)[:, None]
    j = torch.arange(T, device=device)
    return (j <= i) & ((j > i - window) | (j < sinks)) & (i < length) & (j < length)


def attention(q, k, v, window, sinks=0, lengths=None, scale=None, dout=None):
    """A dict of out, lse and the bound's sums: pv = sum p |v|, qk = max sum scale |q| |k|;
    with dout also dq, dk, dv and the sums of the backward (see backward_bounds)."""
    q, k, v = q.double(), k.double(), v.double()
    B, H, Tq, d = q.shape
    Hkv, T = k.shape[1], k.shape[2]
    G = H // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    r = {n: torch.zeros_like(q) for n in ("out", "pv", "dq", "adq", "ddq")}
    r.update({n: torch.zeros_like(k) for n in ("dk", "dv", "adk", "ddk", "adv")})
    r["lse"] = torch.full((B, H, Tq), -math.inf, dtype=torch.float64, device=q.device)
    r["qk"] = 0.0
    for b in range(B):
        n = T if lengths is None else max(0, min(int(lengths[b]), T))
        see = visible(T, Tq, window, sinks, n, q.device)
        rows = see.any(1)
        if not bool(rows.any()):
            continue
        for h in range(H):
            # only the rows and keys below the length take part: what the others hold is never used
            qh, kh, vh = q[b, h][rows], k[b, h // G][:n], v[b, h // G][:n]
            s = (qh @ kh.T * scale).masked_fill(~see[rows][:, :n], -math.inf)
            z = torch.logsumexp(s, 1)
            p = torch.exp(s - z[:, None])
            o = p @ vh
            r["out"][b, h][rows], r["lse"][b, h][rows], r["pv"][b, h][rows] = o, z, p @ vh.abs()
            r["qk"] = max(r["qk"], float((qh.abs() @ kh.abs().T * abs(scale)).max()))
            if dout is None:
                continue
            g = dout[b, h].double()[rows]
            dp = g @ vh.T
            ds = p * (dp - (g * o).sum(1, keepdim=True)) * scale
            r["dq"][b, h][rows] = ds @ kh
            r["dk"][b, h // G][:n] += ds.T @ qh
            r["dv"][b, h // G][:n] += p.T @ g
            # |ds| and p scale sum |dout| (|out| + sum p |v|): what a rounding of ds, and of out, moves
            own = p * abs(scale) * (g.abs() * (o.abs() + p @ vh.abs())).sum(1, keepdim=True)
            # the size of dp's terms, for 32-bit sums
            raw = p * abs(scale) * (g.abs() @ vh.abs().T + (g.abs() * o.abs()).sum(1, keepdim=True))
            r["adq"][b, h][rows] = (ds.abs() + own) @ kh.abs()
            r["adk"][b, h // G][:n] += (ds.abs() + own).T @ qh.abs()
            r["ddq"][b, h][rows] = raw @ kh.abs()
            r["ddk"][b, h // G][:n] += raw.T @ qh.abs()
            r["adv"][b, h // G][:n] += p.T @ g.abs()
    return r


def decode(q, k_new, v_new, k_cache, v_cache, seen, window, sinks=0, scale=None):
    """(out, pv, k_cache, v_cache) of one token per sequence, the caches as new tensors."""
    B, H, _, d = q.shape
    Hkv = k_new.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    kc, vc = k_cache.clone(), v_cache.clone()
    out, pv = torch.zeros_like(q, dtype=torch.float64), torch.zeros_like(q, dtype=torch.float64)
    for b in range(B):
        pos = int(seen[b])
        if pos < 0:
            continue
        slot = pos if pos < sinks else sinks + (pos - sinks) % window
        kc[b, :, slot], vc[b, :, slot] = k_new[b, :, 0], v_new[b, :, 0]
        n = min(pos + 1, sinks + window)
        for h in range(H):
            hk = h // (H // Hkv)
            p = torch.softmax(kc[b, hk, :n].double() @ q[b, h, 0].double() * scale, 0)
            out[b, h, 0], pv[b, h, 0] = p @ vc[b, hk, :n].double(), p @ vc[b, hk, :n].double().abs()
    return out, pv, kc, vc
