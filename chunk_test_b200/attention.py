"""torch-facing wrappers of the block's attention half: rotary positions, the
sliding-window attention with sinks (forward, backward) and its single-token
form over a rolling cache (include/lact.h).

Tensors are [B, heads, T, d] CUDA tensors in bf16 or float32 whose channels
are contiguous; the other strides are free (multiples of 16 bytes), so a
projection's [B, T, heads, d] result is passed as its transpose, and outputs
given by the caller may have that layout too.  Calls run on the tensors'
device, on torch's current stream there (or `stream=`, from whose pool they
then make their results and workspaces).
"""
from __future__ import annotations

import functools
import math
import struct

import torch

from . import _abi
from ._abi import LactError
from .layer import _made, _result

_DT = {torch.float32: _abi.LACT_F32, torch.bfloat16: _abi.LACT_BF16}


# The C structs are packed into bytes, whose address ctypes passes: a quarter of
# the time of a ctypes.Structure, and these calls count microseconds.
_TENSOR = struct.Struct("=4q").pack          # lact_tensor4
_ROTARY = struct.Struct("=7qiifi").pack      # lact_rotary_problem
_SINK = struct.Struct("=8qfi").pack          # lact_swa_sink_problem


def _view(t):
    """The tensor as a lact_tensor4, or NULL."""
    if t is None:
        return None
    s = t.stride()
    return _TENSOR(t.data_ptr(), s[0], s[1], s[2])


def _new(t, stream):
    """A new contiguous result like `t`."""
    if stream is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return _result(stream, torch.empty_like, t, memory_format=torch.contiguous_format)


def _at(t):
    return None if t is None else t.data_ptr()


def _tensor(name, t, shape, like):
    """A [B, heads, T, d] tensor of `like`'s dtype and device, channels contiguous."""
    if t.dtype is not like.dtype or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be a {like.dtype} tensor on {like.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.stride()[3] != 1 and shape[3] > 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    return t


def _dense(name, t, shape, dtype, device):
    if t.dtype is not dtype or t.get_device() != device.index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on {device}")
    return t


def _query(q):
    if q.dim() != 4:
        raise ValueError("q must be a [B, H, T, d] tensor")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    if q.dtype not in _DT:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if q.stride(3) != 1 and q.shape[3] > 1:
        raise ValueError("q's channels must be contiguous")


def _call(name, device, stream, *args):
    """The library's `name` on `device` (made current where another one is) and
    its stream, torch's current one unless given."""
    fn = getattr(_abi.lib(), name)
    st = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    if device.index == torch._C._cuda_getDevice():
        rc = fn(*args, st)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, st)
    if rc != _abi.LACT_OK:
        raise LactError(rc, name)


# ---------------------------------------------------------------------- rotary
def rotary_frequencies(rot, base=10000.0, *, method="none", factor=1.0, context=None, low=1.0, high=32.0,
                       device="cuda"):
    """(freqs, amplitude) for rotary_fwd: `rot` / 2 angular frequencies in
    radians per position (float64), base^(-2i/rot), scaled for contexts
    `factor` times as long as the ones the model was trained on:
      "none"      as they are;
      "linear"    positions divided by factor;
      "base"      the base raised to base * factor^(rot / (rot - 2)), which divides
                  the lowest frequency by factor and leaves the highest;
      "by_parts"  pairs that turn less than `low` times over the trained
                  `context` are divided by factor, those that turn more than
                  `high` times are left, a linear ramp between; the amplitude
                  is 1 + 0.1 ln(factor)."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if factor < 1.0 or base <= 0.0:
        raise ValueError("factor must be at least 1 and base positive")
    i = torch.arange(rot // 2, dtype=torch.float64)
    amplitude = 1.0
    if method == "base":
        if rot == 2:
            raise ValueError('method "base" needs rot > 2')
        base = base * factor ** (rot / (rot - 2))
    f = float(base) ** (-2.0 * i / rot)
    if method == "linear":
        f = f / factor
    elif method == "by_parts":
        if not context or not high > low:
            raise ValueError('method "by_parts" needs the trained context and high > low')
        turns = f * (context / (2.0 * math.pi))
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        amplitude = 1.0 + 0.1 * math.log(factor)
    elif method not in ("none", "base"):
        raise ValueError(f"unknown method {method!r}")
    return f.to(device), amplitude


def _rotary_args(q, k, freqs, positions, start, interleaved, amplitude):
    B, H, T, d = q.shape
    if k is None:
        Hkv = 0
    else:
        if k.dim() != 4:
            raise ValueError("k must be a [B, Hkv, T, d] tensor")
        Hkv = k.shape[1]
        _tensor("k", k, (B, Hkv, T, d), q)
    if freqs.dim() != 1:
        raise ValueError("freqs must be one-dimensional")
    _dense("freqs", freqs, (freqs.shape[0],), torch.float64, q.device)
    if positions is not None:
        _dense("positions", positions, (B, T), torch.int32, q.device)
    return _ROTARY(B, H, Hkv, T, d, 2 * freqs.shape[0], int(start), int(bool(interleaved)), _DT[q.dtype],
                   float(amplitude), 0)


def _params(names, values, q, k):
    """Scales and offsets: all given ([H, d] and [Hkv, d] float32) or none."""
    d = q.shape[3]
    want = [(n, v, (x.shape[1], d)) for n, v, x in zip(names, values, [q] * (len(names) // 2) + [k] * (len(names) // 2))
            if x is not None]
    given = [v is not None for _, v, _ in want]
    if any(given) and not all(given):
        raise ValueError("give all of " + ", ".join(n for n, _, _ in want) + ", or none")
    for n, v, shape in want:
        if v is not None:
            _dense(n, v, shape, torch.float32, q.device)
    if k is None and any(v is not None for v in values[len(values) // 2:]):
        raise ValueError("k's scale and offset need k")
    return given[0]


def rotary_fwd(q, k, freqs, *, positions=None, start=0, interleaved=False, amplitude=1.0, q_scale=None,
               q_offset=None, k_scale=None, k_offset=None, out=None, stream=None):
    """Rotary positions of q [B, H, T, d] and k [B, Hkv, T, d] (or None), after
    x * scale + offset per head and channel where those are given
    (lact_rotary_fwd).  freqs: float64, one per rotated pair (see
    rotary_frequencies); channels from 2 * len(freqs) on are not rotated.
    positions: int32 [B, T], else start + t.  Returns (q_out, k_out), new
    contiguous tensors or the pair `out`, which may be (q, k) itself."""
    _query(q)
    p = _rotary_args(q, k, freqs, positions, start, interleaved, amplitude)
    _params(("q_scale", "q_offset", "k_scale", "k_offset"), (q_scale, q_offset, k_scale, k_offset), q, k)
    if out is None:
        out = (_new(q, stream), None if k is None else _new(k, stream))
    else:
        _tensor("out[0]", out[0], q.shape, q)
        if k is not None:
            _tensor("out[1]", out[1], k.shape, q)
    _call("lact_rotary_fwd", q.device, stream, p, _view(q), _view(k), _at(freqs), _at(positions), _at(q_scale),
          _at(q_offset), _at(k_scale), _at(k_offset), _view(out[0]), None if k is None else _view(out[1]))
    return out[0], (None if k is None else out[1])


def rotary_bwd(dq_out, dk_out, freqs, *, positions=None, start=0, interleaved=False, amplitude=1.0, q=None, k=None,
               q_scale=None, q_offset=None, k_scale=None, k_offset=None, out=None, workspace=None, stream=None):
    """The backward of rotary_fwd (lact_rotary_bwd): from the gradients of its
    results, a dict of dq, dk and, with scales, the float32 dq_scale,
    dq_offset, dk_scale, dk_offset (then q and k are the forward's inputs;
    the offsets' values are not used).  `out`: the pair (dq, dk), which may be
    (dq_out, dk_out) itself."""
    _query(dq_out)
    p = _rotary_args(dq_out, dk_out, freqs, positions, start, interleaved, amplitude)
    affine = _params(("q_scale", "k_scale"), (q_scale, k_scale), dq_out, dk_out)
    res = dict.fromkeys(("dq", "dk", "dq_scale", "dq_offset", "dk_scale", "dk_offset"))
    if out is None:
        res["dq"] = _new(dq_out, stream)
        if dk_out is not None:
            res["dk"] = _new(dk_out, stream)
    else:
        res["dq"] = _tensor("out[0]", out[0], dq_out.shape, dq_out)
        if dk_out is not None:
            res["dk"] = _tensor("out[1]", out[1], dk_out.shape, dq_out)
    need = 0
    if affine:
        if q is None or (dk_out is not None and k is None):
            raise ValueError("the scales' gradients need the forward's q and k")
        _tensor("q", q, dq_out.shape, dq_out)
        like = torch.empty_like if stream is None else functools.partial(_result, stream, torch.empty_like)
        res["dq_scale"], res["dq_offset"] = like(q_scale), like(q_scale)
        if dk_out is not None:
            _tensor("k", k, dk_out.shape, dq_out)
            res["dk_scale"], res["dk_offset"] = like(k_scale), like(k_scale)
        need = int(_abi.lib().lact_rotary_bwd_workspace_bytes(p))
        if need == 0:
            raise LactError(_abi.LACT_EINVAL, "lact_rotary_bwd_workspace_bytes")
        workspace = _workspace(workspace, need, dq_out.device, stream)
    _call("lact_rotary_bwd", dq_out.device, stream, p, _view(dq_out), _view(dk_out), _at(freqs), _at(positions),
          _view(q) if affine else None, _view(k) if affine and dk_out is not None else None, _at(q_scale),
          _at(k_scale), _view(res["dq"]), _view(res["dk"]), _at(res["dq_scale"]), _at(res["dq_offset"]),
          _at(res["dk_scale"]), _at(res["dk_offset"]), _at(workspace) if affine else None, need)
    return res


def _workspace(workspace, need, device, stream):
    if workspace is None:
        if stream is None:
            return torch.empty(need, dtype=torch.uint8, device=device)
        return _made(stream, torch.empty, need, dtype=torch.uint8, device=device)
    if workspace.device != device or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the device of the call")
    if workspace.numel() < need:
        raise ValueError(f"workspace holds {workspace.numel()} bytes; the call needs {need}")
    return workspace


# ---------------------------------------------------------------------- window attention with sinks
def _swa_sink_problem(q, k, window, sinks, scale, T, Tq):
    B, H, _, d = q.shape
    if k.dim() != 4:
        raise ValueError("k must be a [B, Hkv, T, d] tensor")
    return _SINK(B, H, k.shape[1], T, Tq, d, int(window), int(sinks),
                 1.0 / math.sqrt(d) if scale is None else float(scale), _DT[q.dtype])


def _keys(q, k, v, lengths):
    B, _, _, d = q.shape
    _tensor("k", k, (B, k.shape[1], k.shape[2], d), q)
    _tensor("v", v, k.shape, q)
    if lengths is not None:
        _dense("lengths", lengths, (B,), torch.int32, q.device)


def swa_sink_fwd(q, k, v, window, sinks=0, *, lengths=None, scale=None, out=None, lse=None, stream=None):
    """Sliding-window attention whose first `sinks` tokens stay visible
    (lact_swa_sink_fwd): q [B, H, Tq, d] (the last Tq positions), k, v
    [B, Hkv, T, d], H a multiple of Hkv; `lengths` int32 [B] for padded
    batches.  Returns (out [B, H, Tq, d], lse [B, H, Tq] float32)."""
    _query(q)
    p = _swa_sink_problem(q, k, window, sinks, scale, k.shape[2], q.shape[2])
    _keys(q, k, v, lengths)
    if out is None:
        out = _new(q, stream)
    else:
        _tensor("out", out, q.shape, q)
    if lse is None:
        lse = q.new_empty(q.shape[:3], dtype=torch.float32) if stream is None else _result(
            stream, torch.empty, q.shape[:3], dtype=torch.float32, device=q.device)
    else:
        _dense("lse", lse, q.shape[:3], torch.float32, q.device)
    _call("lact_swa_sink_fwd", q.device, stream, p, _view(q), _view(k), _view(v), _at(lengths), _view(out), _at(lse))
    return out, lse


def swa_sink_bwd_workspace_bytes(q, k, window, sinks=0) -> int:
    p = _swa_sink_problem(q, k, window, sinks, None, k.shape[2], q.shape[2])
    return int(_abi.lib().lact_swa_sink_bwd_workspace_bytes(p))


def swa_sink_bwd(q, k, v, out, lse, dout, window, sinks=0, *, lengths=None, scale=None, dq=None, dk=None, dv=None,
                 workspace=None, stream=None):
    """The backward of swa_sink_fwd (lact_swa_sink_bwd) from its inputs, its
    out and lse and the gradient dout of out.  Returns a dict of dq, dk, dv
    in the inputs' dtype (new contiguous tensors, or the ones given)."""
    _query(q)
    p = _swa_sink_problem(q, k, window, sinks, scale, k.shape[2], q.shape[2])
    _keys(q, k, v, lengths)
    _tensor("out", out, q.shape, q)
    _tensor("dout", dout, q.shape, q)
    _dense("lse", lse, q.shape[:3], torch.float32, q.device)
    dq = _new(q, stream) if dq is None else _tensor("dq", dq, q.shape, q)
    dk = _new(k, stream) if dk is None else _tensor("dk", dk, k.shape, q)
    dv = _new(k, stream) if dv is None else _tensor("dv", dv, k.shape, q)
    need = int(_abi.lib().lact_swa_sink_bwd_workspace_bytes(p))
    if need == 0:
        raise LactError(_abi.LACT_EINVAL, "lact_swa_sink_bwd_workspace_bytes")
    workspace = _workspace(workspace, need, q.device, stream)
    _call("lact_swa_sink_bwd", q.device, stream, p, _view(q), _view(k), _view(v), _view(out), _at(lse), _view(dout),
          _at(lengths), _view(dq), _view(dk), _view(dv), _at(workspace), workspace.numel())
    return {"dq": dq, "dk": dk, "dv": dv}


def _caches(q, k, k_cache, v_cache, window, sinks):
    B, Hkv, _, d = k.shape
    shape = (B, Hkv, int(sinks) + int(window), d)
    _dense("k_cache", k_cache, shape, q.dtype, q.device)
    _dense("v_cache", v_cache, shape, q.dtype, q.device)


def swa_sink_decode(q, k, v, k_cache, v_cache, seen, window, sinks=0, *, scale=None, out=None, stream=None):
    """swa_sink_fwd for one new token per sequence over a rolling cache
    (lact_swa_sink_decode): q [B, H, 1, d], the new k, v [B, Hkv, 1, d], caches
    [B, Hkv, sinks + window, d], which the call writes the new token into, and
    seen int32 [B], the tokens each sequence already has there (negative:
    inactive, out 0).  Returns out [B, H, 1, d].  `seen` is the caller's to
    advance (seen.add_(1) on the same stream)."""
    _query(q)
    B, H, n, d = q.shape
    if n != 1:
        raise ValueError("q must hold one token per sequence")
    p = _swa_sink_problem(q, k, window, sinks, scale, 1, 1)
    _tensor("k", k, (B, k.shape[1], 1, d), q)
    _tensor("v", v, k.shape, q)
    _caches(q, k, k_cache, v_cache, window, sinks)
    _dense("seen", seen, (B,), torch.int32, q.device)
    if out is None:
        out = _new(q, stream)
    else:
        _tensor("out", out, q.shape, q)
    _call("lact_swa_sink_decode", q.device, stream, p, _view(q), _view(k), _view(v), _at(k_cache), _at(v_cache),
          _at(seen), _view(out))
    return out


def swa_cache_fill(k, v, k_cache, v_cache, window, sinks=0, *, lengths=None, stream=None):
    """A prompt's k, v [B, Hkv, T, d] into the rolling caches of
    swa_sink_decode (lact_swa_cache_fill): the sinks and the last `window`
    other tokens of each sequence; `seen` is then the sequences' lengths.
    The tokens are those from position 0 on: a prompt in pieces is filled in
    after its last piece."""
    _query(k)
    B, Hkv, T, d = k.shape
    p = _swa_sink_problem(k, k, window, sinks, 1.0, T, 1)
    _keys(k, k, v, lengths)
    _caches(k, k, k_cache, v_cache, window, sinks)
    _call("lact_swa_cache_fill", k.device, stream, p, _view(k), _view(v), _at(lengths), _at(k_cache), _at(v_cache))
