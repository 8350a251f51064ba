"""The operators around RoLA in a video diffusion transformer's block, through the C ABI.

``qk_norm_rope`` (RMS norm and three-axis rotary positions of q and k), ``gated_norm`` (gated
residual with the modulated norm that follows) and ``cross_attend`` (dense attention to an
encoder's states), each with its backward.  ``include/rola.h`` states what they compute; this
module checks shapes, types and devices, allocates results and workspaces with torch (on the
current stream, so calls may be captured into a CUDA graph) and marshals the rest.  A call that
breaks a rule raises ``RolaError`` before anything is launched.

Activations are fp32 or bf16, gains, modulations and their gradients fp32.  ``stream`` is the
stream to run on (default: the current one): results and workspaces are allocated on it, and
what the inputs wait for, and how long they live, is the caller's to see to, as with torch's own
operators under ``torch.cuda.stream``.  Nothing is recorded for autograd: a training step calls
the backwards itself.
"""
from __future__ import annotations

import ctypes
import functools
import numbers

import torch

from . import DTYPES, RolaError, _check, load

_I64, _I32 = ctypes.c_int64, ctypes.c_int
_INVALID, _UNSUPPORTED = 1, 2
_TYPES = {torch.float32: DTYPES["f32"], torch.bfloat16: DTYPES["bf16"]}
NORMS = {"none": 0, "token": 1, "head": 2}
KINDS = {"layer": 0, "rms": 1}
POS_NONE, POS_GRID, POS_GIVEN = 0, 1, 2


class RolaNormRopeParams(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("B", "N", "H", "d", "dtype", "grad_dtype", "norm")] + [("eps", ctypes.c_float)]
                + [(n, _I32) for n in ("pos", "grid_t", "grid_h", "grid_w", "start_t", "start_h", "start_w",
                                       "positions_batched", "rope_pairs_t", "rope_pairs_h", "rope_pairs_w")]
                + [("rope_base", ctypes.c_double)]
                + [(n, _I64 * 3) for n in ("q", "k", "dq_out", "dk_out")])


class RolaGatedNormParams(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("B", "N", "C", "T", "x_dtype", "y_dtype", "norm")] + [("eps", ctypes.c_float)]
                + [(n, _I64) for n in ("gate_b", "gate_t", "scale_b", "scale_t", "shift_b", "shift_t")])


class RolaCrossParams(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("B", "Nq", "Nk", "H", "d", "dtype")] + [("softmax_scale", ctypes.c_float)]
                + [(n, _I64 * 3) for n in ("q", "k", "v", "dout")])


# ---------------------------------------------------------------------------- checks
# Everything that shapes, strides, types and devices decide is checked once per combination and
# kept with the parameter struct that it gives; what a call passes on is only its addresses.


def _need(ok, where, what, code=_INVALID):
    if not ok:
        raise RolaError(code, f"{where}: {what}")


class _Meta:
    """What a call's checks see of a tensor."""
    __slots__ = ("shape", "strides", "dtype", "device")

    def __init__(self, m):
        self.shape, self.strides, self.dtype, self.device = tuple(m[0]), m[1], m[2], m[3]
        if max(self.shape, default=0) >= 2 ** 31:
            raise RolaError(_UNSUPPORTED, f"a tensor of shape {list(self.shape)} has an axis past 31 bits")

    @property
    def contiguous(self):
        want = 1
        for n, s in zip(reversed(self.shape), reversed(self.strides)):
            if n != 1 and s != want:
                return False
            want *= n
        return True


def _ints(where, name, values, n):
    """`values` as n ints of 32 bits."""
    values = tuple(values)
    _need(len(values) == n and all(isinstance(x, int) and -2 ** 31 <= x < 2 ** 31 for x in values), where,
          f"{name} is not {n} 32-bit integers")
    return values


def _m(t):
    if t is None:
        return None
    try:
        return (t.shape, t.stride(), t.dtype, t.get_device())
    except (AttributeError, TypeError, RuntimeError):
        raise RolaError(_INVALID, f"a {type(t).__name__} in the place of a strided tensor") from None


def _number(where, name, x):
    # a tensor is none: checks are kept by their arguments, which must not change behind them
    _need(isinstance(x, numbers.Real), where, f"{name} is not a number")
    try:
        return float(x)
    except OverflowError:
        raise RolaError(_INVALID, f"{where}: {name} is not a number of a double's range") from None


def _results(where, out, n):
    """`out` as n tensors (or None)."""
    _need(isinstance(out, (tuple, list)) and len(out) == n
          and all(t is None or isinstance(t, torch.Tensor) for t in out), where, f"out is not {n} tensors")
    return out


def _metas(*ms):
    return [None if m is None else _Meta(m) for m in ms]


def _type(m, where, name):
    code = _TYPES.get(m.dtype)
    _need(code is not None, where, f"{name} is {m.dtype}, not fp32 or bf16", _UNSUPPORTED)
    return code


def _one_device(where, *metas):
    devices = {m.device for m in metas if m is not None}
    _need(-1 not in devices, where, "tensors are not on a CUDA device")
    _need(len(devices) == 1, where, "tensors are on different devices")


def _param(where, name, m, shape):
    _need(m is None or (m.dtype == torch.float32 and m.shape == shape and m.contiguous), where,
          f"{name} is not a contiguous fp32 {list(shape)}")


def _on_device(call):
    """Runs `call` with its first tensor's device, and the stream that it was given, as the
    current ones: memory that torch hands out in between belongs to that stream's order."""
    @functools.wraps(call)
    def run(*args, **kw):
        first = args[0] if args else next((t for t in kw.values() if isinstance(t, torch.Tensor)), None)
        device = first.get_device() if isinstance(first, torch.Tensor) else -1
        stream = kw.pop("stream", None)
        if stream is not None and device >= 0:
            _need(isinstance(stream, torch.cuda.Stream) and stream.device_index == device, "rola_" + call.__name__,
                  "the stream is another device's, or no stream")
            with torch.cuda.stream(stream):
                return call(*args, **kw)
        if device >= 0 and device != torch.cuda.current_device():
            with torch.cuda.device(device):
                return call(*args, **kw)
        return call(*args, **kw)
    return run


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    return torch._C._cuda_getCurrentRawStream(device)


def _new(t, dtype=None):
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _sized(fn, p):
    n = ctypes.c_size_t()
    _check(fn(ctypes.byref(p), ctypes.byref(n)), fn.__name__)
    return n.value


# ---------------------------------------------------------------------------- qk_norm_rope


@functools.lru_cache(maxsize=512)
def _rope(where, q, k, wq, wk, positions, dq_out, dk_out, norm, eps, grid, start, pairs, rope_base, rope):
    """(params, workspace bytes) of a call; q is None for a backward without a norm."""
    q, k, wq, wk, positions, dq_out, dk_out = _metas(q, k, wq, wk, positions, dq_out, dk_out)
    first = dq_out if q is None else q
    _need(first is not None and len(first.shape) == 4, where, "q is not [B, N, H, d]")
    B, N, H, d = first.shape
    dtype = _type(first, where, "q")
    _need(norm in NORMS, where, f"norm {norm!r} is not one of {sorted(NORMS)}")
    for name, t in (("q", q), ("k", k), ("dq_out", dq_out), ("dk_out", dk_out)):
        if t is not None:
            like = dq_out if name.startswith("d") else q
            _need(t.shape == first.shape and t.dtype == like.dtype and (t.strides[3] == 1 or d == 1), where,
                  f"{name} differs from q in shape or type, or its channels are not contiguous")
    n = {"none": 0, "token": H * d, "head": d}[norm]
    _need(norm != "none" or (wq is None and wk is None), where, "gains come with a norm")
    _param(where, "wq", wq, (n,))
    _param(where, "wk", wk, (n,))
    p = RolaNormRopeParams()
    p.B, p.N, p.H, p.d = B, N, H, d
    p.dtype = dtype
    p.grad_dtype = dtype if dq_out is None else _type(dq_out, where, "dq_out")
    p.norm, p.eps, p.rope_base = NORMS[norm], _number(where, "eps", eps), _number(where, "rope_base", rope_base)
    p.pos = POS_GRID if rope else POS_NONE
    p.grid_t, p.grid_h, p.grid_w = (1, 1, N) if grid is None else _ints(where, "grid", grid, 3)
    p.start_t, p.start_h, p.start_w = _ints(where, "start", start, 3)
    p.rope_pairs_t, p.rope_pairs_h, p.rope_pairs_w = _ints(where, "pairs", pairs, 3)
    if positions is not None:
        _need(rope and grid is None, where, "positions come without a grid, and not with rope=False")
        _need(positions.dtype == torch.int32 and positions.contiguous
              and positions.shape in ((N, 3), (B, N, 3)), where,
              "positions are not a contiguous int32 [N, 3] or [B, N, 3]")
        p.pos, p.positions_batched = POS_GIVEN, len(positions.shape) - 2
    _one_device(where, q, k, wq, wk, positions, dq_out, dk_out)
    for name, t in (("q", q), ("k", k), ("dq_out", dq_out), ("dk_out", dk_out)):
        if t is not None:
            setattr(p, name, (_I64 * 3)(*t.strides[:3]))
    return ctypes.byref(p), _sized(load().rola_qk_norm_rope_workspace_size, p), p


@_on_device
def qk_norm_rope(q, k=None, wq=None, wk=None, *, norm="token", eps=1e-6, grid=None, start=(0, 0, 0), positions=None,
                 pairs=(0, 0, 0), rope_base=10000.0, rope=True, out=None, stream=None):
    """RMS norm and rotary positions of q and k [B, N, H, d] (token, head and batch strides of whole
    16 bytes, d at least).

    norm: "token" (over H*d channels, gains wq, wk [H*d]), "head" (over d, gains [d]) or "none".
    Positions: ``grid`` (t, h, w) for tokens in that order, moved by ``start`` (tokens past the
    grid are not turned; default a 1D grid), or ``positions`` int32 [N, 3] or [B, N, 3]; with
    ``rope=False`` the norm alone.  ``out``: the two results' tensors, contiguous, or q and k
    themselves.  Returns (q_out, k_out), or q_out alone without k.  Nothing is recorded for
    autograd: ``qk_norm_rope_backward`` gives the gradients."""
    where = "rola_qk_norm_rope"
    mq = _m(q)
    p = _rope(where, mq, _m(k), _m(wq), _m(wk), _m(positions), None, None, norm, eps,
              None if grid is None else tuple(grid), tuple(start), tuple(pairs), rope_base, bool(rope))
    if out is None:
        qo, ko = _new(q), None if k is None else _new(k)
    else:
        qo, ko = (out, None) if isinstance(out, torch.Tensor) else _results(where, out, 2)
        for t, src in ((qo, q), (ko, k)):
            _need((t is None) == (src is None) and (t is None or (
                t.shape == q.shape and t.dtype == q.dtype and t.device == q.device
                and (t.stride() == src.stride() if t.data_ptr() == src.data_ptr() else t.is_contiguous()))), where,
                "out is neither contiguous like q nor the input itself")
    _check(load().rola_qk_norm_rope(p[0], q.data_ptr(), _ptr(k), _ptr(wq), _ptr(wk), _ptr(positions), qo.data_ptr(),
                                    _ptr(ko), _stream(mq[3])), where)
    return qo if k is None else (qo, ko)


@_on_device
def qk_norm_rope_backward(dq_out, dk_out=None, q=None, k=None, wq=None, wk=None, *, norm="token", eps=1e-6, grid=None,
                          start=(0, 0, 0), positions=None, pairs=(0, 0, 0), rope_base=10000.0, rope=True,
                          stream=None):
    """Gradients of ``qk_norm_rope`` (same options) from those of its results, which are of q's
    type or fp32 (as ``Plan.backward`` returns them).  Returns a dict: dq, dk of q's type, dwq,
    dwk fp32; entries that do not apply are None.  For norm="none" q and k count by their type
    alone, and one of them or both may be left out (then the results have dq_out's)."""
    where = "rola_qk_norm_rope_backward"
    if norm != "none":
        _need(q is not None and wq is not None and (dk_out is None) == (k is None) == (wk is None), where,
              "q, k and their gains come with a norm")
    elif q is None:
        q = k
    mu, mq = _m(dq_out), _m(q)
    _need(mu is not None, where, "there is no dq_out")
    dtype = mu[2] if q is None else mq[2]
    p = _rope(where, mq, _m(k), _m(wq), _m(wk), _m(positions), mu, _m(dk_out), norm, eps,
              None if grid is None else tuple(grid), tuple(start), tuple(pairs), rope_base, bool(rope))
    if norm == "none":                        # only their type counts
        q = k = None
    dq, dk = _new(dq_out, dtype), None if dk_out is None else _new(dk_out, dtype)
    dwq, dwk = None if wq is None else _new(wq), None if wk is None else _new(wk)
    need = p[1]
    ws = _workspace(need, dq_out.device)
    _check(load().rola_qk_norm_rope_backward(
        p[0], dq_out.data_ptr(), _ptr(dk_out), _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(positions), dq.data_ptr(),
        _ptr(dk), _ptr(dwq), _ptr(dwk), _ptr(ws), need, _stream(mu[3])), where)
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# ---------------------------------------------------------------------------- gated_norm


@functools.lru_cache(maxsize=512)
def _gated(where, x, y_dtype, like_x, like_y, gate, scale, shift, weight, bias, norm, eps):
    """(params, workspace bytes); like_x, like_y: tensors of x's shape in x's type, in y_dtype."""
    x, gate, scale, shift, weight, bias = _metas(x, gate, scale, shift, weight, bias)
    like_x, like_y = _metas(*like_x), _metas(*like_y)
    _need(len(x.shape) == 3, where, "x is not [B, N, C]")
    _need(norm in KINDS, where, f"norm {norm!r} is not one of {sorted(KINDS)}")
    B, N, C = x.shape
    p = RolaGatedNormParams()
    p.B, p.N, p.C = x.shape
    p.x_dtype = _type(x, where, "x")
    _need(y_dtype in _TYPES, where, f"y is {y_dtype}, not fp32 or bf16", _UNSUPPORTED)
    p.y_dtype, p.norm, p.eps = _TYPES[y_dtype], KINDS[norm], _number(where, "eps", eps)
    for t, dt in [(x, x.dtype)] + [(t, x.dtype) for t in like_x] + [(t, y_dtype) for t in like_y]:
        _need(t is None or (t.shape == x.shape and t.dtype == dt and t.contiguous), where,
              f"a tensor beside x is not a contiguous {dt} {[B, N, C]}")
    T = 0
    for name, m in (("gate", gate), ("scale", scale), ("shift", shift)):
        if m is None:
            continue
        _need(m.dtype == torch.float32 and len(m.shape) in (2, 3) and m.strides[-1] == 1, where,
              f"{name} is not an fp32 [B, C] or [B, T, C] with contiguous channels")
        t = 1 if len(m.shape) == 2 else m.shape[1]
        _need(m.shape[0] == B and m.shape[-1] == C and T in (0, t), where,
              f"{name} is not [B, T, C] with one T for all modulations")
        T = t
        setattr(p, name + "_b", m.strides[0])
        setattr(p, name + "_t", m.strides[1] if len(m.shape) == 3 else 0)
    p.T = T or 1
    _param(where, "weight", weight, (C,))
    _param(where, "bias", bias, (C,))
    _one_device(where, x, *like_x, *like_y, gate, scale, shift, weight, bias)
    return ctypes.byref(p), _sized(load().rola_gated_norm_workspace_size, p), p


@_on_device
def gated_norm(x, branch=None, gate=None, scale=None, shift=None, weight=None, bias=None, *, norm="layer", eps=1e-6,
               y_dtype=None, out=None, stream=None):
    """r = x + gate * branch and y = norm(r) * (1 + scale) + shift, or norm(r) * weight + bias.

    x [B, N, C]; branch and y in ``y_dtype`` (default: branch's type, else x's; bf16 beside an
    fp32 x is fine).  gate, scale, shift: fp32 [B, C] or [B, T, C] (views of one modulation
    tensor will do), token n taking row n // (N / T).  norm: "layer" or "rms".  ``out``: the
    tensors (r, y); r may be x.  Returns (r, y); without a branch r is x itself.  Nothing is
    recorded for autograd: ``gated_norm_backward`` gives the gradients."""
    where = "rola_gated_norm"
    mx, mb = _m(x), _m(branch)
    _need(mx is not None, where, "there is no x")
    if y_dtype is None:
        y_dtype = (mx if mb is None else mb)[2]
    p = _gated(where, mx, y_dtype, (), (mb,), _m(gate), _m(scale), _m(shift), _m(weight), _m(bias), norm, eps)
    if out is None:
        r, y = None if branch is None else _new(x), _new(x, y_dtype)
    else:
        r, y = _results(where, out, 2)
        r = None if branch is None else r
        for t, dt, unused in ((r, x.dtype, branch is None), (y, y_dtype, False)):
            _need(unused
                  or (t is not None and t.shape == x.shape and t.dtype == dt and t.is_contiguous()
                      and t.device == x.device), where, "out is not a pair of contiguous tensors like x and y")
    _check(load().rola_gated_norm(p[0], x.data_ptr(), _ptr(branch), _ptr(gate), _ptr(scale), _ptr(shift),
                                  _ptr(weight), _ptr(bias), _ptr(r), y.data_ptr(), _stream(mx[3])), where)
    return (x if r is None else r), y


@_on_device
def gated_norm_backward(dy, r, dr=None, branch=None, gate=None, scale=None, weight=None, *, norm="layer", eps=1e-6,
                        stream=None):
    """Gradients of ``gated_norm`` at the r that it returned, from those of y and of r (``dr``
    None: zero).  branch, gate, scale, weight as they were given to the forward.  Returns a
    dict: dx, dbranch, dgate, dscale, dshift (in the modulations' shape), dweight, dbias;
    entries that do not apply are None."""
    where = "rola_gated_norm_backward"
    mr, md = _m(r), _m(dy)
    _need(mr is not None and md is not None, where, "there is no r or no dy")
    p = _gated(where, mr, md[2], (_m(dr),), (md, _m(branch)), _m(gate), _m(scale), None, _m(weight), None, norm,
               eps)
    res = {"dx": _new(r), "dbranch": None if branch is None else _new(branch)}
    for name, t in (("dgate", gate), ("dscale", scale), ("dshift", scale), ("dweight", weight), ("dbias", weight)):
        res[name] = None if t is None else _new(t)
    need = p[1]
    ws = _workspace(need, r.device)
    _check(load().rola_gated_norm_backward(
        p[0], dy.data_ptr(), _ptr(dr), r.data_ptr(), _ptr(branch), _ptr(gate), _ptr(scale), _ptr(weight),
        *[_ptr(t) for t in res.values()], _ptr(ws), need, _stream(mr[3])), where)
    return res


# ---------------------------------------------------------------------------- cross_attend


@functools.lru_cache(maxsize=512)
def _cross(where, q, k, v, kv_len, key_mask, dout, out, lse, softmax_scale):
    """(params, workspace bytes of the forward, of the backward)."""
    q, k, v, kv_len, key_mask, dout, out, lse = _metas(q, k, v, kv_len, key_mask, dout, out, lse)
    _need(not any(t is None for t in (q, k, v)), where, "q, k or v is missing")
    _need(len(q.shape) == 4 and len(k.shape) == 4, where, "q is not [B, Nq, H, d], or k not [B, Nk, H, d]")
    B, Nq, H, d = q.shape
    Nk = k.shape[1]
    p = RolaCrossParams()
    p.B, p.Nq, p.Nk, p.H, p.d = B, Nq, Nk, H, d
    p.dtype, p.softmax_scale = _type(q, where, "q"), _number(where, "softmax_scale", softmax_scale)
    for name, t, n in (("q", q, Nq), ("k", k, Nk), ("v", v, Nk), ("dout", dout, Nq)):
        if t is not None:
            _need(t.shape == (B, n, H, d) and t.dtype == q.dtype and (t.strides[3] == 1 or d == 1), where,
                  f"{name} is not a {q.dtype} {[B, n, H, d]} with contiguous channels")
            setattr(p, name, (_I64 * 3)(*t.strides[:3]))
    _need(kv_len is None or (kv_len.dtype == torch.int32 and kv_len.shape == (B,) and kv_len.contiguous), where,
          "kv_len is not a contiguous int32 [B]")
    _need(key_mask is None or (key_mask.dtype in (torch.bool, torch.uint8) and key_mask.shape == (B, Nk)
                               and key_mask.contiguous), where, "key_mask is not a contiguous bool or uint8 [B, Nk]")
    _need(out is None or (out.shape == q.shape and out.dtype == q.dtype and out.contiguous), where,
          "out is not contiguous like q")
    _need(lse is None or (lse.shape == (B, H, Nq) and lse.dtype == torch.float32 and lse.contiguous), where,
          "lse is not the forward's")
    _one_device(where, q, k, v, kv_len, key_mask, dout, out, lse)
    lib = load()
    return ctypes.byref(p), _sized(lib.rola_cross_workspace_size, p), _sized(lib.rola_cross_backward_workspace_size, p), p


@_on_device
def cross_attend(q, k, v, *, kv_len=None, key_mask=None, softmax_scale=0.0, return_lse=False, out=None, stream=None):
    """Dense softmax attention of q [B, Nq, H, d] to k, v [B, Nk, H, d] (token, head and batch
    strides of whole 16 bytes, d at least).  Key m counts when m < kv_len[b] (int32 [B]) and key_mask[b, m] (bool or
    uint8 [B, Nk]); a sample without keys gives zeros.  softmax_scale 0: 1/sqrt(d).  Returns
    out [B, Nq, H, d], with ``return_lse`` also the log sum of exponentials fp32 [B, H, Nq].
    In bf16 the probabilities are rounded to bf16 before their product with v (sums are fp32).
    Nothing is recorded for autograd: ``cross_attend_backward`` gives the gradients."""
    where = "rola_cross_attend"
    mq = _m(q)
    p = _cross(where, mq, _m(k), _m(v), _m(kv_len), _m(key_mask), None, _m(out), None, softmax_scale)
    if out is None:
        out = _new(q)
    B, Nq, H, _ = mq[0]
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if return_lse else None
    need = p[1]
    ws = _workspace(need, q.device)
    _check(load().rola_cross_attend(p[0], q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(kv_len), _ptr(key_mask),
                                    out.data_ptr(), _ptr(lse), _ptr(ws), need, _stream(mq[3])), where)
    return (out, lse) if return_lse else out


@_on_device
def cross_attend_backward(dout, q, k, v, out, lse, *, kv_len=None, key_mask=None, softmax_scale=0.0, stream=None):
    """Gradients of ``cross_attend`` from dout, with the forward's inputs, out and lse.  Returns
    a dict: dq, dk, dv, contiguous and of q's type.  In bf16 the probabilities and their gradients
    are rounded to bf16 before their products (sums are fp32)."""
    where = "rola_cross_attend_backward"
    mq = _m(q)
    p = _cross(where, mq, _m(k), _m(v), _m(kv_len), _m(key_mask), _m(dout), _m(out), _m(lse), softmax_scale)
    _need(dout is not None and out is not None and lse is not None, where, "dout, out or lse is missing")
    dq, dk, dv = _new(q), _new(k), _new(v)
    need = p[2]
    ws = _workspace(need, q.device)
    _check(load().rola_cross_attend_backward(
        p[0], dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), _ptr(kv_len),
        _ptr(key_mask), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(ws), need, _stream(mq[3])), where)
    return {"dq": dq, "dk": dk, "dv": dv}


def block_poll_status(stream=None) -> int:
    """Synchronises the stream; returns the status code of the calls of this module on the
    current device since the last poll (0 = ok), clearing it."""
    return load().rola_block_poll_status((torch.cuda.current_stream() if stream is None else stream).cuda_stream)
