"""The operators around RoLA in a video diffusion transformer's block, through the C ABI.

``qk_norm_rope`` (RMS norm and three-axis rotary positions of q and k), ``gated_norm`` (gated
residual with the modulated norm that follows) and ``cross_attend`` (dense attention to an
encoder's states), each with its backward.  ``include/rola.h`` states what they compute; this
module checks shapes, types and devices, allocates results and workspaces with torch (on the
current stream, so calls may be captured into a CUDA graph) and marshals the rest.  A call that
breaks a rule raises ``RolaError`` before anything is launched.

Activations are fp32 or bf16, gains, modulations and their gradients fp32.  ``stream`` is the
stream to launch on (default: the current one); memory is then the caller's to keep alive.
"""
from __future__ import annotations

import ctypes
import functools

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


def _need(ok, where, what, code=_INVALID):
    if not ok:
        raise RolaError(code, f"{where}: {what}")


def _dtype(t, where, name):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise RolaError(_UNSUPPORTED, f"{where}: {name} is {t.dtype}, not fp32 or bf16")
    return code


def _same_device(where, first, *tensors):
    _need(first.is_cuda, where, "tensors are not on a CUDA device")
    for t in tensors:
        _need(t is None or t.device == first.device, where, "tensors are on different devices")


def _param(where, name, t, shape):
    _need(t.dtype == torch.float32 and t.shape == shape and t.is_contiguous(), where,
          f"{name} is not a contiguous fp32 {list(shape)}")


def _on_device(call):
    """Runs `call` with the first tensor's device as the current one."""
    @functools.wraps(call)
    def run(*args, **kw):
        first = args[0] if args else next((t for t in kw.values() if isinstance(t, torch.Tensor)), None)
        if isinstance(first, torch.Tensor) and first.is_cuda and first.get_device() != torch.cuda.current_device():
            with torch.cuda.device(first.device):
                return call(*args, **kw)
        return call(*args, **kw)
    return run


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _sized(fn, p):
    n = ctypes.c_size_t()
    _check(fn(ctypes.byref(p), ctypes.byref(n)), fn.__name__)
    return n.value


# ---------------------------------------------------------------------------- qk_norm_rope


@functools.lru_cache(maxsize=256)
def _rope_params(shape, strides, dtype, grad_dtype, norm, eps, pos, grid, start, batched, pairs, base):
    p = RolaNormRopeParams()
    p.B, p.N, p.H, p.d = shape
    p.dtype, p.grad_dtype, p.norm, p.eps, p.pos = dtype, grad_dtype, norm, eps, pos
    p.grid_t, p.grid_h, p.grid_w = grid
    p.start_t, p.start_h, p.start_w = start
    p.positions_batched = batched
    p.rope_pairs_t, p.rope_pairs_h, p.rope_pairs_w = pairs
    p.rope_base = base
    for name, s in zip(("q", "k", "dq_out", "dk_out"), strides):
        setattr(p, name, (_I64 * 3)(*s[:3]))
    return p, _sized(load().rola_qk_norm_rope_workspace_size, p)


def _rope_setup(where, q, k, wq, wk, up, norm, eps, grid, start, positions, pairs, rope_base, rope):
    first = up[0] if q is None else q
    _need(first.dim() == 4, where, "q is not [B, N, H, d]")
    shape = tuple(first.shape)
    dtype = _dtype(first, where, "q")
    _need(norm in NORMS, where, f"norm {norm!r} is not one of {sorted(NORMS)}")
    n = {"none": 0, "token": shape[2] * shape[3], "head": shape[3]}[norm]
    for name, t in (("q", q), ("k", k)):
        if t is not None:
            _need(t.shape == shape and t.dtype == first.dtype and t.stride(3) == 1, where,
                  f"{name} differs from q in shape or type, or its channels are not contiguous")
    for name, t in (("dq_out", up[0]), ("dk_out", up[1])):
        if t is not None:
            _need(t.shape == shape and t.dtype == up[0].dtype and t.stride(3) == 1, where,
                  f"{name} differs from q in shape, or its channels are not contiguous")
    for name, t in (("wq", wq), ("wk", wk)):
        if t is not None:
            _param(where, name, t, (n,))
    pos, batched, grid_given = POS_NONE, 0, grid
    grid, start = (1, 1, shape[1]) if grid is None else tuple(grid), tuple(start)
    if positions is not None:
        _need(rope and grid_given is None, where, "positions come without a grid, and not with rope=False")
        batched = int(positions.dim() == 3)
        _need(positions.dtype == torch.int32 and positions.is_contiguous()
              and tuple(positions.shape) in ((shape[1], 3), (shape[0], shape[1], 3)), where,
              "positions are not a contiguous int32 [N, 3] or [B, N, 3]")
        pos, grid, start = POS_GIVEN, (1, 1, 1), (0, 0, 0)
    elif rope:
        pos = POS_GRID
    _same_device(where, first, q, k, wq, wk, positions, *up)
    strides = tuple(t.stride() if t is not None else (0, 0, 0) for t in (q, k, *up))
    grad_dtype = dtype if up[0] is None else _dtype(up[0], where, "dq_out")
    return _rope_params(shape, strides, dtype, grad_dtype, NORMS[norm], eps, pos, grid, start, batched, tuple(pairs),
                        float(rope_base))


@_on_device
def qk_norm_rope(q, k=None, wq=None, wk=None, *, norm="token", eps=1e-6, grid=None, start=(0, 0, 0), positions=None,
                 pairs=(0, 0, 0), rope_base=10000.0, rope=True, out=None, stream=None):
    """RMS norm and rotary positions of q and k [B, N, H, d] (any token, head and batch strides).

    norm: "token" (over H*d channels, gains wq, wk [H*d]), "head" (over d, gains [d]) or "none".
    Positions: ``grid`` (t, h, w) for tokens in that order, moved by ``start`` (tokens past the
    grid are not turned; default a 1D grid), or ``positions`` int32 [N, 3] or [B, N, 3]; with
    ``rope=False`` the norm alone.  ``out``: the two results' tensors, contiguous, or q and k
    themselves.  Returns (q_out, k_out), or q_out alone without k."""
    where = "rola_qk_norm_rope"
    p, _ = _rope_setup(where, q, k, wq, wk, (None, None), norm, eps, grid, start, positions, pairs, rope_base, rope)
    if out is None:
        qo = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        ko = None if k is None else torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        qo, ko = (out, None) if isinstance(out, torch.Tensor) else out
        for t, src in ((qo, q), (ko, k)):
            if t is None and src is None:
                continue
            _need(t is not None and src is not None and t.shape == q.shape and t.dtype == q.dtype
                  and t.device == q.device and (t.is_contiguous() or (t.data_ptr() == src.data_ptr()
                                                                      and t.stride() == src.stride())), where,
                  "out is neither contiguous like q nor the input itself")
            _need(t.data_ptr() != src.data_ptr() or t.stride() == src.stride() or t.is_contiguous() == src.is_contiguous(),
                  where, "out starts where the input does but has other strides")
    _check(load().rola_qk_norm_rope(ctypes.byref(p), q.data_ptr(), _ptr(k), _ptr(wq), _ptr(wk), _ptr(positions),
                                    qo.data_ptr(), _ptr(ko), _stream(stream)), where)
    return qo if k is None else (qo, ko)


@_on_device
def qk_norm_rope_backward(dq_out, dk_out=None, q=None, k=None, wq=None, wk=None, *, norm="token", eps=1e-6, grid=None,
                          start=(0, 0, 0), positions=None, pairs=(0, 0, 0), rope_base=10000.0, rope=True,
                          stream=None):
    """Gradients of ``qk_norm_rope`` (same options) from those of its results, which are of q's
    type or fp32 (as ``Plan.backward`` returns them).  Returns a dict: dq, dk of q's type, dwq,
    dwk fp32; entries that do not apply are None.  q and k may be left out for norm="none"."""
    where = "rola_qk_norm_rope_backward"
    if norm == "none":
        dtype = dq_out.dtype if q is None else q.dtype
        wq = wk = None
    else:
        _need(q is not None and wq is not None and (dk_out is None) == (k is None), where,
              "q, k and their gains are needed with a norm")
        dtype = q.dtype
    if norm == "none" and q is not None:      # only its type counts
        p, need = _rope_setup(where, q, k, None, None, (dq_out, dk_out), norm, eps, grid, start, positions, pairs,
                              rope_base, rope)
        q = k = None
    else:
        p, need = _rope_setup(where, q, k, wq, wk, (dq_out, dk_out), norm, eps, grid, start, positions, pairs,
                              rope_base, rope)
    dev = dq_out.device
    dq = torch.empty(dq_out.shape, dtype=dtype, device=dev)
    dk = None if dk_out is None else torch.empty(dq_out.shape, dtype=dtype, device=dev)
    dwq = None if wq is None else torch.empty_like(wq)
    dwk = None if wk is None else torch.empty_like(wk)
    ws = _workspace(need, dev)
    _check(load().rola_qk_norm_rope_backward(
        ctypes.byref(p), dq_out.data_ptr(), _ptr(dk_out), _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(positions),
        dq.data_ptr(), _ptr(dk), _ptr(dwq), _ptr(dwk), _ptr(ws), need, _stream(stream)), where)
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


# ---------------------------------------------------------------------------- gated_norm


@functools.lru_cache(maxsize=256)
def _gated_params(shape, T, x_dtype, y_dtype, norm, eps, strides):
    p = RolaGatedNormParams()
    p.B, p.N, p.C = shape
    p.T, p.x_dtype, p.y_dtype, p.norm, p.eps = T, x_dtype, y_dtype, norm, eps
    p.gate_b, p.gate_t, p.scale_b, p.scale_t, p.shift_b, p.shift_t = strides
    return p, _sized(load().rola_gated_norm_workspace_size, p)


def _gated_setup(where, x, y_dtype, mods, norm, eps, like_x, like_y, params):
    _need(x.dim() == 3, where, "x is not [B, N, C]")
    _need(norm in KINDS, where, f"norm {norm!r} is not one of {sorted(KINDS)}")
    B, N, C = x.shape
    y_code = _TYPES.get(y_dtype)
    _need(y_code is not None, where, f"y is {y_dtype}, not fp32 or bf16", _UNSUPPORTED)
    for name, t, dt in [(n, t, x.dtype) for n, t in like_x] + [(n, t, y_dtype) for n, t in like_y]:
        if t is not None:
            _need(t.shape == x.shape and t.dtype == dt and t.is_contiguous(), where,
                  f"{name} is not a contiguous {dt} {list(x.shape)}")
    T, strides = None, []
    for name, m in mods:
        if m is None:
            strides += [0, 0]
            continue
        _need(m.dtype == torch.float32 and m.stride(-1) == 1 and m.dim() in (2, 3), where,
              f"{name} is not an fp32 [B, C] or [B, T, C] with contiguous channels")
        t = 1 if m.dim() == 2 else m.shape[1]
        _need(m.shape[0] == B and m.shape[-1] == C and T in (None, t), where,
              f"{name} is not [B, T, C] with one T for all modulations")
        T = t
        strides += [m.stride(0), m.stride(1) if m.dim() == 3 else 0]
    for name, w in params:
        if w is not None:
            _param(where, name, w, (C,))
    T = T or 1
    _same_device(where, x, *(t for _, t in (*mods, *like_x, *like_y, *params)))
    return _gated_params((B, N, C), T, _dtype(x, where, "x"), y_code, KINDS[norm], eps, tuple(strides))


@_on_device
def gated_norm(x, branch=None, gate=None, scale=None, shift=None, weight=None, bias=None, *, norm="layer", eps=1e-6,
               y_dtype=None, out=None, stream=None):
    """r = x + gate * branch and y = norm(r) * (1 + scale) + shift, or norm(r) * weight + bias.

    x [B, N, C]; branch and y in ``y_dtype`` (default: branch's type, else x's; bf16 beside an
    fp32 x is fine).  gate, scale, shift: fp32 [B, C] or [B, T, C] (views of one modulation
    tensor will do), token n taking row n // (N / T).  norm: "layer" or "rms".  ``out``: the
    tensors (r, y); r may be x.  Returns (r, y); without a branch r is x itself."""
    where = "rola_gated_norm"
    if y_dtype is None:
        y_dtype = x.dtype if branch is None else branch.dtype
    p, _ = _gated_setup(where, x, y_dtype, (("gate", gate), ("scale", scale), ("shift", shift)), norm, eps,
                        (("x", x),), (("branch", branch),), (("weight", weight), ("bias", bias)))
    if out is None:
        r = None if branch is None else torch.empty_like(x)
        y = torch.empty(x.shape, dtype=y_dtype, device=x.device)
    else:
        r, y = out
        r = None if branch is None else r
        for t, dt in ((r, x.dtype), (y, y_dtype)):
            _need((t is None and t is r and branch is None)
                  or (t is not None and t.shape == x.shape and t.dtype == dt and t.is_contiguous()
                      and t.device == x.device), where, "out is not a pair of contiguous tensors like x and y")
    _check(load().rola_gated_norm(ctypes.byref(p), x.data_ptr(), _ptr(branch), _ptr(gate), _ptr(scale), _ptr(shift),
                                  _ptr(weight), _ptr(bias), _ptr(r), y.data_ptr(), _stream(stream)), where)
    return (x if r is None else r), y


@_on_device
def gated_norm_backward(dy, r, dr=None, branch=None, gate=None, scale=None, weight=None, *, norm="layer", eps=1e-6,
                        stream=None):
    """Gradients of ``gated_norm`` at the r that it returned, from those of y and of r (``dr``
    None: zero).  branch, gate, scale, weight as they were given to the forward.  Returns a
    dict: dx, dbranch, dgate, dscale, dshift (in the modulations' shape), dweight, dbias;
    entries that do not apply are None."""
    where = "rola_gated_norm_backward"
    p, need = _gated_setup(where, r, dy.dtype, (("gate", gate), ("scale", scale), ("shift", None)), norm, eps,
                           (("r", r), ("dr", dr)), (("dy", dy), ("branch", branch)), (("weight", weight),))
    dev = r.device

    def like(t, dtype=None):
        return None if t is None else torch.empty(t.shape, dtype=dtype or t.dtype, device=dev)

    res = {"dx": like(r), "dbranch": like(branch), "dgate": like(gate), "dscale": like(scale), "dshift": like(scale),
           "dweight": like(weight), "dbias": like(weight)}
    ws = _workspace(need, dev)
    _check(load().rola_gated_norm_backward(
        ctypes.byref(p), dy.data_ptr(), _ptr(dr), r.data_ptr(), _ptr(branch), _ptr(gate), _ptr(scale), _ptr(weight),
        *[_ptr(t) for t in res.values()], _ptr(ws), need, _stream(stream)), where)
    return res


# ---------------------------------------------------------------------------- cross_attend


@functools.lru_cache(maxsize=256)
def _cross_params(q_shape, Nk, dtype, scale, strides):
    p = RolaCrossParams()
    p.B, p.Nq, p.H, p.d = q_shape
    p.Nk, p.dtype, p.softmax_scale = Nk, dtype, scale
    for name, s in zip(("q", "k", "v", "dout"), strides):
        setattr(p, name, (_I64 * 3)(*s[:3]))
    lib = load()
    return p, _sized(lib.rola_cross_workspace_size, p), _sized(lib.rola_cross_backward_workspace_size, p)


def _cross_setup(where, q, k, v, kv_len, key_mask, softmax_scale, dout=None):
    _need(q.dim() == 4 and k.dim() == 4, where, "q is not [B, Nq, H, d], or k not [B, Nk, H, d]")
    B, _, H, d = q.shape
    Nk = k.shape[1]
    for name, t, shape in (("q", q, q.shape), ("k", k, (B, Nk, H, d)), ("v", v, (B, Nk, H, d)),
                           ("dout", dout, q.shape)):
        if t is not None:
            _need(t.shape == shape and t.dtype == q.dtype and t.stride(3) == 1, where,
                  f"{name} is not a {q.dtype} {list(shape)} with contiguous channels")
    if kv_len is not None:
        _need(kv_len.dtype == torch.int32 and kv_len.shape == (B,) and kv_len.is_contiguous(), where,
              "kv_len is not a contiguous int32 [B]")
    if key_mask is not None:
        _need(key_mask.dtype in (torch.bool, torch.uint8) and key_mask.shape == (B, Nk) and key_mask.is_contiguous(),
              where, "key_mask is not a contiguous bool or uint8 [B, Nk]")
    _same_device(where, q, k, v, kv_len, key_mask, dout)
    strides = (q.stride(), k.stride(), v.stride(), (0, 0, 0) if dout is None else dout.stride())
    return _cross_params(tuple(q.shape), Nk, _dtype(q, where, "q"), float(softmax_scale), strides)


@_on_device
def cross_attend(q, k, v, *, kv_len=None, key_mask=None, softmax_scale=0.0, return_lse=False, out=None, stream=None):
    """Dense softmax attention of q [B, Nq, H, d] to k, v [B, Nk, H, d] (any token, head and
    batch strides).  Key m counts when m < kv_len[b] (int32 [B]) and key_mask[b, m] (bool or
    uint8 [B, Nk]); a sample without keys gives zeros.  softmax_scale 0: 1/sqrt(d).  Returns
    out [B, Nq, H, d], with ``return_lse`` also the log sum of exponentials fp32 [B, H, Nq]."""
    where = "rola_cross_attend"
    p, need, _ = _cross_setup(where, q, k, v, kv_len, key_mask, softmax_scale)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _need(out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous() and out.device == q.device, where,
              "out is not contiguous like q")
    lse = torch.empty((p.B, p.H, p.Nq), dtype=torch.float32, device=q.device) if return_lse else None
    ws = _workspace(need, q.device)
    _check(load().rola_cross_attend(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(kv_len),
                                    _ptr(key_mask), out.data_ptr(), _ptr(lse), _ptr(ws), need, _stream(stream)), where)
    return (out, lse) if return_lse else out


@_on_device
def cross_attend_backward(dout, q, k, v, out, lse, *, kv_len=None, key_mask=None, softmax_scale=0.0, stream=None):
    """Gradients of ``cross_attend`` from dout, with the forward's inputs, out and lse.  Returns
    a dict: dq, dk, dv, contiguous and of q's type."""
    where = "rola_cross_attend_backward"
    p, _, need = _cross_setup(where, q, k, v, kv_len, key_mask, softmax_scale, dout)
    _need(out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous() and lse.dtype == torch.float32
          and tuple(lse.shape) == (p.B, p.H, p.Nq) and lse.is_contiguous(), where,
          "out and lse are not the forward's results")
    _same_device(where, q, out, lse)
    res = {n: torch.empty(t.shape, dtype=q.dtype, device=q.device) for n, t in (("dq", q), ("dk", k), ("dv", v))}
    ws = _workspace(need, q.device)
    _check(load().rola_cross_attend_backward(
        ctypes.byref(p), dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
        _ptr(kv_len), _ptr(key_mask), *[t.data_ptr() for t in res.values()], _ptr(ws), need, _stream(stream)), where)
    return res


def block_poll_status(stream=None) -> int:
    """Synchronises the stream; returns the status code of the calls of this module on the
    current device since the last poll (0 = ok), clearing it."""
    return load().rola_block_poll_status(_stream(stream))
