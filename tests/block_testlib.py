"""Plain 64-bit forms of the operators around RoLA, with bounds on what 32-bit kernels may be off.

Every bound is arithmetic, per element: u = 2^-24 is the fp32 rounding, half(t) the half step of
the result's type (bf16 2^-8, fp32 2^-24, relative).  A sum of n terms in fp32 is off by at most
about depth * u times the sum of the terms' magnitudes, depth <= n + a few for any order.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24


def half(t):
    return torch.finfo(t).eps / 2


def assert_within(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, f"{what}: shape {tuple(got.shape)}, not {tuple(want.shape)}"
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)) and torch.equal(got[~fine], want[~fine]), f"{what}: non-finite"
    over = (got - want).abs()[fine] - tol.expand_as(want)[fine]
    if over.numel():
        assert float(over.max()) <= 0, f"{what}: exceeds its bound by {float(over.max()):.3e}"


def rand(gen, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    x = torch.randn(*shape, generator=gen, device=gen.device, dtype=torch.float32)
    return (x * scale + shift).to(dtype)


# ---------------------------------------------------------------------------- qk_norm_rope


def pair_split(d, one_axis, pairs=(0, 0, 0)):
    if sum(pairs):
        return pairs
    P = d // 2
    return (0, 0, P) if one_axis else (P - 2 * (P // 3), P // 3, P // 3)


def angles(N, d, grid=None, start=(0, 0, 0), positions=None, pairs=(0, 0, 0), base=10000.0, device="cuda"):
    """[N or B, N, 1, d/2] angles in fp64."""
    if positions is not None:
        pos, split = positions.double(), pair_split(d, False, pairs)
    else:
        gt, gh, gw = grid or (1, 1, N)
        rows = []
        for n in range(N):
            at = (n // (gh * gw), n // gw % gh, n % gw)
            rows.append([a + s for a, s in zip(at, start)] if n < gt * gh * gw else [0, 0, 0])
        pos = torch.tensor(rows, dtype=torch.float64, device=device)
        split = pair_split(d, gt == 1 and gh == 1, pairs)
    cols = [pos[..., i] * base ** (-j / p) for i, p in enumerate(split) for j in range(p)]
    return torch.stack(cols, -1)[..., None, :]


def rotate(x, a):
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack((x0 * a.cos() - x1 * a.sin(), x0 * a.sin() + x1 * a.cos()), -1).flatten(-2)


def pair_norm(x):
    """sqrt(a^2 + b^2) of each pair, at both of its places."""
    return x.unflatten(-1, (-1, 2)).norm(dim=-1, keepdim=True).expand(*x.shape[:-1], x.shape[-1] // 2, 2).flatten(-2)


def _gain(w, norm, H, d):
    return w.double().view(H, d) if norm == "token" else w.double().view(1, d)


def norm_rope_ref(x, w, norm, a, eps=1e-6):
    """(y, bound): fp32 statistics (depth <= 24 sums of squares, all positive, halved by the
    square root), gains and the rotation by an angle good to 3u: within 32u of the pair's length."""
    v = x.double()
    if norm != "none":
        dims = (2, 3) if norm == "token" else (3,)
        v = v / (v.square().mean(dims, keepdim=True) + eps).sqrt() * _gain(w, norm, *x.shape[2:])
    y = v if a is None else rotate(v, a)
    return y, half(x.dtype) * y.abs() + 32 * U * pair_norm(v)


def norm_rope_backward_ref(dy, x, w, norm, a, eps=1e-6):
    """dx, dw and their bounds."""
    g = dy.double() if a is None else rotate(dy.double(), -a)
    ge = 8 * U * pair_norm(dy.double()) if a is not None else 0 * g
    if norm == "none":
        return g, half(x.dtype) * g.abs() + ge, None, None
    dims = (2, 3) if norm == "token" else (3,)
    v = x.double()
    r = (v.square().mean(dims, keepdim=True) + eps).rsqrt()
    xn, wn = v * r, _gain(w, norm, *x.shape[2:])
    over = (0, 1) if norm == "token" else (0, 1, 2)
    n = g.shape[0] * g.shape[1] * (1 if norm == "token" else g.shape[2])
    dw = (g * xn).sum(over).reshape(-1)
    dwe = ((n + 64) * U * (g * xn).abs() + ge * xn.abs()).sum(over).reshape(-1)
    h = g * wn
    inner = (h * xn).mean(dims, keepdim=True)
    dx = r * (h - xn * inner)
    he = ge * wn.abs() + 64 * U * h.abs()
    ie = (he * xn.abs() + 64 * U * (h * xn).abs()).mean(dims, keepdim=True)
    return dx, half(x.dtype) * dx.abs() + r * (he + xn.abs() * (ie + 64 * U * inner.abs())) + 64 * U * dx.abs(), dw, dwe


# ---------------------------------------------------------------------------- gated_norm


def spread(m, N):
    m = m.double()
    m = m[:, None] if m.dim() == 2 else m
    return m.repeat_interleave(N // m.shape[1], 1)


def gated_norm_ref(x, branch, gate, scale, shift, weight, bias, kind, y_dtype, eps=1e-6):
    N = x.shape[1]
    r = x.double()
    re = 0 * r
    if branch is not None:
        g = spread(gate, N) if gate is not None else torch.ones_like(r)
        r = r + g * branch.double()
        re = 2 * U * (r.abs() + (g * branch.double()).abs())
    mean = r.mean(-1, keepdim=True) if kind == "layer" else 0 * r[..., :1]
    rstd = ((r - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    xh = (r - mean) * rstd
    A = 1 + spread(scale, N) if scale is not None else weight.double() if weight is not None else torch.ones_like(r)
    Bv = spread(shift, N) if shift is not None else bias.double() if bias is not None else torch.zeros_like(r)
    y = xh * A + Bv
    # the mean is off by depth <= 24 roundings of the mean magnitude; xhat by that and its own
    mag = r.abs().mean(-1, keepdim=True) if kind == "layer" else 0 * mean
    xe = rstd * (re + re.mean(-1, keepdim=True) + 24 * U * mag + U * r.abs()) \
        + xh.abs() * (24 * U + rstd * (24 * U * mag + re.mean(-1, keepdim=True)))
    return (r, half(x.dtype) * r.abs() + re), (y, half(y_dtype) * y.abs() + xe * A.abs() * (1 + 4 * U)
                                               + 4 * U * (y.abs() + (xh * A).abs() + Bv.abs()))


def gated_norm_backward_ref(dy, r, dr, branch, gate, scale, weight, kind, eps=1e-6):
    """{name: (gradient, bound)}."""
    B, N, C = r.shape
    v, d = r.double(), dy.double()
    mean = v.mean(-1, keepdim=True) if kind == "layer" else 0 * v[..., :1]
    rstd = ((v - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    xh = (v - mean) * rstd
    mag = v.abs().mean(-1, keepdim=True) if kind == "layer" else 0 * mean
    xe = rstd * (24 * U * mag + U * v.abs()) + xh.abs() * (24 * U + rstd * 24 * U * mag)
    A = 1 + spread(scale, N) if scale is not None else weight.double() if weight is not None else torch.ones_like(v)
    g = d * A
    ge = 3 * U * g.abs()
    gm = g.mean(-1, keepdim=True) if kind == "layer" else 0 * mean
    gme = (ge + 24 * U * g.abs()).mean(-1, keepdim=True) if kind == "layer" else 0 * mean
    pr = (g * xh).mean(-1, keepdim=True)
    pe = (ge * xh.abs() + g.abs() * xe + 32 * U * (g * xh).abs()).mean(-1, keepdim=True)
    inner = g - gm - xh * pr
    ie = ge + gme + xe * pr.abs() + xh.abs() * pe + 4 * U * (g.abs() + gm.abs() + (xh * pr).abs())
    up = dr.double() if dr is not None else torch.zeros_like(v)
    dx = up + rstd * inner
    # rstd itself: 24 roundings of its sum of squares and the mean's error in it
    dxe = rstd * (ie + inner.abs() * (32 * U + rstd * 24 * U * mag)) + 2 * U * (up.abs() + dx.abs())
    res = {"dx": (dx, half(r.dtype) * dx.abs() + dxe)}

    def sums(x, e, T):
        shape, n = (B, T, N // T, C), N // T
        return x.view(shape).sum(2), (e + (n + 64) * U * x.abs()).view(shape).sum(2)

    if branch is not None:
        a = branch.double()
        gt = spread(gate, N) if gate is not None else torch.ones_like(v)
        res["dbranch"] = dx * gt, half(dy.dtype) * (dx * gt).abs() + (dxe + 2 * U * dx.abs()) * gt.abs()
        if gate is not None:
            x, e = sums(dx * a, dxe * a.abs(), 1 if gate.dim() == 2 else gate.shape[1])
            res["dgate"] = x.view(gate.shape), e.view(gate.shape)
    if scale is not None:
        T = 1 if scale.dim() == 2 else scale.shape[1]
        for name, x, e in (("dscale", d * xh, d.abs() * xe), ("dshift", d, 0 * d)):
            s, se = sums(x, e, T)
            res[name] = s.view(scale.shape), se.view(scale.shape)
    if weight is not None:
        for name, x, e in (("dweight", d * xh, d.abs() * xe), ("dbias", d, 0 * d)):
            res[name] = x.sum((0, 1)), (e + (B * N + 64) * U * x.abs()).sum((0, 1))
    return res


# ---------------------------------------------------------------------------- cross_attend


def valid_keys(B, Nk, kv_len, key_mask, device):
    ok = torch.ones(B, Nk, dtype=torch.bool, device=device)
    if kv_len is not None:
        ok &= torch.arange(Nk, device=device) < kv_len[:, None]
    if key_mask is not None:
        ok &= key_mask.bool()
    return ok


def _heads(x):
    return x.double().transpose(1, 2)


def _scores(q, k, v, ok, scale):
    """S [B, H, Nq, Nk] (-inf at invalid keys), its bound, k and v with zeros there."""
    keep = ok[:, None, :, None]
    q, k, v = _heads(q), _heads(k).where(keep, 0.0), _heads(v).where(keep, 0.0)
    d = q.shape[-1]
    scale = scale or 1 / math.sqrt(d)
    s = (q @ k.transpose(-1, -2)) * scale
    se = (d + 8) * U * (q.abs() @ k.abs().transpose(-1, -2)) * scale + 8 * U
    return s.masked_fill(~ok[:, None, None, :], -math.inf), se, q, k, v, scale


def _soft(q, k, v, ok, scale):
    s, se, q, k, v, scale = _scores(q, k, v, ok, scale)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse.where(lse > -math.inf, 0.0)[..., None])
    # exponentials: the score's error, their own and the subtraction's rounding of s and lse
    top = s.where(ok[:, None, None, :], 0.0).abs().amax(-1, keepdim=True)
    return s, p, se + 8 * U * (1 + top), lse, q, k, v, scale


def cross_ref(q, k, v, kv_len=None, key_mask=None, scale=0.0):
    ok = valid_keys(q.shape[0], k.shape[1], kv_len, key_mask, q.device)
    s, p, pe, lse, qh, kh, vh, scale = _soft(q, k, v, ok, scale)
    Nk, t = k.shape[1], q.dtype
    row = (pe * p).sum(-1, keepdim=True) + (Nk + 16) * U       # relative error of the denominator
    round_p = half(t) if t != torch.float32 else 0.0             # P enters the second product in t
    out = p @ vh
    oe = (p * (pe + row + round_p + (Nk + 16) * U)) @ vh.abs()
    out, oe = out.transpose(1, 2), oe.transpose(1, 2)
    return (out, half(t) * out.abs() + oe), (lse, row[..., 0] + 4 * U * (1 + lse.where(lse > -math.inf, 0.0).abs()))


def cross_backward_ref(dout, q, k, v, out, lse, kv_len=None, key_mask=None, scale=0.0):
    """The gradients' formula at the out and lse that are given, with bounds."""
    ok = valid_keys(q.shape[0], k.shape[1], kv_len, key_mask, q.device)
    s, se, qh, kh, vh, scale = _scores(q, k, v, ok, scale)
    z = lse.double()
    p = torch.exp(s - z.where(z > -math.inf, 0.0)[..., None])
    pe = se + 8 * U * (1 + z.where(z > -math.inf, 0.0).abs()[..., None] + s.where(p > 0, 0.0).abs())
    do, t, d = _heads(dout), q.dtype, q.shape[-1]
    D = (do * _heads(out)).sum(-1, keepdim=True)
    De = (d + 4) * U * (do.abs() * _heads(out).abs()).sum(-1, keepdim=True)
    dp = do @ vh.transpose(-1, -2)
    dpe = (d + 8) * U * (do.abs() @ vh.abs().transpose(-1, -2))
    ds = p * (dp - D) * scale
    rt = half(t) if t != torch.float32 else 0.0                  # P and dS enter the products in t
    dse = ds.abs() * (pe + rt + 8 * U) + p * scale * (dpe + De + 4 * U * (dp.abs() + D.abs()))
    Nq, Nk = q.shape[1], k.shape[1]
    dq, dqe = ds @ kh, (dse + (Nk + 16) * U * ds.abs()) @ kh.abs()
    dst, dset, pt = ds.transpose(-1, -2), dse.transpose(-1, -2), p.transpose(-1, -2)
    dk, dke = dst @ qh, (dset + (Nq + 16) * U * dst.abs()) @ qh.abs()
    dv, dve = pt @ do, (pt * (pe.transpose(-1, -2) + rt + (Nq + 16) * U)) @ do.abs()
    return {n: (x.transpose(1, 2), (half(t) * x.abs() + e).transpose(1, 2))
            for n, x, e in (("dq", dq, dqe), ("dk", dk, dke), ("dv", dv, dve))}
