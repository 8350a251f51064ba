"""Cases of the operators around RoLA in a video diffusion transformer's block, to be timed.

Three operators, each forward and backward:
  rope   qk_norm_rope   RMS norm of q and k, then rotary positions on three axes (t, h, w)
  norm   gated_norm     gated residual r = x + gate * branch, then the modulated norm of r
  cross  cross_attend   dense attention of video tokens to an encoder's states of another length

With ``own`` false, ``run`` computes them in elementary torch operations (32 bits; angles in 64),
rounded once at the end; with ``own`` true it makes the calls of this repository's package.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_HEADS = (1, 2, 3, 5, 8, 12, 16, 24, 40)


# ---------------------------------------------------------------------------- cases


def _rope(name, back, dtype, B, N, H, d, norm, grid, positions=False):
    return dict(name=name, op="rope", back=back, dtype=dtype, B=B, N=N, H=H, d=d, norm=norm,
                gt=grid[0], gh=grid[1], gw=grid[2], positions=positions)


def _norm(name, back, x, y, B, N, C, T, kind, affine, branch):
    return dict(name=name, op="norm", back=back, x=x, y=y, B=B, N=N, C=C, T=T, kind=kind,
                affine=affine, branch=branch)


def _cross(name, back, dtype, B, Nq, Nk, H, d, mask):
    return dict(name=name, op="cross", back=back, dtype=dtype, B=B, Nq=Nq, Nk=Nk, H=H, d=d, mask=mask)


def listed():
    return [
        # fp32 checks of a small clip: 1000 latent tokens, rotation alone
        _rope("rope f32 n1000", False, "f32", 2, 1000, 2, 64, "none", (2, 20, 25)),
        # q and k of a 14B self-attention layer at 480P, on their way to the attention
        _rope("rope 14b 480p", False, "bf16", 1, 32760, 40, 128, "token", (21, 30, 52)),
        # training the 1.3B model at 480P: back through the rotation and the norm
        _rope("rope backward 1.3b 480p", True, "bf16", 1, 32760, 12, 128, "token", (21, 30, 52)),
        # the norm of a single pooled token (time or image embedding)
        _norm("norm n1", False, "bf16", "bf16", 1, 1, 1536, 1, "layer", "mod", False),
        # between attention and the next block of a 14B model at 720P, residual stream in fp32
        _norm("norm 14b 720p", False, "f32", "bf16", 1, 75600, 5120, 1, "layer", "mod", True),
        # the same in training at 480P
        _norm("norm backward 14b 480p", True, "f32", "bf16", 1, 32760, 5120, 1, "layer", "mod", True),
        # a padded batch in fp32 with a learned gain; odd length
        _norm("norm backward f32 n777", True, "f32", "f32", 3, 777, 1000, 1, "rms", "weight", False),
        # one token (a pooled query) over a prompt, padded batch
        _cross("cross n1", False, "bf16", 2, 1, 512, 12, 128, "len"),
        # every video token of a 14B layer at 720P to 512 text states
        _cross("cross 14b 720p", False, "bf16", 1, 75600, 512, 40, 128, "none"),
        # its training pass at 480P
        _cross("cross backward 14b 480p", True, "bf16", 1, 32760, 512, 40, 128, "len"),
        # fp32 with a key mask, odd lengths on both sides
        _cross("cross f32 mask", False, "f32", 2, 777, 333, 3, 64, "mask"),
        # fp32 training against 257 image states
        _cross("cross backward f32", True, "f32", 1, 1000, 257, 12, 128, "none"),
    ]


def _log_int(rng, lo, hi):
    if hi <= lo:
        return lo
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, back = rng.choice(("rope", "norm", "cross")), rng.random() < 0.5
    if op == "rope":
        H, d = rng.choice(_HEADS), rng.choice((64, 128))
        B = rng.randint(1, 4)
        N = _log_int(rng, 1, 32760 * 40 * 128 // (B * H * d) if H * d * B > 1536 else 75600)
        gt = rng.randint(1, min(21, N))
        gh = rng.randint(1, min(45, N // gt))
        c = _rope("", back, rng.choice(("f32", "bf16", "bf16")), B, N, H, d,
                  rng.choice(("none", "token", "token", "head")), (gt, gh, N // gt // gh), rng.random() < 0.25)
    elif op == "norm":
        C = 8 * _log_int(rng, 8, 1024)
        B = rng.randint(1, 4)
        N = _log_int(rng, 1, min(75600, 32760 * 5120 // (B * C)))
        T = rng.choice((1, 1, N, rng.choice([t for t in range(1, 22) if N % t == 0])))
        x, y = rng.choice((("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")))
        c = _norm("", back, x, y, B, N, C, T, rng.choice(("layer", "rms")),
                  rng.choice(("mod", "mod", "weight", "none")), rng.random() < 0.6)
    else:
        dtype = rng.choice(("f32", "bf16", "bf16"))
        H, d, B = rng.choice(_HEADS), rng.choice((64, 128)), rng.randint(1, 4)
        Nk = _log_int(rng, 1, 8192)
        most = (40_000_000 if dtype == "f32" else 600_000_000) // (B * H * Nk)
        Nq = _log_int(rng, 1, max(1, min(75600, most)))
        c = _cross("", back, dtype, B, Nq, Nk, H, d, rng.choice(("none", "len", "mask")))
    del c["name"]
    return c


# ---------------------------------------------------------------------------- inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1_000_003 + 17)

    def rand(*shape, dtype=torch.float32, scale=1.0, shift=0.0):
        x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
        return x.mul_(scale).add_(shift).to(dtype)

    s = dict(case=case)
    if case["op"] == "rope":
        B, N, H, d, t = case["B"], case["N"], case["H"], case["d"], _TYPES[case["dtype"]]
        s["q"], s["k"] = rand(B, N, H, d, dtype=t), rand(B, N, H, d, dtype=t, scale=2.0)
        n = {"none": 0, "token": H * d, "head": d}[case["norm"]]
        s["wq"], s["wk"] = (rand(n, scale=0.1, shift=1.0), rand(n, scale=0.1, shift=1.0)) if n else (None, None)
        s["positions"] = None
        if case["positions"]:
            far = torch.tensor([2000, 500, 500], device="cuda")
            u = torch.rand(B, N, 3, generator=gen, device="cuda")
            s["positions"] = (u * far).to(torch.int32)
        if case["back"]:
            s["dq"], s["dk"] = rand(B, N, H, d, dtype=t), rand(B, N, H, d, dtype=t)
    elif case["op"] == "norm":
        B, N, C, T = case["B"], case["N"], case["C"], case["T"]
        x, y = _TYPES[case["x"]], _TYPES[case["y"]]
        s["x"] = rand(B, N, C, dtype=x, scale=1.5, shift=0.1)
        for name in ("branch", "gate", "scale", "shift", "weight", "bias"):
            s[name] = None
        if case["branch"]:
            s["branch"], s["gate"] = rand(B, N, C, dtype=y), rand(B, T, C, scale=0.5)
        if case["affine"] == "mod":
            s["scale"], s["shift"] = rand(B, T, C, scale=0.3), rand(B, T, C, scale=0.3)
        elif case["affine"] == "weight":
            s["weight"], s["bias"] = rand(C, scale=0.1, shift=1.0), rand(C, scale=0.1)
        if case["back"]:  # x plays r, the residual stream that the forward returned
            s["dy"], s["dr"] = rand(B, N, C, dtype=y), rand(B, N, C, dtype=x)
    else:
        B, Nq, Nk, H, d = (case[n] for n in ("B", "Nq", "Nk", "H", "d"))
        t = _TYPES[case["dtype"]]
        s["q"] = rand(B, Nq, H, d, dtype=t, scale=1.5)
        s["k"], s["v"] = rand(B, Nk, H, d, dtype=t, scale=1.2), rand(B, Nk, H, d, dtype=t)
        s["kv_len"] = s["key_mask"] = None
        if case["mask"] == "len":
            u = torch.rand(B, generator=gen, device="cuda")
            s["kv_len"] = (Nk * (0.5 + 0.5 * u)).ceil().to(torch.int32)
        elif case["mask"] == "mask":
            s["key_mask"] = torch.rand(B, Nk, generator=gen, device="cuda") < 0.7
        if case["back"]:
            s["dout"] = rand(B, Nq, H, d, dtype=t)
            s["out"], s["lse"] = _attend(s["q"], s["k"], s["v"], s["kv_len"], s["key_mask"])
    return s


# ---------------------------------------------------------------------------- plain forms


def _pairs(d, one_axis):
    P = d // 2
    return (0, 0, P) if one_axis else (P - 2 * (P // 3), P // 3, P // 3)


def _turns(case, positions, dtype):
    """cos and sin of every token's pairs, [N or B, N, 1, d/2]; tokens past the grid are not turned."""
    N, gt, gh, gw = case["N"], case["gt"], case["gh"], case["gw"]
    if positions is None:
        n = torch.arange(N, device="cuda")
        pos = torch.stack((n // (gh * gw), n // gw % gh, n % gw), -1) * (n < gt * gh * gw)[:, None]
        split = _pairs(case["d"], gt == 1 and gh == 1)
    else:
        pos, split = positions, _pairs(case["d"], False)
    pos = pos.to(torch.float64)
    a = [pos[..., i : i + 1] * 10000.0 ** (-torch.arange(p, device="cuda", dtype=torch.float64) / max(p, 1))
         for i, p in enumerate(split)]
    a = torch.cat(a, -1).unsqueeze(-2)
    return torch.cos(a).to(dtype), torch.sin(a).to(dtype)


def _turn(x, c, s):
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)


def _unit(x, norm, eps=1e-6):
    """1 / rms of each token, or of each head of it."""
    dims = (-2, -1) if norm == "token" else (-1,)
    return torch.rsqrt(x.square().mean(dims, keepdim=True) + eps), dims


def _rope_forward(x, w, case, c, s):
    y = x.float()
    if w is not None:
        y = y * _unit(y, case["norm"])[0] * w.view((case["H"], -1) if case["norm"] == "token" else (1, -1))
    return _turn(y, c, s).to(x.dtype)


def _rope_backward(dy, x, w, case, c, s):
    g = _turn(dy.float(), c, -s)
    if w is None:
        return g.to(x.dtype), None
    xf = x.float()
    rstd, dims = _unit(xf, case["norm"])
    xn = xf * rstd
    dw = (g * xn).sum((0, 1) if case["norm"] == "token" else (0, 1, 2)).reshape(-1)
    h = g * w.view((case["H"], -1) if case["norm"] == "token" else (1, -1))
    return (rstd * (h - xn * (h * xn).mean(dims, keepdim=True))).to(x.dtype), dw


def _spread(m, N):
    """A modulation [B, T, C] for every token [B, N, C]."""
    return m if m.shape[1] == 1 else m.repeat_interleave(N // m.shape[1], 1)


def _normed(r, kind, eps=1e-6):
    if kind == "layer":
        r = r - r.mean(-1, keepdim=True)
    rstd = torch.rsqrt(r.square().mean(-1, keepdim=True) + eps)
    return r * rstd, rstd


def _norm_forward(st):
    c, x = st["case"], st["x"]
    r = x.float()
    if st["branch"] is not None:
        r = r + _spread(st["gate"], c["N"]) * st["branch"].float()
    y = _normed(r, c["kind"])[0]
    if st["scale"] is not None:
        y = y * (1 + _spread(st["scale"], c["N"])) + _spread(st["shift"], c["N"])
    elif st["weight"] is not None:
        y = y * st["weight"] + st["bias"]
    return r.to(x.dtype), y.to(_TYPES[c["y"]])


def _norm_backward(st):
    c, r, dy = st["case"], st["x"], st["dy"].float()
    groups = (c["B"], c["T"], c["N"] // c["T"], c["C"])
    xn, rstd = _normed(r.float(), c["kind"])
    g, res = dy, {}
    if st["scale"] is not None:
        res["dscale"], res["dshift"] = (dy * xn).view(groups).sum(2), dy.view(groups).sum(2)
        g = dy * (1 + _spread(st["scale"], c["N"]))
    elif st["weight"] is not None:
        res["dweight"], res["dbias"] = (dy * xn).sum((0, 1)), dy.sum((0, 1))
        g = dy * st["weight"]
    t = g - xn * (g * xn).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        t = t - g.mean(-1, keepdim=True)
    dx = st["dr"].float() + rstd * t
    res["dx"] = dx.to(r.dtype)
    if st["branch"] is not None:
        res["dbranch"] = (dx * _spread(st["gate"], c["N"])).to(st["branch"].dtype)
        res["dgate"] = (dx * st["branch"].float()).view(groups).sum(2)
    return res


def _valid(k, kv_len, key_mask):
    """Which keys count, [B, Nk]."""
    ok = torch.ones(k.shape[:2], dtype=torch.bool, device=k.device)
    if kv_len is not None:
        ok = ok & (torch.arange(k.shape[1], device=k.device) < kv_len[:, None])
    return ok if key_mask is None else ok & key_mask


def _logits(q, k, ok):
    s = torch.matmul(q.permute(0, 2, 1, 3), k.permute(0, 2, 3, 1)).mul_(1 / math.sqrt(q.shape[-1]))
    return s.masked_fill_(~ok[:, None, None, :], -math.inf)


def _attend(q, k, v, kv_len, key_mask):
    ok = _valid(k, kv_len, key_mask)
    keep = ok[:, :, None, None]
    s = _logits(q.float(), k.float().where(keep, 0.0), ok)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.float().where(keep, 0.0).permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    return out.permute(0, 2, 1, 3).to(q.dtype).contiguous(), (m + total.log()).squeeze(-1)


def _attend_backward(dout, q, k, v, out, lse, kv_len, key_mask):
    ok = _valid(k, kv_len, key_mask)
    keep = ok[:, :, None, None]
    kf, vf = k.float().where(keep, 0.0), v.float().where(keep, 0.0)
    qf, do = q.float(), dout.float()
    p = _logits(qf, kf, ok).sub_(torch.where(lse == -math.inf, 0.0, lse)[..., None]).exp_()
    do_h = do.permute(0, 2, 1, 3)
    dv = torch.matmul(p.transpose(-1, -2), do_h)
    dot = (do * out.float()).sum(-1).permute(0, 2, 1)[..., None]
    ds = torch.matmul(do_h, vf.permute(0, 2, 3, 1)).sub_(dot).mul_(p).mul_(1 / math.sqrt(q.shape[-1]))
    dq = torch.matmul(ds, kf.permute(0, 2, 1, 3))
    dk = torch.matmul(ds.transpose(-1, -2), qf.permute(0, 2, 1, 3))
    return {n: g.permute(0, 2, 1, 3).to(q.dtype).contiguous() for n, g in (("dq", dq), ("dk", dk), ("dv", dv))}


def _run_plain(st):
    c = st["case"]
    if c["op"] == "rope":
        co, si = _turns(c, st["positions"], torch.float32)
        if not c["back"]:
            return {"q": _rope_forward(st["q"], st["wq"], c, co, si), "k": _rope_forward(st["k"], st["wk"], c, co, si)}
        dq, dwq = _rope_backward(st["dq"], st["q"], st["wq"], c, co, si)
        dk, dwk = _rope_backward(st["dk"], st["k"], st["wk"], c, co, si)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if c["op"] == "norm":
        if c["back"]:
            return _norm_backward(st)
        r, y = _norm_forward(st)
        return {"r": r, "y": y}
    if c["back"]:
        return _attend_backward(*(st[n] for n in ("dout", "q", "k", "v", "out", "lse", "kv_len", "key_mask")))
    out, lse = _attend(*(st[n] for n in ("q", "k", "v", "kv_len", "key_mask")))
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------- the framework's calls


def _run_own(st):
    import sparse_rank_attention_b200 as rola

    c = st["case"]
    if c["op"] == "rope":
        how = dict(norm=c["norm"], positions=st["positions"])
        if st["positions"] is None:
            how["grid"] = (c["gt"], c["gh"], c["gw"])
        if c["back"]:
            return rola.qk_norm_rope_backward(st["dq"], st["dk"], st["q"], st["k"], st["wq"], st["wk"], **how)
        q, k = rola.qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], **how)
        return {"q": q, "k": k}
    if c["op"] == "norm":
        if c["back"]:
            return rola.gated_norm_backward(st["dy"], st["x"], dr=st["dr"], branch=st["branch"], gate=st["gate"],
                                            scale=st["scale"], weight=st["weight"], norm=c["kind"])
        r, y = rola.gated_norm(st["x"], st["branch"], st["gate"], st["scale"], st["shift"], st["weight"], st["bias"],
                               norm=c["kind"], y_dtype=_TYPES[c["y"]])
        return {"r": r, "y": y}
    if c["back"]:
        return rola.cross_attend_backward(st["dout"], st["q"], st["k"], st["v"], st["out"], st["lse"],
                                          kv_len=st["kv_len"], key_mask=st["key_mask"])
    out, lse = rola.cross_attend(st["q"], st["k"], st["v"], kv_len=st["kv_len"], key_mask=st["key_mask"],
                                 return_lse=True)
    return {"out": out, "lse": lse}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------- the least work


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "rope":
        n = case["B"] * case["N"] * case["H"] * case["d"]
        reads = (2 if case["norm"] != "none" else 1) if case["back"] else 1
        b = 2 * n * size[case["dtype"]] * (1 + reads)
        if case["positions"]:
            b += 12 * case["B"] * case["N"]
        return {"bytes": b, "flops": 2 * n * (8 if case["back"] else 6)}
    if case["op"] == "norm":
        n, m = case["B"] * case["N"] * case["C"], 4 * case["B"] * case["T"] * case["C"]
        x, y = size[case["x"]], size[case["y"]]
        if case["back"]:
            b = n * (2 * x + y + x) + (n * 2 * y + 2 * m if case["branch"] else 0)
            b += 3 * m if case["affine"] == "mod" else 12 * case["C"] if case["affine"] == "weight" else 0
        else:
            b = n * (x + y) + (n * (x + y) + m if case["branch"] else 0)
            b += 2 * m if case["affine"] == "mod" else 8 * case["C"] if case["affine"] == "weight" else 0
        return {"bytes": b, "flops": n * (16 if case["back"] else 10)}
    B, Nq, Nk, H, d = (case[n] for n in ("B", "Nq", "Nk", "H", "d"))
    keys = Nk * (0.75 if case["mask"] == "len" else 0.7 if case["mask"] == "mask" else 1.0)
    q, k = B * Nq * H * d * size[case["dtype"]], B * keys * H * d * size[case["dtype"]]
    if case["back"]:
        return {"bytes": 4 * q + 4 * k + 4 * B * H * Nq, "flops": 10 * B * H * Nq * keys * d}
    return {"bytes": 2 * q + 2 * k + 4 * B * H * Nq, "flops": 4 * B * H * Nq * keys * d}


# ---------------------------------------------------------------------------- the definition in 64 bits


def _exact_rope(case, st):
    B, N, H, d = case["B"], case["N"], case["H"], case["d"]
    half = d // 2
    if st["positions"] is None:
        n = torch.arange(N, device="cuda")
        inside = n < case["gt"] * case["gh"] * case["gw"]
        axes = [n // (case["gh"] * case["gw"]), (n // case["gw"]) % case["gh"], n % case["gw"]]
        axes = [torch.where(inside, a, 0).double()[None] for a in axes]
        one = case["gt"] * case["gh"] == 1
    else:
        axes, one = [st["positions"][..., i].double() for i in range(3)], False
    hw = 0 if one else half // 3
    counts = [0, 0, half] if one else [half - 2 * hw, hw, hw]
    turn = torch.empty(axes[0].shape[0], N, 1, half, dtype=torch.complex128, device="cuda")
    at = 0
    for a, p in zip(axes, counts):
        for j in range(p):
            angle = a * math.pow(10000.0, -j / p)
            turn[:, :, 0, at] = torch.polar(torch.ones_like(angle), angle)
            at += 1

    def rotated(x, z):
        return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], half, 2)) * z).reshape(x.shape)

    over = {"none": None, "token": (2, 3), "head": (3,)}[case["norm"]]

    def gain(w):
        return w.double().reshape((H, d) if case["norm"] == "token" else (1, d))

    out = {}
    for n in ("q", "k"):
        x, w = st[n].double(), st["w" + n]
        if not case["back"]:
            if over is not None:
                x = x / (torch.linalg.vector_norm(x, dim=over, keepdim=True) ** 2
                         / (d * (H if len(over) == 2 else 1)) + 1e-6).sqrt() * gain(w)
            out[n] = rotated(x, turn)
            continue
        g = rotated(st["d" + n].double(), turn.conj())
        if over is None:
            out["d" + n], out["dw" + n] = g, None
            continue
        size = d * (H if len(over) == 2 else 1)
        rms = ((x * x).sum(over, keepdim=True) / size + 1e-6).sqrt()
        out["dw" + n] = (g * x / rms).sum((0, 1) if len(over) == 2 else (0, 1, 2)).reshape(-1)
        h = g * gain(w)
        out["d" + n] = h / rms - x * (h * x).sum(over, keepdim=True) / (size * rms ** 3)
    return out


def _exact_norm(case, st):
    B, N, C, T = case["B"], case["N"], case["C"], case["T"]
    parts = {n: [] for n in ("r", "y", "dx", "dbranch")}
    sums = {n: torch.zeros(B, T, C, dtype=torch.float64, device="cuda") for n in ("dgate", "dscale", "dshift")}
    per = N // T
    step = max(1, min(N, 40_000_000 // (B * C)))
    for lo in range(0, N, step):
        hi = min(N, lo + step)
        group = torch.arange(lo, hi, device="cuda") // per
        at = {n: None if st[n] is None else st[n].double()[:, group] for n in ("gate", "scale", "shift")}
        r = st["x"][:, lo:hi].double()
        a = None if st["branch"] is None else st["branch"][:, lo:hi].double()
        if not case["back"] and a is not None:
            r = r + at["gate"] * a
        mid = r.mean(-1, keepdim=True) if case["kind"] == "layer" else 0.0
        dev = torch.sqrt(((r - mid) ** 2).sum(-1, keepdim=True) / C + 1e-6)
        unit = (r - mid) / dev
        mul = 1 + at["scale"] if at["scale"] is not None else st["weight"].double() if st["weight"] is not None else 1.0
        if not case["back"]:
            add = at["shift"] if at["shift"] is not None else st["bias"].double() if st["bias"] is not None else 0.0
            parts["r"].append(r)
            parts["y"].append(unit * mul + add)
            continue
        dy = st["dy"][:, lo:hi].double()
        g = dy * mul
        inner = (g * unit).sum(-1, keepdim=True) / C
        dn = (g - (g.mean(-1, keepdim=True) if case["kind"] == "layer" else 0.0) - unit * inner) / dev
        dx = dn + st["dr"][:, lo:hi].double()
        parts["dx"].append(dx)
        sums["dscale"].index_add_(1, group, dy * unit)
        sums["dshift"].index_add_(1, group, dy)
        if a is not None:
            parts["dbranch"].append(dx * at["gate"])
            sums["dgate"].index_add_(1, group, dx * a)
    out = {n: torch.cat(v, 1) for n, v in parts.items() if v}
    if case["back"]:
        if a is not None:
            out["dgate"] = sums["dgate"]
        if case["affine"] == "mod":
            out["dscale"], out["dshift"] = sums["dscale"], sums["dshift"]
        elif case["affine"] == "weight":
            out["dweight"], out["dbias"] = sums["dscale"].sum((0, 1)), sums["dshift"].sum((0, 1))
    return out


def _exact_cross(case, st):
    B, Nq, Nk, H, d = (case[n] for n in ("B", "Nq", "Nk", "H", "d"))
    like = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(B, Nq, H, d, **like), torch.full((B, H, Nq), -math.inf, **like)
    dq, dk, dv = torch.zeros(B, Nq, H, d, **like), torch.zeros(B, Nk, H, d, **like), torch.zeros(B, Nk, H, d, **like)
    step = max(1, 200_000_000 // Nk)
    for b in range(B):
        keys = torch.arange(Nk, device="cuda")
        if st["kv_len"] is not None:
            keys = keys[: int(st["kv_len"][b])]
        if st["key_mask"] is not None:
            keys = keys[st["key_mask"][b, keys]]
        if not len(keys):
            continue
        for h in range(H):
            k, v = st["k"][b, keys, h].double(), st["v"][b, keys, h].double()
            for lo in range(0, Nq, step):
                q = st["q"][b, lo : lo + step, h].double()
                s = q @ k.T / math.sqrt(d)
                z = torch.logsumexp(s, -1)
                p = torch.softmax(s, -1)
                if not case["back"]:
                    out[b, lo : lo + step, h], lse[b, h, lo : lo + step] = p @ v, z
                    continue
                do = st["dout"][b, lo : lo + step, h].double()
                dp = do @ v.T
                ds = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(d)
                dq[b, lo : lo + step, h] = ds @ k
                dk[b, keys, h] += ds.T @ q
                dv[b, keys, h] += p.T @ do
    return {"dq": dq, "dk": dk, "dv": dv} if case["back"] else {"out": out, "lse": lse}


def exact(case, seed):
    return {"rope": _exact_rope, "norm": _exact_norm, "cross": _exact_cross}[case["op"]](case, prepare(case, seed))
