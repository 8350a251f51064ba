"""The operators around RoLA on the GPU against their plain 64-bit forms, element by element
within the bounds that tests/block_testlib.py derives."""
import math

import pytest
import torch

import block_testlib as L
import sparse_rank_attention_b200 as rola

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    rola.load()
    yield
    assert rola.block_poll_status() == 0


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---------------------------------------------------------------------------- qk_norm_rope

ROPE = [
    # B, N, H, d, dtype, norm, grid, options
    (1, 1, 1, 64, BF16, "token", None, {}),
    (2, 37, 3, 64, F32, "none", (1, 1, 37), {}),
    (1, 60, 2, 128, BF16, "head", (3, 4, 5), {}),
    (2, 61, 12, 128, BF16, "token", (3, 4, 5), {}),                      # a token past the grid
    (1, 50, 5, 128, F32, "token", (2, 5, 5), dict(start=(70000, 3, -2))),  # far and negative positions
    (3, 33, 40, 128, BF16, "token", None, dict(rope_base=256.0)),
    (1, 40, 64, 128, F32, "token", (2, 4, 5), {}),                       # the widest row
    (2, 24, 16, 64, F32, "head", (2, 3, 4), dict(pairs=(0, 20, 12))),
    (1, 300, 8, 64, BF16, "none", (3, 10, 10), {}),
    (2, 29, 24, 64, BF16, "token", None, dict(rope=False)),
]


def _rope_inputs(B, N, H, d, dtype, norm, seed):
    g = _gen(seed)
    n = {"none": 0, "token": H * d, "head": d}[norm]
    q, k = L.rand(g, B, N, H, d, dtype=dtype), L.rand(g, B, N, H, d, dtype=dtype, scale=3.0)
    w = [L.rand(g, n, scale=0.2, shift=1.0) if n else None for _ in range(2)]
    return g, q, k, *w


def _rope_angles(N, d, grid, opt):
    if not opt.get("rope", True):
        return None
    return L.angles(N, d, grid, opt.get("start", (0, 0, 0)), opt.get("positions"), opt.get("pairs", (0, 0, 0)),
                    opt.get("rope_base", 10000.0))


@pytest.mark.parametrize("B,N,H,d,dtype,norm,grid,opt", ROPE)
def test_qk_norm_rope(B, N, H, d, dtype, norm, grid, opt):
    g, q, k, wq, wk = _rope_inputs(B, N, H, d, dtype, norm, 1)
    a = _rope_angles(N, d, grid, opt)
    out = rola.qk_norm_rope(q, k, wq, wk, norm=norm, grid=grid, **opt)
    for x, w, y in ((q, wq, out[0]), (k, wk, out[1])):
        L.assert_within(y, *L.norm_rope_ref(x, w, norm, a), "y")
    alone = rola.qk_norm_rope(q, None, wq, norm=norm, grid=grid, **opt)
    assert torch.equal(alone, out[0])


@pytest.mark.parametrize("B,N,H,d,dtype,norm,grid,opt", ROPE)
@pytest.mark.parametrize("grad", ["same", "f32"])
def test_qk_norm_rope_backward(B, N, H, d, dtype, norm, grid, opt, grad):
    g, q, k, wq, wk = _rope_inputs(B, N, H, d, dtype, norm, 2)
    t = dtype if grad == "same" else F32
    dq, dk = L.rand(g, B, N, H, d, dtype=t), L.rand(g, B, N, H, d, dtype=t)
    a = _rope_angles(N, d, grid, opt)
    got = rola.qk_norm_rope_backward(dq, dk, q, k, wq, wk, norm=norm, grid=grid, **opt)
    for x, w, dy, n in ((q, wq, dq, "q"), (k, wk, dk, "k")):
        dx, dxe, dw, dwe = L.norm_rope_backward_ref(dy, x, w, norm, a)
        assert got["d" + n].dtype == dtype
        L.assert_within(got["d" + n], dx, dxe, "d" + n)
        if norm == "none":
            assert got["dw" + n] is None
        else:
            L.assert_within(got["dw" + n], dw, dwe, "dw" + n)
    again = rola.qk_norm_rope_backward(dq, dk, q, k, wq, wk, norm=norm, grid=grid, **opt)
    assert all(got[n] is None or torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("batched", [False, True])
def test_qk_norm_rope_given_positions(batched):
    B, N, H, d = 2, 45, 3, 128
    g, q, k, wq, wk = _rope_inputs(B, N, H, d, F32, "head", 3)
    pos = torch.randint(-(2 ** 31), 2 ** 31 - 1, (B, N, 3) if batched else (N, 3), generator=g, device="cuda",
                        dtype=torch.int64).to(torch.int32)
    a = L.angles(N, d, positions=pos)
    # the reference's own fp64 angle (up to 2^31) carries 2^31 * 2^-53 * 2: far below u
    out = rola.qk_norm_rope(q, k, wq, wk, norm="head", positions=pos)
    for x, w, y in ((q, wq, out[0]), (k, wk, out[1])):
        L.assert_within(y, *L.norm_rope_ref(x, w, "head", a), "y")


def test_qk_norm_rope_views_and_in_place():
    B, N, H, d = 2, 50, 4, 64
    g = _gen(4)
    qkv = L.rand(g, B, N, 3, H, d, dtype=BF16)          # a fused projection
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    wq, wk = L.rand(g, H * d), L.rand(g, H * d)
    want = rola.qk_norm_rope(q.contiguous(), k.contiguous(), wq, wk, grid=(2, 5, 5))
    v = qkv[:, :, 2].clone()
    for x, y in zip(rola.qk_norm_rope(q, k, wq, wk, grid=(2, 5, 5)), want):
        assert torch.equal(x, y)
    heads_first = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k)]
    for x, y in zip(rola.qk_norm_rope(*heads_first, wq, wk, grid=(2, 5, 5)), want):
        assert torch.equal(x, y)
    rola.qk_norm_rope(q, k, wq, wk, grid=(2, 5, 5), out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, :, 2], v)


# ---------------------------------------------------------------------------- gated_norm

NORM = [
    # B, N, C, T, x, y, kind, affine, branch, gate
    (1, 1, 8, 1, BF16, BF16, "layer", "mod", False, False),
    (2, 7, 64, 1, F32, F32, "layer", "weight", True, True),
    (1, 33, 1536, 1, F32, BF16, "layer", "mod", True, True),
    (2, 12, 1000, 4, BF16, BF16, "rms", "mod", True, True),
    (3, 5, 5120, 5, F32, BF16, "layer", "mod", True, True),      # a modulation per token
    (1, 40, 8192, 2, F32, F32, "rms", "none", True, False),
    (2, 301, 264, 7, BF16, BF16, "layer", "mod", False, False),
    (1, 700, 136, 1, F32, BF16, "rms", "weight", True, True),
    (4, 9, 2056, 9, BF16, BF16, "layer", "none", True, True),
    (2, 100, 2048, 1, F32, F32, "layer", "weight", False, False),
]


def _norm_inputs(B, N, C, T, x, y, affine, branch, gate, seed):
    g = _gen(seed)
    s = dict(x=L.rand(g, B, N, C, dtype=x, scale=2.0, shift=0.7))
    s["branch"] = L.rand(g, B, N, C, dtype=y) if branch else None
    mods = L.rand(g, B, T, 3, C, scale=0.5)               # one tensor, as a block's modulation is
    s["gate"] = mods[:, :, 0] if gate else None
    s["scale"], s["shift"] = (mods[:, :, 1], mods[:, :, 2]) if affine == "mod" else (None, None)
    s["weight"], s["bias"] = (L.rand(g, C, shift=1.0), L.rand(g, C)) if affine == "weight" else (None, None)
    return g, s


@pytest.mark.parametrize("B,N,C,T,x,y,kind,affine,branch,gate", NORM)
def test_gated_norm(B, N, C, T, x, y, kind, affine, branch, gate):
    g, s = _norm_inputs(B, N, C, T, x, y, affine, branch, gate, 5)
    r, out = rola.gated_norm(**s, norm=kind, y_dtype=y)
    wr, wy = L.gated_norm_ref(*s.values(), kind, y)
    if branch:
        L.assert_within(r, *wr, "r")
    else:
        assert r is s["x"]
    L.assert_within(out, *wy, "y")
    if branch:                                            # the residual stream in place
        x2 = s["x"].clone()
        r2, y2 = rola.gated_norm(**{**s, "x": x2}, norm=kind, out=(x2, torch.empty_like(out)))
        assert r2 is x2 and torch.equal(r2, r) and torch.equal(y2, out)


@pytest.mark.parametrize("B,N,C,T,x,y,kind,affine,branch,gate", NORM)
@pytest.mark.parametrize("with_dr", [False, True])
def test_gated_norm_backward(B, N, C, T, x, y, kind, affine, branch, gate, with_dr):
    g, s = _norm_inputs(B, N, C, T, x, y, affine, branch, gate, 6)
    dy, dr = L.rand(g, B, N, C, dtype=y), L.rand(g, B, N, C, dtype=x) if with_dr else None
    args = dict(dr=dr, branch=s["branch"], gate=s["gate"], scale=s["scale"], weight=s["weight"])
    got = rola.gated_norm_backward(dy, s["x"], **args, norm=kind)
    want = L.gated_norm_backward_ref(dy, s["x"], *args.values(), kind)
    for n, v in got.items():
        assert (v is None) == (n not in want), n
        if v is not None:
            L.assert_within(v, *want[n], n)
    again = rola.gated_norm_backward(dy, s["x"], **args, norm=kind)
    assert all(v is None or torch.equal(v, again[n]) for n, v in got.items())


def test_gated_norm_mean_far_from_zero():
    """A residual stream whose mean is 4096 times its spread: the variance survives (the bound
    scales with mean / spread, not with its square)."""
    g = _gen(7)
    x = L.rand(g, 2, 9, 1536, shift=4096.0)
    _, y = rola.gated_norm(x, y_dtype=F32)
    _, want = L.gated_norm_ref(x, None, None, None, None, None, None, "layer", F32)
    L.assert_within(y, *want, "y")


# ---------------------------------------------------------------------------- cross_attend

CROSS = [
    # B, Nq, Nk, H, d, kv_len, mask
    (1, 1, 1, 1, 64, None, None),
    (2, 1, 512, 3, 128, "some", None),
    (1, 64, 64, 2, 128, None, None),
    (2, 65, 63, 2, 64, None, "random"),
    (3, 127, 129, 1, 128, "empty", None),                 # a sample without keys
    (2, 200, 257, 2, 128, None, "empty"),
    (1, 300, 128, 3, 128, "some", "random"),
    (2, 513, 77, 2, 64, "some", None),
    (1, 3, 2000, 2, 128, None, "random"),                 # few queries, many keys: split over keys
    (1, 2, 4001, 1, 64, "some", None),
    (1, 3001, 5, 1, 128, None, None),                     # many queries, few keys: split over queries
    (2, 1025, 384, 1, 64, None, "random"),
    (1, 257, 640, 1, 128, "some", "random"),
]


def _cross_inputs(B, Nq, Nk, H, d, dtype, lens, mask, seed):
    g = _gen(seed)
    q = L.rand(g, B, Nq, H, d, dtype=dtype, scale=1.5)
    k, v = L.rand(g, B, Nk, H, d, dtype=dtype, scale=1.2), L.rand(g, B, Nk, H, d, dtype=dtype)
    kv_len = key_mask = None
    if lens:
        kv_len = torch.randint(1, Nk + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        if lens == "empty":
            kv_len[1] = 0
    if mask:
        key_mask = torch.rand(B, Nk, generator=g, device="cuda") < 0.6
        if mask == "empty":
            key_mask[-1] = False
    return g, q, k, v, kv_len, key_mask


def _spoil(k, v, ok):
    """k and v with NaN, infinities and the type's lowest value where no key counts."""
    bad = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(k.dtype).min], device="cuda").to(k.dtype)
    fill = bad[torch.arange(k[0, 0].numel(), device="cuda") % 4].view(k.shape[2:])
    return tuple(x.where(ok[:, :, None, None], fill) for x in (k, v))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,Nq,Nk,H,d,lens,mask", CROSS)
def test_cross_attend(B, Nq, Nk, H, d, lens, mask, dtype):
    g, q, k, v, kv_len, key_mask = _cross_inputs(B, Nq, Nk, H, d, dtype, lens, mask, 8)
    (want, oe), (wz, ze) = L.cross_ref(q, k, v, kv_len, key_mask)
    out, lse = rola.cross_attend(q, k, v, kv_len=kv_len, key_mask=key_mask, return_lse=True)
    L.assert_within(out, want, oe, "out")
    L.assert_within(lse, wz, ze, "lse")
    assert torch.equal(rola.cross_attend(q, k, v, kv_len=kv_len, key_mask=key_mask), out)
    ok = L.valid_keys(B, Nk, kv_len, key_mask, "cuda")
    if not bool(ok.all()):
        ks, vs = _spoil(k, v, ok)
        out2, lse2 = rola.cross_attend(q, ks, vs, kv_len=kv_len, key_mask=key_mask, return_lse=True)
        assert torch.equal(out2, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,Nq,Nk,H,d,lens,mask", CROSS)
def test_cross_attend_backward(B, Nq, Nk, H, d, lens, mask, dtype):
    g, q, k, v, kv_len, key_mask = _cross_inputs(B, Nq, Nk, H, d, dtype, lens, mask, 9)
    dout = L.rand(g, B, Nq, H, d, dtype=dtype)
    out, lse = rola.cross_attend(q, k, v, kv_len=kv_len, key_mask=key_mask, return_lse=True)
    got = rola.cross_attend_backward(dout, q, k, v, out, lse, kv_len=kv_len, key_mask=key_mask)
    want = L.cross_backward_ref(dout, q, k, v, out, lse, kv_len, key_mask)
    for n, x in got.items():
        L.assert_within(x, *want[n], n)
    ok = L.valid_keys(B, Nk, kv_len, key_mask, "cuda")
    for n in ("dk", "dv"):
        assert not got[n].where(~ok[:, :, None, None], 0).any(), f"{n} at keys that do not count"
    spoiled = _spoil(k, v, ok)
    again = rola.cross_attend_backward(dout, q, *spoiled, out, lse, kv_len=kv_len, key_mask=key_mask)
    assert all(torch.equal(got[n], again[n]) for n in got)


def test_cross_attend_views_and_scale():
    g = _gen(10)
    B, Nq, Nk, H, d = 2, 70, 90, 3, 128
    q = L.rand(g, B, H, Nq, d, dtype=BF16).transpose(1, 2)          # heads outside tokens
    kv = L.rand(g, B, Nk, 2, H, d, dtype=BF16)                      # a fused projection
    k, v = kv[:, :, 0], kv[:, :, 1]
    dout = L.rand(g, B, H, Nq, d, dtype=BF16).transpose(1, 2)
    out, lse = rola.cross_attend(q, k, v, softmax_scale=0.05, return_lse=True)
    want = rola.cross_attend(q.contiguous(), k.contiguous(), v.contiguous(), softmax_scale=0.05)
    assert torch.equal(out, want)
    L.assert_within(out, *L.cross_ref(q, k, v, scale=0.05)[0], "out")
    got = rola.cross_attend_backward(dout, q, k, v, out, lse, softmax_scale=0.05)
    ref = L.cross_backward_ref(dout, q, k, v, out, lse, scale=0.05)
    for n, x in got.items():
        L.assert_within(x, *ref[n], n)


def test_cross_attend_growing_scores():
    """Keys whose scores rise along the axis by far more than a type's range: the running
    maximum moves at every tile."""
    g = _gen(11)
    for dtype in (F32, BF16):
        q = torch.ones(1, 130, 2, 128, device="cuda", dtype=dtype)
        ramp = torch.linspace(-8, 8, 700, device="cuda")[None, :, None, None].expand(1, 700, 2, 128)
        k = (ramp + 0.01 * L.rand(g, 1, 700, 2, 128)).to(dtype)
        v = L.rand(g, 1, 700, 2, 128, dtype=dtype)
        for kk in (k, k.flip(1)):
            (want, oe), (wz, ze) = L.cross_ref(q, kk, v)
            out, lse = rola.cross_attend(q, kk.contiguous(), v, return_lse=True)
            L.assert_within(out, want, oe, "out")
            L.assert_within(lse, wz, ze, "lse")


@pytest.mark.parametrize("d", [64, 128])
def test_cross_attend_repeats_bit_by_bit(d):
    """Many key tiles through the rings of several blocks, again and again beside another
    stream's traffic: every call gives the same bits and none of its waits runs out."""
    g, q, k, v, _, _ = _cross_inputs(1, 2000, 3001, 8, d, BF16, None, None, 12)
    dout = L.rand(g, 1, 2000, 8, d, dtype=BF16)
    out, lse = rola.cross_attend(q, k, v, return_lse=True)
    want = rola.cross_attend_backward(dout, q, k, v, out, lse)
    other = torch.cuda.Stream()
    big = torch.empty(64 << 20, device="cuda")
    torch.cuda.synchronize()
    for _ in range(40):
        with torch.cuda.stream(other):
            big.mul_(1.0)                                          # moves the loads' arrival around
        again = rola.cross_attend(q, k, v, return_lse=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
        got = rola.cross_attend_backward(dout, q, k, v, out, lse)
        assert all(torch.equal(got[n], want[n]) for n in got)
    assert rola.block_poll_status() == 0
