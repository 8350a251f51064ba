"""The operators around RoLA as a program uses them: on streams of their own and two at once,
captured and replayed, in place, on broadcast and on far memory, with their gradients against
differences of the plain forms, and run together with RoLA as in a transformer block."""
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


# ---------------------------------------------------------------------------- every call, once

# Sizes: long keys beside few queries (the keys are split, so the forward has a workspace) and
# several rows per partial sum.


def _calls(seed, dtype=BF16):
    """{name: call(stream=None) -> list of results}, all inputs fixed."""
    g = _gen(seed)
    B, N, H, d, Nk, C = 2, 300, 3, 128, 1500, 384
    q, k = L.rand(g, B, N, H, d, dtype=dtype), L.rand(g, B, N, H, d, dtype=dtype)
    wq, wk = L.rand(g, H * d, shift=1.0), L.rand(g, H * d, shift=1.0)
    ke, ve = L.rand(g, B, Nk, H, d, dtype=dtype), L.rand(g, B, Nk, H, d, dtype=dtype)
    few = L.rand(g, B, 70, H, d, dtype=dtype)
    kv_len = torch.tensor([1401, 777], dtype=torch.int32, device="cuda")
    mask = torch.rand(B, Nk, generator=g, device="cuda") < 0.8
    out, lse = rola.cross_attend(few, ke, ve, kv_len=kv_len, key_mask=mask, return_lse=True)
    dout = L.rand(g, B, 70, H, d, dtype=dtype)
    x, branch = L.rand(g, B, N, C), L.rand(g, B, N, C, dtype=dtype)
    gate, scale, shift = L.rand(g, B, 3, 3, C, scale=0.5).unbind(2)
    dy, dr = L.rand(g, B, N, C, dtype=dtype), L.rand(g, B, N, C)
    torch.cuda.synchronize()
    return {
        "rope": lambda **s: list(rola.qk_norm_rope(q, k, wq, wk, grid=(3, 10, 10), **s)),
        "rope backward": lambda **s: list(rola.qk_norm_rope_backward(q, k, k, q, wq, wk, grid=(3, 10, 10), **s).values()),
        "norm": lambda **s: list(rola.gated_norm(x, branch, gate, scale, shift, **s)),
        "norm backward": lambda **s: [t for t in rola.gated_norm_backward(dy, x, dr, branch, gate, scale, **s).values()
                                      if t is not None],
        "cross": lambda **s: list(rola.cross_attend(few, ke, ve, kv_len=kv_len, key_mask=mask, return_lse=True, **s)),
        "cross backward": lambda **s: list(rola.cross_attend_backward(dout, few, ke, ve, out, lse, kv_len=kv_len,
                                                                      key_mask=mask, **s).values()),
    }


NAMES = ["rope", "rope backward", "norm", "norm backward", "cross", "cross backward"]


def _same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", NAMES)
def test_own_stream(name, dtype):
    """A call on a busy stream; the current stream goes on at once and fills what it allocates."""
    call = _calls(20, dtype)[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                      # about 10 ms: the call waits behind it
    got = call(stream=side)
    for n in (1 << 12, 1 << 16, 1 << 20, 1 << 23):         # what the allocator would hand out again
        torch.full((n,), math.nan, device="cuda")
    side.synchronize()
    assert _same(got, want)
    assert torch.cuda.current_stream() != side


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(name, dtype):
    a, b = _calls(21, dtype)[name], _calls(22, dtype)[name]
    want = a(), b()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = a(stream=s), b(stream=t)
        torch.cuda.synchronize()
        assert _same(got[0], want[0]) and _same(got[1], want[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", NAMES)
def test_two_graphs(name, dtype):
    """Two captures of one operator, replayed in turn and with calls in between."""
    a, b = _calls(23, dtype)[name], _calls(24, dtype)[name]
    want = a(), b()
    torch.cuda.synchronize()
    graphs, results = [], []
    for call in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append(call())
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for r in results:
            for x in r:
                x.zero_()
        for i in order:
            graphs[i].replay()
            assert _same(a(), want[0])
        torch.cuda.synchronize()
        assert _same(results[0], want[0]) and _same(results[1], want[1])


# ---------------------------------------------------------------------------- odd tensors


def test_broadcast_modulation():
    """One modulation row for all samples (stride 0), gradients per sample."""
    g = _gen(25)
    B, N, C = 3, 40, 256
    x, branch, dy = L.rand(g, B, N, C), L.rand(g, B, N, C), L.rand(g, B, N, C)
    rows = [L.rand(g, C, scale=0.5) for _ in range(3)]
    wide = [r.expand(B, 4, C) for r in rows]
    full = [w.contiguous() for w in wide]
    assert _same(rola.gated_norm(x, branch, *wide), rola.gated_norm(x, branch, *full))
    a = rola.gated_norm_backward(dy, x, None, branch, wide[0], wide[1])
    b = rola.gated_norm_backward(dy, x, None, branch, full[0], full[1])
    assert a["dscale"].shape == (B, 4, C)
    assert all(a[n] is None and b[n] is None or torch.equal(a[n], b[n]) for n in a)


def test_gated_norm_in_place():
    g = _gen(26)
    x, branch = L.rand(g, 2, 500, 1536), L.rand(g, 2, 500, 1536, dtype=BF16)
    gate, scale, shift = L.rand(g, 2, 3, 1536).unbind(1)
    want = rola.gated_norm(x, branch, gate, scale, shift)
    y = torch.empty_like(branch)
    r, _ = rola.gated_norm(x, branch, gate, scale, shift, out=(x, y))
    assert r is x and torch.equal(x, want[0]) and torch.equal(y, want[1])


def test_broadcast_activations_are_refused():
    x = torch.randn(1, 1, 2, 64, device="cuda")
    wide, w = x.expand(1, 40, 2, 64), torch.ones(128, device="cuda")
    for call in (lambda: rola.qk_norm_rope(wide, None, w), lambda: rola.cross_attend(wide, wide, wide),
                 lambda: rola.gated_norm(x[0].expand(30, 2, 64)), lambda: rola.qk_norm_rope(x, None, w.cpu()),
                 lambda: rola.cross_attend(x, x, x.cpu()),
                 lambda: rola.cross_attend(x, x, x, out=x), lambda: rola.qk_norm_rope(x, x, w, w, out=(x, x)),
                 lambda: rola.gated_norm(x[0], x[0], out=(x[0], x[0])),
                 lambda: rola.cross_attend(x, x, x, key_mask=torch.ones(1, 1, dtype=torch.bool))):
        with pytest.raises(rola.RolaError):
            call()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_sample_without_keys_ignores_its_queries(dtype):
    """out = 0, lse = -inf and zero gradients, whatever the sample's q and dout hold."""
    g = _gen(27)
    B, Nq, Nk, H, d = 3, 150, 200, 2, 64
    q, dout = L.rand(g, B, Nq, H, d, dtype=dtype), L.rand(g, B, Nq, H, d, dtype=dtype)
    k, v = L.rand(g, B, Nk, H, d, dtype=dtype), L.rand(g, B, Nk, H, d, dtype=dtype)
    q[0, ::3], dout[0, ::2], q[1, 5], dout[1, 7] = math.nan, math.inf, math.inf, math.nan
    kv_len = torch.tensor([0, Nk, Nk + 9], dtype=torch.int32, device="cuda")     # past Nk: all keys
    mask = torch.ones(B, Nk, dtype=torch.bool, device="cuda")
    mask[1] = False
    out, lse = rola.cross_attend(q, k, v, kv_len=kv_len, key_mask=mask, return_lse=True)
    assert not out[:2].any() and bool((lse[:2] == -math.inf).all())
    got = rola.cross_attend_backward(dout, q, k, v, out, lse, kv_len=kv_len, key_mask=mask)
    for n, x in got.items():
        assert not x[:2].any(), n
    alone = rola.cross_attend(q[2:], k[2:], v[2:], return_lse=True)
    (want, oe), (wz, ze) = L.cross_ref(q[2:], k[2:], v[2:])
    for o, z in ((out[2:], lse[2:]), alone):
        L.assert_within(o, want, oe, "out")
        L.assert_within(z, wz, ze, "lse")
    ref = L.cross_backward_ref(dout[2:], q[2:], k[2:], v[2:], out[2:], lse[2:])
    for n, x in got.items():
        L.assert_within(x[2:], *ref[n], n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("low", [0.0, -300.0])
def test_masks_that_empty_whole_tiles(dtype, low):
    """Runs of invalid keys longer than a tile before, between and behind the valid ones, a
    single valid key, and scores far below zero (their exponentials vanish without the row's
    own maximum)."""
    g = _gen(33)
    B, Nq, Nk, H, d = 5, 140, 900, 2, 128
    q, k, v = L.rand(g, B, Nq, H, d), L.rand(g, B, Nk, H, d), L.rand(g, B, Nk, H, d, dtype=dtype)
    q[..., 0], k[..., 0] = 16.0, low * d ** 0.5 / 16                # adds `low` to every score
    q, k, dout = q.to(dtype), k.to(dtype), L.rand(g, B, Nq, H, d, dtype=dtype)
    mask = torch.zeros(B, Nk, dtype=torch.bool, device="cuda")
    mask[0, 700:] = True
    mask[1, 130:140] = mask[1, 650] = True
    mask[2, -1] = True
    mask[3, 0] = True
    mask[4, :3] = mask[4, 255:257] = True
    out, lse = rola.cross_attend(q, k, v, key_mask=mask, return_lse=True)
    (want, oe), (wz, ze) = L.cross_ref(q, k, v, key_mask=mask)
    L.assert_within(out, want, oe, "out")
    L.assert_within(lse, wz, ze, "lse")
    got = rola.cross_attend_backward(dout, q, k, v, out, lse, key_mask=mask)
    ref = L.cross_backward_ref(dout, q, k, v, out, lse, key_mask=mask)
    for n, x in got.items():
        L.assert_within(x, *ref[n], n)


@pytest.mark.parametrize("x,y", [(F32, F32), (F32, BF16), (BF16, BF16)])
def test_gated_norm_of_a_large_mean(x, y):
    """Rows a thousand spreads away from zero, as fp32 and as bf16 hold them."""
    g = _gen(34)
    r = L.rand(g, 2, 50, 640, dtype=x, shift=1000.0)
    scale, shift = L.rand(g, 2, 2, 640, scale=0.5).unbind(1)
    _, out = rola.gated_norm(r, None, None, scale, shift, y_dtype=y)
    L.assert_within(out, *L.gated_norm_ref(r, None, None, scale, shift, None, None, "layer", y)[1], "y")
    dy = L.rand(g, 2, 50, 640, dtype=y)
    got = rola.gated_norm_backward(dy, r, None, None, None, scale)
    for n, want in L.gated_norm_backward_ref(dy, r, None, None, None, scale, None, "layer").items():
        L.assert_within(got[n], *want, n)


def test_extreme_rows():
    """Zeros (eps alone holds the norm up), the largest finite values and infinities stay in their
    rows."""
    x = torch.zeros(1, 4, 2, 64, device="cuda")
    x[0, 1], x[0, 2, 0, 3], x[0, 3] = 1e18, math.inf, 1.0
    w = torch.ones(128, device="cuda")
    y = rola.qk_norm_rope(x, None, w, rope=False)
    assert not y[0, 0].any() and bool(torch.isfinite(y[0, [1, 3]]).all())
    assert torch.allclose(y[0, 1], torch.ones_like(y[0, 1])) and not bool(torch.isfinite(y[0, 2]).all())
    z = rola.gated_norm(x.view(1, 4, 128), weight=w, norm="rms")[1].view_as(y)
    assert torch.allclose(z[0, [0, 1, 3]], y[0, [0, 1, 3]]) and not bool(torch.isfinite(z[0, 2]).all())


def _room(nbytes):
    if torch.cuda.mem_get_info()[0] < nbytes + (8 << 30):
        pytest.skip(f"needs {nbytes >> 30} GB free")


def _far(x, step):
    """x [1, N, H, d] with its tokens `step` elements apart in a buffer past 2^31 elements."""
    n, hd = x.shape[1], x.shape[2] * x.shape[3]
    assert (n - 1) * step > 2 ** 31
    big = torch.empty((n - 1) * step + hd, dtype=x.dtype, device="cuda")
    y = big.as_strided(x.shape, (n * step, step, x.shape[3], 1))
    return y.copy_(x)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_far_tokens(dtype):
    """Token strides that carry the last rows past 2^32 bytes and 2^31 elements."""
    N, H, d, step = 160, 2, 128, 1 << 24
    _room(2 * N * step * 4)
    g = _gen(28)
    x, y, z = (L.rand(g, 1, N, H, d, dtype=dtype) for _ in range(3))
    w = L.rand(g, H * d, shift=1.0)
    xf, yf = _far(x, step), _far(y, step)
    assert torch.equal(rola.qk_norm_rope(xf, None, w), rola.qk_norm_rope(x, None, w))
    a, b = rola.qk_norm_rope_backward(yf, None, xf, None, w), rola.qk_norm_rope_backward(y, None, x, None, w)
    assert torch.equal(a["dq"], b["dq"]) and torch.equal(a["dwq"], b["dwq"])
    out, lse = rola.cross_attend(z, x, y, return_lse=True)
    assert _same(rola.cross_attend(z, xf, yf, return_lse=True), (out, lse))
    c, e = rola.cross_attend_backward(z, z, xf, yf, out, lse), rola.cross_attend_backward(z, z, x, y, out, lse)
    assert all(torch.equal(c[n], e[n]) for n in c)
    out, lse = rola.cross_attend(x, z, y, return_lse=True)
    assert _same(rola.cross_attend(xf, z, y, return_lse=True), (out, lse))
    c, e = rola.cross_attend_backward(yf, xf, z, z, out, lse), rola.cross_attend_backward(y, x, z, z, out, lse)
    assert all(torch.equal(c[n], e[n]) for n in c)


def test_far_rows():
    """Contiguous results past 2^31 elements: the last rows against the same rows alone."""
    C, tail = 8192, 300
    N = 2 ** 31 // C + tail
    _room(6 * 2 ** 32)
    g = _gen(29)
    x = torch.empty(1, N, C, dtype=BF16, device="cuda")
    x.normal_(generator=g)
    last = x[:, -tail:].contiguous()
    w = L.rand(g, C, shift=1.0)
    _, y = rola.gated_norm(x, weight=w, norm="rms")
    assert torch.equal(y[:, -tail:], rola.gated_norm(last, weight=w, norm="rms")[1])
    res = rola.gated_norm_backward(y, x, x, weight=w, norm="rms")
    ref = rola.gated_norm_backward(y[:, -tail:].contiguous(), last, last, weight=w, norm="rms")
    assert torch.equal(res["dx"][:, -tail:], ref["dx"])
    del y, res
    q, lastq = x.view(1, N, 64, 128), last.view(1, tail, 64, 128)
    out = rola.qk_norm_rope(q, None, w, rope=False)
    assert torch.equal(out[:, -tail:], rola.qk_norm_rope(lastq, None, w, rope=False))
    dq = rola.qk_norm_rope_backward(out, None, q, None, w, rope=False)["dq"]
    assert torch.equal(dq[:, -tail:], rola.qk_norm_rope_backward(out[:, -tail:].contiguous(), None, lastq, None, w,
                                                                 rope=False)["dq"])
    del out, dq
    k, v = (L.rand(g, 1, 5, 64, 128, dtype=BF16) for _ in range(2))
    out, lse = rola.cross_attend(q, k, v, return_lse=True)
    few, z = rola.cross_attend(lastq, k, v, return_lse=True)
    L.assert_within(out[:, -tail:], *L.cross_ref(lastq, k, v)[0], "out")
    L.assert_within(few, *L.cross_ref(lastq, k, v)[0], "out")
    got = rola.cross_attend_backward(out, q, k, v, out, lse)["dq"][:, -tail:]
    o, zz = out[:, -tail:].contiguous(), lse[:, :, -tail:].contiguous()
    L.assert_within(got, *L.cross_backward_ref(o, lastq, k, v, o, zz)["dq"], "dq")


# ---------------------------------------------------------------------------- differences


def _slope(f, xs, vs, eps=1e-4):
    """d/dt f(x + t v) at 0 by a five-point rule in fp64: off by about eps^4 times a fifth
    derivative, and 2^-52 |f| / eps."""
    def at(t):
        return f(*[x + t * v for x, v in zip(xs, vs)])
    return (8 * (at(eps) - at(-eps)) - (at(2 * eps) - at(-2 * eps))) / (12 * eps)


def _check_slopes(f, xs, grads, g, noise=1e-9):
    """<gradient, v> for one input at a time, v random; grads: (gradient, bound) per input."""
    for i, (grad, bound) in enumerate(grads):
        v = [torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64) if j == i else 0 * x
             for j, x in enumerate(xs)]
        got = float((grad.double() * v[i]).sum())
        want = float(_slope(f, xs, v))
        tol = float((bound * v[i].abs()).sum()) + noise * (1 + abs(want))
        assert abs(got - want) <= tol, f"input {i}: {got} against {want}, bound {tol:.2e}"


@pytest.mark.parametrize("norm", ["none", "token", "head"])
def test_qk_norm_rope_slopes(norm):
    g = _gen(30)
    B, N, H, d = 2, 24, 2, 64
    x, u = L.rand(g, B, N, H, d), L.rand(g, B, N, H, d)
    w = None if norm == "none" else L.rand(g, H * d if norm == "token" else d, shift=1.0)
    a = L.angles(N, d, (2, 3, 4))
    got = rola.qk_norm_rope_backward(u, None, x, None, w, norm=norm, grid=(2, 3, 4))
    dx, dxe, dw, dwe = L.norm_rope_backward_ref(u, x, w, norm, a)
    xs = [x.double()] + ([] if w is None else [w.double()])
    _check_slopes(lambda x, w=None: (L.norm_rope_ref(x, w, norm, a)[0] * u.double()).sum(), xs,
                  [(got["dq"], dxe)] + ([] if w is None else [(got["dwq"], dwe)]), g)


@pytest.mark.parametrize("kind,affine", [("layer", "mod"), ("rms", "mod"), ("layer", "weight")])
def test_gated_norm_slopes(kind, affine):
    g = _gen(31)
    B, N, C, T = 2, 12, 72, 3
    x, branch, u, ur = (L.rand(g, B, N, C) for _ in range(4))
    mod = affine == "mod"
    gate, scale, shift = (L.rand(g, B, T, C, scale=0.5) for _ in range(3))
    weight, bias = L.rand(g, C, shift=1.0), L.rand(g, C)
    r, _ = rola.gated_norm(x, branch, gate, *((scale, shift) if mod else (None, None, weight, bias)), norm=kind)
    got = rola.gated_norm_backward(u, r, ur, branch, gate, *((scale,) if mod else (None, weight)), norm=kind)
    ref = L.gated_norm_backward_ref(u, r, ur, branch, gate, scale if mod else None, None if mod else weight, kind)
    # the plain form rounds nothing; at the unrounded r the gradients move by what the formula says
    exact = x.double() + L.spread(gate, N) * branch.double()
    near = L.gated_norm_backward_ref(u.double(), exact, ur.double(), branch.double(), gate.double(),
                                     scale.double() if mod else None, None if mod else weight.double(), kind)
    names = ["dx", "dbranch", "dgate"] + (["dscale", "dshift"] if mod else ["dweight", "dbias"])

    def f(x, branch, gate, p, s):
        (r, _), (y, _) = L.gated_norm_ref(x, branch, gate, p if mod else None, s if mod else None,
                                          None if mod else p, None if mod else s, kind, torch.float64)
        return (y * u.double()).sum() + (r * ur.double()).sum()

    xs = [t.double() for t in (x, branch, gate, *((scale, shift) if mod else (weight, bias)))]
    _check_slopes(f, xs, [(got[n], ref[n][1] + (ref[n][0] - near[n][0]).abs()) for n in names], g)


@pytest.mark.parametrize("masked", [False, True])
def test_cross_attend_slopes(masked):
    g = _gen(32)
    B, Nq, Nk, H, d = 2, 70, 90, 2, 64
    q, k, v, u = L.rand(g, B, Nq, H, d), L.rand(g, B, Nk, H, d), L.rand(g, B, Nk, H, d), L.rand(g, B, Nq, H, d)
    mask = torch.rand(B, Nk, generator=g, device="cuda") < 0.5 if masked else None
    out, lse = rola.cross_attend(q, k, v, key_mask=mask, return_lse=True)
    got = rola.cross_attend_backward(u, q, k, v, out, lse, key_mask=mask)
    ref = L.cross_backward_ref(u, q, k, v, out, lse, key_mask=mask)
    (o, _), (z, _) = L.cross_ref(q.double(), k.double(), v.double(), key_mask=mask)
    near = L.cross_backward_ref(u, q, k, v, o, z, key_mask=mask)     # at the exact out and lse
    _check_slopes(lambda q, k, v: (L.cross_ref(q, k, v, key_mask=mask)[0][0] * u.double()).sum(),
                  [t.double() for t in (q, k, v)],
                  [(got[n], ref[n][1] + (ref[n][0] - near[n][0]).abs()) for n in ("dq", "dk", "dv")], g)


# ---------------------------------------------------------------------------- together


class Block:
    """The attention half of a transformer block around RoLA: modulated norm, q, k, v, their norm
    and positions, RoLA, gated residual with the next norm, cross attention, gated residual with
    the norm of the feed-forward.  Projections are torch's."""

    def __init__(self, dtype, topk, g, B=2, grid=(2, 8, 9), H=2, d=64, Nk=77, r=16):
        self.B, self.N, self.H, self.d, self.grid = B, math.prod(grid), H, d, grid
        C = H * d
        self.plan = rola.Plan(B, H, self.N, d, r, topk, grid, dtype="f32" if dtype == F32 else "bf16")
        s = C ** -0.5
        self.wqkv, self.wo = L.rand(g, 3 * C, C, dtype=dtype, scale=s), L.rand(g, C, C, dtype=dtype, scale=s)
        self.wcq, self.wco = L.rand(g, C, C, dtype=dtype, scale=s), L.rand(g, C, C, dtype=dtype, scale=s)
        self.nq, self.nk, self.ncq = (L.rand(g, C, scale=0.1, shift=1.0) for _ in range(3))
        self.Wq, self.Wk = (L.rand(g, H, d, r, dtype=dtype, scale=d ** -0.5) for _ in range(2))
        self.gains = torch.zeros(H, device="cuda") if topk == 1.0 else torch.full((H,), 0.3, device="cuda")
        self.mod = L.rand(g, B, 5, C, scale=0.3)                   # scale, shift, gate; scale, shift of the last
        self.w3, self.b3 = L.rand(g, C, shift=1.0), L.rand(g, C)
        self.ke, self.ve = (L.rand(g, B, Nk, H, d, dtype=dtype) for _ in range(2))
        self.kv_len = torch.tensor([Nk, 31], dtype=torch.int32, device="cuda")
        self.dtype = dtype

    def heads(self, x):
        return x.view(self.B, -1, self.H, self.d)

    def forward(self, x):
        C, m = self.H * self.d, self.mod
        _, y1 = rola.gated_norm(x, scale=m[:, 0], shift=m[:, 1], y_dtype=self.dtype)
        qkv = (y1 @ self.wqkv.T).view(self.B, self.N, 3, self.H, self.d)
        q, k = rola.qk_norm_rope(qkv[:, :, 0], qkv[:, :, 1], self.nq, self.nk, grid=self.grid)
        v = qkv[:, :, 2].contiguous()
        a = self.plan.forward(q, k, v, self.Wq, self.Wk, self.gains)
        o1 = a.view(self.B, self.N, C) @ self.wo.T
        x1, y2 = rola.gated_norm(x, o1, m[:, 2], weight=self.w3, bias=self.b3)
        c0 = self.heads(y2 @ self.wcq.T)
        cq = rola.qk_norm_rope(c0, None, self.ncq, rope=False)
        ca, lse = rola.cross_attend(cq, self.ke, self.ve, kv_len=self.kv_len, return_lse=True)
        o2 = ca.view(self.B, self.N, C) @ self.wco.T
        x2, y3 = rola.gated_norm(x1, o2, None, m[:, 3], m[:, 4])
        return x2, y3, (x, y1, qkv, q, k, v, o1, x1, y2, c0, cq, ca, lse, o2, x2)

    def backward(self, dx2, dy3, kept):
        """The gradient of x, and those of RoLA's q and k before the norm."""
        x, y1, qkv, q, k, v, o1, x1, y2, c0, cq, ca, lse, o2, x2 = kept
        m, t = self.mod, self.dtype
        g3 = rola.gated_norm_backward(dy3, x2, dx2, o2, None, m[:, 3])
        dca = self.heads(g3["dbranch"] @ self.wco)
        gc = rola.cross_attend_backward(dca, cq, self.ke, self.ve, ca, lse, kv_len=self.kv_len)
        dc0 = rola.qk_norm_rope_backward(gc["dq"], None, c0, None, self.ncq, rope=False)["dq"]
        dy2 = dc0.view(self.B, self.N, -1) @ self.wcq
        g2 = rola.gated_norm_backward(dy2, x1, g3["dx"], o1, m[:, 2], None, self.w3)
        da = self.heads(g2["dbranch"] @ self.wo)
        ga = self.plan.backward(q, k, v, self.Wq, self.Wk, self.gains, da)
        gr = rola.qk_norm_rope_backward(ga["dq"], ga["dk"], qkv[:, :, 0], qkv[:, :, 1], self.nq, self.nk, grid=self.grid)
        dqkv = torch.stack((gr["dq"], gr["dk"], ga["dv"].to(t)), 2)
        dy1 = dqkv.view(self.B, self.N, -1) @ self.wqkv
        return rola.gated_norm_backward(dy1, x, g2["dx"], None, None, m[:, 0])["dx"], gr

    def plain(self, x):
        """x2 and y3 in fp64 for a RoLA that keeps all blocks and has no linear branch."""
        C, m = self.H * self.d, self.mod.double()
        w = {n: getattr(self, n).double() for n in ("wqkv", "wo", "wcq", "wco", "w3", "b3")}
        f64 = torch.float64
        _, (y1, _) = L.gated_norm_ref(x, None, None, m[:, 0], m[:, 1], None, None, "layer", f64)
        qkv = (y1 @ w["wqkv"].T).view(self.B, self.N, 3, self.H, self.d)
        a = L.angles(self.N, self.d, self.grid)
        q, k = (L.norm_rope_ref(qkv[:, :, i], n, "token", a)[0] for i, n in ((0, self.nq), (1, self.nk)))
        o1 = L.cross_ref(q, k, qkv[:, :, 2])[0][0].reshape(self.B, self.N, C) @ w["wo"].T
        (x1, _), (y2, _) = L.gated_norm_ref(x, o1, m[:, 2], None, None, w["w3"], w["b3"], "layer", f64)
        cq = L.norm_rope_ref(self.heads(y2 @ w["wcq"].T), self.ncq, "token", None)[0]
        o2 = L.cross_ref(cq, self.ke.double(), self.ve.double(), self.kv_len)[0][0].reshape(self.B, self.N, C) @ w["wco"].T
        (x2, _), (y3, _) = L.gated_norm_ref(x1, o2, None, m[:, 3], m[:, 4], None, None, "layer", f64)
        return x2, y3


def test_block_against_its_plain_form():
    """fp32, all blocks kept: results and the gradient's slope along itself.

    Tolerances: a stage's fp32 sums of n <= 288 terms are off by at most (n + 64) u < 2.2e-5 of
    their magnitudes, and there are eight stages in a row, each no more than doubling what comes
    in (the norms divide by a spread near 1): 8 * 2.2e-5 < 2e-4 of the root mean square.  RoLA's
    own gradients are held to 5e-5."""
    tf32 = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        g = _gen(40)
        blk = Block(F32, 1.0, g)
        x = L.rand(g, blk.B, blk.N, blk.H * blk.d)
        x2, y3, kept = blk.forward(x)
        for got, want in zip((x2, y3), blk.plain(x.double())):
            rms = float(want.square().mean().sqrt())
            assert float((got.double() - want).square().mean().sqrt()) <= 2e-4 * rms
        u2, u3 = L.rand(g, *x.shape), L.rand(g, *x.shape)
        dx, _ = blk.backward(u2, u3, kept)
        size = float(dx.double().norm())

        def f(x):
            a, b = blk.plain(x)
            return (a * u2.double()).sum() + (b * u3.double()).sum()

        for v in (dx.double() / size, torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)):
            got, want = float((dx.double() * v).sum()), float(_slope(f, [x.double()], [v], 1e-3))
            assert abs(got - want) <= 2e-4 * size * max(1.0, float(v.norm()) / math.sqrt(v.numel())), (got, want)
        assert blk.plan.poll_status() == 0
    finally:
        torch.backends.cuda.matmul.allow_tf32 = tf32


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_block_captured(dtype):
    """Forward and backward of the block in one graph: the bits of the eager calls, again and again."""
    g = _gen(41)
    blk = Block(dtype, 0.5, g)
    x = L.rand(g, blk.B, blk.N, blk.H * blk.d)
    u2, u3 = L.rand(g, *x.shape), L.rand(g, *x.shape, dtype=dtype)

    def step():
        x2, y3, kept = blk.forward(x)
        dx, gr = blk.backward(u2, u3, kept)
        return [x2, y3, dx, *gr.values()]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step()
    for _ in range(3):
        for t in res:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(res, want)
    assert all(bool(torch.isfinite(t).all()) for t in want)
    assert blk.plan.poll_status() == 0
