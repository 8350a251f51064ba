"""The operators around RoLA at the edges of what they accept: as many tokens as an index of 31
bits holds, and calls from several host threads at once."""
import math
import threading

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
    torch.cuda.empty_cache()                  # tests in other processes follow


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _room(nbytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < nbytes + (8 << 30):
        pytest.skip(f"needs {nbytes >> 30} GB free")


@pytest.mark.parametrize("T,N", [(1, 2 ** 31 - 1), (2, 2 ** 31 - 2)])
def test_gated_norm_of_the_most_tokens(T, N):
    """Every row of 2^31 - 1 is written, and the last ones as they are alone."""
    C, tail = 8, 1_500_000                   # several of the runs that a group of warps takes
    _room(3 * 2 * N * C + (1 << 32))
    g = _gen(60)
    x = torch.empty(1, N, C, dtype=BF16, device="cuda")
    x.normal_(generator=g)
    scale, shift = L.rand(g, 1, T, C, scale=0.5), L.rand(g, 1, T, C, scale=0.5)
    last = dict(scale=scale[:, -1], shift=shift[:, -1])
    y = torch.full_like(x, math.nan)
    rola.gated_norm(x, scale=scale, shift=shift, out=(None, y))
    xt = x[:, -tail:].contiguous()
    want = rola.gated_norm(xt, **last)[1]
    assert torch.equal(y[:, -tail:], want)
    assert not any(bool(torch.isnan(part).any()) for part in y[0].split(1 << 26))
    del want
    res = rola.gated_norm_backward(y, x, scale=scale)
    want = rola.gated_norm_backward(y[:, -tail:].contiguous(), xt, scale=last["scale"])
    assert torch.equal(res["dx"][:, -tail:], want["dx"])
    # the sum of dy over a run, from sums of pieces (each within its own roundings)
    parts = [p.double().sum(0) for p in y[0, N // T * (T - 1):].split(1 << 24)]
    size = [p.double().abs().sum(0) for p in y[0, N // T * (T - 1):].split(1 << 24)]
    # a thread adds its rows of a run one by one: depth <= 2^31 / 592 groups + the tree above
    tol = (2 ** 31 / 592 + 64) * L.U * torch.stack(size).sum(0)
    L.assert_within(res["dshift"][0, -1], torch.stack(parts).sum(0), tol, "dshift")


def _two_widths(name):
    """Two calls of one operator that run the same kernel on rows of different widths."""
    g = _gen(61)

    def rope(H, back):
        x, w = L.rand(g, 1, 3, H, 128), L.rand(g, H * 128, shift=1.0)
        if back:
            return lambda: list(t for t in rola.qk_norm_rope_backward(x, None, x, None, w).values() if t is not None)
        return lambda: [rola.qk_norm_rope(x, None, w)]

    def norm(C, back):
        x, b, m = L.rand(g, 1, 3, C), L.rand(g, 1, 3, C), L.rand(g, 1, C)
        if back:
            return lambda: [t for t in rola.gated_norm_backward(x, x, b, b, m).values() if t is not None]
        return lambda: list(rola.gated_norm(x, b, m))

    make = rope if name.startswith("rope") else norm
    wide, narrow = (64, 40) if make is rope else (8192, 5136)
    return make(wide, name.endswith("backward")), make(narrow, name.endswith("backward"))


@pytest.mark.parametrize("name", ["rope", "rope backward", "norm", "norm backward"])
def test_two_host_threads(name):
    """Calls that need different amounts of shared memory of one kernel, from two threads at once:
    neither takes from the other what its launch needs."""
    calls = _two_widths(name)
    want = [c() for c in calls]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(2), []

    def work(call, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait(60)
                for i in range(4000):
                    got = call()
                    if i % 500 == 0:
                        torch.cuda.current_stream().synchronize()
                        assert all(torch.equal(a, b) for a, b in zip(got, want))
                torch.cuda.current_stream().synchronize()
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_widest_rows_beside_a_large_table():
    """8192 fp32 channels with close to 4096 angles in shared memory: all that a block may take."""
    g = _gen(62)
    N, H, d, grid, pairs = 9920, 64, 128, (10, 16, 62), (1, 1, 62)
    x, u, w = L.rand(g, 1, N, H, d), L.rand(g, 1, N, H, d), L.rand(g, H * d, shift=1.0)
    a = L.angles(N, d, grid, pairs=pairs)
    got = rola.qk_norm_rope(x, None, w, grid=grid, pairs=pairs)
    L.assert_within(got, *L.norm_rope_ref(x, w, "token", a), "y")
    got = rola.qk_norm_rope_backward(u, None, x, None, w, grid=grid, pairs=pairs)
    dx, dxe, dw, dwe = L.norm_rope_backward_ref(u, x, w, "token", a)
    L.assert_within(got["dq"], dx, dxe, "dq")
    L.assert_within(got["dwq"], dw, dwe, "dwq")


@pytest.mark.parametrize("layout", ["token", "head", "sample", "heads first", "between heads first"])
def test_parts_of_one_tensor_in_place(layout):
    """q and k side by side in a token, in a head, in a sample, with the heads outside the tokens:
    they share no element and may both be worked on in place, and what lies between stays."""
    g = _gen(63)
    B, N, H, d = 2, 23, 3, 64
    shape, q, k, perm = {
        "token": ((B, N, 3, H, d), (slice(None), slice(None), 0), (slice(None), slice(None), 2), (0, 1, 2, 3)),
        "head": ((B, N, H, 3, d), (..., 0, slice(None)), (..., 1, slice(None)), (0, 1, 2, 3)),
        "sample": ((B, 2, N, H, d), (slice(None), 1), (slice(None), 0), (0, 1, 2, 3)),
        "heads first": ((B, 3, H, N, d), (slice(None), 0), (slice(None), 2), (0, 2, 1, 3)),
        "between heads first": ((B, H, 2, N, d), (slice(None), slice(None), 1), (slice(None), slice(None), 0), (0, 2, 1, 3)),
    }[layout]
    x = L.rand(g, *shape, dtype=BF16)
    wq, wk = L.rand(g, H * d, shift=1.0), L.rand(g, H * d, shift=1.0)
    qv, kv = x[q].permute(perm), x[k].permute(perm)
    want = rola.qk_norm_rope(qv.contiguous(), kv.contiguous(), wq, wk)
    rest = x.clone()
    rola.qk_norm_rope(qv, kv, wq, wk, out=(qv, kv))
    assert torch.equal(qv, want[0]) and torch.equal(kv, want[1])
    for part in (x, rest):
        part[q], part[k] = 0, 0
    assert torch.equal(x, rest)


@pytest.mark.parametrize("dtype,grad", [(F32, F32), (BF16, BF16), (BF16, F32)])
def test_rotation_backward_takes_its_type_from_either(dtype, grad):
    g = _gen(64)
    x, u, v = (L.rand(g, 2, 30, 2, 64, dtype=t) for t in (dtype, grad, grad))
    want = rola.qk_norm_rope_backward(u, v, x, x, norm="none")
    for how in (dict(q=x), dict(k=x), {}):
        got = rola.qk_norm_rope_backward(u, v, **how, norm="none")
        for n in ("dq", "dk"):
            assert got[n].dtype == (dtype if how else grad) and torch.equal(got[n].to(dtype), want[n])


def test_calls_with_missing_parts_are_refused():
    """Each with the rest in order: RolaError, before anything is launched."""
    g = _gen(65)
    q, k, w = L.rand(g, 1, 5, 2, 64), L.rand(g, 1, 7, 2, 64), torch.ones(128, device="cuda")
    x = L.rand(g, 1, 5, 128)
    out, lse = rola.cross_attend(q, k, k, return_lse=True)
    y = torch.empty_like
    for call in (lambda: rola.cross_attend_backward(None, q, k, k, out, lse),
                 lambda: rola.cross_attend_backward(out, q, k, k, None, lse),
                 lambda: rola.cross_attend_backward(out, q, k, k, out, None),
                 lambda: rola.cross_attend(q, k, k, out="out"),
                 lambda: rola.cross_attend(q, k, k, stream="stream"),
                 lambda: rola.qk_norm_rope(q, None, w, out=(y(q),)),
                 lambda: rola.qk_norm_rope(q, None, w, out=(y(q), y(q))),
                 lambda: rola.qk_norm_rope(q, q, w, w, out=(y(q), None)),
                 lambda: rola.qk_norm_rope(q, q, w, w, out=y(q)),
                 lambda: rola.qk_norm_rope(q, None, w, out=3),
                 lambda: rola.gated_norm(x, weight=w, out=(None, None)),
                 lambda: rola.gated_norm(x, weight=w, out=y(x)),
                 lambda: rola.gated_norm(x, x, weight=w, out=(None, y(x))),
                 lambda: rola.gated_norm(x, weight=w, out=(None, y(x), None)),
                 lambda: rola.gated_norm(x, weight=w, out=(None, "y"))):
        with pytest.raises(rola.RolaError):
            call()


@pytest.mark.parametrize("x,y", [(F32, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("C", [888, 904, 1784, 1800, 4096, 4104, 5120, 5128, 6144, 6152, 8184, 8192])
def test_gated_norm_on_both_sides_of_every_variant(C, x, y):
    """Widths where the pieces of a thread, the rows in flight or a block's threads change."""
    g = _gen(66)
    B, N = 2, 7
    r, dr, branch = L.rand(g, B, N, C, dtype=x), L.rand(g, B, N, C, dtype=x), L.rand(g, B, N, C, dtype=y)
    dy, (gate, scale, shift) = L.rand(g, B, N, C, dtype=y), L.rand(g, B, 3, C, scale=0.5).unbind(1)
    for b in (None, branch):
        gb = None if b is None else gate
        wr, wy = L.gated_norm_ref(r, b, gb, scale, shift, None, None, "layer", y)
        res = rola.gated_norm(r, b, gb, scale, shift, y_dtype=y)
        L.assert_within(res[0], *wr, "r")
        L.assert_within(res[1], *wy, "y")
        for up in (None, dr):
            got = rola.gated_norm_backward(dy, r, up, b, gb, scale)
            for n, want in L.gated_norm_backward_ref(dy, r, up, b, gb, scale, None, "layer").items():
                L.assert_within(got[n], *want, n)


@pytest.mark.parametrize("Nq,Nk,d", [(500, 512, 128), (700, 333, 64)])
def test_what_bf16_probabilities_cost(Nq, Nk, d):
    """The rms error that rola.h states.  A rounding to bf16 is uniform within 2^-8 / m of a value
    with mantissa m; for mantissas spread evenly over their logarithm E[1 / m^2] = 3 / (8 ln 2), so
    its rms is e = 2^-8 (1 / 3 * 3 / (8 ln 2))^(1/2) = 0.00166 of the values'.  Against v and dout
    of independent signs the roundings of P (and of dS) add up like the terms that they round:
    another e.  dq and dk see the rounding of `out` in D too, which is no larger than dS: at most
    three e's in squares.  A tenth is left for mantissas that are not spread so."""
    e = 2.0 ** -8 * (1 / (8 * math.log(2))) ** 0.5
    g = _gen(67)
    q, k = (L.rand(g, 2, n, 4, d, dtype=BF16, scale=s) for n, s in ((Nq, 1.5), (Nk, 1.2)))
    v, dout = L.rand(g, 2, Nk, 4, d, dtype=BF16), L.rand(g, 2, Nq, 4, d, dtype=BF16)

    def off(got, want):
        return float((got.double() - want).norm() / want.norm())

    out, lse = rola.cross_attend(q, k, v, return_lse=True)
    (want, _), (z, _) = L.cross_ref(q, k, v)
    assert off(out, want) <= 1.1 * 2 ** 0.5 * e
    got = rola.cross_attend_backward(dout, q, k, v, out, lse)
    ref = L.cross_backward_ref(dout, q, k, v, want, z)
    for n, squares in (("dq", 3), ("dk", 3), ("dv", 2)):
        assert off(got[n], ref[n][0]) <= 1.1 * squares ** 0.5 * e, n


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_past_the_range_of_the_sums(dtype):
    """Up to a sum of squares of 0.9 of the largest fp32 rows come out as any others; past it they
    are zeros or not finite, and the rows beside them keep their bits."""
    g = _gen(68)
    N, H, d = 6, 4, 128
    top, big = torch.finfo(F32).max, torch.finfo(dtype).max
    x, w = L.rand(g, 1, N, H, d, dtype=dtype), L.rand(g, H * d, scale=0.1, shift=1.0)
    x[0, 1] *= (0.9 * top / float(x[0, 1].double().square().sum())) ** 0.5
    x[0, 3], x[0, 5] = 1e19, big
    u = L.rand(g, 1, N, H, d, dtype=dtype)
    rest = x.clone()
    rest[0, [3, 5]] = 1.0
    flat, flat_rest, flat_u = (t.view(1, N, H * d) for t in (x, rest, u))
    for f in (lambda x, y: rola.qk_norm_rope(x, None, w), lambda x, y: rola.gated_norm(y, weight=w, norm="rms")[1],
              lambda x, y: rola.qk_norm_rope_backward(u, None, x, None, w)["dq"],
              lambda x, y: rola.gated_norm_backward(flat_u, y, weight=w, norm="rms")["dx"]):
        got, want = f(x, flat)[0], f(rest, flat_rest)[0]
        assert torch.equal(got[[0, 1, 2, 4]], want[[0, 1, 2, 4]])
        assert not bool((torch.isfinite(got[[3, 5]]) & (got[[3, 5]] != 0)).any())
    y, bound = L.norm_rope_ref(x, w, "token", L.angles(N, d))
    L.assert_within(rola.qk_norm_rope(x, None, w)[:, :3], y[:, :3], bound[:, :3], "y")
