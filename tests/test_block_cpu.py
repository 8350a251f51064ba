"""Refusals of the operators around RoLA, which need no GPU: every call here breaks one rule of
include/rola.h and must come back with its code before anything is launched.  Addresses are made
up; no call that the checks let through is made with them (the complete calls below lack their
workspace, which is checked after every argument and before the launch)."""
import ctypes

import pytest
import torch

import sparse_rank_attention_b200 as rola
from sparse_rank_attention_b200 import block
from sparse_rank_attention_b200 import build as rbuild

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
F32, BF16, FP8 = (rola.DTYPES[n] for n in ("f32", "bf16", "fp8"))
A = 1 << 30                                             # a fake address; regions lie GAP apart
GAP = 1 << 28


@pytest.fixture(scope="module", autouse=True)
def _built():
    rbuild.build()


def at(i, off=0):
    return A + i * GAP + off


def strides(n, H, d):
    return (ctypes.c_int64 * 3)(n * H * d, H * d, d)


# ---------------------------------------------------------------------------- parameters


def rope_params(**kw):
    p = block.RolaNormRopeParams()
    assert rola.load().rola_norm_rope_params_default(ctypes.byref(p)) == 0
    p.B, p.N, p.H, p.d, p.grid_w = 2, 30, 3, 64, 30
    for n in ("q", "k", "dq_out", "dk_out"):
        setattr(p, n, strides(30, 3, 64))
    for n, v in kw.items():
        setattr(p, n, v)
    return p


def norm_params(**kw):
    p = block.RolaGatedNormParams()
    p.B, p.N, p.C, p.T, p.x_dtype, p.y_dtype, p.norm, p.eps = 2, 30, 64, 1, F32, BF16, 0, 1e-6
    p.gate_b = p.scale_b = p.shift_b = p.gate_t = p.scale_t = p.shift_t = 64
    for n, v in kw.items():
        setattr(p, n, v)
    return p


def cross_params(**kw):
    p = block.RolaCrossParams()
    p.B, p.Nq, p.Nk, p.H, p.d, p.dtype = 2, 30, 2000, 3, 64, BF16   # few queries: the keys are split
    p.q, p.dout, p.k, p.v = strides(30, 3, 64), strides(30, 3, 64), strides(2000, 3, 64), strides(2000, 3, 64)
    for n, v in kw.items():
        setattr(p, n, v)
    return p


def size(fn, p):
    n = ctypes.c_size_t()
    return getattr(rola.load(), fn)(ctypes.byref(p), ctypes.byref(n)), n.value


def test_defaults():
    p = block.RolaNormRopeParams()
    assert rola.load().rola_norm_rope_params_default(ctypes.byref(p)) == 0
    assert (p.B, p.N, p.H, p.d, p.dtype, p.norm, p.pos, p.rope_base) == (1, 1, 1, 128, BF16, 1, 1, 10000.0)
    assert rola.load().rola_norm_rope_params_default(None) == INVALID


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(d=96), UNSUPPORTED), (dict(H=129), UNSUPPORTED), (dict(B=65536), UNSUPPORTED), (dict(N=0), INVALID),
    (dict(B=0), INVALID), (dict(H=-1), INVALID), (dict(dtype=7), INVALID), (dict(dtype=FP8), UNSUPPORTED),
    (dict(grad_dtype=F32), 0), (dict(dtype=F32), UNSUPPORTED), (dict(norm=3), INVALID), (dict(pos=-1), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(grid_w=31), INVALID), (dict(grid_h=0), INVALID), (dict(grid_t=65536, grid_h=65536), INVALID),
    (dict(rope_base=1.0), INVALID), (dict(rope_base=float("nan")), INVALID), (dict(rope_pairs_t=1), INVALID),
    (dict(rope_pairs_t=-1, rope_pairs_h=33), INVALID), (dict(pos=0, rope_base=0.0, grid_w=0), 0),
    (dict(pos=2, positions_batched=2), INVALID), (dict(N=1 << 30), UNSUPPORTED),
])
def test_rope_params(kw, code):
    got, need = size("rola_qk_norm_rope_workspace_size", rope_params(**kw))
    assert got == code
    if code == 0:
        assert need > 0 and need % 16 == 0


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(C=12), UNSUPPORTED), (dict(C=8200), UNSUPPORTED), (dict(C=0), INVALID), (dict(T=7), INVALID),
    (dict(T=30), 0), (dict(T=0), INVALID), (dict(x_dtype=BF16), 0), (dict(x_dtype=BF16, y_dtype=F32), UNSUPPORTED),
    (dict(y_dtype=FP8), UNSUPPORTED), (dict(x_dtype=9), INVALID), (dict(norm=2), INVALID), (dict(eps=-0.5), INVALID),
    (dict(N=1 << 30), UNSUPPORTED),
])
def test_gated_norm_params(kw, code):
    assert size("rola_gated_norm_workspace_size", norm_params(**kw))[0] == code


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(d=32), UNSUPPORTED), (dict(Nk=0), INVALID), (dict(Nq=0), INVALID), (dict(H=513), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(dtype=FP8), UNSUPPORTED), (dict(dtype=5), INVALID), (dict(dtype=F32), 0),
    (dict(softmax_scale=-1.0), INVALID), (dict(softmax_scale=float("nan")), INVALID),
    (dict(softmax_scale=float("inf")), INVALID), (dict(Nq=1 << 30), UNSUPPORTED), (dict(Nk=1 << 30), UNSUPPORTED),
])
def test_cross_params(kw, code):
    for fn in ("rola_cross_workspace_size", "rola_cross_backward_workspace_size"):
        assert size(fn, cross_params(**kw))[0] == code


def test_sizes_want_a_place():
    for fn, p in (("rola_qk_norm_rope_workspace_size", rope_params()), ("rola_gated_norm_workspace_size", norm_params()),
                  ("rola_cross_workspace_size", cross_params()), ("rola_cross_backward_workspace_size", cross_params())):
        assert getattr(rola.load(), fn)(ctypes.byref(p), None) == INVALID
        n = ctypes.c_size_t()
        assert getattr(rola.load(), fn)(None, ctypes.byref(n)) == INVALID


# ---------------------------------------------------------------------------- arguments

ROPE = dict(q=at(0), k=at(1), wq=at(2), wk=at(3), positions=None, q_out=at(4), k_out=at(5))
ROPE_BACK = dict(dq_out=at(0), dk_out=at(1), q=at(2), k=at(3), wq=at(4), wk=at(5), positions=None, dq=at(6),
                 dk=at(7), dwq=at(8), dwk=at(9), ws=None, n=0)
NORM = dict(x=at(0), branch=at(1), gate=at(2), scale=at(3), shift=at(4), weight=None, bias=None, r=at(7), y=at(8))
NORM_BACK = dict(dy=at(0), dr=at(1), r=at(2), branch=at(3), gate=at(4), scale=at(5), weight=None, dx=at(7),
                 dbranch=at(8), dgate=at(9), dscale=at(10), dshift=at(11), dweight=None, dbias=None, ws=None, n=0)
CROSS = dict(q=at(0), k=at(1), v=at(2), kv_len=at(3, 4), key_mask=at(4, 1), out=at(5), lse=at(6, 4), ws=None, n=0)
CROSS_BACK = dict(dout=at(0), q=at(1), k=at(2), v=at(3), out=at(4), lse=at(5, 4), kv_len=at(6, 4), key_mask=at(7, 1),
                  dq=at(8), dk=at(9), dv=at(10), ws=None, n=0)


def call(fn, p, base, kw):
    args = {**base, **kw}
    assert set(args) == set(base)
    args["stream"] = None
    return getattr(rola.load(), fn)(ctypes.byref(p), *args.values())


@pytest.mark.parametrize("fn,p,base", [
    ("rola_qk_norm_rope_backward", rope_params, ROPE_BACK), ("rola_gated_norm_backward", norm_params, NORM_BACK),
    ("rola_cross_attend", cross_params, CROSS), ("rola_cross_attend_backward", cross_params, CROSS_BACK)])
def test_complete_calls_lack_only_the_workspace(fn, p, base):
    assert call(fn, p(), base, {}) == WORKSPACE
    assert call(fn, p(), base, dict(ws=at(15), n=16)) == WORKSPACE            # too small
    assert call(fn, p(), base, dict(ws=at(15, 8), n=1 << 27)) == WORKSPACE    # not 16-byte aligned


S = strides(30, 3, 64)
BAD_STRIDES = [(30 * 192, 192, 4), (30 * 192, 192, 0), (30 * 192, 196, 64), (-192, 192, 64), (30 * 192, 1 << 40, 64)]


@pytest.mark.parametrize("pk,kw", [
    ({}, dict(q=None)), ({}, dict(q_out=None)), ({}, dict(k_out=None)), ({}, dict(k=None)), ({}, dict(wq=None)),
    ({}, dict(wk=None)), ({}, dict(positions=at(9))), (dict(pos=2), {}), (dict(pos=2), dict(positions=at(9, 2))),
    (dict(norm=0), {}), ({}, dict(q=at(0, 8))), ({}, dict(k_out=at(5, 4))), ({}, dict(wk=at(3, 4))),
    ({}, dict(q_out=at(0, 16))), ({}, dict(q_out=at(1))), ({}, dict(k_out=at(4, 2 * 30 * 192))),
    ({}, dict(q_out=at(2))), (dict(pos=2), dict(positions=at(4))), ({}, dict(q_out=at(1), k_out=at(0))),
    # in place, where two elements share memory
    (dict(q=(ctypes.c_int64 * 3)(192, 192, 64)), dict(q_out=at(0))),
] + [(dict(q=(ctypes.c_int64 * 3)(*s)), {}) for s in BAD_STRIDES])
def test_rope_refuses(pk, kw):
    assert call("rola_qk_norm_rope", rope_params(**pk), ROPE, kw) == INVALID


@pytest.mark.parametrize("pk,kw", [
    ({}, dict(dq_out=None)), ({}, dict(dq=None)), ({}, dict(dk=None)), ({}, dict(q=None)), ({}, dict(k=None)),
    ({}, dict(wq=None)), ({}, dict(dwk=None)), (dict(norm=0), {}), ({}, dict(dq=at(2))), ({}, dict(dwq=at(9))),
    ({}, dict(dwq=at(4))), ({}, dict(dq=at(0, 32))), ({}, dict(dk=at(0))), ({}, dict(dq=at(6, 8))),
    (dict(grad_dtype=F32), dict(dq=at(0))),            # in place, but of another type
    (dict(dq_out=(ctypes.c_int64 * 3)(30 * 384, 384, 64)), dict(dq=at(0))),   # in place, but strided
    (dict(dq_out=(ctypes.c_int64 * 3)(30 * 192, 0, 64)), {}),
    (dict(k=(ctypes.c_int64 * 3)(30 * 192, 200 + 4, 64)), {}),
])
def test_rope_backward_refuses(pk, kw):
    big = dict(ws=at(15), n=1 << 27, **kw)
    assert call("rola_qk_norm_rope_backward", rope_params(**pk), ROPE_BACK, big) == INVALID


@pytest.mark.parametrize("pk,kw", [
    ({}, dict(x=None)), ({}, dict(y=None)), ({}, dict(r=None)), ({}, dict(branch=None)),
    ({}, dict(branch=None, r=None)),                                        # a gate without a branch
    ({}, dict(shift=None)), ({}, dict(scale=None)), ({}, dict(weight=at(5))), ({}, dict(bias=at(6))),
    ({}, dict(scale=None, shift=None, bias=at(6))), ({}, dict(x=at(0, 4))), ({}, dict(gate=at(2, 4))),
    (dict(gate_b=-64), {}), (dict(scale_b=66), {}), ({}, dict(y=at(0))), ({}, dict(y=at(7))), ({}, dict(r=at(0, 32))),
    ({}, dict(y=at(1))), ({}, dict(r=at(1))), ({}, dict(y=at(3))), ({}, dict(r=at(4, -16))),
])
def test_gated_norm_refuses(pk, kw):
    assert call("rola_gated_norm", norm_params(**pk), NORM, kw) == INVALID


@pytest.mark.parametrize("pk,kw", [
    ({}, dict(dy=None)), ({}, dict(r=None)), ({}, dict(dx=None)), ({}, dict(dbranch=None)), ({}, dict(branch=None)),
    ({}, dict(dgate=None)), ({}, dict(gate=None)), ({}, dict(dscale=None)), ({}, dict(dshift=None)),
    ({}, dict(weight=at(6))), ({}, dict(dweight=at(12))), ({}, dict(dbias=at(12))), ({}, dict(dx=at(2))),
    ({}, dict(dx=at(1, 16))), ({}, dict(dbranch=at(0))), ({}, dict(dgate=at(4))), ({}, dict(dgate=at(10))),
    ({}, dict(dx=at(15))), ({}, dict(dy=at(15))), ({}, dict(dshift=at(11, 8))), (dict(gate_t=-4, T=2), {}),
])
def test_gated_norm_backward_refuses(pk, kw):
    big = dict(ws=at(15), n=1 << 27, **kw)
    assert call("rola_gated_norm_backward", norm_params(**pk), NORM_BACK, big) == INVALID


CROSS_BAD = [(dict(q=(ctypes.c_int64 * 3)(*s)), {}) for s in BAD_STRIDES] + [
    (dict(k=(ctypes.c_int64 * 3)(2000 * 192, 196, 64)), {}), (dict(v=(ctypes.c_int64 * 3)(2000 * 192, 0, 64)), {}),
    ({}, dict(q=None)), ({}, dict(k=None)), ({}, dict(v=None)), ({}, dict(out=None)), ({}, dict(k=at(1, 8))),
    ({}, dict(lse=at(6, 2))), ({}, dict(kv_len=at(3, 1)))]


@pytest.mark.parametrize("pk,kw", CROSS_BAD + [
    ({}, dict(out=at(0))), ({}, dict(out=at(2, 64))), ({}, dict(out=at(3))), ({}, dict(lse=at(5))),
    ({}, dict(lse=at(4))), ({}, dict(out=at(15))), ({}, dict(q=at(15)))])
def test_cross_refuses(pk, kw):
    assert call("rola_cross_attend", cross_params(**pk), CROSS, dict(ws=at(15), n=1 << 27, **kw)) == INVALID


@pytest.mark.parametrize("pk,kw", CROSS_BAD + [
    ({}, dict(lse=None)), ({}, dict(dout=None)), ({}, dict(dq=None)), ({}, dict(dv=None)), ({}, dict(dq=at(9))),
    ({}, dict(dk=at(2))), ({}, dict(dq=at(0))), ({}, dict(dv=at(15))), ({}, dict(dq=at(4))), ({}, dict(dq=at(5))),
    ({}, dict(dv=at(7))), (dict(dout=(ctypes.c_int64 * 3)(0, 0, 0)), {})])
def test_cross_backward_refuses(pk, kw):
    assert call("rola_cross_attend_backward", cross_params(**pk), CROSS_BACK, dict(ws=at(15), n=1 << 27, **kw)) == INVALID


# ---------------------------------------------------------------------------- the Python calls


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


Q, W = t(2, 30, 3, 64), t(192, dtype=torch.float32)
X, M = t(2, 30, 64, dtype=torch.float32), t(2, 64, dtype=torch.float32)
K = t(2, 50, 3, 64)


@pytest.mark.parametrize("make,text", [
    (lambda: rola.qk_norm_rope(Q, Q, W, W), "CUDA device"),
    (lambda: rola.qk_norm_rope(Q[0], None, W), "B, N, H, d"),
    (lambda: rola.qk_norm_rope(Q.half(), None, W), "not fp32 or bf16"),
    (lambda: rola.qk_norm_rope(Q, Q[:, :7], W, W), "differs from q"),
    (lambda: rola.qk_norm_rope(Q, Q.float(), W, W), "differs from q"),
    (lambda: rola.qk_norm_rope(Q, None, W[:64]), "wq is not"),
    (lambda: rola.qk_norm_rope(Q, None, W.bfloat16()), "wq is not"),
    (lambda: rola.qk_norm_rope(Q, None, W, norm="layer"), "norm"),
    (lambda: rola.qk_norm_rope(Q, None, W, norm="none"), "gains"),
    (lambda: rola.qk_norm_rope(Q, None, W, grid=(1, 2)), "grid"),
    (lambda: rola.qk_norm_rope(Q, None, W, grid=(1, 2, 2 ** 32 + 1)), "grid"),
    (lambda: rola.qk_norm_rope(Q, None, W, start=(0, 0, 2 ** 31)), "start"),
    (lambda: rola.qk_norm_rope(Q, None, W, pairs=(0.5, 0, 0)), "pairs"),
    (lambda: rola.qk_norm_rope(Q, None, W, positions=t(30, 3, dtype=torch.int64)), "positions"),
    (lambda: rola.qk_norm_rope(Q, None, W, grid=(1, 1, 30), positions=t(30, 3, dtype=torch.int32)), "grid"),
    (lambda: rola.qk_norm_rope(Q.transpose(2, 3), None, W), "channels"),
    (lambda: rola.qk_norm_rope_backward(Q, None, Q), "gains"),
    (lambda: rola.qk_norm_rope_backward(Q, Q, Q, None, W), "gains"),
    (lambda: rola.gated_norm(X), "CUDA device"),
    (lambda: rola.gated_norm(X[0]), "B, N, C"),
    (lambda: rola.gated_norm(X, X[:, :5]), "beside x"),
    (lambda: rola.gated_norm(X[:, ::2]), "contiguous"),
    (lambda: rola.gated_norm(X, None, None, M.bfloat16(), M), "scale is not"),
    (lambda: rola.gated_norm(X, None, None, M, M[:, None].expand(2, 5, 64)), "one T"),
    (lambda: rola.gated_norm(X, norm="head"), "norm"),
    (lambda: rola.gated_norm(X, weight=M), "weight"),
    (lambda: rola.gated_norm(X, y_dtype=torch.float16), "not fp32 or bf16"),
    (lambda: rola.gated_norm_backward(X, X, X.bfloat16()), "beside x"),
    (lambda: rola.cross_attend(Q, K, K), "CUDA device"),
    (lambda: rola.cross_attend(Q, K, K[:, :9]), "v is not"),
    (lambda: rola.cross_attend(Q, K[:, :, :1].expand(2, 50, 2, 64), K), "k is not"),
    (lambda: rola.cross_attend(Q, K.float(), K), "k is not"),
    (lambda: rola.cross_attend(Q, K, K, kv_len=t(2, dtype=torch.int64)), "kv_len"),
    (lambda: rola.cross_attend(Q, K, K, key_mask=t(2, 51, dtype=torch.bool)), "key_mask"),
    (lambda: rola.cross_attend(Q, K, K, key_mask=t(50, dtype=torch.bool).expand(2, 50)), "key_mask"),
    (lambda: rola.cross_attend(Q, K, K, out=K), "out is not"),
    (lambda: rola.cross_attend_backward(Q, Q, K, K, Q, t(2, 30, 3, dtype=torch.float32)), "lse"),
    (lambda: rola.cross_attend_backward(Q, Q, K, K, Q.transpose(0, 0)[:, ::2], None), "out is not"),
])
def test_python_calls_refuse(make, text):
    with pytest.raises(rola.RolaError) as e:
        make()
    assert text in str(e.value) and e.value.code in (INVALID, UNSUPPORTED)


# ---------------------------------------------------------------------------- sizes at the end of their range


@pytest.mark.parametrize("T", [1, 2])
def test_gated_norm_workspace_of_the_most_tokens(T):
    """2^31 - 1 tokens are cut into about as many runs as half of them."""
    most = size("rola_gated_norm_workspace_size", norm_params(B=1, N=2 ** 31 - T, C=8, T=T))
    half = size("rola_gated_norm_workspace_size", norm_params(B=1, N=2 ** 30, C=8, T=T))
    assert most[0] == half[0] == 0
    assert 0 < most[1] <= 2 * half[1] and half[1] <= 2 * most[1]


# ---------------------------------------------------------------------------- views that share memory


@pytest.mark.parametrize("B,N,H,s,gap", [
    (1, 4, 2, (0, 64, 320), 64),             # heads outside tokens: k one token on
    (1, 4, 2, (0, 64, 320), 192),
    (1, 5, 2, (0, 192, 128), 64),            # heads side by side, the last of a token on the next token's first
    (2, 2, 1, (256, 192, 64), 64),           # side by side in a token, its last on the next sample's first
    (2, 3, 2, (768, 256, 128), 768),         # k one sample on
    (2, 3, 2, (768, 256, 128), 256 + 32),    # half a head off
])
def test_rope_refuses_views_in_one_another(B, N, H, s, gap):
    """q and k in place, with elements of k on elements of q; gaps in elements."""
    st = (ctypes.c_int64 * 3)(*s)
    p = rope_params(B=B, N=N, H=H, grid_w=N, q=st, k=st)
    for k in (at(0, 2 * gap), at(0, -2 * gap)):
        assert call("rola_qk_norm_rope", p, ROPE, dict(k=k, q_out=at(0), k_out=k)) == INVALID


# ---------------------------------------------------------------------------- arguments that are left out


@pytest.mark.parametrize("make,text", [
    (lambda: rola.qk_norm_rope_backward(Q, Q, k=Q, norm="none"), "CUDA device"),       # all but the device
    (lambda: rola.qk_norm_rope_backward(Q.float(), Q.float(), k=Q, norm="none"), "CUDA device"),
    (lambda: rola.qk_norm_rope_backward(Q, None, k=Q, norm="none"), "CUDA device"),
    (lambda: rola.qk_norm_rope_backward(Q, Q, k=Q[:, :7], norm="none"), "differs from q"),
])
def test_rope_backward_without_q(make, text):
    with pytest.raises(rola.RolaError, match=text):
        make()


LSE = t(2, 3, 30, dtype=torch.float32)


@pytest.mark.parametrize("make,text", [
    (lambda: rola.qk_norm_rope(None, Q, W, W), "B, N, H, d"),
    (lambda: rola.qk_norm_rope([1.0], None, W), "a list in the place"),
    (lambda: rola.qk_norm_rope(Q, None, W.numpy()), "a ndarray in the place"),
    (lambda: rola.qk_norm_rope(Q.to_sparse(), None, W), "channels"),
    (lambda: rola.qk_norm_rope(Q, None, W, eps="small"), "eps is not a number"),
    (lambda: rola.qk_norm_rope(Q, None, W, rope_base=None), "rope_base is not a number"),
    (lambda: rola.qk_norm_rope_backward(None, Q, Q, Q, W, W), "no dq_out"),
    (lambda: rola.qk_norm_rope_backward(None, norm="none"), "no dq_out"),
    (lambda: rola.gated_norm(None, X), "no x"),
    (lambda: rola.gated_norm(X, eps=None), "eps is not a number"),
    (lambda: rola.gated_norm_backward(None, X), "no dy"),
    (lambda: rola.gated_norm_backward(X, None), "no r"),
    (lambda: rola.cross_attend(None, K, K), "missing"),
    (lambda: rola.cross_attend(Q, K, None), "missing"),
    (lambda: rola.cross_attend(Q, None, K), "missing"),
    (lambda: rola.cross_attend(Q, K, K, softmax_scale="1"[1:]), "softmax_scale is not a number"),
    (lambda: rola.cross_attend(Q, K, K, kv_len=50), "a int in the place"),
    (lambda: rola.cross_attend_backward(None, Q, K, K, Q, LSE), "CUDA device|missing"),
    (lambda: rola.cross_attend_backward(Q, Q, K, K, None, LSE), "CUDA device|missing"),
])
def test_python_calls_refuse_what_is_no_tensor(make, text):
    with pytest.raises(rola.RolaError, match=text) as e:
        make()
    assert e.value.code == INVALID


@pytest.mark.parametrize("kw", [dict(norm=1), dict(norm=2), dict(dtype=F32, grad_dtype=F32)])
def test_rope_workspace_of_the_most_tokens(kw):
    """A full grid of groups either way: the partial sums do not depend on the last tokens."""
    def need(N):
        return size("rola_qk_norm_rope_workspace_size", rope_params(B=1, N=N, H=1, d=64, pos=0, **kw))
    assert need(2 ** 31 - 1) == need(2 ** 30) and need(2 ** 30)[1] > 0


@pytest.mark.parametrize("n,code", [(2 ** 31 - 1, UNSUPPORTED), (2 ** 31 - 255, UNSUPPORTED), (2 ** 31 - 256, 0)])
def test_cross_of_the_most_tokens(n, code):
    """Tiles that would end past 2^31 are refused."""
    for fn in ("rola_cross_workspace_size", "rola_cross_backward_workspace_size"):
        for dtype in (F32, BF16):
            for kw in (dict(Nq=n, Nk=64), dict(Nq=64, Nk=n)):
                got, need = size(fn, cross_params(B=1, H=1, dtype=dtype, **kw))
                assert got == code and (code or need < 2 ** 50)


@pytest.mark.parametrize("fn,p,base,kw", [
    ("rola_qk_norm_rope", lambda: rope_params(B=1, N=1 << 29, q=(ctypes.c_int64 * 3)(0, 1 << 35, 64)), ROPE, {}),
    ("rola_qk_norm_rope_backward", lambda: rope_params(B=1, N=1 << 29, k=(ctypes.c_int64 * 3)(0, 1 << 35, 64)), ROPE_BACK,
     dict(ws=at(15), n=1 << 27)),
    ("rola_gated_norm", lambda: norm_params(gate_b=1 << 62), NORM, {}),
    ("rola_gated_norm", lambda: norm_params(B=1, T=30, shift_t=1 << 60), NORM, {}),
    ("rola_gated_norm_backward", lambda: norm_params(scale_b=1 << 50), NORM_BACK, dict(ws=at(15), n=1 << 27)),
    ("rola_cross_attend", lambda: cross_params(B=1, H=1, Nk=1 << 29, v=(ctypes.c_int64 * 3)(0, 1 << 35, 64)), CROSS,
     dict(ws=at(15), n=1 << 27)),
])
def test_strides_past_an_address_space(fn, p, base, kw):
    """Whose extents would wrap in 64 bits, and with them the checks against overlaps."""
    assert call(fn, p(), base, kw) == INVALID


@pytest.mark.parametrize("make,text", [
    (lambda x: rola.qk_norm_rope(Q, None, W, eps=x), "eps is not a number"),
    (lambda x: rola.qk_norm_rope(Q, None, W, rope_base=x), "rope_base is not a number"),
    (lambda x: rola.qk_norm_rope(Q, None, W, grid=(1, 1, x)), "grid"),
    (lambda x: rola.gated_norm(X, eps=x), "eps is not a number"),
    (lambda x: rola.cross_attend(Q, K, K, softmax_scale=x), "softmax_scale is not a number"),
])
def test_tensors_are_no_numbers(make, text):
    """Options are kept with the checks of a call; one whose value may change later is refused."""
    with pytest.raises(rola.RolaError, match=text):
        make(torch.tensor(2.0))
    with pytest.raises(rola.RolaError, match="CUDA device|grid"):
        make(2.0)


def test_numbers_of_every_kind():
    import numpy as np
    from fractions import Fraction
    for x in (1, np.float32(1e-6), np.float64(1e-6), np.int64(1), Fraction(1, 4)):
        assert block._number("call", "eps", x) == float(x)
    with pytest.raises(rola.RolaError):
        block._number("call", "eps", 10 ** 400)
