"""The operators around RoLA at the edges of what they accept: as many tokens as an index of 31
bits holds, and calls from several host threads at once."""
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
