"""Routing by scores at the edges of its arguments, against the 64-bit formulas of test_block_gpu.

u = 2^-24 is half a step of float32.
"""
import pytest
import torch

from test_block_gpu import U, check, gen, randn, ref_route, ref_route_grad, ref_scores, ref_weights, run_route

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def m():
    import sparse_expert_ffn_layer_gb300 as mod
    return mod


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E", [48, 256])
@pytest.mark.parametrize("G,top,gt", [(1, 1, 1), (4, 1, 1), (4, 2, 1), (4, 2, 2), (4, 3, 1), (4, 3, 2), (16, 1, 1), (16, 5, 2)])
@pytest.mark.parametrize("alike", [False, True])
def test_experts_that_are_always_taken(m, sigmoid, E, G, top, gt, alike):
    """A bias of +infinity; alike: groups of the same logits in another order, so that 64 bits decide between the others."""
    g = gen(E + G + top)
    T, M = 130, E // G
    k = min(6, top * M)
    x = randn(g, T, E, sigma=1.5)
    if alike:
        x = x[:, None, :M].repeat(1, G, 1).gather(2, torch.rand((T, G, M), generator=g, device="cuda").argsort(2))
        x = x.reshape(T, E).contiguous()
    for forced in ([E - 1], [M - 1, 0], [E // 2, E // 2 + 1, E - 2], [3]):
        bias = torch.full((E,), 0.25, device="cuda")
        bias[forced] = INF
        idx, w, _ = run_route(m, x, k, sigmoid, bias, None, G, top, gt)
        want = ref_route(x, k, sigmoid, bias, G, top, gt)
        assert torch.equal(idx.long(), want), forced
        if len({e // M for e in forced}) <= top:
            taken = sorted(forced)[:k]
            assert (idx[:, :len(taken)].long() == torch.tensor(taken, device="cuda")).all()
        ww = ref_weights(x, want, sigmoid, True, 1.0)
        # as in test_route
        check(w, ww, 70 * U * ww + 1e-37, "topk_w")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E", [48, 256])
def test_an_expert_that_is_always_taken_in_a_group_of_none_other(m, sigmoid, E):
    """The rest of its group switched off, groups by the sum of two: +infinity decides the group."""
    g = gen(E)
    T, G, top, k = 40, 4, 2, 4
    M = E // G
    x = randn(g, T, E)
    bias = torch.zeros(E, device="cuda")
    bias[M:2 * M] = -INF
    bias[M + 5] = INF
    idx, _, _ = run_route(m, x, k, sigmoid, bias, None, G, top, 2)
    other = x.double() if not sigmoid else ref_scores(x, True)
    s = ref_scores(x, sigmoid)
    value = s.view(T, G, M).topk(2, 2).values.sum(2)
    value[:, 1] = -1.0
    best = value.argmax(1, keepdim=True)
    off = torch.arange(E, device="cuda")[None, :] // M != best
    rest = other.masked_fill(off, -INF).sort(dim=1, descending=True, stable=True).indices[:, :k - 1]
    assert (idx[:, 0] == M + 5).all() and torch.equal(idx[:, 1:].long(), rest)


@pytest.mark.parametrize("T,E,k", [(64, 16, 4), (200, 64, 6), (33, 250, 16), (40, 600, 8)])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("offset", [-1000.0, 200.0, 1000.0, 10000.0])
def test_gradient_with_an_offset_of_all_logits(m, T, E, k, renorm, offset):
    """The softmax does not know of it: nothing may be lost by it."""
    g = gen(T + E)
    x = randn(g, T, E, sigma=2.0) + offset
    idx = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    dw, ds = randn(g, T, k), randn(g, T, E)
    for parts in (dict(dtopk_w=dw), dict(dtopk_w=dw, dscores=ds)):
        dl = torch.full((T, E), float("nan"), device="cuda")
        m.moe_route_backward(x, idx, dl, renormalize=renorm, scale=1.5, **parts)
        want, mag = ref_route_grad(x, idx, None, dw, parts.get("dscores"), False, renorm, 1.5)
        # as in test_route_gradient
        check(dl, want, 128 * U * mag + 2.0 ** -47 * mag.sum(1, keepdim=True) + 1e-37, "dlogits")


def test_order_of_scores_that_are_one(m):
    """Logits whose sigmoid is one in 64 bits: by the logits, or by the index where choices are added for groups."""
    x = torch.full((3, 16), -1.0, device="cuda")
    x[:, 2], x[:, 3], x[:, 9] = 40.0, 50.0, 45.0
    assert (run_route(m, x, 3, True)[0].long() == torch.tensor([3, 9, 2], device="cuda")).all()
    assert (run_route(m, x, 3, True, G=4, top=2, gt=1)[0].long() == torch.tensor([3, 9, 2], device="cuda")).all()
    assert (run_route(m, x, 3, True, G=4, top=2, gt=2)[0].long() == torch.tensor([2, 3, 9], device="cuda")).all()
    assert (run_route(m, x, 3, True, bias=torch.zeros(16, device="cuda"))[0].long() == torch.tensor([2, 3, 9], device="cuda")).all()
