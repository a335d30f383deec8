"""A block of routed experts: routing by scores, experts in 8 bits and the norms around the block, against plain
64-bit formulas.

Tolerances.  u = 2^-24 is half a step of float32, h = eps / 2 the half step of the output type (2^-25: that of
f16's subnormals).  A sum of n float32 terms in any order is off by at most n u times the sum of their magnitudes;
the tensor cores' additions truncate, i.e. up to 2 u each.  Each check allows K u (sum of magnitudes) + h |value|
with K counted beside it.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NAN = float("nan")


@pytest.fixture(scope="module")
def m():
    import sparse_expert_ffn_layer_gb300 as mod
    return mod


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, sigma=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def check(got, want, tol, what):
    got, want, tol = got.double(), want.double(), tol.double() if torch.is_tensor(tol) else tol
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: finite values differ"
    err = torch.where(fin, (got - want).abs(), torch.zeros_like(want))
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {float(err.max()):.3e}"


def half(dtype):
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------- routing
def ref_scores(x, sigmoid):
    x = x.double()
    if sigmoid:
        return 1 / (1 + torch.exp(-x))
    empty = torch.isneginf(x).all(1, keepdim=True)
    return torch.softmax(torch.where(empty, torch.zeros_like(x), x), 1) * ~empty


def ref_route(x, k, sigmoid, bias, G, top, gt):
    """Experts by descending choice in 64 bits, ties to the lower index (one stable sort each)."""
    T, E = x.shape
    c = ref_scores(x, sigmoid)
    if bias is not None:
        c = c + bias.double()
    elif top == G or gt == 1 or E == G:
        c = x.double()                              # the same order, without the scores' rounding
    if top < G:
        v = c.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :gt].sum(2)
        best = v.sort(dim=1, descending=True, stable=True).indices[:, :top]
        off = torch.ones((T, G), dtype=torch.bool, device="cuda").scatter_(1, best, False)
        c = c.view(T, G, E // G).masked_fill(off[:, :, None], -float("inf")).reshape(T, E)
        # (masked experts stand behind those of -inf choice in a group that is in)
        order = torch.where(off[:, :, None].expand(T, G, E // G).reshape(T, E), 1, 0)
        idx = c.sort(dim=1, descending=True, stable=True).indices
        idx = idx.gather(1, order.gather(1, idx).sort(dim=1, stable=True).indices)
        return idx[:, :k]
    return c.sort(dim=1, descending=True, stable=True).indices[:, :k]


def ref_weights(x, idx, sigmoid, renorm, scale):
    s = ref_scores(x, sigmoid).gather(1, idx)
    if renorm:
        # in logarithms, so that scores that underflow keep their shares
        xi = x.double().gather(1, idx)
        l = -torch.nn.functional.softplus(-xi) if sigmoid else xi
        s = torch.softmax(torch.where(torch.isneginf(l).all(1, keepdim=True), torch.zeros_like(l), l), 1) \
            * ~torch.isneginf(l).all(1, keepdim=True)
    return s * scale


def run_route(m, x, k, sigmoid, bias=None, mask=None, G=1, top=1, gt=1, renorm=True, scale=1.0, scores=False):
    T, E = x.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), NAN, device="cuda")
    s = torch.full((T, E), NAN, device="cuda") if scores else None
    m.moe_route(None, None, k, idx, w, logits_in=x, bias=bias, token_mask=mask, score=int(sigmoid), n_groups=G,
                top_groups=top, group_top=gt, renormalize=renorm, scale=scale, scores_out=s)
    return idx, w, s


# T, E, k, groups, top_groups, group_top
ROUTES = [(1, 1, 1, 1, 1, 1), (3, 2, 2, 1, 1, 1), (1, 128, 2, 1, 1, 1), (77, 32, 4, 1, 1, 1), (50, 33, 16, 1, 1, 1),
          (129, 60, 6, 1, 1, 1), (65, 64, 8, 4, 2, 1), (300, 256, 8, 8, 4, 2), (41, 15, 5, 3, 2, 2), (20, 96, 3, 32, 7, 2),
          (33, 160, 6, 8, 3, 1), (9, 1024, 16, 16, 5, 2), (13, 1000, 7, 8, 8, 2), (17, 512, 9, 1, 1, 1), (5, 8, 4, 8, 4, 2),
          (7, 24, 12, 12, 6, 1), (2000, 128, 8, 4, 3, 2), (70001, 8, 2, 2, 1, 2)]


@pytest.mark.parametrize("T,E,k,G,top,gt", ROUTES)
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased,renorm,masked", [(False, True, False), (True, True, True), (True, False, False),
                                                  (False, False, True)])
def test_route(m, T, E, k, G, top, gt, sigmoid, biased, renorm, masked):
    g = gen(T * 7 + E + k)
    x = randn(g, T, E, sigma=2.0)
    bias = randn(g, E, sigma=0.1) if biased else None
    mask = (torch.rand(T, generator=g, device="cuda") < 0.8) if masked else None
    given = x.clone()
    if masked:
        given[~mask] = NAN                            # what masked rows hold has no effect
    idx, w, s = run_route(m, given, k, sigmoid, bias, mask, G, top, gt, renorm, 2.5, scores=True)
    on = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask
    want = ref_route(x, k, sigmoid, bias, G, top, gt)
    assert torch.equal(idx[on].long(), want[on]) and (idx[~on] == -1).all()
    # exp 4 u, |x - max| <= 20 costs the subtraction 20 u, a sum of 1024 terms in a tree of 32 + 5, a quotient, a
    # product and the scale: 64; renormalised: two exponentials and a sum of at most 16: less
    ww = ref_weights(x, want, sigmoid, renorm, 2.5) * on[:, None]
    check(w, ww, 70 * U * ww.abs() + 1e-37, "topk_w")
    ws = ref_scores(x, sigmoid) * on[:, None]
    check(s, ws, 70 * U * ws + 1e-37, "scores")
    i2, w2, _ = run_route(m, given, k, sigmoid, bias, mask, G, top, gt, renorm, 2.5)
    assert torch.equal(idx, i2) and torch.equal(w, w2)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("G,top,gt", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
def test_route_near_and_exact_ties(m, sigmoid, G, top, gt):
    """Choices that 32 bits cannot tell apart: the bias cancels the scores to about one rounding."""
    g = gen(5)
    T, E, k = 257, 64, 8
    x = randn(g, T, E)
    x[1:] = x[0]
    x[::3, 7] += 1e-6
    bias = (0.75 - ref_scores(x[:1], sigmoid)[0]).float()
    want = ref_route(x, k, sigmoid, bias, G, top, gt)
    assert torch.equal(run_route(m, x, k, sigmoid, bias, None, G, top, gt)[0].long(), want)
    # few distinct values: ties go to the lower index
    x = torch.randint(-2, 3, (T, E), generator=g, device="cuda").float()
    bias = torch.randint(0, 2, (E,), generator=g, device="cuda").float()
    for b in (None, bias):
        assert torch.equal(run_route(m, x, k, sigmoid, b, None, G, top, gt)[0].long(),
                           ref_route(x, k, sigmoid, b, G, top, gt))
    x = torch.zeros((3, E), device="cuda")
    x[1] = -0.0
    assert torch.equal(run_route(m, x, k, sigmoid, None, None, G, top, gt)[0].long(),
                       ref_route(x, k, sigmoid, None, G, top, gt))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,G,top,gt", [(256, 8, 4, 2), (256, 8, 3, 1), (60, 4, 2, 2), (15, 3, 1, 2), (96, 32, 7, 2),
                                        (128, 4, 2, 1), (1024, 16, 5, 2)])
def test_route_groups_that_hardly_differ(m, sigmoid, E, G, top, gt):
    """Every group holds the first one's logits in another order, some a rounding apart or equal: 64 bits decide."""
    g = gen(E + G)
    T, M, k = 301, E // G, min(5, top * (E // G))
    x = randn(g, T, 1, M, sigma=2.0).repeat(1, G, 1)
    x = x.gather(2, torch.rand((T, G, M), generator=g, device="cuda").argsort(2))
    x = x * (1 + 2.0 ** -23 * torch.randint(-1, 2, (T, G, M), generator=g, device="cuda"))
    x = x.reshape(T, E).float().contiguous()
    for bias in (None, torch.full((E,), 0.3, device="cuda"), randn(g, E, sigma=1e-7)):
        assert torch.equal(run_route(m, x, k, sigmoid, bias, None, G, top, gt)[0].long(),
                           ref_route(x, k, sigmoid, bias, G, top, gt))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_extremes(m, sigmoid, renorm):
    inf = float("inf")
    x = torch.tensor([[-inf, -inf, -inf, -inf, -inf, -inf], [-inf, 3.0, -inf, -inf, -inf, -inf],
                      [-200.0, -201.0, -300.0, -250.0, -inf, -inf], [80.0, 79.0, -80.0, 0.0, 81.0, -inf],
                      [1e30, -1e30, 0.0, 5.0, 3e38, -3e38]], device="cuda")
    idx, w, s = run_route(m, x, 3, sigmoid, renorm=renorm, scores=True)
    assert torch.equal(idx.long(), ref_route(x, 3, sigmoid, None, 1, 1, 1))
    ww, sw = ref_weights(x, idx.long(), sigmoid, renorm, 1.0), ref_scores(x, sigmoid)
    # |x - max| <= 130 where the result is a normal number: 130 u more; below 2^-126 nothing but zero is asked
    check(w, ww, 200 * U * ww + 2e-38, "topk_w")
    check(s, sw, 200 * U * sw + 2e-38, "scores")
    assert (w[0] == 0).all()
    # NaN and +inf: unspecified experts, but in range
    x = torch.full((4, 40), NAN, device="cuda")
    x[1, 3], x[2] = inf, inf
    x[3, ::2] = 1.0
    i = run_route(m, x, 16, sigmoid, bias=torch.zeros(40, device="cuda"), G=4, top=2, gt=2)[0]
    assert ((i >= 0) & (i < 40)).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("G,top,gt", [(1, 1, 1), (4, 2, 1), (4, 3, 2)])
def test_route_with_experts_switched_off(m, sigmoid, G, top, gt):
    """A bias of -infinity, for whole groups among them: the others are taken first, in their order."""
    g = gen(12)
    T, E, k = 50, 48, 6
    x = randn(g, T, E)
    bias = randn(g, E, sigma=0.1)
    bias[::3] = -float("inf")
    bias[12:24] = -float("inf")
    idx, w, _ = run_route(m, x, k, sigmoid, bias, None, G, top, gt)
    want = ref_route(x, k, sigmoid, bias, G, top, gt)
    assert torch.equal(idx.long(), want) and not torch.isneginf(bias[idx.long()]).any()
    ww = ref_weights(x, want, sigmoid, True, 1.0)
    check(w, ww, 70 * U * ww, "topk_w")


@pytest.mark.parametrize("T,d,E,dtype", [(1, 128, 8, torch.float16), (70, 100, 24, torch.float32), (600, 256, 64, torch.float16)])
def test_route_from_tokens(m, T, d, E, dtype):
    """Logits bit for bit those of moe_gate_topk, the rest as with logits_in; logits_in with logits_out copies."""
    g = gen(3)
    x, Wg = randn(g, T, d, dtype=dtype), randn(g, d, E, sigma=0.1)
    k = 4
    lo, l2 = (torch.full((T, E), NAN, device="cuda") for _ in range(2))
    idx, i2 = (torch.empty((T, k), dtype=torch.int32, device="cuda") for _ in range(2))
    w, w2 = (torch.empty((T, k), device="cuda") for _ in range(2))
    m.moe_route(x, Wg, k, idx, w, logits_out=lo, score=m.MOE_SCORE_SIGMOID)
    m.moe_gate_topk(x, Wg, 1, torch.empty((T, 1), dtype=torch.int32, device="cuda"), torch.empty((T, 1), device="cuda"),
                    logits_out=l2)
    assert torch.equal(lo, l2)
    m.moe_route(None, None, k, i2, w2, logits_in=lo, logits_out=l2.zero_(), score=m.MOE_SCORE_SIGMOID)
    assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(l2, lo)


def ref_route_grad(x, idx, mask, dw, ds, sigmoid, renorm, scale):
    """Autograd of the definition in 64 bits, and per element the sum of the magnitudes that make it up."""
    T, E = x.shape
    on = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    xs = torch.where(on[:, None], x, torch.zeros_like(x)).double().requires_grad_()
    s = 1 / (1 + torch.exp(-xs)) if sigmoid else torch.softmax(xs, 1)
    total = 0
    mag = torch.zeros_like(xs)
    sd = s.detach()
    if dw is not None:
        ii = idx.long()
        ok = (ii >= 0) & (ii < E)
        sel = s.gather(1, ii.clamp(0, E - 1)) * ok
        w = scale * (sel / sel.sum(1, keepdim=True).clamp(min=1e-300) if renorm else sel)
        g = dw.double()
        total = total + (w * g * on[:, None]).sum()
        a = w.detach().abs() * (g.abs() + ((w.detach() * g).abs().sum(1, keepdim=True) / scale if renorm else 0)) * ok
        mag = mag.scatter_add(1, ii.clamp(0, E - 1), a)
        if not sigmoid and not renorm:
            mag = mag + sd * (w.detach() * g).abs().sum(1, keepdim=True)
    if ds is not None:
        total = total + torch.where(on[:, None], s * ds.double(), torch.zeros_like(s)).sum()
        a = torch.where(on[:, None], ds.double().abs() * sd, torch.zeros_like(sd))
        mag = mag + a + (0 if sigmoid else sd * a.sum(1, keepdim=True))
    (gr,) = torch.autograd.grad(total, xs)
    return gr * on[:, None], mag * on[:, None]


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 4, 3), (64, 16, 4), (33, 17, 5), (100, 60, 6), (257, 128, 8),
                                   (31, 250, 16), (20, 512, 8), (9, 1000, 16), (4000, 256, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("parts", ["w", "s", "ws"])
def test_route_gradient(m, T, E, k, sigmoid, renorm, parts):
    g = gen(T + E)
    x = randn(g, T, E, sigma=2.0)
    mask = (torch.rand(T, generator=g, device="cuda") < 0.8) if T > 1 else None
    idx = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    idx[torch.rand((T, k), generator=g, device="cuda") < 0.1] = -1
    idx[torch.rand((T, k), generator=g, device="cuda") < 0.05] = E
    dw = randn(g, T, k) if "w" in parts else None
    ds = randn(g, T, E) if "s" in parts else None
    given = x.clone()
    if mask is not None:
        given[~mask] = NAN
        for q in (dw, ds):
            if q is not None:
                q[~mask] = 0.0
    dl = torch.full((T, E), NAN, device="cuda")
    m.moe_route_backward(given, idx, dl, dtopk_w=dw, dscores=ds, token_mask=mask, score=int(sigmoid), renormalize=renorm,
                         scale=1.5)
    want, mag = ref_route_grad(x, idx, mask, dw, ds, sigmoid, renorm, 1.5)
    # the row's softmax takes the hardware's exponential: 2 + 1.2 |x - max| ulp, |x - max| <= 20: 52 u; its sum, the
    # sums over k or E (a tree of 32 + 5) and six products and quotients.  The formula's own 64 bits: a column that
    # nothing reaches (zero here) is what 2^-53 of each of the row's terms leaves, at most some 64 of them deep
    check(dl, want, 128 * U * mag + 2.0 ** -47 * mag.sum(1, keepdim=True) + 1e-37, "dlogits")


@pytest.mark.parametrize("T,E,k", [(5, 1, 1), (40, 3, 3), (300, 128, 8), (21, 600, 16)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_of_an_expert_named_twice(m, T, E, k, sigmoid, renorm):
    """Plans of the caller's own: each mention carries its gradient."""
    g = gen(T * 3 + E)
    d = 128
    x, dw, ds = randn(g, T, E, sigma=2.0), randn(g, T, k), randn(g, T, E)
    idx = torch.randint(0, min(E, 3), (T, k), generator=g, device="cuda").to(torch.int32)
    want, mag = ref_route_grad(x, idx, None, dw, ds, sigmoid, renorm, 1.5)
    tol = 128 * U * mag + 2.0 ** -47 * mag.sum(1, keepdim=True) + 1e-37
    tokens, Wg = randn(g, T, d, dtype=torch.float16), randn(g, d, E, sigma=0.1)
    ws = torch.zeros(m.moe_gate_backward_workspace_size(T, d, E, torch.float16), dtype=torch.uint8, device="cuda")
    for deep in (False, True):
        dl = torch.full((T, E), NAN, device="cuda")
        more = dict(tokens=tokens, Wg=Wg, dWg=torch.empty((d, E), device="cuda"), dtokens=torch.empty_like(tokens),
                    workspace=ws) if deep else {}
        m.moe_route_backward(x, idx, dl, dtopk_w=dw, dscores=ds, score=int(sigmoid), renormalize=renorm, scale=1.5, **more)
        check(dl, want, tol, f"dlogits, deep {deep}")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(m, sigmoid, renorm):
    g = gen(9)
    T, E, k = 12, 20, 5
    x, dw, v = randn(g, T, E), randn(g, T, k), randn(g, T, E).double()
    idx, _, _ = run_route(m, x, k, sigmoid)
    dl = torch.empty((T, E), device="cuda")
    m.moe_route_backward(x, idx, dl, dtopk_w=dw, score=int(sigmoid), renormalize=renorm, scale=0.5)
    eps = 1e-5

    def loss(z):
        s = 1 / (1 + torch.exp(-z)) if sigmoid else torch.softmax(z, 1)
        w = s.gather(1, idx.long())
        return (0.5 * (w / w.sum(1, keepdim=True) if renorm else w) * dw.double()).sum()

    diff = float((loss(x.double() + eps * v) - loss(x.double() - eps * v)) / (2 * eps))
    # the second-order term cancels; the third is below eps^2 |v|^3 = 1e-10 a value, rounding 1e-16 / eps
    assert abs(float((dl.double() * v).sum()) - diff) < 1e-8 + 128 * U * float((dl.double() * v).abs().sum()) * 4


@pytest.mark.parametrize("dtype,T,d,E,k", [(torch.float16, 1, 128, 8, 2), (torch.float16, 300, 256, 60, 6),
                                           (torch.float16, 2000, 512, 128, 8), (torch.float16, 200, 128, 300, 8),
                                           (torch.float32, 150, 68, 24, 4)])
@pytest.mark.parametrize("masked", [False, True])
def test_route_gradient_to_gate(m, dtype, T, d, E, k, masked):
    """dWg and dtokens of the call are the products of its own dlogits."""
    g = gen(T)
    x, Wg = randn(g, T, d, dtype=dtype), randn(g, d, E, sigma=0.05)
    logits = (x.float() @ Wg).contiguous()
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7) if masked else None
    if masked:
        mask[0] = True
    idx, _, _ = run_route(m, logits, k, True)
    dw = randn(g, T, k)
    if masked:
        x[~mask] = NAN
    dl, alone = (torch.full((T, E), NAN, device="cuda") for _ in range(2))
    dWg = torch.full((d, E), NAN, device="cuda")
    dx_in = randn(g, T, d, dtype=dtype)
    dx = torch.full((T, d), NAN, dtype=dtype, device="cuda")
    ws = torch.full((m.moe_gate_backward_workspace_size(T, d, E, dtype),), 0xA5, dtype=torch.uint8, device="cuda")
    kw = dict(dtopk_w=dw, token_mask=mask, score=m.MOE_SCORE_SIGMOID, scale=2.0)
    m.moe_route_backward(logits, idx, dl, tokens=x, Wg=Wg, dWg=dWg, dtokens=dx, dtokens_in=dx_in, workspace=ws, **kw)
    assert m.moe_status_read(ws) == m.MOE_OK
    m.moe_route_backward(logits, idx, alone, **kw)
    # (another kernel, whose sums and products may be fused in other places: each is held to the formula)
    want, mag = ref_route_grad(logits, idx, mask, dw, None, True, True, 2.0)
    for q in (dl, alone):
        check(q, want, 128 * U * mag + 2.0 ** -47 * mag.sum(1, keepdim=True) + 1e-37, "dlogits")
    xd = torch.where(mask[:, None], x, torch.zeros_like(x)).double() if masked else x.double()
    # products of 128 rows in the tensor cores (2 u an addition) or multiply-adds, then T / 128 sums; the split of
    # dlogits: 2^-23 of each value and 2^-36 of the largest (of Wg: by 128 of its rows)
    mag = xd.abs().t() @ dl.double().abs()
    check(dWg, xd.t() @ dl.double(), (300 + T / 64) * U * mag + 2.0 ** -34 * float(dl.abs().max()) * xd.abs().sum(0)[:, None] + 1e-37, "dWg")
    want = dx_in.double() + dl.double() @ Wg.double().t()
    mag = dx_in.double().abs() + dl.double().abs() @ Wg.double().abs().t()
    check(dx, want, (2 * E + 64) * U * mag + half(dtype) * want.abs() + 2.0 ** -25, "dtokens")


# ---------------------------------------------------------------- 8 bits
def step_of(amax):
    """Smallest power of two s with amax <= 448 s (zero: 1), in 64 bits."""
    s = torch.exp2(torch.floor(torch.log2(amax.clamp(min=1e-300) / 448)) - 1)
    for _ in range(3):
        s = torch.where(amax > 448 * s, s * 2, s)
    return torch.where(amax > 0, s.clamp(min=2.0 ** -126), torch.ones_like(amax))


def round8(v):
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def rows8(v):
    s = step_of(v.abs().unflatten(1, (-1, 128)).amax(2)).repeat_interleave(128, 1)
    return round8(v / s) * s


@pytest.mark.parametrize("E,K,N", [(1, 128, 128), (3, 256, 384), (2, 1024, 128), (5, 128, 640)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_fp8_quantize(m, E, K, N, dtype):
    g = gen(K + N)
    W = randn(g, E, K, N, sigma=0.02, dtype=dtype)
    # blocks of zeros, of one size, of values next to the border 448 2^p, of subnormal results and of tiny values
    W[0, :128, :128] = 0
    W[E - 1, :128, :128] = torch.tensor([1.75, -1.75 * 1.0009765625], device="cuda")[torch.randint(0, 2, (128, 128), generator=g, device="cuda")].to(dtype)
    W[E - 1, 0, N - 1] = 440.0
    W[0, K - 1, N - 128:] *= 1e-3
    if K > 128:
        W[0, 128:256, :128] *= 2.0 ** -12 if dtype == torch.float16 else 1e-36
    Wq = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.full((E, N // 128, K // 128), NAN, device="cuda")
    m.moe_fp8_quantize(W, Wq, s)
    Wd = W.double().transpose(1, 2)
    b = Wd.reshape(E, N // 128, 128, K // 128, 128)
    ws = step_of(b.abs().amax(dim=(2, 4)))
    assert torch.equal(s.double(), ws)
    want = round8(b / ws[:, :, None, :, None]).reshape(E, N, K)
    assert torch.equal(Wq.double(), want)
    u8 = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
    m.moe_fp8_quantize(W, u8, s)
    assert torch.equal(u8, Wq.view(torch.uint8))
    # infinities and NaN stay in their block
    W[E - 1, K - 1, N - 1] = float("inf")
    m.moe_fp8_quantize(W, Wq, s)
    assert torch.isnan(s[E - 1, -1, -1]) and torch.isnan(Wq[E - 1, -128:, -128:].float()).all()
    assert int(torch.isnan(s).sum()) == 1


def experts8(m, g, E, n_in, n_out, general=False):
    W = randn(g, E, n_in, n_out, sigma=n_in ** -0.5, dtype=torch.float16)
    q = torch.empty((E, n_out, n_in), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((E, n_out // 128, n_in // 128), device="cuda")
    m.moe_fp8_quantize(W, q, s)
    if general:                                       # scales that are no powers of two
        s *= 0.5 + torch.rand(s.shape, generator=g, device="cuda")
    return q, s


def values8(q, s):
    return q.double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def gelu(x):
    return torch.nn.functional.gelu(x, approximate="tanh")


def ref_ffn8(x, W1, W2, d, f, whole=False):
    """Rows of one expert in 64 bits, and how far the 32-bit calculation may be off: what a hidden value may be off by
    moves its 8-bit value where a border is within that."""
    x = rows8(x.double())
    u, mag = x @ W1.t(), x.abs() @ W1.abs().t()
    # 128 products of a block in the tensor cores (2 u each addition), the block's scale (2 u) and d / 128 sums; whole: all
    # d in the tensor cores, whose scales are exact
    eu = (2 * d if whole else 2 * 128 + 4 + d / 128) * U * mag
    h = gelu(u)
    # |gelu'| <= 1.13; gelu's own steps: three roundings of its exponent z, 3 |z| ln 2 u with |z| <= 29 (beyond that the value
    # is below 1e-8 of the argument): 60 u, the exponential 2 ulp, a sum, a reciprocal and a product: 8 u
    eh = 1.13 * eu + 80 * U * h.abs() + 1e-30
    lo, hi = rows8(h - eh), rows8(h + eh)
    q = rows8(h)
    # (lo and hi are taken with the scales of their own rows: a scale at the border moves all its block)
    move = torch.maximum((hi - q).abs(), (lo - q).abs())
    y = q @ W2.t()
    tol = move @ W2.abs().t() + (2 * f if whole else 2 * 128 + 4 + f / 128) * U * ((q.abs() + move) @ W2.abs().t())
    return y, tol


# slots per expert
LAYOUTS = [[1], [5], [16], [17, 0, 1], [0, 0, 3, 0], [33, 64, 1], [0] * 7 + [2], [160, 161, 3], [255, 256, 257, 1],
           [600, 1, 0, 40], [31, 32, 33, 15, 16, 17, 4, 5], [1] * 40, [130, 0, 97, 12]]


@pytest.mark.parametrize("rows", LAYOUTS, ids=str)
@pytest.mark.parametrize("d,f", [(128, 128), (256, 640), (640, 256)])
@pytest.mark.parametrize("spare", [0, 37])
def test_expert_ffn_fp8(m, rows, d, f, spare, general=True):
    E, S = len(rows), sum(rows)
    g = gen(S * 3 + E + d)
    T = max(1, S // 2 + 3)
    x = randn(g, T, d, dtype=torch.float16)
    perm = torch.randint(0, T, (S + spare,), generator=g, device="cuda").to(torch.int32)
    offsets = torch.tensor([0] + list(np.cumsum(rows)), dtype=torch.int32, device="cuda")
    W1, s1 = experts8(m, g, E, d, f, general=general)
    W2, s2 = experts8(m, g, E, f, d)
    out = torch.full((S + spare + 2, d), 7.5, dtype=torch.float16, device="cuda")
    ws = torch.full((m.moe_expert_fp8_workspace_size(T, d, f, E, S + spare, torch.float16),), 0xA5, dtype=torch.uint8,
                    device="cuda")
    m.moe_expert_ffn_fp8(x, perm, offsets, W1, s1, W2, s2, S + spare, out, ws)
    assert m.moe_status_read(ws) == m.MOE_OK
    assert (out[S:] == 7.5).all()                     # rows behind the last slot are left as they were
    at = 0
    for e, n in enumerate(rows):
        if n:
            want, tol = ref_ffn8(x[perm[at:at + n].long()], values8(W1[e], s1[e]), values8(W2[e], s2[e]), d, f,
                                 whole=not general)
            check(out[at:at + n], want, tol + half(torch.float16) * want.abs() + 2.0 ** -25, f"expert {e}")
        at += n
    again = torch.full_like(out, 7.5)
    m.moe_expert_ffn_fp8(x, perm, offsets, W1.view(torch.uint8), s1, W2.view(torch.uint8), s2, S + spare, again, ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("rows", [[1], [0, 3], [9, 0, 0, 20], [32, 33], [1, 0, 1, 0, 1, 2, 1, 1]], ids=str)
@pytest.mark.parametrize("d,f", [(1024, 128), (1152, 2048), (4096, 1024), (384, 4224)])
def test_expert_ffn_fp8_short_batches(m, rows, d, f):
    """Few items with many inputs each: shared by clusters of two, four and eight blocks."""
    test_expert_ffn_fp8(m, rows, d, f, 2)


@pytest.mark.parametrize("rows,d,f", [([90], 256, 512), ([160, 161, 3], 768, 256), ([65] * 9, 1280, 1024),
                                      ([160, 161, 3], 4352, 6400), ([255, 256, 257, 1], 2304, 5120), ([600, 1, 0, 40], 4352, 3328),
                                      ([240, 241, 239, 0, 480], 1280, 6400), ([1000, 8, 9, 16, 17, 120], 2304, 3328),
                                      ([500, 0, 0, 333], 3328, 3200), ([65] * 33, 2048, 2048), ([3000, 700], 256, 9216),
                                      ([2999, 701, 0], 9216, 256)], ids=str)
def test_expert_ffn_fp8_long_runs(m, rows, d, f):
    """Scales that are powers of two, as the quantiser makes them: applied by the tensor cores where runs are long."""
    test_expert_ffn_fp8(m, rows, d, f, 3, general=False)


@pytest.mark.parametrize("bad", [0.0, -1.0, 3.0, 2.0 ** -140, float("inf"), NAN])
@pytest.mark.parametrize("which", [0, 1])
def test_expert_ffn_fp8_one_other_scale(m, which, bad):
    """One scale that is no power of two (of either product): its column block of every row, and no other."""
    g = gen(7)
    E, n, d, f = 2, 300, 3328, 4608
    x = randn(g, E * n, d, dtype=torch.float16)
    W1, s1 = experts8(m, g, E, d, f)
    W2, s2 = experts8(m, g, E, f, d)
    s = (s1, s2)[which]
    if np.isfinite(bad):
        s[1, 1, 1] *= bad                             # (2^-140: a subnormal)
    else:
        s[1, 1, 1] = bad
    perm = torch.arange(E * n, device="cuda").to(torch.int32)
    offsets = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    out = torch.empty((E * n, d), dtype=torch.float16, device="cuda")
    ws = torch.empty(m.moe_expert_fp8_workspace_size(E * n, d, f, E, E * n, torch.float16), dtype=torch.uint8, device="cuda")
    m.moe_expert_ffn_fp8(x, perm, offsets, W1, s1, W2, s2, E * n, out, ws)
    for e in range(E):
        rows = slice(e * n, (e + 1) * n)
        if e == 1 and not np.isfinite(bad):
            cols = slice(128, 256) if which else slice(0, d)
            assert not torch.isfinite(out[rows, cols]).any() if np.isnan(bad) or which == 0 else True
            if which:
                want, tol = ref_ffn8(x[rows], values8(W1[e], s1[e]), values8(W2[e], s2[e])[:128], d, f, True)
                check(out[rows, :128], want, tol + half(torch.float16) * want.abs() + 2.0 ** -25, "the other columns")
            continue
        want, tol = ref_ffn8(x[rows], values8(W1[e], s1[e]), values8(W2[e], s2[e]), d, f, True)
        check(out[rows], want, tol + half(torch.float16) * want.abs() + 2.0 ** -25, f"expert {e}")


def test_expert_ffn_fp8_bad_indices(m):
    """Plans that leave their bounds: reported, and nothing outside [0, S_max) is written."""
    g = gen(1)
    T, d, f, E, S = 20, 128, 256, 3, 24
    x = randn(g, T, d, dtype=torch.float16)
    W1, s1 = experts8(m, g, E, d, f)
    W2, s2 = experts8(m, g, E, f, d)
    ws = torch.empty(m.moe_expert_fp8_workspace_size(T, d, f, E, S, torch.float16), dtype=torch.uint8, device="cuda")
    good = torch.arange(S, device="cuda").to(torch.int32) % T
    for off, bad in ([0, 8, 16, 24], None), ([0, 8, 16, 900], None), ([0, 20, 4, 24], None), ([-5, 8, 16, 24], None), \
            ([0, 8, 16, 24], 3), ([0, 8, 16, 24], 23):
        perm = good.clone()
        if bad is not None:
            perm[bad] = T if bad == 3 else -1
        out = torch.full((S + 4, d), 7.5, dtype=torch.float16, device="cuda")
        m.moe_expert_ffn_fp8(x, perm, torch.tensor(off, dtype=torch.int32, device="cuda"), W1, s1, W2, s2, S, out, ws)
        fine = off == [0, 8, 16, 24] and bad is None
        assert m.moe_status_read(ws) == (m.MOE_OK if fine else m.MOE_ERR_DEVICE_BOUNDS)
        assert (out[S:] == 7.5).all()


@pytest.mark.parametrize("T,d,f", [(40, 256, 256), (700, 3328, 4608)])
def test_expert_ffn_fp8_special_values(m, T, d, f):
    """A row of zeros gives zeros; infinities and NaN stay in their token's slots."""
    g = gen(2)
    E = 2
    x = randn(g, T, d, dtype=torch.float16)
    x[3] = 0
    x[5, 7], x[9, 200], x[11] = float("inf"), NAN, 65504.0
    W1, s1 = experts8(m, g, E, d, f)
    W2, s2 = experts8(m, g, E, f, d)
    perm = torch.arange(T, device="cuda").to(torch.int32)
    offsets = torch.tensor([0, T - 15, T], dtype=torch.int32, device="cuda")
    out = torch.empty((T, d), dtype=torch.float16, device="cuda")
    ws = torch.empty(m.moe_expert_fp8_workspace_size(T, d, f, E, T, torch.float16), dtype=torch.uint8, device="cuda")
    m.moe_expert_ffn_fp8(x, perm, offsets, W1, s1, W2, s2, T, out, ws)
    assert (out[3] == 0).all() and torch.isnan(out[5]).all() and torch.isnan(out[9]).all()
    rest = [t for t in range(T) if t not in (5, 9, 11)]
    assert torch.isfinite(out[rest]).all()


# ---------------------------------------------------------------- the norms around a block
def norm_inputs(g, T, d, k, dtype, drop=0.2, spare=3):
    S = T * k + spare
    slot = torch.randperm(S, generator=torch.Generator().manual_seed(T + d))[:T * k].to(torch.int32).cuda().view(T, k)
    slot[torch.rand((T, k), generator=g, device="cuda") < drop] = -1
    if T > 2:
        slot[2] = -1                                  # a token that keeps no expert
    if T > 4 and k:
        slot[4, 0] = S                                # (outside: as if dropped)
    return slot.contiguous(), randn(g, S, d, dtype=dtype, sigma=0.7), torch.rand((T, k), generator=g, device="cuda")


def ref_norm(res, rows, slot, w, shared, post, gate, alpha, nxt, eps, S):
    """The block's end in 64 bits, its intermediate values and the magnitudes of y's and h's terms."""
    T, d = res.shape
    y = torch.zeros((T, d), dtype=torch.float64, device="cuda")
    ym = torch.zeros_like(y)
    if slot is not None:
        for j in range(slot.shape[1]):
            on = ((slot[:, j] >= 0) & (slot[:, j] < S)).nonzero()[:, 0]
            t = w[on, j, None].double() * rows[slot[on, j].long()].double()
            y = y.index_add(0, on, t)
            ym = ym.index_add(0, on, t.detach().abs())
    if shared is not None:
        y, ym = y + shared.double(), ym + shared.detach().double().abs()
    rp = torch.rsqrt(y.square().mean(1, keepdim=True) + eps) if post is not None else torch.ones_like(y[:, :1])
    z0 = y * rp * (post.double() if post is not None else 1)
    z = z0 * (gate.double() if gate is not None else 1)
    block = slot is not None or shared is not None
    h = res.double() + (alpha * z if block else 0)
    rn = torch.rsqrt(h.square().mean(1, keepdim=True) + eps)
    n = h * rn * nxt.double() if nxt is not None else None
    return y, ym, rp, z0, z, h, rn, n


NORMS = [(1, 8, 1), (1, 1024, 2), (5, 64, 3), (33, 256, 8), (70, 264, 2), (19, 520, 16), (40, 1032, 4), (9, 3584, 2),
         (11, 4104, 5), (6, 8200, 2), (4, 16384, 3), (700, 128, 1)]


@pytest.mark.parametrize("T,d,k", NORMS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("parts", ["", "s", "p", "g", "pg", "spg"])
def test_block_norm(m, T, d, k, dtype, parts):
    g = gen(T * d + k)
    slot, rows, w = norm_inputs(g, T, d, k, dtype)
    S = rows.shape[0]
    res = randn(g, T, d, dtype=dtype)
    shared = randn(g, T, d, dtype=dtype) if "s" in parts else None
    post = 1 + randn(g, d, sigma=0.2) if "p" in parts else None
    gate = randn(g, d) if "g" in parts else None
    nxt = 1 + randn(g, d, sigma=0.2)
    hid, nrm = (torch.full((T, d), NAN, dtype=dtype, device="cuda") for _ in range(2))
    rp, rn = (torch.full((T,), NAN, device="cuda") for _ in range(2))
    m.moe_block_norm(res, hid, expert_out=rows, slot_of=slot, topk_w=w, shared=shared, post_w=post, gate=gate, alpha=0.6,
                     next_w=nxt, normed_out=nrm, eps=1e-5, rstd_post=rp if post is not None else None, rstd_next=rn)
    y, ym, wp, z0, z, h, wn, n = ref_norm(res, rows, slot, w, shared, post, gate, 0.6, nxt, 1e-5, S)
    # y: k + 1 additions and products; its norm: the error of y against its magnitudes (in the mean square at most
    # (k + 2) u |ym| / |y| twice), a sum of d squares (32 in a thread, then 5 + 16) and a root; four products
    ratio = 1 if post is None else 1 + (ym.norm(dim=1, keepdim=True) / (y.square().sum(1, keepdim=True) + d * 1e-5).sqrt())
    f = wp * (post.double().abs() if post is not None else 1) * (gate.double().abs() if gate is not None else 1)
    ez = (2 * (k + 2) * ratio + 80) * U * ym * f * 0.6 * ratio
    eh = ez + 4 * U * (h.abs() + res.double().abs())
    check(hid, h, eh + half(dtype) * h.abs() + 2.0 ** -25 * (dtype == torch.float16), "hidden")
    en = (eh.norm(dim=1, keepdim=True) / (h.square().sum(1, keepdim=True) + d * 1e-5).sqrt()) + 80 * U
    check(nrm, n, eh * wn * nxt.double().abs() + en * n.abs() + half(dtype) * n.abs() + 2.0 ** -25 * (dtype == torch.float16), "normed")
    check(rn, wn[:, 0], en[:, 0] * wn[:, 0], "rstd_next")
    if post is not None:
        check(rp, wp[:, 0], ((2 * (k + 2) * ratio + 80) * U * ratio * wp)[:, 0], "rstd_post")
    # in place, without the outputs for training
    h2 = res.clone()
    m.moe_block_norm(h2, h2, expert_out=rows, slot_of=slot, topk_w=w, shared=shared, post_w=post, gate=gate, alpha=0.6,
                     next_w=nxt, normed_out=nrm.fill_(NAN), eps=1e-5)
    assert torch.equal(h2, hid)
    # the sum alone
    m.moe_block_norm(res, h2.fill_(NAN), expert_out=rows, slot_of=slot, topk_w=w, shared=shared, post_w=post, gate=gate,
                     alpha=0.6, eps=1e-5)
    assert torch.equal(h2, hid)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_block_norm_without_experts(m, dtype):
    """The norm before the first block; a block that is a dense one."""
    g = gen(8)
    T, d = 37, 512
    res, y = randn(g, T, d, dtype=dtype), randn(g, T, d, dtype=dtype)
    w = 1 + randn(g, d, sigma=0.1)
    nrm, hid = torch.empty_like(res), torch.empty_like(res)
    m.moe_block_norm(res, next_w=w, normed_out=nrm, eps=0.0)
    want = res.double() * torch.rsqrt(res.double().square().mean(1, keepdim=True)) * w.double()
    check(nrm, want, (80 * U + half(dtype)) * want.abs() + 2.0 ** -25, "normed")
    m.moe_block_norm(res, hid, shared=y, next_w=w, normed_out=nrm, alpha=-2.0)
    want = res.double() - 2 * y.double()
    check(hid, want, 2 * U * (res.double().abs() + 2 * y.double().abs()) + half(dtype) * want.abs() + 2.0 ** -25, "hidden")
    res[0] = 0                                        # a row of zeros
    m.moe_block_norm(res, next_w=w, normed_out=nrm)
    assert (nrm[0] == 0).all()
    res[1, 3] = NAN                                   # stays in its row
    m.moe_block_norm(res, next_w=w, normed_out=nrm)
    assert torch.isnan(nrm[1]).all() and torch.isfinite(nrm[2:]).all()


@pytest.mark.parametrize("T,d,k", NORMS + [(3000, 64, 2)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("parts", ["", "sg", "p", "spg"])
@pytest.mark.parametrize("sides", ["hn", "h", "n"])
def test_block_norm_gradient(m, T, d, k, dtype, parts, sides):
    g = gen(T * d + k + 1)
    slot, rows, w = norm_inputs(g, T, d, k, dtype)
    w = w + 0.1
    S = rows.shape[0]
    res = randn(g, T, d, dtype=dtype)
    shared = randn(g, T, d, dtype=dtype) if "s" in parts else None
    post = 1 + randn(g, d, sigma=0.2) if "p" in parts else None
    gate = randn(g, d) if "g" in parts else None
    nxt = 1 + randn(g, d, sigma=0.2)
    eps, alpha = 1e-2, 0.6
    hid, nrm = torch.empty_like(res), torch.empty_like(res)
    rp, rn = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    m.moe_block_norm(res, hid, expert_out=rows, slot_of=slot, topk_w=w, shared=shared, post_w=post, gate=gate, alpha=alpha,
                     next_w=nxt, normed_out=nrm, eps=eps, rstd_post=rp if post is not None else None, rstd_next=rn)
    dhid = randn(g, T, d, dtype=dtype) if "h" in sides else None
    dnrm = randn(g, T, d, dtype=dtype) if "n" in sides else None
    out = dict(dresidual=torch.full((T, d), NAN, dtype=dtype, device="cuda"),
               dexpert_out=torch.full((S, d), 7.5, dtype=dtype, device="cuda"), dtopk_w=torch.full((T, k), NAN, device="cuda"))
    if shared is not None:
        out["dshared"] = torch.full((T, d), NAN, dtype=dtype, device="cuda")
    for name, on in (("dpost_w", post is not None), ("dgate", gate is not None), ("dnext_w", dnrm is not None)):
        if on:
            out[name] = torch.full((d,), NAN, device="cuda")
    ws = torch.full((m.moe_block_norm_workspace_size(T, d, k, dtype),), 0xA5, dtype=torch.uint8, device="cuda")
    given = dict(dhidden=dhid, dnormed=dnrm, expert_out=rows, slot_of=slot, topk_w=w, shared=shared, post_w=post, gate=gate,
                 alpha=alpha)
    if dnrm is not None:
        given.update(hidden=hid, rstd_next=rn, next_w=nxt)
    if post is not None:
        given["rstd_post"] = rp
    m.moe_block_norm_backward(**given, **out, workspace=ws)

    # the formulas in 64 bits at the stored rows and factors, with the magnitudes of their terms
    y, ym, _, _, _, _, _, _ = ref_norm(res, rows, slot, w, shared, post, gate, alpha, nxt, eps, S)
    dh = dhid.double() if dhid is not None else torch.zeros((T, d), dtype=torch.float64, device="cuda")
    dm = dh.abs()
    if dnrm is not None:
        h, r, a = hid.double(), rn.double()[:, None], dnrm.double() * nxt.double()
        dh = dh + r * (a - h * r * r * (h * a).mean(1, keepdim=True))
        dm = dm + r * (a.abs() + h.abs() * r * r * (h * a).abs().mean(1, keepdim=True))
    # sums of d terms: 32 in a thread, then 5 + 16 in a tree; with the products and factors 96
    K = 96 * U
    hf = half(dtype)
    sub = 2.0 ** -25 if dtype == torch.float16 else 0.0
    check(out["dresidual"], dh, K * dm + hf * dh.abs() + sub, "dresidual")
    dz, zm = alpha * dh, alpha * dm
    Ky = (k + 4) * U
    r = rp.double()[:, None] if post is not None else 1.0
    z0 = y * r * (post.double() if post is not None else 1.0)
    z0m = ym * r * (post.double().abs() if post is not None else 1.0)
    many = (T / 100 + 64) * U                          # sums over tokens: ten a team, then 304 of these by eights
    if gate is not None:
        check(out["dgate"], (dz * z0).sum(0), ((K + Ky + many) * zm * z0m).sum(0) + 1e-37, "dgate")
        dz, zm = dz * gate.double(), zm * gate.double().abs()
    dy, em = dz, zm
    if post is not None:
        check(out["dpost_w"], (dz * y * r).sum(0), ((K + Ky + many) * zm * ym * r).sum(0) + 1e-37, "dpost_w")
        b, bm = dz * post.double(), zm * post.double().abs()
        dy = r * (b - y * r * r * (y * b).mean(1, keepdim=True))
        em = r * (bm + ym * r * r * (ym * bm).mean(1, keepdim=True))
    if dnrm is not None:
        t = dnrm.double() * hid.double() * rn.double()[:, None]
        check(out["dnext_w"], t.sum(0), (many + 4 * U) * t.abs().sum(0) + 1e-37, "dnext_w")
    E = 2 * K + 4 * Ky
    if shared is not None:
        check(out["dshared"], dy, E * em + hf * dy.abs() + sub, "dshared")
    named = torch.zeros(S, dtype=torch.bool, device="cuda")
    for j in range(k):
        on = ((slot[:, j] >= 0) & (slot[:, j] < S)).nonzero()[:, 0]
        s = slot[on, j].long()
        named[s] = True
        want = w[on, j, None].double() * dy[on]
        check(out["dexpert_out"][s], want, (E + U) * w[on, j, None].double() * em[on] + hf * want.abs() + sub, "dexpert_out")
        full = torch.zeros(T, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(full)
        full[on] = (dy[on] * rows[s].double()).sum(1)
        tol[on] = ((E + K) * em[on] * rows[s].double().abs()).sum(1)
        check(out["dtopk_w"][:, j], full, tol, "dtopk_w")
    assert (out["dexpert_out"][~named] == 7.5).all()   # slots that no assignment names
    # dresidual in dhidden's place, and nothing but it
    if dhid is not None:
        d2 = dhid.clone()
        m.moe_block_norm_backward(**{**given, "dhidden": d2}, dresidual=d2)
        assert torch.equal(d2, out["dresidual"])


def test_block_norm_gradient_against_differences(m):
    """Central differences of the 64-bit formulas along a random direction of every input."""
    g = gen(17)
    T, d, k = 6, 24, 3
    slot, rows, w = norm_inputs(g, T, d, k, torch.float32)
    S = rows.shape[0]
    p = dict(res=randn(g, T, d), rows=rows, w=w, shared=randn(g, T, d), post=1 + randn(g, d, sigma=0.2),
             gate=randn(g, d), nxt=1 + randn(g, d, sigma=0.2))
    hid, nrm = torch.empty((T, d), device="cuda"), torch.empty((T, d), device="cuda")
    rp, rn = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    m.moe_block_norm(p["res"], hid, expert_out=rows, slot_of=slot, topk_w=w, shared=p["shared"], post_w=p["post"],
                     gate=p["gate"], alpha=0.6, next_w=p["nxt"], normed_out=nrm, eps=1e-2, rstd_post=rp, rstd_next=rn)
    dhid, dnrm = randn(g, T, d), randn(g, T, d)
    out = {q: torch.zeros_like(p[n]) for q, n in (("dresidual", "res"), ("dexpert_out", "rows"), ("dtopk_w", "w"),
                                                  ("dshared", "shared"), ("dpost_w", "post"), ("dgate", "gate"),
                                                  ("dnext_w", "nxt"))}
    ws = torch.empty(m.moe_block_norm_workspace_size(T, d, k, torch.float32), dtype=torch.uint8, device="cuda")
    m.moe_block_norm_backward(dhidden=dhid, dnormed=dnrm, hidden=hid, rstd_next=rn, next_w=p["nxt"], expert_out=rows,
                              slot_of=slot, topk_w=w, shared=p["shared"], post_w=p["post"], rstd_post=rp, gate=p["gate"],
                              alpha=0.6, workspace=ws, **out)
    v = {n: torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64) for n, t in p.items()}

    def loss(eps):
        q = {n: t.double() + eps * v[n] for n, t in p.items()}
        *_, h, _, n = ref_norm(q["res"], q["rows"], slot, q["w"], q["shared"], q["post"], q["gate"], 0.6, q["nxt"], 1e-2, S)
        return (h * dhid.double()).sum() + (n * dnrm.double()).sum()

    eps = 1e-5
    diff = float((loss(eps) - loss(-eps)) / (2 * eps))
    terms = [out[q].double() * v[n] for q, n in (("dresidual", "res"), ("dexpert_out", "rows"), ("dtopk_w", "w"),
                                                 ("dshared", "shared"), ("dpost_w", "post"), ("dgate", "gate"),
                                                 ("dnext_w", "nxt"))]
    total, mag = sum(float(t.sum()) for t in terms), sum(float(t.abs().sum()) for t in terms)
    # the gradient's own error (some 300 u of its terms); the differences': eps^2 times third derivatives of order
    # 10 a value, and rounding / eps
    assert abs(total - diff) < 2000 * U * mag + 1e-6


# ---------------------------------------------------------------- together
def block_step(m, b, st):
    """One forward and backward pass of a block as a user makes it: norm, routing, plan, experts, the block's end."""
    k, E, T = b["k"], b["E"], b["T"]
    m.moe_block_norm(b["res"], next_w=b["w0"], normed_out=st["x"], rstd_next=st["r0"], eps=1e-5)
    m.moe_route(st["x"], b["Wg"], k, st["idx"], st["w"], logits_out=st["logits"], bias=b["bias"], score=m.MOE_SCORE_SIGMOID,
                n_groups=4, top_groups=2, group_top=2, scale=1.5)
    m.moe_dispatch(st["idx"], E, 1.5, st["counts"], st["kept"], st["offsets"], st["perm"], st["slot"])
    m.moe_expert_ffn_fp8(st["x"], st["perm"], st["offsets"], b["W1"], b["s1"], b["W2"], b["s2"], st["perm"].shape[0],
                         st["y"], st["ws8"])
    m.moe_block_norm(b["res"], st["h"], expert_out=st["y"], slot_of=st["slot"], topk_w=st["w"], post_w=b["wp"],
                     gate=b["gate"], alpha=0.5, next_w=b["w1"], normed_out=st["n"], rstd_post=st["rp"], rstd_next=st["rn"],
                     eps=1e-5)
    m.moe_block_norm_backward(dnormed=b["dn"], hidden=st["h"], rstd_next=st["rn"], next_w=b["w1"], expert_out=st["y"],
                              slot_of=st["slot"], topk_w=st["w"], post_w=b["wp"], rstd_post=st["rp"], gate=b["gate"],
                              alpha=0.5, dresidual=st["dres"], dtopk_w=st["dw"], dpost_w=st["dwp"], dgate=st["dgate"],
                              dnext_w=st["dw1"], workspace=st["wsn"])
    m.moe_route_backward(st["logits"], st["idx"], st["dl"], dtopk_w=st["dw"], score=m.MOE_SCORE_SIGMOID, scale=1.5,
                         tokens=st["x"], Wg=b["Wg"], dWg=st["dWg"], dtokens=st["dx"], workspace=st["wsg"])


def block_inputs(m, T, d, f, E, k, seed):
    g = gen(seed)
    W1, s1 = experts8(m, g, E, d, f)
    W2, s2 = experts8(m, g, E, f, d)
    return dict(T=T, E=E, k=k, d=d, f=f, res=randn(g, T, d, dtype=torch.float16), w0=1 + randn(g, d, sigma=0.1),
                w1=1 + randn(g, d, sigma=0.1), wp=1 + randn(g, d, sigma=0.1), gate=randn(g, d), bias=randn(g, E, sigma=0.05),
                Wg=randn(g, d, E, sigma=d ** -0.5), dn=randn(g, T, d, dtype=torch.float16), W1=W1, s1=s1, W2=W2, s2=s2)


def block_state(m, b):
    T, d, f, E, k = b["T"], b["d"], b["f"], b["E"], b["k"]
    h, i = dict(dtype=torch.float16, device="cuda"), dict(dtype=torch.int32, device="cuda")
    S = min(T * k, E * m.moe_capacity(T, E, 1.5))
    st = {q: torch.zeros((T, d), **h) for q in ("x", "h", "n", "dres", "dx")}
    st.update({q: torch.zeros(T, device="cuda") for q in ("r0", "rp", "rn")})
    st.update({q: torch.zeros(d, device="cuda") for q in ("dwp", "dgate", "dw1")})
    st.update(idx=torch.zeros((T, k), **i), w=torch.zeros((T, k), device="cuda"), logits=torch.zeros((T, E), device="cuda"),
              counts=torch.zeros(E, **i), kept=torch.zeros(E, **i), offsets=torch.zeros(E + 1, **i), perm=torch.zeros(S, **i),
              slot=torch.zeros((T, k), **i), y=torch.zeros((S, d), **h), dw=torch.zeros((T, k), device="cuda"),
              dl=torch.zeros((T, E), device="cuda"), dWg=torch.zeros((d, E), device="cuda"))
    u8 = dict(dtype=torch.uint8, device="cuda")
    st["ws8"] = torch.zeros(m.moe_expert_fp8_workspace_size(T, d, f, E, S, torch.float16), **u8)
    st["wsn"] = torch.zeros(m.moe_block_norm_workspace_size(T, d, k, torch.float16), **u8)
    st["wsg"] = torch.zeros(m.moe_gate_backward_workspace_size(T, d, E, torch.float16), **u8)
    return st


RESULTS = ("h", "n", "dres", "dx", "idx", "w", "slot", "dw", "dl", "dWg", "dwp", "dgate", "dw1")


@pytest.mark.parametrize("T,d,f,E,k", [(1, 256, 128, 16, 4), (150, 256, 384, 16, 4), (900, 128, 256, 32, 8)])
def test_block_of_experts(m, T, d, f, E, k):
    """The operators as they are used together, against the same steps in 64 bits (each from the stored results of the
    step before, so that roundings do not add up)."""
    b = block_inputs(m, T, d, f, E, k, 4)
    st = block_state(m, b)
    block_step(m, b, st)
    assert m.moe_status_read(st["ws8"]) == m.MOE_OK and m.moe_status_read(st["wsg"]) == m.MOE_OK
    x = b["res"].double()
    x = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5) * b["w0"].double()
    check(st["x"], x, (80 * U + 2.0 ** -11) * x.abs() + 2.0 ** -25, "x")
    idx = ref_route(st["logits"], k, True, b["bias"], 4, 2, 2)
    assert torch.equal(idx, st["idx"].long())
    w = ref_weights(st["logits"], idx, True, True, 1.5)
    check(st["w"], w, 70 * U * w, "w")
    # the plan: an expert's assignments in token order, up to its capacity
    C = m.moe_capacity(T, E, 1.5)
    flat = idx.flatten().tolist()
    seen, slots = [0] * E, []
    for e in flat:
        slots.append(seen[e] if seen[e] < C else -1)
        seen[e] += 1
    start = np.cumsum([0] + [min(s, C) for s in seen])
    want = torch.tensor([start[e] + r if r >= 0 else -1 for e, r in zip(flat, slots)], device="cuda").view(T, k)
    assert torch.equal(st["slot"].long(), want) and st["offsets"].tolist() == start.tolist()
    y = torch.zeros((T, d), dtype=torch.float64, device="cuda")
    ytol = torch.zeros_like(y)
    for e in range(E):
        n = min(seen[e], C)
        if n:
            rows = slice(int(start[e]), int(start[e]) + n)
            o, tol = ref_ffn8(st["x"][st["perm"][rows].long()], values8(b["W1"][e], b["s1"][e]), values8(b["W2"][e], b["s2"][e]), d, f)
            check(st["y"][rows], o, tol + 2.0 ** -11 * o.abs() + 2.0 ** -25, "expert rows")
    _, ym, _, _, z, h, _, n = ref_norm(b["res"], st["y"], st["slot"], st["w"], None, b["wp"], b["gate"], 0.5, b["w1"], 1e-5,
                                       st["y"].shape[0])
    check(st["h"], h, 1e-5 * (h.abs() + 1) + 2.0 ** -11 * h.abs(), "h")
    check(st["n"], n, 1e-5 * (n.abs() + 1) + 2.0 ** -11 * n.abs(), "n")


@pytest.mark.parametrize("T,d,f", [(130, 256, 256), (2, 1024, 2048), (1500, 1024, 4096)])
def test_block_captured_and_eager(m, T, d, f):
    """A captured step with inputs that change between replays, eager calls of another state between them, and two
    states on two streams: the same bits as eager calls one after another."""
    b = block_inputs(m, T, d, f, 16, 4, 6)
    st, plain = block_state(m, b), block_state(m, b)
    block_step(m, b, st)                              # (first calls set kernels up outside of a capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block_step(m, b, st)
    for seed in (1, 2):
        b["res"].copy_(randn(gen(seed), T, d, dtype=torch.float16))
        block_step(m, b, plain)
        graph.replay()
        torch.cuda.synchronize()
        for q in RESULTS:
            assert torch.equal(st[q], plain[q]), q
    two = [block_state(m, b) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, t in zip(streams, two):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            block_step(m, b, t)
    torch.cuda.synchronize()
    for t in two:
        for q in RESULTS:
            assert torch.equal(t[q], plain[q]), q


@pytest.mark.parametrize("k", [3, 8, 16])
@pytest.mark.parametrize("T,E,cf", [(1, 16, 1.0), (77, 16, 0.5), (500, 64, float("inf")), (5000, 33, 1.25)])
def test_dispatch_of_many_experts(m, T, E, k, cf):
    """moe_dispatch beyond two experts a token."""
    g = gen(T + k)
    idx = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    idx[torch.rand((T, k), generator=g, device="cuda") < 0.1] = -1
    C = m.moe_capacity(T, E, cf)
    S = min(T * k, E * C)
    i = dict(dtype=torch.int32, device="cuda")
    counts, kept, off, perm = torch.zeros(E, **i), torch.zeros(E, **i), torch.zeros(E + 1, **i), torch.full((S,), -9, **i)
    slot = torch.zeros((T, k), **i)
    m.moe_dispatch(idx, E, cf, counts, kept, off, perm, slot)
    flat = idx.flatten().cpu().numpy()
    seen = np.bincount(flat[flat >= 0], minlength=E)
    start = np.concatenate([[0], np.cumsum(np.minimum(seen, C))])
    assert counts.tolist() == seen.tolist() and off.tolist() == start.tolist()
    run = [0] * E
    want, tok = np.full(T * k, -1), {}
    for a, e in enumerate(flat):
        if e >= 0:
            if run[e] < C:
                want[a] = start[e] + run[e]
                tok[want[a]] = a // k
            run[e] += 1
    assert slot.flatten().tolist() == want.tolist()
    assert perm[:start[-1]].tolist() == [tok[s] for s in range(start[-1])]
