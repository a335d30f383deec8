"""Router losses, gate / combine gradients and low-rank adapters against plain 64-bit formulas.

Tolerances.  u = 2^-24 is half a step of float32, h = eps / 2 the half step of the output type.
A sum of n float32 terms in any order is off by at most n u times the sum of their magnitudes;
the tensor cores' additions truncate, i.e. up to 2 u each.  Each check therefore allows
K u (sum of magnitudes) + h |value| with K counted beside it.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


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


# ---------------------------------------------------------------- router
def ref_losses(logits, idx, mask):
    x = logits.double()
    T, E = x.shape
    k = idx.shape[1]
    on = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    empty = torch.isneginf(x).all(1)
    p = torch.softmax(torch.where(empty[:, None], torch.zeros_like(x), x), 1) * (~empty)[:, None]
    lse = torch.where(empty, torch.zeros_like(x[:, 0]), torch.logsumexp(x, 1))
    p, lse = p[on], lse[on]
    n = int(on.sum())
    ii = idx[on].long().flatten()
    ii = ii[(ii >= 0) & (ii < E)]
    counts = torch.bincount(ii, minlength=E)
    P = p.sum(0) / max(n, 1)
    bal = E * (counts.double() / (max(n, 1) * k) * P).sum()
    return counts, P, torch.stack([bal, lse.square().sum() / max(n, 1)]), n


def ref_dlogits(logits, idx, mask, counts, n, dlosses, dw):
    """Autograd of the definition in 64 bits (rows that do not count: zero)."""
    x = logits.double().clone()
    T, E = x.shape
    k = idx.shape[1]
    on = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    use = on & ~torch.isneginf(x).all(1)
    out = torch.zeros_like(x)
    if not use.any():
        return out
    xs = x[use].requires_grad_()
    total = 0
    logp = torch.log_softmax(xs, 1)
    if dlosses is not None:
        g = dlosses.double()
        n = max(n, 1)
        total = g[0] * E * (counts.double() / (n * k) * logp.exp().sum(0) / n).sum()
        total = total + g[1] * torch.logsumexp(xs, 1).square().sum() / n
    if dw is not None:
        ii, w = idx[use].long(), dw[use].double()
        ok = ((ii >= 0) & (ii < E)).all(1) if k == 2 else ((ii >= 0) & (ii < E))[:, 0]
        if k == 2:
            ok &= ii[:, 0] != ii[:, 1]
        sel = logp[ok].gather(1, ii[ok])
        ww = sel.exp() if k == 1 else torch.softmax(sel, 1)
        total = total + (ww * w[ok]).sum()
    (gr,) = torch.autograd.grad(total, xs)
    out[use] = gr
    return out


def run_balance(m, logits, idx, mask=None):
    T, E = logits.shape
    counts = torch.full((E,), -7, dtype=torch.int32, device="cuda")
    P = torch.full((E,), float("nan"), device="cuda")
    losses = torch.full((2,), float("nan"), device="cuda")
    nv = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    ws = torch.full((m.moe_balance_workspace_size(T, E),), 0xA5, dtype=torch.uint8, device="cuda")
    m.moe_balance_loss(logits, idx, counts, P, losses, nv, ws, token_mask=mask)
    return counts, P, losses, nv


def topk(logits, k):
    return torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()


SHAPES = [(1, 1), (1, 2), (2, 3), (7, 4), (64, 8), (33, 16), (100, 17), (129, 31), (65, 32), (77, 33),
          (1000, 60), (50, 64), (201, 65), (513, 127), (3000, 128), (90, 129), (40, 255), (70, 256),
          (31, 257), (25, 512), (19, 513), (11, 1000), (13, 1023), (300, 1024), (20000, 128),
          (70001, 5), (9999, 36), (2500, 257)]


@pytest.mark.parametrize("T,E", SHAPES)
@pytest.mark.parametrize("k", [1, 2])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_and_its_gradient(m, T, E, k, masked):
    k = min(k, E)
    g = gen(T * 1031 + E)
    logits = randn(g, T, E, sigma=2.0)
    idx = topk(logits, k)
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7) if masked else None
    if masked:
        logits[~mask] = float("nan")                 # what padding rows hold has no effect
    counts, P, losses, nv = run_balance(m, logits, idx, mask)
    rc, rP, rl, rn = ref_losses(logits, idx, mask)
    assert int(nv) == rn and torch.equal(counts.long(), rc)
    # p: exponent and sum within 8 u each (|x - max| <= 32 costs the subtraction nothing; expf is
    # within 2 ulp, E <= 1024 terms summed as a tree of <= 32 + 5 steps); the mean over T rows is
    # summed in <= T / 4000 + 40 steps
    K = 64 + T / 4000
    check(P, rP, K * U * rP + 1e-37, "prob_mean")
    check(losses, rl, (K + 80) * U * rl.abs() + 1e-37, "losses")
    dl = torch.full((T, E), float("nan"), device="cuda")
    dloss = torch.tensor([0.7, -0.3], device="cuda")
    dw = randn(g, T, k)
    m.moe_gate_topk_backward(logits, idx, dl, dtopk_w=dw, dlosses=dloss, counts=counts, n_valid=nv,
                             token_mask=mask)
    clean = logits if mask is None else torch.where(mask[:, None], logits, torch.zeros_like(logits))
    want = ref_dlogits(clean, idx, mask, rc, rn, dloss, dw)
    # magnitudes: every term of a row's gradient is at most p (|a| + sum |a| p + |2 g_z lse / n| + |dw|)
    # plus |dw| at the chosen experts
    a = 0.7 * E * rc.double() / (max(rn, 1) ** 2 * k)
    p = torch.softmax(clean.double(), 1)
    lse = torch.logsumexp(clean.double(), 1, keepdim=True)
    mag = p * (a + (a * p).sum(1, keepdim=True) + (0.6 / max(rn, 1)) * lse.abs() +
               dw.abs().double().sum(1, keepdim=True))
    mag.scatter_add_(1, idx.long(), dw.abs().double().sum(1, keepdim=True).expand(T, k).contiguous())
    check(dl, want, 64 * U * mag + 1e-37, "dlogits")
    if mask is not None:
        assert not dl[~mask].any()


@pytest.mark.parametrize("E", [8, 13, 128])
def test_router_odd_values(m, E):
    g = gen(E)
    T = 40
    logits = randn(g, T, E)
    low = torch.finfo(torch.float32).min
    logits[0] = float("-inf")                        # nothing left: adds nothing, counts as a token
    logits[1, 1:] = float("-inf")                    # one expert left
    logits[2] = low                                  # the type's lowest value everywhere
    logits[3, : E // 2] = low
    logits[4] = 80.0 * torch.arange(E, device="cuda")
    logits[5] = -logits[4]
    logits[6] = 0.0
    idx = topk(logits, 2)
    idx[7, 0] = -1                                   # outside: not counted, no gradient
    idx[8, 1] = E
    idx[9, 1] = idx[9, 0]                            # the same expert twice
    counts, P, losses, nv = run_balance(m, logits, idx)
    rc, rP, rl, rn = ref_losses(logits, idx, None)
    assert int(nv) == rn == T and torch.equal(counts.long(), rc)
    check(P, rP, 64 * U * rP + 1e-37, "prob_mean")
    check(losses[:1], rl[:1], 160 * U * rl[:1].abs(), "balance")
    assert torch.isinf(losses[1])                    # lse^2 of the lowest value overflows, as it should
    dl = torch.empty_like(logits)
    dw = randn(g, T, 2)
    dloss = torch.tensor([1.0, 0.0], device="cuda")
    m.moe_gate_topk_backward(logits, idx, dl, dtopk_w=dw, dlosses=dloss, counts=counts, n_valid=nv)
    want = ref_dlogits(logits, idx, None, rc, rn, dloss, dw)
    assert torch.isfinite(dl).all()
    check(dl, want, 64 * U * (1 + dw.abs().double().sum(1, keepdim=True)), "dlogits")
    assert not dl[0].any()
    # NaN and +inf propagate to their own row only
    logits2 = logits.clone()
    logits2[10, 3], logits2[11, 2] = float("nan"), float("inf")
    dl2 = torch.empty_like(dl)
    m.moe_gate_topk_backward(logits2, idx, dl2, dtopk_w=dw, dlosses=dloss, counts=counts, n_valid=nv)
    assert dl2[10].isnan().any() and dl2[11].isnan().any()
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[10:12] = False
    assert torch.equal(dl2[keep], dl[keep])


def test_balance_no_token_counts_and_empty_batch(m):
    logits = torch.full((5, 6), float("nan"), device="cuda")
    idx = torch.zeros((5, 1), dtype=torch.int32, device="cuda")
    mask = torch.zeros(5, dtype=torch.uint8, device="cuda")
    for T in (5, 0):
        counts, P, losses, nv = run_balance(m, logits[:T], idx[:T], mask[:T])
        assert not counts.any() and not P.any() and not losses.any() and int(nv) == 0
    dl = torch.full((5, 6), 3.0, device="cuda")
    m.moe_gate_topk_backward(logits, idx, dl, dlosses=torch.ones(2, device="cuda"), counts=counts,
                             n_valid=nv, token_mask=mask)
    assert not dl.any()


def test_dlogits_against_differences(m):
    """Central differences of the losses that the library itself returns (in 64 bits around it)."""
    g = gen(3)
    T, E, k = 6, 10, 2
    logits = randn(g, T, E)
    idx = topk(logits, k)
    counts, P, losses, nv = run_balance(m, logits, idx)
    dw = randn(g, T, k)
    dloss = torch.tensor([0.5, 0.25], device="cuda")
    dl = torch.empty_like(logits)
    m.moe_gate_topk_backward(logits, idx, dl, dtopk_w=dw, dlosses=dloss, counts=counts, n_valid=nv)

    def total(x):
        p = torch.softmax(x, 1)
        bal = E * (counts.double() / (T * k) * p.mean(0)).sum()
        z = torch.logsumexp(x, 1).square().mean()
        w = torch.softmax(x.gather(1, idx.long()), 1)
        return 0.5 * bal + 0.25 * z + (w * dw.double()).sum()
    x = logits.double()
    h = 1e-5
    for t in range(T):
        for e in range(E):
            d = torch.zeros_like(x)
            d[t, e] = h
            num = (total(x + d) - total(x - d)) / (2 * h)
            assert abs(float(num) - float(dl[t, e])) < 1e-6      # h^2 + 64 u |terms|, terms < 4


GATE = [("f16", 1, 128, 4, 1), ("f16", 5, 8, 1, 1), ("f16", 63, 136, 7, 2), ("f16", 64, 128, 16, 1),
        ("f16", 65, 264, 33, 2), ("f16", 300, 1024, 128, 1), ("f16", 1000, 256, 129, 2),
        ("f16", 2049, 128, 64, 1), ("f16", 130, 392, 1000, 2), ("f16", 257, 520, 256, 2), ("f16", 1300, 776, 190, 1), ("f16", 4096, 1024, 128, 2),
        ("f32", 1, 4, 2, 1), ("f32", 128, 64, 4, 1), ("f32", 77, 68, 13, 2), ("f32", 500, 252, 130, 1),
        ("f32", 2048, 64, 8, 2)]


# where the two forms change over, on both sides, and small ones of the tensor-core form
GATE += [("f16", 16, 136, 256, 2), ("f16", 15, 136, 256, 2), ("f16", 40, 264, 128, 1), ("f16", 64, 8, 64, 2),
         ("f16", 512, 72, 8, 2), ("f16", 511, 72, 8, 2), ("f16", 2048, 264, 2, 1), ("f16", 2521, 136, 13, 2),
         ("f16", 129, 72, 255, 2), ("f16", 128, 72, 255, 2), ("f16", 4097, 64, 4, 1), ("f16", 100, 128, 60, 2), ("f16", 1, 1024, 128, 2),
         ("f16", 3, 264, 256, 2), ("f16", 17, 136, 127, 1), ("f16", 256, 2048, 128, 2), ("f16", 513, 72, 127, 2)]


def gate_inputs(g, dt, T, d, E, k):
    x = randn(g, T, d, dtype=dt)
    Wg = randn(g, d, E, sigma=0.1)
    logits = (x.double() @ Wg.double()).float()
    return x, Wg, logits, topk(logits, k), randn(g, T, k)


@pytest.mark.parametrize("dt,T,d,E,k", GATE)
@pytest.mark.parametrize("form", ["all", "weights", "tokens"])
def test_gate_backward(m, dt, T, d, E, k, form):
    dt = {"f16": torch.float16, "f32": torch.float32}[dt]
    g = gen(T + 7 * d + E)
    x, Wg, logits, idx, dw = gate_inputs(g, dt, T, d, E, k)
    dw[:: 3] *= 1e-6                                 # gradients of very different sizes in one sum
    dx_in = randn(g, T, d, dtype=dt) if form == "all" else None
    ws = torch.empty(m.moe_gate_backward_workspace_size(T, d, E, dt), dtype=torch.uint8, device="cuda")
    dl = torch.full((T, E), float("nan"), device="cuda")
    dWg = torch.full((d, E), float("nan"), device="cuda") if form != "tokens" else None
    dx = torch.full((T, d), float("nan"), device="cuda", dtype=dt) if form != "weights" else None
    m.moe_gate_topk_backward(logits, idx, dl, dtopk_w=dw, tokens=x, Wg=Wg, dWg=dWg, dtokens=dx,
                             dtokens_in=dx_in, workspace=ws)
    assert m.moe_status_read(ws) == m.MOE_OK
    check(dl, ref_dlogits(logits, idx, None, None, T, None, dw),
          64 * U * (dw.abs().double().sum(1, keepdim=True) + 1e-30), "dlogits")
    dd = dl.double()                                 # the products are checked on the dl they had
    if dWg is not None:
        mag = x.double().abs().t() @ dd.abs()
        # f16: dl keeps 22 bits of its chunk's largest value (2 u of it); <= 8 truncating additions per
        # chunk of 64 rows, then chunks and blocks: T / 64 + 16.  f32: T additions at most
        cmax = torch.cat([c.abs().amax(0, keepdim=True).expand(1, E).amax() * c.abs().new_ones(len(c), 1)
                          for c in dd.split(64)])
        slack = (x.double().abs() * cmax).sum(0)[:, None]
        tol = (64 + T / 64) * U * mag + 4 * U * slack if dt == torch.float16 else (T + 8) * U * mag
        check(dWg, x.double().t() @ dd, tol + 1e-37, "dWg")
    if dx is not None:
        want = dd @ Wg.double().t()
        mag = dd.abs() @ Wg.double().abs().t()
        if dx_in is not None:
            want, mag = want + dx_in.double(), mag + dx_in.double().abs()
        # E additions; f16: dl good to 2^-23 of itself and 2^-36 of the largest value of its 128 rows,
        # Wg rounded to f16 once (2^-11; 2^-25 of the largest of 128 rows below f16's range)
        block = lambda v: torch.cat([c.abs().amax().expand(len(c)) for c in v.split(128)])
        slack = 2.0 ** -36 * block(dd)[:, None] * Wg.double().abs().sum(1) + \
            2.0 ** -25 * dd.abs().sum(1, keepdim=True) * block(Wg.double())
        K = 2 * E + 64 + (2 ** 13 if dt == torch.float16 else 0)
        tol = K * U * mag + slack + torch.finfo(dt).eps / 2 * want.abs()
        check(dx, want, tol + (2.0 ** -25 if dt == torch.float16 else 1e-37), "dtokens")


@pytest.mark.parametrize("dt,T,d,E,k", [c for c in GATE if c[0] == "f16"] + [("f16", 700, 1408, 256, 2), ("f16", 700, 1408, 255, 1)])
@pytest.mark.parametrize("with_dWg", [False, True])
def test_gate_dtokens_keep_32_bit_accuracy(m, dt, T, d, E, k, with_dWg):
    """Beside the output's own rounding only what 32-bit sums lose is left, whether dWg is asked for or not."""
    g = gen(T + 7 * d + E + 3)
    dt = torch.float16
    x, Wg, logits, idx, dw = gate_inputs(g, dt, T, d, E, k)
    ws = torch.empty(m.moe_gate_backward_workspace_size(T, d, E, dt), dtype=torch.uint8, device="cuda")
    dl, dx = torch.empty((T, E), device="cuda"), torch.empty((T, d), dtype=dt, device="cuda")
    dWg = torch.empty((d, E), device="cuda") if with_dWg else None
    m.moe_gate_topk_backward(logits, idx, dl, dtopk_w=dw, tokens=x, Wg=Wg, dWg=dWg, dtokens=dx, workspace=ws)
    dd, W = dl.double(), Wg.double()
    want, mag = dd @ W.t(), dd.abs() @ W.abs().t()
    # two parts each: 2 u of either operand and of their low parts' product, 2^-36 of the largest of 128
    # rows; E additions at two units each at most (f16 products: chains of 3 E / 16 and one join)
    block = lambda v: torch.cat([c.abs().amax().expand(len(c)) for c in v.split(128)])
    slack = 2.0 ** -36 * (block(dd)[:, None] * W.abs().sum(1) + dd.abs().sum(1, keepdim=True) * block(W))
    tol = (2 * E + 64) * U * mag + slack + 2.0 ** -11 * want.abs() * (1 + 2 ** -10) + 2.0 ** -25
    check(dx, want, tol, "dtokens")


def test_gate_backward_masked_rows_and_in_place(m):
    g = gen(5)
    T, d, E, k = 200, 128, 24, 2
    x, Wg, logits, idx, dw = gate_inputs(g, torch.float16, T, d, E, k)
    mask = torch.rand(T, generator=g, device="cuda") < 0.6
    x[~mask] = float("nan")                          # padding rows hold anything
    logits[~mask] = float("inf")
    ws = torch.empty(m.moe_gate_backward_workspace_size(T, d, E, x.dtype), dtype=torch.uint8, device="cuda")
    dl, dWg = torch.empty((T, E), device="cuda"), torch.empty((d, E), device="cuda")
    dx = randn(g, T, d, dtype=torch.float16)
    before = dx.clone()
    m.moe_gate_topk_backward(logits, idx, dl, dtopk_w=dw, token_mask=mask, tokens=x, Wg=Wg, dWg=dWg,
                             dtokens=dx, dtokens_in=dx, workspace=ws)
    assert torch.isfinite(dWg).all() and not dl[~mask].any()
    assert torch.equal(dx[~mask], before[~mask])
    want = x[mask].double().t() @ dl[mask].double()
    mag = x[mask].double().abs().t() @ dl[mask].double().abs()
    check(dWg, want, 80 * U * (mag + x[mask].double().abs().sum(0)[:, None] * dl.abs().max().double()), "dWg")
    dWg0 = torch.ones((d, E), device="cuda")         # an empty batch clears the sum
    m.moe_gate_topk_backward(logits[:0], idx[:0], dl[:0], dtopk_w=dw[:0], tokens=x[:0], Wg=Wg, dWg=dWg0,
                             workspace=ws)
    assert not dWg0.any()


@pytest.mark.parametrize("T,d,E", [(1, 8, 4), (70, 136, 64), (130, 264, 128), (1000, 520, 128), (4100, 1024, 64),
                                   (2050, 776, 255), (700, 392, 300), (900, 3584, 256)])
@pytest.mark.parametrize("kind", ["some", "blocks", "tail", "one", "none"])
@pytest.mark.parametrize("form", ["all", "weights"])
def test_gate_backward_masks(m, T, d, E, kind, form):
    """Masked tokens hold NaN and infinities: they add nothing to dWg, and their dlogits are zero."""
    g = gen(T + d + E)
    x, Wg, logits, idx, dw = gate_inputs(g, torch.float16, T, d, E, 2)
    t = torch.arange(T, device="cuda")
    mask = {"some": torch.rand(T, generator=g, device="cuda") < 0.7, "blocks": (t // 64) % 3 != 1,
            "tail": t < (T * 5) // 8, "one": t == T // 2, "none": t < 0}[kind]
    x[~mask] = torch.where(t[~mask] % 2 == 0, float("nan"), float("inf"))[:, None].half()
    logits[~mask] = float("nan")
    ws = torch.empty(m.moe_gate_backward_workspace_size(T, d, E, x.dtype), dtype=torch.uint8, device="cuda")
    dl, dWg = torch.full((T, E), 5.0, device="cuda"), torch.full((d, E), 5.0, device="cuda")
    dx = randn(g, T, d, dtype=torch.float16) if form == "all" else None
    before = dx.clone() if form == "all" else None
    m.moe_gate_topk_backward(logits, idx, dl, dtopk_w=dw, token_mask=mask, tokens=x, Wg=Wg, dWg=dWg,
                             dtokens=dx, dtokens_in=dx, workspace=ws)
    assert m.moe_status_read(ws) == m.MOE_OK
    assert not dl[~mask].any() and torch.isfinite(dl).all()
    xd, dd = x[mask].double(), dl[mask].double()
    mag = xd.abs().t() @ dd.abs()
    top = dd.abs().max() if len(dd) else 0           # as in test_gate_backward, by the largest of all rows
    check(dWg, xd.t() @ dd, (64 + T / 64) * U * mag + 4 * U * xd.abs().sum(0)[:, None] * top, "dWg")
    if form == "all":
        assert torch.equal(dx[~mask], before[~mask])
        want = before[mask].double() + dd @ Wg.double().t()
        mag = before[mask].double().abs() + dd.abs() @ Wg.double().abs().t()
        check(dx[mask], want, 2.0 ** -11 * 1.02 * (want.abs() + mag) + 2.0 ** -24 + 2.0 ** -36 * top * d, "dtokens")


@pytest.mark.parametrize("T", [40, 300])
def test_gate_backward_infinities_stay_where_they_are(m, T):
    """A token whose gradient is NaN spoils its own row of dtokens and nothing of the others'."""
    g = gen(T)
    d, E = 136, 20
    x, Wg, logits, idx, dw = gate_inputs(g, torch.float16, T, d, E, 2)
    dw *= 1e-7                                       # small beside what a NaN might leave unscaled
    ws = torch.empty(m.moe_gate_backward_workspace_size(T, d, E, x.dtype), dtype=torch.uint8, device="cuda")
    out = []
    for bad in (False, True):
        if bad:
            logits = logits.clone()
            logits[5, 3] = float("nan")
        dl, dWg = torch.empty((T, E), device="cuda"), torch.empty((d, E), device="cuda")
        dx = torch.empty((T, d), dtype=torch.float16, device="cuda")
        m.moe_gate_topk_backward(logits, idx, dl, dtopk_w=dw * 1e3, tokens=x, Wg=Wg, dWg=dWg, dtokens=dx, workspace=ws)
        out.append((dl, dWg, dx))
    keep = torch.arange(T, device="cuda") != 5
    assert out[1][2][5].isnan().any() and torch.equal(out[1][2][keep], out[0][2][keep])
    assert torch.equal(out[1][0][keep], out[0][0][keep])
    # columns of dWg that no NaN reaches are those of the batch without that token
    clean = ~out[1][0][5].isnan()
    dd = out[1][0][keep].double()
    want, mag = x[keep].double().t() @ dd, x[keep].double().abs().t() @ dd.abs()
    add = x[5].double()[:, None] * out[1][0][5].double().nan_to_num()[None]
    tol = 80 * U * (mag + add.abs() + x.double().abs().sum(0)[:, None] * dd.abs().max())
    check(out[1][1][:, clean], (want + add)[:, clean], tol[:, clean], "dWg")


@pytest.mark.parametrize("T,cut,d,E,k", [(500, 130, 136, 24, 2), (3000, 2999, 264, 128, 1), (900, 450, 64, 300, 2)])
@pytest.mark.parametrize("masked", [False, True])
def test_one_batch_over_two_callers(m, T, cut, d, E, k, masked):
    """Each caller has a part of the batch's tokens: with counts and n_valid summed over both first, the
    gradients of their rows are the whole batch's, and their dWg add up to its."""
    g = gen(T + E)
    x, Wg, logits, idx, dw = gate_inputs(g, torch.float16, T, d, E, k)
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7) if masked else None
    dloss = torch.tensor([0.7, -0.3], device="cuda")
    parts = [slice(0, cut), slice(cut, T)]
    cutm = lambda s: None if mask is None else mask[s].clone()
    # (a slice need not start on 16 bytes: a caller has tensors of its own)
    own = [run_balance(m, logits[s].clone(), idx[s].clone(), cutm(s)) for s in parts]
    counts, nv = own[0][0] + own[1][0], own[0][3] + own[1][3]
    whole = run_balance(m, logits, idx, mask)
    assert torch.equal(counts, whole[0]) and torch.equal(nv, whole[3])
    # the losses from the parts' means: prob_mean and z weighted by their tokens
    w = [o[3].double() / max(int(nv), 1) for o in own]
    P = w[0] * own[0][1] + w[1] * own[1][1]
    check(P, whole[1].double(), 128 * U * P + 1e-37, "prob_mean")
    bal = E * (counts.double() / (max(int(nv), 1) * k) * P).sum()
    check(whole[2], torch.stack([bal, (w[0] * own[0][2][1] + w[1] * own[1][2][1])[0]]), 256 * U * whole[2].double().abs(), "losses")

    def back(s, mk):
        n = logits[s].shape[0]
        ws = torch.empty(m.moe_gate_backward_workspace_size(n, d, E, x.dtype), dtype=torch.uint8, device="cuda")
        dl, dWg = torch.full((n, E), 5.0, device="cuda"), torch.full((d, E), 5.0, device="cuda")
        m.moe_gate_topk_backward(logits[s].clone(), idx[s].clone(), dl, dtopk_w=dw[s].clone(), dlosses=dloss, counts=counts,
                                 n_valid=nv, token_mask=mk, tokens=x[s].clone(), dWg=dWg, workspace=ws)
        return dl, dWg
    a, b = (back(s, cutm(s)) for s in parts)
    dl, dWg = back(slice(0, T), mask)
    clean = logits if mask is None else torch.where(mask[:, None], logits, torch.zeros_like(logits))
    want = ref_dlogits(clean, idx, mask, counts, int(nv), dloss, dw)
    got = torch.cat([a[0], b[0]])
    # as in test_balance_and_its_gradient
    c = 0.7 * E * counts.double() / (max(int(nv), 1) ** 2 * k)
    p = torch.softmax(clean.double(), 1)
    lse = torch.logsumexp(clean.double(), 1, keepdim=True)
    mag = p * (c + (c * p).sum(1, keepdim=True) + 0.6 / max(int(nv), 1) * lse.abs() + dw.abs().double().sum(1, keepdim=True))
    mag.scatter_add_(1, idx.long(), dw.abs().double().sum(1, keepdim=True).expand(T, k).contiguous())
    check(got, want, 64 * U * mag + 1e-37, "dlogits of the parts")
    check(dl, want, 64 * U * mag + 1e-37, "dlogits of the batch")
    xd, dd = x.double(), got.double()
    both = (64 + T / 64 + 2) * U * (xd.abs().clamp(min=2.0 ** -14).t() @ dd.abs()) + 2.0 ** -36 * xd.abs().sum(0)[:, None] * dd.abs().max()
    check(a[1].double() + b[1].double(), xd.t() @ dd, both + 1e-37, "dWg of the parts")


# ---------------------------------------------------------------- combine
@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
@pytest.mark.parametrize("T,d,k", [(1, 8, 1), (3, 7, 2), (64, 128, 2), (129, 1001, 1), (1000, 264, 2),
                                   (5000, 72, 2), (2433, 8, 1), (40, 3584, 2)])
@pytest.mark.parametrize("form", ["both", "dy", "dw"])
def test_combine_backward(m, dt, T, d, k, form):
    g = gen(T + d)
    kept = torch.rand((T, k), generator=g, device="cuda") < 0.8
    S = int(kept.sum())
    slot = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    slot[kept.flatten()] = torch.randperm(S, generator=g, device="cuda").to(torch.int32)
    slot = slot.view(T, k)
    w = torch.rand((T, k), generator=g, device="cuda")
    dout, y = randn(g, T, d, dtype=dt), randn(g, T * k + 3, d, dtype=dt)
    y[S:] = float("nan")                             # behind the last slot: not read
    dy = torch.full((T * k + 3, d), 7.0, dtype=dt, device="cuda") if form != "dw" else None
    dw = torch.full((T, k), float("nan"), device="cuda") if form != "dy" else None
    m.moe_combine_backward(dout, y if dw is not None else None, slot, w if dy is not None else None, dy, dw)
    dd, yy = dout.double(), y.double()
    if dw is not None:
        ii = slot.long().clamp(min=0)
        prod = dd[:, None, :] * yy[ii] * (slot >= 0)[:, :, None]
        prod = torch.where((slot >= 0)[:, :, None], prod, torch.zeros_like(prod))
        check(dw, prod.sum(2), (d / 32 + 16) * U * prod.abs().sum(2) + 1e-37, "dtopk_w")
    if dy is not None:
        want = torch.full_like(yy, 7.0)
        for j in range(k):
            on = slot[:, j] >= 0
            want[slot[on, j].long()] = w[on, j].double()[:, None] * dd[on]
        # rounded to 32 bits, then to the type
        check(dy, want, want.abs() * (torch.finfo(dt).eps / 2 + U) + (2.0 ** -25 if dt == torch.float16 else 0),
              "dexpert_out")
        assert (dy[S:] == 7.0).all()


def test_combine_backward_slots_outside_are_dropped(m):
    dout = torch.ones((4, 8), device="cuda")
    y = torch.ones((2, 8), device="cuda")
    slot = torch.tensor([[0], [2], [1 << 30], [-5]], dtype=torch.int32, device="cuda")
    w = torch.full((4, 1), 0.5, device="cuda")
    dy, dw = torch.zeros_like(y), torch.full((4, 1), -1.0, device="cuda")
    m.moe_combine_backward(dout, y, slot, w, dy, dw)
    assert dw.flatten().tolist() == [8.0, 0.0, 0.0, 0.0]
    assert dy[0].eq(0.5).all() and dy[1].eq(0).all()


# ---------------------------------------------------------------- adapters
def plan(m, ids, N):
    """perm and offsets of adapter ids, by the library's own dispatch."""
    T = ids.numel()
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, kept, off = torch.zeros(N, **i32), torch.zeros(N, **i32), torch.zeros(N + 1, **i32)
    perm, slot = torch.zeros(T, **i32), torch.zeros((T, 1), **i32)
    m.moe_dispatch(ids.view(T, 1), N, float("inf"), counts, kept, off, perm, slot)
    return perm, off


def adapter_inputs(m, g, dt, T, di, do, r, N, none=0.2, one=False):
    ids = torch.randint(0, N, (T,), generator=g, device="cuda", dtype=torch.int32)
    if one:
        ids[:] = N - 1
    ids[torch.rand(T, generator=g, device="cuda") < none] = -1
    perm, off = plan(m, ids, N)
    return dict(ids=ids, perm=perm, off=off, x=randn(g, T, di, dtype=dt),
                A=randn(g, N, di, r, sigma=di ** -0.5, dtype=dt), B=randn(g, N, r, do, sigma=0.3, dtype=dt),
                scale=randn(g, N, sigma=1.5), base=randn(g, T, do, dtype=dt))


def adapter_ws(m, T, di, do, r, N, dt):
    return torch.full((m.moe_adapter_workspace_size(T, di, do, r, N, T, dt),), 0x5A, dtype=torch.uint8,
                      device="cuda")


def tiny(dt):
    return 2.0 ** -25 if dt == torch.float16 else 1e-37


ADAPT = [("f16", 1, 8, 8, 8, 1), ("f16", 1, 1024, 1024, 16, 32), ("f16", 2, 64, 8, 8, 3), ("f16", 17, 72, 136, 24, 2),
         ("f16", 64, 3584, 264, 16, 64), ("f16", 100, 520, 1000, 40, 1), ("f16", 300, 128, 2048, 64, 5),
         ("f16", 333, 1032, 72, 128, 3), ("f16", 1000, 256, 256, 8, 1000), ("f16", 2000, 200, 328, 104, 7),
         ("f16", 4097, 512, 512, 32, 2), ("f16", 500, 136, 200, 8, 2), ("f16", 3000, 2048, 64, 16, 4),
         ("f16", 700, 64, 1032, 48, 20), ("f16", 65, 128, 128, 128, 1024), ("f32", 1, 4, 4, 8, 1),
         ("f32", 128, 64, 256, 8, 4), ("f32", 33, 68, 100, 24, 3), ("f32", 500, 1028, 36, 64, 9),
         ("f32", 70, 128, 260, 128, 2), ("f32", 1111, 32, 32, 16, 1)]


# long runs of every rank's form, and where short ones change over
ADAPT += [("f16", 1300, 136, 1000, 16, 1), ("f16", 1184, 72, 64, 8, 1), ("f16", 1500, 264, 136, 128, 3),
          ("f16", 1400, 328, 200, 64, 2), ("f16", 900, 1032, 72, 24, 2), ("f16", 784, 128, 264, 64, 1),
          ("f16", 768, 128, 264, 64, 1), ("f16", 600, 64, 72, 112, 1), ("f16", 128, 200, 72, 16, 2)]


@pytest.mark.parametrize("dt,T,di,do,r,N", ADAPT)
@pytest.mark.parametrize("form", ["base", "in_place", "bare", "one"])
def test_adapter_forward(m, dt, T, di, do, r, N, form):
    dt = {"f16": torch.float16, "f32": torch.float32}[dt]
    g = gen(T + di + do + r)
    c = adapter_inputs(m, g, dt, T, di, do, r, N, none=0.0 if form == "one" else 0.2, one=form == "one")
    ws = adapter_ws(m, T, di, do, r, N, dt)
    out = c["base"].clone() if form == "in_place" else torch.full((T, do), 9.0, dtype=dt, device="cuda")
    base = out if form == "in_place" else None if form == "bare" else c["base"]
    hid = torch.full((T, r), 5.0, device="cuda")
    before = out.clone()
    m.moe_adapter_forward(c["x"], c["perm"], c["off"], c["A"], c["B"], c["scale"], out, ws, base=base,
                          hidden=hid)
    assert m.moe_status_read(ws) == m.MOE_OK
    S = int(c["off"][-1])
    assert (hid[S:] == 5.0).all()
    t = c["perm"][:S].long()
    a = c["ids"][t].long()
    for n in a.unique().tolist():
        s = (a == n).nonzero()[:, 0]
        tt = t[s]
        x, A, B, sc = c["x"][tt].double(), c["A"][n].double(), c["B"][n].double(), float(c["scale"][n])
        h = x @ A
        hm = x.abs() @ A.abs()
        # a block sums at most ceil(di / 8 / 64) chunks of four products of 16, the cluster eight blocks,
        # two units per truncating addition (f32: di / 8 + 32 + 8 additions)
        K = 2 * (4 * (di / 512 + 1) + 16) if dt == torch.float16 else di / 8 + 48
        check(hid[s], h, K * U * hm + 1e-37, "hidden")
        y = sc * (h @ B)
        ym = abs(sc) * (hm @ B.abs())
        # h off by K, and for f16 rounded once (2^-11 of each term, values 2^-25 of the row's largest
        # below its range); the second sum r / 4 + 8 additions
        slack = abs(sc) * h.abs().amax(1, keepdim=True) * B.abs().sum(0)
        K2 = K + (r / 2 + 24 + 2 ** 13 * (1 + 2 ** -10) if dt == torch.float16 else r + 8)
        b = c["base"][tt].double() if form != "bare" else torch.zeros_like(y)
        want = b + y
        tol = K2 * U * (ym + b.abs()) + 2 * U * slack + torch.finfo(dt).eps / 2 * want.abs() * (1 + 2 ** -10)
        check(out[tt], want, tol + tiny(dt), "out")
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[t] = False
    assert torch.equal(out[rest], before[rest])


@pytest.mark.parametrize("dt,T,di,do,r,N", ADAPT)
@pytest.mark.parametrize("form", ["all", "dA", "dB", "dx", "one"])
def test_adapter_backward(m, dt, T, di, do, r, N, form):
    dt = {"f16": torch.float16, "f32": torch.float32}[dt]
    g = gen(T + di + do + r + 1)
    c = adapter_inputs(m, g, dt, T, di, do, r, N, none=0.0 if form == "one" else 0.2, one=form == "one")
    ws = adapter_ws(m, T, di, do, r, N, dt)
    dout = randn(g, T, do, sigma=0.1, dtype=dt)
    dout[:: 3] *= 1e-3
    hid = randn(g, T, r)
    din = randn(g, T, di, dtype=dt)
    full = form in ("all", "one")
    dx = torch.full((T, di), 9.0, dtype=dt, device="cuda") if full or form == "dx" else None
    dA = torch.full((N, di, r), float("nan"), device="cuda") if full or form == "dA" else None
    dB = torch.full((N, r, do), float("nan"), device="cuda") if full or form == "dB" else None
    m.moe_adapter_backward(dout, c["x"], hid, c["perm"], c["off"], c["A"], c["B"], c["scale"], ws,
                           dtokens=dx, dtokens_in=din if full else None, dA=dA, dB=dB)
    assert m.moe_status_read(ws) == m.MOE_OK
    S = int(c["off"][-1])
    t = c["perm"][:S].long()
    a = c["ids"][t].long()
    half = dt == torch.float16
    for n in range(N):
        s = (a == n).nonzero()[:, 0]
        if not len(s):
            assert dA is None or not dA[n].any()
            assert dB is None or not dB[n].any()
            continue
        tt = t[s]
        x, dy, A, B = c["x"][tt].double(), dout[tt].double(), c["A"][n].double(), c["B"][n].double()
        sc, H = float(c["scale"][n]), hid[s].double()
        dh, dhm = dy @ B.t(), dy.abs() @ B.abs().t()
        K = 2 * (4 * (do / 512 + 1) + 16) if half else do / 8 + 48
        if dx is not None:
            b = din[tt].double() if full else torch.zeros_like(x)
            want = b + sc * (dh @ A.t())
            mag = abs(sc) * (dhm @ A.abs().t()) + b.abs()
            slack = abs(sc) * dh.abs().amax(1, keepdim=True) * A.abs().sum(1)
            K2 = K + (r / 2 + 24 + 2 ** 13 * (1 + 2 ** -10) if half else r + 8)   # dh rounded, as above
            tol = K2 * U * mag + 2 * U * slack + torch.finfo(dt).eps / 2 * want.abs() * (1 + 2 ** -10)
            check(dx[tt], want, tol + tiny(dt), "dtokens")
        rows = len(s)
        # sums over rows: f16 parts keep 2 u of the largest value of the rows, 8 truncating additions
        # per chunk, rows / 64 + 16 more; f32: one addition per row
        KW = 64 + rows / 64 if half else rows + 16
        if dA is not None:
            mag = x.abs().t() @ dhm
            slack = x.abs().sum(0)[:, None] * dh.abs().max() if half else 0
            check(dA[n], sc * (x.t() @ dh), abs(sc) * ((KW + K) * U * mag + 2 * U * slack) + 1e-37, "dA")
        if dB is not None:
            # an f16 operand below 2^-14 (a subnormal q 2^-24, q < 2^10) enters the tensor core's adder
            # with its stored exponent and leading zeros: the sum of a product keeps its 23 bits below
            # 2^-14 |h|, not below |dy h|, so such an operand counts as 2^-14 in the bound
            dyf = torch.where(dy == 0, dy, dy.abs().clamp(min=2.0 ** -14)) if half else dy.abs()
            mag = H.abs().t() @ dyf
            slack = dyf.sum(0)[None, :] * H.abs().max() if half else 0
            check(dB[n], sc * (H.t() @ dy), abs(sc) * (KW * U * mag + 2 * U * slack) + 1e-37, "dB")
    if dx is not None:
        rest = torch.ones(T, dtype=torch.bool, device="cuda")
        rest[t] = False
        assert (dx[rest] == 9.0).all()


@pytest.mark.parametrize("dt,T,di,do,r,N", [c for c in ADAPT if c[0] == "f16"])
@pytest.mark.parametrize("back", [False, True])
def test_adapter_hidden_rows_keep_32_bit_accuracy(m, dt, T, di, do, r, N, back):
    """The second product takes h (dh) with more than f16's 11 bits: beside the output's own rounding
    only what 32-bit sums lose is left."""
    g = gen(T + di + do + r + 2)
    dt = torch.float16
    c = adapter_inputs(m, g, dt, T, di, do, r, N)
    ws = adapter_ws(m, T, di, do, r, N, dt)
    e, dk = (di, do) if back else (do, di)
    src, out = randn(g, T, dk, dtype=dt), torch.full((T, e), 9.0, dtype=dt, device="cuda")
    if back:
        m.moe_adapter_backward(src, None, None, c["perm"], c["off"], c["A"], c["B"], c["scale"], ws, dtokens=out)
    else:
        m.moe_adapter_forward(src, c["perm"], c["off"], c["A"], c["B"], c["scale"], out, ws)
    t = c["perm"][:int(c["off"][-1])].long()
    a = c["ids"][t].long()
    for n in a.unique().tolist():
        tt = t[(a == n).nonzero()[:, 0]]
        P, Q = (c["B"][n].double().t(), c["A"][n].double().t()) if back else (c["A"][n].double(), c["B"][n].double())
        x, sc = src[tt].double(), float(c["scale"][n])
        h, hm = x @ P, x.abs() @ P.abs()
        y, ym = sc * (h @ Q), abs(sc) * (hm @ Q.abs())
        # h: as in test_adapter_forward.  Its parts leave 2 u of it and 2^-25 of the row's largest; the
        # second chain has r / 8 products of two units each, and the scale and the addition 4 more
        K = 2 * (4 * (dk / 512 + 1) + 16) + r / 2 + 24
        slack = abs(sc) * h.abs().amax(1, keepdim=True) * Q.abs().sum(0)
        tol = K * U * ym + 2 * U * slack + 2.0 ** -11 * y.abs() * (1 + 2 ** -10) + 2.0 ** -25
        check(out[tt], y, tol, "dtokens" if back else "out")


@pytest.mark.parametrize("T,N", [(300, 1), (1500, 3), (70, 1)])
@pytest.mark.parametrize("r", [16, 40, 128])
def test_adapter_gradients_of_small_columns(m, T, N, r):
    """Columns of h far smaller than others (and one row far larger) keep their own bits in dA and dB."""
    g = gen(T + r)
    dt, di, do = torch.float16, 264, 136
    c = adapter_inputs(m, g, dt, T, di, do, r, N, none=0.0)
    # f16 weights and upstream rows in their normal range: dh spans 2^15, hidden 2^30
    j = torch.arange(r, device="cuda") % 16
    c["B"] = (c["B"].float() * 2.0 ** (8 - j.float())[None, :, None]).to(dt)
    dout = randn(g, T, do, dtype=dt)
    hid = randn(g, T, r) * 2.0 ** (-2.0 * j.float())
    hid[T // 2] *= 2.0 ** 8
    ws = adapter_ws(m, T, di, do, r, N, dt)
    dA, dB = torch.empty((N, di, r), device="cuda"), torch.empty((N, r, do), device="cuda")
    m.moe_adapter_backward(dout, c["x"], hid, c["perm"], c["off"], c["A"], c["B"], c["scale"], ws, dA=dA, dB=dB)
    for n in range(N):
        s = slice(int(c["off"][n]), int(c["off"][n + 1]))
        t, sc = c["perm"][s].long(), float(c["scale"][n])
        x, y, h, B = c["x"][t].double(), dout[t].double(), hid[s].double(), c["B"][n].double()
        dh, dhm = y @ B.t(), y.abs() @ B.abs().t()
        rows, K = len(t), 2 * (4 * (do / 512 + 1) + 16)
        # h to 2 u, 8 truncating products per 64 rows (one more for the low part), rows / 64 + 16 additions;
        # 2^-39 of the chunk's largest h; f16 operands below 2^-14 count as that (see test_adapter_backward)
        KW = 66 + rows / 64
        up = lambda v: torch.where(v == 0, v, v.abs().clamp(min=2.0 ** -14))
        check(dA[n], sc * (x.t() @ dh), abs(sc) * ((KW + K) * U * (up(x).t() @ dhm) +
              2.0 ** -39 * up(x).sum(0)[:, None] * dh.abs().max()) + 1e-37, "dA")
        check(dB[n], sc * (h.t() @ y), abs(sc) * (KW * U * (h.abs().t() @ up(y)) +
              2.0 ** -39 * up(y).sum(0)[None, :] * h.abs().max()) + 1e-37, "dB")


@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
@pytest.mark.parametrize("T,E", [(300, 300), (1100, 1000), (70, 300), (300, 64), (2100, 200), (40, 13)])
def test_gate_gradient_of_small_columns(m, dt, T, E):
    """Experts whose probabilities are far below the others' keep their bits in dWg, at every E."""
    g = gen(T + E)
    d = 264
    x = randn(g, T, d, dtype=dt)
    logits = randn(g, T, E) - torch.arange(E, device="cuda") % 24    # p down to 2^-33 of the largest
    idx, dw = topk(logits, 1), randn(g, T, 1)
    dw[T // 2] *= 2.0 ** 8
    ws = torch.empty(m.moe_gate_backward_workspace_size(T, d, E, dt), dtype=torch.uint8, device="cuda")
    dl, dWg = torch.empty((T, E), device="cuda"), torch.empty((d, E), device="cuda")
    m.moe_gate_topk_backward(logits, idx, dl, dtopk_w=dw, tokens=x, dWg=dWg, workspace=ws)
    dd, xd = dl.double(), x.double()
    # as above; the tensor-core form of up to 256 experts: 2^-36 of the largest of 128 rows, separate sums of
    # both parts
    K, low = (70 + T / 64, 2.0 ** -36) if dt == torch.float16 else (T + 8, 0)
    up = xd.abs().clamp(min=2.0 ** -14)
    check(dWg, xd.t() @ dd, K * U * (up.t() @ dd.abs()) + low * up.sum(0)[:, None] * dd.abs().max() + 1e-37, "dWg")


def test_adapter_single_row_gradient_keeps_22_bits(m):
    """One row: dA = scale x dh has one term, so nothing but the operands' precision shows."""
    g = gen(11)
    c = adapter_inputs(m, g, torch.float16, 1, 256, 256, 16, 1, none=0.0)
    ws = adapter_ws(m, 1, 256, 256, 16, 1, torch.float16)
    hid, dout = randn(g, 1, 16), randn(g, 1, 256, dtype=torch.float16)
    dB = torch.empty((1, 16, 256), device="cuda")
    m.moe_adapter_backward(dout, c["x"], hid, c["perm"], c["off"], c["A"], c["B"], c["scale"], ws, dB=dB)
    want = float(c["scale"]) * hid.double().t() @ dout.double()
    check(dB[0], want, 4 * U * want.abs() + 2 * U * hid.abs().max().double() * dout.double().abs() *
          abs(float(c["scale"])), "dB")


@pytest.mark.parametrize("T", [3, 300, 1300])
def test_adapter_wide_range_and_infinities(m, T):
    """h far outside f16's range, and rows with infinities or NaN that leave the others alone."""
    g = gen(T)
    c = adapter_inputs(m, g, torch.float16, T, 128, 128, 16, 1, none=0.0)
    c["x"] = (c["x"].double() * 3e4).clamp(-6e4, 6e4).half()
    c["A"] = (c["A"].double() * 1e3).half()
    c["B"] = (c["B"].double() * 1e-3).half()
    c["scale"][:] = 1e-4
    ws = adapter_ws(m, T, 128, 128, 16, 1, torch.float16)

    def fwd(x):
        out = torch.empty((T, 128), dtype=torch.float16, device="cuda")
        hid = torch.empty((T, 16), device="cuda")
        m.moe_adapter_forward(x, c["perm"], c["off"], c["A"], c["B"], c["scale"], out, ws, base=c["base"],
                              hidden=hid)
        return out, hid
    out, hid = fwd(c["x"])
    assert hid.abs().max() > 65504
    h = c["x"].double() @ c["A"][0].double()
    want = c["base"].double() + 1e-4 * (h @ c["B"][0].double())
    mag = 1e-4 * (c["x"].double().abs() @ c["A"][0].double().abs() @ c["B"][0].double().abs())
    hm = 1e-4 * (h.abs() @ c["B"][0].double().abs())          # h is rounded to f16 once
    check(out, want, 2.0 ** -11 * (want.abs() + hm) * 1.001 + 128 * U * (mag + 1) + 2.0 ** -25, "out")
    x2 = c["x"].clone()
    x2[1, 5], x2[2, 7] = float("inf"), float("nan")
    out2, _ = fwd(x2)
    assert not torch.isfinite(out2[1]).any() and out2[2].isnan().all()
    assert torch.equal(out2[0], out[0]) and torch.equal(out2[3:], out[3:])
    # a NaN in one column of hidden reaches that column of dB only, whatever its rows' scale
    hid2 = torch.randn(hid.shape, generator=g, device="cuda") * 1e-6
    dy = randn(g, T, 128, dtype=torch.float16)
    dB = [torch.empty((1, 16, 128), device="cuda") for _ in range(2)]
    for q in range(2):
        if q:
            hid2[2, 7] = float("nan")
        m.moe_adapter_backward(dy, c["x"], hid2, c["perm"], c["off"], c["A"], c["B"], c["scale"], ws, dB=dB[q])
    keep = torch.arange(16, device="cuda") != 7
    assert dB[1][0, 7].isnan().all()
    t = c["perm"].long()
    want = 1e-4 * hid2.double().t() @ dy[t].double()
    mag = 1e-4 * hid2.double().nan_to_num().abs().t() @ dy[t].double().abs().clamp(min=2.0 ** -14)
    slack = 1e-4 * dy[t].double().abs().clamp(min=2.0 ** -14).sum(0) * hid2.nan_to_num().abs().max()
    check(dB[1][0][keep], want[keep], 80 * U * mag[keep] + 2 * U * slack + 1e-37, "dB")


def test_adapter_rows_behind_the_last_slot_and_bad_indices(m):
    g = gen(2)
    T, d, r, N = 70, 64, 8, 4
    c = adapter_inputs(m, g, torch.float16, T, d, d, r, N)
    ws = adapter_ws(m, T, d, d, r, N, torch.float16)

    def fwd(perm, off):
        out = torch.full((T, d), 3.0, dtype=torch.float16, device="cuda")
        hid = torch.full((T, r), 3.0, device="cuda")
        m.moe_adapter_forward(c["x"], perm, off, c["A"], c["B"], c["scale"], out, ws, base=c["base"], hidden=hid)
        return m.moe_status_read(ws), out, hid
    st, good, hid = fwd(c["perm"], c["off"])
    assert st == m.MOE_OK
    # entries that point outside are skipped and reported; the next good call reports OK again
    S = int(c["off"][-1])
    bad = c["perm"].clone()
    lost = [int(bad[0]), int(bad[S - 1])]
    bad[0], bad[S - 1] = T, -1
    st, out, _ = fwd(bad, c["off"])
    assert st == m.MOE_ERR_DEVICE_BOUNDS
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[lost] = False
    assert torch.equal(out[keep], good[keep]) and (out[lost] == 3.0).all()
    assert fwd(c["perm"], c["off"])[0] == m.MOE_OK
    for off in ([0, 10, 5, 20, S], [0, 10, 20, 30, T + 9], [-4, 10, 20, 30, S],
                [0, 1 << 30, 1 << 30, 1 << 30, 1 << 30], [S, S, S, S, 0]):
        st, out, hid = fwd(c["perm"], torch.tensor(off, dtype=torch.int32, device="cuda"))
        assert st == m.MOE_ERR_DEVICE_BOUNDS
        dA, dB = torch.empty((N, d, r), device="cuda"), torch.empty((N, r, d), device="cuda")
        m.moe_adapter_backward(c["x"], c["x"], hid, c["perm"], torch.tensor(off, dtype=torch.int32, device="cuda"),
                               c["A"], c["B"], c["scale"], ws, dA=dA, dB=dB)
        assert m.moe_status_read(ws) == m.MOE_ERR_DEVICE_BOUNDS
    # no adapter at all
    st, out, hid = fwd(c["perm"], torch.zeros(N + 1, dtype=torch.int32, device="cuda"))
    assert st == m.MOE_OK and (out == 3.0).all() and (hid == 3.0).all()


@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
def test_adapter_gradients_under_decreasing_offsets(m, dt):
    """Offsets that decrease are reported, and the sums are those of the runs that the other products
    take: a boundary is the largest offset up to it.  (Long runs: their partial sums are joined.)"""
    g = gen(31)
    T, d, r, N = 1900, 64, 16, 5
    c = adapter_inputs(m, g, dt, T, d, d, r, N, none=0.0)
    ws = adapter_ws(m, T, d, d, r, N, dt)
    off = torch.tensor([0, 1100, 100, 1500, 1200, T], dtype=torch.int32, device="cuda")
    bound = [0, 1100, 1100, 1500, 1500, T]
    dy, hid = randn(g, T, d, dtype=dt), randn(g, T, r)
    dA, dB = torch.full((N, d, r), 7.0, device="cuda"), torch.full((N, r, d), 7.0, device="cuda")
    m.moe_adapter_backward(dy, c["x"], hid, c["perm"], off, c["A"], c["B"], c["scale"], ws, dA=dA, dB=dB)
    assert m.moe_status_read(ws) == m.MOE_ERR_DEVICE_BOUNDS
    for n in range(N):
        s = slice(bound[n], bound[n + 1])
        t, sc = c["perm"][s].long(), float(c["scale"][n])
        x, y, h, B = c["x"][t].double(), dy[t].double(), hid[s].double(), c["B"][n].double()
        dh, dhm = y @ B.t(), y.abs() @ B.abs().t()
        if not len(t):
            assert not dA[n].any() and not dB[n].any()
            continue
        # as in test_adapter_backward
        half = dt == torch.float16
        K = 2 * (4 * (d / 512 + 1) + 16) if half else d / 8 + 48
        KW = 64 + len(t) / 64 if half else len(t) + 16
        yf = torch.where(y == 0, y, y.abs().clamp(min=2.0 ** -14)) if half else y.abs()
        sa = x.abs().sum(0)[:, None] * dh.abs().max() if half else 0
        sb = yf.sum(0)[None, :] * h.abs().max() if half else 0
        check(dA[n], sc * (x.t() @ dh), abs(sc) * ((KW + K) * U * (x.abs().t() @ dhm) + 2 * U * sa) + 1e-37, "dA")
        check(dB[n], sc * (h.t() @ y), abs(sc) * (KW * U * (h.abs().t() @ yf) + 2 * U * sb) + 1e-37, "dB")


@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
@pytest.mark.parametrize("T", [40, 700, 1500])
def test_adapter_bad_entries_take_nothing_into_the_gradients(m, dt, T):
    """Entries outside [0, T) are left out of every sum, whatever a token without an adapter holds."""
    g = gen(37 + T)
    d, r, N = 64, 16, 2
    c = adapter_inputs(m, g, dt, T, d, d, r, N, none=0.0)
    ws = adapter_ws(m, T, d, d, r, N, dt)
    ids = c["ids"].clone()
    ids[0] = -1
    perm, off = plan(m, ids, N)
    S = T - 1
    assert int(off[-1]) == S
    bad = perm.clone()
    lost = torch.tensor([0, 3, 5, S - 1], device="cuda")
    bad[lost] = torch.tensor([-1, T, 1 << 30, -(1 << 30)], dtype=torch.int32, device="cuda")
    x, dy, hid = c["x"].clone(), randn(g, T, d, dtype=dt), randn(g, T, r)
    x[0], dy[0] = float("nan"), float("inf")
    dx = torch.full((T, d), 9.0, dtype=dt, device="cuda")
    got = []
    for h in (hid, hid.clone().index_fill_(0, lost, 0.0)):
        # the second call names row 1 in the slots that the first skips, with nothing to add
        dA, dB = torch.empty((N, d, r), device="cuda"), torch.empty((N, r, d), device="cuda")
        p = bad if h is hid else bad.clone().index_fill_(0, lost, 1)
        m.moe_adapter_backward(dy, x, h, p, off, c["A"], c["B"], c["scale"], ws, dtokens=dx if h is hid else None,
                               dA=dA, dB=dB)
        assert m.moe_status_read(ws) == (m.MOE_ERR_DEVICE_BOUNDS if h is hid else m.MOE_OK)
        got.append((dA, dB))
    for n in range(N):
        s = torch.arange(int(off[n]), int(off[n + 1]), device="cuda")
        s = s[~torch.isin(s, lost)]
        t, sc = perm[s].long(), float(c["scale"][n])
        xx, y, B = x[t].double(), dy[t].double(), c["B"][n].double()
        dh, dhm = y @ B.t(), y.abs() @ B.abs().t()
        half = dt == torch.float16
        K = (2 * (4 * (d / 512 + 1) + 16) if half else d / 8 + 48) + (64 + len(t) / 64 if half else len(t) + 16)
        slack = xx.abs().sum(0)[:, None] * dh.abs().max() if half else 0
        check(got[0][0][n], sc * (xx.t() @ dh), abs(sc) * (K * U * (xx.abs().t() @ dhm) + 2 * U * slack) + 1e-37, "dA")
        assert torch.isfinite(got[0][1][n]).all()
        h = hid[s].double()
        want = sc * (h.t() @ y)
        yf = torch.where(y == 0, y, y.abs().clamp(min=2.0 ** -14)) if half else y.abs()
        tol = abs(sc) * (K * U * (h.abs().t() @ yf) + (2 * U * yf.sum(0)[None, :] * h.abs().max() if half else 0)) + 1e-37
        check(got[0][1][n], want, tol, "dB")
        check(got[1][1][n], want, tol, "dB with zero rows")
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[perm[:S].long()] = False
    rest[perm[lost].long()] = True
    assert (dx[rest] == 9.0).all()


def behind(m, size, extra=16 << 20):
    """A workspace of exactly `size` bytes with a guard behind it."""
    buf = torch.full((size + extra,), 0x5A, dtype=torch.uint8, device="cuda")
    return buf[:size], buf[size:]


@pytest.mark.parametrize("r", [8, 24, 64, 128])
@pytest.mark.parametrize("off", [[19000, 20000], [18200, 18900, 18900, 20000], [19500, 19700, 100, 20000],
                                 [12000, 12500, 13000]])
@pytest.mark.parametrize("di,do", [(2048, 1032), (72, 136)])     # several column parts, one
def test_adapter_long_plan_that_starts_late(m, off, di, do, r):
    """Slots before offsets[0] belong to no adapter (a slice of a larger plan): nothing is read from or
    written for them, nor behind the workspace, and the rows are those of the plan without the gap."""
    g = gen(41 + r)
    S, T, N = 20000, 1900, len(off) - 1
    dt, i32 = torch.float16, dict(dtype=torch.int32, device="cuda")
    bound = [max(off[:n + 1]) for n in range(N + 1)]
    rows = bound[N] - bound[0]
    tok = torch.randperm(T, generator=g, device="cuda")[:rows].to(torch.int32)
    perm = torch.full((S,), -1, **i32)               # entries that no adapter owns are not looked at
    perm[bound[0]:bound[N]] = tok
    perm0 = torch.full((S,), -1, **i32)
    perm0[:rows] = tok
    x, base = randn(g, T, di, dtype=dt), randn(g, T, do, dtype=dt)
    A, B = randn(g, N, di, r, sigma=di ** -0.5, dtype=dt), randn(g, N, r, do, sigma=0.3, dtype=dt)
    scale = randn(g, N)
    got = []
    for p, o in ((perm, off), (perm0, [b - bound[0] for b in bound])):
        o = torch.tensor(o, **i32)
        size = m.moe_adapter_workspace_size(T, di, do, r, N, S, dt)
        e = lambda *s, t=torch.float32: torch.full(s, 3.0, dtype=t, device="cuda")
        out, hid, dx, dA, dB = e(T, do, t=dt), e(S, r), e(T, di, t=dt), e(N, di, r), e(N, r, do)
        want_status = m.MOE_ERR_DEVICE_BOUNDS if p is perm and off != bound else m.MOE_OK
        ws, guard = behind(m, size)
        m.moe_adapter_forward(x, p, o, A, B, scale, out, ws, base=base, hidden=hid)
        assert m.moe_status_read(ws) == want_status
        assert (guard == 0x5A).all()
        ws, guard = behind(m, size)
        m.moe_adapter_backward(base, x, hid, p, o, A, B, scale, ws, dtokens=dx, dtokens_in=x, dA=dA, dB=dB)
        assert m.moe_status_read(ws) == want_status
        assert (guard == 0x5A).all()
        # without hidden rows, and without their gradient
        bare, ws = e(T, do, t=dt), behind(m, size)[0]
        m.moe_adapter_forward(x, p, o, A, B, scale, bare, ws, base=base)
        assert torch.equal(bare, out)
        dx2 = e(T, di, t=dt)
        m.moe_adapter_backward(base, None, None, p, o, A, B, scale, ws, dtokens=dx2, dtokens_in=x)
        assert torch.equal(dx2, dx)
        first = bound[0] if p is perm else 0
        assert (hid[:first] == 3.0).all() and (hid[first + rows:] == 3.0).all()
        got.append((out, hid[first:first + rows], dx, dA, dB))
    for a, b in zip(got[0][:3], got[1][:3]):
        assert torch.equal(a, b)
    for n in range(N):
        s = slice(bound[n] - bound[0], bound[n + 1] - bound[0])
        t, sc = tok[s].long(), scale[n].double()
        xx, y, h = x[t].double(), base[t].double(), got[0][1][s].double()
        # a chain of K truncating additions per hidden value, then one of rows / 64 + 64 for the sums
        K = 2 * (4 * (di / 512 + 1) + 16)
        check(h, xx @ A[n].double(), K * U * (xx.abs() @ A[n].double().abs()) + 1e-37, "hidden")
        yf = torch.where(y == 0, y, y.abs().clamp(min=2.0 ** -14))
        dh, dhm = y @ B[n].double().t(), y.abs() @ B[n].double().abs().t()
        KW, top = 64 + len(t) / 64, lambda v: v.abs().max() if len(t) else 0
        for q in got:
            check(q[3][n], sc * (xx.t() @ dh), sc.abs() * ((KW + K) * U * (xx.abs().t() @ dhm) +
                  2 * U * xx.abs().sum(0)[:, None] * top(dh)) + 1e-37, "dA")
            check(q[4][n], sc * (h.t() @ y), sc.abs() * (KW * U * (h.abs().t() @ yf) +
                  2 * U * yf.sum(0)[None, :] * top(h)) + 1e-37, "dB")


def test_adapter_few_tokens_of_many(m):
    """Most tokens without an adapter: the plans go by the caller's bound, the work by the offsets."""
    g = gen(21)
    T, di, do, r, N = 6000, 520, 1048, 24, 3
    dt = torch.float16
    c = adapter_inputs(m, g, dt, T, di, do, r, N, none=0.97)
    ws = adapter_ws(m, T, di, do, r, N, dt)
    out, hid = c["base"].clone(), torch.full((T, r), 4.0, device="cuda")
    m.moe_adapter_forward(c["x"], c["perm"], c["off"], c["A"], c["B"], c["scale"], out, ws, base=out, hidden=hid)
    dA, dB = torch.empty((N, di, r), device="cuda"), torch.empty((N, r, do), device="cuda")
    m.moe_adapter_backward(c["base"], c["x"], hid, c["perm"], c["off"], c["A"], c["B"], c["scale"], ws, dA=dA, dB=dB)
    S = int(c["off"][-1])
    assert 50 < S < 400 and (hid[S:] == 4.0).all()
    # the same tokens as a batch of their own give the same bits of what belongs to a row
    t = c["perm"][:S].long()
    x2, b2 = c["x"][t].contiguous(), c["base"][t].contiguous()
    perm2 = torch.arange(S, device="cuda", dtype=torch.int32)
    ws2 = adapter_ws(m, S, di, do, r, N, dt)
    out2, hid2 = b2.clone(), torch.empty((S, r), device="cuda")
    m.moe_adapter_forward(x2, perm2, c["off"], c["A"], c["B"], c["scale"], out2, ws2, base=out2, hidden=hid2)
    K = 2 * (4 * (di / 512 + 1) + 16)
    a = c["ids"][t].long()
    hm = torch.einsum("ti,tij->tj", x2.double().abs(), c["A"].double().abs()[a])
    check(hid[:S], hid2.double(), 2 * K * U * hm, "hidden")
    check(out[t], out2.double(), 2.0 ** -10 * out2.double().abs() + 2.0 ** -24 +
          2.0 ** -10 * c["scale"].double().abs()[a][:, None] *
          torch.einsum("tj,tjo->to", hid2.double().abs(), c["B"].double().abs()[a]), "out")
    for n in range(N):
        s = (a == n).nonzero()[:, 0]
        dy, x = c["base"][t[s]].double(), x2[s].double()
        dhm = dy.abs() @ c["B"][n].double().abs().t()
        want = float(c["scale"][n]) * x.t() @ (dy @ c["B"][n].double().t())
        Kd = 2 * (4 * (do / 512 + 1) + 16) + 64 + len(s) / 64
        check(dA[n], want, abs(float(c["scale"][n])) * (Kd * U * (x.abs().t() @ dhm) +
              2 * U * x.abs().sum(0)[:, None] * dhm.max()) + 1e-37, "dA")


def test_offsets_past_32_bits(m):
    """Rows whose elements lie behind 2^31: 4.4 GB per matrix."""
    T, d, r, N, E = 620_000, 3584, 8, 2, 4
    dt = torch.float16
    x = torch.empty((T, d), dtype=dt, device="cuda").normal_()
    rows = torch.cat([torch.arange(3), torch.arange(599_180, 599_190), torch.arange(T - 200, T)]).cuda()
    g = gen(31)
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) % 3) - 1
    perm, off = plan(m, ids, N)
    A, B = randn(g, N, d, r, sigma=d ** -0.5, dtype=dt), randn(g, N, r, d, sigma=0.3, dtype=dt)
    scale = torch.tensor([0.5, -1.5], device="cuda")
    ws = adapter_ws(m, T, d, d, r, N, dt)
    out = x.clone()
    m.moe_adapter_forward(x, perm, off, A, B, scale, out, ws, base=out)
    xs, a = x[rows].double(), ids[rows].long()
    delta = torch.einsum("ti,tij,tjo->to", xs, A.double()[a.clamp(min=0)], B.double()[a.clamp(min=0)])
    want = xs + delta * (scale.double()[a.clamp(min=0)] * (a >= 0))[:, None]
    mag = torch.einsum("ti,tij,tjo->to", xs.abs(), A.double().abs()[a.clamp(min=0)], B.double().abs()[a.clamp(min=0)])
    check(out[rows], want, 2.0 ** -11 * (1 + 2 ** -9) * want.abs() + 2.0 ** -25 + 1.5 * mag * (256 * U) +
          1.5 * 2.0 ** -11 * torch.einsum("tj,tjo->to", torch.einsum("ti,tij->tj", xs, A.double()[a.clamp(min=0)]).abs(),
                                          B.double().abs()[a.clamp(min=0)]), "out")
    # gate: dtokens row by row, dWg over all rows
    Wg = randn(g, d, E, sigma=0.1)
    logits = randn(g, T, E)
    idx, dw = topk(logits, 1), randn(g, T, 1)
    dl, dWg, dx = torch.empty((T, E), device="cuda"), torch.empty((d, E), device="cuda"), out
    gws = torch.empty(m.moe_gate_backward_workspace_size(T, d, E, dt), dtype=torch.uint8, device="cuda")
    m.moe_gate_topk_backward(logits, idx, dl, dtopk_w=dw, tokens=x, Wg=Wg, dWg=dWg, dtokens=dx, workspace=gws)
    assert m.moe_status_read(gws) == m.MOE_OK
    want = dl[rows].double() @ Wg.double().t()
    mag = dl[rows].double().abs() @ Wg.double().abs().t()
    check(dx[rows], want, 2.0 ** -11 * 1.01 * (want.abs() + mag) + 2.0 ** -24, "dtokens")
    want, mag = torch.zeros((d, E), dtype=torch.double, device="cuda"), torch.zeros((d, E), dtype=torch.double, device="cuda")
    for c in range(0, T, 20_000):
        xd, dd = x[c:c + 20_000].double(), dl[c:c + 20_000].double()
        want += xd.t() @ dd
        mag += xd.abs().t() @ dd.abs()
    check(dWg, want, (80 + T / 128 / 8) * U * mag, "dWg")
    # combine: slots in reverse order, so that high slots meet low tokens
    slot = torch.arange(T - 1, -1, -1, device="cuda", dtype=torch.int32).view(T, 1)
    w = torch.rand((T, 1), generator=g, device="cuda")
    dy, dwo = torch.empty_like(x), torch.empty((T, 1), device="cuda")
    m.moe_combine_backward(x, out, slot, w, dy, dwo)
    s = slot[rows, 0].long()
    check(dy[s], w[rows].double() * xs, 2.0 ** -11 * 1.01 * (w[rows].double() * xs).abs() + 2.0 ** -25, "dexpert_out")
    prod = xs * out[s].double()
    check(dwo[rows, 0], prod.sum(1), 128 * U * prod.abs().sum(1), "dtopk_w")


def test_empty_batches(m):
    z = torch.zeros
    dA, dB = torch.ones((2, 16, 8), device="cuda"), torch.ones((2, 8, 16), device="cuda")
    x = z((0, 16), dtype=torch.float16, device="cuda")
    perm = z((0,), dtype=torch.int32, device="cuda")
    off = z((3,), dtype=torch.int32, device="cuda")
    A, B = z((2, 16, 8), dtype=torch.float16, device="cuda"), z((2, 8, 16), dtype=torch.float16, device="cuda")
    ws = adapter_ws(m, 0, 16, 16, 8, 2, torch.float16)
    m.moe_adapter_forward(x, perm, off, A, B, z(2, device="cuda"), x.clone(), ws)
    m.moe_adapter_backward(x, x, z((0, 8), device="cuda"), perm, off, A, B, z(2, device="cuda"), ws, dA=dA, dB=dB)
    assert not dA.any() and not dB.any()
    m.moe_combine_backward(x, x, z((0, 1), dtype=torch.int32, device="cuda"), z((0, 1), device="cuda"), x, None)


def test_empty_calls_set_the_status_word(m):
    """An empty call after one that found a bad index, or on a workspace that holds anything, reads OK."""
    z = lambda *s, t=torch.float16: torch.zeros(s, dtype=t, device="cuda")
    i32 = torch.int32
    d, r, N, E = 16, 8, 2, 4
    off = z(N + 1, t=i32)
    A, B, sc = z(N, d, r), z(N, r, d), z(N, t=torch.float32)
    for S in (0, 3):                                 # no token, or no slot
        T = 3 - S
        perm, x = z(S if T == 0 else 0, t=i32), z(T, d)
        for fill in (0x5A, 6):
            ws = torch.full((m.moe_adapter_workspace_size(8, d, d, r, N, 8, x.dtype),), fill, dtype=torch.uint8, device="cuda")
            m.moe_adapter_forward(x, perm, off, A, B, sc, x.clone(), ws)
            assert m.moe_status_read(ws) == m.MOE_OK
            ws.fill_(fill)
            m.moe_adapter_backward(x, x, z(perm.numel(), r, t=torch.float32), perm, off, A, B, sc, ws, dtokens=x.clone())
            assert m.moe_status_read(ws) == m.MOE_OK
    gws = torch.full((m.moe_gate_backward_workspace_size(8, d, E, torch.float16),), 0x5A, dtype=torch.uint8, device="cuda")
    f = lambda *s: z(*s, t=torch.float32)
    m.moe_gate_topk_backward(f(0, E), z(0, 1, t=i32), f(0, E), dtopk_w=f(0, 1), tokens=z(0, d), dWg=f(d, E), workspace=gws)
    assert m.moe_status_read(gws) == m.MOE_OK
    # a bad plan, then an empty one
    ws.zero_()
    m.moe_adapter_forward(z(4, d), z(4, t=i32) + 9, torch.tensor([0, 2, 4], dtype=i32, device="cuda"), A, B, sc, z(4, d), ws)
    assert m.moe_status_read(ws) == m.MOE_ERR_DEVICE_BOUNDS
    m.moe_adapter_forward(z(0, d), z(0, t=i32), off, A, B, sc, z(0, d), ws)
    assert m.moe_status_read(ws) == m.MOE_OK
    # captured as well
    x0, p0 = z(0, d), z(0, t=i32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_adapter_forward(x0, p0, off, A, B, sc, x0, ws)
    ws.fill_(6)
    g.replay()
    assert m.moe_status_read(ws) == m.MOE_OK


def test_empty_gate_call_for_the_tokens_alone_sets_the_status_word(m):
    f = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")
    x = f(0, 16, t=torch.float16)
    ws = torch.full((m.moe_gate_backward_workspace_size(8, 16, 4, x.dtype),), 6, dtype=torch.uint8, device="cuda")
    m.moe_gate_topk_backward(f(0, 4), f(0, 1, t=torch.int32), f(0, 4), dtopk_w=f(0, 1), Wg=f(16, 4), dtokens=x, workspace=ws)
    assert m.moe_status_read(ws) == m.MOE_OK


# ---------------------------------------------------------------- together, streams, graphs
def step_buffers(m, T, d, r, N, E, k):
    f16, f32, i32 = torch.float16, torch.float32, torch.int32
    e = lambda *s, t=f32: torch.zeros(s, dtype=t, device="cuda")
    S = T * k
    return dict(logits=e(T, E), idx=e(T, k, t=i32), w=e(T, k), counts=e(E, t=i32), kept=e(E, t=i32),
                off=e(E + 1, t=i32), perm=e(S, t=i32), slot=e(T, k, t=i32), y=e(S, d, t=f16), out=e(T, d, t=f16),
                ws=e(m.moe_workspace_size(T, d, 4 * d, E, k, float("inf"), 0, 0, m.MOE_F16), t=torch.uint8),
                bc=e(E, t=i32), P=e(E), losses=e(2), nv=e(1, t=i32),
                bws=e(m.moe_balance_workspace_size(T, E), t=torch.uint8),
                hid=e(T, r), aws=e(m.moe_adapter_workspace_size(T, d, d, r, N, T, f16), t=torch.uint8),
                acnt=e(N, t=i32), akept=e(N, t=i32), aoff=e(N + 1, t=i32), aperm=e(T, t=i32), aslot=e(T, 1, t=i32),
                dw=e(T, k), dl=e(T, E), dWg=e(d, E), dx=e(T, d, t=f16), dA=e(N, d, r), dB=e(N, r, d),
                gws=e(m.moe_gate_backward_workspace_size(T, d, E, f16), t=torch.uint8))


def step(m, c, b, stream=None):
    """A training step of the router and the adapters of a layer whose experts stay as they are."""
    kw = dict(stream=stream)
    E, k = c["Wg"].shape[1], b["idx"].shape[1]
    N = c["A"].shape[0]
    m.moe_gate_topk(c["x"], c["Wg"], k, b["idx"], b["w"], logits_out=b["logits"], **kw)
    m.moe_dispatch(b["idx"], E, 1.0, b["counts"], b["kept"], b["off"], b["perm"], b["slot"], **kw)
    m.moe_expert_ffn(c["x"], b["perm"], b["off"], c["W1"], c["W2"], b["y"].shape[0], b["y"], b["ws"], **kw)
    m.moe_combine(b["y"], b["slot"], b["w"], b["out"], **kw)
    m.moe_balance_loss(b["logits"], b["idx"], b["bc"], b["P"], b["losses"], b["nv"], b["bws"], **kw)
    m.moe_dispatch(c["ids"], N, float("inf"), b["acnt"], b["akept"], b["aoff"], b["aperm"], b["aslot"], **kw)
    m.moe_adapter_forward(c["x"], b["aperm"], b["aoff"], c["A"], c["B"], c["scale"], b["out"], b["aws"],
                          base=b["out"], hidden=b["hid"], **kw)
    m.moe_combine_backward(c["dout"], b["y"], b["slot"], b["w"], None, b["dw"], **kw)
    m.moe_gate_topk_backward(b["logits"], b["idx"], b["dl"], dtopk_w=b["dw"], dlosses=c["dloss"],
                             counts=b["bc"], n_valid=b["nv"], tokens=c["x"], Wg=c["Wg"], dWg=b["dWg"],
                             dtokens=b["dx"], workspace=b["gws"], **kw)
    m.moe_adapter_backward(c["dout"], c["x"], b["hid"], b["aperm"], b["aoff"], c["A"], c["B"], c["scale"],
                           b["aws"], dtokens=b["dx"], dtokens_in=b["dx"], dA=b["dA"], dB=b["dB"], **kw)


OUTS = ("out", "losses", "bc", "P", "dw", "dl", "dWg", "dx", "dA", "dB")


def step_inputs(seed, T, d, r, N, E, k):
    g = gen(seed)
    f16 = torch.float16
    ids = torch.randint(-1, N, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    return dict(x=randn(g, T, d, dtype=f16), Wg=randn(g, d, E, sigma=d ** -0.5), ids=ids,
                W1=randn(g, E, d, 4 * d, sigma=d ** -0.5, dtype=f16),
                W2=randn(g, E, 4 * d, d, sigma=0.5 * d ** -0.5, dtype=f16),
                A=randn(g, N, d, r, sigma=d ** -0.5, dtype=f16), B=randn(g, N, r, d, sigma=0.1, dtype=f16),
                scale=torch.rand(N, generator=g, device="cuda") + 0.5, dout=randn(g, T, d, sigma=0.1, dtype=f16),
                dloss=torch.tensor([0.01, 0.001], device="cuda"))


@pytest.mark.parametrize("T,d,r,N,E,k", [(96, 128, 16, 5, 8, 2), (700, 256, 24, 3, 12, 1), (1700, 128, 40, 2, 16, 2)])
def test_training_step_of_router_and_adapters(m, T, d, r, N, E, k):
    c, b = step_inputs(1, T, d, r, N, E, k), step_buffers(m, T, d, r, N, E, k)
    step(m, c, b)
    torch.cuda.synchronize()
    assert m.moe_status_read(b["ws"]) == m.MOE_OK and m.moe_status_read(b["aws"]) == m.MOE_OK
    # the same step by autograd in 64 bits (experts' outputs as the library rounded them)
    x = c["x"].double().requires_grad_()
    Wg, A, B = (c[q].double().requires_grad_() for q in ("Wg", "A", "B"))
    logits = x @ Wg
    idx, slot = b["idx"].long(), b["slot"].long()
    sel = torch.log_softmax(logits, 1).gather(1, idx)
    w = sel.exp() if k == 1 else torch.softmax(sel, 1)
    y = torch.where((slot >= 0)[..., None], b["y"].double()[slot.clamp(min=0)], torch.zeros((), device="cuda", dtype=torch.double))
    comb = (w[..., None] * y).sum(1)
    ids = c["ids"].flatten().long()
    on = ids >= 0
    delta = torch.einsum("ti,tij,tjo->to", x[on], A[ids[on]], B[ids[on]]) * c["scale"].double()[ids[on]][:, None]
    out = comb.index_add(0, on.nonzero()[:, 0], delta)
    p = torch.softmax(logits, 1)
    bal = E * (b["bc"].double() / (T * k) * p.mean(0)).sum()
    z = torch.logsumexp(logits, 1).square().mean()
    total = (out * c["dout"].double()).sum() + 0.01 * bal + 0.001 * z
    gx, gW, gA, gB = torch.autograd.grad(total, (x, Wg, A, B), retain_graph=True)
    (gx_adapter,) = torch.autograd.grad((delta * c["dout"].double()[on]).sum(), x)
    gx_gate = gx - gx_adapter
    assert abs(float(b["losses"][0]) - bal.item()) < 1e-5 and abs(float(b["losses"][1]) - z.item()) < 1e-4
    # out is rounded twice, after the combine and after the adapter (rows without one: once), dtokens
    # after the gate and after the adapter; 32-bit sums of a row's terms add less than 2^-16 of its
    # largest value.  dlogits come from logits of 32 bits (d products: 2^-24 d of their magnitudes).
    half = 2.0 ** -11 * (1 + 2.0 ** -9)
    ids_on = ids[on]
    hmag = torch.einsum("ti,tij->tj", c["x"].double()[on], c["A"].double()[ids_on]).abs()
    dhmag = torch.einsum("to,tjo->tj", c["dout"].double()[on], c["B"].double()[ids_on]).abs()
    sc = c["scale"].double()[ids_on][:, None]
    # h (and dh) rounded to f16 before the second product, Wg before the gate's
    gate_h = b["dl"].double().abs() @ c["Wg"].double().abs().t()
    out_h, dx_h = torch.zeros_like(out), torch.zeros_like(gx)
    out_h[on] = sc * torch.einsum("tj,tjo->to", hmag, c["B"].double()[ids_on].abs())
    dx_h[on] = sc * torch.einsum("tj,tij->ti", dhmag, c["A"].double()[ids_on].abs())
    row = lambda v: 2.0 ** -16 * v.abs().amax(1, keepdim=True) + 2.0 ** -24
    check(b["out"], out, half * (comb.abs() + out.abs() + out_h) + row(out), "out")
    check(b["dx"], gx, half * (gx_gate.abs() + gx.abs() + dx_h + gate_h) + row(gx), "dx")
    for name, want in (("dWg", gW), ("dA", gA), ("dB", gB)):
        check(b[name], want, 2.0 ** -14 * want.abs().max(), name)


@pytest.mark.parametrize("shape", [(300, 128, 16, 4, 8, 2), (1300, 256, 40, 2, 64, 2)])
def test_training_step_streams_graph_and_repeats(m, shape):
    c, b = step_inputs(2, *shape), step_buffers(m, *shape)
    step(m, c, b)
    torch.cuda.synchronize()
    want = {q: b[q].clone() for q in OUTS}
    # again, and on another stream
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s):
        for q in OUTS:
            b[q].zero_()
        torch.cuda.synchronize()
        step(m, c, b, stream=stream)
        torch.cuda.synchronize()
        for q in OUTS:
            assert torch.equal(b[q], want[q]), (q, stream)
    # captured and replayed with new inputs; two graphs share every workspace and run one after the other
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(m, c, b)
        graphs.append(g)
    c2 = step_inputs(3, *shape)
    keep = {q: c[q].clone() for q in c}
    for q in ("x", "Wg", "A", "B", "dout", "ids"):
        c[q].copy_(c2[q])
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    got = {q: b[q].clone() for q in OUTS}
    step(m, c, b)
    torch.cuda.synchronize()
    for q in OUTS:
        assert torch.equal(b[q], got[q]), q
    for q in keep:
        c[q].copy_(keep[q])
    graphs[0].replay()
    torch.cuda.synchronize()
    for q in OUTS:
        assert torch.equal(b[q], want[q]), q


def test_two_router_calls_at_once(m):
    """Losses and gate gradients of two batches on two streams, each with its own workspace."""
    g = gen(10)
    T, d, E, k = 3000, 512, 64, 2
    x, Wg, logits, idx, dw = gate_inputs(g, torch.float16, T, d, E, k)
    dloss = torch.tensor([0.01, 0.001], device="cuda")
    e = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")
    out = [dict(c=e(E, t=torch.int32), p=e(E), l=e(2), n=e(1, t=torch.int32), dl=e(T, E), dWg=e(d, E),
                dx=e(T, d, t=torch.float16), bws=e(m.moe_balance_workspace_size(T, E), t=torch.uint8),
                gws=e(m.moe_gate_backward_workspace_size(T, d, E, x.dtype), t=torch.uint8)) for _ in range(3)]

    def run(o, stream=None):
        m.moe_balance_loss(logits, idx, o["c"], o["p"], o["l"], o["n"], o["bws"], stream=stream)
        m.moe_gate_topk_backward(logits, idx, o["dl"], dtopk_w=dw, dlosses=dloss, counts=o["c"], n_valid=o["n"],
                                 tokens=x, Wg=Wg, dWg=o["dWg"], dtokens=o["dx"], workspace=o["gws"], stream=stream)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for o, s in zip(out, streams):
            run(o, s)
    run(out[2])
    torch.cuda.synchronize()
    for q in ("c", "p", "l", "n", "dl", "dWg", "dx"):
        assert torch.equal(out[0][q], out[2][q]) and torch.equal(out[1][q], out[2][q]), q
    assert all(m.moe_status_read(o["gws"]) == m.MOE_OK for o in out)


def test_two_adapter_calls_at_once(m):
    """Different workspaces and outputs: calls may overlap on two streams."""
    g = gen(9)
    c = adapter_inputs(m, g, torch.float16, 2000, 512, 512, 32, 6)
    outs = [torch.zeros((2000, 512), dtype=torch.float16, device="cuda") for _ in range(3)]
    wss = [adapter_ws(m, 2000, 512, 512, 32, 6, torch.float16) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, s in enumerate(streams):
        for _ in range(4):
            m.moe_adapter_forward(c["x"], c["perm"], c["off"], c["A"], c["B"], c["scale"], outs[i], wss[i],
                                  base=c["base"], stream=s)
    m.moe_adapter_forward(c["x"], c["perm"], c["off"], c["A"], c["B"], c["scale"], outs[2], wss[2], base=c["base"])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])
