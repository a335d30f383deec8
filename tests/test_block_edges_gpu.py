"""The block calls where their documentation allows something out of the ordinary."""
import pytest
import torch

import test_block_gpu
from test_block_gpu import check, experts8, gen, half, norm_inputs, randn, ref_ffn8, rows8, values8

pytestmark = pytest.mark.gpu
F16 = torch.float16
NAN = float("nan")


@pytest.fixture(scope="module")
def m():
    import sparse_expert_ffn_layer_gb300 as mod
    return mod


def test_outputs_that_may_be_inputs(m):
    """Same bits as with outputs of their own."""
    g = gen(3)
    T, d, f, E, k = 300, 256, 512, 8, 2
    # the experts' outputs over the tokens
    x = randn(g, T, d, dtype=F16)
    (W1, s1), (W2, s2) = experts8(m, g, E, d, f), experts8(m, g, E, f, d)
    perm = torch.randperm(T, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    off = torch.tensor([0, 10, 80, 80, 130, 200, 230, 290, T], dtype=torch.int32, device="cuda")
    ws = torch.empty(m.moe_expert_fp8_workspace_size(T, d, f, E, T, F16), dtype=torch.uint8, device="cuda")
    want, got = torch.empty_like(x), x.clone()
    m.moe_expert_ffn_fp8(x, perm, off, W1, s1, W2, s2, T, want, ws)
    m.moe_expert_ffn_fp8(got, perm, off, W1, s1, W2, s2, T, got, ws)
    assert torch.equal(got, want)
    # logits in place, the tokens' gradient added up in place
    li = randn(g, T, E)
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    i2, w2 = torch.empty_like(idx), torch.empty_like(w)
    m.moe_route(None, None, k, idx, w, logits_in=li)
    m.moe_route(None, None, k, i2, w2, logits_in=li, logits_out=li)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    Wg, dw, dl, dx = randn(g, d, E), randn(g, T, k), torch.empty_like(li), torch.empty_like(x)
    ws = torch.empty(m.moe_gate_backward_workspace_size(T, d, E, F16), dtype=torch.uint8, device="cuda")
    got = x.clone()
    m.moe_route_backward(li, idx, dl, dtopk_w=dw, Wg=Wg, dtokens=dx, dtokens_in=x, workspace=ws)
    m.moe_route_backward(li, idx, dl, dtopk_w=dw, Wg=Wg, dtokens=got, dtokens_in=got, workspace=ws)
    assert torch.equal(got, dx)
    # the residual's gradient in place, sums in one buffer side by side
    slot, rows, w = norm_inputs(g, T, d, k, F16)
    post, gate = 1 + randn(g, d, sigma=0.1), randn(g, d)
    hid, rp, dh = torch.empty_like(x), torch.empty(T, device="cuda"), randn(g, T, d, dtype=F16)
    m.moe_block_norm(x, hid, expert_out=rows, slot_of=slot, topk_w=w, post_w=post, gate=gate, rstd_post=rp)
    ws = torch.empty(m.moe_block_norm_workspace_size(T, d, k, F16), dtype=torch.uint8, device="cuda")
    given = dict(expert_out=rows, slot_of=slot, topk_w=w, post_w=post, gate=gate, rstd_post=rp, workspace=ws)
    want, sums, one = torch.empty_like(x), [torch.empty(d, device="cuda") for _ in range(2)], torch.empty(2 * d, device="cuda")
    m.moe_block_norm_backward(dh, dresidual=want, dpost_w=sums[0], dgate=sums[1], **given)
    m.moe_block_norm_backward(dh, dresidual=dh, dpost_w=one[:d], dgate=one[d:], **given)
    assert torch.equal(dh, want) and torch.equal(one, torch.cat(sums))


def test_gradients_over_their_weights_are_refused(m):
    """They are factors of each other's sums."""
    g = gen(4)
    T, d = 40, 128
    dh, y = randn(g, T, d, dtype=F16), randn(g, T, d, dtype=F16)
    post, gate, rp = randn(g, d), randn(g, d), torch.ones(T, device="cuda")
    ws = torch.empty(m.moe_block_norm_workspace_size(T, d, 0, F16), dtype=torch.uint8, device="cuda")
    given = dict(shared=y, post_w=post, gate=gate, rstd_post=rp, workspace=ws)
    for over in (dict(dgate=gate, dpost_w=torch.empty_like(gate)), dict(dpost_w=post), dict(dgate=post), dict(dshared=y),
                 dict(dgate=rp.new_empty(d), dpost_w=None, dshared=y)):
        with pytest.raises(m.MoeError) as e:
            m.moe_block_norm_backward(dh, **over, **given)
        assert e.value.code == m.MOE_ERR_INVALID_ARG
    Wg, li, idx = randn(g, d, 8), randn(g, T, 8), torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    ws = torch.empty(m.moe_gate_backward_workspace_size(T, d, 8, F16), dtype=torch.uint8, device="cuda")
    with pytest.raises(m.MoeError) as e:
        m.moe_route_backward(li, idx, torch.empty_like(li), dtopk_w=randn(g, T, 1), tokens=y, Wg=Wg, dWg=Wg,
                             dtokens=torch.empty_like(y), workspace=ws)
    assert e.value.code == m.MOE_ERR_INVALID_ARG


def layer8(m, g, T, d, f, E, S):
    """An input, experts and a workspace; run(perm, offsets) gives the outputs (rows that nothing wrote: 7.5) and status."""
    x = randn(g, T, d, dtype=F16)
    (W1, s1), (W2, s2) = experts8(m, g, E, d, f), experts8(m, g, E, f, d)

    def run(perm, offsets):
        size = m.moe_expert_fp8_workspace_size(T, d, f, E, S, F16)
        ws = torch.full((size + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        out = torch.full((S + 3, d), 7.5, dtype=F16, device="cuda")
        n0 = m.get_lib().moe_kernel_launches()
        m.moe_expert_ffn_fp8(x, perm, torch.tensor(offsets, dtype=torch.int32, device="cuda"), W1, s1, W2, s2, S, out, ws[:size])
        launches = m.get_lib().moe_kernel_launches() - n0
        status = m.moe_status_read(ws[:size])
        assert (ws[size:] == 0x5A).all() and (out[S:] == 7.5).all()
        return out[:S], status, launches
    return run


# short runs with clusters, tiles of 32 and of more rows; long runs: each product in two forms of which one returns at once
SHAPES = [(60, 1024, 512, 3, 40, 3), (300, 256, 384, 3, 290, 3), (700, 2048, 2048, 3, 2100, 5)]


@pytest.mark.parametrize("T,d,f,E,S,launches", SHAPES)
@pytest.mark.parametrize("start", [1, 13, 38])
def test_experts_in_8_bits_of_a_plan_that_starts_late(m, T, d, f, E, S, launches, start):
    """A slice of a larger plan: what stands before its first slot is not looked at, and the rows are those of the plan
    without the gap."""
    g = gen(start)
    run = layer8(m, g, T, d, f, E, S)
    n = S - 38
    cut = [0, n // 3, n // 3 + 1, n]
    tokens = torch.randint(0, T, (n,), generator=g, device="cuda").to(torch.int32)
    perm0 = torch.full((S,), -1, dtype=torch.int32, device="cuda")
    perm0[:n] = tokens
    want, status, took = run(perm0, cut)
    assert status == m.MOE_OK and took == launches
    perm = torch.full((S,), T + 9, dtype=torch.int32, device="cuda")
    perm[start:start + n] = tokens
    out, status, _ = run(perm, [start + c for c in cut])
    assert status == m.MOE_OK
    assert torch.equal(out[start:start + n], want[:n])
    assert (out[:start] == 7.5).all() and (out[start + n:] == 7.5).all()
    # as moe_expert_ffn has it
    W1, W2 = randn(g, E, d, f, sigma=0.05, dtype=F16), randn(g, E, f, d, sigma=0.05, dtype=F16)
    x = randn(g, T, d, dtype=F16)
    ws = torch.empty(512 + S * f * 2, dtype=torch.uint8, device="cuda")
    m.moe_expert_ffn(x, perm, torch.tensor([start + c for c in cut], dtype=torch.int32, device="cuda"), W1, W2, S,
                     out.contiguous(), ws)
    assert m.moe_status_read(ws) == m.MOE_OK


@pytest.mark.parametrize("T,d,f,E,S,launches", SHAPES)
def test_experts_in_8_bits_of_plans_that_leave_their_bounds(m, T, d, f, E, S, launches):
    """Offsets that fall, exceed S_max or are negative are clamped, tokens out of range give rows of zeros, both are
    reported; everything else is as in the plan that this amounts to."""
    g = gen(S)
    run = layer8(m, g, T, d, f, E, S)
    perm = torch.randint(0, T, (S,), generator=g, device="cuda").to(torch.int32)
    a, b = S // 3, S // 3 * 2
    for given, clamped in (([0, a, b, S + 900], [0, a, b, S]), ([0, b, a, S], [0, b, b, S]), ([-7, a, b, S], [0, a, b, S]),
                           ([0, a, 2 ** 31 - 1, S], [0, a, S, S]), ([S + 5, 0, a, b], [S, S, S, S]),
                           ([0, a, -2 ** 31, b], [0, a, a, b])):
        want, status, took = run(perm, clamped)
        assert status == m.MOE_OK and took == launches
        out, status, _ = run(perm, given)
        assert status == m.MOE_ERR_DEVICE_BOUNDS, given
        assert torch.equal(out, want), given
    want, _, _ = run(perm, [0, a, b, S])
    for at, token in ((0, T), (a, -1), (S - 1, 2 ** 31 - 1), (b + 3, -2 ** 31)):
        bad = perm.clone()
        bad[at] = token
        out, status, _ = run(bad, [0, a, b, S])
        assert status == m.MOE_ERR_DEVICE_BOUNDS
        assert (out[at] == 0).all()
        rest = torch.arange(S, device="cuda") != at
        assert torch.equal(out[rest], want[rest])
        # the next call sets the word anew
        assert run(perm, [0, a, b, S])[1] == m.MOE_OK


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_a_slot_that_two_tokens_name(m, dtype):
    """Each element of its gradient is one of theirs; the other slots and gradients do not notice."""
    g = gen(6)
    T, d, k = 64, 2048, 2
    slot, rows, w = norm_inputs(g, T, d, k, dtype, drop=0.0)
    dh = randn(g, T, d, dtype=dtype)
    a, b = int(slot[10, 0]), int(slot[50, 1])
    one, two = slot.clone(), slot.clone()
    one[50, 1], two[50, 1] = -1, a
    got = {}
    for name, s in (("one", one), ("two", two)):
        dy, dw = torch.full_like(rows, 7.5), torch.empty((T, k), device="cuda")
        m.moe_block_norm_backward(dh, expert_out=rows, slot_of=s, topk_w=w, dexpert_out=dy, dtopk_w=dw)
        got[name] = dy, dw
    (y1, w1), (y2, w2) = got["one"], got["two"]
    other = torch.arange(rows.shape[0], device="cuda") != a
    assert torch.equal(y1[other], y2[other]) and (y2[b] == 7.5).all()
    theirs = (w[50, 1].double() * dh[50].double()).to(dtype)
    assert ((y2[a] == y1[a]) | (y2[a] == theirs)).all()
    same = torch.ones_like(w, dtype=torch.bool)
    same[50, 1] = False
    assert torch.equal(w1[same], w2[same]) and float(w2[50, 1]) != 0.0


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("factor", [0.0, -1.0, 3.0, 2.0 ** -140, float("inf"), -float("inf")])
def test_one_scale_that_is_no_power_of_two(m, which, factor):
    """Long runs, in the form for any scales and to its tolerance; an infinite scale makes its columns infinite with the
    sign of the block's sum."""
    g = gen(17)
    E, n, d, f = 2, 300, 3328, 4608
    x = randn(g, E * n, d, dtype=F16)
    (W1, s1), (W2, s2) = experts8(m, g, E, d, f), experts8(m, g, E, f, d)
    s = (s1, s2)[which]
    s[1, 1, 1] = s[1, 1, 1] * factor if abs(factor) < 1e30 else factor
    perm, off = torch.arange(E * n, device="cuda").to(torch.int32), torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    out = torch.empty((E * n, d), dtype=F16, device="cuda")
    ws = torch.empty(m.moe_expert_fp8_workspace_size(E * n, d, f, E, E * n, F16), dtype=torch.uint8, device="cuda")
    m.moe_expert_ffn_fp8(x, perm, off, W1, s1, W2, s2, E * n, out, ws)
    assert m.moe_status_read(ws) == m.MOE_OK
    for e in range(E):
        rows, cols = slice(e * n, (e + 1) * n), torch.ones(d, dtype=torch.bool, device="cuda")
        w1, w2 = values8(W1[e], s1[e]), values8(W2[e], s2[e])
        if e == 1 and abs(factor) > 1e30:
            if which == 0:                            # GeLU(-infinity) is NaN in its formula: all of each row
                assert not torch.isfinite(out[rows]).any()
                continue
            cols[128:256] = False
            got = out[rows, 128:256].float()
            h = rows8(torch.nn.functional.gelu(rows8(x[rows].double()) @ values8(W1[e], s1[e]).t(), approximate="tanh"))
            sign = h[:, 128:256] @ W2[e, 128:256, 128:256].double().t()
            # (a sum that is near zero may have either sign, or be zero: 0 times infinity is NaN)
            clear = sign.abs() > 0.05 * (h[:, 128:256].abs() @ W2[e, 128:256, 128:256].double().abs().t())
            assert clear.float().mean() > 0.5 and not torch.isfinite(got).any()
            assert torch.equal(got[clear], (torch.sign(sign[clear]) * factor).float())
            w2 = w2.clone()
            w2[128:256] = 0.0
        want, tol = ref_ffn8(x[rows], w1, w2, d, f)
        check(out[rows][:, cols], want[:, cols], (tol + half(F16) * want.abs() + 2.0 ** -25)[:, cols], f"expert {e}")


@pytest.mark.parametrize("T,d,k,dtype", [(2500, 1024, 2, F16), (700, 4104, 1, F16), (700, 8192, 2, F16), (500, 8200, 1, F16),
                                         (700, 2560, 2, torch.float32), (500, 4100, 1, torch.float32), (900, 520, 3, torch.float32)])
def test_gradients_where_each_team_has_several_rows(m, T, d, k, dtype):
    """Every width of a team, two of them to a block, and sums over tokens of more rows than there are teams."""
    test_block_gpu.test_block_norm_gradient(m, T, d, k, dtype, "spg", "hn")
