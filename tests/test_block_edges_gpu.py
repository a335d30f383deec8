"""The block calls where their documentation allows something out of the ordinary."""
import pytest
import torch

from test_block_gpu import experts8, gen, norm_inputs, randn

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
