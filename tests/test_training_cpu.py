"""Training and adapter calls on the CPU: workspace sizes and refusals.  Every call returns before
any CUDA work is enqueued."""
import ctypes
import os
import re

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    from sparse_expert_ffn_layer_gb300 import _build
    _build.build()
    import sparse_expert_ffn_layer_gb300 as mod
    return mod


P = ctypes.c_void_p(0x10000)       # never dereferenced: every call below fails its host checks
ODD = ctypes.c_void_p(0x10002)
S0 = ctypes.c_void_p(0)


def test_workspace_sizes(m):
    assert m.moe_balance_workspace_size(64, 8) % 256 == 0
    assert m.moe_balance_workspace_size(1 << 20, 1024) >= 4 * 2 * 1024 * 2 * 148
    # room for the status word and dh [S_max, r]
    for r in (8, 16, 128):
        assert m.moe_adapter_workspace_size(100, 64, 64, r, 4, 100, torch.float16) >= 256 + 400 * r
    assert m.moe_adapter_workspace_size(0, 64, 64, 8, 4, 0, m.MOE_F32) >= 256
    assert m.moe_gate_backward_workspace_size(64, 128, 8, torch.float16) >= 256
    for args, code in [((-1, 8), 1), ((4, 0), 1), ((4, 1025), 2), ((1 << 22, 1024), 2)]:
        with pytest.raises(m.MoeError) as e:
            m.moe_balance_workspace_size(*args)
        assert e.value.code == code
    for args, code in [((8, 100, 64, 8, 4, 8, torch.float16), 2), ((8, 64, 100, 8, 4, 8, torch.float16), 2),
                       ((8, 64, 64, 12, 4, 8, torch.float16), 2), ((8, 64, 64, 136, 4, 8, torch.float16), 2),
                       ((8, 64, 64, 8, 1025, 8, torch.float16), 2), ((8, 64, 66, 8, 4, 8, torch.float32), 2),
                       ((8, 64, 64, 0, 4, 8, torch.float16), 1), ((8, 64, 64, 8, 0, 8, torch.float16), 1),
                       ((8, 64, 64, 8, 4, -1, torch.float16), 1), ((8, 64, 64, 8, 4, 8, 7), 1)]:
        with pytest.raises(m.MoeError) as e:
            m.moe_adapter_workspace_size(*args)
        assert e.value.code == code
    with pytest.raises(m.MoeError):
        m.moe_gate_backward_workspace_size(8, 100, 8, torch.float16)
    with pytest.raises(TypeError):
        m.moe_adapter_workspace_size(8, 64, 64, 8, 4, 8, torch.bfloat16)


def test_one_workspace_serves_every_smaller_batch(m):
    rows = [*range(0, 1400, 9), *range(1400, 20000, 311)]
    for dt in (torch.float16, torch.float32):
        for d, E in [(1024, 64), (256, 8), (3584, 128), (1024, 13), (512, 1000)]:
            size = [m.moe_gate_backward_workspace_size(T, d, E, dt) for T in rows]
            assert size == sorted(size)
        for di, do, r, N in [(1024, 1024, 16, 8), (2048, 8192, 32, 4), (3584, 3584, 64, 64), (64, 256, 128, 1)]:
            size = [m.moe_adapter_workspace_size(T, di, do, r, N, T, dt) for T in rows]
            assert size == sorted(size)
    for E in (8, 1000):
        size = [m.moe_balance_workspace_size(T, E) for T in rows]
        assert size == sorted(size)


def test_balance_and_gate_refusals(m):
    f = m.lib.moe_balance_loss

    def bal(logits=P, idx=P, T=8, E=4, k=1, counts=P, pm=P, losses=P, nv=P, ws=P, n=1 << 24):
        return f(logits, idx, None, T, E, k, counts, pm, losses, nv, ws, n, S0)
    assert bal(k=3) == bal(k=2, E=1) == bal(T=-1) == bal(E=0) == m.MOE_ERR_INVALID_ARG
    assert bal(logits=None) == bal(idx=None) == bal(counts=None) == bal(losses=None) == \
        bal(pm=None) == bal(nv=None) == m.MOE_ERR_INVALID_ARG
    assert bal(E=1025) == bal(T=1 << 28, E=1000) == bal(logits=ODD) == m.MOE_ERR_UNSUPPORTED
    assert bal(ws=None) == bal(n=100) == m.MOE_ERR_WORKSPACE
    g = m.lib.moe_gate_topk_backward

    def gate(logits=P, idx=P, dw=P, dl=P, counts=P, nv=P, mask=None, x=P, Wg=P, dt=1, T=8, d=64, E=4,
             k=1, dlogits=P, dWg=P, din=None, dx=P, ws=P, n=1 << 24):
        return g(logits, idx, dw, dl, counts, nv, mask, x, Wg, dt, T, d, E, k, dlogits, dWg, din, dx,
                 ws, n, S0)
    inv = m.MOE_ERR_INVALID_ARG
    assert gate(dw=None, dl=None) == inv                       # nothing to differentiate
    assert gate(counts=None) == gate(nv=None) == gate(dlogits=None) == inv
    assert gate(x=None) == gate(Wg=None) == gate(dt=5) == gate(d=0) == inv
    assert gate(dx=None, din=P) == inv
    assert gate(d=68) == gate(dt=0, d=66) == gate(x=ODD) == m.MOE_ERR_UNSUPPORTED
    assert gate(ws=None) == gate(n=8) == m.MOE_ERR_WORKSPACE
    assert gate(T=0, dWg=None) == m.MOE_OK


def test_combine_backward_refusals(m):
    f = m.lib.moe_combine_backward

    def comb(dout=P, y=P, slot=P, w=P, dt=1, T=8, d=64, k=1, S=8, dy=P, dw=P):
        return f(dout, y, slot, w, dt, T, d, k, S, dy, dw, S0)
    inv = m.MOE_ERR_INVALID_ARG
    assert comb(dy=None, dw=None) == comb(dout=None) == comb(slot=None) == inv
    assert comb(w=None) == comb(y=None) == comb(k=3) == comb(dt=9) == comb(S=-1) == comb(d=0) == inv
    assert comb(dout=ODD) == comb(y=ODD) == m.MOE_ERR_UNSUPPORTED
    assert comb(T=0) == m.MOE_OK


def test_combine_backward_refuses_lengths_beyond_its_indices(m):
    f = m.lib.moe_combine_backward
    for T, d in [((1 << 31) - 1, 8), ((1 << 30) + 1, 8), (8, (1 << 31) - 8), (8, (1 << 20) + 8)]:
        assert f(P, P, P, P, 1, T, d, 1, 8, P, P, S0) == m.MOE_ERR_UNSUPPORTED


def test_adapter_refusals(m):
    f, b = m.lib.moe_adapter_forward, m.lib.moe_adapter_backward

    def fwd(x=P, perm=P, off=P, A=P, B=P, sc=P, base=None, dt=1, T=8, di=64, do=64, r=8, N=4, S=8, out=P,
            hid=None, ws=P, n=1 << 20):
        return f(x, perm, off, A, B, sc, base, dt, T, di, do, r, N, S, out, hid, ws, n, S0)
    inv, uns = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED
    assert fwd(x=None) == fwd(perm=None) == fwd(off=None) == fwd(A=None) == fwd(sc=None) == inv
    assert fwd(out=None) == fwd(T=-1) == fwd(S=-1) == fwd(r=0) == fwd(N=0) == fwd(dt=3) == inv
    assert fwd(di=60) == fwd(do=4) == fwd(r=12) == fwd(r=136) == fwd(N=1025) == uns
    assert fwd(x=ODD) == fwd(base=ODD) == fwd(hid=ODD) == fwd(off=ODD) == uns
    assert fwd(ws=None) == fwd(n=256) == m.MOE_ERR_WORKSPACE
    assert fwd(T=0) == fwd(S=0) == m.MOE_OK

    def bwd(dy=P, x=P, hid=P, perm=P, off=P, A=P, B=P, sc=P, din=None, dt=1, T=8, di=64, do=64, r=8,
            N=4, S=8, dx=P, dA=P, dB=P, ws=P, n=1 << 20):
        return b(dy, x, hid, perm, off, A, B, sc, din, dt, T, di, do, r, N, S, dx, dA, dB, ws, n, S0)
    assert bwd(dx=None, dA=None, dB=None) == bwd(x=None) == bwd(hid=None) == bwd(dy=None) == inv
    assert bwd(dx=None, din=P) == bwd(A=None) == inv
    assert bwd(dA=ODD) == bwd(di=60) == uns
    assert bwd(n=256) == m.MOE_ERR_WORKSPACE
    assert bwd(T=0, dA=None, dB=None) == m.MOE_OK


def test_empty_batch_whose_only_output_has_no_rows(m):
    """The tokens' gradient of an empty batch is an empty tensor, whose pointer is null."""
    assert m.lib.moe_adapter_backward(None, None, None, P, P, P, P, P, None, 1, 0, 64, 64, 8, 4, 8, None, None, None,
                                      None, 0, S0) == m.MOE_OK
    assert m.lib.moe_adapter_backward(P, P, P, P, P, P, P, P, None, 1, 8, 64, 64, 8, 4, 8, None, None, None,
                                      P, 1 << 20, S0) == m.MOE_ERR_INVALID_ARG
    assert m.lib.moe_combine_backward(None, None, None, None, 1, 0, 64, 1, 8, None, None, S0) == m.MOE_OK


def test_outputs_that_would_overwrite_what_is_read(m):
    """The same buffer as an input that other blocks still read is refused."""
    Q, inv = ctypes.c_void_p(0x20000), m.MOE_ERR_INVALID_ARG
    n = 1 << 24
    assert m.lib.moe_adapter_forward(P, Q, Q, Q, Q, Q, P, 1, 8, 64, 64, 8, 4, 8, P, None, Q, n, S0) == inv
    b = m.lib.moe_adapter_backward
    assert b(P, Q, Q, Q, Q, Q, Q, Q, None, 1, 8, 64, 64, 8, 4, 8, P, None, None, Q, n, S0) == inv
    assert b(Q, P, Q, Q, Q, Q, Q, Q, None, 1, 8, 64, 64, 8, 4, 8, P, Q, None, Q, n, S0) == inv
    assert m.lib.moe_combine_backward(P, Q, Q, Q, 1, 8, 64, 1, 8, P, Q, S0) == inv
    assert m.lib.moe_gate_topk_backward(Q, Q, Q, None, None, None, None, P, Q, 1, 8, 64, 4, 1, Q, Q, None, P,
                                        Q, n, S0) == inv


def test_binding_refuses_what_the_kernels_would_misread(m):
    T, d, r, N = 4, 16, 8, 2
    x, out = torch.zeros(T, d, dtype=torch.float16), torch.zeros(T, d, dtype=torch.float16)
    perm, off = torch.zeros(T, dtype=torch.int32), torch.zeros(N + 1, dtype=torch.int32)
    A, B = torch.zeros(N, d, r, dtype=torch.float16), torch.zeros(N, r, d, dtype=torch.float16)
    sc, ws = torch.zeros(N), torch.zeros(1 << 16, dtype=torch.uint8)

    def fwd(**kw):
        a = dict(tokens=x, perm=perm, offsets=off, A=A, B=B, scale=sc, out=out, workspace=ws)
        a.update(kw)
        return m.moe_adapter_forward(**a)
    with pytest.raises(ValueError, match="CUDA device"):
        fwd()
    with pytest.raises(TypeError, match="perm"):
        fwd(perm=perm.long())
    with pytest.raises(ValueError, match="B has shape"):
        fwd(B=torch.zeros(N, r + 1, d, dtype=torch.float16))
    with pytest.raises(TypeError, match="A is"):
        fwd(A=A.float())
    with pytest.raises(ValueError, match="contiguous"):
        fwd(tokens=torch.zeros(d, T, dtype=torch.float16).t())
    with pytest.raises(ValueError, match="offsets has shape"):
        fwd(offsets=off[:N].contiguous())
    with pytest.raises(TypeError, match="unsupported dtype"):
        fwd(tokens=x.bfloat16(), A=A.bfloat16(), B=B.bfloat16(), out=out.bfloat16())
    logits, idx = torch.zeros(T, 4), torch.zeros(T, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="counts is required"):
        m.moe_gate_topk_backward(logits, idx, logits, dlosses=torch.zeros(2))
    with pytest.raises(ValueError, match="tokens is required"):
        m.moe_gate_topk_backward(logits, idx, logits, dtopk_w=torch.zeros(T, 1), dWg=torch.zeros(d, 4))
    with pytest.raises(TypeError, match="token_mask"):
        m.moe_balance_loss(logits, idx, torch.zeros(4, dtype=torch.int32), torch.zeros(4), torch.zeros(2),
                           torch.zeros(1, dtype=torch.int32), ws, token_mask=torch.zeros(T))
    with pytest.raises(ValueError, match="expert_out has shape"):
        m.moe_combine_backward(x, torch.zeros(T, d + 1, dtype=torch.float16), idx, torch.zeros(T, 1),
                               dtopk_w=torch.zeros(T, 1))


CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_expert_ffn_layer_gb300", "csrc")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def block_behind(text, at):
    """The braces' content that opens at or behind `at`."""
    i = text.index("{", at)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i + 1:j]
    raise AssertionError("unbalanced")


def test_no_warp_leaves_a_loop_whose_barrier_others_wait_at():
    """A bounded wait may give up in one warp and not in the next.  In a loop that meets at a barrier of
    several warps, each warp therefore goes round as often as the others, whatever its waits say."""
    text = source("gate_grad.cu")
    seen = 0
    for mt in re.finditer(r"\bfor \(", text):
        head = text[mt.start():text.index("{", mt.start())]
        body = block_behind(text, mt.start())
        if "bar.sync" not in body:
            continue
        seen += 1
        assert not re.search(r"\b(break|return|continue|goto)\b", body.split("bar.sync")[0]), head
        assert not re.search(r"\bok\b", head), head
    assert seen >= 1


def test_combine_backward_needs_the_experts_output_for_the_gate_weights(m):
    """Without it (and without a dexpert_out that says how many slots there are) the gradient was zero."""
    x, idx = torch.zeros(4, 16, dtype=torch.float16), torch.zeros(4, 1, dtype=torch.int32)
    for dy in (None, torch.zeros(4, 16, dtype=torch.float16)):
        with pytest.raises(ValueError, match="expert_out is required"):
            m.moe_combine_backward(x, None, idx, torch.zeros(4, 1), dy, torch.zeros(4, 1))


def test_blocks_that_give_up_wait_for_their_copies():
    """Each kernel with bounded waits on bulk copies waits for those in flight at its end: its block's
    shared memory may be another's a moment later."""
    for name, body, end in [("gate_grad.cu", "void wgrad_block(", "end_block"), ("gate_grad.cu", "void dx_block(", "end_block"),
                            ("adapter.cu", "adapter_shrink_kernel(", "ring.finish"),
                            ("adapter.cu", "adapter_expand_kernel(", "ring.finish")]:
        text = source(name)
        last = block_behind(text, text.index(body)).strip().splitlines()[-1]
        assert last.strip().startswith(end), (name, body, last)
    assert "mbar_drain" in block_behind(source("gate_grad.cu"), source("gate_grad.cu").index("void end_block("))
    assert "mbar_drain" in block_behind(source("adapter.cu"), source("adapter.cu").index("void finish("))


def test_no_block_writes_to_another_before_the_cluster_has_met():
    """Another block's shared memory may be touched only once that block has started, which a cluster
    barrier says.  (Reads through map_shared_rank in the kernels are of complete data, behind cl.sync.)"""
    for name, body in [("router_loss.cu", "void join_records("), ("adapter.cu", "adapter_f16_kernel("),
                       ("adapter.cu", "adapter_f32_kernel(")]:
        text = source(name)
        kernel = block_behind(text, text.index(body))
        first = kernel.index("map_shared_rank")
        assert "cl.sync()" in kernel[:first] or "cluster_wait()" in kernel[:first], (name, body)
