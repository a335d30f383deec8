"""The block calls on the CPU: workspace sizes and refusals.  Every call returns before any CUDA work is enqueued."""
import ctypes
import re

import pytest
import torch

from test_training_cpu import block_behind, source


@pytest.fixture(scope="module")
def m():
    from sparse_expert_ffn_layer_gb300 import _build
    _build.build()
    import sparse_expert_ffn_layer_gb300 as mod
    return mod


def ptr(n):                        # never dereferenced: every call below fails its host checks
    return ctypes.c_void_p(0x10000 * n)


P, Q, R = ptr(1), ptr(2), ptr(3)
ODD = ctypes.c_void_p(0x10002)
S0 = ctypes.c_void_p(0)
INF, NAN = float("inf"), float("nan")


def test_workspace_sizes(m):
    rows = [*range(0, 700, 7), *range(700, 20000, 611)]
    for d, f, E in [(128, 128, 1), (1024, 4096, 128), (3584, 14336, 64)]:
        size = [m.moe_expert_fp8_workspace_size(S, d, f, E, S, torch.float16) for S in rows]
        assert size == sorted(size) and size[-1] >= rows[-1] * (d + f) and all(s % 256 == 0 for s in size)
    for dt, d in [(torch.float16, 8), (torch.float16, 3584), (torch.float32, 1024), (torch.float16, 16384)]:
        size = [m.moe_block_norm_workspace_size(T, d, 2, dt) for T in rows]
        assert size == sorted(size) and size[0] >= 8 * d
    for args, code in [((4, 100, 128, 2, 4, torch.float16), 2), ((4, 128, 200, 2, 4, torch.float16), 2),
                       ((4, 128, 128, 1025, 4, torch.float16), 2), ((4, 128, 128, 2, 4, torch.float32), 2),
                       ((4, 128, 128, 0, 4, torch.float16), 1), ((4, 128, 128, 2, -1, torch.float16), 1),
                       ((-1, 128, 128, 2, 4, torch.float16), 1), ((4, 128, 128, 2, 4, 9), 1),
                       ((4, 1 << 21, 128, 2, 4, torch.float16), 2)]:
        with pytest.raises(m.MoeError) as e:
            m.moe_expert_fp8_workspace_size(*args)
        assert e.value.code == code, args
    for args, code in [((4, 12, 2, torch.float16), 2), ((4, 6, 2, torch.float32), 2), ((4, 16392, 2, torch.float16), 2),
                       ((4, 64, 17, torch.float16), 2), ((-1, 64, 2, torch.float16), 1), ((4, 0, 2, torch.float16), 1),
                       ((4, 64, -1, torch.float16), 1), ((4, 64, 2, 5), 1)]:
        with pytest.raises(m.MoeError) as e:
            m.moe_block_norm_workspace_size(*args)
        assert e.value.code == code, args


def test_route_refusals(m):
    inv, uns = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED

    def route(x=None, dt=1, Wg=None, li=P, b=None, mask=None, T=8, d=64, E=16, k=4, score=0, G=1, top=1, gt=1, scale=1.0,
              lo=None, so=None, i=Q, w=R):
        return m.lib.moe_route(x, dt, Wg, li, b, mask, T, d, E, k, score, G, top, gt, 1, scale, lo, so, i, w, S0)
    assert route(T=0) == m.MOE_OK
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=17, E=17 - 1), dict(score=2), dict(G=3), dict(G=0), dict(top=0),
                dict(G=4, top=5), dict(gt=0), dict(gt=3), dict(scale=NAN), dict(scale=INF), dict(d=0), dict(dt=4),
                dict(i=None), dict(w=None), dict(li=None), dict(li=None, x=P, Wg=P), dict(li=None, x=P, lo=P),
                dict(E=16, G=8, top=1, k=3), dict(so=P), dict(li=None, x=P, Wg=P, lo=R, so=R)):
        assert route(**bad) == inv, bad
    for bad in (dict(k=17, E=32), dict(E=1025), dict(E=64, G=64, top=64), dict(T=1 << 22, E=1024), dict(li=ODD), dict(i=ODD),
                dict(b=ODD), dict(w=ODD), dict(so=ODD)):
        assert route(**bad) == uns, bad

    def back(l=P, i=Q, dw=Q, ds=None, x=None, Wg=None, dt=1, T=8, d=64, E=16, k=4, score=0, scale=1.0, dl=R, dWg=None,
             dxi=None, dx=None, ws=None, n=0):
        return m.lib.moe_route_backward(l, i, dw, ds, None, x, Wg, dt, T, d, E, k, score, 1, scale, dl, dWg, dxi, dx, ws, n, S0)
    assert back(T=0) == m.MOE_OK
    for bad in (dict(l=None), dict(i=None), dict(dw=None), dict(dl=None), dict(k=0), dict(score=-1), dict(scale=INF),
                dict(dWg=P), dict(dx=P), dict(dxi=P), dict(dl=P), dict(ds=R), dict(dWg=P, x=P, dt=3, ws=Q, n=1 << 30),
                dict(dWg=Q, x=P, Wg=Q, dx=P, ws=Q, n=1 << 30)):
        assert back(**bad) == inv, bad
    for bad in (dict(k=17, E=64), dict(dWg=P, x=P, d=60, ws=Q, n=1 << 30), dict(ds=ODD), dict(dw=ODD)):
        assert back(**bad) == uns, bad
    assert back(dWg=P, x=P) == back(dWg=P, x=P, ws=Q, n=64) == m.MOE_ERR_WORKSPACE
    # two experts a token and no more where the layer's own calls take them, up to 16 for the plan
    assert m.lib.moe_dispatch(P, 0, 32, 16, 1.0, P, P, P, P, P, S0) == m.MOE_OK
    for k in (0, 17, 5):
        assert m.lib.moe_dispatch(P, 8, 32 if k != 5 else 4, k, 1.0, P, P, P, P, P, S0) == inv


def test_fp8_refusals(m):
    inv, uns, n = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED, 1 << 30
    quant = m.lib.moe_fp8_quantize
    for a in ((None, 1, 2, 128, 128, Q, R), (P, 5, 2, 128, 128, Q, R), (P, 1, 0, 128, 128, Q, R), (P, 1, 2, 0, 128, Q, R),
              (P, 1, 2, 128, 128, None, R), (P, 1, 2, 128, 128, Q, None), (P, 1, 2, 128, 128, P, R)):
        assert quant(*a, S0) == inv, a
    for a in ((P, 1, 2, 100, 128, Q, R), (P, 1, 2, 128, 64, Q, R), (ODD, 1, 2, 128, 128, Q, R), (P, 0, 2, 128, 128, ODD, R),
              (P, 1, 2, 128, 128, Q, ODD), (P, 1, 1 << 10, 1 << 20, 1 << 20, Q, R)):
        assert quant(*a, S0) == uns, a

    def ffn(x=P, perm=P, off=P, W1=P, s1=P, W2=P, s2=P, dt=1, T=8, d=128, f=256, E=4, S=8, out=Q, ws=R, n=n):
        return m.lib.moe_expert_ffn_fp8(x, perm, off, W1, s1, W2, s2, dt, T, d, f, E, S, out, ws, n, S0)
    assert ffn(T=0, ws=None, n=0) == ffn(S=0, ws=None, n=0) == m.MOE_OK
    for q in ("x", "perm", "off", "W1", "s1", "W2", "s2", "out"):
        assert ffn(**{q: None}) == inv, q
        assert ffn(**{q: ODD}) == uns, q
    for bad in (dict(T=-1), dict(S=-1), dict(E=0), dict(d=0), dict(dt=2)):
        assert ffn(**bad) == inv, bad
    for bad in (dict(d=64), dict(f=100), dict(E=1025), dict(dt=0), dict(ws=ODD)):
        assert ffn(**bad) == uns, bad
    assert ffn(ws=None) == ffn(n=1024) == m.MOE_ERR_WORKSPACE


def test_norm_refusals(m):
    inv, uns = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED
    H, N, Y = ptr(4), ptr(5), ptr(6)

    def norm(res=P, y=Y, slot=Q, w=Q, sh=None, pw=None, gate=None, alpha=1.0, nw=Q, eps=1e-6, dt=1, T=8, d=64, k=2, S=16,
             h=H, n=N, rp=None, rn=None):
        return m.lib.moe_block_norm(res, y, slot, w, sh, pw, gate, alpha, nw, eps, dt, T, d, k, S, h, n, rp, rn, S0)
    assert norm(T=0) == m.MOE_OK
    none = dict(y=None, slot=None, w=None, k=0, S=0)
    for bad in (dict(T=-1), dict(d=0), dict(k=-1), dict(S=-1), dict(dt=7), dict(eps=-1e-6), dict(eps=NAN), dict(eps=INF),
                dict(alpha=NAN), dict(alpha=INF), dict(res=None), dict(y=None), dict(slot=None), dict(w=None), dict(k=0),
                dict(h=None), dict(nw=None), dict(n=None), dict(rp=Q), dict(n=None, nw=None, rn=Q), dict(n=H), dict(n=P),
                dict(h=Y), dict(n=Y), dict(sh=H), dict(**none, pw=Q), dict(**none, gate=Q), dict(**none, h=None, n=None, nw=None)):
        assert norm(**bad) == inv, bad
    for bad in (dict(d=60), dict(d=16392), dict(k=17), dict(res=ODD), dict(y=ODD), dict(slot=ODD), dict(w=ODD), dict(sh=ODD),
                dict(pw=ODD), dict(gate=ODD), dict(nw=ODD), dict(h=ODD), dict(n=ODD), dict(dt=0, d=66)):
        assert norm(**bad) == uns, bad

    def back(dh=P, dn=None, h=None, rn=None, nw=None, y=Y, slot=Q, w=Q, sh=None, pw=None, rp=None, gate=None, alpha=1.0,
             dt=1, T=8, d=64, k=2, S=16, dr=H, de=None, dw=None, dsh=None, dpw=None, dg=None, dnw=None, ws=None, n=0):
        return m.lib.moe_block_norm_backward(dh, dn, h, rn, nw, y, slot, w, sh, pw, rp, gate, alpha, dt, T, d, k, S, dr, de,
                                             dw, dsh, dpw, dg, dnw, ws, n, S0)
    assert back(T=0) == m.MOE_OK
    nxt = dict(dn=N, h=N, rn=Q, nw=Q)
    for bad in (dict(T=-1), dict(S=-1), dict(alpha=INF), dict(dt=3), dict(dh=None), dict(dn=N), dict(dn=N, h=N, rn=Q),
                dict(dn=N, h=N, nw=Q), dict(y=None), dict(slot=None), dict(w=None), dict(k=0), dict(pw=Q), dict(dg=Q),
                dict(dpw=Q), dict(dnw=Q), dict(dr=None), dict(**none, dw=Q), dict(**none, de=Q), dict(**none, dsh=Q),
                dict(**none, pw=Q, rp=Q), dict(de=Y), dict(de=P), dict(dsh=P), dict(**nxt, dr=N), dict(de=H), dict(de=Q, dsh=Q)):
        assert back(**bad) == inv, bad
    for bad in (dict(d=60), dict(k=17), dict(dh=ODD), dict(dr=ODD), dict(de=ODD), dict(dw=ODD), dict(y=ODD)):
        assert back(**bad) == uns, bad
    assert back(**nxt, dnw=Q) == back(**nxt, dnw=Q, ws=R, n=128) == m.MOE_ERR_WORKSPACE


def test_binding_refuses_what_the_kernels_would_misread(m):
    T, E, k, d = 4, 8, 2, 128
    x, li = torch.zeros(T, d, dtype=torch.float16), torch.zeros(T, E)
    idx, w = torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k)
    with pytest.raises(ValueError, match="CUDA device"):
        m.moe_route(None, None, k, idx, w, logits_in=li)
    with pytest.raises(TypeError, match="topk_idx"):
        m.moe_route(None, None, k, idx.long(), w, logits_in=li)
    with pytest.raises(ValueError, match="topk_w has shape"):
        m.moe_route(None, None, k, idx, torch.zeros(T, k + 1), logits_in=li)
    with pytest.raises(ValueError, match="logits_out is required"):
        m.moe_route(x, torch.zeros(d, E), k, idx, w)
    with pytest.raises(ValueError, match="bias has shape"):
        m.moe_route(None, None, k, idx, w, logits_in=li, bias=torch.zeros(E + 1))
    with pytest.raises(TypeError, match="token_mask"):
        m.moe_route(None, None, k, idx, w, logits_in=li, token_mask=torch.zeros(T))
    with pytest.raises(ValueError, match="tokens is required"):
        m.moe_route_backward(li, idx, li, dtopk_w=w, dWg=torch.zeros(d, E))
    with pytest.raises(ValueError, match="dscores has shape"):
        m.moe_route_backward(li, idx, li, dscores=torch.zeros(T, E - 1))
    W = torch.zeros(2, d, 256, dtype=torch.float16)
    q, s = torch.zeros(2, 256, d, dtype=torch.float8_e4m3fn), torch.zeros(2, 2, 1)
    with pytest.raises(ValueError, match="Wq has shape"):
        m.moe_fp8_quantize(W, q.view(2, d, 256), s)
    with pytest.raises(TypeError, match="Wq is"):
        m.moe_fp8_quantize(W, q.float(), s)
    with pytest.raises(ValueError, match="scales has shape"):
        m.moe_fp8_quantize(W, q, torch.zeros(2, 1, 2))
    perm, off, ws = torch.zeros(T, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.uint8)
    W2, s2 = torch.zeros(2, d, 256, dtype=torch.float8_e4m3fn), torch.zeros(2, 1, 2)

    def ffn(**kw):
        a = dict(tokens=x, perm=perm, offsets=off, W1q=q, W1s=s, W2q=W2, W2s=s2, S_max=T, expert_out=torch.zeros_like(x), workspace=ws)
        a.update(kw)
        return m.moe_expert_ffn_fp8(**a)
    with pytest.raises(ValueError, match="CUDA device"):
        ffn()
    with pytest.raises(ValueError, match="S_max"):
        ffn(S_max=T + 1)
    with pytest.raises(ValueError, match="W2q has shape"):
        ffn(W2q=q)
    with pytest.raises(ValueError, match="contiguous"):
        ffn(W1q=W2.transpose(1, 2))
    with pytest.raises(ValueError, match="offsets has shape"):
        ffn(offsets=perm)
    with pytest.raises(ValueError, match="slot_of has shape"):
        m.moe_block_norm(x, x, expert_out=x, slot_of=idx[:2], topk_w=w)
    with pytest.raises(TypeError, match="expert_out"):
        m.moe_block_norm(x, x, expert_out=x.float(), slot_of=idx, topk_w=w)
    with pytest.raises(TypeError, match="post_w"):
        m.moe_block_norm(x, x, shared=x, post_w=torch.zeros(d, dtype=torch.float16))
    with pytest.raises(ValueError, match="dhidden or dnormed"):
        m.moe_block_norm_backward(dresidual=x)


def test_no_warp_leaves_a_loop_whose_barrier_others_wait_at():
    """A bounded wait may give up in one warp and not in the next.  Around each barrier of several warps, each warp goes
    round as often as the others, whatever its waits say."""
    text = source("fp8.cu")

    def without(before, heads):                       # inner loops may end early: they are over before the barrier
        for inner in heads:
            while inner in before:
                at = before.index(inner)
                end = before.index("{", at) + len(block_behind(before, at)) + 2
                before = before[:at] + before[end:]
        return before

    results = block_behind(text, text.index("void finish("))
    assert results.count("bar.sync") == 1
    before = without(results.split("bar.sync")[0], ("for (int c = 0; c < C8; ++c) {",))
    assert not re.search(r"\b(break|return|continue|goto)\b", before)
    for name in ("fp8_gemm_kernel(", "fp8_long_kernel("):
        kernel = block_behind(text, text.index(name))
        assert "bar.sync" not in kernel
        seen = 0
        for mt in re.finditer(r"\bfor \(", kernel):
            head = kernel[mt.start():kernel.index("{", mt.start())]
            body = block_behind(kernel, mt.start())
            if "finish<" not in body:
                continue
            seen += 1
            before = body.split("finish<")[0]
            # blocks that hand their sums to another one of the cluster: all warps of the block
            if "if (part > 0)" in body:
                before = before.replace(block_behind(body, body.index("if (part > 0)")), "")
            before = without(before, ("for (int kb",))
            assert not re.search(r"\b(break|return|continue|goto)\b", before), head
            assert not re.search(r"\bok\b", head), head
        assert seen == (1 if name == "fp8_gemm_kernel(" else 2)   # items, and their parts


def test_blocks_that_give_up_wait_for_their_copies():
    """The block's shared memory may be another's a moment after its end."""
    text = source("fp8.cu")
    for name, rings in (("fp8_gemm_kernel(", "a_full : b_full"), ("fp8_long_kernel(", "&full[st]")):
        end = block_behind(text, text.index(name))
        end = end[end.rindex("__syncthreads()"):]
        # the rings' loads by the warps that issued them, and the products
        assert rings in end and end.count("mbar_drain") == 2 and "tmem_dealloc" in end
        assert end.rindex("mbar_drain") < end.index("tmem_dealloc")


def test_no_block_of_a_cluster_writes_to_another_that_is_not_there():
    """Before the first write to another block's shared memory the cluster has met, and it meets again before a block
    leaves: also where a wait gave up."""
    kernel = block_behind(source("fp8.cu"), source("fp8.cu").index("fp8_gemm_kernel("))
    assert kernel.count("cluster_meet()") == 2
    assert kernel.index("cluster_meet()") < kernel.index("store_remote")
    assert kernel.rindex("cluster_meet()") > kernel.rindex("tmem_dealloc")
    kernel = block_behind(source("fp8.cu"), source("fp8.cu").index("fp8_long_kernel("))
    first = kernel.index("cluster_meet()")
    assert first < min(kernel.index(w) for w in ("load_rows_pair", "commit_pair", "arrive_remote_tmem"))
    last = kernel.rindex("__syncthreads()")
    assert kernel.index("cluster_meet()", last) < kernel.index("tmem_dealloc_pair") < kernel.rindex("cluster_meet()")
    # the warps that wait for arrivals of the other block see the last of them before they end
    assert "n < a.na && ok" in kernel and "n < 2 && ok" in kernel
