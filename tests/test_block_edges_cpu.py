"""The block calls on the CPU: outputs that share memory with what is read, or with each other, are refused.

Every call returns before any CUDA work is enqueued."""
import ctypes
import itertools

import pytest


@pytest.fixture(scope="module")
def m():
    from sparse_expert_ffn_layer_gb300 import _build
    _build.build()
    import sparse_expert_ffn_layer_gb300 as mod
    return mod


BIG = 1 << 24                          # the arguments lie this far apart (never dereferenced)


def addresses(names):
    return {n: (i + 1) * BIG for i, n in enumerate(names)}


def pairs(outputs, inputs, allowed):
    for o, i in itertools.chain(itertools.product(outputs, inputs), itertools.combinations(outputs, 2)):
        if (o, i) not in allowed:
            yield o, i


def refused(m, call, outputs, inputs, sizes, allowed=()):
    """Each output at each input's address, in its last 16 bytes, and ending 16 bytes into it."""
    base = addresses(outputs + inputs)
    for o, i in pairs(outputs, inputs, allowed):
        for at in (base[i], base[i] + (sizes[i] - 1) // 16 * 16, base[i] - (sizes[o] - 1) // 16 * 16):
            assert call({**base, o: at}) == m.MOE_ERR_INVALID_ARG, (o, i, at - base[i])


def ptr(a):
    return ctypes.c_void_p(a)


T, d, E, k = 50, 128, 16, 4
S = T * k


def test_norm(m):
    td, row, t4 = T * d * 2, d * 4, T * 4
    sizes = dict(residual=td, y=S * d * 2, slot=t4 * k, w=t4 * k, shared=td, post=row, gate=row, nxt=row, hidden=td, normed=td,
                 rp=t4, rn=t4)

    def call(a):
        p = {n: ptr(v) for n, v in a.items()}
        return m.lib.moe_block_norm(p["residual"], p["y"], p["slot"], p["w"], p["shared"], p["post"], p["gate"], 1.0, p["nxt"],
                                    1e-6, 1, T, d, k, S, p["hidden"], p["normed"], p["rp"], p["rn"], None)
    outs = ["hidden", "normed", "rp", "rn"]
    refused(m, call, outs, [n for n in sizes if n not in outs], sizes, {("hidden", "residual")})
    base = addresses(outs + [n for n in sizes if n not in outs])
    # the same rows may be residual and hidden, rows a few further on not
    assert call({**base, "hidden": base["residual"] + d * 2}) == m.MOE_ERR_INVALID_ARG


def test_norm_backward(m):
    td, row, t4 = T * d * 2, d * 4, T * 4
    sizes = dict(dresidual=td, dy=S * d * 2, dw=t4 * k, dshared=td, dpost=row, dgate=row, dnxt=row,
                 ws=m.moe_block_norm_workspace_size(T, d, k, 1), dh=td, dn=td, hidden=td, rn=t4, nxt=row, y=S * d * 2,
                 slot=t4 * k, w=t4 * k, shared=td, post=row, rp=t4, gate=row)
    outs = ["dresidual", "dy", "dw", "dshared", "dpost", "dgate", "dnxt", "ws"]

    def call(a):
        p = {n: ptr(v) for n, v in a.items()}
        return m.lib.moe_block_norm_backward(p["dh"], p["dn"], p["hidden"], p["rn"], p["nxt"], p["y"], p["slot"], p["w"],
                                             p["shared"], p["post"], p["rp"], p["gate"], 1.0, 1, T, d, k, S, p["dresidual"],
                                             p["dy"], p["dw"], p["dshared"], p["dpost"], p["dgate"], p["dnxt"], p["ws"],
                                             sizes["ws"], None)
    refused(m, call, outs, [n for n in sizes if n not in outs], sizes, {("dresidual", "dh")})
    base = addresses(outs + [n for n in sizes if n not in outs])
    assert call({**base, "dresidual": base["dh"] + d * 2}) == m.MOE_ERR_INVALID_ARG


def test_route(m):
    te, tk = T * E * 4, T * k * 4
    sizes = dict(lo=te, so=te, i=tk, w=tk, x=T * d * 2, Wg=d * E * 4, bias=E * 4, mask=T)
    outs = ["lo", "so", "i", "w"]

    def call(a, given=False):
        p = {n: ptr(v) for n, v in a.items()}
        return m.lib.moe_route(None if given else p["x"], 1, None if given else p["Wg"], p["li"] if given else None, p["bias"],
                               p["mask"], T, d, E, k, 0, 1, 1, 1, 1, 1.0, p["lo"], p["so"], p["i"], p["w"], None)
    refused(m, call, outs, [n for n in sizes if n not in outs], sizes)
    sizes["li"] = te
    refused(m, lambda a: call(a, True), outs, ["li", "bias", "mask"], sizes, {("lo", "li")})
    base = addresses(outs + ["li", "bias", "mask"])
    assert call({**base, "lo": base["li"] + E * 4}, True) == m.MOE_ERR_INVALID_ARG


def test_route_backward(m):
    te, tk, de, td = T * E * 4, T * k * 4, d * E * 4, T * d * 2
    size = ctypes.c_size_t(0)
    assert m.lib.moe_gate_backward_workspace_size(T, d, E, 1, ctypes.byref(size)) == m.MOE_OK
    sizes = dict(dl=te, dWg=de, dx=td, ws=size.value, l=te, i=tk, dw=tk, ds=te, mask=T, x=td, Wg=de, dxi=td)
    outs = ["dl", "dWg", "dx", "ws"]

    def call(a):
        p = {n: ptr(v) for n, v in a.items()}
        return m.lib.moe_route_backward(p["l"], p["i"], p["dw"], p["ds"], p["mask"], p["x"], p["Wg"], 1, T, d, E, k, 0, 1, 1.0,
                                        p["dl"], p["dWg"], p["dxi"], p["dx"], p["ws"], size.value, None)
    refused(m, call, outs, [n for n in sizes if n not in outs], sizes, {("dx", "dxi")})


def test_experts_in_8_bits(m):
    f = 256
    sizes = dict(out=S * d * 2, ws=m.moe_expert_fp8_workspace_size(T, d, f, E, S, 1), x=T * d * 2, perm=S * 4, off=(E + 1) * 4,
                 W1=E * d * f, s1=E * d * f // 16384 * 4, W2=E * d * f, s2=E * d * f // 16384 * 4)

    def call(a):
        p = {n: ptr(v) for n, v in a.items()}
        return m.lib.moe_expert_ffn_fp8(p["x"], p["perm"], p["off"], p["W1"], p["s1"], p["W2"], p["s2"], 1, T, d, f, E, S,
                                        p["out"], p["ws"], sizes["ws"], None)
    refused(m, call, ["out", "ws"], [n for n in sizes if n not in ("out", "ws")], sizes, {("out", "x")})
    sizes = dict(q=2 * 128 * 256, s=2 * 2 * 4, W=2 * 128 * 256 * 2)

    def quantize(a):
        return m.lib.moe_fp8_quantize(ptr(a["W"]), 1, 2, 128, 256, ptr(a["q"]), ptr(a["s"]), None)
    refused(m, quantize, ["q", "s"], ["W"], sizes)
