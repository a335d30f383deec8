"""Operators around a block of routed experts as measured work: cases, plain forms and calls.

Three operators: routing to experts by softmax or sigmoid scores with a balance bias, expert groups,
top-k and renormalised weights, with its gradient down to the gate (`route`: moe_route, `route_grad`:
moe_route_backward); the experts' products in 8-bit floating point with a scale for each block of 128
(`quantize`: moe_fp8_quantize, `ffn`: moe_expert_ffn_fp8); and the block's end and the next one's start,
the sum over a token's experts, its norm, gate and residual, and the norm after it, with their gradient
(`norm`: moe_block_norm, `norm_grad`: moe_block_norm_backward).  With `own` false, `run` computes them
from elementary torch operations; with `own` true it makes the library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f16": torch.float16, "f32": torch.float32}
_FP8_MAX = 448.0                       # largest finite value of e4m3


def listed():
    return [
        # routing of one token while serving (latency), of a ragged batch with padding tokens by plain
        # softmax, and of a long prefill over many experts in groups
        dict(name="route_T1_E128_k2", op="route", T=1, E=128, k=2, score="softmax", groups=1, top_groups=1,
             group_top=1, bias=False, mask=False, renorm=True),
        dict(name="route_T4099_E60_k4_padded", op="route", T=4099, E=60, k=4, score="softmax", groups=1,
             top_groups=1, group_top=1, bias=False, mask=True, renorm=False),
        dict(name="route_T16384_E256_k8_groups", op="route", T=16384, E=256, k=8, score="sigmoid", groups=8,
             top_groups=4, group_top=2, bias=True, mask=False, renorm=True),
        # its gradient: a small 32-bit layer, and the accumulated batch of a wide one
        dict(name="route_grad_T500_d64_E16_f32", op="route_grad", T=500, d=64, E=16, k=4, score="softmax",
             renorm=False, mask=True, dtype="f32"),
        dict(name="route_grad_T16384_d2048_E128_k8", op="route_grad", T=16384, d=2048, E=128, k=8,
             score="sigmoid", renorm=True, mask=False, dtype="f16"),
        # a layer's weights brought to 8 bits when it is loaded: 16 experts of the PR-MoE shape
        dict(name="quantize_E16_2048x8192", op="quantize", E=16, K=2048, N=8192),
        # experts in 8 bits: the 350M+MoE-128 layer at decode size, many small experts with eight
        # a token (a prefill bound by the products), the 2.4B+MoE-128 top-2 layer with capacity drops
        dict(name="ffn_T8_d1024_f4096_E128", op="ffn", T=8, d=1024, f=4096, E=128, k=1, cf=0.0, skew=0.0),
        dict(name="ffn_T4096_d2048_f2048_E64_k8", op="ffn", T=4096, d=2048, f=2048, E=64, k=8, cf=0.0,
             skew=0.4),
        dict(name="ffn_T16384_d3584_f14336_E128_k2", op="ffn", T=16384, d=3584, f=14336, E=128, k=2, cf=1.25,
             skew=0.2),
        # the block's end: one token while serving, the 2.4B top-2 layer's prefill; and its gradient in a
        # training step of a ragged batch with dropped assignments
        dict(name="norm_T1_d1024_k1", op="norm", T=1, d=1024, k=1, shared=False, post=True, gate=False,
             drop=0.0, dtype="f16"),
        dict(name="norm_T16384_d3584_k2", op="norm", T=16384, d=3584, k=2, shared=False, post=True, gate=True,
             drop=0.1, dtype="f16"),
        dict(name="norm_grad_T8191_d2048_k4", op="norm_grad", T=8191, d=2048, k=4, shared=True, post=True,
             gate=True, drop=0.1, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "quantize", "ffn", "norm", "norm_grad"])
    score = rng.choice(["softmax", "sigmoid"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log_int(rng, max(1, 4 // groups), 512 // groups)
        top_groups = rng.randint((groups + 1) // 2, groups)
        return dict(op=op, T=_log_int(rng, 1, 16384 * 256 // max(256, E)), E=E,
                    k=rng.randint(1, min(16, E // groups * top_groups)), score=score, groups=groups,
                    top_groups=top_groups, group_top=rng.choice([1, 2]), bias=rng.random() < 0.5,
                    mask=rng.random() < 0.5, renorm=rng.random() < 0.7)
    dtype = "f16" if rng.random() < 0.75 else "f32"
    if op == "route_grad":
        T, E = _log_int(rng, 1, 16384 if dtype == "f16" else 2048), _log_int(rng, 4, 256)
        d = 128 * _log_int(rng, 1, 16) if dtype == "f16" else 4 * _log_int(rng, 8, 256)
        while T * d * E > 16384 * 2048 * 128:
            T //= 2
        return dict(op=op, T=T, d=d, E=E, k=rng.randint(1, min(8, E)), score=score,
                    renorm=rng.random() < 0.7, mask=rng.random() < 0.5, dtype=dtype)
    if op == "quantize":
        K, N = (128 * _log_int(rng, 1, 64) for _ in range(2))
        return dict(op=op, E=_log_int(rng, 1, max(1, 16 * 2048 * 8192 // (K * N))), K=K, N=N)
    if op == "ffn":
        d, f = 128 * _log_int(rng, 1, 28), 128 * _log_int(rng, 1, 64)
        E = _log_int(rng, 1, 128)
        T, k = _log_int(rng, 1, 16384), rng.choice([1, 2, 4, 8])
        k = min(k, E)
        while T > 1 and T * k * d * f > 32768 * 3584 * 2048:
            T //= 2
        return dict(op=op, T=T, d=d, f=f, E=E, k=k, cf=rng.choice([0.0, 0.0, 1.25]), skew=rng.choice([0.0, 0.5]))
    d = 8 * _log_int(rng, 8, 448)
    T, k = _log_int(rng, 1, 16384 if dtype == "f16" else 8192), rng.choice([1, 2, 4, 8])
    while T * (k + 3) * d > 16384 * 5 * 3584:
        T //= 2
    shared = rng.random() < 0.5 or k == 1
    return dict(op=op, T=T, d=d, k=k, shared=shared, post=rng.random() < 0.7, gate=rng.random() < 0.5,
                drop=rng.choice([0.0, 0.1, 0.5]), dtype=dtype)


# ---------------------------------------------------------------- inputs
class _Make:
    """Inputs of one seed, drawn on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, shape, sigma, dtype=torch.float32):
        return torch.randn(shape, generator=self.g, device="cuda").mul_(sigma).to(dtype)

    def uniform(self, shape):
        return torch.rand(shape, generator=self.g, device="cuda")


def _plan(mk, T, E, k, cf, skew):
    """Slots of a routed batch, as moe_dispatch lays them out: k distinct experts a token, an expert's slots
    in token order and no more than its capacity (cf = 0: no limit)."""
    scores = mk.normal((T, E), 1.0) + mk.normal((E,), skew)
    idx = torch.topk(scores, k, dim=1).indices.flatten()
    order = torch.argsort(idx, stable=True)
    counts = torch.bincount(idx, minlength=E)
    C = math.ceil(cf * T / E) if cf else T
    start = torch.cumsum(counts, 0) - counts
    rank = torch.arange(T * k, device="cuda") - start[idx[order]]
    kept = torch.clamp(counts, max=C)
    slots = (order // k)[rank < C]
    S_max = min(T * k, E * C)
    perm = torch.zeros(S_max, dtype=torch.int32, device="cuda")
    perm[:slots.numel()] = slots.to(torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(kept, 0)
    return perm, offsets, [int(v) for v in kept.tolist()], S_max


def _weights8(mk, E, n_out, n_in):
    """Expert weights in 8 bits, each output's inputs side by side, and the scale of each 128 x 128 block."""
    q = torch.empty((E, n_out, n_in), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((E, n_out // 128, n_in // 128), device="cuda")
    for e in range(E):
        q[e], s[e] = _quantize_blocks(mk.normal((n_out, n_in), 0.02))
    return q, s


def prepare(case, seed):
    mk = _Make(seed)
    op = case["op"]
    st = dict(case=case)
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        # logits of a router whose experts differ in popularity; the bias works against it
        pull = mk.normal((E,), 0.5)
        st["mask"] = (mk.uniform((T,)) < 0.9) if case["mask"] else None
        st["topk_w"] = torch.zeros((T, k), device="cuda")
        if op == "route":
            st["logits"] = mk.normal((T, E), 1.0) + pull
            st["bias"] = (-0.1 * pull + mk.normal((E,), 0.01)) if case["bias"] else None
            st["topk_idx"] = torch.zeros((T, k), dtype=torch.int32, device="cuda")
        else:
            d, dt = case["d"], _DT[case["dtype"]]
            st["tokens"] = mk.normal((T, d), 1.0, dt)
            st["Wg"] = mk.normal((d, E), d ** -0.5)
            st["logits"] = st["tokens"].float() @ st["Wg"]
            st["topk_idx"] = torch.topk(st["logits"], k, dim=1).indices.to(torch.int32).contiguous()
            st["dtopk_w"] = mk.normal((T, k), 0.1)
            st["dtokens_in"] = mk.normal((T, d), 0.01, dt)
            st["dlogits"] = torch.zeros((T, E), device="cuda")
            st["dWg"] = torch.zeros((d, E), device="cuda")
            st["dtokens"] = torch.zeros((T, d), dtype=dt, device="cuda")
    elif op == "quantize":
        E, K, N = case["E"], case["K"], case["N"]
        st["W"] = mk.normal((E, K, N), 0.02, torch.float16)
        st["Wq"] = torch.zeros((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
        st["scales"] = torch.zeros((E, N // 128, K // 128), device="cuda")
    elif op == "ffn":
        T, d, f, E, k = (case[q] for q in ("T", "d", "f", "E", "k"))
        st["perm"], st["offsets"], st["lengths"], S_max = _plan(mk, T, E, k, case["cf"], case["skew"])
        st["tokens"] = mk.normal((T, d), 1.0, torch.float16)
        st["W1q"], st["W1s"] = _weights8(mk, E, f, d)
        st["W2q"], st["W2s"] = _weights8(mk, E, d, f)
        st["expert_out"] = torch.zeros((S_max, d), dtype=torch.float16, device="cuda")
    else:
        T, d, k, dt = case["T"], case["d"], case["k"], _DT[case["dtype"]]
        kept = mk.uniform((T, k)) >= case["drop"]
        S = int(kept.sum())
        # every kept assignment has a slot of its own, spread as experts spread tokens
        slot = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
        slot[kept.flatten()] = torch.argsort(mk.uniform((S,))).to(torch.int32)
        st["slot_of"] = slot.view(T, k)
        w = mk.uniform((T, k)) + 0.05
        st["topk_w"] = w / w.sum(1, keepdim=True)
        st["expert_out"] = mk.normal((T * k, d), 0.5, dt)
        st["shared"] = mk.normal((T, d), 0.5, dt) if case["shared"] else None
        st["residual"] = mk.normal((T, d), 1.0, dt)
        st["post_w"] = 1 + mk.normal((d,), 0.1) if case["post"] else None
        st["gate"] = 0.5 + mk.normal((d,), 0.1) if case["gate"] else None
        st["next_w"] = 1 + mk.normal((d,), 0.1)
        st["alpha"], st["eps"] = 0.7, 1e-6
        st["hidden"] = torch.zeros((T, d), dtype=dt, device="cuda")
        if op == "norm":
            st["normed"] = torch.zeros((T, d), dtype=dt, device="cuda")
        else:
            hidden, _, st["rstd_post"], st["rstd_next"] = _block_norm(st)
            st["hidden"] = hidden.to(dt)
            st["dhidden"] = mk.normal((T, d), 0.1, dt)
            st["dnormed"] = mk.normal((T, d), 0.1, dt)
            st["dresidual"] = torch.zeros((T, d), dtype=dt, device="cuda")
            st["dexpert_out"] = torch.zeros((T * k, d), dtype=dt, device="cuda")
            st["dtopk_w"] = torch.zeros((T, k), device="cuda")
            for name, given in (("dpost_w", "post_w"), ("dgate", "gate"), ("dnext_w", "next_w")):
                st[name] = torch.zeros(d, device="cuda") if st[given] is not None else None
            st["dshared"] = torch.zeros((T, d), dtype=dt, device="cuda") if case["shared"] else None
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    import sparse_expert_ffn_layer_gb300 as moe
    c = st["case"]
    if c["op"] == "route_grad":
        size = moe.moe_gate_backward_workspace_size(c["T"], c["d"], c["E"], st["tokens"].dtype)
    elif c["op"] == "ffn":
        size = moe.moe_expert_fp8_workspace_size(c["T"], c["d"], c["f"], c["E"], st["perm"].shape[0],
                                                 torch.float16)
    elif c["op"] == "norm_grad":
        size = moe.moe_block_norm_workspace_size(c["T"], c["d"], c["k"], st["hidden"].dtype)
    else:
        return
    st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- one pass
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import sparse_expert_ffn_layer_gb300 as moe
    c = st["case"]
    op = c["op"]
    if op in ("route", "route_grad"):
        score = moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX
    if op == "route":
        moe.moe_route(None, None, c["k"], st["topk_idx"], st["topk_w"], logits_in=st["logits"],
                      bias=st["bias"], token_mask=st["mask"], score=score, n_groups=c["groups"],
                      top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renorm"], scale=2.5)
        return st["topk_idx"], st["topk_w"]
    if op == "route_grad":
        moe.moe_route_backward(st["logits"], st["topk_idx"], st["dlogits"], dtopk_w=st["dtopk_w"],
                               token_mask=st["mask"], score=score, renormalize=c["renorm"], scale=2.5,
                               tokens=st["tokens"], Wg=st["Wg"], dWg=st["dWg"], dtokens=st["dtokens"],
                               dtokens_in=st["dtokens_in"], workspace=st["workspace"])
        return st["dlogits"], st["dWg"], st["dtokens"]
    if op == "quantize":
        moe.moe_fp8_quantize(st["W"], st["Wq"], st["scales"])
        return st["Wq"], st["scales"]
    if op == "ffn":
        moe.moe_expert_ffn_fp8(st["tokens"], st["perm"], st["offsets"], st["W1q"], st["W1s"], st["W2q"],
                               st["W2s"], st["perm"].shape[0], st["expert_out"], st["workspace"])
        return st["expert_out"]
    if op == "norm":
        moe.moe_block_norm(st["residual"], st["hidden"], expert_out=st["expert_out"], slot_of=st["slot_of"],
                           topk_w=st["topk_w"], shared=st["shared"], post_w=st["post_w"], gate=st["gate"],
                           alpha=st["alpha"], next_w=st["next_w"], normed_out=st["normed"], eps=st["eps"])
        return st["hidden"], st["normed"]
    moe.moe_block_norm_backward(st["dhidden"], dnormed=st["dnormed"], hidden=st["hidden"],
                                rstd_next=st["rstd_next"], next_w=st["next_w"], expert_out=st["expert_out"],
                                slot_of=st["slot_of"], topk_w=st["topk_w"], shared=st["shared"],
                                post_w=st["post_w"], rstd_post=st["rstd_post"], gate=st["gate"],
                                alpha=st["alpha"], dresidual=st["dresidual"], dexpert_out=st["dexpert_out"],
                                dtopk_w=st["dtopk_w"], dshared=st["dshared"], dpost_w=st["dpost_w"],
                                dgate=st["dgate"], dnext_w=st["dnext_w"], workspace=st["workspace"])
    return {q: st[q] for q in _grads(st)}


def _grads(st):
    names = ("dresidual", "dexpert_out", "dtopk_w", "dshared", "dpost_w", "dgate", "dnext_w")
    return [q for q in names if st[q] is not None]


def _scores(x, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.max(dim=1, keepdim=True).values)
    return e / e.sum(dim=1, keepdim=True)


def _power_of_two(amax):
    """The smallest power of two that brings amax to the largest 8-bit value or below (1 for zero)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 127)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))


def _quantize_blocks(w):
    """[out, in] -> 8-bit values and the scale of each 128 x 128 block."""
    n, k = w.shape
    b = w.view(n // 128, 128, k // 128, 128)
    s = _power_of_two(b.abs().amax(dim=(1, 3)))
    return (b / s[:, None, :, None]).to(torch.float8_e4m3fn).view(n, k), s


def _quantize_rows(x):
    """Rows brought to 8 bits by blocks of 128 columns: the values that these stand for."""
    b = x.view(x.shape[0], -1, 128)
    s = _power_of_two(b.abs().amax(dim=2, keepdim=True))
    return ((b / s).to(torch.float8_e4m3fn).float() * s).view(x.shape)


def _values(q, s):
    n, k = q.shape
    return (q.float().view(n // 128, 128, k // 128, 128) * s[:, None, :, None]).view(n, k)


def _gelu(x):
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _block_norm(st):
    """The block's end in 32 bits: hidden, normed and the two norms' factors."""
    T, d = st["residual"].shape
    k = st["slot_of"].shape[1]
    slot = st["slot_of"].flatten().long()
    w = st["topk_w"] * (st["slot_of"] >= 0)
    y = (st["expert_out"][slot.clamp(min=0)].view(T, k, d).float() * w[:, :, None]).sum(1)
    if st["shared"] is not None:
        y = y + st["shared"].float()
    rp = None
    z = y
    if st["post_w"] is not None:
        rp = 1 / torch.sqrt((y * y).mean(1) + st["eps"])
        z = y * rp[:, None] * st["post_w"]
    if st["gate"] is not None:
        z = z * st["gate"]
    h = st["residual"].float() + st["alpha"] * z
    rn = 1 / torch.sqrt((h * h).mean(1) + st["eps"])
    return h, h * rn[:, None] * st["next_w"], rp, rn


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "route":
        # the order of two scores next to each other needs 64 bits
        T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
        s = _scores(st["logits"].double(), c["score"])
        choice = s if st["bias"] is None else s + st["bias"].double()
        if G > 1:
            members = choice.view(T, G, E // G)
            value = torch.sort(members, dim=2, descending=True).values[:, :, :c["group_top"]].sum(2)
            best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
            off = torch.ones((T, G), dtype=torch.bool, device="cuda").scatter_(1, best, False)
            choice = members.masked_fill(off[:, :, None], -math.inf).view(T, E)
        idx = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
        w = s.gather(1, idx)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        w = w * 2.5
        if st["mask"] is not None:
            idx = torch.where(st["mask"][:, None], idx, torch.full_like(idx, -1))
            w = torch.where(st["mask"][:, None], w, torch.zeros_like(w))
        return idx.to(torch.int32), w.float()
    if op == "route_grad":
        s = _scores(st["logits"], c["score"])
        idx, dw = st["topk_idx"].long(), st["dtopk_w"] * 2.5
        if st["mask"] is not None:
            dw = dw * st["mask"][:, None]
        if c["renorm"]:
            chosen = s.gather(1, idx)
            total = chosen.sum(1, keepdim=True)
            dw = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
        ds = torch.zeros_like(s).scatter_(1, idx, dw)
        if c["score"] == "sigmoid":
            dl = ds * s * (1 - s)
        else:
            dl = s * (ds - (ds * s).sum(1, keepdim=True))
        x = st["tokens"].float()
        if st["mask"] is not None:
            x = x * st["mask"][:, None]
        return dl, x.t() @ dl, (st["dtokens_in"].float() + dl @ st["Wg"].t()).to(st["tokens"].dtype)
    if op == "quantize":
        E, K, N = c["E"], c["K"], c["N"]
        w = st["W"].transpose(1, 2).float().reshape(E * N, K)
        q, s = _quantize_blocks(w)
        return q.view(E, N, K), s.view(E, N // 128, K // 128)
    if op == "ffn":
        out = torch.zeros_like(st["expert_out"])
        x = _quantize_rows(st["tokens"].float())
        s0 = 0
        for e, n in enumerate(st["lengths"]):
            if n:
                rows = x[st["perm"][s0:s0 + n].long()]
                h = _quantize_rows(_gelu(rows @ _values(st["W1q"][e], st["W1s"][e]).t()))
                out[s0:s0 + n] = (h @ _values(st["W2q"][e], st["W2s"][e]).t()).to(out.dtype)
            s0 += n
        return out
    dt = st["residual"].dtype
    if op == "norm":
        h, n, _, _ = _block_norm(st)
        return h.to(dt), n.to(dt)
    T, d = st["residual"].shape
    k = c["k"]
    g = {}
    h, dn, rn = st["hidden"].float(), st["dnormed"].float(), st["rstd_next"][:, None]
    a = dn * st["next_w"]
    dh = st["dhidden"].float() + rn * (a - h * rn * rn * (h * a).mean(1, keepdim=True))
    g["dnext_w"] = (dn * h * rn).sum(0)
    g["dresidual"] = dh.to(dt)
    slot = st["slot_of"].flatten().long()
    kept = st["slot_of"] >= 0
    rows = st["expert_out"][slot.clamp(min=0)].view(T, k, d).float()
    y = (rows * (st["topk_w"] * kept)[:, :, None]).sum(1)
    if st["shared"] is not None:
        y = y + st["shared"].float()
    dz = st["alpha"] * dh
    if st["post_w"] is not None:
        rp = st["rstd_post"][:, None]
        z = y * rp * st["post_w"]
    else:
        z = y
    if st["gate"] is not None:
        g["dgate"] = (dz * z).sum(0)
        dz = dz * st["gate"]
    dy = dz
    if st["post_w"] is not None:
        g["dpost_w"] = (dz * y * rp).sum(0)
        b = dz * st["post_w"]
        dy = rp * (b - y * rp * rp * (y * b).mean(1, keepdim=True))
    if st["shared"] is not None:
        g["dshared"] = dy.to(dt)
    g["dtopk_w"] = (rows * dy[:, None, :]).sum(2) * kept
    # dropped assignments go to a spare last row
    de = torch.zeros((T * k + 1, d), dtype=dt, device="cuda")
    to = torch.where(kept.flatten(), slot, torch.full_like(slot, T * k))
    de[to] = (dy[:, None, :] * st["topk_w"][:, :, None]).view(T * k, d).to(dt)
    g["dexpert_out"] = de[:T * k]
    return {q: g[q] for q in _grads(st)}


# ---------------------------------------------------------------- definition in 64 bits
def _round8(v):
    """64-bit values to the nearest e4m3 value (ties to even; none is above the largest)."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _step_of(amax):
    """Power of two by counting up from the exact quotient's exponent."""
    e = torch.floor(torch.log2(amax.clamp(min=1e-300) / _FP8_MAX)) - 1
    for _ in range(3):
        e = torch.where(amax > _FP8_MAX * torch.exp2(e), e + 1, e)
    return torch.where(amax > 0, torch.exp2(e), torch.ones_like(amax))


def exact(case, seed):
    """The operators from their definitions in 64 bits; gradients by differentiating these."""
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
        x = st["logits"].double()
        s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
        left = s if st["bias"] is None else s + st["bias"].double()
        if G > 1:
            value = left.view(T, G, E // G).topk(min(case["group_top"], E // G), dim=2).values.sum(2)
            # a group is in when fewer than top_groups are before it
            at = torch.arange(G, device="cuda")
            ahead = (value[:, None, :] > value[:, :, None]) | (
                (value[:, None, :] == value[:, :, None]) & (at[None, None, :] < at[None, :, None]))
            inside = ahead.sum(2) < case["top_groups"]
            left = left.masked_fill(~inside.repeat_interleave(E // G, dim=1), -math.inf)
        left = left.clone()
        picks = []
        for _ in range(k):
            top = left.max(dim=1, keepdim=True).values
            pick = (left == top).to(torch.int8).argmax(dim=1, keepdim=True)
            picks.append(pick)
            left.scatter_(1, pick, -math.inf)
        idx = torch.cat(picks, 1)
        w = torch.gather(s, 1, idx)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        w = 2.5 * w
        if st["mask"] is not None:
            idx, w = idx.clone(), w.clone()
            idx[~st["mask"]] = -1
            w[~st["mask"]] = 0
        return idx.to(torch.int32), w
    if op == "route_grad":
        x = st["tokens"].double().requires_grad_()
        Wg = st["Wg"].double().requires_grad_()
        # the logits are an input of their own (the forward pass rounded them to 32 bits)
        logits = st["logits"].double().requires_grad_()
        s = torch.sigmoid(logits) if case["score"] == "sigmoid" else torch.softmax(logits, 1)
        w = s.gather(1, st["topk_idx"].long())
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        on = torch.ones(case["T"], device="cuda") if st["mask"] is None else st["mask"]
        (dl,) = torch.autograd.grad((2.5 * w * st["dtopk_w"].double() * on.double()[:, None]).sum(), logits)
        dx, dWg = torch.autograd.grad(((x @ Wg) * dl).sum(), (x, Wg))
        return dl, dWg, st["dtokens_in"].double() + dx
    if op == "quantize":
        E, K, N = case["E"], case["K"], case["N"]
        q = torch.empty((E, N, K), dtype=torch.float64, device="cuda")
        s = torch.empty((E, N // 128, K // 128), dtype=torch.float64, device="cuda")
        for e in range(E):
            w = st["W"][e].double()
            s[e] = _step_of(w.abs().view(K // 128, 128, N // 128, 128).amax(dim=(1, 3))).t()
            q[e] = _round8(w.t() / s[e].repeat_interleave(128, 0).repeat_interleave(128, 1))
        return q, s
    if op == "ffn":
        def rows8(v):
            s = _step_of(v.abs().unflatten(1, (-1, 128)).amax(dim=2)).repeat_interleave(128, 1)
            return _round8(v / s) * s

        def weight(q, s):
            return q.double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)

        if 4 * case["T"] * case["k"] * case["d"] * case["f"] > 1e13:
            return None                                   # over 20 seconds
        out = torch.zeros(st["expert_out"].shape, dtype=torch.float64, device="cuda")
        off = st["offsets"].tolist()
        for e in range(case["E"]):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            x = rows8(st["tokens"][st["perm"][a:b].long()].double())
            u = torch.einsum("sk,nk->sn", x, weight(st["W1q"][e], st["W1s"][e]))
            h = rows8(torch.nn.functional.gelu(u, approximate="tanh"))
            out[a:b] = torch.einsum("sk,nk->sn", h, weight(st["W2q"][e], st["W2s"][e]))
        return out
    leaf = {q: st[q].double().requires_grad_() for q in ("residual", "expert_out", "topk_w", "shared", "post_w",
                                                         "gate", "next_w") if st[q] is not None}
    T, d = st["residual"].shape
    y = torch.zeros((T, d), dtype=torch.float64, device="cuda")
    for j in range(case["k"]):
        on = (st["slot_of"][:, j] >= 0).nonzero()[:, 0]
        y = y.index_add(0, on, leaf["topk_w"][on, j, None] * leaf["expert_out"][st["slot_of"][on, j].long()])
    if "shared" in leaf:
        y = y + leaf["shared"]
    z = y
    if "post_w" in leaf:
        r = torch.rsqrt(y.square().mean(1, keepdim=True) + st["eps"])
        if op == "norm_grad":
            # differentiated at the factor that the forward pass gave (rounded to 32 bits)
            r = r * (st["rstd_post"].double()[:, None] / r.detach())
        z = y * r * leaf["post_w"]
    if "gate" in leaf:
        z = z * leaf["gate"]
    h = leaf["residual"] + st["alpha"] * z
    if op == "norm":
        n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + st["eps"]) * leaf["next_w"]
        return h.detach(), n.detach()
    # the stored hidden rows are an input of their own (rounded to their type), as is their norm's factor
    hin = st["hidden"].double().requires_grad_()
    rn = st["rstd_next"].double()[:, None]
    dn = st["dnormed"].double()
    a = dn * leaf["next_w"].detach()
    dh = st["dhidden"].double() + rn * a - hin.detach() * rn ** 3 * (hin.detach() * a).mean(1, keepdim=True)
    names = [q for q in ("expert_out", "topk_w", "shared", "post_w", "gate") if q in leaf]
    got = dict(zip(names, torch.autograd.grad((h * dh).sum(), [leaf[q] for q in names])))
    got["residual"] = dh
    got["next_w"] = (dn * hin.detach() * rn).sum(0)
    return {"d" + q: got[q] for q in (n[1:] for n in _grads(st))}


# ---------------------------------------------------------------- unavoidable work
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0) + (T if case["mask"] else 0),
                "flops": 8 * T * E}
    if op == "quantize":
        n = case["E"] * case["K"] * case["N"]
        return {"bytes": 3 * n + 4 * n // 16384, "flops": 3 * n}
    if op == "ffn":
        T, d, f, E, k = (case[q] for q in ("T", "d", "f", "E", "k"))
        S = min(T * k, E * math.ceil(case["cf"] * T / E)) if case["cf"] else T * k
        hit = max(1, round(E * (1 - (1 - k / E) ** T)))      # experts that a token reaches
        return {"bytes": hit * 2 * d * f * (1 + 4 / 16384) + T * d * 2 + S * d * 2 + 4 * (S + E),
                "flops": 4 * S * d * f}
    e = 2 if case["dtype"] == "f16" else 4
    if op == "route_grad":
        T, d, E, k = case["T"], case["d"], case["E"], case["k"]
        return {"bytes": 3 * T * d * e + 8 * T * E + 8 * T * k + 8 * d * E + (T if case["mask"] else 0),
                "flops": 4 * T * d * E + 10 * T * E}
    T, d, k = case["T"], case["d"], case["k"]
    S = int(T * k * (1 - case["drop"]))
    weights = 4 * d * (1 + case["post"] + case["gate"])
    sh = T * d * e if case["shared"] else 0
    if op == "norm":
        return {"bytes": (S + 3 * T) * d * e + sh + 8 * T * k + weights, "flops": 2 * S * d + 10 * T * d}
    return {"bytes": (2 * S + 4 * T) * d * e + 2 * sh + 12 * T * k + 8 * T + 2 * weights,
            "flops": 6 * S * d + 24 * T * d}
