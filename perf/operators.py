"""The training and adapter operators of the MoE layer as measured work: cases, plain forms and calls.

Five operators: the router's losses (`balance`: moe_balance_loss, then their gradient by
moe_gate_topk_backward), the gate's whole gradient (`gate`: moe_gate_topk_backward down to Wg and the
tokens), the combine's gradient (`combine`: moe_combine_backward), and the low-rank adapters of many
requests (`adapter`: moe_adapter_forward, `adapter_grad`: moe_adapter_backward).  With `own` false,
`run` computes them from elementary torch operations in 32 bits; with `own` true it makes the
library's calls.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # router losses: a decode-sized batch of a small layer (latency), a ragged batch with
        # padding tokens, and the accumulated batch of one optimizer step of a 128-expert layer
        dict(name="balance_T64_E8", op="balance", T=64, E=8, k=1, mask=False),
        dict(name="balance_T4099_E60_k2_padded", op="balance", T=4099, E=60, k=2, mask=True),
        dict(name="balance_T262144_E128_k2", op="balance", T=262144, E=128, k=2, mask=False),
        # gate gradient: the 350M+MoE-128 layer at its prefill size and the 2.4B+MoE-128 top-2 layer
        dict(name="gate_T4096_d1024_E128", op="gate", T=4096, d=1024, E=128, k=1, dtype="f16"),
        dict(name="gate_T16384_d3584_E128_k2", op="gate", T=16384, d=3584, E=128, k=2, dtype="f16"),
        # combine gradient: a ragged batch in 32 bits, and the 2.4B top-2 layer with capacity drops
        dict(name="combine_T1001_d1024_f32", op="combine", T=1001, d=1024, k=2, drop=0.1, dtype="f32"),
        dict(name="combine_T16384_d3584_k2", op="combine", T=16384, d=3584, k=2, drop=0.1, dtype="f16"),
        # adapters while serving: one token; 64 requests with an adapter each at the 2.4B width;
        # a prefill of eight tenants (Zipf lengths) at the same width
        dict(name="adapter_T1_d1024_r16", op="adapter", T=1, d_in=1024, d_out=1024, r=16, N=32,
             base_model=0.0, skew=0.0, dtype="f16"),
        dict(name="adapter_T64_d3584_r16_N64", op="adapter", T=64, d_in=3584, d_out=3584, r=16, N=64,
             base_model=0.1, skew=0.0, dtype="f16"),
        dict(name="adapter_T16384_d3584_r64_N8", op="adapter", T=16384, d_in=3584, d_out=3584, r=64,
             N=8, base_model=0.0, skew=1.1, dtype="f16"),
        # adapters in training: a small 32-bit layer, and adapters on the PR-MoE layer's first dense
        # projection (2048 -> 8192)
        dict(name="adapter_grad_T500_d64_r8_f32", op="adapter_grad", T=500, d_in=64, d_out=256, r=8,
             N=4, base_model=0.1, skew=0.0, dtype="f32"),
        dict(name="adapter_grad_T8192_d2048_f8192_r32", op="adapter_grad", T=8192, d_in=2048,
             d_out=8192, r=32, N=16, base_model=0.0, skew=1.1, dtype="f16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "gate", "combine", "adapter", "adapter_grad"])
    if op == "balance":
        E = _log_int(rng, 2, 1024)
        return dict(op=op, T=_log_int(rng, 1, min(262144, (262144 * 128) // E)), E=E,
                    k=rng.choice([1, 2]), mask=rng.random() < 0.5)
    dtype = "f16" if rng.random() < 0.75 else "f32"
    if op == "gate":
        T, E = _log_int(rng, 1, 16384 if dtype == "f16" else 2048), _log_int(rng, 4, 256)
        d = 128 * _log_int(rng, 1, 28) if dtype == "f16" else 4 * _log_int(rng, 8, 256)
        while T * d * E > 16384 * 3584 * 128:
            T //= 2
        return dict(op=op, T=T, d=d, E=E, k=rng.choice([1, 2]), dtype=dtype)
    if op == "combine":
        return dict(op=op, T=_log_int(rng, 1, 16384 if dtype == "f16" else 8192),
                    d=8 * _log_int(rng, 8, 448), k=rng.choice([1, 2]),
                    drop=rng.choice([0.0, 0.1, 0.5]), dtype=dtype)
    big = dtype == "f16"
    T = _log_int(rng, 1, 16384 if big else 2048)
    d_in, d_out = (8 * _log_int(rng, 8, 1024 if big else 128) for _ in range(2))
    r = 8 * rng.randint(1, 16 if big else 4)
    N = _log_int(rng, 1, 64)
    while T * (d_in + d_out) > 8192 * (2048 + 8192) or T * r * (d_in + d_out) > 16384 * 64 * 7168:
        T //= 2
    return dict(op=op, T=T, d_in=d_in, d_out=d_out, r=r, N=N, base_model=rng.choice([0.0, 0.1, 0.9]),
                skew=rng.choice([0.0, 1.1]), dtype=dtype)


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


def _router_inputs(mk, T, E, k):
    # logits of a router whose experts differ in popularity
    logits = mk.normal((T, E), 1.0) + mk.normal((E,), 0.5)
    topk_idx = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    return logits, topk_idx


def _spread(mk, T, N, base_model, skew):
    """Adapter of each token (-1: none), and its slot-ordered plan: what moe_dispatch returns for
    these ids with k = 1 and no capacity limit."""
    w = torch.arange(1, N + 1, dtype=torch.float32, device="cuda").pow(-skew)
    cdf = torch.cumsum(w / w.sum(), 0)
    ids = torch.searchsorted(cdf, mk.uniform((T,))).clamp_(max=N - 1)
    ids = torch.where(mk.uniform((T,)) < base_model, torch.full_like(ids, -1), ids)
    order = torch.argsort(ids, stable=True)
    lengths = torch.bincount(ids + 1, minlength=N + 1)
    perm = order[int(lengths[0]):].to(torch.int32)
    offsets = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(lengths[1:], 0)
    pad = torch.zeros(T - perm.numel(), dtype=torch.int32, device="cuda")
    return torch.cat([perm, pad]), offsets, [int(v) for v in lengths[1:].tolist()]


def prepare(case, seed):
    mk = _Make(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "balance":
        T, E, k = case["T"], case["E"], min(case["k"], case["E"])
        st["logits"], st["topk_idx"] = _router_inputs(mk, T, E, k)
        st["mask"] = (mk.uniform((T,)) < 0.9) if case["mask"] else None
        # loss coefficients (balance 0.01, z 0.001) times the upstream gradient
        st["dlosses"] = torch.tensor([0.01, 0.001], device="cuda") * (1 + mk.uniform((1,)))
        st["dlogits"] = torch.zeros((T, E), device="cuda")
    elif op == "gate":
        T, d, E, k = case["T"], case["d"], case["E"], min(case["k"], case["E"])
        dt = _DT[case["dtype"]]
        st["tokens"] = mk.normal((T, d), 1.0, dt)
        st["Wg"] = mk.normal((d, E), 0.02)
        st["logits"] = st["tokens"].float() @ st["Wg"]
        st["topk_idx"] = torch.topk(st["logits"], k, dim=1).indices.to(torch.int32).contiguous()
        st["dtopk_w"] = mk.normal((T, k), 0.1)
        st["counts"] = torch.bincount(st["topk_idx"].flatten(), minlength=E).to(torch.int32)
        st["n_valid"] = torch.tensor([T], dtype=torch.int32, device="cuda")
        st["dlosses"] = torch.tensor([0.01, 0.001], device="cuda") * (1 + mk.uniform((1,))) * T
        st["dtokens_in"] = mk.normal((T, d), 0.01, dt)
        st["dlogits"] = torch.zeros((T, E), device="cuda")
        st["dWg"] = torch.zeros((d, E), device="cuda")
        st["dtokens"] = torch.zeros((T, d), dtype=dt, device="cuda")
    elif op == "combine":
        T, d, k, dt = case["T"], case["d"], case["k"], _DT[case["dtype"]]
        kept = mk.uniform((T, k)) >= case["drop"]
        S = int(kept.sum())
        # every kept assignment has a slot of its own, spread as experts spread tokens
        slot = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
        slot[kept.flatten()] = torch.argsort(mk.uniform((S,))).to(torch.int32)
        st["slot_of"] = slot.view(T, k)
        w = mk.uniform((T, k)) + 0.05
        st["topk_w"] = w / w.sum(1, keepdim=True) if k == 2 else w
        st["dout"] = mk.normal((T, d), 0.1, dt)
        st["expert_out"] = mk.normal((T * k, d), 1.0, dt)
        st["dexpert_out"] = torch.zeros((T * k, d), dtype=dt, device="cuda")
        st["dtopk_w"] = torch.zeros((T, k), device="cuda")
    else:
        T, d_in, d_out, r, N = (case[q] for q in ("T", "d_in", "d_out", "r", "N"))
        dt = _DT[case["dtype"]]
        st["perm"], st["offsets"], st["lengths"] = _spread(mk, T, N, case["base_model"], case["skew"])
        st["tokens"] = mk.normal((T, d_in), 1.0, dt)
        st["A"] = mk.normal((N, d_in, r), d_in ** -0.5, dt)
        st["B"] = mk.normal((N, r, d_out), 0.02, dt)
        st["scale"] = 0.5 + mk.uniform((N,))
        if op == "adapter":
            st["base"] = mk.normal((T, d_out), 1.0, dt)
            st["out"] = torch.zeros((T, d_out), dtype=dt, device="cuda")
        else:
            st["dout"] = mk.normal((T, d_out), 0.1, dt)
            hidden = torch.zeros((T, r), device="cuda")
            for n, s0, s1 in _segments(st["lengths"]):
                rows = st["tokens"][st["perm"][s0:s1].long()].float()
                hidden[s0:s1] = rows @ st["A"][n].float()
            st["hidden"] = hidden
            st["dtokens_in"] = mk.normal((T, d_in), 0.01, dt)
            st["dtokens"] = torch.zeros((T, d_in), dtype=dt, device="cuda")
            st["dA"] = torch.zeros((N, d_in, r), device="cuda")
            st["dB"] = torch.zeros((N, r, d_out), device="cuda")
    if own:
        _prepare_own(st)
    return st


def _segments(lengths):
    s = 0
    for n, length in enumerate(lengths):
        if length:
            yield n, s, s + length
        s += length


def _prepare_own(st):
    import sparse_expert_ffn_layer_gb300 as moe
    c = st["case"]
    op = c["op"]
    if op == "balance":
        E = c["E"]
        st["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        st["prob_mean"] = torch.empty(E, device="cuda")
        st["losses"] = torch.empty(2, device="cuda")
        st["n_valid"] = torch.empty(1, dtype=torch.int32, device="cuda")
        size = moe.moe_balance_workspace_size(c["T"], E)
    elif op == "gate":
        size = moe.moe_gate_backward_workspace_size(c["T"], c["d"], c["E"], st["tokens"].dtype)
    elif op == "combine":
        return
    else:
        size = moe.moe_adapter_workspace_size(c["T"], c["d_in"], c["d_out"], c["r"], c["N"], c["T"],
                                              st["tokens"].dtype)
    st["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- one pass
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    import sparse_expert_ffn_layer_gb300 as moe
    op = st["case"]["op"]
    if op == "balance":
        moe.moe_balance_loss(st["logits"], st["topk_idx"], st["counts"], st["prob_mean"], st["losses"],
                             st["n_valid"], st["workspace"], token_mask=st["mask"])
        moe.moe_gate_topk_backward(st["logits"], st["topk_idx"], st["dlogits"], dlosses=st["dlosses"],
                                   counts=st["counts"], n_valid=st["n_valid"], token_mask=st["mask"])
        return st["losses"], st["counts"], st["prob_mean"], st["dlogits"]
    if op == "gate":
        moe.moe_gate_topk_backward(st["logits"], st["topk_idx"], st["dlogits"], dtopk_w=st["dtopk_w"],
                                   dlosses=st["dlosses"], counts=st["counts"], n_valid=st["n_valid"],
                                   tokens=st["tokens"], Wg=st["Wg"], dWg=st["dWg"],
                                   dtokens=st["dtokens"], dtokens_in=st["dtokens_in"],
                                   workspace=st["workspace"])
        return st["dlogits"], st["dWg"], st["dtokens"]
    if op == "combine":
        moe.moe_combine_backward(st["dout"], st["expert_out"], st["slot_of"], st["topk_w"],
                                 st["dexpert_out"], st["dtopk_w"])
        return st["dexpert_out"], st["dtopk_w"]
    if op == "adapter":
        moe.moe_adapter_forward(st["tokens"], st["perm"], st["offsets"], st["A"], st["B"], st["scale"],
                                st["out"], st["workspace"], base=st["base"])
        return st["out"]
    moe.moe_adapter_backward(st["dout"], st["tokens"], st["hidden"], st["perm"], st["offsets"],
                             st["A"], st["B"], st["scale"], st["workspace"], dtokens=st["dtokens"],
                             dtokens_in=st["dtokens_in"], dA=st["dA"], dB=st["dB"])
    return st["dtokens"], st["dA"], st["dB"]


def _softmax(logits):
    m = logits.max(dim=1, keepdim=True).values
    e = torch.exp(logits - m)
    s = e.sum(dim=1, keepdim=True)
    return e / s, m + torch.log(s)


def _plain_dlogits(logits, topk_idx, p, lse, n, counts, dlosses, mask, dtopk_w):
    T, E = logits.shape
    k = topk_idx.shape[1]
    a = dlosses[0] * E * counts.float() / (n * n * k)
    dl = p * (a - (p * a).sum(1, keepdim=True)) + p * (2 * dlosses[1] / n * lse)
    if mask is not None:
        dl = dl * mask.float()[:, None]
    if dtopk_w is not None:
        idx = topk_idx.long()
        if k == 1:
            q = p.gather(1, idx) * dtopk_w
            dl = dl - p * q
            dl = dl.scatter_add(1, idx, q)
        else:
            pk = p.gather(1, idx)
            w = pk / pk.sum(1, keepdim=True)
            q = w * (dtopk_w - (w * dtopk_w).sum(1, keepdim=True))
            dl = dl.scatter_add(1, idx, q)
    return dl


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op == "balance":
        logits, idx, mask = st["logits"], st["topk_idx"], st["mask"]
        T, E = logits.shape
        k = idx.shape[1]
        p, lse = _softmax(logits)
        if mask is None:
            n = torch.full((), float(T), device="cuda")
            cnt = torch.zeros(E, dtype=torch.int32, device="cuda")
            cnt.scatter_add_(0, idx.flatten().long(), torch.ones_like(idx).flatten())
            P, z = p.sum(0), (lse * lse).sum()
        else:
            on = mask.float()[:, None]
            n = on.sum()
            cnt = torch.zeros(E, dtype=torch.int32, device="cuda")
            cnt.scatter_add_(0, idx.flatten().long(),
                             mask.to(torch.int32)[:, None].expand(T, k).reshape(-1))
            P, z = (p * on).sum(0), (lse * lse * on).sum()
        n1 = n.clamp(min=1)
        P = P / n1
        losses = torch.stack([E * (cnt.float() / (n1 * k) * P).sum(), z / n1])
        dl = _plain_dlogits(logits, idx, p, lse, n1, cnt, st["dlosses"], mask, None)
        return losses, cnt, P, dl
    if op == "gate":
        p, lse = _softmax(st["logits"])
        dl = _plain_dlogits(st["logits"], st["topk_idx"], p, lse, st["n_valid"].float(), st["counts"],
                            st["dlosses"], None, st["dtopk_w"])
        dWg = st["tokens"].float().t() @ dl
        dx = st["dtokens_in"].float() + dl @ st["Wg"].t()
        return dl, dWg, dx.to(st["tokens"].dtype)
    if op == "combine":
        T, d = st["dout"].shape
        k = st["slot_of"].shape[1]
        dt = st["dout"].dtype
        slot = st["slot_of"].flatten().long()
        kept = slot >= 0
        rows = st["expert_out"][slot.clamp(min=0)].float().view(T, k, d)
        dout = st["dout"].float()
        dw = (rows * dout[:, None, :]).sum(2) * kept.view(T, k).float()
        # dropped assignments go to a spare last row
        dy = torch.zeros((T * k + 1, d), dtype=dt, device="cuda")
        to = torch.where(kept, slot, torch.full_like(slot, T * k))
        dy[to] = (dout[:, None, :] * st["topk_w"][:, :, None]).view(T * k, d).to(dt)
        return dy[:T * k], dw
    lengths = st["lengths"]
    S = sum(lengths)
    perm = st["perm"][:S].long()
    if op == "adapter":
        dt = st["base"].dtype
        out = torch.zeros_like(st["out"])
        if S <= 256:                       # few tokens: a batched product over gathered adapters
            s = torch.arange(S, device="cuda")
            a = torch.searchsorted(st["offsets"].long(), s, right=True) - 1
            x = st["tokens"][perm].float()
            h = torch.bmm(x[:, None, :], st["A"][a].float())
            y = torch.bmm(h, st["B"][a].float())[:, 0] * st["scale"][a][:, None]
            out[perm] = (st["base"][perm].float() + y).to(dt)
            return out
        for n, s0, s1 in _segments(lengths):
            t = perm[s0:s1]
            h = st["tokens"][t].float() @ st["A"][n].float()
            y = (h @ st["B"][n].float()) * st["scale"][n]
            out[t] = (st["base"][t].float() + y).to(dt)
        return out
    dtokens = torch.zeros_like(st["dtokens"])
    dA, dB = torch.zeros_like(st["dA"]), torch.zeros_like(st["dB"])
    for n, s0, s1 in _segments(lengths):
        t = perm[s0:s1]
        dy = st["dout"][t].float() * st["scale"][n]
        dh = dy @ st["B"][n].float().t()
        dtokens[t] = (st["dtokens_in"][t].float() + dh @ st["A"][n].float().t()).to(dtokens.dtype)
        dA[n] = st["tokens"][t].float().t() @ dh
        dB[n] = st["hidden"][s0:s1].t() @ dy
    return dtokens, dA, dB


# ---------------------------------------------------------------- definition in 64 bits
def exact(case, seed):
    """The operators by differentiating their definitions in 64 bits."""
    st = prepare(case, seed)
    op = case["op"]
    if op in ("balance", "gate"):
        x = st["logits"].double().requires_grad_()
        idx = st["topk_idx"].long()
        T, E = x.shape
        k = idx.shape[1]
        on = torch.ones(T, dtype=torch.float64, device="cuda")
        if st.get("mask") is not None:
            on = st["mask"].double()
        n = on.sum().clamp(min=1)
        logp = torch.log_softmax(x, 1)
        P = (logp.exp() * on[:, None]).sum(0) / n
        hot = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, idx, 1.0)
        counts = (hot * on[:, None]).sum(0)
        losses = torch.stack([E * (counts / (n * k) * P).sum(),
                              (torch.logsumexp(x, 1).square() * on).sum() / n])
        total = (losses * st["dlosses"].double()).sum()
        if op == "gate":
            sel = logp.gather(1, idx)
            w = sel.exp() if k == 1 else torch.softmax(sel, 1)
            total = total + (w * st["dtopk_w"].double()).sum()
        (dl,) = torch.autograd.grad(total, x)
        if op == "balance":
            return (losses.detach(), counts.to(torch.int32), P.detach(), dl)
        dWg = st["tokens"].double().t() @ dl
        return (dl, dWg, st["dtokens_in"].double() + dl @ st["Wg"].double().t())
    if op == "combine":
        k = case["k"]
        T, d = st["dout"].shape
        dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        dy = torch.zeros(st["dexpert_out"].shape, dtype=torch.float64, device="cuda")
        dout = st["dout"].double()
        for j in range(k):
            on = (st["slot_of"][:, j] >= 0).nonzero()[:, 0]
            s = st["slot_of"][on, j].long()
            dw[on, j] = torch.einsum("td,td->t", dout[on], st["expert_out"][s].double())
            dy[s] = st["topk_w"][on, j].double()[:, None] * dout[on]
        return dy, dw
    perm, off = st["perm"].long().cpu(), st["offsets"].cpu().tolist()
    if op == "adapter":
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        for n in range(case["N"]):
            t = perm[off[n]:off[n + 1]].cuda()
            if t.numel():
                delta = torch.linalg.multi_dot([st["tokens"][t].double(), st["A"][n].double(),
                                                st["B"][n].double()])
                out[t] = st["base"][t].double() + st["scale"][n].double() * delta
        return out
    dx = torch.zeros(st["dtokens"].shape, dtype=torch.float64, device="cuda")
    dA = torch.zeros(st["dA"].shape, dtype=torch.float64, device="cuda")
    dB = torch.zeros(st["dB"].shape, dtype=torch.float64, device="cuda")
    for n in range(case["N"]):
        s0, s1 = off[n], off[n + 1]
        t = perm[s0:s1].cuda()
        if not t.numel():
            continue
        x = st["tokens"][t].double().requires_grad_()
        A = st["A"][n].double().requires_grad_()
        B = st["B"][n].double().requires_grad_()
        dy = st["dout"][t].double()
        sc = st["scale"][n].double()
        h = x @ A
        # the hidden rows are an input of their own (the forward pass rounded them to 32 bits)
        gh, gx, gA = torch.autograd.grad(((h @ B.detach()) * sc * dy).sum(), (h, x, A))
        (gB,) = torch.autograd.grad(((st["hidden"][s0:s1].double() @ B) * sc * dy).sum(), B)
        dx[t] = st["dtokens_in"][t].double() + gx
        dA[n], dB[n] = gA, gB
    return dx, dA, dB


# ---------------------------------------------------------------- unavoidable work
def work(case):
    op = case["op"]
    if op == "balance":
        T, E, k = case["T"], case["E"], min(case["k"], case["E"])
        # logits and top-k indices in, logits' gradient out
        by = 8 * T * E + 4 * T * k + 8 * E + 8 + (T if case["mask"] else 0)
        return {"bytes": by, "flops": 14 * T * E}
    e = 2 if case["dtype"] == "f16" else 4
    if op == "gate":
        T, d, E, k = case["T"], case["d"], case["E"], min(case["k"], case["E"])
        by = 3 * T * d * e + 8 * T * E + 8 * T * k + 8 * d * E + 4 * E
        return {"bytes": by, "flops": 4 * T * d * E + 10 * T * E}
    if op == "combine":
        T, d, k = case["T"], case["d"], case["k"]
        S = int(T * k * (1 - case["drop"]))
        return {"bytes": T * d * e + 2 * S * d * e + 12 * T * k, "flops": 3 * S * d}
    T, d_in, d_out, r, N = (case[q] for q in ("T", "d_in", "d_out", "r", "N"))
    S = max(1, int(T * (1 - case["base_model"])))
    used = min(N, S)
    weights = used * r * (d_in + d_out) * e
    if op == "adapter":
        return {"bytes": S * (d_in + 2 * d_out) * e + weights + 4 * (S + N),
                "flops": 2 * S * r * (d_in + d_out)}
    return {"bytes": S * (3 * d_in + d_out) * e + 4 * S * r + weights + 4 * N * r * (d_in + d_out),
            "flops": 4 * S * r * (d_in + d_out)}
