"""Experts in 8 bits where the right answer is known exactly, or to a few units: values, scales and sums of long runs.

u = 2^-24 is half a step of float32.  Inputs are small integers times powers of two, so that 8-bit values, scales and
sums (below 2^24 of their unit, in any order and however additions are cut off) are exact; then outputs are the
exact ones, rounded once to float16.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F16 = torch.float16


@pytest.fixture(scope="module")
def m():
    import sparse_expert_ffn_layer_gb300 as mod
    return mod


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(g, lo, hi, *shape):
    """Whole numbers from lo to hi, both among them."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").double()


def spread(b, n, k):
    return b.repeat_interleave(n, -2).repeat_interleave(k, -1)


def to8(m, W):
    """[E, n_out, n_in] in 64 bits to 8 bits by the library; the values have to survive that."""
    E, n, k = W.shape
    q = torch.empty((E, n, k), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((E, n // 128, k // 128), device="cuda")
    m.moe_fp8_quantize(W.transpose(1, 2).float().contiguous(), q, s)
    for e in range(E):
        assert torch.equal(q[e].double() * spread(s[e].double(), 128, 128), W[e])
    return q, s


def run(m, x, rows, W1, W2, other=False, status=None):
    """moe_expert_ffn_fp8 over slots in order; other: one more expert without slots, whose scales are no powers of two,
    which brings all products to the form for any scales.  Also the launches that the call took."""
    (q1, s1), (q2, s2) = W1, W2
    T, d = x.shape
    off = [0]
    for n in rows:
        off.append(off[-1] + n)
    if other:
        more = lambda t, v: torch.cat([t, torch.full((1,) + t.shape[1:], v, dtype=t.dtype, device="cuda")])
        q1, q2 = (more(q.view(torch.uint8), 0) for q in (q1, q2))
        s1, s2, off = more(s1, 3.0), more(s2, 3.0), off + off[-1:]
    E, f, S = q1.shape[0], q1.shape[1], off[-1]
    out = torch.full((S, d), float("nan"), dtype=F16, device="cuda")
    ws = torch.full((m.moe_expert_fp8_workspace_size(T, d, f, E, S, F16),), 0xA5, dtype=torch.uint8, device="cuda")
    n0 = m.get_lib().moe_kernel_launches()
    m.moe_expert_ffn_fp8(x, torch.arange(T, device="cuda").to(torch.int32), torch.tensor(off, dtype=torch.int32, device="cuda"),
                         q1, s1, q2, s2, S, out, ws)
    launches = m.get_lib().moe_kernel_launches() - n0
    assert m.moe_status_read(ws) == m.MOE_OK
    return out, launches


# Rows to 8 bits and two products; where products are long enough, each in two forms of which one returns at once.
ONE_FORM, TWO_FORMS = 3, 5
LONG = [([3000, 700], 256, 9216), ([160, 161, 3], 4352, 6400), ([2999, 701, 0], 9216, 256), ([1000, 8, 9, 16, 17, 120], 2304, 3328),
        ([241, 0, 480, 65], 1280, 8448), ([700], 2560, 14336)]
SHORT = [([90], 256, 512), ([160, 161, 3], 768, 256), ([65] * 9, 1280, 1024), ([33, 0, 2], 384, 1152)]


def first_half(g, T, d):
    """Rows whose second half is the first but for a few entries: what a sum of both halves leaves is small."""
    x = 4 * ints(g, 4, 7, T, d // 2)                  # 16, 20, 24 or 28: GeLU leaves them as they are
    step = 4 * ints(g, -1, 1, T, d // 2) * (torch.rand((T, d // 2), generator=g, device="cuda") < 1 / 64)
    return torch.cat([x, (x + step).clamp(16, 28)], 1)


@pytest.mark.parametrize("rows,d,f", LONG + SHORT, ids=str)
@pytest.mark.parametrize("other", [False, True])
def test_second_product_is_exact(m, rows, d, f, other):
    """Each hidden value is one of the inputs; the two halves of a sum of f inputs nearly cancel.  GeLU(x) for x >= 16 is
    x / (1 + e) with e below 2^-300; its reciprocal is off by 1 ulp at most, which the rounding to 8 bits takes away."""
    g = gen(d + f)
    E, T = len(rows), sum(rows)
    x = first_half(g, T, d)
    j = torch.arange(f // 2, device="cuda")
    W1 = torch.zeros((E, f, d), dtype=torch.float64, device="cuda")
    pick = torch.cat([j % (d // 2), d // 2 + j % (d // 2)])
    W1[:, torch.arange(f, device="cuda"), pick] = 1.0
    # whole numbers 1 to 3 times a power of two for each block; a half of f is whole blocks where f is a multiple of 256,
    # else (a block in the middle) all have one scale
    b = ints(g, 0, 3, E, d // 128, max(1, f // 256)) if f % 256 == 0 else ints(g, 0, 0, E, d // 128, 1)
    w = ints(g, 1, 3, E, d, f // 2) * torch.exp2(spread(b, 128, 128 if f % 256 == 0 else f // 2) - 6)
    W2 = torch.cat([w, -w], 2)
    out, launches = run(m, x.half(), rows, to8(m, W1), to8(m, W2), other)
    assert launches == (TWO_FORMS if (rows, d, f) in LONG else ONE_FORM)
    at = 0
    for e, n in enumerate(rows):
        h = x[at:at + n][:, pick]
        want = h @ W2[e].t()                          # |sum of the magnitudes| < 2^24 of its unit: exact
        assert torch.equal(out[at:at + n], want.half()), f"expert {e}"
        if n:                                         # (and a block that is left out would be seen)
            assert not torch.equal(out[at:at + n], (h[:, 128:] @ W2[e, :, 128:].t()).half())
        at += n


@pytest.mark.parametrize("rows,d,f", LONG + SHORT, ids=str)
@pytest.mark.parametrize("other", [False, True])
def test_first_product_to_one_step(m, rows, d, f, other):
    """Sums of d whole numbers times 16 with scales of their own for each block; GeLU leaves x >= 16 and makes the others
    zero; each output is one hidden value, which is within half a step of 8 bits of the exact sum (and 1 ulp of GeLU's
    reciprocal)."""
    g = gen(d * 3 + f)
    E, T = len(rows), sum(rows)
    x = ints(g, -2, 2, T, d) * torch.exp2(ints(g, 0, 2, T, d // 128)).repeat_interleave(128, 1)
    W1 = ints(g, -2, 2, E, f, d) * torch.exp2(spread(ints(g, 4, 7, E, f // 128, d // 128), 128, 128))
    W2 = torch.zeros((E, d, f), dtype=torch.float64, device="cuda")
    j = torch.arange(d, device="cuda")
    pick = (j * 37 + 5) % f
    W2[:, j, pick] = 2.0 ** -6                        # (so that they are within f16's range)
    out, launches = run(m, x.half(), rows, to8(m, W1), to8(m, W2), other)
    assert launches == (TWO_FORMS if (rows, d, f) in LONG else ONE_FORM)
    at = 0
    for e, n in enumerate(rows):
        h = (x[at:at + n] @ W1[e].t()).clamp(min=0)
        top = h.unflatten(1, (-1, 128)).amax(2)
        # e4m3 at a scale s with top <= 448 s (top 1 ulp off): steps of 2^-3 of a value's power of two, at least s 2^-9
        s = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1.0) * (1 + 2 * U) / 448))).repeat_interleave(128, 1)
        step = torch.maximum(torch.exp2(torch.floor(torch.log2(h.clamp(min=1.0))) - 3), s * 2.0 ** -9)
        got = out[at:at + n].double() * 64
        err = (got - h[:, pick]).abs()
        assert bool((err <= (step / 2 + 4 * U * h)[:, pick]).all()), f"expert {e}: {float(err.max())}"
        at += n


@pytest.mark.parametrize("rows,d,f", [([480], 3584, 14336), ([1900, 148], 256, 16384), ([500], 2048, 8192)], ids=str)
@pytest.mark.parametrize("other", [False, True])
def test_sums_of_one_sign(m, rows, d, f, other):
    """Additions that are cut off always lose: over f positive terms this must not add up.  A tensor core's addition of 32
    products loses at most 2 u of the sum so far; of 1024 terms, whose sum so far grows evenly, 2 u (1 + .. + 32) / 32 =
    33 u.  The sums of those, at most 16, are rounded: u / 2 (1 + .. + 16) / 16 = 4 u.  The mean of N outputs rounded to
    f16 (each off by at most 2^-11, evenly spread) has a deviation of 2^-11 / sqrt(3 N), of which four are allowed."""
    g = gen(f)
    E, T = len(rows), sum(rows)
    x = 4 * ints(g, 4, 7, T, d)
    W1 = torch.zeros((E, f, d), dtype=torch.float64, device="cuda")
    j = torch.arange(f, device="cuda")
    W1[:, j, j % d] = 1.0
    q2 = torch.empty((E, d, f), dtype=torch.float8_e4m3fn, device="cuda")
    s2 = torch.empty((E, d // 128, f // 128), device="cuda")
    # weights of all sizes down to the smallest that 8 bits hold, so that each sum has bits to lose
    m.moe_fp8_quantize(torch.exp2(-14 * torch.rand((E, f, d), generator=g, device="cuda")) * 2.0 ** -5, q2, s2)
    out, launches = run(m, x.half(), rows, to8(m, W1), (q2, s2), other)
    assert launches == TWO_FORMS
    at, off = 0, []
    for e, n in enumerate(rows):
        want = x[at:at + n][:, j % d] @ (q2[e].double() * spread(s2[e].double(), 128, 128)).t()
        off.append((out[at:at + n].double() / want - 1).flatten())
        at += n
    off = torch.cat(off)
    assert abs(float(off.mean())) <= 37 * U + 4 * 2.0 ** -11 / (3 * off.numel()) ** 0.5
    assert float(off.abs().max()) <= 2.0 ** -11 + 37 * U


@pytest.mark.parametrize("rows,d,f", [([1200], 256, 27136), ([160, 161, 3, 90], 4352, 6400), ([700, 650, 1], 768, 8192),
                                      ([65] * 99, 1280, 1024)], ids=str)
def test_random_values_on_the_whole(m, rows, d, f):
    """Outputs of random values in the mean square.  Rounding to f16 is at most 2^-11 of each; a hidden value next to the
    border of two 8-bit values, at least 2^-4 of it apart, may take the other, which moves it by at most 2^-3: 240 u of
    a hidden value's size would move 2.3e-4 of them, and the outputs by sqrt(2.3e-4) 2^-3 = 1.9e-3 of their size.  With
    the rounding 2^-9; a block of 128 of 27136 inputs that is left out would be 35 times that."""
    g = gen(f + 1)
    E, T = len(rows), sum(rows)
    x = torch.randn((T, d), generator=g, device="cuda").half()

    def weights(n_in, n_out):
        q = torch.empty((E, n_out, n_in), dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty((E, n_out // 128, n_in // 128), device="cuda")
        m.moe_fp8_quantize((torch.randn((E, n_in, n_out), generator=g, device="cuda") * n_in ** -0.5).half(), q, s)
        return q, s
    W1, W2 = weights(d, f), weights(f, d)
    out, launches = run(m, x, rows, W1, W2)
    assert launches == TWO_FORMS

    def rows8(v):
        b = v.unflatten(1, (-1, 128))
        _, e = torch.frexp(b.abs().amax(2, keepdim=True) / 448)
        s = torch.exp2(e.double())                    # (a power of two: amax / 448 below it)
        s = torch.where(b.abs().amax(2, keepdim=True) <= 448 * s / 2, s / 2, s)
        return ((b / s).float().to(torch.float8_e4m3fn).double() * s).flatten(1)
    at, num, den = 0, 0.0, 0.0
    for e, n in enumerate(rows):
        w1, w2 = (q[e].double() * spread(s[e].double(), 128, 128) for q, s in (W1, W2))
        h = torch.nn.functional.gelu(rows8(x[at:at + n].double()) @ w1.t(), approximate="tanh")
        want = rows8(h) @ w2.t()
        num += float((out[at:at + n].double() - want).square().sum())
        den += float(want.square().sum())
        at += n
    assert num ** 0.5 <= 2.0 ** -9 * den ** 0.5
