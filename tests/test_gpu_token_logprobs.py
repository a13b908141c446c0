"""Log probabilities of tokens, entropy, the most likely tokens, and the gradient of the
logits, against 64 bits (tests/decoder_oracle.py).

Bounds.  e^d of d = x - max is off by 2^-22 + |d| 2^-23 of itself (the difference, the product
with log2 e and the exponential), sums of non-negative terms by (32 + 6 + units / 64 + 6) roundings
and as much from the moves between maxima: below 2^-17 of themselves for |d| <= 60, beyond
which e^d counts less than 2^-60.  So log_sum and T / S are within 2^-16 of max(1, magnitude), a log
probability adds two roundings of its own magnitude.
"""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests import decoder_oracle as ref
from tests.helpers import dev

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
LOG = 2.0 ** -16
INF, NAN = float("inf"), float("nan")


def make(rows, V, dt, seed, spread=3.0, n=1):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, V, generator=g) * spread).to(DT[dt]).to(dev())
    t = torch.randint(0, V, (rows, n), generator=g).to(dev())
    return x, t, torch.randn(rows, n, generator=g).to(dev()), torch.randn(rows, generator=g).to(dev())


def check(x, t, top, what=""):
    lp, ent, *best = torch_ops.token_logprobs(x, t, top)
    wl, we, wt, wi = ref.logprobs(x, t if t.dim() == 2 else t[:, None], top)
    ref.close(lp, wl.reshape(lp.shape), LOG + wl.reshape(lp.shape).abs().nan_to_num(posinf=0) * 2.0 ** -22, f"logprob {what}")
    ref.close(ent, we, LOG * (1 + we.abs().nan_to_num()), f"entropy {what}")
    if top:
        assert best[1].dtype == torch.int64 and torch.equal(best[1], wi), f"tokens {what}"
        ref.close(best[0], wt, LOG + wt.abs().nan_to_num(posinf=0) * 2.0 ** -22, f"top {what}")
    return lp, ent, *best


# below, at and above a vector, a lane's vectors, a unit (2048), a workgroup's units (8192)
VOCABS = [1, 2, 7, 8, 9, 64, 511, 513, 2047, 2048, 2049, 8191, 8193, 32000, 50257, 131072, 300007]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", VOCABS)
def test_matches_the_formula(V, dt):
    x, t, _, _ = make(5, V, dt, V)
    check(x, t[:, 0], min(20, V))


@pytest.mark.parametrize("rows", [1, 2, 63, 511, 512, 1023, 1024, 1500])
def test_numbers_of_rows_and_their_bits(rows):
    x, t, _, _ = make(1500, 9001, "bf16", 3)
    whole = torch_ops.token_logprobs(x, t, 9)
    part = check(x[:rows], t[:rows], 9)
    assert all(torch.equal(a[:rows], b) for a, b in zip(whole, part))
    one = torch_ops.token_logprobs(x[rows - 1:rows].clone(), t[rows - 1:rows], 9)
    assert all(torch.equal(a[rows - 1:rows], b) for a, b in zip(whole, one))


@pytest.mark.parametrize("top", [0, 1, 2, 33, 63, 64])
def test_numbers_of_alternatives(top):
    x, t, _, _ = make(3, 70001, "f32", 4)
    check(x, t, top)


def test_ties_go_to_the_lower_token():
    V = 20011
    x = torch.zeros(6, V, dtype=torch.bfloat16, device=dev())
    x[1] = -0.0
    x[1, 100:20000:7] = 0.0
    x[2, ::3] = 2.0
    x[3] = torch.arange(V, device=dev()) // 64   # ascending: each unit is better than all before
    x[4] = -(torch.arange(V, device=dev()) // 64)
    x[5, 17000:] = 1.0
    check(x, torch.zeros(6, 1, dtype=torch.int64, device=dev()), 64)
    check(x.float(), torch.zeros(6, 1, dtype=torch.int64, device=dev()), 20)


def test_masked_and_bad_logits():
    x, t, _, _ = make(8, 5000, "f32", 5)
    x[0, 1:] = -INF              # one token left
    t[0] = 0
    x[1, ::2] = -INF
    t[1] = 4                     # a masked one
    x[2] = torch.finfo(torch.float32).min
    x[3] = -INF                  # nothing left
    x[4, 77] = NAN
    x[5, 78] = INF
    x[6, 2:] = torch.finfo(torch.float32).min
    check(x, t, 10)
    clean, _, _, _ = make(8, 5000, "f32", 5)
    a, b = torch_ops.token_logprobs(x, t, 10), torch_ops.token_logprobs(clean, t, 10)
    assert all(torch.equal(u[7], v[7]) for u, v in zip(a, b))
    for dt in (torch.bfloat16, torch.float16):
        y = x.clamp(min=torch.finfo(dt).min).to(dt)
        y[1, ::2] = y[3] = -INF
        check(y, t, 10)


def test_large_offsets():
    # the difference to the largest logit counts, not the logits' own magnitude
    x, t, g, h = make(4, 3001, "f32", 6)
    x = (x * 2 ** 10).round() / 2 ** 10 + 2.0 ** 12
    check(x, t, 5)


def test_tokens_of_a_row():
    x, t, g, h = make(6, 1001, "bf16", 7, n=70)
    t[0, :] = 5                  # the same token over and over
    t[1, ::2] = -100             # padding
    t[2, 3] = 1001               # past the vocabulary
    lp, _ = check(x, t, 0)
    assert (lp[1, ::2] == 0).all() and torch.isnan(lp[2, 3]) and torch.isfinite(lp[2, 4:]).all()
    y = x.reshape(2, 3, 1001)
    again = torch_ops.token_logprobs(y, t.reshape(2, 3, 70), 3)
    assert again[0].shape == (2, 3, 70) and again[1].shape == (2, 3) and again[2].shape == again[3].shape == (2, 3, 3)
    assert torch.equal(again[0].reshape(6, 70).nan_to_num(7), lp.nan_to_num(7))
    none = torch_ops.token_logprobs(x, t[:, :0], 1)
    assert none[0].shape == (6, 0) and torch.equal(none[1], again[1].reshape(6))


def gradient_bound(x, t, g, h):
    """p is off by 2^-20 of itself plus 2^-23 of |logp| and the logarithm's LOG, entropy by LOG"""
    logp = torch.log_softmax(x.double(), 1)
    p = logp.exp()
    logp = torch.where(p > 0, logp, torch.zeros_like(logp))
    ent = -(p * logp).sum(1, keepdim=True)
    G, H = g.double().abs().sum(1, keepdim=True), h.double().abs()[:, None]
    terms = p * (G + H * (logp.abs() + ent)) * (2 * LOG) + p * H * LOG * (1 + ent)
    return terms + (G + H) * 2.0 ** -60


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [1, 7, 8, 1000, 2047, 2049, 50257, 131072])
@pytest.mark.parametrize("n", [1, 3])
def test_gradient_matches_the_formula(V, dt, n):
    x, t, g, h = make(5, V, dt, 8 + V, n=n)
    if n == 3:
        t[0, 1] = t[0, 0]
        t[1, 0] = -1
    lp, ent, norm = torch_ops.token_logprobs_forward(x, t)
    dx = torch_ops.token_logprobs_backward(g, h, x, t, norm, ent)
    assert dx.dtype == x.dtype and dx.is_contiguous()
    cases = [(dx, g, h)]
    if n == 1:
        cases += [(torch_ops.token_logprobs_backward(g, None, x, t, norm, ent), g, 0 * h),
                  (torch_ops.token_logprobs_backward(None, h, x, t, norm, ent), 0 * g, h)]
    for got, g1, h1 in cases:
        want = ref.logprobs_gradient(x, t, g1, h1)
        gm = torch.where(t >= 0, g1, torch.zeros_like(g1))
        # p, logp and the entropy; the final rounding, half a step of the value that is compared
        # (and 2^-22 of it for the fp32 operations before); the roundings of the sum of g
        tol = gradient_bound(x, t, gm, h1) + want.abs() * (ref.half(x.dtype) + 2.0 ** -22) + ref.tiny(x.dtype)
        tol = tol + (gm.abs().sum(1, keepdim=True).double()) * 2.0 ** -22
        ref.close(got, want, tol, "dx")


def test_gradient_of_masked_logits():
    x, t, g, h = make(4, 3000, "f32", 9)
    x[0, 10:] = -INF
    t[0] = 3
    x[1, 1:] = -INF
    t[1] = 0
    x[2, ::2] = torch.finfo(torch.float32).min
    t[2] = 1
    lp, ent, norm = torch_ops.token_logprobs_forward(x, t)
    dx = torch_ops.token_logprobs_backward(g, h, x, t, norm, ent)
    want = ref.logprobs_gradient(x, t, g, h)
    ref.close(dx, want, gradient_bound(x, t, g, h) + want.abs() * 2.0 ** -21 + 2.0 ** -22 * g.abs().double(), "masked")
    assert (dx[0, 10:] == 0).all() and (dx[2, ::2] == 0).all()


def test_autograd_and_differences():
    x, t, g, h = make(3, 257, "f32", 10, spread=1.5)
    leaf = x.clone().requires_grad_()
    lp, ent, top, tok = torch_ops.token_logprobs(leaf, t, 4)
    assert not top.requires_grad and not tok.requires_grad
    torch.autograd.backward((lp, ent), (g, h))
    _, e, norm = torch_ops.token_logprobs_forward(x, t)
    assert torch.equal(leaf.grad, torch_ops.token_logprobs_backward(g, h, x, t, norm, e))

    def loss(y):
        a, b, _, _ = ref.logprobs(y, t, 0)
        return (a * g.double()).sum() + (b * h.double()).sum()

    d = torch.randn(x.shape, generator=torch.Generator().manual_seed(11)).double().to(dev())
    step = 1e-5
    want = (loss(x.double() + step * d) - loss(x.double() - step * d)) / (2 * step)
    tol = ((gradient_bound(x, t, g, h) + 2.0 ** -20 * (g.abs() + h.abs()[:, None]).double()) * d.abs()).sum() + 1e-6
    assert abs((leaf.grad.double() * d).sum() - want) <= tol
    leaf.grad = None
    torch_ops.token_logprobs(leaf, t)[0].sum().backward()  # an expanded gradient
    assert torch.equal(leaf.grad, torch_ops.token_logprobs_backward(torch.ones_like(g), None, x, t, norm, e))


def test_strided_rows():
    x, t, g, h = make(6, 4099, "bf16", 12)
    wide = torch.full((6, 5003), NAN, dtype=torch.bfloat16, device=dev())
    wide[:, 11:11 + 4099] = x
    view = wide[:, 11:11 + 4099]
    want = torch_ops.token_logprobs(x, t, 6)
    for y in (view, x.t().contiguous().t()):
        assert all(torch.equal(a, b) for a, b in zip(torch_ops.token_logprobs(y, t, 6), want))
    _, e, norm = torch_ops.token_logprobs_forward(view, t)
    assert torch.equal(torch_ops.token_logprobs_backward(g, h, view, t, norm, e),
                       torch_ops.token_logprobs_backward(g, h, x, t, norm, e))


def test_no_rows_and_refusals():
    x, t, g, h = make(3, 100, "bf16", 13)
    lp, ent, top, tok = torch_ops.token_logprobs(x[:0], t[:0], 2)
    assert lp.shape == (0, 1) and ent.shape == (0,) and top.shape == tok.shape == (0, 2)
    for bad in (lambda: torch_ops.token_logprobs(x.double(), t), lambda: torch_ops.token_logprobs(x.cpu(), t.cpu()),
                lambda: torch_ops.token_logprobs(x, t.int()), lambda: torch_ops.token_logprobs(x, t[:2]),
                lambda: torch_ops.token_logprobs(x, t, 65), lambda: torch_ops.token_logprobs(x, t, -1),
                lambda: torch_ops.token_logprobs(x[:, :5], t, 6), lambda: torch_ops.token_logprobs(x, t.cpu()),
                lambda: torch_ops.token_logprobs_backward(g.half(), h, x, t, torch.empty(3, 2, device=dev()), h),
                lambda: torch_ops.token_logprobs_backward(g, h, x, t, h, h)):
        with pytest.raises(ValueError):
            bad()
