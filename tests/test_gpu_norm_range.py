"""The norm over the whole range of its type: rows whose sum of squares is no
fp32 value of full precision.

The oracle is the formula in 64 bits, the tolerances those of the other norm
tests (an fp32 value within 2^-18 of its terms' magnitudes, half a step of the
output's type), with half of fp32's smallest subnormal, 2^-150, where a value
itself is that small: rstd of rows near the type's end is 2^-128 and keeps 21
bits, 2^-22 of itself.
"""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8_TINY = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}
F32, HALF, TINY = 2.0 ** -18, 2.0 ** -8, 2.0 ** -134
# every thread layout
COLS = [8, 128, 256, 512, 1040, 2048, 4104, 8192, 14336, 32768]
# powers of two that a row is scaled by: sums that overflow from 2^56.5 on (32768
# columns) and below 2^-50 are no longer exact to fp32's last bits
HUGE = [50, 56, 57, 58, 60, 63, 64, 100, 124]
SMALL = [-45, -55, -63, -64, -75, -100, -110, -124]


def close(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).max())} of the bound"


def make(cols, powers, seed):
    """Rows of normal values times a power of two each; then a uniform row at the
    type's largest value, and one with a lone element there."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(len(powers) + 2, cols, generator=g).clamp(-4, 4)
    x[:len(powers)] *= 2.0 ** torch.tensor([float(p) for p in powers])[:, None]
    x = x.bfloat16()
    top = torch.finfo(torch.bfloat16).max
    x[-2] = top if max(powers) > 0 else 2.0 ** -126
    x[-1, cols // 2] = -top if max(powers) > 0 else 2.0 ** -60
    w = (1 + 0.3 * torch.randn(cols, generator=g)).bfloat16()
    return x.to(dev()), w.to(dev())


def formula(h, w, eps):
    h = h.double()
    rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    return rstd, h * rstd * w.double()


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("powers,eps", [(HUGE, 1e-6), (HUGE, 0.0), (SMALL, 0.0), (SMALL, 1e-30), (SMALL, 1e-40),
                                        (SMALL, 1e-6), (SMALL, 2.0 ** -61), (SMALL, 2.0 ** -59)])
def test_rows_over_the_whole_range(cols, powers, eps):
    x, w = make(cols, powers, cols)
    eps32 = float(torch.tensor(eps))
    rstd64, t = formula(x, w, eps32)
    y, h, rstd = torch_ops.rms_norm_forward(x, w, eps)
    close(rstd, rstd64[:, 0], rstd64[:, 0] * F32 + 2.0 ** -150, "rstd")
    close(y, t, t.abs() * (HALF + F32) + TINY, "y")
    assert torch.equal(torch_ops.rms_norm(x, w, eps), y)
    zero = torch.zeros_like(x)
    assert all(torch.equal(a, b) for a, b in zip(torch_ops.rms_norm(x, w, eps, residual=zero), (y, x)))
    for i in range(x.shape[0]):  # each row alone
        assert torch.equal(torch_ops.rms_norm(x[i:i + 1], w, eps)[0], y[i])
    if cols % 16 == 0:
        for out, dt in F8.items():
            q, scale = torch_ops.rms_norm_quant(x, w, eps, dtype=dt)
            want = (t.abs().amax(1) / FMAX[out]).clamp(min=2.0 ** -120)
            close(scale, want, want * F32, "scale")
            back = q.double() * scale.double()[:, None]
            close(back, t, t.abs() * (torch.finfo(dt).eps / 2 + 2 * F32) + F8_TINY[out] * scale.double()[:, None], out)


@pytest.mark.parametrize("cols", [128, 1040, 2048, 8192, 32768])
@pytest.mark.parametrize("powers,eps", [(HUGE, 1e-6), (SMALL[:-2], 0.0), (SMALL[:-2], 1e-30)])
def test_gradients_over_the_whole_range(cols, powers, eps):
    x, w = make(cols, powers, 7 + cols)
    x = x[:-2]
    g = torch.Generator().manual_seed(5)
    dy = torch.randn(x.shape, generator=g).bfloat16().to(dev())
    leaves = [x.clone().requires_grad_(), w.clone().requires_grad_()]
    dx, dw = torch.autograd.grad(torch_ops.rms_norm(*leaves, eps), leaves, dy)
    rstd, _ = formula(x, w, float(torch.tensor(eps)))
    n, gw = x.double() * rstd, dy.double() * w.double()
    want = rstd * (gw - n * (gw * n).mean(1, keepdim=True))
    bound = rstd * (gw.abs() + n.abs() * (gw * n).abs().mean(1, keepdim=True))
    close(dx, want, want.abs() * HALF + bound * F32 + TINY, "dx")
    wdw, bdw = (dy.double() * n).sum(0), (dy.double() * n).abs().sum(0)
    close(dw, wdw, wdw.abs() * HALF + bdw * F32 + TINY, "dw")


@pytest.mark.parametrize("cols", [8, 264, 4096])
def test_rows_of_subnormal_values(cols):
    """eps = 0 and a root mean square below 2^-128: its reciprocal is no fp32 value (rstd is
    infinite), the norm is."""
    g = torch.Generator().manual_seed(cols)
    x = (torch.randint(1, 16, (6, cols), generator=g) * torch.randint(0, 2, (6, cols), generator=g).mul(2).sub(1))
    x = (x.double() * 2.0 ** -133).bfloat16().to(dev())
    w = torch.ones(cols, dtype=torch.bfloat16, device=dev())
    rstd64, t = formula(x, w, 0.0)
    y, _, rstd = torch_ops.rms_norm_forward(x, w, 0.0)
    want = rstd64[:, 0].float().double()
    assert torch.isinf(want).any() and torch.equal(torch.isinf(rstd), torch.isinf(want))
    close(y, t, t.abs() * (HALF + F32) + TINY, "y")


@pytest.mark.parametrize("cols", [64, 1040, 4096, 16384])
@pytest.mark.parametrize("eps", [1e-5, 0.0])
def test_bad_rows_stay_alone_beside_the_largest(cols, eps):
    """NaN, infinities and zeros among rows at the ends of the range."""
    g = torch.Generator().manual_seed(13)
    x = torch.randn(12, cols, generator=g).bfloat16().to(dev())
    w = (1 + 0.3 * torch.randn(cols, generator=g)).bfloat16().to(dev())
    clean = torch_ops.rms_norm(x, w, eps)
    x[1, 3] = float("nan")
    x[4, cols - 1] = float("inf")
    x[7, 0] = -float("inf")
    x[9] = 0
    x[2], x[5] = 3.0e38, 1e-38
    ok = [0, 3, 6, 8, 10, 11]
    y = torch_ops.rms_norm(x, w, eps)
    q, sq = torch_ops.rms_norm_quant(x, w, eps)
    assert torch.equal(y[ok], clean[ok])
    assert y[1].isnan().all() and q[1].float().isnan().all() and sq[1].isnan()
    for i, k in ((4, cols - 1), (7, 0)):  # 1 / inf = 0: the other elements are zero
        rest = [j for j in range(cols) if j != k]
        assert y[i, k].isnan() and (y[i, rest] == 0).all()
        assert q[i].float().isnan().all() and not torch.isfinite(sq[i])
    if eps:
        assert (y[9] == 0).all() and (q[9].float() == 0).all() and sq[9] == 2.0 ** -120
    else:
        assert y[9].isnan().all()  # 0 / 0
    _, t = formula(x, w, float(torch.tensor(eps)))
    for i in (2, 5):
        close(y[i], t[i], t[i].abs() * (HALF + F32) + TINY, "y")
