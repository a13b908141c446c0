"""fp8 rows have the bits of their definition: q = round8(t / row_scale) with the
division and row_scale = max(max |t| / FMAX, 2^-120) rounded in fp32, and for the
norm t = (h rstd) weight, each product rounded in fp32.  The oracle is those
operations on the CPU, one by one.
"""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def defined(t, out):
    """(codes, scales) of fp32 rows t on the CPU."""
    scale = (t.abs().amax(1) / FMAX[out]).clamp(min=2.0 ** -120)
    return (t / scale[:, None]).to(F8[out]), scale


def same(q, scale, t, out):
    want, ws = defined(t, out)
    assert torch.equal(scale.cpu(), ws)
    bad = q.cpu().view(torch.uint8) != want.view(torch.uint8)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} codes differ"


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", [(200, 4096), (4000, 128), (50, 14336), (700, 1040), (20, 32768)])
def test_codes_of_quantize_rows(rows, cols, out, dt):
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g).to(DT[dt])
    q, scale = torch_ops.quantize_rows(x.to(dev()), F8[out])
    same(q, scale, x.float(), out)


@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
def test_codes_at_the_ends_of_the_range(out):
    """Rows from bf16's smallest values to its largest, and from fp16's."""
    g = torch.Generator().manual_seed(11)
    for dt, lo, hi in (("bf16", -133, 126), ("f16", -24, 14)):
        x = torch.randn(4 * (hi - lo), 256, generator=g, dtype=torch.float64).clamp(-1.9, 1.9)
        x = (x * 2.0 ** (lo + torch.arange(x.shape[0]) // 4).double()[:, None]).to(DT[dt])
        assert torch.isfinite(x.float()).all()
        q, scale = torch_ops.quantize_rows(x.to(dev()), F8[out])
        same(q, scale, x.float(), out)


@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
def test_codes_of_zeros_and_rows_of_zeros(out):
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    x[0, ::2], x[1, 1::3], x[1, 5], x[2, 7] = -0.0, -0.0, 3.0, -1.7
    q, scale = torch_ops.quantize_rows(x.to(dev()), F8[out])
    same(q, scale, x.float(), out)


@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
def test_codes_at_ties(out):
    """Quotients halfway between two codes, exact and a bit of fp32 to either side."""
    codes = torch.arange(256, dtype=torch.uint8).view(F8[out]).float()
    codes = codes[torch.isfinite(codes) & (codes >= 0)].sort().values
    mid = (codes[1:] + codes[:-1]) / 2
    for m in range(64):  # scales of every 16-bit significand: bf16 amax = FMAX (1 + m / 128)
        s = (1 + m / 128) * 2.0 ** (m % 5 - 2)
        x = torch.zeros(1, 512, dtype=torch.bfloat16)
        x[0, :mid.numel()] = (mid * s).bfloat16()
        x[0, -1] = FMAX[out] * s
        q, scale = torch_ops.quantize_rows(x.to(dev()), F8[out])
        same(q, scale, x.float(), out)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", [(300, 1040), (130, 4096), (40, 16384), (1000, 128)])
def test_codes_of_the_norm(rows, cols, out, dt):
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, cols, generator=g).to(DT[dt]).to(dev())
    r = torch.randn(rows, cols, generator=g).to(DT[dt]).to(dev())
    w = (1 + 0.3 * torch.randn(cols, generator=g)).to(DT[dt]).to(dev())
    _, h, rstd = torch_ops.rms_norm_forward(x, w, 1e-5, residual=r)
    q, scale, h2 = torch_ops.rms_norm_quant(x, w, 1e-5, residual=r, dtype=F8[out])
    assert torch.equal(h, h2)
    same(q, scale, (h.cpu().float() * rstd.cpu()[:, None]) * w.cpu().float(), out)
