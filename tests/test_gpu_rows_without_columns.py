"""Rows without columns: the values that the formulas give are written."""
import pytest
import torch

import invariant_matmul_amd as imm
from invariant_matmul_amd import torch_ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LEAST = 2.0 ** -120  # the scale of a row whose largest magnitude is zero, as that of no values is


def poison():
    """Freed blocks full of NaN, for the operators' new tensors to land in."""
    blocks = [torch.full((128,), float("nan"), device=dev()) for _ in range(64)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
@pytest.mark.parametrize("lead", [(1,), (5,), (2, 3), (300,)])
def test_rows_without_columns(lead, out, dt):
    x = torch.empty(*lead, 0, dtype=dt, device=dev())
    w = torch.empty(0, dtype=dt, device=dev())
    poison()
    for q, scale, *h in (torch_ops.quantize_rows(x, F8[out]), torch_ops.rms_norm_quant(x, w, dtype=F8[out]),
                         torch_ops.rms_norm_quant(x, None, residual=x, dtype=F8[out])):
        assert q.shape == x.shape and scale.shape == lead and (scale == LEAST).all()
        y = torch_ops.linear_f8(q, scale, torch.empty(16, 0, dtype=F8[out], device=dev()),
                                torch.ones(16, device=dev()), bias=torch.arange(16., device=dev()))
        assert torch.equal(y, torch.arange(16.).bfloat16().to(dev()).expand(*lead, 16))
    poison()
    y, h, rstd = torch_ops.rms_norm_forward(x, w)
    assert y.shape == h.shape == x.shape and rstd.shape == lead and rstd.isnan().all()  # the mean of nothing
    assert torch_ops.rms_norm(x, w, residual=x)[0].shape == x.shape
    dx, dw = torch_ops.rms_norm_backward(x, x, w, rstd)
    assert dx.shape == x.shape and dw.shape == (0,)


def test_rows_without_columns_in_c():
    x = torch.empty(5, 0, dtype=torch.bfloat16, device=dev())
    q = torch.empty(5, 0, dtype=torch.float8_e4m3fn, device=dev())
    for call in (lambda s, r: imm.rms_norm_run(imm.rms_norm_plan(5, 0, "bf16", "e4m3"), x, q, row_scale=s, rstd=r),
                 lambda s, r: imm.quantize_rows(x, q, s)):
        scale, rstd = torch.full((7,), 7.0, device=dev()), torch.full((7,), 7.0, device=dev())
        call(scale[:5], rstd[:5])
        assert (scale[:5] == LEAST).all() and (scale[5:] == 7).all() and (rstd[5:] == 7).all()
    rstd = torch.full((7,), 7.0, device=dev())
    imm.rms_norm_run(imm.rms_norm_plan(5, 0, "bf16"), x, x, rstd=rstd[:5])
    assert rstd[:5].isnan().all() and (rstd[5:] == 7).all()
