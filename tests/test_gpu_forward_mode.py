"""Forward-mode derivatives: the operators have none, so a tangent is refused, not dropped."""
import pytest
import torch
from torch.autograd import forward_ad

from invariant_matmul_amd import torch_ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu


def test_tangents_are_refused():
    g = torch.Generator().manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=g).bfloat16().to(dev())

    x, w, r = normal(4, 64), normal(64), normal(4, 64)
    q, s = torch_ops.quantize_rows(x)
    wq, ws = torch_ops.quantize_rows(normal(32, 64))
    codes = torch.randint(0, 256, (32, 32), generator=g, dtype=torch.uint8).to(dev())
    scales = normal(32, 1)
    w4 = torch_ops.pack_w4(codes, scales)
    bias = torch.randn(32, generator=g).to(dev())
    dy = normal(4, 64)
    rstd = torch_ops.rms_norm_forward(x, w)[2]

    def calls(x, w, r, s, ws, bias, scales, dy, rstd):
        return {
            "rms_norm": ((x, w, r), lambda: torch_ops.rms_norm(x, w, residual=r)),
            "rms_norm_forward": ((x, w, r), lambda: torch_ops.rms_norm_forward(x, w, residual=r)),
            "rms_norm_backward": ((x, w, dy, rstd, r), lambda: torch_ops.rms_norm_backward(dy, x, w, rstd, r)),
            "rms_norm_quant": ((x, w, r), lambda: torch_ops.rms_norm_quant(x, w, residual=r)),
            "quantize_rows": ((x,), lambda: torch_ops.quantize_rows(x)),
            "linear_f8": ((s, ws, bias), lambda: torch_ops.linear_f8(q, s, wq, ws, bias=bias)),
            "pack_w4": ((scales,), lambda: torch_ops.pack_w4(codes, scales)),
            "linear_w4": ((x, bias), lambda: torch_ops.linear_w4(x, w4, bias)),
        }

    plain = (x, w, r, s, ws, bias, scales, dy, rstd)
    want = {k: f() for k, (_, f) in calls(*plain).items()}
    with forward_ad.dual_level():
        for i, t in enumerate(plain):
            dual = forward_ad.make_dual(t, torch.ones_like(t))
            for name, (reads, f) in calls(*plain[:i], dual, *plain[i + 1:]).items():
                if any(a is dual for a in reads):
                    with pytest.raises(ValueError, match=name), torch.no_grad():
                        f()
                    with pytest.raises(ValueError, match=name):
                        f()
        leaf = forward_ad.make_dual(x.clone().requires_grad_(), torch.ones_like(x))
        with pytest.raises(ValueError, match="rms_norm"):
            torch_ops.rms_norm(leaf, w)
        # plain tensors, and duals without their tangents, are what they are outside
        for k, (_, f) in calls(*plain).items():
            if k != "pack_w4":
                got, ref = f(), want[k]
                for a, b in zip(got if isinstance(got, tuple) else (got,), ref if isinstance(ref, tuple) else (ref,)):
                    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        assert torch.equal(torch_ops.rms_norm(forward_ad.unpack_dual(dual).primal, w), torch_ops.rms_norm(x, w))
