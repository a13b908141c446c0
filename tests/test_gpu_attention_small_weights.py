"""The gradient of values that many keys share: probabilities below the normal numbers of fp16."""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests import decoder_oracle as ref
from tests.helpers import dev
from tests.test_gpu_attention import DT, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("std", [0.3, 1.5])
@pytest.mark.parametrize("n,m,hq,D", [(1, 65536, 1, 64), (5, 65536, 2, 128), (40, 16384, 1, 96), (1, 300, 1, 64)])
def test_dv(n, m, hq, D, std, dt):
    q, k, v, do = make(n, m, hq, 1, D, dt, 60 + n, std)
    do = do * 1024  # (so that dv is not below fp16's normal numbers itself)
    o, saved = torch_ops.attention_forward(q, k, v, causal=False)
    _, _, dv = torch_ops.attention_backward(do, q, k, v, o, saved, causal=False)
    _, lse, p, _ = ref.attend(q, k, v, False, D ** -0.5)                                  # [hq, n, m]
    qd, kd, dod = q.double().transpose(0, 1), k.double()[:, 0], do.double().transpose(0, 1)
    want = sum(p[h].T @ dod[h] for h in range(hq))
    # p: a chain of D products and the scale; lse, which sums 16 values of a lane and step, 4 steps, 4 lanes and
    # m / 256 chunks, all positive; the exponential's argument, whose terms reach |lse| and the logit in
    # magnitude and 14 more (four roundings of them); exponential and logarithm; then half a step of the type, or
    # of its smallest subnormal number 14 places down
    U = ref.U
    mag = D ** -0.5 * torch.stack([qd[h].abs() @ kd.abs().T for h in range(hq)])
    top = lse.abs().amax() + 14 + 2 * mag.amax()
    eps = 2 * (D + 4) * U * mag + (m / 256 + 32) * U + 8 * U * top + 2.0 ** -20
    # (the lowest places are the products': 2^-14 of a subnormal step of fp16)
    e_p = p * (eps + ref.half(DT[dt]) * (1 + eps) + n * hq * U) + ref.tiny(DT[dt]) * 2.0 ** -14
    tol = sum(e_p[h].T @ dod[h].abs() for h in range(hq)) + want.abs() * ref.half(DT[dt]) + ref.tiny(DT[dt])
    ref.close(dv[:, 0], want, tol, "dv")
    # on the whole: the roundings of p (of n hq terms) and of dv are independent, each 0.6 of half a step in the mean
    off = (dv[:, 0].double() - want).norm() / want.norm()
    assert off <= 1.5 * ref.half(DT[dt]), float(off)
