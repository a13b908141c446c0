"""Log probabilities of one row agree with each other bit by bit: in whatever column a token is asked for, as a
given token and as an alternative, and with the numbers that the backward pass takes."""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests import decoder_oracle as ref
from tests.helpers import dev
from tests.test_gpu_token_logprobs import DT, gradient_bound, make

pytestmark = pytest.mark.gpu


def confident(rows, V, dt, seed):
    """Rows whose largest logits stand far above the rest, so that units' maxima differ."""
    x, _, _, _ = make(rows, V, dt, seed, spread=2.0)
    g = torch.Generator().manual_seed(seed + 1)
    at = torch.randint(0, V, (rows, 40), generator=g).to(dev())
    up = torch.rand(rows, 40, generator=g).to(dev()) * 12
    return x.scatter(1, at, (x.gather(1, at).float() + up).to(x.dtype)), at


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [5000, 50257, 300007])
@pytest.mark.parametrize("rows", [3, 1100])  # rows cut into parts, and whole
def test_columns_and_alternatives(rows, V, dt):
    if rows * V > 10 ** 8:
        rows = 1024 if V < 10 ** 5 else 3
    x, at = confident(rows, V, dt, 80 + rows)
    x[:, 100:140] = x[:, 100:101]  # equal logits
    tokens = torch.cat((at[:, :1].expand(-1, 64), at[:, 1:], torch.arange(100, 140, device=dev()).expand(rows, -1)), 1).contiguous()
    lp, ent, top_lp, top = torch_ops.token_logprobs(x, tokens, 64)
    _, _, norm = torch_ops.token_logprobs_forward(x, tokens)
    own = (x.gather(1, tokens).float() - norm[:, :1]) - norm[:, 1:]
    assert torch.equal(lp, own), int((lp != own).sum())
    assert (lp[:, :64] == lp[:, :1]).all() and (lp[:, 103:] == lp[:, 103:104]).all()
    again = torch_ops.token_logprobs(x, top, 0)[0]
    assert torch.equal(again, top_lp), int((again != top_lp).sum())
    assert (top_lp[:, 1:] <= top_lp[:, :-1]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradient_of_a_thousand_tokens_a_row(dt):
    x, t, g, h = make(2, 3001, dt, 90, n=1024)
    t[0, 5:900] = -1
    t[1, ::3] = 17
    lp, ent, norm = torch_ops.token_logprobs_forward(x, t)
    dx = torch_ops.token_logprobs_backward(g, h, x, t, norm, ent)
    want = ref.logprobs_gradient(x, t, g, h)
    gm = torch.where(t >= 0, g, torch.zeros_like(g)).double().abs()
    # the sums of g, over a row's tokens and over those that are the same logit: 1024 roundings of 2^-24 at most
    tol = gradient_bound(x, t, gm, h) + want.abs() * (ref.half(DT[dt]) + 2.0 ** -22) + gm.sum(1, keepdim=True) * 1024 * ref.U
    ref.close(dx, want, tol + ref.tiny(DT[dt]), "dx")
