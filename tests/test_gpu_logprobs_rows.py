"""Log probabilities of logits whose rows are not one stride apart, or only through several dimensions: the same
results, and copies of the logits only where they are needed, once for both directions."""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

B, T, V = 6, 40, 50000


def inputs():
    g = torch.Generator(device=dev()).manual_seed(95)
    x = torch.randn(B, T, V, generator=g, device=dev()).bfloat16()
    return x, torch.randint(0, V, (B, T), generator=g, device=dev())


@pytest.mark.parametrize("view", [lambda x: x[:, :-1], lambda x: x[..., 3:-5], lambda x: x[:, ::2], lambda x: x[:, 3:4], lambda x: x.transpose(0, 1),
                                  lambda x: x[0], lambda x: x[2, 7]], ids=range(7))
def test_views_have_the_results_of_their_values(view):
    x, t = inputs()
    y = view(x)
    tok = torch.randint(0, y.shape[-1], y.shape[:-1], device=dev())
    leaf, dense = y.detach().requires_grad_(), y.detach().contiguous().requires_grad_()
    a, b = torch_ops.token_logprobs(leaf, tok, 5), torch_ops.token_logprobs(dense, tok, 5)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    ga, = torch.autograd.grad(a[0].sum() + a[1].sum(), leaf)
    gb, = torch.autograd.grad(b[0].sum() + b[1].sum(), dense)
    assert torch.equal(ga, gb) and ga.shape == leaf.shape


@pytest.mark.parametrize("shifted", [True, False])
def test_memory(shifted):
    x, t = inputs()
    leaf = (x[:, :-1] if shifted else x[..., :-8]).detach().requires_grad_()
    tok = t[:, :leaf.shape[1]].contiguous().clamp(max=leaf.shape[2] - 1)
    size, small = leaf.numel() * 2, 1 << 21

    def grown(f):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        r = f()
        return r, torch.cuda.max_memory_allocated() - before

    (lp, _), more = grown(lambda: torch_ops.token_logprobs(leaf, tok))
    assert more < small + (size if shifted else 0)
    _, more = grown(lambda: torch.autograd.grad(lp.sum(), leaf))
    assert size <= more < size + small  # the gradient alone


def test_a_change_after_the_call_is_noticed():
    x, t = inputs()
    x.requires_grad_()
    lp, _ = torch_ops.token_logprobs(x, t)
    with torch.no_grad():
        x.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        lp.sum().backward()
