"""Attention's gradients with a NaN or an infinity in q, k, v or the gradient of o: the bits follow from the
sequence alone, whatever the call's size and so its kernels are, and how far it reaches is bounded."""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests.helpers import dev
from tests.test_gpu_attention import INF, NAN, ints, make, starts

pytestmark = pytest.mark.gpu

REACH = 15 + 63  # places beyond what the formula gives


def backward_groups(Tq, Tk, hq, hk, batch):
    """Workgroups of 128 rows or keys: waves take 32 from 801 on."""
    return (Tq * (hq // hk) // 128 + 2 * (Tk // 128) + 3 * batch) * hk


def gradients(q, k, v, do, cu_q=None, cu_k=None, lens=None, causal=True):
    o, saved = torch_ops.attention_forward(q, k, v, cu_q, cu_k, k_lens=lens, causal=causal)
    return torch_ops.attention_backward(do, q, k, v, o, saved, cu_q, cu_k, k_lens=lens, causal=causal)


def same(a, b):
    return torch.equal(a.nan_to_num(3, 4, 5), b.nan_to_num(3, 4, 5)) and torch.equal(a.isnan(), b.isnan())


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("which", ["q", "k", "v", "do"])
@pytest.mark.parametrize("n,m,group,D,dt", [(330, 340, 1, 128, "bf16"), (300, 377, 2, 64, "f16"), (130, 511, 3, 96, "f16"), (400, 333, 1, 64, "bf16")])
def test_small_and_large_calls(n, m, group, D, dt, which, bad):
    hk = 130
    q, k, v, do = make(n, m, hk * group, hk, D, dt, n + m)
    t = {"q": q, "k": k, "v": v, "do": do}[which]
    for at in (m - n + 32 if which in ("k", "v") else 32, 127, 200, t.shape[0] - 1):
        if 0 <= at < t.shape[0]:
            for head in range(0, t.shape[1], 3):
                t[at, head, (5 + head) % D] = bad
    assert backward_groups(n, m, hk * group, hk, 1) > 800
    cu_q, cu_k = ints([0, n]), ints([0, m])
    large = gradients(q, k, v, do, cu_q, cu_k)
    few = 7
    assert backward_groups(n, m, few * group, few, 1) <= 800
    small = gradients(q[:, :few * group], k[:, :few], v[:, :few], do[:, :few * group].contiguous(), cu_q, cu_k)
    for a, b, name in zip(small, large, ("dq", "dk", "dv")):
        assert same(a, b[:, :a.shape[1]]), name
    # and beside another sequence
    q2, k2, v2, do2 = make(200, 200, hk * group, hk, D, dt, 70)
    cu_q, cu_k = starts([200, n]), starts([200, m])
    both = gradients(torch.cat((q2, q)), torch.cat((k2, k)), torch.cat((v2, v)), torch.cat((do2, do)), cu_q, cu_k)
    for a, b, lo, name in zip(large, both, (200,) * 3, ("dq", "dk", "dv")):
        assert same(a, b[lo:]) and torch.isfinite(b[:lo]).all(), name


@pytest.mark.parametrize("hk", [2, 160])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_reach(hk, bad):
    # causal, query t sees keys up to t + 10
    n, m, D = 330, 340, 64
    q, k, v, do = make(n, m, hk, hk, D, "bf16", 71)
    assert (backward_groups(n, m, hk, hk, 1) > 800) == (hk == 160)
    cu_q, cu_k = ints([0, n]), ints([0, m])
    clean = gradients(q, k, v, do, cu_q, cu_k)
    for at in (127, 190, 200, 300):
        for name, t in (("k", k), ("v", v)):  # a key: queries from at - 10 on see it
            kept = t[at, 0, 5].clone()
            t[at, 0, 5] = bad
            dq, dk, dv = gradients(q, k, v, do, cu_q, cu_k)
            t[at, 0, 5] = kept
            free = max(0, at - 10 - REACH)
            assert torch.equal(dq[:free], clean[0][:free]), (name, at)
            for x, y in zip((dq, dk, dv), clean):  # the other heads
                assert torch.equal(x[:, 1:], y[:, 1:])
            assert not torch.isfinite(dq[at - 10:, 0]).all(1).any()
        for name, t in (("q", q), ("do", do)):  # a query: it sees the keys up to at + 10
            kept = t[at, 0, 5].clone()
            t[at, 0, 5] = bad
            dq, dk, dv = gradients(q, k, v, do, cu_q, cu_k)
            t[at, 0, 5] = kept
            others = torch.arange(n, device=dev()) != at
            assert torch.equal(dq[others], clean[0][others]), (name, at)
            free = at + 11 + REACH
            assert torch.equal(dk[free:], clean[1][free:]) and torch.equal(dv[free:], clean[2][free:]), (name, at)
            assert not torch.isfinite(dk[:at + 11, 0]).all(1).any()


@pytest.mark.parametrize("hk", [2, 160])
def test_what_has_no_keys_and_no_queries_stays_zero(hk):
    # queries before the first key, and the room of a cache, beside bad queries and keys
    n, D = 300, 64
    q, k, v, do = make(n, 2 * n, hk, hk, D, "f16", 72)
    cu_q, cu_k, lens = ints([0, n]), ints([0, 2 * n]), ints([n - 75])
    assert (backward_groups(n, 2 * n, hk, hk, 1) > 800) == (hk == 160)
    q[::7], do[3::7], k[::5], v[2::5] = NAN, INF, NAN, INF
    dq, dk, dv = gradients(q, k, v, do, cu_q, cu_k, lens)
    assert (dq[:75] == 0).all() and (dk[n - 75:] == 0).all() and (dv[n - 75:] == 0).all()
