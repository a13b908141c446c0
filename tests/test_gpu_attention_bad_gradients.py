"""Attention's gradients with a NaN or an infinity in q, k, v or the gradient of o."""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests.helpers import dev
from tests.test_gpu_attention import INF, NAN, ints, make

pytestmark = pytest.mark.gpu


def backward_groups(Tq, Tk, hq, hk, batch):
    """Workgroups of 128 rows or keys: waves take 32 from 801 on."""
    return (Tq * (hq // hk) // 128 + 2 * (Tk // 128) + 3 * batch) * hk


def gradients(q, k, v, do, cu_q=None, cu_k=None, lens=None, causal=True):
    o, saved = torch_ops.attention_forward(q, k, v, cu_q, cu_k, k_lens=lens, causal=causal)
    return torch_ops.attention_backward(do, q, k, v, o, saved, cu_q, cu_k, k_lens=lens, causal=causal)


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
