"""The kernels of few and of many rows where the reference of a row's logits is set again and again, within
chunks of 256 keys and from chunk to chunk: o, lse, o_low and the gradients have the same bits."""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests.helpers import dev
from tests.test_gpu_attention import ints, make, starts
from tests.test_gpu_attention_kernels import groups, takes_few

pytestmark = pytest.mark.gpu


def spread(q, k, room, how):
    """Logits whose steps' maxima rise by more than 8 (binary) at many steps."""
    if how == "wide":  # a standard deviation of 19
        q.mul_(8.0)
    else:  # growing along the keys, by 3 a step of 64, or by 12 a chunk
        at = torch.arange(k.shape[0], device=dev()) % room
        q[:, :, 0] = 2.0
        k[:, :, 0] = (0.25 * at if how == "steps" else 64.0 * (at // 256)).to(k.dtype)[:, None]


@pytest.mark.parametrize("how", ["wide", "steps", "chunks"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 1, 64), (3, 3, 96)])
def test_few_and_many_rows(heads, dt, how):
    hq, hk, D = heads
    count, room, new = 100, 1500, 3
    q, k, v, do = make(count * new, count * room, hq, hk, D, dt, 50 + hq)
    spread(q, k, room, how)
    lens = torch.randint(900, room + 1, (count,), generator=torch.Generator().manual_seed(51)).int().to(dev())
    cu_q = starts([new] * count)
    cu_k = cu_q // new * room
    assert takes_few(q, k, count, new) and not takes_few(q, k, count, None)
    results = []
    for max_q in (new, None):
        o, saved = torch_ops.attention_forward(q, k, v, cu_q, cu_k, k_lens=lens, max_q=max_q)
        results.append((o, *saved, *torch_ops.attention_backward(do, q, k, v, o, saved, cu_q, cu_k, k_lens=lens)))
    for few, many, name in zip(*results, ("o", "lse", "o_low", "dq", "dk", "dv")):
        assert torch.isfinite(few).all() and torch.equal(few, many), (name, int((few != many).sum()))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_sums_that_a_new_reference_scales(dt):
    # Within a chunk: a step at 2^-8.6, one with eight keys at 2^-4, one with a key at 1, which sets the reference
    # again.  The row's sum is 1.7, half of it scaled by an odd factor, and its logarithm as small: a product
    # rounded before its sum in one kernel and not in the other is a different lse in one row of ten.
    count, room, new, hq, D = 100, 1500, 3, 8, 128
    q, k, v, _ = make(count * new, room, hq, 1, D, dt, 53)
    binary = torch.full((room,), -60.0)
    binary[:64], binary[70:78], binary[150] = -8.6, -4.0, 0.0
    q[:, :, 2:] = 0
    q[:, :, 0], q[:, :, 1] = 1.0, 0.05 * q[:, :, 1]
    k[:, 0, 0] = (binary * 0.6931 * D ** 0.5).to(k.dtype).to(dev())
    k[:, 0, 1] = k[:, 0, 1] * (0.5 * D ** 0.5)
    k, v = k.repeat(count, 1, 1), v.repeat(count, 1, 1)
    cu_q = starts([new] * count)
    cu_k = cu_q // new * room
    assert takes_few(q, k, count, new) and not takes_few(q, k, count, None)
    few, a = torch_ops.attention_forward(q, k, v, cu_q, cu_k, max_q=new)
    many, b = torch_ops.attention_forward(q, k, v, cu_q, cu_k)
    assert (a.lse.abs() < 2).all() and a.lse.unique().numel() > 500
    assert torch.equal(few, many) and torch.equal(a.lse, b.lse) and torch.equal(a.o_low, b.o_low), int((a.lse != b.lse).sum())


@pytest.mark.parametrize("how", ["wide", "steps", "chunks"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_pieces_tokens_and_rows_a_wave(dt, how):
    n, hk, D = 1100, 60, 128
    q, k, v, _ = make(n, n, hk, hk, D, dt, 52)
    spread(q, k, n, how)
    assert groups(q, k, 1) > 512
    whole, saved = torch_ops.attention_forward(q, k, v)
    few_heads = q[:, :2], k[:, :2], v[:, :2]
    assert groups(*few_heads[:2], 1) <= 512
    o, s = torch_ops.attention_forward(*few_heads)
    assert all(torch.equal(a, b[:, :2]) for a, b in zip((o, *s), (whole, *saved)))
    room = 9000
    cache_k, cache_v = (torch.zeros(room, 2, D, dtype=k.dtype, device=dev()) for _ in "kv")
    cache_k[:n], cache_v[:n] = k[:, :2], v[:, :2]
    for lo, hi in [(t, t + 1) for t in range(0, n, 37)] + [(100, 107), (500, 540), (1090, n)]:
        assert takes_few(q[lo:hi, :2], cache_k, 1, hi - lo)
        o, s = torch_ops.attention_forward(q[lo:hi, :2], cache_k, cache_v, ints([0, hi - lo]), ints([0, room]), k_lens=ints([hi]),
                                           max_q=hi - lo)
        for a, b, name in zip((o, *s), (whole, *saved), ("o", "lse", "o_low")):
            assert torch.equal(a, b[lo:hi, :2]), (name, lo, hi)
