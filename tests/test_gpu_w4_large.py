"""A 4-bit weight with more scale words than a launch has threads (2^32)."""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu


def test_more_scale_words_than_one_launch_has_threads():
    """2^20 + 16 outputs x 4096 groups: the last outputs and groups against their own product."""
    N, K, group = (1 << 20) + 16, 1 << 17, 32
    groups = K // group
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 190 << 30:
        pytest.skip("needs 190 GiB of device memory")
    g = torch.Generator(device=dev()).manual_seed(103)
    q = torch.empty(N, K // 2, dtype=torch.uint8, device=dev())
    for lo in range(0, N, 1 << 16):
        part = q[lo:lo + (1 << 16)]
        part.copy_(torch.randint(0, 256, part.shape, generator=g, dtype=torch.uint8, device=dev()))
    sc = torch.empty(N, groups, dtype=torch.bfloat16, device=dev()).uniform_(0.5, 1.5, generator=g)
    x = torch.randn(2, K, generator=g, device=dev()).bfloat16()
    w = torch_ops.pack_w4(q, sc)
    y = torch_ops.linear_w4(x, w)
    for lo, hi in ((0, 64), (N // 2, N // 2 + 64), (N - 64, N)):
        assert torch.equal(y[:, lo:hi], torch_ops.linear_w4(x, torch_ops.pack_w4(q[lo:hi], sc[lo:hi])))
    # the words behind the blocks: [groups, N rounded up to 16], the scale's bits and -8
    np = (N + 15) // 16 * 16
    words = w.packed[w.packed.numel() - 4 * groups * np:].view(torch.int16).view(groups, np, 2)
    for gr in (0, groups // 2, groups - 1):
        assert torch.equal(words[gr, :N, 0], sc[:, gr].contiguous().view(torch.int16))
        assert (words[gr, :N, 1] == torch.tensor(-8.0).bfloat16().view(torch.int16).to(dev())).all()
    del q, sc, w, words
    torch.cuda.empty_cache()
