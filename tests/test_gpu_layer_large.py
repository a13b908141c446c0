"""Batches whose rows pass 2^32 bytes, and the rows around the limits where a call is cut
into several launches or changes its kernel: each against its own small batch."""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GiB of device memory")
    yield
    torch.cuda.empty_cache()


def bits(t):
    return t.view(torch.uint8)


def test_w4_rows_at_the_limit_of_the_tiles():
    """2^28 sums of x: one row fewer and the tiles take the product, from there on the kernel
    of few rows does, in two launches (17 column groups on 2^21 workgroups)."""
    M, N, K, group = 4194341, 520, 2048, 32
    g = torch.Generator(device=dev()).manual_seed(107)
    x = torch.empty(M, K, dtype=torch.bfloat16, device=dev())
    for lo in range(0, M, 1 << 19):
        part = x[lo:lo + (1 << 19)]
        part.copy_(torch.randn(part.shape, generator=g, device=dev()))
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device=dev())
    w = torch_ops.pack_w4(q, (torch.rand(N, K // group, generator=g, device=dev()) * 0.01).bfloat16())
    y = torch_ops.linear_w4(x, w)
    cut = (1 << 21) // 17 * 32
    for lo in (0, cut - 40, cut, M - 70, 1 << 20):
        assert torch.equal(y[lo:lo + 70], torch_ops.linear_w4(x[lo:lo + 70], w)), lo
    tiles = torch_ops.linear_w4(x[:4194000], w)
    assert torch.equal(tiles, y[:4194000])


def test_f8_rows_past_32_bits():
    M, N, K = 600000, 48, 8192
    g = torch.Generator(device=dev()).manual_seed(109)
    x = torch.randint(0, 0x70, (M, K), generator=g, dtype=torch.uint8, device=dev()).view(torch.float8_e4m3fn)
    w, ws = torch_ops.quantize_rows(torch.randn(N, K, generator=g, device=dev()).bfloat16())
    s = torch.rand(M, generator=g, device=dev()) * 2.0 ** -6
    for wide in (False, True):
        y = torch_ops.linear_f8(x, s, w, ws, fp32_accum=wide)
        for lo in (0, (1 << 32) // K - 30, M // 2, M - 65):
            part = torch_ops.linear_f8(x[lo:lo + 65], s[lo:lo + 65], w, ws, fp32_accum=wide)
            assert torch.equal(y[lo:lo + 65], part), (wide, lo)


def test_norm_rows_past_32_bits():
    rows, cols = (1 << 19) + 77, 8200
    g = torch.Generator(device=dev()).manual_seed(113)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev())
    for lo in range(0, rows, 1 << 16):
        part = x[lo:lo + (1 << 16)]
        part.copy_(torch.randn(part.shape, generator=g, device=dev()))
    w = torch.rand(cols, generator=g, device=dev()).bfloat16()
    y, h, rstd = torch_ops.rms_norm_forward(x, w, residual=x)
    dx, dw = torch_ops.rms_norm_backward(y, h, w, rstd, x)
    part = 64
    for lo in (0, (1 << 31) // cols - 30, (1 << 32) // cols - 30, rows - part):
        s = slice(lo, lo + part)
        y2, h2, r2 = torch_ops.rms_norm_forward(x[s], w, residual=x[s])
        assert torch.equal(y[s], y2) and torch.equal(h[s], h2) and torch.equal(rstd[s], r2), lo
        assert torch.equal(dx[s], torch_ops.rms_norm_backward(y[s], h[s], w, rstd[s], x[s])[0]), lo
    # dw = sum over the rows of dy n, in 64 bits.  A workgroup (one of 512) adds its 1025
    # rows, then 512 parts in at most 17 steps, on terms of three fp32 roundings
    want, mag = torch.zeros(cols, dtype=torch.float64, device=dev()), torch.zeros(cols, dtype=torch.float64, device=dev())
    for lo in range(0, rows, 1 << 14):
        t = y[lo:lo + (1 << 14)].double() * (h[lo:lo + (1 << 14)].double() * rstd[lo:lo + (1 << 14), None].double())
        want, mag = want + t.sum(0), mag + t.abs().sum(0)
    assert ((dw.double() - want).abs() <= want.abs() * 2.0 ** -8 + mag * 1050 * 2.0 ** -24).all()
    del y, h, dx


def test_quantised_rows_past_32_bits():
    rows, cols = (1 << 19) + 77, 8208
    g = torch.Generator(device=dev()).manual_seed(127)
    x = torch.empty(rows, cols, dtype=torch.float16, device=dev())
    for lo in range(0, rows, 1 << 16):
        part = x[lo:lo + (1 << 16)]
        part.copy_(torch.randn(part.shape, generator=g, device=dev()))
    w = torch.rand(cols, generator=g, device=dev()).half()
    q, s = torch_ops.quantize_rows(x)
    n, ns = torch_ops.rms_norm_quant(x, w)
    for lo in (0, (1 << 31) // cols - 30, (1 << 32) // cols - 30, rows - 64):
        r = slice(lo, lo + 64)
        q2, s2 = torch_ops.quantize_rows(x[r])
        n2, ns2 = torch_ops.rms_norm_quant(x[r], w)
        assert torch.equal(bits(q[r]), bits(q2)) and torch.equal(s[r], s2), lo
        assert torch.equal(bits(n[r]), bits(n2)) and torch.equal(ns[r], ns2), lo
