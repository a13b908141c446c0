"""Linear layers with 4-bit weights and group scales (linear_w4, w4_run).

Oracles.  In 64 bits: y = sum_g s (sum x (q - z)) + b, with a bound from the
arithmetic: a group's two fp32 chains are off by at most group 2^-24 of their
magnitudes, the groups' sum by (groups + 1) 2^-24, so y by
  (group + groups + 4) 2^-24 sum |s| |x| (q + z) + |b| 2^-24
before the rounding to the output type (half a step).  Bitwise: for integer x a
group's sums are exact, so the documented chain of fused multiply-adds can be
replayed in 64 bits, rounding to fp32 after each.
"""
import threading

import pytest
import torch

import invariant_matmul_amd as imm
from invariant_matmul_amd import torch_ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def make(M, N, K, group, dt, seed, integers=False):
    g = torch.Generator().manual_seed(seed)
    s = {"q": torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8),
         "s": ((torch.rand(N, K // group, generator=g) + 0.5) * 0.2 * max(1, K) ** -0.5).to(DT[dt]),
         "z": torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8),
         "b": torch.randn(N, generator=g)}
    s["x"] = (torch.randint(-8, 9, (M, K), generator=g).to(DT[dt]) if integers
              else torch.randn(M, K, generator=g).to(DT[dt]))
    return {k: v.to(dev()) for k, v in s.items()}


def unpacked(s):
    q = torch.empty(s["q"].shape[0], 2 * s["q"].shape[1], device=dev(), dtype=torch.float64)
    q[:, 0::2] = (s["q"] & 15).double()
    q[:, 1::2] = (s["q"] >> 4).double()
    return q


def oracle(s, group, zeros, bias):
    q, sc = unpacked(s), s["s"].double().repeat_interleave(group, 1)
    z = s["z"].double().repeat_interleave(group, 1) if zeros else torch.full_like(q, 8.0)
    x = s["x"].double()
    y = x @ (sc * (q - z)).t()
    mag = x.abs() @ (sc.abs() * (q + z)).t()
    if bias:
        y = y + s["b"].double()
    return y, mag


def check(y, s, group, zeros, bias, dt):
    want, mag = oracle(s, group, zeros, bias)
    groups = s["s"].shape[1]
    tol = mag * (group + groups + 4) * 2.0 ** -24 + want.abs() * (torch.finfo(DT[dt]).eps / 2) * (1 + 2.0 ** -20)
    tol = tol + TINY[dt] + (s["b"].double().abs() * 2.0 ** -23 if bias else 0)
    err = (y.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())


# few rows, with units of 1, 2 and 4 column blocks; the 64 x 128 tile (545 x 4112); the 128 x 256
# tile (2048 x 4096, which small tiles would fill unevenly); ragged rows and columns
SHAPES = [(2100, 4000, 256), (2048, 4096, 512), (545, 4112, 384), (5, 8216, 256), (40, 8216, 384), (9, 4120, 1152),
          (50, 4120, 1152), (29, 4096, 640), (100, 1024, 384), (1, 8, 128), (1, 4096, 4096), (3, 264, 256), (16, 1024, 1152), (17, 40, 640), (31, 520, 2048),
          (64, 256, 14336), (65, 1032, 384), (129, 136, 1024), (300, 512, 512), (1030, 264, 896)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_64_bits(shape, group, dt):
    s = make(*shape, group, dt, sum(shape) + group)
    w = torch_ops.pack_w4(s["q"], s["s"], s["z"])
    y = torch_ops.linear_w4(s["x"], w, bias=s["b"])
    assert y.dtype == DT[dt] and y.shape == shape[:2]
    check(y, s, group, True, True, dt)
    y = torch_ops.linear_w4(s["x"], torch_ops.pack_w4(s["q"], s["s"]))
    check(y, s, group, False, False, dt)


@pytest.mark.parametrize("K,group", [(32, 32), (96, 32), (160, 32), (4128, 32), (64, 64), (192, 64), (4160, 64)])
@pytest.mark.parametrize("M,N", [(1, 56), (20, 56), (90, 56), (400, 56), (30, 8216), (600, 4112), (1100, 6000)])
def test_groups_that_end_inside_a_block(K, group, M, N):
    s = make(M, N, K, group, "bf16", K + M)
    y = torch_ops.linear_w4(s["x"], torch_ops.pack_w4(s["q"], s["s"], s["z"]), bias=s["b"])
    check(y, s, group, True, True, "bf16")


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N", [(1, 72), (16, 72), (40, 72), (100, 72), (260, 72), (700, 72), (3, 8200), (33, 8200), (29, 4096), (100, 1024),
                                 (600, 4112), (1100, 6000)])
def test_bits_of_the_documented_chain(M, N, group, dt):
    K = 2176
    s = make(M, N, K, group, dt, 61, integers=True)
    y = torch_ops.linear_w4(s["x"], torch_ops.pack_w4(s["q"], s["s"], s["z"]), bias=s["b"])
    q, x = unpacked(s), s["x"].double()
    acc = torch.zeros(M, N, dtype=torch.float64, device=dev())
    for g in range(K // group):
        k = slice(g * group, (g + 1) * group)
        v = x[:, k] @ (q[:, k] - s["z"][:, g].double()[:, None]).t()  # exact integers
        acc = (acc + v * s["s"][:, g].double()).float().double()
    want = (acc.float() + s["b"]).to(DT[dt])
    assert torch.equal(y, want)


@pytest.mark.parametrize("N,K,group", [(4096, 2048, 128), (1032, 4096, 64), (264, 14336, 32), (8216, 512, 128)])
def test_rows_do_not_depend_on_the_batch(N, K, group):
    s = make(2050, N, K, group, "bf16", 67)
    w = torch_ops.pack_w4(s["q"], s["s"], s["z"])
    y = torch_ops.linear_w4(s["x"], w, bias=s["b"])
    for lo, hi in ((0, 1), (2049, 2050), (599, 600), (1, 2049), (5, 13), (3, 19), (9, 26), (0, 48), (7, 71), (100, 228), (11, 300)):
        assert torch.equal(torch_ops.linear_w4(s["x"][lo:hi], w, bias=s["b"]), y[lo:hi]), (lo, hi)


def test_every_code_and_zero_point():
    """All 16 codes against all 256 zero points: one column and group per pair."""
    K, group = 64, 32
    q = torch.arange(16).repeat_interleave(256)
    z = torch.arange(256).repeat(16)
    N = 4096
    s = {"q": (q | (q << 4)).to(torch.uint8)[:, None].expand(N, K // 2).contiguous().to(dev()),
         "s": torch.full((N, 2), 0.25, dtype=torch.float16, device=dev()),
         "z": torch.stack((z, z), 1).to(torch.uint8).to(dev())}
    x = torch.zeros(2, K, dtype=torch.float16, device=dev())
    x[0, 3], x[1, 40] = 1.0, -2.0
    y = torch_ops.linear_w4(x, torch_ops.pack_w4(s["q"], s["s"], s["z"]))
    v = 0.25 * (q - z).double().to(dev())
    assert torch.equal(y.double(), torch.stack((v, -2 * v)))


@pytest.mark.parametrize("M,N", [(12, 136), (80, 136), (300, 136), (600, 4112)])
def test_bad_rows_and_scales_stay_alone(M, N):
    s = make(M, N, 512, 64, "bf16", 71)
    y = torch_ops.linear_w4(s["x"], torch_ops.pack_w4(s["q"], s["s"], s["z"]))
    x, sc = s["x"].clone(), s["s"].clone()
    x[3, 100], x[M - 1, 511], x[5] = float("nan"), float("inf"), 0
    sc[7, 2], sc[9] = float("nan"), 0
    z = torch_ops.linear_w4(x, torch_ops.pack_w4(s["q"], sc, s["z"]))
    rows = [i for i in range(M) if i not in (3, 5, M - 1)]
    cols = [j for j in range(N) if j not in (7, 9)]
    assert torch.equal(z[rows][:, cols], y[rows][:, cols])
    assert not torch.isfinite(z[3]).any() and not torch.isfinite(z[M - 1][cols]).any()
    assert z[:, 7].isnan().all() and (z[rows, 9] == 0).all() and (z[5, cols] == 0).all()


def test_views_shapes_and_empty():
    s = make(24, 72, 256, 64, "f16", 73)
    w = torch_ops.pack_w4(s["q"], s["s"], s["z"])
    y = torch_ops.linear_w4(s["x"], w)
    z = torch_ops.linear_w4(s["x"].view(2, 3, 4, 256), w)
    assert z.shape == (2, 3, 4, 72) and torch.equal(z.view(24, 72), y)
    assert torch.equal(torch_ops.linear_w4(s["x"][5], w), y[5])
    wide = torch.zeros(24, 301, dtype=torch.float16, device=dev())
    wide[:, 1:257] = s["x"]
    assert torch.equal(torch_ops.linear_w4(wide[:, 1:257], w), y)
    flat = torch.zeros(24 * 256 + 4, dtype=torch.float16, device=dev())
    flat[4:] = s["x"].reshape(-1)
    assert torch.equal(torch_ops.linear_w4(flat[4:].view(24, 256), w), y)
    qt, st, zt = (t.t().contiguous().t() for t in (s["q"], s["s"], s["z"]))
    w2 = torch_ops.pack_w4(qt, st, zt)
    assert torch.equal(w2.packed, w.packed)
    assert torch_ops.linear_w4(s["x"][:0], w).shape == (0, 72)
    assert torch.equal(torch_ops.linear_w4(s["x"], w.to(dev())), y)


@pytest.mark.parametrize("M,N", [(1, 1032), (24, 1032), (200, 1032), (600, 4112)])
def test_streams_graphs_and_rows_behind(M, N):
    s = make(M, N, 1024, 128, "bf16", 79)
    w = torch_ops.pack_w4(s["q"], s["s"], s["z"])
    want = torch_ops.linear_w4(s["x"], w, bias=s["b"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = torch_ops.linear_w4(s["x"], w, bias=s["b"])
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = torch_ops.linear_w4(s["x"], w, bias=s["b"])
    for _ in range(4):
        out.fill_(0)
        torch_ops.linear_w4(s["x"] * 2, w)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    buf = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=dev())
    plan = imm.w4_plan(M, N, 1024, "bf16", 128)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=dev())
    imm.w4_run(plan, s["x"], w.packed, buf[:M], bias=s["b"], workspace=ws)
    assert torch.equal(buf[:M], want) and (buf[M:] == 7).all()


@pytest.mark.parametrize("M", [1, 20, 800])
def test_weights_past_32_bits(M):
    """A weight of more than 2^32 dwords and bytes: its last columns against their own product."""
    N, K = 262144 + 16, 131072
    g = torch.Generator(device=dev()).manual_seed(97)
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device=dev())
    sc = (torch.rand(N, K // 128, generator=g, device=dev()) * K ** -0.5).bfloat16()
    x = torch.randn(M, K, generator=g, device=dev()).bfloat16()
    y = torch_ops.linear_w4(x, torch_ops.pack_w4(q, sc))
    for lo, hi in ((0, 64), (131072, 131136), (N - 64, N)):
        assert torch.equal(y[:, lo:hi], torch_ops.linear_w4(x, torch_ops.pack_w4(q[lo:hi], sc[lo:hi])))


def test_norm_then_product():
    """What a serving layer runs: norm with the residual, then the 4-bit product."""
    s = make(33, 520, 1024, 128, "bf16", 83)
    g = torch.Generator().manual_seed(84)
    r = torch.randn(33, 1024, generator=g).bfloat16().to(dev())
    nw = (1 + 0.1 * torch.randn(1024, generator=g)).bfloat16().to(dev())
    w = torch_ops.pack_w4(s["q"], s["s"], s["z"])
    h, stream = torch_ops.rms_norm(s["x"], nw, 1e-6, residual=r)
    y = torch_ops.linear_w4(h, w, bias=s["b"])
    check(y, {**s, "x": h}, 128, True, True, "bf16")
    for i in (0, 20, 32):
        h1, _ = torch_ops.rms_norm(s["x"][i:i + 1], nw, 1e-6, residual=r[i:i + 1])
        assert torch.equal(torch_ops.linear_w4(h1, w, bias=s["b"])[0], y[i])


def test_threads_on_their_own_streams():
    """Four host threads, a batch size each, through norm, fp8 and 4-bit products at once."""
    N, K = 4112, 1024
    g = torch.Generator(device=dev()).manual_seed(101)
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device=dev())
    w4 = torch_ops.pack_w4(q, (torch.rand(N, K // 64, generator=g, device=dev()) * 0.01).bfloat16())
    w8, s8 = torch_ops.quantize_rows(torch.randn(N, K, generator=g, device=dev()).bfloat16())
    nw = torch.rand(K, generator=g, device=dev()).bfloat16()
    xs = [torch.randn(m, K, generator=g, device=dev()).bfloat16() for m in (1, 20, 600, 1100)]

    def run(x):
        h, stream = torch_ops.rms_norm(x, nw, 1e-6, residual=x)
        r8, sx = torch_ops.quantize_rows(h)
        return torch_ops.linear_w4(h, w4), torch_ops.linear_f8(r8, sx, w8, s8), stream

    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    wrong, done = [], []

    def worker(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for k in range(12):
                got = run(xs[i])
                if k % 4 == 3:
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        wrong.append((i, k))
            torch.cuda.current_stream().synchronize()
        done.append(i)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted(done) == [0, 1, 2, 3] and not wrong


def test_refusals_on_the_gpu():
    s = make(4, 64, 256, 64, "f16", 89)
    w = torch_ops.pack_w4(s["q"], s["s"], s["z"])
    for call in (lambda: torch_ops.linear_w4(s["x"].bfloat16(), w),
                 lambda: torch_ops.linear_w4(s["x"][:, :128], w),
                 lambda: torch_ops.linear_w4(s["x"].cpu(), w),
                 lambda: torch_ops.linear_w4(s["x"], w.to("cpu")),
                 lambda: torch_ops.linear_w4(s["x"], w, bias=s["b"][:3]),
                 lambda: torch_ops.linear_w4(s["x"].clone().requires_grad_(), w),
                 lambda: torch_ops.pack_w4(s["q"].to(torch.int8), s["s"]),
                 lambda: torch_ops.pack_w4(s["q"], s["s"].float()),
                 lambda: torch_ops.pack_w4(s["q"], s["s"][:, :3]),
                 lambda: torch_ops.pack_w4(s["q"], s["s"][:, :1]),
                 lambda: torch_ops.pack_w4(s["q"], s["s"], s["z"][:, :2]),
                 lambda: torch_ops.pack_w4(s["q"], s["s"], s["z"].half()),
                 lambda: torch_ops.pack_w4(s["q"][:60], s["s"][:60])):
        with pytest.raises(ValueError):
            call()
    L, p = imm.lib(), imm.w4_plan(4, 64, 256, "f16", 64)
    y = torch.empty(4, 64, dtype=torch.float16, device=dev())
    pinned = torch.zeros(4, 256, dtype=torch.float16).pin_memory()
    assert L.w4_run(p.handle, pinned.data_ptr(), w.packed.data_ptr(), None, y.data_ptr(),
                    None, 0, None) == 1
    big = imm.w4_plan(1 << 24, 64, 256, "f16", 64)  # rows past any allocation here
    assert L.w4_run(big.handle, s["x"].data_ptr(), w.packed.data_ptr(), None, y.data_ptr(),
                    w.packed.data_ptr(), big.workspace_bytes, None) == 1
