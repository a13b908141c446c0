"""The product of fp8 rows with their scales (linear_f8, gemm_run_scaled).

Two oracles.  Bitwise: the fp32 output of the unscaled product (checked against
the CPU oracle elsewhere) scaled, biased and rounded by separate fp32 torch
operations, in the documented order.  In 64 bits: the formula, with the fp32
accumulation bound K 2^-24 sum |a||b| (times the scales), what the fp8 step's
8-product window may drop (tests/helpers.py: at most min(|a b|, 2^(E - 13)) a
product, so at most 2^-12 of the group's largest and 2^-12 sum |a||b| in
all), three fp32 roundings and half a step of the output type.
"""
import pytest
import torch

import invariant_matmul_amd as imm
from invariant_matmul_amd import torch_ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
OUT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make(M, N, K, dt, seed):
    g = torch.Generator().manual_seed(seed)
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    s = {"x": x.to(F8[dt]), "w": w.to(F8[dt]), "sx": torch.rand(M, generator=g) + 0.5,
         "sw": (torch.rand(N, generator=g) + 0.5) * max(1, K) ** -0.5, "b": torch.randn(N, generator=g)}
    return {k: v.to(dev()) for k, v in s.items()}


def unscaled(s, wide=False):
    """The fp32 sums of the unscaled single pass."""
    M, K = s["x"].shape
    N = s["w"].shape[0]
    flags = imm.PLAN_TILE_BY_M | imm.PLAN_B_TRANSPOSED | (imm.PLAN_FP8_FP32_ACCUM if wide else 0)
    plan = imm.gemm_plan_ex2(M, N, K, s["x"].dtype, "f32", flags=flags)
    C = torch.empty(M, N, device=dev())
    imm.gemm_run(plan, s["x"], s["w"], C)
    return C


def scaled(C, s, bias, out):
    y = (C * s["sx"][:, None]) * s["sw"]
    return (y + s["b"] if bias else y).to(OUT[out])


# long and short K, small and large B; ragged rows, every tile of the plans
SHAPES = [(1, 256, 256), (7, 16, 16), (33, 272, 1040), (64, 512, 4096), (100, 4096, 4096), (257, 1040, 528),
          (300, 6144, 256), (513, 2048, 2048), (1, 4096, 14336), (40, 1024, 8192), (1, 16, 1008),
          (16, 4112, 1040), (17, 4096, 144), (31, 8208, 528), (64, 8208, 2064), (65, 4112, 1536), (250, 2064, 640),
          (64, 4096, 528), (60, 2000, 2000), (300, 240, 2064), (2051, 4096, 1024), (2112, 4096, 2048), (4097, 4096, 4096)]


@pytest.mark.parametrize("dt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("out,bias,wide", [("bf16", True, False), ("f16", False, False),
                                           ("f32", True, False), ("f32", False, True),
                                           ("bf16", True, True)])
def test_scales_bias_and_rounding_are_those_of_the_definition(shape, dt, out, bias, wide):
    s = make(*shape, dt, sum(shape))
    y = torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"] if bias else None,
                            out_dtype=OUT[out], fp32_accum=wide)
    assert torch.equal(y, scaled(unscaled(s, wide), s, bias, out))


@pytest.mark.parametrize("dt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("shape", [(5, 48, 16), (65, 400, 2000), (130, 272, 4096)])
def test_against_64_bits(shape, dt, wide):
    M, N, K = shape
    s = make(M, N, K, dt, 31)
    y = torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"], fp32_accum=wide)
    a, b = s["x"].double() * s["sx"].double()[:, None], s["w"].double() * s["sw"].double()[:, None]
    want = a @ b.t() + s["b"].double()
    mag = a.abs() @ b.abs().t()
    tol = mag * (K * 2.0 ** -24 + (0 if wide else 2.0 ** -12)) + (mag + s["b"].abs()) * 2.0 ** -22
    tol = tol + want.abs() * 2.0 ** -8
    err = (y.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())


def test_rows_behind_whole_rounds_of_tiles():
    """2048 rows on tiles and 3 on the kernel of few rows, into their places and no further."""
    s = make(2051, 4096, 4096, "e4m3", 39)
    y = torch.full((2053, 4096), 7.0, dtype=torch.float32, device=dev())
    plan = imm.gemm_plan_ex2(2051, 4096, 4096, "e4m3", "f32", flags=imm.PLAN_B_TRANSPOSED | imm.PLAN_TILE_BY_M)
    imm.gemm_run_scaled(plan, s["x"], s["w"], s["sx"], s["sw"], y[:2051], bias=s["b"])
    assert (y[2051:] == 7).all()
    assert torch.equal(y[:2051], torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"],
                                                     out_dtype=torch.float32))
    for lo, hi in ((2040, 2051), (2048, 2051), (1000, 1100)):
        assert torch.equal(torch_ops.linear_f8(s["x"][lo:hi], s["sx"][lo:hi], s["w"], s["sw"], bias=s["b"],
                                               out_dtype=torch.float32), y[lo:hi])


@pytest.mark.parametrize("N,K", [(4096, 4096), (1024, 4096), (6144, 512)])
def test_rows_do_not_depend_on_the_batch(N, K):
    s = make(700, N, K, "e4m3", 37)
    y = torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"])
    for lo, hi in ((0, 1), (13, 29), (5, 30), (3, 67), (100, 228), (500, 700), (699, 700)):
        p = torch_ops.linear_f8(s["x"][lo:hi], s["sx"][lo:hi], s["w"], s["sw"], bias=s["b"])
        assert torch.equal(p, y[lo:hi]), (lo, hi)


def test_bad_rows_and_scales_stay_alone():
    s = make(20, 512, 512, "e4m3", 41)
    y = torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"])
    x, sx, sw = s["x"].clone(), s["sx"].clone(), s["sw"].clone()
    x.view(torch.uint8)[3, 5] = 0x7f            # NaN
    sx[7], sx[9], sw[11], sw[12] = float("inf"), float("nan"), 0.0, float("nan")
    z = torch_ops.linear_f8(x, sx, s["w"], sw)
    rows = [i for i in range(20) if i not in (3, 7, 9)]
    cols = [j for j in range(512) if j not in (11, 12)]
    assert torch.equal(z[rows][:, cols], y[rows][:, cols])
    assert z[3].isnan().all() and z[9].isnan().all() and z[:, 12].isnan().all()
    assert not torch.isfinite(z[7, cols]).any() and (z[rows, 11] == 0).all()


def test_shapes_views_and_empty():
    s = make(24, 64, 128, "e5m2", 43)
    y = torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"])
    z = torch_ops.linear_f8(s["x"].view(2, 12, 128), s["sx"].view(2, 12), s["w"], s["sw"])
    assert z.shape == (2, 12, 64) and torch.equal(z.view(24, 64), y)
    one = torch_ops.linear_f8(s["x"][4], s["sx"][4], s["w"], s["sw"])
    assert one.shape == (64,) and torch.equal(one, y[4])
    wide = torch.zeros(24, 160, dtype=torch.uint8, device=dev())
    wide[:, 16:144] = s["x"].view(torch.uint8)
    view = wide.view(F8["e5m2"])[:, 16:144]
    assert torch.equal(torch_ops.linear_f8(view, s["sx"], s["w"], s["sw"]), y)
    wt = s["w"].view(torch.uint8).t().contiguous().t().view(F8["e5m2"])
    sw2 = torch.stack((s["sw"], s["sw"]), 1)[:, 0]
    assert torch.equal(torch_ops.linear_f8(s["x"], s["sx"], wt, sw2), y)
    assert torch_ops.linear_f8(s["x"][:0], s["sx"][:0], s["w"], s["sw"]).shape == (0, 64)
    k0 = torch_ops.linear_f8(s["x"][:, :0], s["sx"], s["w"][:, :0], s["sw"], bias=s["b"])
    assert torch.equal(k0, s["b"].bfloat16().expand(24, 64))
    assert torch.equal(torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"].half()),
                       torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"].half().float()))


@pytest.mark.parametrize("shape", [(16, 6144, 1024), (5, 512, 4096), (300, 1024, 1024), (50, 8208, 528), (700, 4096, 512)])
def test_streams_graphs_and_rows_behind(shape):
    M, N, K = shape
    s = make(M, N, K, "e4m3", 47)
    want = torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"])
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"])
    for _ in range(4):
        out.fill_(0)
        torch_ops.linear_f8(s["x"], s["sx"], s["w"], s["sw"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    buf = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=dev())
    plan = imm.gemm_plan_ex2(M, N, K, "e4m3", "bf16", flags=imm.PLAN_B_TRANSPOSED | imm.PLAN_TILE_BY_M)
    imm.gemm_run_scaled(plan, s["x"], s["w"], s["sx"], s["sw"], buf[:M], bias=s["b"])
    assert (buf[M:] == 7).all()


@pytest.mark.parametrize("M", [1, 50, 600])
def test_weights_past_32_bits(M):
    """A weight of more than 2^32 bytes: its last columns against their own product."""
    N, K = (1 << 19) + 16, 8208
    g = torch.Generator(device=dev()).manual_seed(97)
    w = torch.randint(0, 0x78, (N, K), generator=g, dtype=torch.uint8, device=dev()).view(torch.float8_e4m3fn)
    x = torch.randn(M, K, generator=g, device=dev()).to(torch.float8_e4m3fn)
    sx, sw = torch.rand(M, generator=g, device=dev()), torch.rand(N, generator=g, device=dev()) * 2.0 ** -12
    y = torch_ops.linear_f8(x, sx, w, sw)
    for lo, hi in ((0, 64), (1 << 18, (1 << 18) + 64), (N - 64, N)):
        assert torch.equal(y[:, lo:hi], torch_ops.linear_f8(x, sx, w[lo:hi], sw[lo:hi]))


def test_norm_quant_product_together():
    """What a serving layer runs: norm with the residual to fp8 rows, then the product."""
    g = torch.Generator().manual_seed(53)
    K, N = 1024, 2048
    x = torch.randn(37, K, generator=g).bfloat16().to(dev())
    r = torch.randn(37, K, generator=g).bfloat16().to(dev())
    nw = (1 + 0.1 * torch.randn(K, generator=g)).bfloat16().to(dev())
    W = (torch.randn(N, K, generator=g) * K ** -0.5).bfloat16().to(dev())
    wq, ws = torch_ops.quantize_rows(W)
    q, s, h = torch_ops.rms_norm_quant(x, nw, 1e-6, residual=r)
    y = torch_ops.linear_f8(q, s, wq, ws)
    h64 = h.double()
    t = h64 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + 1e-6) * nw.double()
    want = t @ W.double().t()
    # an e4m3 value is off by at most 2^-4 of itself (or half the smallest step, 2^-10 of its scale)
    at, aw = t.abs(), W.double().abs()
    et = at * 2.0 ** -4 + 2.0 ** -10 * s.double()[:, None]
    ew = aw * 2.0 ** -4 + 2.0 ** -10 * ws.double()[:, None]
    tol = et @ aw.t() + at @ ew.t() + et @ ew.t() + 2.0 ** -11 * (at @ aw.t()) + want.abs() * 2.0 ** -8
    assert ((y.double() - want).abs() <= tol).all()
    rel = float((y.double() - want).norm() / want.norm())
    assert rel < 2.0 ** -4  # each operand's roundings alone stay under that
    for i in (0, 11, 36):  # the whole run, one row at a time
        q1, s1, _ = torch_ops.rms_norm_quant(x[i:i + 1], nw, 1e-6, residual=r[i:i + 1])
        assert torch.equal(torch_ops.linear_f8(q1, s1, wq, ws)[0], y[i])


def test_refusals_on_the_gpu():
    s = make(4, 64, 128, "e4m3", 59)
    f = torch_ops.linear_f8
    for call in (lambda: f(s["x"].half(), s["sx"], s["w"], s["sw"]),
                 lambda: f(s["x"], s["sx"], s["w"].to(F8["e5m2"]), s["sw"]),
                 lambda: f(s["x"], s["sx"][:3], s["w"], s["sw"]),
                 lambda: f(s["x"], s["sx"].half(), s["w"], s["sw"]),
                 lambda: f(s["x"], s["sx"], s["w"], s["sw"][:5]),
                 lambda: f(s["x"], s["sx"], s["w"][:40], s["sw"][:40]),
                 lambda: f(s["x"][:, :120], s["sx"], s["w"][:, :120], s["sw"]),
                 lambda: f(s["x"], s["sx"], s["w"], s["sw"], bias=s["b"][:3]),
                 lambda: f(s["x"], s["sx"], s["w"], s["sw"].cpu()),
                 lambda: f(s["x"], s["sx"], s["w"], s["sw"], out_dtype=torch.float64),
                 lambda: f(s["x"], s["sx"].clone().requires_grad_(), s["w"], s["sw"])):
        with pytest.raises(ValueError):
            call()
    C = torch.empty(4, 64, device=dev())
    for flags, dt in ((0, "e4m3"), (imm.PLAN_B_TRANSPOSED, "f16")):
        plan = imm.gemm_plan_ex2(4, 64, 128, dt, "f32", flags=flags)
        assert imm.lib().gemm_run_scaled(plan.handle, s["x"].data_ptr(), s["w"].data_ptr(), s["sx"].data_ptr(),
                                         s["sw"].data_ptr(), None, C.data_ptr(), None) == 2
