"""The row norm, its fp8 form, its backward pass and the fp8 quantisation of rows.

The oracle is the formula in 64 bits.  Tolerances, derived from the kernels'
arithmetic: fp32 sums of a row run over at most 32 values in a thread, 6
halvings in a wave and 16 waves, so a sum of magnitudes is off by at most
54 * 2^-24 of itself; with the square root, the division and the few products
after it, every fp32 value is within 2^-18 of the sum of its terms'
magnitudes.  Then comes one rounding: half a step, eps / 2 of the value (or
half the smallest subnormal).
"""
import numpy as np
import pytest
import torch

import invariant_matmul_amd as imm
from invariant_matmul_amd import torch_ops
from tests.helpers import dev

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
      "e5m2": torch.float8_e5m2}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F32 = 2.0 ** -18
EPS = 1e-5


def half(dt):
    return torch.finfo(DT[dt]).eps / 2


def make(rows, cols, dt, seed, names="xrw"):
    g = torch.Generator().manual_seed(seed)
    out = {}
    for n in names:
        shape = (cols,) if n == "w" else (rows, cols)
        v = torch.randn(shape, generator=g)
        out[n] = (1 + 0.3 * v if n == "w" else v * 1.5).to(DT[dt]).to(dev())
    return out


def close(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).max())} of the bound"


def reference(x, w, r, eps=EPS):
    h = x.double() if r is None else (x.float() + r.float()).to(x.dtype).double()
    rstd = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    t = h * rstd if w is None else h * rstd * w.double()
    return h, rstd, t


# every thread layout (cols / 8 = 1 .. 4096 vectors), with full and partial last vectors
COLS = [8, 64, 120, 128, 136, 256, 264, 512, 520, 1024, 1040, 2048, 2056, 4096, 4104, 8192, 8200,
        14336, 16384, 16392, 32768]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_matches_the_formula(cols, dt, residual):
    rows = 19 if cols <= 2048 else 5
    s = make(rows, cols, dt, cols)
    r = s["r"] if residual else None
    got = torch_ops.rms_norm(s["x"], s["w"], EPS, residual=r)
    h, _, t = reference(s["x"], s["w"], r)
    y = got[0] if residual else got
    close(y, t, t.abs() * (half(dt) + F32) + TINY[dt], "y")
    if residual:
        assert torch.equal(got[1], s["x"] + s["r"])  # the stream, bit for bit


@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
@pytest.mark.parametrize("cols", [16, 128, 256, 528, 1040, 2048, 4096, 8192, 14336, 32768])
@pytest.mark.parametrize("residual", [False, True])
def test_quantised_norm_matches_the_formula(cols, out, residual):
    dt = "bf16"
    s = make(9, cols, dt, 100 + cols)
    r = s["r"] if residual else None
    got = torch_ops.rms_norm_quant(s["x"], s["w"], EPS, residual=r, dtype=DT[out])
    q, scale = got[:2]
    _, _, t = reference(s["x"], s["w"], r)
    assert q.dtype == DT[out] and scale.dtype == torch.float32 and scale.shape == (9,)
    close(scale, t.abs().amax(1) / FMAX[out], scale.double() * F32, "scale")
    back = q.double() * scale.double()[:, None]
    close(back, t, t.abs() * (half(out) + 2 * F32) + TINY[out] * scale.double()[:, None], "q scale")
    assert torch.equal(q.float().abs().amax(1), torch.full((9,), FMAX[out], device=q.device))
    if residual:
        assert torch.equal(got[2], s["x"] + s["r"])


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("out", ["e4m3", "e5m2"])
@pytest.mark.parametrize("cols", [16, 144, 4096, 16384])
def test_quantize_rows(cols, out, dt):
    x = make(7, cols, dt, 7, "x")["x"]
    x[3] = 0
    q, scale = torch_ops.quantize_rows(x, DT[out])
    want = x.double().abs().amax(1) / FMAX[out]
    want[3] = 2.0 ** -120
    close(scale, want, want * F32, "scale")
    close(q.double() * scale.double()[:, None], x.double(),
          x.double().abs() * (half(out) + 2 * F32) + TINY[out] * scale.double()[:, None], "q scale")
    assert (q[3].float() == 0).all()


def grads(s, rstd, h, dh):
    n = h * rstd
    g = s["d"].double() * (s["w"].double() if "w" in s else 1.0)
    dot = (g * n).mean(1, keepdim=True)
    dx = rstd * (g - n * dot)
    bound = rstd * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, bound = dx + dh.double(), bound + dh.double().abs()
    return dx, bound, (s["d"].double() * n).sum(0), (s["d"].double() * n).abs().sum(0)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 128), (1000, 136), (17, 264), (515, 512), (70, 1040),
                                       (33, 2048), (700, 4096), (5, 8200), (3, 16384), (2, 32768)])
def test_backward_matches_the_formula(rows, cols, dt):
    s = make(rows, cols, dt, rows + cols, "xrwde")
    y, h, rstd = torch_ops.rms_norm_forward(s["x"], s["w"], EPS, residual=s["r"])
    h64, rstd64, _ = reference(s["x"], s["w"], s["r"])
    close(rstd, rstd64[:, 0], rstd64[:, 0] * F32, "rstd")
    for dh in (s["e"], None):
        dx, dw = torch_ops.rms_norm_backward(s["d"], h, s["w"], rstd, dh)
        want, bound, wdw, bdw = grads(s, rstd64, h64, dh)
        close(dx, want, want.abs() * half(dt) + bound * F32 + TINY[dt], "dx")
        # a column adds its rows in at most rows + 32 steps
        close(dw, wdw, wdw.abs() * half(dt) + bdw * (rows + 96) * 2.0 ** -24 + TINY[dt], "dw")
        again = torch_ops.rms_norm_backward(s["d"], h, s["w"], rstd, dh)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_gradients_against_differences():
    """Directional derivatives of the 64-bit forward formula by differences."""
    rows, cols, dt = 11, 272, "bf16"
    s = make(rows, cols, dt, 5, "xrwde")
    x, w, r = (s[k].clone().requires_grad_() for k in "xwr")
    y, h = torch_ops.rms_norm(x, w, EPS, residual=r)
    dx, dw, dr = torch.autograd.grad((y, h), (x, w, r), (s["d"], s["e"]))
    assert torch.equal(dx, dr)
    h64, rstd64, _ = reference(s["x"], s["w"], s["r"])
    want, bound, wdw, bdw = grads(s, rstd64, h64, s["e"])

    def loss(hh, ww):
        rs = 1 / torch.sqrt((hh * hh).mean(1, keepdim=True) + EPS)
        return (hh * rs * ww * s["d"].double()).sum() + (hh * s["e"].double()).sum()

    g = torch.Generator().manual_seed(9)
    step = 1e-4
    for k in range(4):
        dirh = torch.randn(rows, cols, generator=g, dtype=torch.float64).to(dev())
        dirw = torch.randn(cols, generator=g, dtype=torch.float64).to(dev())
        w64 = s["w"].double()
        num = (loss(h64 + step * dirh, w64) - loss(h64 - step * dirh, w64)) / (2 * step)
        tol = (dirh.abs() * (want.abs() * half(dt) + bound * F32)).sum() + 1e-5 * num.abs() + 1e-5
        assert abs((dx.double() * dirh).sum() - num) <= tol
        num = (loss(h64, w64 + step * dirw) - loss(h64, w64 - step * dirw)) / (2 * step)
        tol = (dirw.abs() * (wdw.abs() * half(dt) + bdw * (rows + 96) * 2.0 ** -24)).sum() + 1e-5
        assert abs((dw.double() * dirw).sum() - num) <= tol


def test_autograd_uses():
    """Every subset of inputs and outputs that a model may ask gradients for."""
    s = make(6, 64, "bf16", 3, "xrwde")
    full = [s[k].clone().requires_grad_() for k in "xwr"]
    y, h = torch_ops.rms_norm(*full[:2], EPS, residual=full[2])
    gx, gw, gr = torch.autograd.grad((y, h), full, (s["d"], s["e"]))
    # the norm's output alone; the stream alone; an expanded gradient
    y, h = torch_ops.rms_norm(*full[:2], EPS, residual=full[2])
    a = torch.autograd.grad(y, full, s["d"], retain_graph=True)
    assert torch.equal(a[0], torch_ops.rms_norm_backward(
        s["d"], h.detach(), s["w"], torch_ops.rms_norm_forward(s["x"], s["w"], EPS, s["r"])[2])[0])
    assert torch.equal(a[1], gw)
    b = torch.autograd.grad(h, full, s["e"], retain_graph=True)
    assert torch.equal(b[0], s["e"]) and torch.equal(b[2], s["e"]) and (b[1] == 0).all()
    c = torch.autograd.grad(y.float().sum(), full)
    d = torch_ops.rms_norm_backward(torch.ones_like(s["d"]), h.detach(), s["w"],
                                    torch_ops.rms_norm_forward(s["x"], s["w"], EPS, s["r"])[2])
    assert torch.equal(c[0], d[0]) and torch.equal(c[1], d[1])
    # only the weight, only the input, no weight at all
    w = s["w"].clone().requires_grad_()
    y = torch_ops.rms_norm(s["x"], w, EPS)
    (gw1,) = torch.autograd.grad(y, w, s["d"])
    x = s["x"].clone().requires_grad_()
    (gx1,) = torch.autograd.grad(torch_ops.rms_norm(x, s["w"], EPS), x, s["d"])
    (gx2,) = torch.autograd.grad(torch_ops.rms_norm(x, None, EPS), x, s["d"])
    rstd = torch_ops.rms_norm_forward(s["x"], None, EPS)[2]
    dx, dw = torch_ops.rms_norm_backward(s["d"], s["x"], s["w"], rstd)
    assert torch.equal(dx, gx1) and torch.equal(dw, gw1)
    assert torch.equal(torch_ops.rms_norm_backward(s["d"], s["x"], None, rstd)[0], gx2)
    ones = torch.ones_like(s["w"])
    assert torch.equal(torch_ops.rms_norm_backward(s["d"], s["x"], ones, rstd)[0], gx2)


@pytest.mark.parametrize("cols", [64, 256, 512, 1024, 2048, 4096, 8192, 16384])
def test_rows_do_not_depend_on_the_batch(cols):
    rows = 130
    s = make(rows, cols, "bf16", 11, "xrwde")
    y, h, rstd = torch_ops.rms_norm_forward(s["x"], s["w"], EPS, residual=s["r"])
    q, sc, _ = torch_ops.rms_norm_quant(s["x"], s["w"], EPS, residual=s["r"])
    dx, _ = torch_ops.rms_norm_backward(s["d"], h, s["w"], rstd, s["e"])
    # the fused addition has the bits of the addition and the norm
    assert torch.equal(torch_ops.rms_norm(s["x"] + s["r"], s["w"], EPS), y)
    for lo, hi in ((0, 1), (5, 6), (129, 130), (3, 40), (64, 128)):
        part = {k: (v if k == "w" else v[lo:hi]) for k, v in s.items()}
        y2, h2, r2 = torch_ops.rms_norm_forward(part["x"], s["w"], EPS, residual=part["r"])
        assert torch.equal(y2, y[lo:hi]) and torch.equal(h2, h[lo:hi]) and torch.equal(r2, rstd[lo:hi])
        q2, sc2, _ = torch_ops.rms_norm_quant(part["x"], s["w"], EPS, residual=part["r"])
        assert torch.equal(q2.view(torch.uint8), q[lo:hi].view(torch.uint8)) and torch.equal(sc2, sc[lo:hi])
        dx2, _ = torch_ops.rms_norm_backward(part["d"], h2, s["w"], r2, part["e"])
        assert torch.equal(dx2, dx[lo:hi])


@pytest.mark.parametrize("cols", [64, 1040, 4096])
def test_bad_rows_stay_alone(cols):
    s = make(12, cols, "bf16", 13)
    clean = torch_ops.rms_norm(s["x"], s["w"], EPS)
    qc, sc = torch_ops.rms_norm_quant(s["x"], s["w"], EPS)
    x = s["x"].clone()
    x[1, 3] = float("nan")
    x[4, cols - 1] = float("inf")
    x[7, 0] = -float("inf")
    x[9] = 0
    ok = [i for i in range(12) if i not in (1, 4, 7, 9)]
    y = torch_ops.rms_norm(x, s["w"], EPS)
    q, sq = torch_ops.rms_norm_quant(x, s["w"], EPS)
    assert torch.equal(y[ok], clean[ok]) and torch.equal(sq[ok], sc[ok])
    assert torch.equal(q[ok].view(torch.uint8), qc[ok].view(torch.uint8))
    assert y[1].isnan().all() and q[1].float().isnan().all() and sq[1].isnan()
    for i, k in ((4, cols - 1), (7, 0)):  # 1 / inf = 0: the other elements are zero
        rest = [j for j in range(cols) if j != k]
        assert y[i, k].isnan() and (y[i, rest] == 0).all()
        assert q[i].float().isnan().all() and not torch.isfinite(sq[i])
    assert (y[9] == 0).all() and (q[9].float() == 0).all() and sq[9] == 2.0 ** -120
    for v in (3.0e38, 1e-38):  # the ends of the range: sums overflow, or vanish beside eps
        x[2] = v
        want = 0.0 if v > 1 else v * EPS ** -0.5
        got = torch_ops.rms_norm(x, None, EPS)[2].double()
        assert ((got - want).abs() <= want * (half("bf16") + F32)).all()
    x[2] = 60000.0
    qi, si = torch_ops.quantize_rows(x.to(torch.float16))
    assert (qi[2].float() == 448).all()


def test_views_offsets_and_shapes():
    s = make(24, 256, "bf16", 17)
    y = torch_ops.rms_norm(s["x"], s["w"], EPS, residual=s["r"])
    wide = torch.zeros(24, 300, dtype=torch.bfloat16, device=dev())
    wide[:, 3:259] = s["x"]
    assert torch.equal(torch_ops.rms_norm(wide[:, 3:259], s["w"], EPS, residual=s["r"])[0], y[0])
    flat = torch.zeros(24 * 256 + 1, dtype=torch.bfloat16, device=dev())
    flat[1:] = s["x"].reshape(-1)        # contiguous, but off the 16-byte grid
    off = flat[1:].view(24, 256)
    wo = torch.zeros(257, dtype=torch.bfloat16, device=dev())
    wo[1:] = s["w"]
    assert torch.equal(torch_ops.rms_norm(off, wo[1:], EPS, residual=s["r"])[0], y[0])
    z = torch_ops.rms_norm(s["x"].view(2, 3, 4, 256), s["w"], EPS, residual=s["r"].view(2, 3, 4, 256))
    assert z[0].shape == (2, 3, 4, 256) and torch.equal(z[0].view(24, 256), y[0])
    q, sc = torch_ops.rms_norm_quant(s["x"].view(2, 12, 256), s["w"], EPS)
    assert q.shape == (2, 12, 256) and sc.shape == (2, 12)
    one = torch_ops.rms_norm(s["x"][0], s["w"], EPS)
    assert one.shape == (256,) and torch.equal(one, torch_ops.rms_norm(s["x"], s["w"], EPS)[0])
    tr = s["x"].t().contiguous().t()
    assert torch.equal(torch_ops.rms_norm(tr, s["w"], EPS, residual=s["r"])[0], y[0])


def test_empty_batches():
    x = torch.empty(0, 64, dtype=torch.float16, device=dev())
    w = torch.ones(64, dtype=torch.float16, device=dev())
    y, h = torch_ops.rms_norm(x, w, EPS, residual=x)
    assert y.shape == h.shape == (0, 64)
    q, sc = torch_ops.rms_norm_quant(x, w, EPS)
    assert q.shape == (0, 64) and sc.shape == (0,)
    dx, dw = torch_ops.rms_norm_backward(x, x, w, torch.empty(0, device=dev()))
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_in_place_stream_and_rows_behind():
    """residual_out may be the residual itself, and nothing is written past the rows."""
    rows, cols = 5, 264
    s = make(rows, cols, "f16", 19)
    y, h = torch_ops.rms_norm(s["x"], s["w"], EPS, residual=s["r"])
    plan = imm.rms_norm_plan(rows, cols, "f16", eps=EPS)
    buf = torch.full((rows + 2, cols), 7.0, dtype=torch.float16, device=dev())
    out = torch.full((rows + 2, cols), 7.0, dtype=torch.float16, device=dev())
    rstd = torch.full((rows + 2,), 7.0, device=dev())
    buf[:rows] = s["r"]
    imm.rms_norm_run(plan, s["x"], out[:rows], weight=s["w"], residual=buf[:rows],
                     residual_out=buf[:rows], rstd=rstd[:rows])
    assert torch.equal(buf[:rows], h) and torch.equal(out[:rows], y)
    assert (buf[rows:] == 7).all() and (out[rows:] == 7).all() and (rstd[rows:] == 7).all()


def test_streams_and_graph_replays():
    s = make(37, 1024, "bf16", 23, "xrwde")
    want = torch_ops.rms_norm_forward(s["x"], s["w"], EPS, residual=s["r"])
    wq = torch_ops.rms_norm_quant(s["x"], s["w"], EPS, residual=s["r"])
    wb = torch_ops.rms_norm_backward(s["d"], want[1], s["w"], want[2], s["e"])

    def step():
        f = torch_ops.rms_norm_forward(s["x"], s["w"], EPS, residual=s["r"])
        q = torch_ops.rms_norm_quant(s["x"], s["w"], EPS, residual=s["r"])
        b = torch_ops.rms_norm_backward(s["d"], f[1], s["w"], f[2], s["e"])
        return (*f, q[0].view(torch.uint8), q[1], q[2], *b)

    expect = (*want, wq[0].view(torch.uint8), wq[1], wq[2], *wb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, expect))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(4):
        for o in outs:
            o.fill_(0)
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, expect))


def test_refusals_on_the_gpu():
    s = make(4, 64, "bf16", 29)
    x, w = s["x"], s["w"]
    for call in (lambda: torch_ops.rms_norm(x.float(), w), lambda: torch_ops.rms_norm(x, w.half()),
                 lambda: torch_ops.rms_norm(x, w[:32]), lambda: torch_ops.rms_norm(x[:, :12], None),
                 lambda: torch_ops.rms_norm(x, w, residual=x[:2]),
                 lambda: torch_ops.rms_norm(x, w, residual=x.half()),
                 lambda: torch_ops.rms_norm(x, w.cpu()),
                 lambda: torch_ops.rms_norm_quant(x[:, :24], None),
                 lambda: torch_ops.rms_norm_quant(x, w, dtype=torch.float16),
                 lambda: torch_ops.rms_norm_quant(x, w.clone().requires_grad_()),
                 lambda: torch_ops.quantize_rows(x.clone().requires_grad_()),
                 lambda: torch_ops.rms_norm_backward(x, x, w, torch.zeros(3, device=dev()))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(imm.GemmError):
        torch_ops.rms_norm(x, w, float("nan"))
    with torch.no_grad():
        torch_ops.rms_norm_quant(x, w.clone().requires_grad_())
    # the C ABI's own checks: a scale where none belongs, host memory, a short workspace
    plan = imm.rms_norm_plan(4, 64, "bf16")
    out = torch.empty_like(x)
    sc = torch.empty(4, device=dev())
    with pytest.raises(imm.GemmError):
        imm.rms_norm_run(plan, x, out, weight=w, row_scale=sc)
    L = imm.lib()
    pinned = torch.zeros(4, 64, dtype=torch.bfloat16).pin_memory()
    args = [plan.handle, pinned.data_ptr(), 0, 0, out.data_ptr(), 0, 0, 0, 0]
    assert L.rms_norm_run(*args) == 1
    ws = torch.empty(plan.workspace_bytes - 4, dtype=torch.uint8, device=dev())
    with pytest.raises(imm.GemmError) as e:
        imm.rms_norm_backward(plan, x, x, sc, out, weight=w, dweight=torch.empty_like(w), workspace=ws)
    assert e.value.status == 3
    # beyond one allocation: the rows of a larger plan do not fit in these operands
    big = imm.rms_norm_plan(1 << 24, 1024, "bf16")
    assert L.rms_norm_run(big.handle, x.data_ptr(), 0, 0, out.data_ptr(), 0, 0, 0, 0) == 1


def test_more_rows_than_one_launch_holds():
    """2^28 + 5 rows of 8 (16 threads a row): the rows behind the first launch's threads."""
    rows = (1 << 28) + 5
    x = torch.empty(rows, 8, dtype=torch.bfloat16, device=dev())
    g = torch.Generator().manual_seed(91)
    part = torch.randn(64, 8, generator=g).bfloat16().to(dev())
    x.zero_()
    places = ((0, 64), ((1 << 27) - 32, (1 << 27) + 32), (rows - 64, rows))
    for lo, hi in places:
        x[lo:hi] = part
    want = torch_ops.rms_norm(part, None, 1e-6)
    y = torch_ops.rms_norm(x, None, 1e-6)
    for lo, hi in places:
        assert torch.equal(y[lo:hi], want)
    assert (y[1000:2000] == 0).all()
    assert torch.equal(torch_ops.rms_norm_forward(x)[2][rows - 64:], torch_ops.rms_norm_forward(part)[2])
