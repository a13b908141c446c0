"""The norm of query and key heads with the rotation of their position, and its backward
pass, against the formula in 64 bits (tests/decoder_oracle.py)."""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests import decoder_oracle as ref
from tests.helpers import dev

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def make(T, hq, hk, D, R, dt, seed, axes=1, far=100000, fused=True):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (mean + std * torch.randn(*shape, generator=g)).to(DT[dt]).to(dev())

    if fused:
        qkv = normal(T, (hq + 2 * hk) * D, std=2.0)
        q, k = qkv[:, :hq * D].unflatten(1, (hq, D)), qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    else:
        q, k = normal(T, hq, D, std=2.0), normal(T, hk, D, std=2.0)
    pos = torch.randint(-far // 10, far, (T,) if axes == 1 else (axes, T), generator=g).to(dev())
    freq = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))).to(dev())
    return {"q": q, "k": k, "pos": pos, "freq": freq, "wq": normal(D, std=0.2, mean=1.0), "wk": normal(D, std=0.2, mean=1.0),
            "dq": normal(T, hq, D), "dk": normal(T, hk, D)}


# (T, hq, hk, D, R): dimensions of every lane layout, full and partial; one token; odd numbers
SHAPES = [(1, 32, 8, 128, 128), (7, 5, 1, 64, 64), (33, 3, 3, 80, 64), (3, 2, 1, 8, 0), (5, 1, 1, 16, 16), (65, 8, 2, 96, 96),
          (9, 4, 4, 256, 128), (4, 3, 1, 512, 512), (19, 1, 2, 136, 96), (130, 40, 8, 128, 64), (2, 70, 1, 128, 128)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_matches_the_formula(shape, interleaved, dt):
    T, hq, hk, D, R = shape
    s = make(*shape, dt, 1)
    got = torch_ops.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], s["wq"], s["wk"], EPS, interleaved=interleaved)
    for y, x, w, name in zip(got, (s["q"], s["k"]), (s["wq"], s["wk"]), "qk"):
        want, tol = ref.rope(x, s["pos"], s["freq"], w, EPS, True, interleaved, None)
        assert y.is_contiguous() and y.shape == x.shape and y.dtype == x.dtype
        ref.close(y, want, tol, name)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sections", [None, [16, 24, 24], [1, 63], [0, 64], [10, 20, 30, 4]])
@pytest.mark.parametrize("norm,weights", [(True, True), (True, False), (False, False)])
def test_axes_norm_and_weights(norm, weights, sections, interleaved):
    axes = 1 if sections is None else len(sections)
    s = make(37, 6, 2, 128, 128, "bf16", 2, axes)
    w = (s["wq"], s["wk"]) if weights else (None, None)
    got = torch_ops.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], *w, EPS, norm=norm, interleaved=interleaved,
                                 sections=sections)
    for y, x, u in zip(got, (s["q"], s["k"]), w):
        want, tol = ref.rope(x, s["pos"], s["freq"], u, EPS, norm, interleaved, sections)
        ref.close(y, want, tol, "out")


def test_far_positions():
    # the angle's whole turns go in fp64: 2^31 positions lose 2^-22 of a radian there
    s = make(64, 2, 1, 64, 64, "f16", 3)
    pos = torch.randint(0, 1 << 31, (64,), generator=torch.Generator().manual_seed(4)).to(dev())
    y, _ = torch_ops.qk_norm_rope(s["q"], s["k"], pos, s["freq"], norm=False)
    want, tol = ref.rope(s["q"], pos, s["freq"], None, EPS, False, False, None)
    ref.close(y, want, tol, "far")


def test_rows_are_their_own():
    s = make(300, 16, 4, 128, 128, "bf16", 5)
    whole = torch_ops.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], s["wq"], s["wk"])
    for a, b in ((0, 1), (17, 18), (100, 300), (0, 299)):
        part = torch_ops.qk_norm_rope(s["q"][a:b], s["k"][a:b], s["pos"][a:b], s["freq"], s["wq"], s["wk"])
        assert all(torch.equal(x[a:b], y) for x, y in zip(whole, part))
    alone = torch_ops.qk_norm_rope(s["q"][:, 3:4], s["k"][:, :0], s["pos"], s["freq"], s["wq"], None)
    assert torch.equal(alone[0], whole[0][:, 3:4]) and alone[1].shape == (300, 0, 128)


@pytest.mark.parametrize("scale", [1e37, 3e38, 1e-20, 1e-38])
def test_finite_heads_of_every_magnitude(scale):
    s = make(5, 3, 1, 128, 64, "bf16", 6)
    q = (s["q"].float() * (scale / 8)).bfloat16()
    y, _ = torch_ops.qk_norm_rope(q, s["k"], s["pos"], s["freq"], None, None, 0.0)
    want, tol = ref.rope(q, s["pos"], s["freq"], None, 0.0, True, False, None)
    ref.close(y, want, tol, "magnitude")


def test_bad_heads_stay_alone():
    s = make(9, 4, 2, 64, 64, "bf16", 7)
    clean = torch_ops.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], s["wq"], s["wk"])
    q = s["q"].clone()
    q[3, 2, 5] = float("nan")
    q[4, 0, 0] = float("inf")
    y, k = torch_ops.qk_norm_rope(q, s["k"], s["pos"], s["freq"], s["wq"], s["wk"])
    bad = torch.zeros(9, 4, dtype=torch.bool, device=y.device)
    bad[3, 2] = bad[4, 0] = True
    assert torch.isnan(y[3, 2]).all() and not torch.isfinite(y[4, 0]).all()
    assert torch.equal(y[~bad], clean[0][~bad]) and torch.equal(k, clean[1])


def backward_reference(s, x, dy, w, norm, interleaved, sections):
    """(dx, bound, dw, bound).  dx is x, dy and w in a few fp32 operations: 2^-17 of the magnitudes of
    its terms; a weight's gradient sums T heads in fp32 chains."""
    cos, sin = ref.turns(s["pos"], s["freq"], sections)
    g = ref.rotate(dy.double(), cos, -sin, interleaved)
    mag = ref.rotate(dy.double().abs(), torch.ones_like(cos), -torch.ones_like(sin), interleaved).abs() + dy.double().abs()
    if not norm:
        return g, g.abs() * ref.half(x.dtype) + mag * 2.0 ** -18 + ref.tiny(x.dtype), None, None
    xd, D = x.double(), x.shape[-1]
    rstd = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True) + EPS)
    n = xd * rstd
    wd = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
    dx = rstd * (g * wd - n * (g * wd * n).mean(-1, keepdim=True))
    m = rstd * (mag * wd.abs() + n.abs() * (mag * wd.abs() * n.abs()).mean(-1, keepdim=True))
    dw = (g * n).sum((0, 1))
    terms = x.shape[0] * x.shape[1]
    bw = (mag * n.abs()).sum((0, 1)) * (2.0 ** -17 + terms * ref.U) + dw.abs() * ref.half(x.dtype) + ref.tiny(x.dtype)
    return dx, dx.abs() * ref.half(x.dtype) + m * 2.0 ** -17 + ref.tiny(x.dtype), dw, bw


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("norm,weights", [(True, True), (True, False), (False, False)])
@pytest.mark.parametrize("shape", SHAPES)
def test_gradients_match_the_formula(shape, norm, weights, dt):
    s = make(*shape, dt, 8)
    w = (s["wq"], s["wk"]) if weights else (None, None)
    interleaved = shape[0] % 2 == 0
    got = torch_ops.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["freq"], *w, EPS, norm=norm,
                                          interleaved=interleaved)
    for i, (x, dy) in enumerate(((s["q"], s["dq"]), (s["k"], s["dk"]))):
        dx, bx, dw, bw = backward_reference(s, x, dy, w[i], norm, interleaved, None)
        ref.close(got[i], dx, bx, "dx")
        if weights:
            ref.close(got[2 + i], dw, bw, "dw")
        else:
            assert got[2 + i] is None


def test_many_tokens_and_the_weights_gradient():
    s = make(3001, 16, 8, 128, 128, "bf16", 9)
    got = torch_ops.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["freq"], s["wq"], s["wk"], EPS)
    again = torch_ops.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["freq"], s["wq"], s["wk"], EPS)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    for i, (x, dy, w) in enumerate(((s["q"], s["dq"], s["wq"]), (s["k"], s["dk"], s["wk"]))):
        dx, bx, dw, bw = backward_reference(s, x, dy, w, True, False, None)
        ref.close(got[i], dx, bx, "dx")
        ref.close(got[2 + i], dw, bw, "dw")


def test_autograd_and_differences():
    s = make(6, 3, 1, 64, 32, "bf16", 10, fused=False)
    leaves = [s[n].clone().requires_grad_() for n in ("q", "k", "wq", "wk")]
    y, z = torch_ops.qk_norm_rope(leaves[0], leaves[1], s["pos"], s["freq"], leaves[2], leaves[3], EPS)
    torch.autograd.backward((y, z), (s["dq"], s["dk"]))
    direct = torch_ops.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["freq"], s["wq"], s["wk"], EPS)
    for a, b in zip(leaves, direct):
        assert torch.equal(a.grad, b)

    def loss(q, wq):
        return (ref.rope(q, s["pos"], s["freq"], wq, EPS, True, False, None)[0] * s["dq"].double()).sum()

    g = torch.Generator().manual_seed(11)
    for name, i in (("q", 0), ("wq", 2)):
        d = torch.randn(s[name].shape, generator=g).double().to(dev())
        at = {"q": s["q"].double(), "wq": s["wq"].double()}
        h = 1e-5
        up, down = ({**at, name: at[name] + e * d} for e in (h, -h))
        want = (loss(**{"q": up["q"], "wq": up["wq"]}) - loss(**{"q": down["q"], "wq": down["wq"]})) / (2 * h)
        dx, bx, dw, bw = backward_reference(s, s["q"], s["dq"], s["wq"], True, False, None)
        tol = ((bx if i == 0 else bw) * d.abs()).sum() + 1e-6 * (1 + want.abs())
        assert abs((direct[i].double() * d).sum() - want) <= tol


def test_strided_and_unaligned_heads():
    s = make(11, 4, 2, 72, 64, "f16", 12, fused=False)
    want = torch_ops.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], s["wq"], s["wk"])
    odd = torch.empty(11 * 4 * 72 + 1, dtype=torch.float16, device=dev())[1:].view(11, 4, 72).copy_(s["q"])
    turned = s["k"].permute(2, 0, 1).contiguous().permute(1, 2, 0)
    got = torch_ops.qk_norm_rope(odd, turned, s["pos"], s["freq"], s["wq"], s["wk"])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    heads = s["q"].transpose(0, 1).contiguous().transpose(0, 1)  # heads outside tokens: read in place
    assert torch.equal(torch_ops.qk_norm_rope(heads, s["k"], s["pos"], s["freq"], s["wq"], s["wk"])[0], want[0])


def test_no_tokens():
    s = make(3, 2, 1, 64, 64, "bf16", 13)
    y, z = torch_ops.qk_norm_rope(s["q"][:0], s["k"][:0], s["pos"][:0], s["freq"], s["wq"], s["wk"])
    assert y.shape == (0, 2, 64) and z.shape == (0, 1, 64)
    dq, dk, dwq, dwk = torch_ops.qk_norm_rope_backward(y, z, s["q"][:0], s["k"][:0], s["pos"][:0], s["freq"], s["wq"], s["wk"])
    assert dq.shape == (0, 2, 64) and (dwq == 0).all() and (dwk == 0).all()


def test_refusals():
    s = make(3, 2, 1, 64, 64, "bf16", 14)
    a = dict(q=s["q"], k=s["k"], positions=s["pos"], inv_freq=s["freq"])
    for change in ({"q": s["q"].float()}, {"k": s["k"].half()}, {"q": s["q"].cpu()}, {"positions": s["pos"].int()},
                   {"positions": s["pos"][:2]}, {"inv_freq": s["freq"].float()}, {"k": s["k"][:2]}, {"q": s["q"][0]},
                   {"sections": [16, 16, 1]}, {"q_weight": s["wq"][:32]}, {"q_weight": s["wq"].half()},
                   {"norm": False, "q_weight": s["wq"]}, {"sections": [-1, 33]}, {"inv_freq": s["freq"].cpu()}):
        with pytest.raises(ValueError):
            torch_ops.qk_norm_rope(**{**a, **change})
    for change in ({"inv_freq": s["freq"][:7]}, {"eps": -1.0}, {"eps": float("nan")}):  # R = 14
        with pytest.raises(RuntimeError):
            torch_ops.qk_norm_rope(**{**a, **change})
