"""The decoder operators in 64 bits, straight from their formulas, with error bounds.

Bounds count roundings: one to the result's type is at most half a step,
``half(dtype)`` = eps / 2 of the value (or half the smallest subnormal,
``tiny(dtype)``); an fp32 operation U = 2^-24 of its result, a chain of n
additions at most n U of the sum of magnitudes.
"""
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2


def close(got, want, tol, what):
    """|got - want| <= tol everywhere; NaN and infinities of the reference in the same places."""
    got, want = got.double(), want.double()
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    same = odd & ~torch.isnan(want)
    assert torch.equal(got[same], want[same]), f"{what}: infinities"
    err = (got - want).abs()
    tol = torch.as_tensor(tol, dtype=torch.float64, device=want.device).expand_as(want)
    bad = ~odd & ~(err <= tol)
    if bad.any():
        i = tuple(int(x[0]) for x in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, the first at {i}: {float(got[i])} for "
                             f"{float(want[i])}, allowed {float(tol[i])}")


# ---- norm and rotation of heads ----------------------------------------------------

def turns(positions, inv_freq, sections):
    """cos and sin [T, 1, R / 2]"""
    if sections is None:
        angle = positions.double()[:, None] * inv_freq
    else:
        axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(positions.device)
        angle = positions.double()[axis].t() * inv_freq
    return angle.cos()[:, None], angle.sin()[:, None]


def rotate(y, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    z = y.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    z[..., a] = y[..., a] * cos - y[..., b] * sin
    z[..., b] = y[..., b] * cos + y[..., a] * sin
    return z


def rope(x, positions, inv_freq, weight, eps, norm, interleaved, sections):
    """(out, bound) in fp64 for one tensor of heads.  With the norm, x rstd w is within 2^-19 of itself
    (64 squares in a lane and its 6 halvings at most, a division, a root, three products);
    cosine and sine are within 2^-21 (the angle's fraction of a turn rounded to fp32, 2^-25 of
    a half turn times 2 pi, and an fp32 function); then one rounding."""
    h = x.double()
    if norm:
        h = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
        if weight is not None:
            h = h * weight.double()
    cos, sin = turns(positions, inv_freq, sections)
    out = rotate(h, cos, sin, interleaved)
    mag = rotate(h.abs(), torch.ones_like(cos), -torch.ones_like(sin), interleaved).abs() + h.abs()
    return out, out.abs() * half(x.dtype) + mag * 2.0 ** -18 + tiny(x.dtype)


# ---- attention ---------------------------------------------------------------------

def attend(q, k, v, causal, scale):
    """One sequence in fp64: (o, lse, p, seen); q [n, hq, D], k and v [m, hk, D]."""
    n, hq, _ = q.shape
    m, hk, _ = k.shape
    kd = k.double().repeat_interleave(hq // hk, 1)
    vd = v.double().repeat_interleave(hq // hk, 1)
    s = scale * torch.matmul(q.double().transpose(0, 1), kd.permute(1, 2, 0).contiguous())
    seen = torch.ones(n, m, dtype=torch.bool, device=q.device)
    if causal:
        seen = torch.arange(m, device=q.device)[None] <= (m - n + torch.arange(n, device=q.device))[:, None]
    s = s.masked_fill(~seen, float("-inf"))
    top = s.amax(-1, keepdim=True) if m else s.new_full((hq, n, 1), float("-inf"))
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    o = torch.matmul(p, vd.transpose(0, 1).contiguous()).transpose(0, 1)
    lse = (top + torch.log(total))[..., 0].transpose(0, 1)
    return o, lse, p, seen


def attention_case(q, k, v, do, causal, scale):
    """One sequence: fp64 results (o, lse, dq, dk, dv) and their bounds, as two dicts."""
    dt = q.dtype
    n, hq, D = q.shape
    m, hk, _ = k.shape
    G = hq // hk
    o, lse, p, seen = attend(q, k, v, causal, scale)
    qd, dod = q.double().transpose(0, 1), do.double().transpose(0, 1)          # [hq, n, D]
    kd, vd = (t.double().transpose(0, 1).repeat_interleave(G, 0) for t in (k, v))  # [hq, m, D]

    def mm(a, b):
        return torch.matmul(a.contiguous(), b.contiguous())

    # logits: a chain of D products, the scale, the maximum's subtraction (each an fp32
    # rounding of numbers up to the logits' magnitudes), and the exponential
    mag = scale * mm(qd.abs(), kd.abs().transpose(1, 2))
    ds_ = (D + 4) * U * mag + 2.0 ** -21
    eps_p = (2 * ds_.masked_fill(~seen, 0).amax(-1, keepdim=True) if m else ds_.new_zeros(hq, n, 1)) + (m + 64) * U
    sub = tiny(dt) / (1.0 if dt != torch.float16 else 1.0)  # of a probability below the type's normals
    rnd = half(dt)
    bound = {}
    ov = mm(p, vd.abs())
    # a probability about the running maximum is at most 1 and its share of the sum at least as small
    bo = ov * (rnd + eps_p) + sub * (vd.abs().sum(1, keepdim=True) if m else 0)
    bound["o"] = (bo + o.transpose(0, 1).abs() * rnd).transpose(0, 1) + tiny(dt)
    bound["lse"] = (eps_p[..., 0] + 2.0 ** -21 * (1 + lse.transpose(0, 1).abs().nan_to_num(posinf=0))).transpose(0, 1)
    delta = (dod * o.transpose(0, 1)).sum(-1, keepdim=True)
    dp = mm(dod, vd.transpose(1, 2))
    ds = p * (dp - delta)
    e_dp = (D + 2) * U * mm(dod.abs(), vd.abs().transpose(1, 2))
    e_delta = (dod.abs() * bound["o"].transpose(0, 1)).sum(-1, keepdim=True) + (D + 2) * U * (
        dod * o.transpose(0, 1)).abs().sum(-1, keepdim=True)
    e_lse = bound["lse"].transpose(0, 1).unsqueeze(-1)
    eps_q = eps_p + e_lse  # p again, from the stored lse
    e_ds = p * (e_dp + e_delta) * (1 + rnd) + ds.abs() * (rnd + 2 * eps_q) + tiny(dt)
    e_ds = e_ds.masked_fill(~seen, 0)
    dq = scale * mm(ds, kd)
    bound["dq"] = (scale * mm(e_ds + (m + 8) * U * ds.abs(), kd.abs()) + dq.abs() * rnd).transpose(0, 1) + tiny(dt)

    def shared(t):  # over the query heads of a key head
        return t.reshape(hk, G, m, D).sum(1).transpose(0, 1)

    rows = (n * G + 8) * U
    dk = shared(scale * mm(ds.transpose(1, 2), qd))
    dv = shared(mm(p.transpose(1, 2), dod))
    bound["dk"] = shared(scale * mm((e_ds + rows * ds.abs()).transpose(1, 2), qd.abs())) + dk.abs() * rnd + tiny(dt)
    e_p = (p * (rnd + 2 * eps_q + rows) + sub).masked_fill(~seen, 0)
    bound["dv"] = shared(mm(e_p.transpose(1, 2), dod.abs())) + dv.abs() * rnd + tiny(dt)
    want = {"o": o, "lse": lse, "dq": dq.transpose(0, 1), "dk": dk, "dv": dv}
    return want, bound


# ---- log probabilities ---------------------------------------------------------------

def logprobs(x, tokens, top):
    """(logprob, entropy, top_logprob, top_token) of rows x [rows, V], tokens [rows, n], in fp64."""
    x = x.double()
    V = x.shape[1]
    logp = torch.log_softmax(x, 1)
    p = logp.exp()
    ent = -torch.where(p > 0, p * logp, torch.where(torch.isnan(p), p, torch.zeros_like(p))).sum(1)
    inside = (tokens >= 0) & (tokens < V)
    lp = logp.gather(1, tokens.clamp(0, V - 1))
    lp = torch.where(inside, lp, torch.where(tokens < 0, torch.zeros_like(lp), torch.full_like(lp, float("nan"))))
    # NaN above every number, then by value, then by place
    key = torch.where(torch.isnan(x), torch.full_like(x, float("inf")), x)
    key = torch.where(torch.isnan(x), key, torch.minimum(key, torch.full_like(x, 1e300)))
    best = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :top]
    return lp, ent, logp.gather(1, best), best


def logprobs_gradient(x, tokens, g, h):
    """The gradient of the logits in fp64; g [rows, n], h [rows]."""
    x = x.double()
    V = x.shape[1]
    logp = torch.log_softmax(x, 1)
    p = logp.exp()
    safe = torch.where(p > 0, logp, torch.zeros_like(logp))
    ent = -(p * safe).sum(1, keepdim=True)
    inside = (tokens >= 0) & (tokens < V)
    gd = torch.where(inside, g.double(), torch.zeros_like(g, dtype=torch.float64))
    dx = -p * gd.sum(1, keepdim=True) - h.double()[:, None] * p * (safe + ent)
    return dx.scatter_add(1, tokens.clamp(0, V - 1), gd)
