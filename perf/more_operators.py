"""Operators between and behind the products of a transformer: what is measured, with plain forms.

Three operators that a decoder needs next to its linear layers: the norm of every
query and key head with the rotation of its position ("rope", and its training
step), attention over packed sequences, over a cache and in training
("attention"), and the log probabilities of given tokens with the entropy and the
most likely alternatives ("logprobs", and its training step).

``own = False`` computes them with elementary torch operations in 32 bits (angles
in 64); ``own = True`` makes the calls of invariant_matmul_amd.torch_ops.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one token through a layer: latency alone
        {"name": "rope_token", "op": "rope", "tokens": 1, "hq": 32, "hk": 8, "dim": 128, "rot": 128, "axes": 1,
         "interleaved": False, "norm": True, "train": False, "far": 100000, "dtype": "bf16"},
        # a long prompt behind a fused query, key and value projection
        {"name": "rope_prompt", "op": "rope", "tokens": 8191, "hq": 32, "hk": 8, "dim": 128, "rot": 128, "axes": 1,
         "interleaved": False, "norm": True, "train": False, "far": 1000000, "dtype": "bf16"},
        # patches of a video: time, height and width, no norm, part of each head rotated
        {"name": "rope_video", "op": "rope", "tokens": 5003, "hq": 16, "hk": 16, "dim": 80, "rot": 64, "axes": 3,
         "interleaved": True, "norm": False, "train": False, "far": 500, "dtype": "f16"},
        # a training step: outputs and the gradients of heads and weights
        {"name": "rope_train", "op": "rope", "tokens": 4096, "hq": 16, "hk": 8, "dim": 128, "rot": 128, "axes": 1,
         "interleaved": False, "norm": True, "train": True, "far": 4096, "dtype": "bf16"},
        # one new token of one conversation over its cache: latency
        {"name": "attention_token", "op": "attention", "kind": "cache", "seqs": 1, "new": 1, "room": 8192, "hq": 32,
         "hk": 8, "dim": 128, "causal": True, "dtype": "bf16"},
        # a decode batch over caches filled to different lengths: the stream of the caches
        {"name": "attention_batch", "op": "attention", "kind": "cache", "seqs": 61, "new": 1, "room": 8192, "hq": 32,
         "hk": 4, "dim": 128, "causal": True, "dtype": "f16"},
        # prompts of different lengths packed into one call, small heads
        {"name": "attention_packed", "op": "attention", "kind": "prompt", "seqs": 13, "tokens": 8191, "hq": 16, "hk": 2,
         "dim": 64, "causal": True, "dtype": "f16"},
        # one long prompt: the matrix rate
        {"name": "attention_long", "op": "attention", "kind": "prompt", "seqs": 1, "tokens": 16384, "hq": 32, "hk": 8,
         "dim": 128, "causal": True, "dtype": "bf16"},
        # a training step over packed documents: output and the gradients of queries, keys and values
        {"name": "attention_train", "op": "attention", "kind": "train", "seqs": 5, "tokens": 8195, "hq": 16, "hk": 8,
         "dim": 128, "causal": True, "dtype": "bf16"},
        # a decode batch's sampled tokens with twenty alternatives
        {"name": "logprobs_decode", "op": "logprobs", "rows": 16, "vocab": 131072, "top": 20, "train": False,
         "dtype": "bf16"},
        # scoring a prompt: odd vocabulary, 32-bit logits
        {"name": "logprobs_prompt", "op": "logprobs", "rows": 4093, "vocab": 100003, "top": 5, "train": False,
         "dtype": "f32"},
        # a policy's training step: log probability, entropy and the gradient of the logits
        {"name": "logprobs_train", "op": "logprobs", "rows": 4096, "vocab": 65536, "top": 0, "train": True,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over its logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["rope", "attention", "attention", "logprobs"])
    if op == "rope":
        hk = rng.choice([1, 2, 4, 8, 16])
        hq = min(64, hk * rng.choice([1, 2, 4, 5, 8]))
        dim = rng.choice([64, 80, 96, 128, 256])
        train = rng.random() < 0.4
        norm = rng.random() < 0.7
        return {"op": "rope", "tokens": _log(rng, 1, (4096 if train else 8191) * 48 * 128 // ((hq + hk) * dim * 2)),
                "hq": hq, "hk": hk, "dim": dim, "rot": rng.choice([dim, dim // 32 * 16]), "axes": rng.choice([1, 1, 2, 3]),
                "interleaved": rng.random() < 0.4, "norm": norm, "train": train,
                "far": _log(rng, 1000, 1000000), "dtype": rng.choice(["bf16", "f16"])}
    if op == "logprobs":
        train = rng.random() < 0.4
        vocab = _log(rng, 300, 200000)
        return {"op": "logprobs", "rows": _log(rng, 1, min(20000, (4096 * 65536 if train else 4093 * 100003 // 2) // vocab)),
                "vocab": vocab, "top": 0 if train else rng.choice([0, 1, 5, 20]), "train": train,
                "dtype": rng.choice(["bf16", "f16", "f32"])}
    kind = rng.choice(["cache", "cache", "prompt", "train"])
    hk = rng.choice([1, 2, 4, 8])
    case = {"op": "attention", "kind": kind}
    if kind == "cache":
        case["seqs"] = _log(rng, 1, 96)
        case["new"] = rng.choice([1, 1, 1, 2, 5, 100])
        case["room"] = _log(rng, 128, min(65536, 61 * 8192 // case["seqs"]))
        case["new"] = min(case["new"], case["room"])
    else:
        case["seqs"] = _log(rng, 1, 24)
        case["tokens"] = _log(rng, max(16, 2 * case["seqs"]), 8195 if kind == "prompt" else 5000)
    case.update({"hq": hk * rng.choice([1, 2, 4, 5, 8] if hk < 8 else [1, 2, 4]), "hk": hk,
                 "dim": rng.choice([64, 80, 96, 128]), "causal": kind == "cache" or rng.random() < 0.8,
                 "dtype": rng.choice(["bf16", "f16"])})
    return case


def _lengths(case):
    """(queries, keys) of each sequence, fixed by the case."""
    rng = random.Random(case["seqs"] * 1000003 + case.get("tokens", case.get("room")))
    if case["kind"] == "cache":
        least = max(case["new"], case["room"] // 8)
        keys = [rng.randint(least, case["room"]) for _ in range(case["seqs"])]
        keys[0] = case["room"]
        return [case["new"]] * case["seqs"], keys
    cuts = sorted(rng.sample(range(1, case["tokens"]), case["seqs"] - 1))
    lens = [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]
    return lens, lens


def _sections(case):
    """Frequencies of each axis: a quarter for time, the rest shared."""
    half, axes = case["rot"] // 2, case["axes"]
    if axes == 1:
        return None
    first = half // 4 if axes == 3 else half // 2
    return [first, half - first] if axes == 2 else [first, (half - first) // 2, half - first - (half - first) // 2]


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    if case["op"] == "rope":
        T, hq, hk, D, R = (case[n] for n in ("tokens", "hq", "hk", "dim", "rot"))
        # the projection's output: queries, keys and values of a token in one row
        qkv = normal(T, (hq + 2 * hk) * D, std=2.0).to(dt)
        s = {"q": qkv[:, :hq * D].unflatten(1, (hq, D)), "k": qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D)),
             "freq": 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)}
        shape = (T,) if case["axes"] == 1 else (case["axes"], T)
        s["pos"] = torch.randint(0, case["far"], shape, generator=g, device="cuda")
        if case["norm"]:
            s["wq"], s["wk"] = ((1 + normal(D, std=0.2)).to(dt) for _ in "qk")
        if case["train"]:
            s["dq"], s["dk"] = normal(T, hq, D, std=0.1).to(dt), normal(T, hk, D, std=0.1).to(dt)
        return s
    if case["op"] == "logprobs":
        rows, V = case["rows"], case["vocab"]
        # logits of a model that is sure of some tokens and undecided on others
        x = normal(rows, V)
        x *= 1 + 2 * torch.rand(rows, 1, generator=g, device="cuda")
        s = {"x": x.to(dt), "t": torch.randint(0, V, (rows,), generator=g, device="cuda")}
        if case["train"]:
            s["dl"], s["dh"] = normal(rows), normal(rows, std=0.01)
        return s
    nq, nk = _lengths(case)
    hq, hk, D = case["hq"], case["hk"], case["dim"]
    Tq = sum(nq)
    Tk = case["seqs"] * case["room"] if case["kind"] == "cache" else Tq
    s = {"q": normal(Tq, hq, D, std=1.7).to(dt), "k": normal(Tk, hk, D, std=1.7).to(dt), "v": normal(Tk, hk, D).to(dt),
         "cu_q": torch.tensor([sum(nq[:i]) for i in range(len(nq) + 1)], dtype=torch.int32, device="cuda")}
    if case["kind"] == "cache":
        # one slab of `room` rows a sequence, filled to its length
        s["cu_k"] = torch.arange(case["seqs"] + 1, dtype=torch.int32, device="cuda") * case["room"]
        s["lens"] = torch.tensor(nk, dtype=torch.int32, device="cuda")
    if case["kind"] == "train":
        s["do"] = normal(Tq, hq, D, std=0.1).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    return s


def run(state):
    return {"rope": _rope, "attention": _attention, "logprobs": _logprobs}[state["case"]["op"]](state, state["case"])


def _rope(s, case):
    sections = _sections(case)
    if own:
        from invariant_matmul_amd import torch_ops
        kw = {"norm": case["norm"], "interleaved": case["interleaved"], "sections": sections}
        args = (s["q"], s["k"], s["pos"], s["freq"], s.get("wq"), s.get("wk"), EPS)
        out = torch_ops.qk_norm_rope(*args, **kw)
        if not case["train"]:
            return out
        dq, dk, dwq, dwk = torch_ops.qk_norm_rope_backward(s["dq"], s["dk"], *args, **kw)
        return (*out, dq, dk, dwq, dwk) if case["norm"] else (*out, dq, dk)
    pos = s["pos"].double()
    if sections is None:
        angle = pos[:, None] * s["freq"]
    else:  # each frequency turns by its own axis' position
        angle = torch.cat([p[:, None] * f for p, f in zip(pos, s["freq"].split(sections))], 1)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out, grads, dws = [], [], []
    for name in "qk":
        x = s[name].float()
        n = w = 1.0
        if case["norm"]:
            rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            n, w = x * rstd, s["w" + name].float()
            out.append(_turn(n * w, cos, sin, case))
        else:
            out.append(_turn(x, cos, sin, case))
        if case["train"]:
            g = _turn(s["d" + name].float(), cos, -sin, case)  # the rotation's transpose
            if case["norm"]:
                dws.append((g * n).sum((0, 1)))
                g = g * w
                g = rstd * (g - n * (g * n).mean(-1, keepdim=True))
            grads.append(g)
    return tuple(t.to(s["q"].dtype) for t in out + grads + dws)


def _turn(x, cos, sin, case):
    R = case["rot"]
    if case["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., R:]), -1)


def _attention(s, case):
    q, k, v = s["q"], s["k"], s["v"]
    if own:
        from invariant_matmul_amd import torch_ops
        cu_k = s.get("cu_k", s["cu_q"])
        if case["kind"] != "train":
            return torch_ops.attention(q, k, v, s["cu_q"], cu_k, k_lens=s.get("lens"), max_q=case.get("new"),
                                       causal=case["causal"])
        o, lse = torch_ops.attention_forward(q, k, v, s["cu_q"], cu_k, causal=case["causal"])
        return o, *torch_ops.attention_backward(s["do"], q, k, v, o, lse, s["cu_q"], cu_k, causal=case["causal"])
    nq, nk = _lengths(case)
    hk, D = case["hk"], case["dim"]
    group = case["hq"] // hk
    o = torch.empty_like(q)
    grads = [torch.zeros_like(t, dtype=torch.float32) for t in (q, k, v)] if "do" in s else None
    q0 = k0 = 0
    for n, m in zip(nq, nk):
        # the keys of a head, once for the whole group of query heads that share it
        kf, vf = (t[k0:k0 + m].float().transpose(0, 1).contiguous() for t in (k, v))
        step = max(1, (1 << 29) // (m * case["hq"]))
        for a in range(0, n, step):
            b = min(n, a + step)

            def rows(t):
                return t[q0 + a:q0 + b].float().unflatten(1, (hk, group)).permute(1, 2, 0, 3).reshape(hk, -1, D)

            qf = rows(q) * D ** -0.5
            p = qf @ kf.transpose(1, 2)
            if case["causal"]:
                at = torch.arange(m - n + a, m - n + b, device="cuda").repeat(group)
                p.masked_fill_(torch.arange(m, device="cuda") > at[:, None], float("-inf"))
            p -= p.amax(-1, keepdim=True)
            p.exp_()
            p /= p.sum(-1, keepdim=True)
            of = p @ vf

            def back(t):
                return t.reshape(hk, group, b - a, D).permute(2, 0, 1, 3).reshape(b - a, hk * group, D)

            o[q0 + a:q0 + b] = back(of).to(q.dtype)
            if grads:
                do = rows(s["do"])
                grads[2][k0:k0 + m] += (p.transpose(1, 2) @ do).transpose(0, 1)
                ds = do @ vf.transpose(1, 2)
                ds -= (do * of).sum(-1, keepdim=True)
                ds *= p
                grads[0][q0 + a:q0 + b] = back(ds @ kf) * D ** -0.5
                grads[1][k0:k0 + m] += (ds.transpose(1, 2) @ qf).transpose(0, 1)
        q0 += n
        k0 += case.get("room", m)
    return (o, *(t.to(q.dtype) for t in grads)) if grads else o


def _logprobs(s, case):
    if own:
        from invariant_matmul_amd import torch_ops
        if not case["train"]:
            return torch_ops.token_logprobs(s["x"], s["t"], case["top"])
        lp, ent, lse = torch_ops.token_logprobs_forward(s["x"], s["t"])
        return lp, ent, torch_ops.token_logprobs_backward(s["dl"], s["dh"], s["x"], s["t"], lse, ent)
    x = s["x"].float()
    logp = x - x.amax(1, keepdim=True)
    logp -= logp.exp().sum(1, keepdim=True).log()
    p = logp.exp()
    lp = logp.gather(1, s["t"][:, None])[:, 0]
    ent = -(p * logp).sum(1)
    if case["train"]:
        dx = -p * (s["dl"][:, None] + s["dh"][:, None] * (logp + ent[:, None]))
        dx.scatter_add_(1, s["t"][:, None], s["dl"][:, None])
        return lp, ent, dx.to(s["x"].dtype)
    if not case["top"]:
        return lp, ent
    where = []
    for _ in range(case["top"]):  # the first of equal logits each time
        where.append(x.argmax(1, keepdim=True))
        x = x.scatter(1, where[-1], float("-inf"))
    where = torch.cat(where, 1)
    return lp, ent, logp.gather(1, where), where


def _pairs(case):
    """Products of one query with one key, over all query heads."""
    n = 0
    for a, b in zip(*_lengths(case)):
        n += a * b - a * (a - 1) // 2 if case["causal"] else a * b
    return n * case["hq"]


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        n = case["tokens"] * (case["hq"] + case["hk"]) * case["dim"]
        per_token = case["tokens"] * case["axes"] * 8 + case["rot"] * 4
        if case["train"]:  # heads in and out, both gradients in and out; the heads are read for each direction
            return {"bytes": 2 * n * 5 + 2 * per_token, "flops": 24 * n}
        return {"bytes": 2 * n * 2 + per_token, "flops": 8 * n}
    if case["op"] == "logprobs":
        n = case["rows"] * case["vocab"]
        small = case["rows"] * (16 + 12 * case["top"])
        # the gradient has to read the logits again: its factors are the whole row's
        return {"bytes": size * n * (3 if case["train"] else 1) + small, "flops": (8 if case["train"] else 4) * n}
    nq, nk = _lengths(case)
    D, hq, hk = case["dim"], case["hq"], case["hk"]
    heads, cache = 2 * sum(nq) * hq * D, 2 * sum(nk) * hk * D
    if case["kind"] == "train":
        # forward: q, k, v in, o out; backward: q, k, v, o and its gradient in, three gradients out
        return {"bytes": heads * 6 + cache * 6, "flops": 14 * _pairs(case) * D}
    return {"bytes": 2 * heads + 2 * cache, "flops": 4 * _pairs(case) * D}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s, case)
    if case["op"] == "logprobs":
        return _exact_logprobs(s, case)
    return _exact_attention(s, case)


def _exact_rope(s, case):
    R, T = case["rot"], case["tokens"]
    axis = torch.zeros(R // 2, dtype=torch.long, device="cuda")
    at = 0
    for i, n in enumerate(_sections(case) or [R // 2]):
        axis[at:at + n] = i
        at += n
    pos = s["pos"].reshape(case["axes"], T)[axis].T.double()
    unit = torch.polar(torch.ones_like(pos), pos * s["freq"]).unsqueeze(1)  # e^(i angle)

    def turn(x, u):
        z = torch.complex(x[..., 0:R:2], x[..., 1:R:2]) if case["interleaved"] else \
            torch.complex(x[..., :R // 2], x[..., R // 2:R])
        z = z * u
        y = x.clone()
        if case["interleaved"]:
            y[..., 0:R:2], y[..., 1:R:2] = z.real, z.imag
        else:
            y[..., :R // 2], y[..., R // 2:R] = z.real, z.imag
        return y

    outs, grads, dws = [], [], []
    for x, name in ((s["q"], "q"), (s["k"], "k")):
        x = x.double()
        D = x.shape[-1]
        if case["norm"]:
            ms = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / D + EPS
            w = s["w" + name].double()
            outs.append(turn(x / ms.sqrt() * w, unit))
        else:
            outs.append(turn(x, unit))
        if not case["train"]:
            continue
        g = turn(s["d" + name].double(), unit.conj())
        if case["norm"]:
            dws.append((g * x / ms.sqrt()).sum((0, 1)))
            g = g * w
            g = g / ms.sqrt() - x * torch.linalg.vecdot(g, x).unsqueeze(-1) / (D * ms ** 1.5)
        grads.append(g)
    return tuple(outs + grads + dws)


def _exact_attention(s, case):
    nq, nk = _lengths(case)
    hq, D, train = case["hq"], case["dim"], case["kind"] == "train"
    share = hq // case["hk"]
    scale = 1 / math.sqrt(D)
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    dq, dk, dv = ((torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in "qkv") if train else (None,) * 3)
    first = first_k = 0
    for n, m in zip(nq, nk):
        for h in range(hq):
            K, V = s["k"][first_k:first_k + m, h // share].double(), s["v"][first_k:first_k + m, h // share].double()
            step = max(1, (1 << 27) // m)
            for a in range(first, first + n, step):
                b = min(a + step, first + n)
                Q = s["q"][a:b, h].double()
                logits = Q @ K.T * scale
                if case["causal"]:  # query i of n stands at key m - n + i
                    logits += torch.full_like(logits, -math.inf).triu(m - n + a - first + 1)
                P = torch.softmax(logits, 1)
                o[a:b, h] = P @ V
                if train:
                    G = s["do"][a:b, h].double()
                    dv[first_k:first_k + m, h // share] += P.T @ G
                    dS = P * (G @ V.T - torch.linalg.vecdot(G, o[a:b, h]).unsqueeze(1)) * scale
                    dq[a:b, h] = dS @ K
                    dk[first_k:first_k + m, h // share] += dS.T @ Q
        first += n
        first_k += case["room"] if case["kind"] == "cache" else m
    return (o, dq, dk, dv) if train else o


def _exact_logprobs(s, case):
    parts = []
    rows = max(1, (1 << 28) // case["vocab"])
    for a in range(0, case["rows"], rows):
        x = s["x"][a:a + rows]
        t = s["t"][a:a + rows].unsqueeze(1)
        logp = torch.log_softmax(x.double(), 1)
        p = torch.exp(logp)
        lp, ent = logp.gather(1, t).squeeze(1), -torch.linalg.vecdot(p, logp)
        if case["train"]:
            dl, dh = s["dl"][a:a + rows].double().unsqueeze(1), s["dh"][a:a + rows].double().unsqueeze(1)
            dx = torch.zeros_like(p).scatter(1, t, dl) - p * dl - dh * p * (logp + ent.unsqueeze(1))
            parts.append((lp, ent, dx))
        elif case["top"]:
            # by value, then by place: a stable sort of the largest
            best = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            parts.append((lp, ent, logp.gather(1, best), best))
        else:
            parts.append((lp, ent))
    return tuple(torch.cat(c) for c in zip(*parts))
