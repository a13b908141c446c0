"""The operators between and behind a decoder's products as a program uses them: together, on other
streams, from several threads, captured into graphs, at operands past 32 bits."""
import threading

import pytest
import torch
from torch.autograd import forward_ad
from torch.nn import functional as F

import invariant_matmul_amd as imm
from invariant_matmul_amd import torch_ops
from tests import decoder_oracle as ref
from tests.helpers import dev

pytestmark = pytest.mark.gpu

# (the products of batch_invariant_mode take multiples of 8)
HQ, HK, D, HIDDEN, VOCAB = 8, 2, 64, 256, 1000


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def weights(dt, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std):
        return (torch.randn(*shape, generator=g) * std).to(dt).to(dev())

    return {"norm1": 1 + normal(HIDDEN, std=0.1), "qkv": normal((HQ + 2 * HK) * D, HIDDEN, std=HIDDEN ** -0.5),
            "wq": 1 + normal(D, std=0.1), "wk": 1 + normal(D, std=0.1), "out": normal(HIDDEN, HQ * D, std=(HQ * D) ** -0.5),
            "norm2": 1 + normal(HIDDEN, std=0.1), "head": normal(VOCAB, HIDDEN, std=3 * HIDDEN ** -0.5),
            "embed": normal(VOCAB, HIDDEN, std=1.0)}


FREQ = 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)


def layer(w, tokens, positions, attend):
    """One attention layer and the head's logits; attend(q, k, v) -> o."""
    x = w["embed"][tokens]
    qkv = F.linear(torch_ops.rms_norm(x, w["norm1"]), w["qkv"])
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split((HQ * D, HK * D, HK * D), 1))
    q, k = torch_ops.qk_norm_rope(q, k, positions, FREQ.to(x.device), w["wq"], w["wk"])
    h = x + F.linear(attend(q, k, v).flatten(1), w["out"])
    return F.linear(torch_ops.rms_norm(h, w["norm2"]), w["head"])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_a_prompt_and_its_tokens_one_by_one(dt):
    # logits of prefill, of pieces and of steps over the cache: the same bits
    w = weights(dt)
    T, room = 300, 2048
    tokens = torch.randint(0, VOCAB, (T,), generator=torch.Generator().manual_seed(1)).to(dev())
    at = torch.arange(T, device=dev())
    with torch.no_grad(), torch_ops.batch_invariant_mode():
        whole = layer(w, tokens, at, lambda q, k, v: torch_ops.attention(q, k, v))
        lp, ent, top_lp, top = torch_ops.token_logprobs(whole[:-1], tokens[1:], 5)
        cache = torch.zeros(2, room, HK, D, dtype=dt, device=dev())

        def over_cache(start):
            def attend(q, k, v):
                n = q.shape[0]
                cache[0, start:start + n], cache[1, start:start + n] = k, v
                return torch_ops.attention(q, cache[0], cache[1], ints([0, n]), ints([0, room]), k_lens=ints([start + n]),
                                           max_q=n)
            return attend

        for start, n in ((0, 100), (100, 7), (107, 1), (108, 1), (109, 91), (200, 1), (201, 99)):
            part = layer(w, tokens[start:start + n], at[start:start + n], over_cache(start))
            assert torch.equal(part, whole[start:start + n]), start
            known = min(n, T - 1 - start)
            if known > 0:
                got = torch_ops.token_logprobs(part[:known], tokens[start + 1:start + 1 + known], 5)
                for a, b in zip(got, (lp, ent, top_lp, top)):
                    assert torch.equal(a, b[start:start + known]), start
    # (a logarithm and differences of fp32 numbers up to 32: a few times 2^-24 32)
    want = ref.logprobs(whole[:-1], tokens[1:, None], 5)[0]
    assert (lp.double() - want[:, 0]).abs().max() < 2 ** -16


def test_a_training_step_of_packed_documents():
    # gradients of a loss through all operators: those of each document alone add up (in fp32, from the
    # gradients of the logits on), and they follow the loss's differences
    dt = torch.bfloat16
    w = weights(dt, 2)
    lens = [70, 1, 129]
    T = sum(lens)
    tokens = torch.randint(0, VOCAB, (T,), generator=torch.Generator().manual_seed(3)).to(dev())
    at = torch.cat([torch.arange(n) for n in lens]).to(dev())
    cu = ints([0, 70, 71, T])
    leaves = {n: t.clone().requires_grad_() for n, t in w.items()}

    def loss_of(w, tokens, at, cu):
        logits = layer(w, tokens, at, lambda q, k, v: torch_ops.attention(q, k, v, cu))
        lp, ent = torch_ops.token_logprobs(logits, tokens.roll(-1))
        return -lp.sum() - 0.01 * ent.sum(), logits

    with torch_ops.batch_invariant_mode():
        loss, logits = loss_of(leaves, tokens, at, cu)
        loss.backward()
        again = {n: t.clone().requires_grad_() for n, t in w.items()}
        loss_of(again, tokens, at, cu)[0].backward()
    for n, t in leaves.items():
        assert t.grad is not None and torch.isfinite(t.grad).all() and t.grad.abs().sum() > 0, n
        if n != "embed":  # (torch sums the embedding's gradient in no fixed order)
            assert torch.equal(t.grad, again[n].grad), n

    # the same layer in fp64
    def exact(p):
        x = p["embed"][tokens]

        def norm(x, w):
            return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w

        q, k, v = (t.unflatten(1, (-1, D)) for t in (norm(x, p["norm1"]) @ p["qkv"].T).split((HQ * D, HK * D, HK * D), 1))
        cos, sin = ref.turns(at, FREQ.to(dev()), None)
        q, k = ref.rotate(norm(q, p["wq"]), cos, sin, False), ref.rotate(norm(k, p["wk"]), cos, sin, False)
        o = torch.cat([ref.attend(q[a:b], k[a:b], v[a:b], True, D ** -0.5)[0] for a, b in ((0, 70), (70, 71), (71, T))])
        h = x + o.flatten(1) @ p["out"].T
        z = (norm(h, p["norm2"]) @ p["head"].T).log_softmax(1)
        lp = z.gather(1, tokens.roll(-1)[:, None]).sum()
        return -lp + 0.01 * (z.exp() * z).sum()

    wide = {n: t.double().requires_grad_() for n, t in w.items()}
    exact(wide).backward()
    # each of the dozen 16-bit results on the way is off by 2^-9 to 2^-8 of itself and these
    # add up as independent errors at least as large as the result: 2^-8 sqrt(12 * 2) < 2^-5
    for n, t in leaves.items():
        off = (t.grad.double() - wide[n].grad).norm() / wide[n].grad.norm()
        assert off < 2 ** -5, (n, float(off))


def calls(seed, dt=torch.bfloat16):
    """Inputs of the three operators and a call of all of them, forward and backward."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g).to(dt).to(dev())

    T, V = 70, 5003
    q, k, v, do = normal(T, HQ, D), normal(T, HK, D), normal(T, HK, D), normal(T, HQ, D)
    wq, wk, x, cache = normal(D), normal(D), normal(9, V), normal(2, 3000, HK, D)
    at = torch.randint(0, 5000, (T,), generator=g).to(dev())
    tok = torch.randint(0, V, (9,), generator=g).to(dev())
    freq = FREQ.to(dev())
    dl = torch.randn(9, generator=g).to(dev())
    cu_q, cu_k, lens = ints([0, 1, 3]), ints([0, 1500, 3000]), ints([1400, 700])

    def run():
        a, b = torch_ops.qk_norm_rope(q, k, at, freq, wq, wk)
        o, saved = torch_ops.attention_forward(a, b, v)
        dq, dk, dv = torch_ops.attention_backward(do, a, b, v, o, saved)
        few = torch_ops.attention(a[:3], cache[0], cache[1], cu_q, cu_k, k_lens=lens, max_q=2)
        grads = torch_ops.qk_norm_rope_backward(dq, dk, q, k, at, freq, wq, wk)
        lp, ent, norm = torch_ops.token_logprobs_forward(x, tok)
        tops = torch_ops.token_logprobs(x, tok, 7)
        dx = torch_ops.token_logprobs_backward(dl, None, x, tok, norm, ent)
        return (a, b, o, *saved, dv, few, *grads, lp, ent, norm, *tops, dx)

    return run, (q, x, lens, at)


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want, strict=True))


def test_captured_and_replayed():
    run, (q, x, lens, at) = calls(4)
    run()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs of the same call, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append((graph, out))
    for i in range(5):
        q.mul_(-0.5 if i % 2 else -2.0)
        x.add_(0.25)
        at.add_(1)
        lens.sub_(3)
        torch.ones(5000, device=dev()).sum().item()
        for graph, out in graphs if i % 2 else reversed(graphs):
            graph.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        assert all(same(out, want) for _, out in graphs), i


def test_a_captured_backward_pass():
    # forward and backward by autograd in one graph, of leaves that no graph made outside holds
    g = torch.Generator().manual_seed(8)
    q, k, v, wq = (torch.randn(*n, generator=g).bfloat16().to(dev()) for n in ((70, HQ, D), (70, HK, D), (70, HK, D), (D,)))
    at, tok, cu, freq = torch.arange(70, device=dev()), torch.arange(70, device=dev()), ints([0, 30, 70]), FREQ.to(dev())

    def step(leaves):
        q, k, v, wq = leaves
        a, b = torch_ops.qk_norm_rope(q, k, at, freq, wq, wq)
        lp, ent = torch_ops.token_logprobs(torch_ops.attention(a, b, v, cu).flatten(1), tok)
        return torch.autograd.grad(-lp.sum() - 0.1 * ent.sum(), leaves)

    def eager():
        return step([t.clone().requires_grad_() for t in (q, k, v, wq)])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        eager()
    torch.cuda.synchronize()
    leaves = [t.clone().requires_grad_() for t in (q, k, v, wq)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step(leaves)
    for i in range(4):
        with torch.no_grad():
            for t, leaf in zip((q, k, v, wq), leaves):
                t.mul_(-0.75)
                leaf.copy_(t)
        graph.replay()
        torch.ones(3000, device=dev()).sum().item()
        want = eager()
        torch.cuda.synchronize()
        assert same(grads, want), i


def test_on_other_streams_at_once():
    runs = [calls(5 + i)[0] for i in range(3)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [[] for _ in runs]
    for _ in range(4):
        for i, (run, stream) in enumerate(zip(runs, streams)):
            with torch.cuda.stream(stream):
                got[i].append(run())
    torch.cuda.synchronize()
    assert all(same(g, w) for gs, w in zip(got, want) for g in gs)


def test_several_threads():
    runs = [calls(9 + i)[0] for i in range(4)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    failed = []

    def work(run, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got = run()
                    torch.cuda.current_stream().synchronize()
                    if not same(got, want):
                        failed.append("other bits")
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(runs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_tangents_are_refused():
    g = torch.Generator().manual_seed(13)

    def normal(*shape):
        return torch.randn(*shape, generator=g).bfloat16().to(dev())

    q, k, v, do = normal(5, 4, 64), normal(5, 2, 64), normal(5, 2, 64), normal(5, 4, 64)
    wq, x = normal(64), normal(3, 100)
    at, tok = torch.arange(5, device=dev()), torch.tensor([1, 2, 3], device=dev())
    freq = FREQ.to(dev())
    o, saved = torch_ops.attention_forward(q, k, v)
    lp, ent, norm = torch_ops.token_logprobs_forward(x, tok)

    def ops(q, k, v, do, wq, freq, x, o, lse, o_low, norm, ent, lp):
        return {
            "qk_norm_rope": ((q, k, wq, freq), lambda: torch_ops.qk_norm_rope(q, k, at, freq, wq, wq)),
            "qk_norm_rope_backward": ((q, k, wq, freq, do),
                                      lambda: torch_ops.qk_norm_rope_backward(do, k, q, k, at, freq, wq, wq)),
            "attention": ((q, k, v), lambda: torch_ops.attention(q, k, v)),
            "attention_forward": ((q, k, v), lambda: torch_ops.attention_forward(q, k, v)),
            "attention_backward": ((do, q, k, v, o, lse, o_low), lambda: torch_ops.attention_backward(
                do, q, k, v, o, torch_ops.AttentionSaved(lse, o_low))),
            "token_logprobs": ((x,), lambda: torch_ops.token_logprobs(x, tok, 2)),
            "token_logprobs_forward": ((x,), lambda: torch_ops.token_logprobs_forward(x, tok)),
            "token_logprobs_backward": ((lp, x, norm, ent),
                                        lambda: torch_ops.token_logprobs_backward(lp, ent, x, tok, norm, ent)),
        }

    plain = (q, k, v, do, wq, freq, x, o, *saved, norm, ent, lp)
    with forward_ad.dual_level():
        for i, t in enumerate(plain):
            dual = forward_ad.make_dual(t, torch.ones_like(t))
            for name, (reads, f) in ops(*plain[:i], dual, *plain[i + 1:]).items():
                if any(a is dual for a in reads):
                    with pytest.raises(ValueError, match=name), torch.no_grad():
                        f()
                    with pytest.raises(ValueError, match=name):
                        f()


def test_gradients_asked_of_frequencies_and_twice():
    q, k = (torch.randn(3, 2, 64, device=dev()).bfloat16().requires_grad_() for _ in "qk")
    at, freq = torch.arange(3, device=dev()), FREQ.to(dev())
    with pytest.raises(ValueError, match="inv_freq"):
        torch_ops.qk_norm_rope(q, k, at, freq.clone().requires_grad_())
    # a second derivative would be left out of what create_graph=True gives
    x = torch.randn(3, 100, device=dev()).requires_grad_()
    for name, out, leaf in (("qk_norm_rope", torch_ops.qk_norm_rope(q, k, at, freq)[0], q), ("attention", torch_ops.attention(q, k, k), q),
                            ("token_logprobs", torch_ops.token_logprobs(x, at)[0], x)):
        (once,) = torch.autograd.grad(out.sum(), leaf, retain_graph=True)
        assert not once.requires_grad
        with pytest.raises(RuntimeError, match=name + " is differentiable once"):
            torch.autograd.grad(out.sum(), leaf, create_graph=True)


def test_heads_of_more_than_32_bits_of_bytes():
    T, hq, hk, dim = 600_000, 28, 4, 128  # 4.9 GB
    g = torch.Generator(device=dev()).manual_seed(14)
    qkv = torch.empty(T, hq + 2 * hk, dim, dtype=torch.bfloat16, device=dev()).normal_(generator=g)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]
    at = torch.randint(0, 10 ** 6, (T,), generator=g, device=dev())
    freq = 10000.0 ** (-torch.arange(0, dim, 2, device=dev(), dtype=torch.float64) / dim)
    w = torch.randn(dim, generator=g, device=dev()).bfloat16()
    a, b = torch_ops.qk_norm_rope(q, k, at, freq, w, w)
    dq, dk, dw, _ = torch_ops.qk_norm_rope_backward(a, b, q, k, at, freq, w, w)
    for lo in (0, 290_000, T - 50):
        part = slice(lo, lo + 50)
        a1, b1 = torch_ops.qk_norm_rope(q[part], k[part], at[part], freq, w, w)
        assert torch.equal(a[part], a1) and torch.equal(b[part], b1)
        g1 = torch_ops.qk_norm_rope_backward(a1, b1, q[part], k[part], at[part], freq, w, w)
        assert torch.equal(dq[part], g1[0]) and torch.equal(dk[part], g1[1])
    assert torch.isfinite(dw).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_logits_of_more_than_32_bits_of_bytes(dt):
    rows, V = 17_000, 131_072 if dt == torch.bfloat16 else 65_537  # 4.5 GB
    g = torch.Generator(device=dev()).manual_seed(15)
    x = torch.empty(rows, V, dtype=dt, device=dev()).normal_(generator=g)
    tok = torch.randint(0, V, (rows,), generator=g, device=dev())
    lp, ent, top_lp, top = torch_ops.token_logprobs(x, tok, 3)
    _, _, norm = torch_ops.token_logprobs_forward(x, tok)
    dl = torch.randn(rows, generator=g, device=dev())
    dx = torch_ops.token_logprobs_backward(dl, dl, x, tok, norm, ent)
    for i in (0, 8191, 16_500, rows - 1):
        one = torch_ops.token_logprobs(x[i:i + 1], tok[i:i + 1], 3)
        assert all(torch.equal(a[i:i + 1], b) for a, b in zip((lp, ent, top_lp, top), one)), i
        d1 = torch_ops.token_logprobs_backward(dl[i:i + 1], dl[i:i + 1], x[i:i + 1], tok[i:i + 1], norm[i:i + 1], ent[i:i + 1])
        assert torch.equal(dx[i:i + 1], d1), i
        want = ref.logprobs(x[i:i + 1], tok[i:i + 1, None], 3)
        assert torch.equal(top[i:i + 1], want[3]) and (lp[i].double() - want[0][0, 0]).abs() < 2 ** -16


def test_rows_of_logits_far_apart():
    V, rows, apart = 1000, 5, 1 << 30  # 2 GB between rows in 16 bits
    far = torch.empty(rows * apart, dtype=torch.bfloat16, device=dev())
    x = far.as_strided((rows, V), (apart, 1))
    g = torch.Generator().manual_seed(16)
    x.copy_(torch.randn(rows, V, generator=g))
    tok = torch.randint(0, V, (rows,), generator=g).to(dev())
    near = x.contiguous()
    assert same(torch_ops.token_logprobs(x, tok, 9), torch_ops.token_logprobs(near, tok, 9))
    _, ent, norm = torch_ops.token_logprobs_forward(x, tok)
    got = torch_ops.token_logprobs_backward(ent, ent, x, tok, norm, ent)
    assert torch.equal(got, torch_ops.token_logprobs_backward(ent, ent, near, tok, norm, ent))


def test_the_plans_of_the_package():
    # the library's own wrappers give what the operators give
    g = torch.Generator().manual_seed(17)

    def normal(*shape, dt=torch.bfloat16):
        return torch.randn(*shape, generator=g).to(dt).to(dev())

    def bytes_of(n):
        return torch.empty(n, dtype=torch.uint8, device=dev())

    T, V = 40, 5003
    q, k, v, do, w = normal(T, HQ, D), normal(T, HK, D), normal(T, HK, D), normal(T, HQ, D), normal(D)
    at, freq = torch.arange(T, device=dev()), FREQ.to(dev())
    plan = imm.head_rope_plan(T, HQ, HK, D, D, "bf16")
    a, b, dq, dk, dw, dw2 = (torch.empty_like(t) for t in (q, k, q, k, w, w))
    imm.head_rope_run(plan, q, k, at, freq, a, b, w, w)
    imm.head_rope_backward(plan, do, v, q, k, at, freq, dq, dk, w, w, dw, dw2, bytes_of(imm.head_rope_workspace_size(plan)))
    assert same((a, b), torch_ops.qk_norm_rope(q, k, at, freq, w, w))
    assert same((dq, dk, dw, dw2), torch_ops.qk_norm_rope_backward(do, v, q, k, at, freq, w, w))

    plan = imm.attention_plan(T, T, 2, HQ, HK, D, "bf16")
    cu = ints([0, 13, T])
    o, low, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(T, HQ, device=dev())
    imm.attention_run(plan, q, k, v, o, cu, cu, lse=lse, o_low=low)
    want, saved = torch_ops.attention_forward(q, k, v, cu)
    assert same((o, lse, low), (want, *saved))
    dv = torch.empty_like(v)
    imm.attention_backward(plan, do, q, k, v, o, lse, dq, dk, dv, cu, cu, o_low=low,
                           workspace=bytes_of(imm.attention_backward_workspace_size(plan)))
    assert same((dq, dk, dv), torch_ops.attention_backward(do, q, k, v, o, saved, cu))
    keys, values = normal(3000, HK, D), normal(3000, HK, D)
    cu_q, cu_k, lens = ints([0, 1, 3]), ints([0, 1500, 3000]), ints([1400, 700])
    plan = imm.attention_plan(3, 3000, 2, HQ, HK, D, "bf16", max_q=2)
    size = imm.attention_workspace_size(plan)
    assert size > 0
    imm.attention_run(plan, q[:3], keys, values, o[:3], cu_q, cu_k, lens, workspace=bytes_of(size))
    assert torch.equal(o[:3], torch_ops.attention(q[:3], keys, values, cu_q, cu_k, k_lens=lens, max_q=2))

    x, tok, dl = normal(9, V), torch.randint(0, V, (9,), generator=g).to(dev()), normal(9, dt=torch.float32)
    plan = imm.logprobs_plan(9, V, "bf16", 1, 4)
    lp, ent, norm = (torch.empty(n, device=dev()) for n in (9, 9, (9, 2)))
    top_lp, top = torch.empty(9, 4, device=dev()), torch.empty(9, 4, dtype=torch.int64, device=dev())
    size = imm.logprobs_workspace_size(plan)
    imm.logprobs_run(plan, x, tok, lp, ent, norm, top_lp, top, workspace=bytes_of(size) if size else None)
    assert same((lp, ent, top_lp, top), torch_ops.token_logprobs(x, tok, 4))
    dx = torch.empty_like(x)
    plan = imm.logprobs_plan(9, V, "bf16", 1, 0)
    imm.logprobs_backward(plan, x, tok, norm, ent, dx, dl, None)
    assert torch.equal(dx, torch_ops.token_logprobs_backward(dl, None, x, tok, norm, ent))
