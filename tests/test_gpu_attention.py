"""Attention and its gradients against the formula in 64 bits (bounds derived in
tests/decoder_oracle.py), and the bits of its rows: a prompt at once, in pieces and token by token."""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests import decoder_oracle as ref
from tests.helpers import dev

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
NAN, INF = float("nan"), float("inf")


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return ints(out)


def make(Tq, Tk, hq, hk, D, dt, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, s=std):
        return (torch.randn(*shape, generator=g) * s).to(DT[dt]).to(dev())

    return normal(Tq, hq, D), normal(Tk, hk, D), normal(Tk, hk, D, s=1.0), normal(Tq, hq, D, s=1.0)


def check(q, k, v, do, nq, nk, causal, scale=None, grads=True, max_q=None):
    """Packed sequences of nq queries and nk keys: o, lse and the gradients within their bounds."""
    D = q.shape[2]
    same = list(nq) == list(nk)
    cu_q, cu_k = starts(nq), starts(nk)
    o, saved = torch_ops.attention_forward(q, k, v, cu_q, None if same else cu_k, causal=causal, scale=scale, max_q=max_q)
    if grads:
        got = torch_ops.attention_backward(do, q, k, v, o, saved, cu_q, cu_k, causal=causal, scale=scale)
    a = b = 0
    for n, m in zip(nq, nk):
        want, tol = ref.attention_case(q[a:a + n], k[b:b + m], v[b:b + m], do[a:a + n], causal,
                                       D ** -0.5 if scale is None else scale)
        ref.close(o[a:a + n], want["o"], tol["o"], f"o of {n} over {m}")
        ref.close(saved.lse[a:a + n], want["lse"], tol["lse"], f"lse of {n} over {m}")
        if grads:
            for x, name, lo, hi in zip(got, ("dq", "dk", "dv"), (a, b, b), (a + n, b + m, b + m)):
                ref.close(x[lo:hi], want[name], tol[name], f"{name} of {n} over {m}")
        a, b = a + n, b + m
    return o, saved


# (queries, keys of each sequence): lengths of one, around steps (64), chunks (256) and tiles (128, 256);
# no keys, fewer keys than queries (rows that see nothing), empty sequences
LENGTHS = [([1], [1]), ([3], [3]), ([64], [64]), ([65], [65]), ([255, 1, 257], [255, 1, 257]), ([300], [300]),
           ([5, 0, 7], [5, 0, 7]), ([1, 1, 1], [700, 1, 256]), ([2, 9], [513, 260]), ([70], [20]), ([4, 3], [0, 3]),
           ([130, 600], [130, 600]), ([17], [1030])]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(4, 2, 128), (1, 1, 64), (5, 1, 96), (6, 2, 80), (2, 2, 8)])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_matches_the_formula(lengths, heads, causal, dt):
    nq, nk = lengths
    hq, hk, D = heads
    q, k, v, do = make(sum(nq), sum(nk), hq, hk, D, dt, sum(nq) * 7 + hq)
    check(q, k, v, do, nq, nk, causal)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_long_sequences(dt):
    nq = [2051, 640]
    q, k, v, do = make(sum(nq), sum(nq), 4, 1, 128, dt, 3)
    check(q, k, v, do, nq, nq, True)


@pytest.mark.parametrize("scale", [1e-3, 0.3, 1.0])
def test_scales(scale):
    q, k, v, do = make(200, 200, 2, 1, 64, "bf16", 4)
    check(q, k, v, do, [200], [200], True, scale)


@pytest.mark.parametrize("group,max_q", [(1, 1), (4, 1), (8, 1), (16, 4), (3, 5), (8, 8), (64, 1), (7, 9)])
def test_few_queries_over_a_cache(group, max_q):
    # every sequence has up to max_q new tokens over a cache with room
    hk, D, room = 2, 128, 1500
    new = [max_q, 1, max(1, max_q - 1), 1]
    lens = [room, 1, 257, 700]
    lens = [max(a, b) for a, b in zip(lens, new)]
    q, k, v, do = make(sum(new), room * 4, hk * group, hk, D, "bf16", 5 + group)
    for i, n in enumerate(lens):  # what lies behind a cache's end is not read
        k[i * room + n:(i + 1) * room] = NAN
        v[i * room + n:(i + 1) * room] = INF
    cu_k = ints([i * room for i in range(5)])
    o, saved = torch_ops.attention_forward(q, k, v, starts(new), cu_k, k_lens=ints(lens), max_q=max_q)
    many, _ = torch_ops.attention_forward(q, k, v, starts(new), cu_k, k_lens=ints(lens))
    a = 0
    for i, (n, m) in enumerate(zip(new, lens)):
        b = i * room
        want, tol = ref.attention_case(q[a:a + n], k[b:b + m], v[b:b + m], do[a:a + n], True, D ** -0.5)
        ref.close(o[a:a + n], want["o"], tol["o"], f"o {i}")
        ref.close(saved.lse[a:a + n], want["lse"], tol["lse"], f"lse {i}")
        a += n
    assert torch.equal(o, many)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (5, 1, 64), (3, 3, 96), (2, 1, 40)])
def test_pieces_have_the_bits_of_the_whole(heads, dt):
    hq, hk, D = heads
    n = 901
    q, k, v, _ = make(n, n, hq, hk, D, dt, 6)
    whole, (lse, _) = torch_ops.attention_forward(q, k, v)
    for t in (0, 1, 63, 64, 255, 256, 257, 512, 767, 900):  # token by token, over the cache so far
        one, (l1, _) = torch_ops.attention_forward(q[t:t + 1], k, v, ints([0, 1]), ints([0, n]), k_lens=ints([t + 1]), max_q=1)
        assert torch.equal(one[0], whole[t]) and torch.equal(l1[0], lse[t]), t
    for a, b in ((0, 100), (100, 107), (300, 700), (640, 901)):  # in pieces
        for max_q in (None, b - a):
            part = torch_ops.attention(q[a:b], k[:b], v[:b], ints([0, b - a]), ints([0, b]), max_q=max_q)
            assert torch.equal(part, whole[a:b]), (a, b)
    # beside other sequences, in other places
    q2, k2, v2, _ = make(333, 333, hq, hk, D, dt, 7)
    both = torch_ops.attention(torch.cat((q2, q)), torch.cat((k2, k)), torch.cat((v2, v)), ints([0, 333, 333 + n]))
    assert torch.equal(both[333:], whole)


def test_gradients_of_a_sequence_are_its_own():
    n, m = 300, 190
    q, k, v, do = make(n + m, n + m, 4, 2, 64, "bf16", 8)
    cu = ints([0, n, n + m])
    o, saved = torch_ops.attention_forward(q, k, v, cu)
    both = torch_ops.attention_backward(do, q, k, v, o, saved, cu)
    for lo, hi in ((0, n), (n, n + m)):
        o1, s1 = torch_ops.attention_forward(q[lo:hi], k[lo:hi], v[lo:hi])
        alone = torch_ops.attention_backward(do[lo:hi], q[lo:hi], k[lo:hi], v[lo:hi], o1, s1)
        assert all(torch.equal(a[lo:hi], b) for a, b in zip(both, alone))


def test_rows_and_keys_outside_sequences():
    q, k, v, do = make(200, 400, 4, 2, 64, "bf16", 9)
    cu_q, cu_k, lens = ints([10, 60, 150]), ints([20, 170, 330]), ints([100, 160])
    for max_q in (None, 8):
        if max_q:
            cu_q = ints([10, 17, 25])
        o, saved = torch_ops.attention_forward(q, k, v, cu_q, cu_k, k_lens=lens, max_q=max_q)
        first, last = int(cu_q[0]), int(cu_q[-1])
        out = torch.ones(200, dtype=torch.bool, device=dev())
        out[first:last] = False
        assert (o[out] == 0).all() and (saved.lse[out] == -INF).all()
        dq, dk, dv = torch_ops.attention_backward(do, q, k, v, o, saved, cu_q, cu_k, k_lens=lens)
        assert (dq[out] == 0).all()
        keys = torch.ones(400, dtype=torch.bool, device=dev())
        keys[20:120] = keys[170:330] = False
        assert (dk[keys] == 0).all() and (dv[keys] == 0).all()
        a = int(cu_q[0])
        for i, (b, m) in enumerate(((20, 100), (170, 160))):
            n = int(cu_q[i + 1]) - int(cu_q[i])
            want, tol = ref.attention_case(q[a:a + n], k[b:b + m], v[b:b + m], do[a:a + n], True, 0.125)
            for x, name, lo, hi in ((o, "o", a, a + n), (dq, "dq", a, a + n), (dk, "dk", b, b + m), (dv, "dv", b, b + m)):
                ref.close(x[lo:hi], want[name], tol[name], name)
            a += n


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_later_tokens_do_not_reach_earlier_rows(dt, bad):
    n = 333
    q, k, v, _ = make(n, n, 4, 2, 128, dt, 10)
    clean = torch_ops.attention(q, k, v)
    for at in (5, 64, 255, 300):
        k2, v2 = k.clone(), v.clone()
        v2[at, 1, 7] = bad
        k2[at + 3, 0] = bad
        o = torch_ops.attention(q, k2, v2)
        assert torch.equal(o[:at], clean[:at]), at
        assert torch.equal(o[at:at + 3, :2], clean[at:at + 3, :2])  # the other key head's
        seen = o[at:at + 3, 2:, 7].float()
        assert torch.isnan(seen).all() if bad != bad else (seen == bad).all(), at
        rest = torch.cat((o[at:at + 3, 2:, :7], o[at:at + 3, 2:, 8:]), 2)
        assert torch.equal(rest, torch.cat((clean[at:at + 3, 2:, :7], clean[at:at + 3, 2:, 8:]), 2))
        # the same rows as drafted tokens over a cache
        few = torch_ops.attention(q[at - 2:at + 3], k2[:at + 3], v2[:at + 3], ints([0, 5]), ints([0, at + 3]), max_q=5)
        assert torch.equal(few.nan_to_num(3, 4, 5), o[at - 2:at + 3].nan_to_num(3, 4, 5))


def test_masked_lowest_values():
    # logits of the type's lowest values, and one value throughout
    q, k, v, do = make(100, 100, 2, 1, 64, "bf16", 11)
    q[:] = 1.0
    k[::2] = -1e4
    check(q, k, v, do, [100], [100], True)
    k[:] = 2.0
    check(q, k, v, do, [100], [100], False)


def test_more_queries_than_said():
    for keys in (100, 2000):  # either kernel
        q, k, v, _ = make(9, 3 * keys, 2, 1, 64, "bf16", 12)
        o = torch_ops.attention(q, k, v, ints([0, 2, 9]), ints([0, keys, 3 * keys]), max_q=4)
        full = torch_ops.attention(q, k, v, ints([0, 2, 9]), ints([0, keys, 3 * keys]))
        assert torch.equal(o[:6], full[:6]) and torch.isnan(o[6:]).all() and torch.isfinite(full).all()


def test_contents_of_the_arrays_stay_inside():
    # values that do not ascend or pass the operands are clamped: nothing outside is read or written
    q, k, v, do = make(50, 60, 2, 1, 64, "bf16", 13)
    for cu_q, cu_k, lens in (([0, 90, 40], [0, 10, 1000], [5, 5000]), ([-5, 60, 50], [70, -3, 60], [-1, 9]),
                             ([30, 10, 2 ** 31 - 1], [0, 2 ** 31 - 1, -2 ** 31], [2 ** 31 - 1, 2 ** 31 - 1])):
        for max_q in (None, 3):
            o, saved = torch_ops.attention_forward(q, k, v, ints(cu_q), ints(cu_k), k_lens=ints(lens), max_q=max_q)
            torch_ops.attention_backward(do, q, k, v, o, saved, ints(cu_q), ints(cu_k), k_lens=ints(lens))
    torch.cuda.synchronize()


def test_views_of_a_fused_projection():
    T, hq, hk, D = 130, 4, 2, 64
    qkv = torch.randn(T, (hq + 2 * hk) * D, generator=torch.Generator().manual_seed(14)).bfloat16().to(dev())
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split((hq * D, hk * D, hk * D), 1))
    want = torch_ops.attention(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(torch_ops.attention(q, k, v), want)
    heads_first = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    assert torch.equal(torch_ops.attention(*heads_first), want)
    odd = [torch.empty(x.numel() + 1, dtype=x.dtype, device=dev())[1:].view(x.shape).copy_(x) for x in (q, k, v)]
    assert torch.equal(torch_ops.attention(*odd), want)
    one = k[:1].expand(T, hk, D)  # a broadcast key
    assert torch.equal(torch_ops.attention(q, one, v), torch_ops.attention(q, one.contiguous(), v))
    for n in (1, 3):
        last = torch_ops.attention(q[-n:], k, v, ints([0, n]), ints([0, T]), max_q=n)
        assert torch.equal(last, want[-n:])


def test_autograd_and_differences():
    n = 40
    q, k, v, do = make(n, n, 4, 2, 64, "bf16", 15)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    cu = ints([0, 13, n])
    o = torch_ops.attention(*leaves, cu)
    o.backward(do)
    o1, saved = torch_ops.attention_forward(q, k, v, cu)
    direct = torch_ops.attention_backward(do, q, k, v, o1, saved, cu)
    assert torch.equal(o.detach(), o1) and all(torch.equal(a.grad, b) for a, b in zip(leaves, direct))

    def loss(q, k, v):
        total = 0.0
        for a, b in ((0, 13), (13, n)):
            total = total + (ref.attend(q[a:b], k[a:b], v[a:b], True, 0.125)[0] * do[a:b].double()).sum()
        return total

    g = torch.Generator().manual_seed(16)
    bounds = [ref.attention_case(q[a:b], k[a:b], v[a:b], do[a:b], True, 0.125)[1] for a, b in ((0, 13), (13, n))]
    at = [t.double() for t in (q, k, v)]
    for i, name in enumerate(("dq", "dk", "dv")):
        d = torch.randn(at[i].shape, generator=g).double().to(dev())
        h = 1e-5
        up, down = ([t + s * h * d if j == i else t for j, t in enumerate(at)] for s in (1, -1))
        want = (loss(*up) - loss(*down)) / (2 * h)
        tol = (torch.cat([b[name] for b in bounds]) * d.abs()).sum() + 1e-6 * (1 + want.abs())
        assert abs((direct[i].double() * d).sum() - want) <= tol, name


def test_captured_and_replayed():
    q, k, v, do = make(64, 64, 4, 2, 64, "bf16", 17)
    cache_k, cache_v, _, _ = make(2 * 600, 2 * 600, 2, 2, 64, "bf16", 18)
    lens, cu_q, cu_k = ints([100, 599]), ints([0, 1, 2]), ints([0, 600, 1200])

    def step():
        one = torch_ops.attention(q[:2], cache_k, cache_v, cu_q, cu_k, k_lens=lens, max_q=1)
        o, saved = torch_ops.attention_forward(q, k, v)
        return (one, o, *torch_ops.attention_backward(do, q, k, v, o, saved))

    step()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        lens.copy_(ints([101 + 57 * i, 600 - i]))
        q.mul_(-1.0)
        torch.ones(1000, device=dev()).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_nothing_to_do_and_refusals():
    q, k, v, do = make(3, 5, 4, 2, 64, "bf16", 19)
    o, saved = torch_ops.attention_forward(q[:0], k, v)
    assert o.shape == (0, 4, 64) and saved.lse.shape == (0, 4)
    dq, dk, dv = torch_ops.attention_backward(do[:0], q[:0], k, v, o, saved)
    assert dq.shape == (0, 4, 64) and (dk == 0).all() and (dv == 0).all()
    o, saved = torch_ops.attention_forward(q, k[:0], v[:0])
    assert (o == 0).all() and (saved.lse == -INF).all()
    dq, dk, dv = torch_ops.attention_backward(do, q, k[:0], v[:0], o, saved)
    assert (dq == 0).all() and dk.shape == (0, 2, 64)
    cu = ints([0, 3])
    for args, kw in (((q.float(), k, v), {}), ((q, k.half(), v), {}), ((q, k, v[:4]), {}), ((q[:, :3], k, v), {}),
                     ((q.cpu(), k.cpu(), v.cpu()), {}), ((q[0], k, v), {}), ((q, k, v, None, cu), {}), ((q, k, v, cu.long()), {}),
                     ((q, k, v, cu.cpu()), {}), ((q, k, v, cu, ints([0, 1, 2])), {}), ((q, k, v, cu, cu), {"k_lens": ints([1, 2])}),
                     ((q[..., :12], k[..., :12], v[..., :12]), {}), ((q, k, v, ints([0])), {})):
        with pytest.raises(ValueError):
            torch_ops.attention(*args, **kw)
    wide = torch.zeros(2, 2, 136, dtype=torch.bfloat16, device=dev())
    with pytest.raises(ValueError):
        torch_ops.attention(wide, wide, wide)
    for scale in (0.0, -1.0, INF, NAN):
        with pytest.raises(RuntimeError):
            torch_ops.attention(q, k, v, scale=scale)
    with pytest.raises(ValueError):
        torch_ops.attention_backward(do, q, k, v, q, (saved.lse[:2], q), None)
