"""Attention's kernels at sizes that choose each of them: few rows, 16 rows a wave, 32 rows a wave, and
sequences taken by length.  The bits are the same; each is checked against the formula too."""
import pytest
import torch

import invariant_matmul_amd as imm
from invariant_matmul_amd import torch_ops
from tests import decoder_oracle as ref
from tests.helpers import dev
from tests.test_gpu_attention import DT, INF, NAN, check, ints, make, starts

pytestmark = pytest.mark.gpu


def takes_few(q, k, batch, max_q):
    """Whether the kernel of few rows takes such a call: it alone has a workspace."""
    dt = {v: n for n, v in DT.items()}[q.dtype]
    return imm.attention_workspace_size(imm.attention_plan(q.shape[0], k.shape[0], batch, q.shape[1], k.shape[1], q.shape[2], dt,
                                                           max_q=max_q or 0)) > 0


def groups(q, k, batch):
    """Workgroups of 128 rows: waves take 32 rows from 513 on, sequences go by length up to 2048."""
    return (q.shape[0] * (q.shape[1] // k.shape[1]) // 128 + batch) * k.shape[1]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(96, 48, 128), (64, 64, 64), (60, 60, 96), (64, 64, 8)])
@pytest.mark.parametrize("lengths", [([700, 1, 257, 142], [700, 1, 257, 142]), ([1100], [1100]), ([64, 900, 0, 200], [700, 20, 9, 513])],
                         ids=str)
def test_32_rows_a_wave(lengths, heads, causal, dt):
    nq, nk = lengths
    hq, hk, D = heads
    q, k, v, do = make(sum(nq), sum(nk), hq, hk, D, dt, sum(nq) + hq)
    assert groups(q, k, len(nq)) > 512 and not takes_few(q, k, len(nq), None)
    o, saved = check(q, k, v, do, nq, nk, causal)
    grads = torch_ops.attention_backward(do, q, k, v, o, saved, starts(nq), starts(nk), causal=causal)
    # without what the backward pass takes, and a few key heads alone (16 rows or keys a wave)
    assert torch.equal(torch_ops.attention(q, k, v, starts(nq), starts(nk), causal=causal), o)
    g = hq // hk
    for lo in (0, hk - 3):
        part = q[:, lo * g:(lo + 3) * g], k[:, lo:lo + 3], v[:, lo:lo + 3]
        assert groups(*part[:2], len(nq)) <= 512
        o1, s1 = torch_ops.attention_forward(*part, starts(nq), starts(nk), causal=causal)
        assert torch.equal(o1, o[:, lo * g:(lo + 3) * g]) and torch.equal(s1.lse, saved.lse[:, lo * g:(lo + 3) * g])
        assert torch.equal(s1.o_low, saved.o_low[:, lo * g:(lo + 3) * g])
        alone = torch_ops.attention_backward(do[:, lo * g:(lo + 3) * g], *part, o1, s1, starts(nq), starts(nk), causal=causal)
        for one, all_, h in zip(alone, grads, (g, 1, 1)):
            assert torch.equal(one, all_[:, lo * h:(lo + 3) * h])


def test_32_rows_a_wave_and_bad_values():
    n, hk = 1300, 56
    q, k, v, _ = make(n, n, hk, hk, 128, "bf16", 30)
    assert groups(q, k, 1) > 512
    clean = torch_ops.attention(q, k, v)
    for at, bad in ((5, NAN), (64, INF), (700, -INF)):
        k2, v2 = k.clone(), v.clone()
        v2[at, 1, 7] = bad
        k2[at + 3, 0] = bad
        o = torch_ops.attention(q, k2, v2)
        assert torch.equal(o[:at], clean[:at]) and torch.equal(o[at:at + 3, 2:], clean[at:at + 3, 2:])
        assert torch.equal(o[:, 2:], clean[:, 2:])
        seen = o[at:at + 3, 1, 7].float()
        assert torch.isnan(seen).all() if bad != bad else (seen == bad).all(), at


def sequences(count, seed):
    """Lengths 0 to 40, some longer."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, 41, (count,), generator=g)
    lens[count // 3] = 300
    lens[-1] = 131
    return lens.tolist()


@pytest.mark.parametrize("count", [29, 30, 31, 61, 62, 63, 64, 100, 127, 4095, 5000])
def test_many_sequences(count):
    nq = sequences(count, count)
    q, k, v, do = make(sum(nq), sum(nq), 4, 2, 64, "bf16", count)
    cu = starts(nq)
    o, saved = torch_ops.attention_forward(q, k, v, cu)
    grads = torch_ops.attention_backward(do, q, k, v, o, saved, cu)
    at = cu.tolist()
    for i in sorted({0, 1, count // 3, count // 2, count - 2, count - 1, *range(5, count, max(1, count // 23))}):
        lo, hi = at[i], at[i + 1]
        if lo == hi:
            continue
        part = q[lo:hi], k[lo:hi], v[lo:hi]
        want, tol = ref.attention_case(*part, do[lo:hi], True, 0.125)
        for x, name in zip((o, saved.lse, *grads), ("o", "lse", "dq", "dk", "dv")):
            ref.close(x[lo:hi], want[name], tol[name], f"{name} of sequence {i} of {count}")


@pytest.mark.parametrize("count", [2, 62, 63, 100, 5000])
def test_many_sequences_with_a_new_token(count):
    room, hk, D = 700, 1, 128
    g = torch.Generator(device=dev()).manual_seed(count)
    q, k, v = (torch.randn(n, h, D, generator=g, device=dev()).bfloat16() for n, h in ((count, 2), (count * room, hk), (count * room, hk)))
    lens = torch.randint(0, room + 1, (count,), generator=torch.Generator().manual_seed(count))
    lens[0], lens[-1] = room, 1
    assert takes_few(q, k, count, 1)
    cu_q = torch.arange(count + 1, dtype=torch.int32, device=dev())
    o, saved = torch_ops.attention_forward(q, k, v, cu_q, cu_q * room, k_lens=lens.int().to(dev()), max_q=1)
    for i in sorted({0, 1, count - 2, count - 1, *range(0, count, max(1, count // 23))}):
        b, m = i * room, int(lens[i])
        want, tol = ref.attention_case(q[i:i + 1], k[b:b + m], v[b:b + m], q[i:i + 1], True, D ** -0.5)
        ref.close(o[i:i + 1], want["o"], tol["o"], f"o of sequence {i} of {count}")
        ref.close(saved.lse[i:i + 1], want["lse"], tol["lse"], f"lse of sequence {i} of {count}")


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_few_rows_and_bad_values(bad):
    m = 3000
    q, k, v, _ = make(5, m, 4, 2, 128, "bf16", 31)
    cu_q, cu_k = ints([0, 5]), ints([0, m])
    assert takes_few(q, k, 1, 5)
    clean = torch_ops.attention(q, k, v, cu_q, cu_k, max_q=5)
    # query t sees keys up to m - 5 + t: a bad value at the third's last key
    k2, v2 = k.clone(), v.clone()
    v2[m - 3, 1, 7] = bad
    k2[m - 3, 0] = bad
    o = torch_ops.attention(q, k2, v2, cu_q, cu_k, max_q=5)
    assert torch.equal(o[:2], clean[:2])
    assert torch.equal(o[2:, 2:, :7], clean[2:, 2:, :7]) and torch.equal(o[2:, 2:, 8:], clean[2:, 2:, 8:])
    seen = o[2:, 2:, 7].float()
    assert torch.isnan(seen).all() if bad != bad else (seen == bad).all()


def test_few_rows_outside_sequences():
    q, k, v, do = make(30, 9000, 4, 2, 128, "bf16", 32)
    cu_q, cu_k, lens = ints([10, 17, 25]), ints([20, 4170, 8330]), ints([3999, 4160])
    assert takes_few(q, k, 2, 8)
    o, saved = torch_ops.attention_forward(q, k, v, cu_q, cu_k, k_lens=lens, max_q=8)
    assert (o[:10] == 0).all() and (o[25:] == 0).all()
    assert (saved.lse[:10] == -INF).all() and (saved.lse[25:] == -INF).all()
    for a, e, b, m in ((10, 17, 20, 3999), (17, 25, 4170, 4160)):
        want, tol = ref.attention_case(q[a:e], k[b:b + m], v[b:b + m], do[a:e], True, 128 ** -0.5)
        ref.close(o[a:e], want["o"], tol["o"], "o")
        ref.close(saved.lse[a:e], want["lse"], tol["lse"], "lse")


def test_contents_of_the_arrays_stay_inside_in_each_kernel():
    bad = (([0, 90, 40], [0, 10, 10 ** 6], [5, 5000]), ([-5, 60, 50], [70, -3, 60], [-1, 9]),
           ([30, 10, 2 ** 31 - 1], [0, 2 ** 31 - 1, -2 ** 31], [2 ** 31 - 1, 2 ** 31 - 1]),
           ([0, 2 ** 31 - 1, 0], [0, 2 ** 31 - 1, 0], [2 ** 31 - 1, -2 ** 31]))
    for (Tq, Tk, hq, hk), max_q, few in (((50, 6000, 2, 1), 3, True), ((1200, 60, 56, 56), None, False), ((2500, 2500, 8, 8), None, False)):
        q, k, v, do = make(Tq, Tk, hq, hk, 64, "bf16", 33)
        assert takes_few(q, k, 2, max_q) == few
        for cu_q, cu_k, lens in bad:
            o, saved = torch_ops.attention_forward(q, k, v, ints(cu_q), ints(cu_k), k_lens=ints(lens), max_q=max_q)
            torch_ops.attention_backward(do, q, k, v, o, saved, ints(cu_q), ints(cu_k), k_lens=ints(lens))
        torch.cuda.synchronize()


def test_a_cache_past_32_bits_of_bytes():
    # the second sequence's rows begin at byte 5.1e9; its keys against those of a small cache
    rows, D = 20_000_000, 128
    k, v = (torch.zeros(rows, 1, D, dtype=torch.bfloat16, device=dev()) for _ in "kv")
    q, ks, vs, do = make(3000, 1500, 4, 1, D, "bf16", 34)
    lo = rows - 1500
    k[lo:], v[lo:] = ks, vs
    cu_k = ints([0, lo, rows])
    for max_q, cu_q in ((1, [0, 1, 2]), (3, [0, 1, 4]), (None, [0, 1, 3000])):
        n = cu_q[-1]
        assert takes_few(q[:n], k, 2, max_q) == (n < 5)
        o, saved = torch_ops.attention_forward(q[:n], k, v, ints(cu_q), cu_k, k_lens=ints([700, 1500]), max_q=max_q)
        want, (lse, _) = torch_ops.attention_forward(q[1:n], ks, vs, ints([0, n - 1]), ints([0, 1500]), max_q=max_q)
        assert (o[0] == 0).all() and torch.equal(o[1:], want) and torch.equal(saved.lse[1:], lse)
    # one sequence of 20 million keys, one of which has all the weight
    k[:], v[:] = 0, 1
    at = 17_500_000
    q[:] = 1
    k[at], v[at] = 30, vs[0]
    for length, found in ((rows, True), (at + 1, True), (at, False)):
        o = torch_ops.attention(q[:1], k, v, ints([0, 1]), ints([0, rows]), k_lens=ints([length]), max_q=1)
        assert torch.equal(o[0], vs[0].expand(4, D) if found else torch.ones(4, D, dtype=o.dtype, device=dev())), length


def test_heads_4_gb_apart():
    rows, n, D = 17_000_000, 300, 128
    far = torch.empty(2, rows, 1, D, dtype=torch.bfloat16, device=dev())
    q, k, v, do = make(n, n, 4, 2, D, "bf16", 35)
    want = torch_ops.attention(q, k, v)
    for x in (k, v):
        far[:, :n, 0] = x.transpose(0, 1)
        view = far[:, :n, 0].transpose(0, 1)
        args = (view, v) if x is k else (k, view)
        assert torch.equal(torch_ops.attention(q, *args), want)
        assert torch.equal(torch_ops.attention(q[-2:], *args, ints([0, 2]), ints([0, n]), max_q=2), want[-2:])
    far[:, :n, 0] = q[:, ::2].transpose(0, 1)
    view = far[:, :n, 0].transpose(0, 1)
    o, saved = torch_ops.attention_forward(view, k, v)
    assert torch.equal(o, want[:, ::2])
    got = torch_ops.attention_backward(do[:, ::2].contiguous(), view, k, v, o, saved)
    same = torch_ops.attention_backward(do[:, ::2].contiguous(), q[:, ::2].contiguous(), k, v, o, saved)
    assert all(torch.equal(a, b) for a, b in zip(got, same))


def test_more_rows_than_a_launch_has_threads():
    # 2^28 rows and heads: 16 lanes each for delta, and a wave each where results are joined
    T, hq, D = (1 << 24) + 5, 16, 8
    g = torch.Generator(device=dev()).manual_seed(36)
    q, do = (torch.empty(T, hq, D, dtype=torch.bfloat16, device=dev()).normal_(generator=g) for _ in range(2))
    k, v = (torch.empty(9, 1, D, dtype=torch.bfloat16, device=dev()).normal_(generator=g) for _ in range(2))
    o, saved = torch_ops.attention_forward(q, k, v, causal=False)
    dq, _, _ = torch_ops.attention_backward(do, q, k, v, o, saved, causal=False)
    for lo in (0, T // 2, T - 50):
        part = slice(lo, lo + 50)
        o1, s1 = torch_ops.attention_forward(q[part], k, v, causal=False)
        assert torch.equal(o[part], o1) and torch.equal(saved.lse[part], s1.lse)
        assert torch.equal(dq[part], torch_ops.attention_backward(do[part], q[part], k, v, o1, s1, causal=False)[0])
    assert takes_few(q, k, 2, 1)
    few = torch_ops.attention(q, k, v, ints([T - 3, T - 2, T - 1]), ints([0, 4, 9]), max_q=1)
    assert (few[:T - 3] == 0).all() and (few[T - 1] == 0).all()
    assert torch.equal(few[T - 2], torch_ops.attention(q[T - 2:T - 1], k[4:], v[4:])[0])


@pytest.mark.parametrize("nq,nk", [([5], [3000]), ([1, 3, 2], [2500, 2900, 2100])], ids=str)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_gradients_of_few_rows(nq, nk, dt):
    q, k, v, do = make(sum(nq), sum(nk), 8, 2, 128, dt, 37)
    assert takes_few(q, k, len(nq), max(nq))
    check(q, k, v, do, nq, nk, True, max_q=max(nq))


@pytest.mark.parametrize("heads", [(64, 1, 64), (100, 1, 128), (129, 1, 8), (146, 2, 40)])
def test_many_heads_of_a_group(heads):
    # more heads of a group than a step has rows
    hq, hk, D = heads
    nq, nk = [70, 1, 33], [70, 5, 90]
    q, k, v, do = make(sum(nq), sum(nk), hq, hk, D, "bf16", hq)
    for causal in (True, False):
        check(q, k, v, do, nq, nk, causal)
