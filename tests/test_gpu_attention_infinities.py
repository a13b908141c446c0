"""Values of attention that are not finite: a row that sees one has it in its result, whatever weight the
row gives it, in each of the kernels and at every place of a row in its tile; a row that does not has the
bits that it has without."""
import pytest
import torch

from invariant_matmul_amd import torch_ops
from tests import decoder_oracle as ref
from tests.helpers import dev
from tests.test_gpu_attention import INF, NAN, ints, make
from tests.test_gpu_attention_kernels import groups, takes_few

pytestmark = pytest.mark.gpu

N, D = 700, 128
PLACES = (10, 64, 255, 300, 513)


def weights_of_every_size(hk, dt, rising):
    """Queries and keys whose logits spread over hundreds; rising: each later key has more, so that what came
    before falls to 0 again and again."""
    q, k, v, _ = make(N, N, hk, hk, D, dt, 40 + hk)
    q[:, :, 0] = 4.0
    at = torch.arange(N, device=dev(), dtype=torch.float32)
    grown = 3.0 * at if rising else 300.0 * torch.sin(at * 1.7)
    k[:, :, 0] = grown.to(k.dtype)[:, None]
    return q, k, v


@pytest.mark.parametrize("rising", [False, True])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hk", [2, 90])  # 16 and 32 rows a wave
def test_whatever_its_weight(hk, dt, bad, rising):
    q, k, v = weights_of_every_size(hk, dt, rising)
    assert (groups(q, k, 1) > 512) == (hk == 90) and not takes_few(q, k, 1, None)
    clean, saved = torch_ops.attention_forward(q, k, v)
    assert torch.isfinite(clean).all()
    for at in PLACES:
        v2 = v.clone()
        v2[at, 1, 7] = bad
        o, again = torch_ops.attention_forward(q, k, v2)
        odd = torch.zeros(N, hk, D, dtype=torch.bool, device=dev())
        odd[at:, 1, 7] = True
        assert torch.equal(o[~odd], clean[~odd]) and torch.equal(again.lse, saved.lse), at
        got = o[odd].float()
        assert torch.isnan(got).all() if bad != bad else (got == bad).all(), at
        # token by token over a longer cache, and a piece
        room = 9000
        kc, vc = (torch.zeros(room, 2, D, dtype=k.dtype, device=dev()) for _ in "kv")
        kc[:N], vc[:N] = k[:, :2], v2[:, :2]
        assert takes_few(q[:1, :2], kc, 1, 1)
        for t in (at - 1, at, at + 1, at + 31, 699):
            one = torch_ops.attention(q[t:t + 1, :2], kc, vc, ints([0, 1]), ints([0, room]), k_lens=ints([t + 1]), max_q=1)
            assert torch.equal(one.nan_to_num(3, 4, 5), o[t:t + 1, :2].nan_to_num(3, 4, 5)), (at, t)
        piece = torch_ops.attention(q[at - 2:at + 3, :2], kc, vc, ints([0, 5]), ints([0, room]), k_lens=ints([at + 3]), max_q=5)
        assert torch.equal(piece.nan_to_num(3, 4, 5), o[at - 2:at + 3, :2].nan_to_num(3, 4, 5)), at


@pytest.mark.parametrize("hk", [2, 90])
def test_several_and_of_both_signs(hk):
    q, k, v = weights_of_every_size(hk, "f16", False)
    v2 = v.clone()
    v2[20, 0, 3] = v2[400, 0, 3] = INF
    v2[30, 0, 5], v2[410, 0, 5] = INF, -INF
    v2[N - 1] = -INF
    o = torch_ops.attention(q, k, v2)
    whole = torch_ops.attention(q, k, v)
    assert torch.equal(o[:20], whole[:20]) and (o[20:-1, 0, 3] == INF).all() and torch.equal(o[:-1, 1:], whole[:-1, 1:])
    assert (o[30:410, 0, 5] == INF).all() and torch.isnan(o[410:, 0, 5]).all()
    assert torch.isnan(o[-1, 0, 3]) and (o[-1, 1:] == -INF).all()
    # without order every row sees all
    o = torch_ops.attention(q, k, v2, causal=False)
    assert torch.isnan(o[:, 0, 3]).all() and torch.isnan(o[:, 0, 5]).all() and (o[:, 1:] == -INF).all()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_the_finite_dimensions_are_the_formulas(dt):
    q, k, v, do = make(300, 300, 4, 2, 64, dt, 41)
    v2 = v.clone()
    v2[17, :, 9] = INF
    o = torch_ops.attention(q, k, v2)
    want, tol = ref.attention_case(q, k, v, do, True, 0.125)
    keep = torch.ones(64, dtype=torch.bool, device=dev())
    keep[9] = False
    ref.close(o[:, :, keep], want["o"][:, :, keep], tol["o"][:, :, keep], "o")
    assert (o[17:, :, 9] == INF).all()


@pytest.mark.parametrize("room", [200, 3000])
def test_other_sequences_and_rooms(room):
    # packed sequences that share a tile of rows, and free room that holds anything
    q, k, v, _ = make(90, 3 * room, 4, 2, 64, "f16", 42)
    cu_q, cu_k, lens = ints([0, 30, 31, 90]), ints([0, room, 2 * room, 3 * room]), ints([room - 50, 1, room - 1])
    assert takes_few(q, k, 3, 59) == (room == 3000)
    clean = torch_ops.attention(q, k, v, cu_q, cu_k, k_lens=lens, max_q=59)
    v2, k2 = v.clone(), k.clone()
    for a, b in ((room - 50, room), (room + 1, 2 * room), (3 * room - 1, 3 * room)):
        v2[a:b] = INF
        k2[a:b] = NAN
    assert torch.equal(torch_ops.attention(q, k2, v2, cu_q, cu_k, k_lens=lens, max_q=59), clean)
    v2[room] = INF
    o = torch_ops.attention(q, k2, v2, cu_q, cu_k, k_lens=lens, max_q=59)
    assert torch.equal(o[:30], clean[:30]) and torch.equal(o[31:], clean[31:]) and (o[30] == INF).all()
