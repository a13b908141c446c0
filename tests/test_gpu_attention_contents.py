"""Arrays of attention that do not ascend or pass the operands: nothing outside the outputs and the
workspace is written, by any of the kernels.  (Which rows and keys they read is checked on the host,
tests/test_attention_sequences_cpu.py.)"""
import pytest
import torch

import invariant_matmul_amd as imm
from tests.helpers import dev
from tests.test_gpu_attention import DT, ints, make

pytestmark = pytest.mark.gpu

BIG = 2 ** 31 - 1
BAD = [([0, 90, 40], [0, 10, 10 ** 6], [5, 5000]), ([-5, 60, 50], [70, -3, 60], [-1, 9]), ([30, 10, BIG], [0, BIG, -BIG - 1], [BIG, BIG]),
       ([0, BIG, 0], [0, BIG, 0], [BIG, -BIG - 1]), ([0, 1000, 5], [0, 0, 900], [BIG, BIG]), ([1000, 500, 0], [1000, 500, 0], [BIG, BIG])]
GUARD = 1 << 16  # bytes on each side


class Guarded:
    """Outputs inside larger buffers whose other bytes hold a pattern."""

    def __init__(self):
        self.all = []

    def __call__(self, *shape, dtype):
        size = torch.empty(0, dtype=dtype).element_size()
        n = size
        for s in shape:
            n *= s
        buf = torch.full((n + 2 * GUARD,), 0x5a, dtype=torch.uint8, device=dev())
        self.all.append((buf, n))
        return buf[GUARD:GUARD + n].view(dtype).view(shape)

    def untouched(self):
        return all((buf[:GUARD] == 0x5a).all() and (buf[GUARD + n:] == 0x5a).all() for buf, n in self.all)


# few rows; 16 and 32 rows a wave, sequences by length and in their order; more sequences than a wave has lanes
CALLS = [(50, 6000, 2, 1, 3, 2), (300, 300, 6, 2, 0, 2), (1200, 60, 56, 56, 0, 2), (2500, 2500, 8, 8, 0, 2), (1100, 1100, 120, 60, 0, 40),
         (70, 160000, 4, 2, 2, 80)]


@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("call", CALLS, ids=str)
def test_nothing_outside_is_written(call, heads_first):
    Tq, Tk, hq, hk, max_q, batch = call
    D, dt = 64, DT["bf16"]
    q, k, v, do = make(Tq, Tk, hq, hk, D, "bf16", Tq)
    if heads_first:
        q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    plan = imm.attention_plan(Tq, Tk, batch, hq, hk, D, "bf16", max_q=max_q)
    assert (imm.attention_workspace_size(plan) > 0) == (max_q > 0)
    guarded = Guarded()
    o, low, dq = (guarded(Tq, hq, D, dtype=dt) for _ in range(3))
    dk, dv = (guarded(Tk, hk, D, dtype=dt) for _ in range(2))
    lse = guarded(Tq, hq, dtype=torch.float32)
    ws = guarded(imm.attention_workspace_size(plan), dtype=torch.uint8) if max_q else None
    ws2 = guarded(imm.attention_backward_workspace_size(plan), dtype=torch.uint8)
    for cu_q, cu_k, lens in BAD:
        if batch > 2:  # the same values over and over
            cu_q, cu_k = ((c * batch)[:batch + 1] for c in (cu_q, cu_k))
            lens = lens * (batch // 2)
        arrays = ints(cu_q), ints(cu_k), ints(lens)
        for t in (o, low, lse):
            t.zero_()
        imm.attention_run(plan, q, k, v, o, *arrays, lse=lse, o_low=low, workspace=ws)
        imm.attention_backward(plan, do, q, k, v, o, lse, dq, dk, dv, *arrays, o_low=low, workspace=ws2)
        torch.cuda.synchronize()
        assert guarded.untouched(), (cu_q, cu_k, lens)
