"""Host-side checks of the calls around a linear layer (no GPU needed): sizes of zero in
the norm and fp8 calls, and the packed bytes of a 4-bit weight."""
import copy

import pytest
import torch

import invariant_matmul_amd as imm
from invariant_matmul_amd import torch_ops

OK, INVALID = 0, 1
P = 4096  # an aligned address that no check reads


def test_arguments_of_rows_without_columns():
    """Without columns a call with nothing per row to write is done; one with a row's scale
    or rstd goes on, and its pointers are checked."""
    L = imm.lib()
    p, f8 = imm.rms_norm_plan(4, 0, "f16"), imm.rms_norm_plan(4, 0, "f16", "e4m3")

    def run(plan, scale=0, rstd=0):
        return L.rms_norm_run(plan.handle, 0, 0, 0, 0, scale, 0, rstd, None)

    assert run(p) == run(f8) == OK
    assert run(p, rstd=P + 2) == run(f8, scale=P + 2) == run(f8, scale=P, rstd=P + 2) == INVALID
    assert run(p, scale=P) == run(p, scale=P, rstd=P) == INVALID  # no scale of a 16-bit output
    none = imm.rms_norm_plan(0, 0, "f16", "e4m3")
    assert run(none) == run(none, scale=P) == OK

    def quantize(rows=4, scale=0):
        return L.quantize_rows(rows, 0, 0, 2, 0, 0, scale, None)

    assert quantize() == quantize(rows=0) == quantize(rows=0, scale=P) == OK
    assert quantize(scale=P + 1) == INVALID


def test_packed_bytes_of_a_4_bit_weight():
    size = imm.w4_packed_size(imm.w4_plan(1, 56, 256, "f16", 64))
    packed = torch.zeros(size, dtype=torch.uint8)
    w = torch_ops.W4Weight(packed, 56, 256, 64, torch.float16)
    for same in (w.to("cpu"), copy.deepcopy(w)):
        assert (same.N, same.K, same.group, same.dtype) == (56, 256, 64, torch.float16)
        assert torch.equal(same.packed, packed)
    torch_ops.W4Weight(packed[:0], 0, 256, 64, torch.float16)
    for bad in (packed[:-1], packed[:-16], torch.zeros(2 * size, dtype=torch.uint8)[::2], packed.view(4, -1),
                packed.view(torch.int8), packed.view(torch.int16)):
        with pytest.raises(ValueError):
            torch_ops.W4Weight(bad, 56, 256, 64, torch.float16)
    for sizes in ((72, 256, 64), (56, 384, 64), (56, 256, 32)):
        with pytest.raises(ValueError):
            torch_ops.W4Weight(packed, *sizes, torch.float16)
    with pytest.raises(imm.GemmError):
        torch_ops.W4Weight(packed, 56, 256, 48, torch.float16)
