"""Host-side checks of the calls around a linear layer (no GPU needed): what
the C ABI and the torch operators refuse before anything is enqueued."""
import os
import re

import pytest
import torch

import invariant_matmul_amd as imm
from invariant_matmul_amd import build, torch_ops
from tests.lds_read_check import file_hazards

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "invariant_matmul.h")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 4096  # an aligned address that no check reads


def test_tile_kernels_have_no_in_flight_read_hazard():
    """The 4-bit tile kernels issue LDS reads the compiler does not track (see
    tests/lds_read_check.py)."""
    if not os.path.exists(build.W4_ASM):
        pytest.skip("device assembly not built (run invariant_matmul_amd.build)")
    with open(build.W4_ASM) as f:
        text = f.read()
    hazards, n = file_hazards(text, "w4_tile_kernel")
    assert n >= 12, n
    assert not hazards, {k[:90]: list(v.items())[:3] for k, v in list(hazards.items())[:5]}
    # a spilled register would be stored before its read has landed
    spills = re.findall(r"\.vgpr_spill_count:\s+(\d+)", text)
    assert len(spills) >= n and set(spills) == {"0"}, spills


def status(call, *args, **kw):
    try:
        call(*args, **kw)
        return OK
    except imm.GemmError as e:
        return e.status


def test_library_exports_the_layer_calls():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)
    names = set(re.findall(r"\b((?:rms_norm|quantize|w4)_[a-z_0-9]+)\s*\(", text))
    assert names == set(imm.LAYER_SYMBOLS)
    for n in names:
        assert hasattr(imm.lib(), n), n


@pytest.mark.parametrize("args,want", [
    ((4, 64, "bf16"), OK), ((0, 64, "f16"), OK), ((4, 0, "f16"), OK), ((4, 32768, "f16"), OK),
    ((-1, 64, "f16"), INVALID), ((4, -8, "f16"), INVALID), ((4, 60, "f16"), UNSUPPORTED),
    ((4, 32776, "f16"), UNSUPPORTED), ((1 << 31, 64, "f16"), UNSUPPORTED),
    ((4, 64, "f32"), UNSUPPORTED), ((4, 64, "e4m3"), UNSUPPORTED), ((4, 64, "f16", "bf16"), UNSUPPORTED),
    ((4, 64, "f16", "f32"), UNSUPPORTED), ((4, 64, "f16", "e4m3"), OK), ((4, 64, "bf16", "e5m2"), OK),
    ((4, 72, "f16", "e4m3"), UNSUPPORTED),
    ((4, 64, "f16", "f16", -1e-6), UNSUPPORTED), ((4, 64, "f16", "f16", float("inf")), UNSUPPORTED),
    ((4, 64, "f16", "f16", 0.0), OK),
])
def test_rms_norm_plan_arguments(args, want):
    assert status(imm.rms_norm_plan, *args) == want


def test_rms_norm_run_arguments():
    L = imm.lib()
    assert L.rms_norm_plan(4, 64, 0, 0, 1e-6, None) == INVALID
    p = imm.rms_norm_plan(4, 64, "f16")
    f8 = imm.rms_norm_plan(4, 64, "f16", "e4m3")

    def run(plan, x=P, r=0, w=0, out=P, scale=0, rout=0, rstd=0):
        return L.rms_norm_run(plan.handle if plan else None, x, r, w, out, scale, rout, rstd, None)

    assert run(None) == INVALID
    assert run(p, x=0) == run(p, out=0) == run(p, x=P + 8) == run(p, out=P + 2) == INVALID
    assert run(p, w=P + 8) == run(p, rstd=P + 2) == INVALID
    assert run(p, r=P) == run(p, rout=P) == run(p, r=P + 8, rout=P) == run(p, r=P, rout=P + 8) == INVALID
    assert run(p, scale=P) == INVALID                      # no scale of a 16-bit output
    assert run(f8) == run(f8, scale=P + 2) == INVALID      # an fp8 output needs one
    assert run(imm.rms_norm_plan(0, 64, "f16"), x=0, out=0) == OK
    assert run(imm.rms_norm_plan(4, 0, "f16"), x=0, out=0) == OK


def test_rms_norm_backward_arguments():
    L = imm.lib()
    p = imm.rms_norm_plan(100, 64, "f16")
    need = p.workspace_bytes
    assert need % (64 * 4) == 0 and need > 0
    assert imm.rms_norm_plan(0, 64, "f16").workspace_bytes == 0
    assert imm.rms_norm_plan(4, 64, "f16", "e4m3").workspace_bytes == 0
    assert L.rms_norm_workspace_size(None) == 0

    def run(plan=p, dy=P, h=P, w=0, rstd=P, dh=0, dx=P, dw=0, ws=0, n=0):
        return L.rms_norm_backward(plan.handle if plan else None, dy, h, w, rstd, dh, dx, dw, ws, n, None)

    assert run(None) == INVALID
    assert run(imm.rms_norm_plan(4, 64, "f16", "e4m3")) == UNSUPPORTED
    for bad in ({"dy": 0}, {"h": 0}, {"rstd": 0}, {"dx": 0}, {"dy": P + 8}, {"h": P + 8}, {"w": P + 8},
                {"rstd": P + 2}, {"dh": P + 8}, {"dx": P + 8}, {"dw": P + 8, "ws": P, "n": need},
                {"dw": P, "ws": P + 8, "n": need}):
        assert run(**bad) == INVALID, bad
    assert run(dw=P) == run(dw=P, ws=P, n=need - 1) == WORKSPACE
    assert run(imm.rms_norm_plan(0, 64, "f16"), dy=0, h=0, rstd=0, dx=0) == OK


def test_quantize_rows_arguments():
    L = imm.lib()

    def run(rows=4, cols=64, i=0, o=2, x=P, q=P, s=P):
        return L.quantize_rows(rows, cols, i, o, x, q, s, None)

    assert run(rows=-1) == run(x=0) == run(q=0) == run(s=0) == run(x=P + 8) == run(s=P + 2) == INVALID
    assert run(o=0) == run(o=4) == run(i=4) == run(i=2) == run(cols=72) == UNSUPPORTED
    assert run(cols=32784) == UNSUPPORTED
    assert run(rows=0, x=0, q=0, s=0) == OK


def test_scaled_product_arguments():
    L = imm.lib()
    plan = imm.gemm_plan_ex2(4, 64, 128, "e4m3", "bf16", flags=imm.PLAN_B_TRANSPOSED)

    def run(p=plan, a=P, b=P, rs=P, cs=P, bias=0, c=P):
        h = p.handle if p else None
        return L.gemm_run_scaled(h, a, b, rs, cs, bias, c, None)

    assert run(None) == INVALID
    for bad in ({"a": 0}, {"b": 0}, {"c": 0}, {"rs": 0}, {"cs": 0}, {"a": P + 8}, {"b": P + 4}, {"c": P + 2},
                {"rs": P + 2}, {"cs": P + 1}, {"bias": P + 2}):
        assert run(**bad) == INVALID, bad
    for other in (imm.gemm_plan_ex2(4, 64, 128, "e4m3", "bf16"),
                  imm.gemm_plan_ex2(4, 64, 128, "f16", "f16", flags=imm.PLAN_B_TRANSPOSED)):
        assert run(other) == UNSUPPORTED
    empty = imm.gemm_plan_ex2(0, 64, 128, "e4m3", "bf16", flags=imm.PLAN_B_TRANSPOSED)
    assert run(empty, a=0, b=0, rs=0, cs=0, c=0) == OK


@pytest.mark.parametrize("args,want", [
    ((4, 64, 256, "bf16", 128), OK), ((0, 64, 256, "f16", 64), OK), ((4, 0, 256, "f16", 32), OK),
    ((4, 64, 0, "f16", 32), OK), ((4, 8, 96, "f16", 32), OK), ((-1, 64, 256, "f16", 128), INVALID),
    ((4, -8, 256, "f16", 128), INVALID), ((4, 64, -128, "f16", 128), INVALID),
    ((4, 60, 256, "f16", 128), UNSUPPORTED), ((4, 64, 192, "f16", 128), UNSUPPORTED),
    ((4, 64, 256, "f16", 16), UNSUPPORTED), ((4, 64, 256, "f16", 256), UNSUPPORTED),
    ((4, 64, 256, "f16", 0), UNSUPPORTED), ((4, 64, 256, "f16", -32), UNSUPPORTED),
    ((4, 64, 256, "f32", 128), UNSUPPORTED), ((4, 64, 256, "e4m3", 128), UNSUPPORTED),
    ((1 << 31, 64, 256, "f16", 128), UNSUPPORTED), ((1 << 30, 1 << 20, 256, "f16", 128), UNSUPPORTED),
    ((4, 1 << 30, 1 << 20, "f16", 128), UNSUPPORTED), ((4, 1 << 22, 128, "f16", 128), UNSUPPORTED),
    ((1 << 30, 128, 128, "f16", 128), UNSUPPORTED), (((1 << 30) - 64, 128, 128, "f16", 128), OK),
    ((4, 4000000, 128, "f16", 128), OK), ((4, 64, 1 << 25, "f16", 128), UNSUPPORTED), ((4, 64, 33000064, "f16", 32), OK),
])
def test_w4_plan_arguments(args, want):
    assert status(imm.w4_plan, *args) == want


def test_w4_arguments():
    L = imm.lib()
    assert L.w4_plan(4, 64, 256, 0, 128, None) == INVALID
    assert L.w4_packed_size(None) == 0
    # 4 column blocks x 2 K blocks of 1 KB, and 4 groups x 64 scale words
    p = imm.w4_plan(4, 56, 256, "f16", 64)
    assert imm.w4_packed_size(p) == 4 * 2 * 1024 + 4 * 64 * 4
    assert imm.w4_packed_size(imm.w4_plan(9999, 56, 256, "f16", 64)) == imm.w4_packed_size(p)

    def pack(plan=p, q=P, s=P, z=0, packed=P):
        return L.w4_pack(plan.handle if plan else None, q, s, z, packed, None)

    def run(plan=p, x=P, packed=P, b=0, y=P, ws=0, n=0):
        return L.w4_run(plan.handle if plan else None, x, packed, b, y, ws, n, None)

    assert pack(None) == pack(q=0) == pack(s=0) == pack(packed=0) == pack(s=P + 1) == pack(packed=P + 8) == INVALID
    assert run(None) == run(x=0) == run(packed=0) == run(y=0) == INVALID
    assert run(x=P + 8) == run(packed=P + 4) == run(y=P + 2) == run(b=P + 2) == INVALID
    assert run(imm.w4_plan(0, 64, 128, "f16"), x=0, packed=0, y=0) == OK
    assert run(imm.w4_plan(4, 0, 128, "f16"), x=0, packed=0, y=0) == OK
    assert pack(imm.w4_plan(4, 64, 0, "f16"), q=0, s=0, packed=0) == OK
    # many rows: the sums of x per group, rows rounded up to 128
    many = imm.w4_plan(600, 4112, 256, "f16", 64)
    assert many.workspace_bytes == imm.w4_workspace_size(many) == 4 * 640 * 8
    assert imm.w4_workspace_size(p) == L.w4_workspace_size(None) == 0
    assert run(many) == run(many, ws=P, n=4 * 640 * 8 - 1) == WORKSPACE
    assert run(many, ws=P + 8, n=1 << 20) == INVALID


def test_operators_refuse_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    for call in (lambda: torch_ops.rms_norm(x, w), lambda: torch_ops.rms_norm_quant(x, w),
                 lambda: torch_ops.quantize_rows(x), lambda: torch_ops.rms_norm_forward(x, w),
                 lambda: torch_ops.rms_norm_backward(x, x, w, torch.zeros(4)),
                 lambda: torch_ops.linear_f8(x.to(torch.float8_e4m3fn), torch.ones(4),
                                             x.to(torch.float8_e4m3fn), torch.ones(4)),
                 lambda: torch_ops.pack_w4(torch.zeros(8, 64, dtype=torch.uint8),
                                           torch.ones(8, 1).half())):
        with pytest.raises(ValueError):
            call()
    p = imm.rms_norm_plan(4, 64, "bf16")
    with pytest.raises(ValueError):
        imm.rms_norm_run(p, x, x)
    with pytest.raises(ValueError):
        imm.quantize_rows(x, x.to(torch.float8_e4m3fn), torch.zeros(4))


