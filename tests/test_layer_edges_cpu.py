"""Host-side checks of the norm and fp8 calls at sizes of zero (no GPU needed)."""
import invariant_matmul_amd as imm

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
