"""Host logic of the calls between and behind a decoder's products: exported names, plan
arguments, sizes of workspaces, and every refusal that needs no GPU."""
import ctypes
import os
import re

import pytest
import torch

import invariant_matmul_amd as imm
from invariant_matmul_amd import torch_ops

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "invariant_matmul.h")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 1 << 20  # an aligned address that no call reaches: it is refused before


def status(call, *args, **kw):
    try:
        call(*args, **kw)
        return OK
    except imm.GemmError as e:
        return e.status


def test_library_exports_the_decoder_calls():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)
    names = set(re.findall(r"\b((?:head_rope|attention|logprobs)_[a-z_0-9]+)\s*\(", text))
    assert names == set(imm.DECODER_SYMBOLS)
    for n in names:
        assert hasattr(imm.lib(), n), n


@pytest.mark.parametrize("args,kw,want", [
    ((4, 8, 2, 128, 128, "bf16"), {}, OK), ((0, 8, 2, 128, 64, "f16"), {}, OK), ((4, 8, 0, 512, 512, "f16"), {}, OK),
    ((4, 0, 0, 8, 0, "f16"), {}, OK), ((4, 8, 2, 128, 128, "bf16"), {"sections": [16, 24, 24]}, OK),
    ((4, 8, 2, 128, 128, "bf16"), {"sections": [1, 2, 3, 58]}, OK),
    ((-1, 8, 2, 128, 128, "bf16"), {}, INVALID), ((4, -8, 2, 128, 128, "bf16"), {}, INVALID),
    ((4, 8, 2, 128, -16, "bf16"), {}, INVALID), ((4, 8, 2, 128, 128, "bf16"), {"sections": [16, 24, 23]}, INVALID),
    ((4, 8, 2, 128, 128, "bf16"), {"sections": [65, -1]}, INVALID), ((4, 8, 2, 128, 128, "bf16"), {"sections": [2 ** 31 - 1, 65]}, INVALID),
    ((4, 8, 2, 128, 128, "bf16"), {"sections": [16, 16, 16, 8, 8]}, UNSUPPORTED),
    ((4, 8, 2, 128, 128, "bf16"), {"sections": []}, UNSUPPORTED),
    ((4, 8, 2, 132, 128, "bf16"), {}, UNSUPPORTED), ((4, 8, 2, 520, 128, "bf16"), {}, UNSUPPORTED),
    ((4, 8, 2, 0, 0, "bf16"), {}, UNSUPPORTED), ((4, 8, 2, 128, 72, "bf16"), {}, UNSUPPORTED),
    ((4, 8, 2, 64, 80, "bf16"), {}, UNSUPPORTED), ((4, 8, 2, 128, 128, "f32"), {}, UNSUPPORTED),
    ((4, 8, 2, 128, 128, "bf16"), {"eps": -1.0}, UNSUPPORTED), ((4, 8, 2, 128, 128, "bf16"), {"eps": float("nan")}, UNSUPPORTED),
    ((1 << 31, 8, 2, 128, 128, "bf16"), {}, UNSUPPORTED),
])
def test_head_rope_plan_arguments(args, kw, want):
    assert status(imm.head_rope_plan, *args, **kw) == want


def test_head_rope_refusals():
    L = imm.lib()
    plan = imm.head_rope_plan(4, 8, 2, 128, 128, "bf16")

    def run(q=P, qt=1280, qh=128, k=P, kt=1280, kh=128, pos=P, freq=P, wq=P, wk=P, yq=P, yk=P, plan=plan):
        return L.head_rope_run(plan.handle if plan else None, q, qt, qh, k, kt, kh, pos, freq, wq, wk, yq, yk, None)

    for bad in ({"plan": None}, {"q": 0}, {"q": P + 8}, {"k": 0}, {"qt": 1284}, {"kh": 4}, {"qt": -8}, {"qt": 1 << 41},
                {"pos": 0}, {"pos": P + 4}, {"freq": 0}, {"wq": P + 2}, {"yq": 0}, {"yk": P + 8}):
        assert run(**bad) == INVALID, bad
    plain = imm.head_rope_plan(4, 8, 2, 128, 128, "bf16", norm=False)
    assert run(plan=plain) == INVALID  # weights without the norm
    assert imm.head_rope_workspace_size(plain) == 0
    ws = imm.head_rope_workspace_size(plan)
    assert ws > 0 and ws % (2 * 128 * 4) == 0

    def back(w=P, dwq=P, n=ws, dy=P, plan=plan):
        return L.head_rope_backward(plan.handle, dy, P, P, 1280, 128, P, 1280, 128, P, P, 0, 0, P, P, dwq, 0, w, n, None)

    assert back(w=0) == WORKSPACE and back(n=ws - 1) == WORKSPACE and back(w=P + 4) == INVALID
    assert back(dy=0) == INVALID and back(dwq=P + 2) == INVALID and back(plan=plain) == INVALID
    # nothing to do
    none = imm.head_rope_plan(0, 8, 2, 128, 128, "bf16")
    assert run(plan=none, q=0, k=0, yq=0, yk=0) == OK


@pytest.mark.parametrize("args,kw,want", [
    ((10, 100, 2, 8, 2, 128, "bf16"), {}, OK), ((0, 0, 1, 1, 1, 8, "f16"), {}, OK), ((5, 5, 1, 7, 7, 72, "f16"), {"max_q": 9}, OK),
    ((-1, 100, 2, 8, 2, 128, "bf16"), {}, INVALID), ((10, -1, 2, 8, 2, 128, "bf16"), {}, INVALID),
    ((10, 100, 0, 8, 2, 128, "bf16"), {}, INVALID), ((10, 100, 2, 8, 2, 128, "bf16"), {"max_q": -1}, INVALID),
    ((10, 100, 2, 8, 3, 128, "bf16"), {}, UNSUPPORTED), ((10, 100, 2, 8, 0, 128, "bf16"), {}, UNSUPPORTED),
    ((10, 100, 2, 8, 2, 136, "bf16"), {}, UNSUPPORTED), ((10, 100, 2, 8, 2, 100, "bf16"), {}, UNSUPPORTED),
    ((10, 100, 2, 8, 2, 0, "bf16"), {}, UNSUPPORTED), ((10, 100, 2, 8, 2, 128, "f32"), {}, UNSUPPORTED),
    ((10, 100, 2, 8, 2, 128, "e4m3"), {}, UNSUPPORTED), ((10, 100, 2, 8, 2, 128, "bf16"), {"scale": 0.0}, UNSUPPORTED),
    ((10, 100, 2, 8, 2, 128, "bf16"), {"scale": -0.1}, UNSUPPORTED), ((10, 100, 2, 8, 2, 128, "bf16"), {"scale": float("inf")}, UNSUPPORTED),
    ((10, 100, 2, 8, 2, 128, "bf16"), {"scale": float("nan")}, UNSUPPORTED),
    ((10, (1 << 30) + 1, 2, 8, 2, 128, "bf16"), {}, UNSUPPORTED), ((1 << 28, 100, 2, 8, 2, 128, "bf16"), {}, UNSUPPORTED),
    ((10, 100, 1 << 22, 8, 2, 128, "bf16"), {}, UNSUPPORTED),
])
def test_attention_plan_arguments(args, kw, want):
    assert status(imm.attention_plan, *args, **kw) == want


def test_attention_refusals():
    L = imm.lib()
    plan = imm.attention_plan(10, 6000, 2, 8, 2, 128, "bf16", max_q=4)

    def run(q=P, qt=1024, qh=128, k=P, kt=256, kh=128, v=P, vt=256, vh=128, cq=P, ck=P, lens=0, o=P, low=0, lse=0, ws=P,
            n=None, plan=plan):
        n = imm.attention_workspace_size(plan) if n is None else n
        return L.attention_run(plan.handle if plan else None, q, qt, qh, k, kt, kh, v, vt, vh, cq, ck, lens, o, low, lse, ws, n,
                               None)

    # few rows: a chunk slot per 256 keys and sequence, for 4 queries of 8 heads
    need = (6000 // 256 + 2) * 4 * 8 * (128 + 4) * 4
    assert imm.attention_workspace_size(plan) == need
    for bad in ({"q": 0}, {"q": P + 8}, {"k": 0}, {"v": P + 4}, {"qt": 1028}, {"kh": -8}, {"vt": 12}, {"cq": 0}, {"ck": 0},
                {"cq": 0, "ck": 0}, {"cq": P + 2}, {"lens": P + 1}, {"o": 0}, {"o": P + 8}, {"low": P + 8}, {"lse": P + 2},
                {"ws": P + 8}, {"kt": 1 << 39}):
        assert run(**bad) == INVALID, bad
    assert L.attention_run(None, *[P] * 3, *[P] * 3, *[P] * 3, P, P, 0, P, 0, 0, P, need, None) == INVALID
    assert run(ws=0) == WORKSPACE and run(n=need - 1) == WORKSPACE
    assert run(kt=1 << 23) == UNSUPPORTED and run(vt=1 << 23) == UNSUPPORTED  # 256 rows past 31 bits
    many = imm.attention_plan(1000, 600, 2, 8, 2, 128, "bf16")
    assert imm.attention_workspace_size(many) == 0
    assert imm.attention_backward_workspace_size(many) == 2 * 1000 * 8 * 4
    # new tokens over long caches go to the kernel of few rows, prompts and long pieces do not
    few = lambda *args, **kw: imm.attention_workspace_size(imm.attention_plan(*args, "bf16", **kw)) > 0  # noqa: E731
    assert few(1, 8192, 1, 32, 8, 128) and few(61, 61 * 8192, 61, 32, 4, 128, max_q=1) and few(100, 8192, 1, 32, 8, 128)
    assert not few(8192, 8192, 1, 32, 8, 128) and not few(512, 16384, 1, 32, 8, 128) and not few(61, 61 * 8192, 61, 32, 4, 128)

    def back(do=P, o=P, low=P, lse=P, dq=P, dk=P, dv=P, ws=P, n=2 * 1000 * 8 * 4):
        return L.attention_backward(many.handle, do, P, 1024, 128, P, 256, 128, P, 256, 128, o, low, lse, P, P, 0, dq, dk, dv, ws,
                                    n, None)

    for name in ("do", "o", "lse", "dq", "dk", "dv"):
        assert back(**{name: 0}) == INVALID and back(**{name: P + 2}) == INVALID, name
    assert back(low=P + 2) == INVALID and back(ws=0) == WORKSPACE and back(n=2 * 1000 * 8 * 4 - 1) == WORKSPACE
    empty = imm.attention_plan(0, 600, 2, 8, 2, 128, "bf16")
    assert run(plan=empty, q=0, o=0, n=0) == OK


@pytest.mark.parametrize("args,kw,want", [
    ((4, 1000, "f32"), {}, OK), ((4, 1, "bf16"), {"top": 1}, OK), ((0, 1000, "f16"), {"top": 64, "tokens_per_row": 0}, OK),
    ((4, 1 << 22, "f32"), {"tokens_per_row": 1024}, OK),
    ((-1, 1000, "f32"), {}, INVALID), ((4, 0, "f32"), {}, INVALID), ((4, 10, "f32"), {"top": 11}, INVALID),
    ((4, 10, "f32"), {"top": -1}, INVALID), ((4, 10, "f32"), {"tokens_per_row": -1}, INVALID),
    ((4, 1000, "f32"), {"top": 65}, UNSUPPORTED), ((4, (1 << 22) + 1, "f32"), {}, UNSUPPORTED),
    ((4, 1000, "e4m3"), {}, UNSUPPORTED), ((1 << 31, 1000, "f32"), {}, UNSUPPORTED),
    ((4, 1000, "f32"), {"tokens_per_row": 1025}, UNSUPPORTED),
])
def test_logprobs_plan_arguments(args, kw, want):
    assert status(imm.logprobs_plan, *args, **kw) == want


def test_logprobs_refusals():
    L = imm.lib()
    plan = imm.logprobs_plan(4, 100000, "f32", 1, 5)
    need = imm.logprobs_workspace_size(plan)
    assert need > 0 and imm.logprobs_workspace_size(imm.logprobs_plan(1024, 100000, "f32", 1, 5)) == 0

    def run(x=P, stride=100000, t=P, lp=P, ent=P, norm=0, tl=P, tt=P, ws=P, n=need):
        return L.logprobs_run(plan.handle, x, stride, t, lp, ent, norm, tl, tt, ws, n, None)

    for bad in ({"x": 0}, {"x": P + 2}, {"stride": -1}, {"stride": 1 << 45}, {"t": 0}, {"t": P + 4}, {"lp": 0}, {"ent": 0},
                {"norm": P + 2}, {"tl": 0}, {"tt": P + 4}, {"ws": P + 8}):
        assert run(**bad) == INVALID, bad
    assert run(ws=0) == WORKSPACE and run(n=need - 1) == WORKSPACE

    def back(x=P, t=P, norm=P, ent=P, dx=P, g=P, h=P):
        return L.logprobs_backward(plan.handle, g, h, x, 100000, t, norm, ent, dx, None)

    for bad in ({"x": 0}, {"t": 0}, {"norm": 0}, {"ent": 0}, {"dx": 0}, {"dx": P + 8}, {"g": P + 2}, {"h": P + 1}):
        assert back(**bad) == INVALID, bad


def test_host_pointers_are_refused():
    # what passes the host's checks is refused as memory of no device (or for want of one)
    buf = ctypes.create_string_buffer(1 << 16)
    at = (ctypes.addressof(buf) + 63) & ~63
    plan = imm.logprobs_plan(2, 16, "f32", 1, 0)
    assert imm.lib().logprobs_run(plan.handle, at, 16, at + 1024, at + 2048, at + 4096, 0, 0, 0, 0, 0, None) in (INVALID, 4)
    rope = imm.head_rope_plan(1, 1, 1, 16, 16, "bf16")
    assert imm.lib().head_rope_run(rope.handle, at, 16, 16, at, 16, 16, at, at, 0, 0, at, at, None) in (INVALID, 4)
    att = imm.attention_plan(100, 2, 1, 1, 1, 16, "bf16")
    assert imm.lib().attention_run(att.handle, at, 16, 16, at, 16, 16, at, 16, 16, 0, 0, 0, at, 0, 0, 0, 0, None) in (INVALID, 4)


def test_torch_operators_refuse_cpu_tensors():
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="qk_norm_rope"):
        torch_ops.qk_norm_rope(x, x, torch.zeros(2, dtype=torch.int64), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="attention"):
        torch_ops.attention(x, x, x)
    with pytest.raises(ValueError, match="token_logprobs"):
        torch_ops.token_logprobs(torch.zeros(2, 5), torch.zeros(2, dtype=torch.int64))
