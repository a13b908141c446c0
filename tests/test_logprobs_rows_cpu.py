"""Which logits token_logprobs reads in place."""
import pytest
import torch

from invariant_matmul_amd import torch_ops

WIDE = torch.arange(4 * 6 * 11, dtype=torch.float32).view(4, 6, 11)


@pytest.mark.parametrize("view,stride", [
    (WIDE, 11), (WIDE[..., 2:9], 11), (WIDE[:, :1, 1:], 66), (WIDE[:, ::2], 22), (WIDE[:, ::3, :5], 33), (WIDE[1:, 2:3], 66), (WIDE[0], 11), (WIDE[0, ::2, :4], 22),
    (WIDE[0, 0], 11), (WIDE[0, 0, 3:], 8), (WIDE[:, 0], 66), (WIDE[:1, 1:, 2:], 11), (WIDE[0, :1].expand(5, 11), 0),
    (WIDE[0, :1].expand(3, 5, 11), 0), (WIDE[..., :1].transpose(0, 1).transpose(0, 1), 11), (WIDE[0, :, :1].t()[..., :1], 1),
    (WIDE[:0], 11), (WIDE.unflatten(0, (2, 2)), 11),
], ids=lambda v: str(tuple(v.shape)) + str(v.stride()) if isinstance(v, torch.Tensor) else str(v))
def test_read_in_place(view, stride):
    rows, got = torch_ops._rows_of(view)
    assert rows is view and got == stride or view.numel() <= view.shape[-1]
    flat = torch.as_strided(rows, (view.numel() // view.shape[-1], view.shape[-1]), (got, 1))
    assert torch.equal(flat, view.reshape(-1, view.shape[-1]))


@pytest.mark.parametrize("view", [WIDE[:, :-1], WIDE[:, 1:, 2:], WIDE[::2, ::3], WIDE.transpose(0, 1), WIDE.transpose(1, 2), WIDE[..., ::2],
                                  WIDE[0, 0, ::2], WIDE[:1].expand(3, 6, 11)], ids=lambda v: str(v.stride()))
def test_copied(view):
    rows, got = torch_ops._rows_of(view)
    assert rows.shape == view.shape and rows.is_contiguous() and got == view.shape[-1] and torch.equal(rows, view)
    assert rows.data_ptr() != view.data_ptr()
