"""Outputs of the prompt calls whose rows or heads share elements are refused, without a GPU: nothing here is launched."""
from __future__ import annotations

import pytest
import torch

from tests.test_prompt_refusals import INVALID, append, dfv, prompt, read, rows  # noqa: F401

OVERLAP = [(0, 128), (4096, 0), (64, 128), (4096, 120), (128, 128), (512, 512)]


@pytest.mark.parametrize("row,head", OVERLAP)
def test_overlapping_outputs(dfv, row, head):  # noqa: F811
    for status in (append(dfv, orow=row, oh=head), append(dfv, ko=0x7000, kor=row, koh=head), read(dfv, kr=row, kh=head), read(dfv, v=0, kr=row, kh=head),
                   read(dfv, k=0, vr=row, vh=head), prompt(dfv, orow=row, oh=head)):
        assert status == INVALID and b"overlap" in dfv.lib().dfv_last_error_detail()


def test_keys_and_values_into_one_tensor(dfv):  # noqa: F811
    assert read(dfv, k=0x3000, v=0x3000) == INVALID and b"v_out" in dfv.lib().dfv_last_error_detail()


def test_inputs_may_share_rows_of_values(dfv):  # noqa: F811
    """The append reads q, k and v with any strides; what is refused next (a layer out of range) shows that they passed."""
    assert append(dfv, layer=9, qr=0, kr=0, vr=0, kh=0, vh=0) == INVALID and b"layer" in dfv.lib().dfv_last_error_detail()


def test_binding(dfv):  # noqa: F811
    off = torch.tensor([0, 3, 5], dtype=torch.int32)
    r = dfv.RowBatch(off, 5, 3)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):  # (host tensors: refused before the library sees them)
        dfv.prompt_attention(r, q, q[:, :2], q[:, 2:], ws, out=q.new_zeros(1, 4, 64).expand(5, 4, 64))
