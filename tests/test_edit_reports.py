"""What edit_logits reports of lists without an entry: offsets and penalties are looked at all the same."""
import numpy as np
import pytest

from device_logits_sampling_gb300 import edit
from test_logit_edit import Case, records


@pytest.mark.gpu
@pytest.mark.parametrize("offsets,penalties,bias_offsets,err", [
    ([0, 0, 0], [(1.5, 1, 1)] * 2, [0, 0, 0], 0), ([0, 3, 3], [(1.5, 1, 1)] * 2, [0, 0, 0], edit.ARC_EDIT_ERR_HIST),
    ([0, 0, 0], [(1.5, 1, 1), (0.0, 1, 1)], [0, 0, 0], edit.ARC_EDIT_ERR_PARAM),
    ([0, 0, 0], [(1.5, 1, 1)] * 2, [0, 0, -1], edit.ARC_EDIT_ERR_BIAS)])
def test_empty_lists(cuda_lib, offsets, penalties, bias_offsets, err):
    import torch

    c = Case(2, 300)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    none, word = i32([]), i32([0])
    got = edit.edit_logits(c.logits, params=records(penalties), hist_offsets=i32(offsets), hist_ids=none,
                           bias_offsets=i32(bias_offsets), bias_ids=none, bias=none.float(), err_word=word)
    assert torch.equal(got, c.logits) and int(word) == err
    c.host.update(penalties=penalties, hist_offsets=offsets, hist_ids=np.zeros(0, int), bias_offsets=bias_offsets,
                  bias_ids=np.zeros(0, int), bias=np.zeros(0))
    assert c.want()[1] == err  # what a list with room for entries reports
