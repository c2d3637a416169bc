"""Parked sequences of attend_shared: their rows are 0 whatever lies in their queries and in the prefix, as in attend."""
import numpy as np
import pytest

from test_attend_shared import run, shared_case


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,front", [(64, 16, 10), (128, 64, 3), (256, 32, 5)])
@pytest.mark.parametrize("what", ["nan query", "infinite query", "nan key", "bad page"])
def test_rows_of_parked_sequences_are_zero(cuda_lib, dim, page, front, what):
    import torch

    c = shared_case(91, dim, page, 2, 4, front, [3, None, 20, None, 0], [2, 1, 1, 3, 1])
    parked = [2, 4, 5, 6]  # rows of sequences 1 and 3
    if what == "nan query":
        c.q[parked] = float("nan")
    elif what == "infinite query":
        c.q[parked] = float("inf")
    elif what == "nan key":
        c.k[c.prefix[1], :, 3, 5] = 0x7F
    else:
        c.prefix[2] = len(c.k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(c, err_word=err).float().cpu().numpy()
    assert int(err) == (1 if what == "bad page" else 0)
    assert (got[parked] == 0).all()
    others = np.delete(got, parked, 0)
    assert np.isnan(others).all() if what in ("nan key", "bad page") else np.isfinite(others).all()


@pytest.mark.gpu
def test_a_batch_of_parked_sequences(cuda_lib):
    """Nobody is behind the prefix; more rows than a unit has, all of them NaN."""
    import torch

    c = shared_case(92, 128, 16, 1, 4, 9, [5] + [None] * 80, [1] * 81)
    c.q[:] = float("nan")
    c.positions[0] = -3
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert (run(c, single=True, err_word=err) == 0).all() and int(err) == 0
