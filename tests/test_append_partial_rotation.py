"""Keys whose rotation ends inside a thread's sixteen values, or between two threads': NaN values past its end are
stored as those of any other key are (as 0), beside values that turn."""
import math

import pytest

from test_kv_cache import Case, check_append

SHAPES = [(64, 20, "half"), (64, 20, "interleaved"), (128, 50, "half"), (128, 50, "interleaved"), (256, 254, "interleaved"),
          (256, 254, "half"), (64, 32, "half"), (64, 0, "half")]


def keys_with(value, dim, rot, layout, single):
    c = Case(41, dim, 16, 2, 2, [0, 5, 16, 40], [1] * 4 if single else [2, 3, 1, 20], "bf16", rot=rot, layout=layout)
    for t in range(len(c.nk)):
        c.nk[t, t % 2, rot + t % (dim - rot)] = value
    c.nk[0, 0, dim - 1] = value
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("single", [True, False])
@pytest.mark.parametrize("dim,rot,layout", SHAPES)
def test_nan_past_the_rotation(cuda_lib, dim, rot, layout, single):
    check_append(keys_with(math.nan, dim, rot, layout, single), single=single, err_want=4)
