"""norm.join where rows go through rings in shared memory (dim above 2,048, at least four rows an SM) and where a thread has
four groups of a row of odd length, against the fp64 oracle with the tolerances of test_norm_join."""
import pytest

from device_logits_sampling_gb300 import norm
from test_norm_join import case, check

# rows that are no multiple of the blocks, once and several times around the rings
ROWS = (613, 1300)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("dim", (2056, 5120, 8192))
@pytest.mark.parametrize("stream", (None, "float32"))
@pytest.mark.parametrize("post,gate", [(False, None), (True, "sigmoid"), (False, "token"), (True, "channel")])
def test_forms(cuda_lib, rows, dim, stream, post, gate):
    """Rings of three rows and of two; rows that have no room for two."""
    kind = "bfloat16" if rows == 613 else "float16"
    x, kw = case(rows, dim, kind, stream, post, gate, seed=dim + rows)
    check(x, kw, norm.join(x, **kw, alpha=0.3, offset=1.0), alpha=0.3, offset=1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,stream,gate", [(14336, None, None), (9552, "float32", None), (7168, "float32", "token"), (2056, None, None)])
def test_long_rings_wide_weights_and_strides(cuda_lib, dim, stream, gate):
    x, kw = case(2001, dim, "bfloat16", stream, True, gate, wide=True, pad=8, seed=dim)
    check(x, kw, norm.join(x, **kw, alpha=-1.5, eps=1e-3), alpha=-1.5, eps=1e-3)


@pytest.mark.gpu
@pytest.mark.parametrize("stream", (None, "float32"))
def test_in_place_again_and_in_a_graph(cuda_lib, stream):
    """h over x and n over y; the same bits each time, on another stream and replayed."""
    import torch

    x, kw = case(1300, 5120, "bfloat16", stream, True, "sigmoid", seed=5)
    want = norm.join(x, **kw)
    again = norm.join(x, **kw)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = norm.join(x, **kw, stream=side)
    side.synchronize()
    assert torch.equal(got[0].cpu(), want[0].cpu()) and torch.equal(got[1].cpu(), want[1].cpu())
    y = kw.pop("y")
    x2, y2 = x.clone(), y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm.join(x2, y2, **kw, h=x2, n=y2)
    for _ in range(2):
        x2.copy_(x)
        y2.copy_(y)
        graph.replay()
        assert torch.equal(x2, want[0]) and torch.equal(y2, want[1])


@pytest.mark.gpu
def test_a_bad_row_is_alone(cuda_lib):
    import torch

    x, kw = case(1300, 4096, post=False)
    want = norm.join(x, **kw)
    x[304, 3], kw["y"][700, 5] = float("nan"), float("inf")
    h, n = norm.join(x, **kw)
    keep = torch.ones(1300, dtype=torch.bool)
    keep[[304, 700]] = False
    assert torch.isnan(n[304]).all() and torch.isnan(n[700]).any()
    assert torch.equal(h[keep], want[0][keep]) and torch.equal(n[keep], want[1][keep])


@pytest.mark.gpu
@pytest.mark.parametrize("dim", (8184, 8185, 8201, 9999, 12345, 16375, 16376, 16377, 16384))
@pytest.mark.parametrize("pad", (0, 3))
@pytest.mark.parametrize("kind,stream", [("bfloat16", None), ("float16", "float32")])
def test_long_rows_of_any_length(cuda_lib, dim, pad, kind, stream):
    """Two, four and eight groups a thread: rows that all begin alike, and (padded inputs, packed outputs) that do not."""
    x, kw = case(5, dim, kind, stream, gate="sigmoid", pad=pad, seed=dim)
    check(x, kw, norm.join(x, **kw, alpha=0.3, offset=1.0), alpha=0.3, offset=1.0)
