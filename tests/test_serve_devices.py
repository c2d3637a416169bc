"""Host tensors never reach a kernel: the calls refuse them, whichever argument they are, and check the device and
type of the error word and of a workspace as they do those of the operands."""
import pytest

from device_logits_sampling_gb300 import kv_cache, serve, w4


def operands(device, rows=3):
    import torch

    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=device)  # noqa: E731
    k = z(4, 2, 16, 64, t=torch.uint8)
    s = torch.ones(4, 2, device=device)
    return dict(cache=kv_cache.PagedCache(k, k.clone(), s, s.clone()), q=z(rows, 4, 64), k=z(rows, 2, 64), v=z(rows, 2, 64),
                pos=z(rows, t=torch.int32), table=z(rows, 2, t=torch.int32), x=z(rows, 256),
                weight=z(10, 128, t=torch.uint8), scales=z(10, 2))


def test_host_tensors_are_refused():
    import torch

    o = operands("cpu")
    args = (o["pos"], o["table"])
    for call in (lambda **kw: kv_cache.append(o["cache"], o["k"], o["v"], *args, **kw),
                 lambda **kw: kv_cache.append(o["cache"], o["k"], o["v"], *args, q=o["q"], **kw),
                 lambda **kw: kv_cache.attend(o["cache"], o["q"], *args, **kw),
                 lambda **kw: kv_cache.attend(o["cache"], o["q"], *args, workspace=torch.zeros(1 << 24, dtype=torch.uint8), **kw),
                 lambda **kw: w4.matvec(o["x"], o["weight"], o["scales"], **kw),
                 lambda **kw: w4.matvec(torch.cat([o["x"]] * 4), o["weight"], o["scales"], **kw)):
        for kw in ({}, dict(check=False), dict(stream=object())):
            with pytest.raises(ValueError, match="CUDA"):
                call(**kw)


def test_error_word_and_workspace_checks():
    import torch

    assert serve.err_word_ptr(None, 0) is None
    with pytest.raises(TypeError):
        serve.err_word_ptr(torch.zeros(1, dtype=torch.int64), -1)
    for word in (torch.zeros(1, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError):
            serve.err_word_ptr(word, 0)
    with pytest.raises(ValueError):
        serve.workspace_of(torch.zeros(64, dtype=torch.uint8), 0)
    with pytest.raises(ValueError):
        serve.workspace_of(torch.zeros(8, 8, dtype=torch.uint8).T, -1)
    w = torch.zeros(16, dtype=torch.int32)
    assert serve.workspace_of(w, -1) == (w.data_ptr(), 64)  # bytes, whatever its type


def test_the_current_stream_without_the_short_way(monkeypatch):
    import torch

    class Stream:
        cuda_stream = 7

    monkeypatch.setattr(serve, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream())
    assert serve.stream_of(None, 0) == 7 and serve.stream_of(Stream(), 0) == 7


@pytest.mark.gpu
def test_one_host_tensor_among_the_others_is_refused(cuda_lib):
    import torch

    o = operands("cuda")
    host = {n: t.cpu() for n, t in o.items() if n != "cache"}
    word = torch.zeros(1, dtype=torch.int32)
    ws = o["cache"].attend_workspace()

    def append(**kw):
        a = {**o, **kw}
        return kv_cache.append(o["cache"], a["k"], a["v"], a["pos"], a["table"], q=a["q"], q_out=a.get("q_out"),
                               err_word=a.get("err_word"))

    def attend(**kw):
        a = {**o, **kw}
        return kv_cache.attend(o["cache"], a["q"], a["pos"], a["table"], out=a.get("out"), workspace=a.get("workspace"),
                               err_word=a.get("err_word"))

    def matvec(rows=1, **kw):
        a = {**o, **kw}
        return w4.matvec(torch.cat([a["x"]] * rows), a["weight"], a["scales"], out=a.get("out"), workspace=a.get("workspace"))

    for kw in [{n: host[n]} for n in ("q", "k", "v", "pos", "table")] + [dict(err_word=word), dict(q_out=host["q"])]:
        with pytest.raises(ValueError):
            append(**kw)
    for kw in [{n: host[n]} for n in ("q", "pos", "table")] + [dict(err_word=word), dict(out=host["q"]), dict(workspace=ws.cpu())]:
        with pytest.raises(ValueError):
            attend(**kw)
    for kw in [{n: host[n]} for n in ("x", "weight", "scales")] + [dict(out=torch.zeros(3, 10, dtype=torch.bfloat16)),
                                                                  dict(rows=4, workspace=ws.cpu())]:
        with pytest.raises(ValueError):
            matvec(**kw)
    with pytest.raises(TypeError):
        append(err_word=torch.zeros(1, dtype=torch.int64, device="cuda"))
    # and the same calls without them run
    append(err_word=word.cuda())
    attend(workspace=ws.view(torch.int32))
    matvec(rows=4)
    torch.cuda.synchronize()
