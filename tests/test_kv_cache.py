"""The paged 8-bit cache (include/serve/arc_kv.h): append and attend against the
fp64 oracle, their refusals, and the oracle against closed forms.

Stored codes and scales have to be the oracle's, bit for bit.  Floating outputs
may be off by half a step of their type and by what the kernels' own roundings
add: a rotated value 2^-21 (|a| + |b|); an attention output, with weights that
enter the products in fp16, (2^-11 + 2^-12) sum p |v| (a weight's half step, and
the fp32 scores) plus 2^-25 times the tokens times the largest value (weights
below fp16's normal range)."""
import ctypes
import math

import numpy as np
import pytest

from conftest import ROOT  # noqa: F401
from device_logits_sampling_gb300 import kv_cache, sampler, serve
from oracle import kv_cache as ok


# ------------------------------------------------------------------ host
@pytest.fixture(scope="module")
def lib():
    import os

    if not os.path.exists(serve.LIB_PATH):
        from device_logits_sampling_gb300 import build

        build.build_serve()
    return serve.load()


def test_library_exports_what_its_headers_declare(lib):
    import os
    import re
    import subprocess

    inc = os.path.join(ROOT, "include", "serve")
    text = "\n".join(open(os.path.join(inc, f)).read() for f in sorted(os.listdir(inc)))
    declared = set(re.findall(r"^\s*(?:int|size_t|const char\s*\*)\s*(arc_\w+)\s*\(", text, re.M))
    out = subprocess.run(["nm", "-D", "--defined-only", serve.LIB_PATH], capture_output=True, text=True).stdout
    assert set(re.findall(r"\bT (arc_\w+)", out)) == declared == set(serve.SIGNATURES)
    assert lib.arc_serve_abi_version() == 1
    for rc in range(-8, 1):
        assert "unknown" not in lib.arc_serve_strerror(rc).decode()
    assert "unknown" in lib.arc_serve_strerror(-99).decode()


def test_struct_sizes():
    sizes = [ctypes.sizeof(s) for s in (serve.KvCache, serve.KvStep, serve.RopeArgs, serve.KvRows, serve.KvQuery,
                                        serve.W4Weight)]
    assert sizes == [64, 56, 24, 104, 64, 48]


FAKE = 0x1000  # a non-NULL, aligned address that is never dereferenced


def fake_cache(**kw):
    d = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, page_stride=4 * 64 * 128, head_stride=64 * 128, pages=10, heads=4,
             page_size=64, head_dim=128)
    d.update(kw)
    return serve.KvCache(**d)


def fake_step(**kw):
    d = dict(page_table=FAKE, table_stride=5, positions=FAKE, row_offsets=None, B=3, T=3, max_pages=5, reserved=0)
    d.update(kw)
    return serve.KvStep(**d)


def fake_rows(**kw):
    d = dict(q=FAKE, k=FAKE, v=FAKE, q_out=2 * FAKE, q_token_stride=1024, q_head_stride=128, k_token_stride=512,
             k_head_stride=128, v_token_stride=512, v_head_stride=128, out_token_stride=1024, out_head_stride=128, q_heads=8,
             dtype=1)
    d.update(kw)
    return serve.KvRows(**d)


def fake_query(**kw):
    d = dict(q=FAKE, out=FAKE, q_token_stride=1024, q_head_stride=128, out_token_stride=1024, out_head_stride=128, q_heads=8,
             dtype=1, scale=0.1, window=0)
    d.update(kw)
    return serve.KvQuery(**d)


ref = ctypes.addressof

CACHE_REFUSALS = [(dict(k=None), -1), (dict(v=None), -1), (dict(k_scale=None), -1), (dict(v_scale=None), -1),
                  (dict(head_dim=96), -5), (dict(head_dim=0), -5), (dict(page_size=48), -5), (dict(page_size=512), -5),
                  (dict(pages=0), -2), (dict(heads=0), -2), (dict(head_stride=64), -2), (dict(page_stride=64 * 128), -2),
                  (dict(k=FAKE + 8), -4), (dict(page_stride=4 * 64 * 128 + 8), -4), (dict(v_scale=FAKE + 2), -4)]
STEP_REFUSALS = [(dict(page_table=None), -1), (dict(positions=None), -1), (dict(B=0), -2), (dict(T=0), -2), (dict(T=4), -2),
                 (dict(B=(1 << 20) + 1, T=(1 << 20) + 1), -2), (dict(T=(1 << 24) + 1, row_offsets=FAKE), -2),
                 (dict(max_pages=0), -2), (dict(max_pages=6), -2), (dict(max_pages=1 << 26, table_stride=1 << 26), -2),
                 (dict(reserved=1), -6), (dict(positions=FAKE + 2), -4), (dict(page_table=FAKE + 1), -4)]


def test_append_refusals(lib):
    def call(cache=fake_cache(), step=fake_step(), rows=fake_rows(), rope=None, err=None):
        return lib.arc_kv_append(ref(cache), ref(step), ref(rows), None if rope is None else ref(rope), err, None)

    for kw, rc in CACHE_REFUSALS:
        assert call(cache=fake_cache(**kw)) == rc, kw
    for kw, rc in STEP_REFUSALS:
        assert call(step=fake_step(**kw)) == rc, kw
    for kw, rc in [(dict(k=None), -1), (dict(v=None), -1), (dict(q=None), -1), (dict(q_out=None), -1), (dict(dtype=0), -3),
                   (dict(dtype=7), -3), (dict(q_heads=-1), -2), (dict(k=FAKE + 1), -4), (dict(q_out=FAKE + 1), -4),
                   (dict(q_out=FAKE, out_token_stride=2048), -6)]:
        assert call(rows=fake_rows(**kw)) == rc, kw
    good = dict(turns=FAKE, amplitude=1.0, rot_dim=128, layout=0, reserved=0)
    for kw, rc in [(dict(turns=None), -1), (dict(rot_dim=130), -2), (dict(rot_dim=63), -2), (dict(rot_dim=-2), -2),
                   (dict(layout=2), -6), (dict(reserved=1), -6), (dict(amplitude=0.0), -6), (dict(amplitude=math.nan), -6),
                   (dict(amplitude=math.inf), -6), (dict(turns=FAKE + 4), -4)]:
        assert call(rope=serve.RopeArgs(**{**good, **kw})) == rc, kw
    assert call(err=FAKE + 2) == -4
    assert lib.arc_kv_append(None, ref(fake_step()), ref(fake_rows()), None, None, None) == -1
    assert lib.arc_kv_append(ref(fake_cache()), None, ref(fake_rows()), None, None, None) == -1
    assert lib.arc_kv_append(ref(fake_cache()), ref(fake_step()), None, None, None, None) == -1


def test_attend_refusals(lib):
    def call(cache=fake_cache(), step=fake_step(), query=fake_query(), err=None, ws=FAKE, n=1 << 30):
        return lib.arc_kv_attend(ref(cache), ref(step), ref(query), err, ws, n, None)

    for kw, rc in CACHE_REFUSALS:
        assert call(cache=fake_cache(**kw)) == rc, kw
    for kw, rc in STEP_REFUSALS:
        assert call(step=fake_step(**kw)) == rc, kw
    for kw, rc in [(dict(q=None), -1), (dict(out=None), -1), (dict(dtype=0), -3), (dict(q_heads=0), -2), (dict(q_heads=6), -2),
                   (dict(window=-1), -6), (dict(scale=math.nan), -6), (dict(scale=math.inf), -6), (dict(q=FAKE + 1), -4)]:
        assert call(query=fake_query(**kw)) == rc, kw
    assert call(ws=None) == -8 and call(n=0) == -8 and call(ws=FAKE + 8) == -4 and call(err=FAKE + 1) == -4
    need = lib.arc_kv_attend_workspace_bytes(ref(fake_cache()))
    assert need > 0 and call(n=need - 1) == -8
    assert lib.arc_kv_attend_workspace_bytes(ref(fake_cache(head_dim=96))) == 0
    assert lib.arc_kv_attend_workspace_bytes(None) == 0


def test_python_refusals():
    import torch

    k = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    s = torch.ones(4, 2)
    cache = kv_cache.PagedCache(k, k.clone(), s, s.clone())
    for bad in (k[:, :, :, :32], k.transpose(2, 3), k[:, :, ::2]):
        with pytest.raises(ValueError):
            kv_cache.PagedCache(bad, bad, s, s)
    with pytest.raises(TypeError):
        kv_cache.PagedCache(k.float(), k.float(), s, s)
    with pytest.raises(ValueError):
        kv_cache.PagedCache(k, k.clone(), s[:3], s)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    pos, table = torch.zeros(3, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32)
    good = dict(k=x, v=x, positions=pos, page_table=table)
    for kw in (dict(k=x[:, :1]), dict(v=x[:2]), dict(v=x[..., :32]), dict(positions=pos[:2]), dict(page_table=table[0]),
               dict(k=x.transpose(1, 2).contiguous().transpose(1, 2)), dict(row_offsets=pos), dict(q_out=x),
               dict(q=x[..., :32]), dict(q=x, q_out=x[:2])):
        with pytest.raises(ValueError):
            kv_cache.append(cache, **{**good, **kw})
    for kw in (dict(positions=pos.long()), dict(page_table=table.float()), dict(k=x.float(), v=x.float())):
        with pytest.raises(TypeError):
            kv_cache.append(cache, **{**good, **kw})
    for kw in (dict(q=x[:2]), dict(q=x[..., :32]), dict(q=x, out=x[:2]), dict(q=x, out=x.half())):
        with pytest.raises(ValueError):
            kv_cache.attend(cache, positions=pos, page_table=table, workspace=k, **kw)
    with pytest.raises(TypeError):
        kv_cache.attend(cache, x.float(), pos, table, workspace=k)
    for kw in (dict(layout="other"), dict(turns=torch.zeros(2, 2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            kv_cache.Rope(**{**dict(turns=torch.zeros(2, dtype=torch.int64)), **kw})
    with pytest.raises(TypeError):
        kv_cache.Rope(torch.zeros(2))


def test_rope_turns():
    t, amp = kv_cache.rope_turns(8, base=100.0)
    want = 100.0 ** (-np.arange(4) / 4.0) / (2 * math.pi)
    assert amp == 1.0 and np.allclose(t / 2.0 ** 64, want, rtol=1e-15)
    assert np.array_equal(kv_cache.rope_turns(8, base=100.0, scaling="linear", factor=4.0)[0], t // 4)
    tb, _ = kv_cache.rope_turns(8, base=100.0, scaling="base", factor=4.0)
    assert tb[0] == t[0] and abs(tb[3] / t[3] * 4.0 - 1.0) < 1e-12
    tp, amp = kv_cache.rope_turns(64, scaling="parts", factor=8.0, original_length=4096)
    base = kv_cache.rope_turns(64)[0]
    assert amp == 0.1 * math.log(8.0) + 1.0 and tp[0] == base[0] and abs(tp[-1] / base[-1] * 8.0 - 1.0) < 1e-12
    for kw in (dict(rot_dim=7), dict(rot_dim=8, base=1.0), dict(rot_dim=8, scaling="x"),
               dict(rot_dim=8, scaling="linear", factor=0.5), dict(rot_dim=8, scaling="parts", factor=2.0)):
        with pytest.raises(ValueError):
            kv_cache.rope_turns(**kw)


def test_oracle_pins():
    import torch

    mine, theirs = ok.TABLE, torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(mine, theirs, equal_nan=True)
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    assert np.array_equal(ok.encode(ok.TABLE[codes]), codes)
    x = np.array([17.0, 19.0, 464.0, 1e9, -1e9, 2.0 ** -10, 3 * 2.0 ** -10, math.nan])  # 17, 19: ties of step 2
    assert ok.TABLE[ok.encode(x)].tolist() == [16.0, 20.0, 448.0, 448.0, -448.0, 0.0, 2.0 ** -8, 0.0]
    r = np.random.default_rng(0).standard_normal(20000) * 100
    assert np.array_equal(ok.TABLE[ok.encode(r)], torch.from_numpy(r).float().to(torch.float8_e4m3fn).double().numpy())
    assert [ok.scale_exponent(a) for a in (448.0, 448.1, 0.0, 1e30, 896.0, 1.0)] == [0, 1, -32, 32, 1, -8]
    y = ok.rotate(np.array([1.0, 0.0, 0.0, 0.0]), 3, [1 << 62], 1.0, "half")  # three quarter turns
    assert np.allclose(y, [0.0, -1.0, 0.0, 0.0])
    y = ok.rotate(np.array([0.0, 0.0, 1.0, 2.0]), 1 << 40, [1 << 30, 1 << 22], 2.0, "interleaved")
    assert np.allclose(y, [0.0, 0.0, -4.0, 2.0])  # 2^62: a quarter turn
    k = np.full((1, 1, 16, 4), 0x38, dtype=np.uint8)  # ones
    s = np.ones((1, 1))
    out, spread = ok.attend(k, k, s, s, np.ones((1, 1, 4)), [9], np.zeros((1, 1), int), [0, 1])
    assert np.allclose(out, 1.0) and np.allclose(spread, 1.0)


# ------------------------------------------------------------------ GPU
class Case:
    """A cache with stale bytes everywhere, sequences of random pages, and their new tokens."""

    def __init__(self, seed, dim, page, heads, q_heads, positions, news, dtype, max_pages=None, spare=3, amp=1.0, rot=None,
                 layout="half", base=10000.0, head_major=False, fill=True):
        import torch

        rng = self.rng = np.random.default_rng(seed)
        self.dim, self.page, self.heads, self.q_heads, self.layout, self.amp = dim, page, heads, q_heads, layout, amp
        self.positions, self.news = np.array(positions, np.int32), np.array(news, np.int64)
        self.dtype = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
        self.offsets = np.concatenate([[0], np.cumsum(self.news)]).astype(np.int32)
        B = len(positions)
        need = [max(0, -(-(int(p) + int(n)) // page)) if p >= 0 else 0 for p, n in zip(positions, news)]
        self.max_pages = max_pages or max(max(need), 1)
        total = sum(need) + spare
        ids = rng.permutation(total)
        self.table = np.full((B, self.max_pages), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            m = min(n, self.max_pages)
            self.table[b, :m] = ids[at:at + m]
            at += n
        shape = (total, heads, page, dim)
        self.k, self.v = (rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2))
        self.ks, self.vs = (2.0 ** rng.integers(-9, -2, shape[:2]) for _ in range(2))
        # what sequences hold is finite; everything else may be NaN codes
        if fill:
            for b in range(B):
                for j in range(min(max(0, int(positions[b])), self.max_pages * page)):
                    p = self.table[b, j // page]
                    for x in (self.k, self.v):
                        r = x[p, :, j % page]
                        r[(r & 0x7F) == 0x7F] = 0x30
        T = int(self.offsets[-1])
        host = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(self.dtype)  # noqa: E731
        self.q, self.nk, self.nv = host(T, q_heads, dim), host(T, heads, dim), host(T, heads, dim)
        rot = dim if rot is None else rot
        self.turns = kv_cache.rope_turns(rot, base=base)[0]
        self.head_major = head_major

    def device(self):
        import torch

        def place(x):
            t = torch.from_numpy(x).cuda()
            return t.transpose(0, 1).contiguous().transpose(0, 1) if self.head_major else t

        f32 = lambda x: torch.from_numpy(x.astype(np.float32)).cuda()  # noqa: E731
        cache = kv_cache.PagedCache(place(self.k), place(self.v), f32(self.ks), f32(self.vs))
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()  # noqa: E731
        return cache, i32(self.positions), i32(self.table), i32(self.offsets)

    def rope(self):
        import torch

        return kv_cache.Rope(torch.from_numpy(self.turns).cuda(), layout=self.layout, amplitude=self.amp)


def check_append(c, single=False, inplace=False, strided=None, err_want=0, times=1):
    """Append on the device and in the oracle; codes and scales equal, q within half a step and the rotation's bound."""
    import torch

    cache, pos, table, offs = c.device()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = c.q.cuda(), c.nk.cuda(), c.nv.cuda()
    if strided:  # one projection's output with an odd gap: no 16-byte alignment
        T, D = q.shape[0], c.dim
        wide = torch.zeros(T, (c.q_heads + 2 * c.heads) * D + strided, dtype=q.dtype, device="cuda")
        views = []
        at = strided
        for x in (q, k, v):
            n = x.shape[1] * D
            wide[:, at:at + n] = x.reshape(T, n)
            views.append(wide[:, at:at + n].unflatten(1, (x.shape[1], D)))
            at += n
        q, k, v = views
    for _ in range(times):
        src = q.clone() if inplace else q
        got_q = kv_cache.append(cache, k, v, pos, table, q=src, q_out=src if inplace else None, rope=c.rope(),
                                row_offsets=None if single else offs, err_word=err)
    torch.cuda.synchronize()
    ek, ev, eks, evs = c.k.copy(), c.v.copy(), c.ks.copy(), c.vs.copy()
    e = ok.append(ek, ev, eks, evs, c.nk.double().numpy(), c.nv.double().numpy(), c.positions, c.table, c.offsets, c.turns,
                  float(np.float32(c.amp)), c.layout)
    assert int(err.item()) == e == err_want
    assert np.array_equal(cache.k_scale.cpu().numpy(), eks) and np.array_equal(cache.v_scale.cpu().numpy(), evs)
    for got, want in ((cache.k, ek), (cache.v, ev)):
        got = got.cpu().numpy()
        zero = (want & 0x7F) == 0  # the sign of a zero carries nothing
        assert np.array_equal(got & 0x7F, want & 0x7F) and np.array_equal(got[~zero], want[~zero])
    eps = torch.finfo(c.dtype).eps / 2
    for b in range(len(c.positions)):
        for i in range(int(c.news[b])):
            t = int(c.offsets[b]) + i
            x = c.q[t].double().numpy()
            y = got_q[t].double().cpu().numpy()
            if c.positions[b] < 0:
                assert not y.any()
                continue
            want = ok.rotate(x, int(c.positions[b]) + i, c.turns, float(np.float32(c.amp)), c.layout)
            tol = eps * np.abs(want) + 2.0 ** -21 * c.amp * 2 * np.abs(x).max() + 2.0 ** -25
            assert (np.abs(y - want) <= tol).all()
    return cache


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,page,heads,q_heads,rot,layout", [
    (64, 16, 2, 8, 64, "half"), (128, 64, 3, 3, 128, "half"), (256, 32, 1, 7, 256, "half"), (128, 16, 2, 10, 64, "half"),
    (64, 256, 4, 4, 64, "interleaved"), (128, 128, 1, 5, 32, "interleaved"), (256, 16, 2, 2, 254, "interleaved"),
    (64, 32, 2, 2, 12, "half"), (128, 64, 2, 4, 0, "half"), (64, 16, 1, 1, 50, "half")])
def test_append_one_token_each(cuda_lib, dtype, dim, page, heads, q_heads, rot, layout):
    c = Case(1, dim, page, heads, q_heads, [0, 1, page - 1, page, 3 * page + 5, -1, 2 * page + page // 2], [1] * 7, dtype,
             rot=rot, layout=layout, amp=1.0 if rot != 64 else 1.2)
    check_append(c, single=True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,news", [(64, 16, [3, 1, 40, 0, 17]), (128, 64, [130, 7, 1, 64, 0]), (256, 256, [300, 2, 0, 1, 5]),
                                           (128, 16, [1, 1, 1, 1, 1]), (64, 128, [128, 129, 127, 1, 260])])
def test_append_pieces(cuda_lib, dim, page, news):
    c = Case(2, dim, page, 2, 4, [0, page - 1, 5, 9, 2 * page + 3], news, "bf16", rot=dim // 2, amp=1.1)
    check_append(c)


@pytest.mark.gpu
def test_append_many_sequences(cuda_lib):
    rng = np.random.default_rng(3)
    n = 700  # more sequences than a block has threads
    c = Case(3, 64, 16, 1, 2, rng.integers(-1, 60, n), rng.integers(0, 4, n), "fp16", layout="interleaved")
    check_append(c)
    c = Case(4, 64, 16, 1, 2, rng.integers(-1, 60, n), np.ones(n, int), "fp16")
    check_append(c, single=True)


@pytest.mark.gpu
def test_append_far_positions(cuda_lib):
    far = [(1 << 20) - 3, 777_777, 499_999]
    for base in (10000.0, 5e6):
        c = Case(5, 128, 256, 1, 2, [0] * 3, [2] * 3, "bf16", base=base)
        c.positions = np.array(far, np.int32)
        c.max_pages = (1 << 20) // 256
        c.table = np.full((3, c.max_pages), -1, np.int32)
        for b, p in enumerate(far):
            c.table[b, p // 256:(p + 1) // 256 + 1] = b
        check_append(c)


@pytest.mark.gpu
@pytest.mark.parametrize("single", [True, False])
def test_append_layouts_of_memory(cuda_lib, single):
    for kw in (dict(inplace=True), dict(strided=3), dict(strided=8), dict(strided=3, inplace=True)):
        for rot, layout in ((128, "half"), (20, "half"), (64, "interleaved")):
            c = Case(6, 128, 32, 2, 6, [0, 31, 70], [1] * 3 if single else [4, 2, 33], "bf16", rot=rot, layout=layout)
            check_append(c, single=single, **kw)
    c = Case(7, 64, 16, 3, 6, [0, 15, 70], [1] * 3, "bf16", head_major=True)
    check_append(c, single=single)


@pytest.mark.gpu
@pytest.mark.parametrize("single", [True, False])
def test_append_scale_growth_and_special_values(cuda_lib, single):
    import torch

    c = Case(8, 64, 16, 2, 2, [3, 15, 16, 40, 7, 9], [1] * 6 if single else [2, 3, 1, 20, 1, 1], "bf16")
    c.nv[0] *= 1000  # grows the page's scale over what it holds
    c.nk[0] *= 300
    c.nv[1] = 0.0
    c.nk[2], c.nv[2] = 0.0, 0.0  # a page that starts with zeros (or holds them)
    c.nv[3] = 448.0  # exactly on a scale's border
    c.nv[4, 0, 0], c.nv[4, 1, 5], c.nk[4, 1, 2] = math.inf, -math.inf, math.inf
    c.nv[5, 1, 3], c.nk[5, 0, 1] = math.nan, math.nan
    c.q[1, 0, 0] = 0.0
    check_append(c, single=single, err_want=4)
    c = Case(9, 128, 64, 1, 1, [0, 70], [1] * 2, "bf16")
    c.nk *= 1e30  # saturates at 448 * 2^32
    c.nv *= 1e-30  # below the least scale
    c.q[:] = torch.zeros_like(c.q)
    check_append(c, single=single)
    # the same token again changes nothing
    c = Case(10, 64, 16, 2, 2, [3, 15, 16], [1] * 3, "bf16")
    c.nv *= 50
    check_append(c, single=single, times=2)


@pytest.mark.gpu
@pytest.mark.parametrize("single", [True, False])
def test_append_bad_pages_and_positions(cuda_lib, single):
    c = Case(11, 64, 16, 2, 2, [3, 15, 16, 40], [1] * 4, "bf16", max_pages=3)
    c.table[1, 0] = 9999
    check_append(c, single=single, err_want=1)
    c.table[1, 0] = -5
    check_append(c, single=single, err_want=1)
    c = Case(12, 64, 16, 2, 2, [3, 48, 16], [1] * 3, "bf16", max_pages=3)
    check_append(c, single=single, err_want=2)


@pytest.mark.gpu
def test_bad_offsets_leave_their_sequence_out(cuda_lib):
    import torch

    c = Case(13, 64, 16, 1, 1, [0, 5, 9], [2, 2, 2], "bf16")
    cache, pos, table, offs = c.device()
    before = cache.k.clone()
    for bad in ([0, 4, 2, 6], [0, 2, 4, 9], [0, -2, 4, 6]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        o = torch.tensor(bad, dtype=torch.int32, device="cuda")
        kv_cache.append(cache, c.nk.cuda(), c.nv.cuda(), pos, table, q=c.q.cuda(), rope=c.rope(), row_offsets=o, err_word=err)
        assert int(err.item()) & 8
        err.zero_()
        kv_cache.attend(cache, c.q.cuda(), pos, table, row_offsets=o, err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) & 8
    assert before.shape == cache.k.shape


def check_attend(c, single=False, window=0, scale=None, err_want=0, strided=0, workspace=None):
    import torch

    cache, pos, table, offs = c.device()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = c.q.cuda()
    out = None
    if strided:
        wide = torch.full((q.shape[0], q.shape[1] + 1, c.dim + strided), 7.0, dtype=q.dtype, device="cuda")
        out = torch.full_like(wide, 7.0)[:, 1:, strided:]
        wide[:, 1:, strided:] = q
        q = wide[:, 1:, strided:]
    got = kv_cache.attend(cache, q, pos, table, out=out, row_offsets=None if single else offs, window=window, scale=scale,
                          err_word=err, workspace=workspace)
    torch.cuda.synchronize()
    assert int(err.item()) == err_want
    want, spread = ok.attend(c.k, c.v, c.ks, c.vs, c.q.double().numpy(), c.positions, c.table, c.offsets, scale, window)
    got = got.double().cpu().numpy()
    n = max(1, int((c.positions + c.news).max()))
    finite = c.v[(c.v & 0x7F) != 0x7F]
    vmax = float(np.abs(ok.TABLE[finite]).max() * c.vs.max()) if finite.size else 0.0
    eps = torch.finfo(c.dtype).eps / 2
    tol = eps * np.abs(want) + (2.0 ** -11 + 2.0 ** -12) * spread + 2.0 ** -25 * n * vmax + 2.0 ** -25
    assert np.array_equal(np.isnan(got), np.isnan(want))
    bad = ~(np.abs(got - want) <= tol) & ~np.isnan(want)
    assert not bad.any(), (np.argwhere(bad)[:5], float(np.nanmax(np.abs(got - want) / tol)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,page,heads,group", [(64, 16, 2, 1), (64, 64, 1, 4), (128, 16, 2, 8), (128, 64, 3, 5),
                                                  (128, 256, 1, 16), (256, 32, 2, 2), (256, 128, 1, 9), (64, 128, 1, 17),
                                                  (128, 32, 2, 40)])
def test_attend_one_token_each(cuda_lib, dtype, dim, page, heads, group):
    pos = [0, 1, 14, 15, 16, 17, 63, 64, 127, 130, 255, -1, 300, 511, 777]
    c = Case(21, dim, page, heads, heads * group, pos, [1] * len(pos), dtype)
    c.v[:] = np.where((c.v & 0x7F) == 0x7F, 0x7F, c.v)
    put_new(c)
    check_attend(c, single=True)


def put_new(c):
    """Finite codes where the new tokens lie (attend reads them; append is tested apart)."""
    for b in range(len(c.positions)):
        if c.positions[b] < 0:
            continue
        for j in range(int(c.positions[b]), int(c.positions[b] + c.news[b])):
            if j // c.page >= c.max_pages or not 0 <= c.table[b, j // c.page] < len(c.k):
                continue
            p = c.table[b, j // c.page]
            for x in (c.k, c.v):
                r = x[p, :, j % c.page]
                r[(r & 0x7F) == 0x7F] = 0x41


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page,heads,group,window", [(64, 16, 2, 4, 0), (128, 64, 1, 1, 0), (128, 32, 2, 5, 33), (256, 16, 1, 3, 1),
                                                         (64, 32, 1, 8, 16), (128, 16, 1, 16, 100)])
def test_attend_several_tokens(cuda_lib, dim, page, heads, group, window):
    pos, news = [0, 3, 15, 100, 0, 250, -1, 60], [1, 5, 17, 8, 33, 2, 3, 0]
    c = Case(22, dim, page, heads, heads * group, pos, news, "bf16")
    put_new(c)
    check_attend(c, window=window)


@pytest.mark.gpu
def test_attend_long_and_many(cuda_lib):
    c = Case(23, 128, 64, 2, 8, [20000], [1], "bf16", fill=False)
    c.k[(c.k & 0x7F) == 0x7F] = 0x30
    c.v[(c.v & 0x7F) == 0x7F] = 0x30
    check_attend(c, single=True)
    check_attend(c, single=True, window=5000)
    rng = np.random.default_rng(24)
    n = 1500
    c = Case(24, 64, 16, 1, 4, rng.integers(-1, 40, n), np.ones(n, int), "fp16")
    put_new(c)
    check_attend(c, single=True)


@pytest.mark.gpu
def test_attend_scales_far_apart(cuda_lib):
    """Pages whose value scales differ by 2^40: the small ones still count where their weights are large."""
    c = Case(25, 64, 16, 1, 2, [95, 63], [1, 1], "bf16")
    put_new(c)
    c.vs[:] = 2.0 ** c.rng.integers(-20, 21, c.vs.shape)
    c.ks[:] = 2.0 ** -7
    # tolerance: relative to the spread, which the largest scales carry
    check_attend(c, single=True)
    c.vs[:] = c.vs * 1.37  # scales that are no powers of two
    c.vs = c.vs.astype(np.float32).astype(np.float64)
    check_attend(c, single=True)


@pytest.mark.gpu
def test_attend_extreme_scores(cuda_lib):
    """Scores of thousands (one token takes all the weight) and of zero (all alike)."""
    import torch

    for factor in (200.0, 0.0, 1e-30):
        c = Case(26, 128, 16, 1, 3, [0, 40, 77], [1] * 3, "bf16")
        put_new(c)
        c.ks[:] = 2.0 ** -6
        c.q = (c.q.float() * factor).to(torch.bfloat16)
        # the scores' fp32 error, 2^-22 of their size, is what moves the weights here
        if factor > 1:
            c.q = torch.round(c.q.float() / 64).mul(64).to(torch.bfloat16)  # few bits: exact products
        check_attend(c, single=True)


@pytest.mark.gpu
def test_attend_nan_where_it_is_not_seen(cuda_lib):
    """NaN values of later tokens, of other pages and of slots past the end do not reach a row; a NaN it sees does."""
    c = Case(27, 64, 16, 1, 2, [30, 30], [4, 4], "bf16")
    put_new(c)
    p = c.table[0, 33 // 16]
    c.v[p, 0, 33 % 16, 5] = 0x7F  # the last new token of sequence 0
    c.v[p, 0, 33 % 16 + 1:] = 0xFF
    c.k[p, 0, 33 % 16 + 1:] = 0xFF
    import torch

    cache, pos, table, offs = c.device()
    got = kv_cache.attend(cache, c.q.cuda(), pos, table, row_offsets=offs).float().cpu().numpy()
    nan = np.zeros_like(got, dtype=bool)
    nan[3, :, 5] = True
    assert np.array_equal(np.isnan(got), nan)
    # a NaN or infinite query spoils its own row alone
    c = Case(28, 64, 16, 1, 4, [30, 30], [1, 1], "bf16")
    put_new(c)
    c.q[0, 1, 3], c.q[1, 2, 7] = math.nan, math.inf
    cache, pos, table, offs = c.device()
    got = kv_cache.attend(cache, c.q.cuda(), pos, table).float().cpu().numpy()
    want = np.zeros((2, 4), dtype=bool)
    want[0, 1] = want[1, 2] = True
    assert np.array_equal(np.isnan(got).any(-1), want)
    assert torch.isfinite(torch.from_numpy(got[0, 0])).all()


@pytest.mark.gpu
def test_attend_bad_pages_and_positions(cuda_lib):
    c = Case(29, 64, 16, 2, 4, [30, 50, 16], [1] * 3, "bf16")
    put_new(c)
    c.table[1, 1] = len(c.k)
    check_attend(c, single=True, err_want=1)
    c = Case(30, 64, 16, 2, 4, [30, 50, 16], [1, 2, 1], "bf16", max_pages=3)
    put_new(c)
    check_attend(c, err_want=2)


@pytest.mark.gpu
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 32), (128, 16), (256, 16)])
def test_attend_window_needs_no_older_pages(cuda_lib, dim, page):
    """Pages that lie wholly before the first new token's window may be gone from the table."""
    pos, news, window = [200, 333, 90, 17], [1, 4, 7, 2], 50
    c = Case(34, dim, page, 1, 6, pos, news, "bf16")
    put_new(c)
    for b, p in enumerate(pos):
        c.table[b, : max(0, p + 1 - window) // page] = -1
    check_attend(c, window=window)


@pytest.mark.gpu
def test_attend_memory_and_workspace(cuda_lib):
    import torch

    c = Case(31, 128, 16, 2, 6, [30, 50, 2000, 16], [1] * 4, "bf16", head_major=True)
    put_new(c)
    check_attend(c, single=True)
    c.head_major = False
    ws = c.device()[0].attend_workspace()
    for strided in (0, 1, 8):
        for _ in range(3):  # a workspace serves call after call
            check_attend(c, single=True, strided=strided, scale=0.3, workspace=ws)
    s = torch.cuda.Stream()
    cache, pos, table, _ = c.device()
    q = c.q.cuda()
    torch.cuda.synchronize()
    a = kv_cache.attend(cache, q, pos, table, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        b = kv_cache.attend(cache, q, pos, table, workspace=ws)
    s.synchronize()
    assert torch.equal(a, b)  # and the same bits every time


@pytest.mark.gpu
def test_cache_past_32_bits(cuda_lib):
    """Pages whose byte offsets pass 2^32."""
    import torch

    pages, heads, ps, d = 17000, 8, 256, 128
    cache = kv_cache.PagedCache.empty(pages, heads, ps, d)
    assert pages * heads * ps * d > 1 << 32
    c = Case(32, d, ps, heads, 16, [0, 300], [40, 3], "bf16")
    hi = np.where(c.table >= 0, pages - 1 - c.table, -1).astype(np.int32)
    offs, pos = torch.from_numpy(c.offsets).cuda(), torch.tensor(c.positions, device="cuda")
    small, _, table, _ = c.device()
    big = torch.from_numpy(hi).cuda()
    for p in range(len(c.k)):
        for a, b in ((cache.k, small.k), (cache.v, small.v)):
            a.view(torch.uint8)[pages - 1 - p] = b[p]
        cache.k_scale[pages - 1 - p], cache.v_scale[pages - 1 - p] = small.k_scale[p], small.v_scale[p]
    outs = []
    for x, t in ((cache, big), (small, table)):
        q = kv_cache.append(x, c.nk.cuda(), c.nv.cuda(), pos, t, q=c.q.cuda(), rope=c.rope(), row_offsets=offs)
        outs.append(kv_cache.attend(x, q, pos, t, row_offsets=offs))
    torch.cuda.synchronize()
    assert torch.equal(*outs) and bool(torch.isfinite(outs[0].float()).all())
    for p in range(len(c.k)):
        assert torch.equal(cache.k.view(torch.uint8)[pages - 1 - p], small.k[p])


@pytest.mark.gpu
def test_replayed_from_a_graph(cuda_lib):
    """Positions advance on the device between replays; each replay is the eager step."""
    import torch

    c = Case(33, 64, 16, 2, 4, [0, 9, 30, -1], [1] * 4, "bf16", max_pages=6)
    for b in (0, 1, 2):
        c.table[b] = np.arange(6) + 6 * b
    c.k, c.v = (np.zeros((18, 2, 16, 64), np.uint8) for _ in range(2))
    c.ks, c.vs = np.ones((18, 2)), np.ones((18, 2))
    steps = 20
    feed = torch.randn(steps, 4, 8, 64, device="cuda").to(torch.bfloat16)
    res = []
    for graphed in (False, True):
        cache, pos, table, _ = c.device()
        ws = cache.attend_workspace()
        x = torch.zeros_like(feed[0])
        rope = c.rope()
        live = (pos >= 0).to(torch.int32)

        def step():
            q = kv_cache.append(cache, x[:, 4:6], x[:, 6:8], pos, table, q=x[:, :4], rope=rope)
            o = kv_cache.attend(cache, q, pos, table, workspace=ws)
            pos.add_(live)
            return o

        outs = []
        if graphed:
            g = torch.cuda.CUDAGraph()
            keep = [t.clone() for t in (pos, cache.k, cache.v, cache.k_scale, cache.v_scale)]
            with torch.cuda.graph(g):
                o = step()
            for t, s in zip((pos, cache.k, cache.v, cache.k_scale, cache.v_scale), keep):
                t.copy_(s)
        for i in range(steps):
            x.copy_(feed[i])
            if graphed:
                g.replay()
            else:
                o = step()
            outs.append(o.clone())
        torch.cuda.synchronize()
        res.append(torch.stack(outs))
    assert torch.equal(res[0], res[1])
