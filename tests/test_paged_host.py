"""Host-side checks of the paged cache's entry points: every refusal that needs no GPU (the
addresses are never dereferenced), the binding's own checks, and the models that the GPU tests
compare with."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from _paged import Case, Tables, attend


def P(i, off=0):
    return 0x7f0000000000 + i * (1 << 34) + off


@pytest.fixture(scope="module")
def g():
    from gated_deltanet_state_gdn_b200 import build
    build.build()
    import gated_deltanet_state_gdn_b200 as g
    g.lib()
    return g


def cache(**kw):
    from gated_deltanet_state_gdn_b200._paged import _Cache
    a = dict(k=P(1), v=P(2), page_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64, k_scale=None,
             v_scale=None, block_table=P(3), seq_lens=P(4), table_stride=8, rows=4, width=8, num_pages=20,
             page_size=16, heads=2, head_dim=64, dtype=1)
    a.update(kw)
    return _Cache(*[a[n] for n, _ in _Cache._fields_])


def append(g, c=None, **kw):
    a = dict(k=P(5), v=P(6), kt=128, kh=64, vt=128, vh=64, slots=P(7), off=P(8), B=3, N=30, dtype=1)
    a.update(kw)
    return g.lib().gdn_kv_append(a["k"], a["v"], a["kt"], a["kh"], a["vt"], a["vh"],
                                 None if c is False else ctypes.byref(c or cache()), a["slots"], a["off"],
                                 a["B"], a["N"], a["dtype"], None, None)


def test_append_refusals(g):
    assert append(g, dtype=0) == g.GDN_ERR_DTYPE                     # fp32 rows
    assert append(g, dtype=g.GDN_E4M3) == g.GDN_ERR_DTYPE
    assert append(g, dtype=2) == g.GDN_ERR_DTYPE                     # fp16 rows, bf16 cache
    assert append(g, cache(dtype=0)) == g.GDN_ERR_DTYPE
    assert append(g, cache(k_scale=P(9))) == g.GDN_ERR_DTYPE         # scales of a 16-bit cache
    assert append(g, False) == g.GDN_ERR_NULL
    for f in ("k", "v", "block_table", "seq_lens"):
        assert append(g, cache(**{f: None})) == g.GDN_ERR_NULL
    assert append(g, k=None) == g.GDN_ERR_NULL
    for f in ("rows", "width", "num_pages", "page_size", "heads", "head_dim"):
        assert append(g, cache(**{f: 0})) == g.GDN_ERR_SHAPE
    assert append(g, cache(head_dim=264)) == g.GDN_ERR_UNSUPPORTED
    assert append(g, cache(head_dim=60)) == g.GDN_ERR_UNSUPPORTED
    assert append(g, cache(head_dim=24, dtype=3)) == g.GDN_ERR_UNSUPPORTED
    assert append(g, cache(width=1 << 27, table_stride=1 << 27)) == g.GDN_ERR_UNSUPPORTED
    assert append(g, cache(table_stride=7)) == g.GDN_ERR_SHAPE
    assert append(g, cache(head_stride=32)) == g.GDN_ERR_SHAPE       # heads over one another
    assert append(g, cache(token_stride=64)) == g.GDN_ERR_SHAPE
    assert append(g, cache(page_stride=64)) == g.GDN_ERR_SHAPE
    assert append(g, cache(page_stride=-2048)) == g.GDN_ERR_SHAPE
    assert append(g, cache(page_stride=2052)) == g.GDN_ERR_ALIGN
    assert append(g, cache(k=P(1, 8))) == g.GDN_ERR_ALIGN
    assert append(g, k=P(5, 8)) == g.GDN_ERR_ALIGN
    assert append(g, kt=132) == g.GDN_ERR_ALIGN
    assert append(g, slots=P(7, 2)) == g.GDN_ERR_ALIGN
    assert append(g, B=-1) == g.GDN_ERR_SHAPE
    assert append(g, off=None, N=31) == g.GDN_ERR_SHAPE
    assert append(g, slots=None, B=5) == g.GDN_ERR_SHAPE             # more requests than rows
    assert append(g, N=1 << 31) == g.GDN_ERR_UNSUPPORTED
    assert append(g, k=P(1, 1024)) == g.GDN_ERR_ALIAS
    assert append(g, cache(v=P(1))) == g.GDN_ERR_ALIAS
    assert append(g, cache(seq_lens=P(2, 64))) == g.GDN_ERR_ALIAS
    assert append(g, B=0, N=0) == g.GDN_OK
    assert append(g, N=0) == g.GDN_OK
    # one head, one token a page: their strides do not matter
    assert append(g, cache(heads=1, head_stride=3), kh=5, vh=7, N=0) == g.GDN_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: no call may be launched")
def test_calls_without_a_device_return(g):
    """Valid calls where there is no GPU return an error, in a process of their own (a call that
    ends the process would end these tests)."""
    import subprocess
    import sys
    code = """if 1:
        import sys
        sys.path[:0] = ["tests", "."]
        import gated_deltanet_state_gdn_b200 as g
        import test_paged_host as t
        assert t.append(g) == g.GDN_ERR_CUDA
        assert t.append(g, t.cache(dtype=3, page_stride=32 * 64)) == g.GDN_ERR_CUDA
        assert t.attn(g) == g.GDN_ERR_CUDA
        L, P = g.lib(), t.P
        assert L.gdn_page_resize(bytes(t.table()), P(5), P(6), 3, None, 0, P(7), 1 << 20, None, None) == g.GDN_ERR_CUDA
        assert L.gdn_page_fork(bytes(t.table()), P(5), P(6), 3, None, 0, None, None) == g.GDN_ERR_CUDA
        assert L.gdn_page_compact(bytes(t.table()), P(5), None, 0, P(7), 1 << 20, None, None) == g.GDN_ERR_CUDA
        print("returned")
    """
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "returned" in r.stdout, r.stdout + r.stderr


def vectors(base, c):
    """First bytes of all vectors of a cache, [pages, tokens, heads]."""
    es = 1 if c.dtype == 3 else 2
    i, j, h = (np.arange(n) for n in (c.num_pages, c.page_size, c.heads))
    return base + es * (i[:, None, None] * c.page_stride + j[:, None] * c.token_stride + h * c.head_stride)


@pytest.mark.parametrize("dtype", [1, 3])
@pytest.mark.parametrize("pages,page,heads,D,order,gaps", [
    (5, 4, 3, 16, "tokens", (0, 0, 0)), (5, 4, 3, 16, "heads", (0, 0, 0)), (4, 3, 2, 16, "tokens", (16, 0, 0)),
    (4, 3, 2, 32, "tokens", (0, 96, 0)), (4, 3, 2, 16, "heads", (32, 16, 128)), (3, 1, 4, 16, "tokens", (16, 0, 0)),
    (3, 5, 1, 16, "heads", (0, 16, 32)), (1, 1, 1, 16, "tokens", (0, 0, 0))])
def test_keys_over_values(g, dtype, pages, page, heads, D, order, gaps):
    """Caches whose keys and values share bytes are refused for writing, wherever they start; values
    in the gaps between keys are not."""
    inner = D + gaps[0]
    if order == "tokens":
        hs, ts = inner, heads * inner + gaps[1]
        ps = page * ts + gaps[2]
    else:
        ts, hs = inner, page * inner + gaps[1]
        ps = heads * hs + gaps[2]
    es = 1 if dtype == 3 else 2
    a = dict(dtype=dtype, num_pages=pages, page_size=page, heads=heads, head_dim=D, head_stride=hs, token_stride=ts,
             page_stride=ps)
    k = vectors(P(1), cache(**a)).reshape(-1)
    end = (pages * ps + 4 * D) * es
    got = {}
    for off in range(-end // 16 * 16, end, 16):
        status = append(g, cache(v=P(1, off), **a), kt=heads * D, kh=D, vt=heads * D, vh=D, dtype=1, N=0)
        v = vectors(P(1, off), cache(**a)).reshape(-1)
        at = np.searchsorted(v, k)              # a key's vector meets the values' next or last one
        gap = np.minimum(np.abs(v[np.minimum(at, len(v) - 1)] - k), np.abs(v[np.maximum(at - 1, 0)] - k)) \
            if (np.diff(v) > 0).all() else np.abs(v[:, None] - k).min(0)
        want = g.GDN_ERR_ALIAS if (gap < D * es).any() else g.GDN_OK
        assert status == want, off
        got[status] = got.get(status, 0) + 1
    assert len(got) == 2


def attn(g, c=None, **kw):
    a = dict(q=P(5), qt=256, qh=64, slots=P(7), B=3, T=2, Hq=4, dtype=1, scale=0.1, window=0, out=P(8), lse=P(9),
             flags=0, ws=P(10), nbytes=1 << 30)
    a.update(kw)
    return g.lib().gdn_paged_attn(a["q"], a["qt"], a["qh"], None if c is False else ctypes.byref(c or cache()),
                                  a["slots"], a["B"], a["T"], a["Hq"], a["dtype"], a["scale"], a["window"],
                                  a["out"], a["lse"], a["flags"], a["ws"], a["nbytes"], None, None)


def test_attn_refusals(g):
    assert attn(g, dtype=0) == g.GDN_ERR_DTYPE
    assert attn(g, dtype=2) == g.GDN_ERR_DTYPE
    assert attn(g, flags=1) == g.GDN_ERR_UNSUPPORTED
    assert attn(g, False) == g.GDN_ERR_NULL
    assert attn(g, T=0) == g.GDN_ERR_SHAPE
    assert attn(g, T=17) == g.GDN_ERR_UNSUPPORTED
    assert attn(g, Hq=5) == g.GDN_ERR_SHAPE
    assert attn(g, window=-1) == g.GDN_ERR_SHAPE
    assert attn(g, slots=None, B=5) == g.GDN_ERR_SHAPE
    for f in ("q", "out", "ws"):
        assert attn(g, **{f: None}) == g.GDN_ERR_NULL
    assert attn(g, q=P(5, 2)) == g.GDN_ERR_ALIGN
    assert attn(g, qt=255) == g.GDN_ERR_ALIGN
    assert attn(g, out=P(8, 2)) == g.GDN_ERR_ALIGN
    assert attn(g, ws=P(10, 8)) == g.GDN_ERR_ALIGN
    assert attn(g, out=P(5, 64)) == g.GDN_ERR_ALIAS
    assert attn(g, out=P(1, 64)) == g.GDN_ERR_ALIAS
    assert attn(g, lse=P(8, 64)) == g.GDN_ERR_ALIAS
    assert attn(g, lse=P(4)) == g.GDN_ERR_ALIAS
    assert attn(g, B=0) == g.GDN_OK
    size = g.lib().gdn_paged_attn_workspace_size
    assert size(0, 1, 4, 2, 64, 1) == 0 and size(1, 17, 4, 2, 64, 1) == 0 and size(1, 1, 5, 2, 64, 1) == 0


def test_expanded_caches_are_refused(g):
    """A stride of zero, of a dimension of more than one (nothing is launched: B or N is zero)."""
    for f, kw in ((attn, dict(B=0)), (append, dict(N=0))):
        for n in ("page_stride", "token_stride", "head_stride"):
            assert f(g, cache(**{n: 0}), **kw) == g.GDN_ERR_SHAPE
        assert f(g, cache(heads=1, head_stride=0), **kw) == g.GDN_OK
        assert f(g, cache(page_size=1, token_stride=0, page_stride=128), **kw) == g.GDN_OK
        assert f(g, cache(num_pages=1, page_stride=0), **kw) == g.GDN_OK


def table(**kw):
    from gated_deltanet_state_gdn_b200._paged import _Table
    a = dict(block_table=P(1), ref_count=P(2), seq_lens=P(3), table_stride=8, rows=4, width=8, num_pages=20,
             page_size=16)
    a.update(kw)
    return _Table(*[a[n] for n, _ in _Table._fields_])


def pools(*rows):
    from gated_deltanet_state_gdn_b200._paged import _Pool
    return (_Pool * max(len(rows), 1))(*[_Pool(*r) for r in rows]), len(rows)


def test_page_refusals(g):
    L = g.lib()

    def resize(t=None, p=(), r=P(5), n=P(6), count=3, ws=P(7), nbytes=1 << 20):
        arr, k = pools(*p)
        return L.gdn_page_resize(None if t is False else ctypes.byref(t or table()), r, n, count, arr, k, ws,
                                 nbytes, None, None)

    def fork(t=None, p=(), a=P(5), b=P(6), count=3):
        arr, k = pools(*p)
        return L.gdn_page_fork(None if t is False else ctypes.byref(t or table()), a, b, count, arr, k, None, None)

    def compact(t=None, p=(), m=P(5), ws=P(7), nbytes=1 << 20):
        arr, k = pools(*p)
        return L.gdn_page_compact(None if t is False else ctypes.byref(t or table()), m, arr, k, ws, nbytes, None,
                                  None)

    for f in (resize, fork, compact):
        assert f(False) == g.GDN_ERR_NULL
        for n in ("block_table", "ref_count", "seq_lens"):
            assert f(table(**{n: None})) == g.GDN_ERR_NULL
        for n in ("rows", "width", "num_pages", "page_size"):
            assert f(table(**{n: 0})) == g.GDN_ERR_SHAPE
        assert f(table(table_stride=7)) == g.GDN_ERR_SHAPE
        assert f(table(width=1 << 27, table_stride=1 << 27)) == g.GDN_ERR_UNSUPPORTED
        assert f(table(ref_count=P(2, 2))) == g.GDN_ERR_ALIGN
        assert f(table(ref_count=P(1, 64))) == g.GDN_ERR_ALIAS
        assert f(p=[(None, 64, 64)]) == g.GDN_ERR_NULL
        assert f(p=[(P(8), 64, 128)]) == g.GDN_ERR_SHAPE            # rows over one another
        assert f(p=[(P(8), 64, 0)]) == g.GDN_ERR_SHAPE
        assert f(p=[(P(8), 64, 64), (P(8), 64, 64)]) == g.GDN_ERR_ALIAS
        assert f(p=[(P(3, 4), 64, 64)]) == g.GDN_ERR_ALIAS          # a pool over the table
    assert resize(r=None) == g.GDN_ERR_NULL and resize(ws=None) == g.GDN_ERR_NULL
    assert resize(nbytes=64) == g.GDN_ERR_SHAPE and compact(nbytes=64) == g.GDN_ERR_SHAPE
    assert resize(count=-1) == g.GDN_ERR_SHAPE and fork(count=-1) == g.GDN_ERR_SHAPE
    assert resize(n=P(6, 2)) == g.GDN_ERR_ALIGN and compact(ws=P(7, 4)) == g.GDN_ERR_ALIGN
    assert resize(r=P(3, 4)) == g.GDN_ERR_ALIAS and fork(b=P(1, 8)) == g.GDN_ERR_ALIAS
    assert compact(m=P(2)) == g.GDN_ERR_ALIAS and compact(m=P(7, 16)) == g.GDN_ERR_ALIAS
    assert compact(p=[(P(8), 64, 64)], m=P(8, 128)) == g.GDN_ERR_ALIAS
    assert resize(count=0) == g.GDN_OK and fork(count=0) == g.GDN_OK
    assert L.gdn_page_workspace_size(0, 1) == 0 and L.gdn_page_workspace_size(5, -1) == 0
    assert L.gdn_page_workspace_size(20, 3) > 0 and L.gdn_page_workspace_size(20, 0) > 0


def meet(a, b, rows):
    """Whether a row of one pool shares a byte with a row of another (addresses, strides, lengths)."""
    x, y = ({(p, p + n) for p in range(at, at + (rows - 1) * s + 1, max(s, 1))} for at, s, n in (a, b))
    return any(p < e2 and p2 < e for p, e in x for p2, e2 in y)


def test_pools_over_one_another(g):
    """Pools that share bytes are refused, wherever they start; pools in each other's gaps are not.
    (No row is listed: nothing is launched.)"""
    L = g.lib()
    rng = np.random.default_rng(1)

    def fork(rows, some):
        arr, k = pools(*some)
        t = table(rows=rows)
        return L.gdn_page_fork(ctypes.byref(t), P(5), P(6), 0, arr, k, None, None)

    seen = set()
    for _ in range(3000):
        rows, n = int(rng.integers(1, 6)), int(rng.integers(2, 6))
        stride = int(rng.integers(1, 40))
        some = []
        for _ in range(n):
            s = stride if rng.random() < 0.8 else int(rng.integers(1, 90))
            some.append((P(8, int(rng.integers(0, 120))), s, int(rng.integers(1, min(s, 9) + 1))))
        want = any(meet(some[i], some[j], rows) for i in range(n) for j in range(i))
        assert fork(rows, some) == (g.GDN_ERR_ALIAS if want else g.GDN_OK), (rows, some)
        seen.add((want, len({s for _, s, _ in some}) > 1))
    assert len(seen) == 4
    # layers of one tensor, in any order and more than are gone through in order; then one too many
    for n in (2, 96, 512, 700):
        some = [(P(8, 64 * int(i)), 64 * n, 64) for i in rng.permutation(n)]
        assert fork(4, some) == g.GDN_OK
        assert fork(4, some + [(P(8, 64 * (n + 3) + 8), 64 * n, 8)]) == g.GDN_ERR_ALIAS
    apart_ = [(P(8, 1000 * int(i)), 64, 64) for i in rng.permutation(300)]
    assert fork(4, apart_) == g.GDN_OK and fork(4, apart_ + [(P(8, 255), 64, 1)]) == g.GDN_ERR_ALIAS


def test_binding_takes_gpu_tensors_only(g):
    x = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    t = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        g.gdn_paged_attn(x, x, x, t, t[0])
    with pytest.raises(TypeError, match="CUDA"):
        g.gdn_kv_append(x, x, x, x, t, t[0])
    for f in (g.gdn_page_resize, g.gdn_page_fork):
        with pytest.raises(TypeError, match="CUDA"):
            f(t, t[0], t[0], t[0], t[0], 16)
    with pytest.raises(TypeError, match="CUDA"):
        g.gdn_page_compact(t, t[0], t[0], 16)


def test_packed_structures():
    """The bytes that the binding packs are the structures that the header declares."""
    from gated_deltanet_state_gdn_b200 import _paged as p
    for cls, packed in ((p._Cache, p._CACHE_BYTES), (p._Table, p._TABLE_BYTES)):
        assert ctypes.sizeof(cls) == packed.size
        values = [1000 + 7 * i for i in range(len(cls._fields_))]
        assert bytes(cls(*values)) == packed.pack(*values)


def test_status_word():
    """What the kernels write their status to: an int32 tensor of the call's device."""
    from gated_deltanet_state_gdn_b200._paged import _status
    dev = torch.device("cpu")
    t = torch.zeros(4, dtype=torch.int32)
    assert _status(None, dev) is None and _status(t, dev) == t.data_ptr() and _status(t[2], dev) == t[2].data_ptr()
    for bad in (t.long(), t.float(), t[:0], [0], 0):
        with pytest.raises(TypeError, match="dev_status"):
            _status(bad, dev)
    with pytest.raises(TypeError, match="dev_status"):
        _status(t, torch.device("cuda", 0))


def test_row_strides():
    """What the binding takes for evenly spaced tokens, and what it copies."""
    from gated_deltanet_state_gdn_b200._paged import _row_strides
    x = torch.zeros(4, 3, 10, 64, dtype=torch.bfloat16)
    y, ts, hs = _row_strides("x", x[:, :, 2:6], 4, 64, 2)
    assert y.data_ptr() == x[:, :, 2:6].data_ptr() and (ts, hs) == (640, 64)
    y, ts, hs = _row_strides("x", x.transpose(0, 1), 10, 64, 2)      # tokens not evenly spaced
    assert y.data_ptr() != x.data_ptr() and (ts, hs) == (640, 64)
    y, ts, hs = _row_strides("x", x[0].transpose(0, 1)[None], 3, 64, 8)
    assert (ts, hs) == (64, 640)
    flat = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16)[1:].view(2, 2, 64)
    y, ts, hs = _row_strides("x", flat, 2, 64, 8)                    # off its alignment
    assert y.data_ptr() % 16 == 0 and (ts, hs) == (128, 64)
    with pytest.raises(ValueError):
        _row_strides("x", x, 4, 64, 2)


def test_pool_rows():
    """Rows of a pool may be transposed inside, but not have holes."""
    from gated_deltanet_state_gdn_b200._paged import _pools
    dev = torch.device("cpu")
    kv = torch.zeros(5, 2, 8, 4, 16, dtype=torch.bfloat16)
    arr, n = _pools([kv[:, 0].transpose(1, 2), kv[:, 1]], 5, dev)
    assert n == 2 and arr[0].row_bytes == 8 * 4 * 16 * 2 and arr[0].row_stride == 2 * arr[0].row_bytes
    assert arr[1].data == kv[:, 1].data_ptr()
    with pytest.raises(ValueError, match="dense"):
        _pools([kv[:, 0, :, 1:]], 5, dev)
    with pytest.raises(ValueError, match="rows"):
        _pools([kv], 6, dev)
    with pytest.raises(TypeError):
        _pools(kv, 5, dev)


def test_pools_without_elements():
    """The window pool of a conv of one tap, [slots, channels, 0], is taken and left out."""
    from gated_deltanet_state_gdn_b200._paged import _pools
    dev = torch.device("cpu")
    x, y = torch.zeros(5, 4), torch.zeros(5, 7)
    arr, n = _pools([torch.zeros(5, 64, 0), x, torch.zeros(5, 0), y], 5, dev)
    assert n == 2 and [arr[i].data for i in range(2)] == [x.data_ptr(), y.data_ptr()]
    assert _pools([torch.zeros(5, 64, 0)], 5, dev)[1] == 0
    with pytest.raises(ValueError, match="rows"):
        _pools([torch.zeros(4, 64, 0)], 5, dev)


# ---------------------------------------------------------------- the models themselves
def test_model_of_attention():
    """Against torch's own softmax on whole rows, and a window and a cut by hand."""
    c = Case(1, [7, 0, 20], T=2, device="cpu", dtype=torch.float16)
    out, lse, size, dx, count = attend(c)
    row = c.table[int(c.slots[2])]
    k, v = (torch.cat([x[int(p)] for p in row[:2]])[:20].double() for x in (c.k, c.v))
    x = torch.einsum("hgd,lhd->hgl", c.q[2, 1].double().reshape(2, 2, 64), k) / 8
    want = torch.einsum("hgl,lhd->hgd", torch.softmax(x, -1), v).reshape(4, 64)
    np.testing.assert_allclose(out[2, 1], want.numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(lse[2, 1], torch.logsumexp(x, -1).reshape(-1).numpy(), rtol=1e-12)
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all() and count[2, 0, 0] == 19
    assert attend(c, window=3)[4][2, 1, 0] == 3 and attend(c, window=1)[4][0, 0, 0] == 1
    one = attend(c, window=1)[0][2, 1, 0]
    np.testing.assert_allclose(one, v[19, 0].numpy())


def test_model_of_tables():
    """A few steps by hand: shared pages, copies, the lowest free pages, compaction."""
    t = Tables(torch.full((3, 4), -1), torch.zeros(8, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 4)
    x = torch.arange(8)
    t.resize([1], [6], [x])
    assert t.t[1] == [0, 1, -1, -1] and t.ref[:3] == [1, 1, 0] and t.seq == [0, 6, 0]
    t.fork([1], [2])
    assert t.t[2] == t.t[1] and t.ref[:2] == [2, 2]
    t.resize([2], [7], [x])
    assert t.t[2] == [0, 2, -1, -1] and t.ref[:3] == [2, 1, 1] and x.tolist() == [0, 1, 1, 3, 4, 5, 6, 7]
    t.resize([1], [0])
    assert t.ref[:3] == [1, 0, 1] and t.t[1] == [-1] * 4
    assert t.compact([x]) == [0, -1, 1, -1, -1, -1, -1, -1]
    assert t.t[2] == [0, 1, -1, -1] and t.ref[:3] == [1, 1, 0]
    assert t.status == 0
