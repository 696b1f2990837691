"""The paged cache's calls as programs use them: captured graphs, several streams, the checked
build, a wait that runs out."""
import time

import pytest
import torch

from _paged import Case, attend, check_attend

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_state_gdn_b200 as g
    from gated_deltanet_state_gdn_b200 import build
    build.build(checked=True)   # rebuilds only when missing or older than the sources
    product = g._binding.LIB_PATH
    yield g
    g.use_library(product)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """A cache and the tensors of one decoding step over it."""

    def __init__(self, seed, rows=6, T=2, H=2, Hq=8, D=128, page=16, cache=torch.bfloat16):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.page, self.H, self.D = T, page, H, D
        self.P = 80
        self.k, self.v = (torch.randn(self.P, page, H, D, device="cuda", generator=g).to(torch.bfloat16).to(cache)
                          for _ in range(2))
        self.table = torch.full((rows, 20), -1, dtype=torch.int32, device="cuda")
        self.ref, self.seq = ints([0] * self.P), ints([0] * rows)
        self.slots = ints(list(range(rows))[::-1])
        self.lens = ints([5, 17, 40, 3, 64, 90])
        self.rows = ints(list(range(rows)))
        new = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
        self.q, self.kn, self.vn = new(rows, T, Hq, D), new(rows, T, H, D), new(rows, T, H, D)
        self.out = torch.zeros_like(self.q)
        self.status = ints([0])

    def start(self, gdn):
        gdn.gdn_page_resize(self.table, self.ref, self.seq, self.rows, self.lens, self.page, [self.k, self.v])

    def step(self, gdn, **kw):
        gdn.gdn_page_resize(self.table, self.ref, self.seq, self.rows, self.lens, self.page, [self.k, self.v],
                            dev_status=self.status, **kw)
        gdn.gdn_kv_append(self.kn, self.vn, self.k, self.v, self.table, self.seq, self.slots, dev_status=self.status,
                          **kw)
        return gdn.gdn_paged_attn(self.q, self.k, self.v, self.table, self.seq, self.slots, out=self.out,
                                  dev_status=self.status, **kw)

    def everything(self):
        return [x.clone() for x in (self.table, self.ref, self.seq, self.k, self.v, self.out)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.dtype == E4M3 else x,
                           y.view(torch.uint8) if y.dtype == E4M3 else y) for x, y in zip(a, b))


def advance(s, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s.lens += s.T
    for x in (s.q, s.kn, s.vn):
        x.copy_(torch.randn(x.shape, device="cuda", generator=g))


@pytest.mark.parametrize("cache", [torch.bfloat16, E4M3])
def test_captured_step_replays(gdn, cache):
    """A whole step captured once and replayed on new inputs does what the calls do one by one."""
    a, b = Server(1, cache=cache), Server(1, cache=cache)
    a.start(gdn)
    b.start(gdn)
    for s in (a, b):
        advance(s, 7)
    a.step(gdn)                         # warm-up outside the capture
    b.step(gdn)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    advance(a, 8)
    advance(b, 8)
    keep = a.everything()
    with torch.cuda.graph(graph):
        a.step(gdn)
    assert same(keep, a.everything())   # a capture runs nothing
    for n in range(5):
        graph.replay()
        b.step(gdn)
        torch.cuda.synchronize()
        assert same(a.everything(), b.everything()), n
        for s in (a, b):
            advance(s, 20 + n)
    assert int(a.status.item()) == 0


def test_two_graphs_and_two_streams_at_once(gdn):
    """Two captured steps replayed at the same time, and two eager ones on streams of their own,
    do not meet."""
    servers = [Server(s) for s in range(4)]
    alone = [Server(s) for s in range(4)]
    for s in servers + alone:
        s.start(gdn)
        advance(s, 3)
        s.step(gdn)
        advance(s, 4)
    for s in alone:
        s.step(gdn)
    torch.cuda.synchronize()
    graphs = []
    for s in servers[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step(gdn)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for g, st in zip(graphs, streams):
        with torch.cuda.stream(st):
            g.replay()
    for s, st in zip(servers[2:], streams[2:]):
        s.step(gdn, stream=st)
    torch.cuda.synchronize()
    for s, x in zip(servers, alone):
        assert same(s.everything(), x.everything())


def test_given_stream_orders_the_call(gdn):
    """`stream` runs the whole call there, copies of its arguments included: inputs that the stream
    itself makes late are seen, on a stream that is not the current one."""
    c = Case(3, [500, 20, 90], T=1, D=128)
    want = c.attend(gdn)
    args = [c.to(x) for x in (c.q, c.k, c.v, c.table, c.seq, c.slots)]
    q = torch.zeros(3, 4, 1, 128, dtype=torch.bfloat16, device="cuda").transpose(1, 2)[:, :, ::1]
    late = torch.zeros(3, 1, 4, 132, dtype=torch.bfloat16, device="cuda")[..., 1:129]   # off its alignment
    st = torch.cuda.Stream()
    big = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(20):
            big.add_(1.0)               # keeps the stream busy for a while
        late.copy_(args[0])
        q.copy_(args[0])
    got = gdn.gdn_paged_attn(late, *args[1:], return_lse=True, stream=st)
    got2 = gdn.gdn_paged_attn(q, *args[1:], return_lse=True, stream=st)
    st.synchronize()
    assert same(got, want) and same(got2, want)


def test_captured_tables_replay(gdn):
    """A fork, a growth into shared pages and a compaction, captured together."""
    a, b = Server(11), Server(11)
    states = [torch.randn(6, 4, 33, device="cuda") for _ in range(2)]
    states[1].copy_(states[0])

    def turn(s, state):
        gdn.gdn_page_fork(s.table, s.ref, s.seq, ints_[0], ints_[1], s.page, [state], dev_status=s.status)
        gdn.gdn_page_resize(s.table, s.ref, s.seq, s.rows, s.lens, s.page, [s.k, s.v], dev_status=s.status)
        return gdn.gdn_page_compact(s.table, s.ref, s.seq, s.page, [s.k, s.v], dev_status=s.status)

    ints_ = ints([2, 2, 5]), ints([0, 4, 1])
    for s in (a, b):
        s.start(gdn)
    for s, state in zip((a, b), states):
        turn(s, state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        to = turn(a, states[0])
    for n in range(4):
        for s in (a, b):
            s.lens.copy_(ints([9 + n, 70, 33 + 2 * n, 5, 64 - 7 * n, 90]))
        states[0][n] += 1
        states[1][n] += 1
        graph.replay()
        want = turn(b, states[1])
        torch.cuda.synchronize()
        assert same(a.everything(), b.everything()) and torch.equal(states[0], states[1])
        assert torch.equal(to, want)
    assert int(a.status.item()) == 0


def test_views_of_larger_tensors(gdn):
    """Keys and values of one tensor, heads cut out of it, a table that is part of a wider one."""
    a, b = Server(12), Server(12)
    kv = torch.zeros(b.P, 2, b.page, 5, b.D, dtype=torch.bfloat16, device="cuda")
    kv[:, 0, :, 1:3], kv[:, 1, :, 1:3] = b.k, b.v
    b.k, b.v = kv[:, 0, :, 1:3], kv[:, 1, :, 1:3]
    wide = torch.full((6, 33), -9, dtype=torch.int32, device="cuda")
    wide[:, 4:24] = b.table
    b.table = wide[:, 4:24]
    pages = [kv[:, 0], kv[:, 1]]
    for s, pools in ((a, [a.k, a.v]), (b, pages)):
        gdn.gdn_page_resize(s.table, s.ref, s.seq, s.rows, s.lens, s.page, pools)
        gdn.gdn_page_fork(s.table, s.ref, s.seq, ints([5]), ints([3]), s.page)
        s.lens[3] = 90
        advance(s, 2)
        gdn.gdn_page_resize(s.table, s.ref, s.seq, s.rows, s.lens, s.page, pools)
        gdn.gdn_kv_append(s.kn, s.vn, s.k, s.v, s.table, s.seq, s.slots)
        gdn.gdn_paged_attn(s.q, s.k, s.v, s.table, s.seq, s.slots, out=s.out)
        gdn.gdn_page_compact(s.table, s.ref, s.seq, s.page, pools)
    assert same(a.everything(), b.everything())
    assert (kv[:, :, :, 0] == 0).all() and (kv[:, :, :, 3:] == 0).all()
    assert (wide[:, :4] == -9).all() and (wide[:, 24:] == -9).all()


@pytest.mark.parametrize("D,cache", [(8, torch.bfloat16), (16, E4M3), (256, torch.float16)])
def test_smallest_cache(gdn, D, cache):
    """One page of one token of one head."""
    dtype = torch.float16 if cache == torch.float16 else torch.bfloat16
    k, v = (torch.zeros(1, 1, 1, D, device="cuda").to(cache) for _ in range(2))
    table, seq = ints([[0]]), ints([1])
    kn = torch.randn(1, 1, 1, D, device="cuda").to(dtype)
    gdn.gdn_kv_append(kn, -kn, k, v, table, seq)
    assert torch.equal(k.float(), kn.to(cache).float()) and torch.equal(v.float(), (-kn).to(cache).float())
    out, lse = gdn.gdn_paged_attn(kn, k, v, table, seq, return_lse=True)
    assert torch.equal(out.float(), v.float().to(dtype).float())
    x = (kn.double() * k.double()).sum() / D ** 0.5
    assert abs(float(lse) - float(x)) <= (D + 8) * 2.0 ** -22 * float((kn.double() * k.double()).abs().sum())


def test_wrong_devices_are_refused(gdn):
    c = Case(4, [5])
    args = [c.to(x) for x in (c.q, c.k, c.v, c.table, c.seq, c.slots)]
    for i in range(6):
        bad = list(args)
        bad[i] = args[i].cpu()
        with pytest.raises(TypeError):
            gdn.gdn_paged_attn(*bad)
    with pytest.raises(ValueError):
        gdn.gdn_paged_attn(args[0], args[1], args[2].transpose(1, 2).contiguous().transpose(1, 2), *args[3:])
    with pytest.raises(ValueError):
        gdn.gdn_paged_attn(args[0][..., ::2], *args[1:])
    with pytest.raises(TypeError):
        gdn.gdn_paged_attn(args[0].float(), *args[1:])
    with pytest.raises(TypeError):
        gdn.gdn_paged_attn(*args[:5], args[5].long())
    with pytest.raises(gdn.GdnError):
        gdn.gdn_paged_attn(args[0].half(), *args[1:])
    with pytest.raises(gdn.GdnError):
        gdn.gdn_paged_attn(args[0].expand(1, 17, 4, 64).contiguous(), *args[1:])
    with pytest.raises(ValueError):
        gdn.gdn_paged_attn(*args, lse=torch.zeros(1, 1, 3, device="cuda"))


def test_status_on_the_host_is_refused(gdn):
    s = Server(21)
    calls = [lambda st: gdn.gdn_kv_append(s.kn, s.vn, s.k, s.v, s.table, s.seq, s.slots, dev_status=st),
             lambda st: gdn.gdn_paged_attn(s.q, s.k, s.v, s.table, s.seq, s.slots, dev_status=st),
             lambda st: gdn.gdn_page_resize(s.table, s.ref, s.seq, s.rows, s.lens, s.page, dev_status=st),
             lambda st: gdn.gdn_page_fork(s.table, s.ref, s.seq, ints([0]), ints([1]), s.page, dev_status=st),
             lambda st: gdn.gdn_page_compact(s.table, s.ref, s.seq, s.page, dev_status=st)]
    before = s.everything()
    for call in calls:
        for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, device="cuda"),
                    torch.zeros(1, dtype=torch.int64, device="cuda")):
            with pytest.raises(TypeError, match="dev_status"):
                call(bad)
    assert same(before, s.everything())


def both(gdn, fn):
    """fn(status) through the product library, then through the checked build."""
    product = gdn._binding.LIB_PATH
    r0 = fn(None)
    st = ints([0])
    gdn.use_library(gdn.CHECKED_LIB_PATH)
    try:
        r1 = fn(st)
    finally:
        gdn.use_library(product)
    return r0, r1, int(st.item())


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float16, E4M3])
@pytest.mark.parametrize("D,Hq,T,page", [(64, 4, 1, 16), (128, 4, 5, 24), (48, 32, 2, 1), (256, 16, 4, 272),
                                         (192, 2, 1, 16)])
def test_attention_in_bounds(gdn, cache, D, Hq, T, page):
    dtype = torch.float16 if cache == torch.float16 else torch.bfloat16
    c = Case(D, [1, 0, 900, 17, 64, 3], D=D, Hq=Hq, T=T, page=page, dtype=dtype, cache=cache, pad=(3,))
    r0, r1, st = both(gdn, lambda status: c.attend(gdn, window=300, dev_status=status))
    assert st == 0 and same(r0, r1)


@pytest.mark.parametrize("cache", [torch.bfloat16, E4M3])
def test_append_and_tables_in_bounds(gdn, cache):
    def run(status):
        s = Server(5, cache=cache)
        s.status = status
        s.start(gdn)
        advance(s, 1)
        s.step(gdn)
        state = torch.arange(6 * 1001, device="cuda", dtype=torch.float32).reshape(6, 1001)
        gdn.gdn_page_fork(s.table, s.ref, s.seq, ints([1, 2, -1]), ints([5, 0, 3]), s.page, [state], dev_status=status)
        s.lens += 3
        gdn.gdn_page_resize(s.table, s.ref, s.seq, s.rows, s.lens, s.page, [s.k, s.v], dev_status=status)
        gdn.gdn_page_resize(s.table, s.ref, s.seq, ints([3, 0]), ints([0, 7]), s.page, [s.k, s.v], dev_status=status)
        to = gdn.gdn_page_compact(s.table, s.ref, s.seq, s.page, [s.k, s.v], dev_status=status)
        return s.everything() + [state, to]
    r0, r1, st = both(gdn, run)
    assert st == 0 and same(r0, r1)


def test_attention_wait_runs_out_on_request(gdn):
    """GDN_DEV_TEST_STALL makes the first tile of the call expect 16 bytes more than its copies
    deliver: its waits run out after about a second, GDN_DEV_TIMEOUT is set, every warp leaves,
    and a normal call on the same context then matches the product library bit for bit."""
    c = Case(6, [700, 40], T=2, D=128)
    want = c.attend(gdn)
    product = gdn._binding.LIB_PATH
    gdn.use_library(gdn.CHECKED_LIB_PATH)
    try:
        st = ints([gdn.GDN_DEV_TEST_STALL])
        t0 = time.time()
        c.attend(gdn, dev_status=st)
        torch.cuda.synchronize()
        took = time.time() - t0
        s = int(st.item())
        assert s & gdn.GDN_DEV_TIMEOUT and not s & gdn.GDN_DEV_BOUNDS and took < 60
        st2 = ints([0])
        got = c.attend(gdn, dev_status=st2)
        assert int(st2.item()) == 0
    finally:
        gdn.use_library(product)
    assert same(got, want)
    check_attend(c, got, attend(c))


def test_first_calls_inside_a_capture(gdn):
    """A program whose first calls are captured, without one before: what a call sets up on the device
    it can set up there."""
    import os
    import subprocess
    import sys
    code = """if 1:
        import sys
        sys.path[:0] = ["tests", "."]
        import torch
        import gated_deltanet_state_gdn_b200 as gdn
        from test_gpu_paged_use import Server, ints, same
        a, b = Server(1), Server(1)
        wide = [torch.full((6, 40000), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
        refs = [ints([0] * 70000) for _ in range(2)]        # (planned by a cluster)
        seqs = [ints([0] * 6) for _ in range(2)]
        long = ints([9000, 1, 20000, 7, 0, 5])

        def turn(s, i):
            s.start(gdn)
            gdn.gdn_page_fork(s.table, s.ref, s.seq, ints_[0], ints_[1], s.page, dev_status=s.status)
            gdn.gdn_page_resize(s.table, s.ref, s.seq, s.rows, grown, s.page, [s.k, s.v], dev_status=s.status)
            gdn.gdn_kv_append(s.kn, s.vn, s.k, s.v, s.table, s.seq, s.slots, dev_status=s.status)
            gdn.gdn_paged_attn(s.q, s.k, s.v, s.table, s.seq, s.slots, out=s.out, dev_status=s.status)
            gdn.gdn_page_resize(wide[i], refs[i], seqs[i], s.rows, long, 1, dev_status=s.status)
            return (gdn.gdn_page_compact(s.table, s.ref, s.seq, s.page, [s.k, s.v], dev_status=s.status),
                    gdn.gdn_page_compact(wide[i], refs[i], seqs[i], 1, dev_status=s.status))

        ints_ = ints([2, 5]), ints([0, 1])
        grown = ints([42, 92, 42, 5, 66, 92])               # two tokens more each: shared pages are copied
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            to = turn(a, 0)
        graph.replay()
        want = turn(b, 1)
        torch.cuda.synchronize()
        assert same(a.everything(), b.everything()) and same(to, want)
        assert same([wide[0], refs[0], seqs[0]], [wide[1], refs[1], seqs[1]]) and int(seqs[0].sum()) == 29013
        assert int(a.status.item()) == 0
        print("replayed")
    """
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "replayed" in r.stdout, r.stdout + r.stderr
