"""gdn_page_resize, gdn_page_fork and gdn_page_compact against a model of plain lists, call by
call; and the cache's calls together, as a decoding loop makes them."""
import math

import numpy as np
import pytest
import torch

from _paged import Case, Tables, attend, check_attend, pages_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_state_gdn_b200 as g
    g.lib()
    return g


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class State:
    def __init__(self, rows, width, P, page, pools=2, slots=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.page = page
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(P, dtype=torch.int32, device="cuda")
        self.seq = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.pools = [torch.randn(P, page, 2, 8, device="cuda", generator=g).to(torch.bfloat16)
                      for _ in range(pools)]
        self.slots = [torch.randn(rows, 3, 5, device="cuda", generator=g) for _ in range(slots)]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.model = Tables(self.table.cpu(), self.ref.cpu(), self.seq.cpu(), page)
        self.mp = [x.clone() for x in self.pools]
        self.ms = [x.clone() for x in self.slots]

    def check(self):
        self.model.same(self.table.cpu(), self.ref.cpu(), self.seq.cpu())
        for a, b in zip(self.pools + self.slots, self.mp + self.ms):
            assert torch.equal(a, b)
        assert int(self.status.item()) == self.model.status

    def resize(self, gdn, rows, lens):
        gdn.gdn_page_resize(self.table, self.ref, self.seq, ints(rows), ints(lens), self.page,
                            self.pools, dev_status=self.status)
        self.model.resize(rows, lens, self.mp)
        self.check()

    def fork(self, gdn, parents, children):
        gdn.gdn_page_fork(self.table, self.ref, self.seq, ints(parents), ints(children), self.page,
                          self.slots, dev_status=self.status)
        self.model.fork(parents, children, self.ms)
        self.check()

    def compact(self, gdn):
        to = gdn.gdn_page_compact(self.table, self.ref, self.seq, self.page, self.pools,
                                  dev_status=self.status)
        assert to.tolist() == self.model.compact(self.mp)
        self.check()


def test_grow_shrink_free(gdn):
    s = State(6, 9, 40, 4)
    s.resize(gdn, [3, 0, 5], [10, 1, 36])
    s.resize(gdn, [0, 3], [4, 3])              # within a page; back by pages
    s.resize(gdn, [3, 1, 0], [0, 8, 5])        # what one gives another takes
    s.resize(gdn, [-1, 2, -4], [7, 4, 2])      # padding
    s.resize(gdn, [5], [36])                   # the same length
    assert s.model.status == 0


def test_out_of_pages(gdn):
    s = State(5, 8, 10, 4)
    s.resize(gdn, [0, 1], [12, 8])
    s.resize(gdn, [1, 2, 0, 3], [20, 12, 12, 4])    # three more, then two are left: row 2 and 3 wait
    assert s.model.status == gdn.GDN_DEV_NO_PAGES
    s.resize(gdn, [1, 2], [0, 28])
    s.resize(gdn, [0, 4], [0, 32])


def test_bad_requests(gdn):
    s = State(4, 5, 30, 4)
    s.resize(gdn, [0, 1], [6, 9])
    s.resize(gdn, [0, 1, 0, 2], [8, 4, 9, 3])       # row 0 twice: neither
    s.resize(gdn, [4, 2, 99], [1, 5, 1])
    s.resize(gdn, [2, 1, 3], [21, -1, 20])
    s.model.seq[3] = 77
    s.seq[3] = 77
    s.resize(gdn, [3], [4])
    assert s.model.status == gdn.GDN_DEV_CONFLICT | gdn.GDN_DEV_BAD_SLOT | gdn.GDN_DEV_BAD_LENGTH


def test_bad_table_entries(gdn):
    s = State(4, 6, 30, 4)
    s.resize(gdn, [0, 1, 2], [18, 18, 6])
    for r, j, v in ((0, 3, 30), (1, 4, -5)):
        s.table[r, j] = v
        s.model.t[r][j] = v
    s.resize(gdn, [0, 1], [2, 20])    # a bad page is dropped; a bad last page cannot be grown into
    s.fork(gdn, [1], [3])
    s.compact(gdn)
    assert s.model.status == gdn.GDN_DEV_BAD_PAGE


def test_fork_and_copy_on_growth(gdn):
    s = State(8, 9, 60, 4)
    s.resize(gdn, [0, 1], [10, 8])
    s.fork(gdn, [0, 0, 1, 4], [2, 3, 5, -1])
    s.resize(gdn, [2], [11])                # its own copy of the last page
    s.resize(gdn, [0, 3], [14, 11])         # both share still: both copy
    s.resize(gdn, [5, 1], [9, 9])           # the last page is full: nothing to copy
    s.resize(gdn, [2], [6])                 # into a page that others hold
    s.resize(gdn, [2], [7])
    s.fork(gdn, [2, 0], [5, 3])             # children that held pages
    s.fork(gdn, [2, 0], [5, 3])             # again
    s.resize(gdn, [3, 5], [0, 0])
    assert s.model.status == 0


def test_fork_conflicts(gdn):
    s = State(8, 4, 60, 4)
    s.resize(gdn, [0, 1, 2], [10, 8, 3])
    s.fork(gdn, [0, 1, 2], [3, 3, 4])       # one child twice
    s.fork(gdn, [0, 4, 5], [4, 5, 5])       # a chain, a self
    s.fork(gdn, [0, 8, 1], [8, 6, 6])       # rows that are not there
    s.seq[7] = -4
    s.model.seq[7] = -4
    s.fork(gdn, [7, 0], [6, 7])
    assert s.model.status & gdn.GDN_DEV_CONFLICT and s.model.status & gdn.GDN_DEV_BAD_SLOT


@pytest.mark.parametrize("P", [1, 2, 7, 64, 1000])
@pytest.mark.parametrize("share", [0.0, 0.3, 0.9, 1.0])
def test_compact(gdn, P, share):
    rng = np.random.default_rng(P)
    s = State(4, P + 1, P, 2)
    used = sorted(rng.permutation(P)[:int(round(P * share))].tolist())
    order = rng.permutation(used).tolist()
    half = len(order) // 2
    for r, pages in ((1, order[:half]), (3, order[half:])):
        for j, p in enumerate(pages):
            s.model.t[r][j] = p
            s.model.ref[p] = int(rng.integers(1, 4))
        s.model.seq[r] = max(2 * len(pages) - 1, 0)
    s.table.copy_(torch.tensor(s.model.t))
    s.ref.copy_(torch.tensor(s.model.ref))
    s.seq.copy_(torch.tensor(s.model.seq))
    s.compact(gdn)
    s.compact(gdn)                          # nothing to move
    assert s.model.status == 0


@pytest.mark.parametrize("seed", range(4))
def test_random_walks(gdn, seed):
    rng = np.random.default_rng(seed)
    rows, page = int(rng.integers(2, 40)), int(rng.integers(1, 9))
    s = State(rows, int(rng.integers(3, 30)), int(rng.integers(10, 400)), page, seed=seed)
    cap = s.model.width * page
    for _ in range(25):
        what = rng.random()
        n = int(rng.integers(1, rows + 1))
        if what < 0.6:
            r = rng.permutation(rows)[:n]
            lens = [int(rng.integers(0, cap + 1)) if rng.random() < 0.5
                    else min(cap, max(0, s.model.seq[i] + int(rng.integers(-3, 6)))) for i in r]
            s.resize(gdn, r.tolist(), lens)
        elif what < 0.85:
            r = rng.permutation(rows)
            k = max(1, rows // 2)
            s.fork(gdn, rng.choice(r[:k], k).tolist()[:rows - k], r[k:2 * k].tolist()[:rows - k])
        else:
            s.compact(gdn)


def test_many_rows_and_pages(gdn):
    # more listed rows than a block has threads, more pages than the cluster takes in one pass
    rows, P = 2500, 60000
    s = State(rows, 130, P, 1, pools=1, slots=1, seed=9)
    rng = np.random.default_rng(2)
    s.resize(gdn, list(range(rows)), [int(x) for x in rng.integers(0, 40, rows)])
    s.resize(gdn, rng.permutation(rows)[:1500].tolist(), [int(x) for x in rng.integers(0, 45, 1500)])
    s.resize(gdn, [5, 7], [130, 0])
    s.compact(gdn)
    assert s.model.status == 0


def test_small_steps_of_a_wide_table(gdn):
    """Decoding steps: hundreds of rows of a wide table, each longer by a token or two, or cut."""
    rng = np.random.default_rng(8)
    s = State(400, 100, 5000, 4, pools=1, slots=1, seed=8)
    rows = rng.permutation(400).tolist()
    s.resize(gdn, rows, [int(x) for x in rng.integers(1, 30, 400)])
    for step in range(6):
        rows = rng.permutation(400)[:380].tolist()
        s.resize(gdn, rows, [max(0, s.model.seq[r] + int(rng.integers(-2, 4))) for r in rows])
        if step == 2:
            s.fork(gdn, [int(x) for x in range(50)], [int(x) for x in range(350, 400)])
    assert s.model.status == 0


@pytest.mark.parametrize("n", [700, 2000, 3500])
def test_rows_listed_twice(gdn, n):
    """Among hundreds and thousands of listed rows (some of them far past the table), a few twice."""
    rng = np.random.default_rng(n)
    s = State(4000, 3, 9000, 4, pools=1, slots=1, seed=n)
    rows = rng.permutation(4000)[:n].tolist()
    for i in range(0, n - 50, 97):
        rows[i + 50] = rows[i]
    rows[3] = rows[4] = 0x7fffffff
    rows[8] = -3
    s.resize(gdn, rows, [int(x) for x in rng.integers(0, 13, n)])
    assert s.model.status == gdn.GDN_DEV_CONFLICT | gdn.GDN_DEV_BAD_SLOT


def test_many_children(gdn):
    s = State(1800, 4, 300, 4, pools=1, slots=1, seed=3)
    s.resize(gdn, [7, 9], [13, 6])
    s.fork(gdn, [7] * 900 + [9] * 800, list(range(10, 910)) + list(range(950, 1750)))
    # a copy of the shared last page for each: 290 of the 300 - 4 - 2 free pages
    s.resize(gdn, list(range(10, 300)), [14] * 290)
    assert s.model.status == 0
    s.resize(gdn, list(range(300, 310)), [14] * 10)       # four are left
    assert s.model.status == gdn.GDN_DEV_NO_PAGES


def test_more_asked_for_than_32_bits_count(gdn):
    """2200 rows that ask for a million pages each: more than 2^31 in all, of a hundred there are.
    The row ahead of them fits; the ones behind the shortage wait, however little they ask for."""
    rows, width, P = 2203, 1 << 20, 100
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    ref, seq, st = ints([0] * P), ints([0] * rows), ints([0])
    lens = [60] + [width] * 2200 + [3, 0]
    gdn.gdn_page_resize(table, ref, seq, ints(list(range(rows))), ints(lens), 1, dev_status=st)
    assert int(st.item()) == gdn.GDN_DEV_NO_PAGES
    assert seq.tolist() == [60] + [0] * 2202
    assert ref.tolist() == [1] * 60 + [0] * 40 and table[0, :61].tolist() == list(range(60)) + [-1]
    assert int((table[1:] != -1).sum()) == 0


def test_no_rows(gdn):
    s = State(3, 3, 5, 4)
    s.resize(gdn, [], [])
    s.fork(gdn, [], [])


@pytest.mark.parametrize("shape,dtype", [((8, 128), torch.bfloat16), ((5,), torch.float32),
                                         ((7,), torch.bfloat16), ((9,), torch.uint8),
                                         ((9, 4099), torch.bfloat16), ((3, 16384), torch.uint8)])
def test_pools_of_all_widths(gdn, shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.randint(0, 250, (12, *shape), device="cuda", generator=g).to(dtype)
    other = torch.randint(0, 250, (2, 12, *shape), device="cuda", generator=g).to(dtype)
    want, ow = pool.clone(), other.clone()
    table = torch.full((12, 2), -1, dtype=torch.int32, device="cuda")
    ref = torch.zeros(4, dtype=torch.int32, device="cuda")
    seq = torch.zeros(12, dtype=torch.int32, device="cuda")
    gdn.gdn_page_fork(table, ref, seq, ints([3, 3, 0]), ints([7, 11, 1]), 4, [pool, other[1]])
    for p, c in ((3, 7), (3, 11), (0, 1)):
        want[c] = want[p]
        ow[1, c] = ow[1, p]
    assert torch.equal(pool, want) and torch.equal(other, ow)


def test_more_pools_than_a_launch_takes(gdn):
    big = torch.randn(250, 6, 40, device="cuda")
    want = big.clone()
    table = torch.full((6, 2), -1, dtype=torch.int32, device="cuda")
    ref, seq = ints([0] * 6), ints([0] * 6)
    gdn.gdn_page_fork(table, ref, seq, ints([2]), ints([5]), 4, list(big.unbind(0)))
    want[:, 5] = want[:, 2]
    assert torch.equal(big, want)
    # pages 1, 4 and 5 are used: 4 moves to 0 and 5 to 2, in every pool
    table[0, 0], seq[0] = 4, 3
    table[1, :2], seq[1] = ints([1, 5]), 5
    ref.copy_(ints([0, 1, 0, 0, 1, 1]))
    to = gdn.gdn_page_compact(table, ref, seq, 4, list(big.unbind(0)))
    want[:, 0], want[:, 2] = want[:, 4].clone(), want[:, 5].clone()
    assert torch.equal(big, want) and to.tolist() == [-1, 1, -1, -1, 0, 2]
    assert table[0].tolist() == [0, -1] and table[1].tolist() == [1, 2]


# ---------------------------------------------------------------- together
def decode_loop(gdn, dtype, cache, steps=12, stream=None):
    """Prompts, steps of two tokens of which one is sometimes taken back, a fork, a compaction:
    after each step the attention must be that of the tokens each row has, kept apart in lists."""
    page, H, Hq, D, T = 4, 2, 4, 64, 2
    rows, P = 6, 120
    g = torch.Generator(device="cuda").manual_seed(5)
    new = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    k, v = (torch.full((P, page, H, D), math.nan, device="cuda").to(cache) for _ in range(2))
    state = new(rows, 4, 3)
    table = torch.full((rows, 30), -1, dtype=torch.int32, device="cuda")
    ref, seq = ints([0] * P), ints([0] * rows)
    st = ints([0])
    have = {r: [] for r in range(rows)}             # (key, value) of each position
    scale = dict(k_scale=torch.tensor([0.03, 0.05], device="cuda"),
                 v_scale=torch.tensor([0.04, 0.02], device="cuda")) if cache == torch.float8_e4m3fn else {}

    def stored(x, s):
        x = x.to(dtype)
        if not scale:
            return x.float()
        s = scale[s]
        return (x.float() / s[:, None]).clamp(-448, 448).to(cache).float() * s[:, None]

    def append(live, counts):
        n = sum(counts)
        kk, vv = new(n, H, D).to(dtype), new(n, H, D).to(dtype)
        off = ints(np.concatenate([[0], np.cumsum(counts)]).tolist())
        gdn.gdn_page_resize(table, ref, seq, ints(live), ints([len(have[r]) + c for r, c in zip(live, counts)]),
                            page, [k, v], dev_status=st)
        gdn.gdn_kv_append(kk, vv, k, v, table, seq, ints(live), off, dev_status=st, **scale)
        at = 0
        for r, c in zip(live, counts):
            have[r] = have[r] + [(stored(kk[i], "k_scale"), stored(vv[i], "v_scale")) for i in range(at, at + c)]
            at += c

    live = [4, 0, 2]
    append(live, [7, 1, 12])
    for step in range(steps):
        append(live, [T] * len(live))
        q = new(len(live), T, Hq, D).to(dtype)
        out, lse = gdn.gdn_paged_attn(q, k, v, table, seq, ints(live), return_lse=True, dev_status=st, **scale)
        for i, r in enumerate(live):
            kr, vr = (torch.stack([x[j] for x in have[r]]).double() for j in (0, 1))
            for t in range(T):
                m = len(have[r]) - T + t + 1
                x = torch.einsum("hgd,lhd->hgl", q[i, t].double().reshape(H, Hq // H, D), kr[:m]) / 8
                w = torch.softmax(x, -1)
                ref_o = torch.einsum("hgl,lhd->hgd", w, vr[:m]).reshape(Hq, D)
                size = torch.einsum("hgl,lhd->hgd", w, vr[:m].abs()).reshape(Hq, D)
                half = torch.finfo(dtype).eps / 2
                lim = half * 1.01 * ref_o.abs() + (half * 1.01 + 2.0 ** -14) * size
                assert ((out[i, t].double() - ref_o).abs() <= lim).all(), (step, r, t)
                assert ((lse[i, t].double() - torch.logsumexp(x, -1).reshape(-1)).abs() < 2.0 ** -14).all()
        if step % 3 == 0:                           # a token is not accepted
            back = live[step % len(live)]
            have[back] = have[back][:-1]
            gdn.gdn_page_resize(table, ref, seq, ints([back]), ints([len(have[back])]), page, [k, v], dev_status=st)
        if step == 4:
            gdn.gdn_page_fork(table, ref, seq, ints([4, 4]), ints([1, 5]), page, [state], dev_status=st)
            have[1], have[5] = list(have[4]), list(have[4])
            live = [4, 0, 2, 5, 1]
            assert torch.equal(state[1], state[4]) and torch.equal(state[5], state[4])
        if step == 8:
            gdn.gdn_page_resize(table, ref, seq, ints([0, 4]), ints([0, 0]), page, [k, v], dev_status=st)
            have[0], have[4] = [], []
            live = [2, 5, 1]
            gdn.gdn_page_compact(table, ref, seq, page, [k, v], dev_status=st)
            assert (ref[:int((ref > 0).sum())] > 0).all()
    assert int(st.item()) == 0
    held = sum(pages_of(len(have[r]), page) for r in live)
    assert int(ref.sum()) == held


@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                         (torch.bfloat16, torch.float8_e4m3fn)])
def test_decoding_loop(gdn, dtype, cache):
    decode_loop(gdn, dtype, cache)
