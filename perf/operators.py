"""Cases of the paged key-value cache operators, with their plain forms.

Five kinds of case, one for each entry point of the cache (a branch also grows its rows):

  attend    gdn_paged_attn: the last T tokens of each request attend to its pages
  append    gdn_kv_append: new keys and values go to the pages of their positions
  branch    gdn_page_fork, then gdn_page_resize: children share their parents' pages, take a
            copy of their recurrent states, and grow, which copies the shared partial pages
  turnover  gdn_page_resize twice: a batch retires while another is admitted, and back
  compact   gdn_page_compact: the used pages move to the lowest numbers

Request lengths are the evenly spaced quantiles of U[lo, hi], dealt out by the seed, so that the
work of a case does not depend on the seed.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "e4m3": 1}


def listed():
    return [
        # one interactive request early in its conversation: latency counts
        dict(name="attend-one", kind="attend", B=1, pad=0, T=1, Hq=16, Hkv=2, D=128, page=16,
             lo=200, hi=200, window=0, dtype="bf16", cache="bf16", layout="tokens"),
        # a full decode batch, the rows and padding of the state-pool workload, ragged contexts
        dict(name="attend-batch", kind="attend", B=256, pad=13, T=1, Hq=32, Hkv=8, D=128, page=64,
             lo=1, hi=4096, window=0, dtype="bf16", cache="bf16", layout="tokens"),
        # one long document, wide heads: the work has to be split over the cache's length
        dict(name="attend-long", kind="attend", B=1, pad=0, T=1, Hq=16, Hkv=2, D=256, page=16,
             lo=131072, hi=131072, window=0, dtype="fp16", cache="fp16", layout="tokens"),
        # verification of four drafted tokens a row over an 8-bit cache, head-major pages
        dict(name="attend-verify-8bit", kind="attend", B=64, pad=3, T=4, Hq=16, Hkv=4, D=64,
             page=32, lo=1, hi=8192, window=0, dtype="bf16", cache="e4m3", layout="heads"),
        # the write of one decode step
        dict(name="append-step", kind="append", B=256, pad=13, lo=1, hi=1, Hkv=8, D=128, page=64,
             dtype="bf16", cache="bf16"),
        # the write of a ragged prompt batch (8 requests of U[1, 4096] tokens) into 8 bits
        dict(name="append-prompts-8bit", kind="append", B=8, pad=0, lo=1, hi=4096, Hkv=8, D=128,
             page=16, dtype="bf16", cache="e4m3"),
        # one request tried two ways, the states of the multi-token workload
        dict(name="branch-one", kind="branch", parents=1, fan=1, lo=100, hi=100, grow=4, layers=1,
             page=16, Hkv=2, D=128, states=1, Hv=16, Dv=64, conv=4096),
        # sixteen requests sampled five ways each, states of the decode workload, several layers
        dict(name="branch-samples", kind="branch", parents=16, fan=4, lo=1, hi=4096, grow=1,
             layers=4, page=64, Hkv=8, D=128, states=3, Hv=32, Dv=128, conv=8192),
        # a small server's batch changes hands
        dict(name="turnover-few", kind="turnover", rows=8, lo=1, hi=2048, page=16),
        # a large server's: thousands of rows' worth of pages change hands at once
        dict(name="turnover-many", kind="turnover", rows=512, lo=1, hi=16384, page=16),
        # a small cache is put in order
        dict(name="compact-small", kind="compact", P=500, used=0.5, rows=20, layers=1, page=16,
             Hkv=2, D=128),
        # gigabytes of pages are
        dict(name="compact-large", kind="compact", P=40000, used=0.5, rows=300, layers=2, page=16,
             Hkv=8, D=128),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "append", "branch", "turnover", "compact"])
    if kind == "attend":
        B, T = _spread(rng, 1, 300), rng.choice([1, 1, 1, 2, 3, 4, 8, 16])
        Hkv, group = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16])
        cache = rng.choice(["same", "same", "e4m3"])
        dtype = rng.choice(["bf16", "fp16"])
        D = rng.choice([64, 80, 96, 128, 192, 256])
        most = max(64, min(131072, int(9e8 / (B * Hkv * D * 4))))   # well below the largest's bytes
        hi = _spread(rng, 20, most)
        return dict(kind=kind, B=B, pad=B // 20, T=T, Hq=Hkv * group, Hkv=Hkv, D=D,
                    page=rng.choice([1, 16, 24, 32, 64, 272]), lo=rng.choice([1, hi]), hi=hi,
                    window=rng.choice([0, 0, max(1, hi // 3)]), dtype=dtype,
                    cache=dtype if cache == "same" else cache,
                    layout=rng.choice(["tokens", "heads"]))
    if kind == "append":
        B, dtype = _spread(rng, 1, 300), rng.choice(["bf16", "fp16"])
        hi = 1 if rng.random() < 0.5 else _spread(rng, 2, max(4, 16000 // B))
        return dict(kind=kind, B=B, pad=B // 20, lo=1, hi=hi, Hkv=rng.choice([1, 2, 3, 4, 8]),
                    D=rng.choice([64, 80, 128, 256]), page=rng.choice([1, 16, 24, 64, 272]),
                    dtype=dtype, cache=rng.choice([dtype, "e4m3"]))
    if kind == "branch":
        return dict(kind=kind, parents=_spread(rng, 1, 16), fan=rng.randint(1, 4), lo=1,
                    hi=_spread(rng, 20, 4000), grow=rng.choice([1, 2, 4, 16]),
                    layers=rng.randint(1, 4), page=rng.choice([16, 24, 64, 272]),
                    Hkv=rng.choice([2, 3, 8]), D=rng.choice([64, 128, 256]),
                    states=rng.randint(1, 3), Hv=rng.choice([4, 16, 32]),
                    Dv=rng.choice([64, 128]), conv=rng.choice([1001, 4096, 8192]))
    if kind == "turnover":
        return dict(kind=kind, rows=_spread(rng, 1, 500), lo=1, hi=_spread(rng, 20, 16000),
                    page=rng.choice([16, 24, 64, 272]))
    return dict(kind=kind, P=_spread(rng, 60, 30000), used=rng.choice([0.2, 0.5, 0.8]),
                rows=_spread(rng, 3, 300), layers=rng.randint(1, 2), page=rng.choice([8, 16, 24]),
                Hkv=rng.choice([2, 3, 8]), D=rng.choice([64, 128]))


def _lengths(n, lo, hi):
    return [lo + int((hi - lo) * (i + 0.5) / n) for i in range(n)]


def _pages(length, page):
    return -(-length // page)


class _Draw:
    """Seeded tensors on the GPU."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32):
        if dtype.itemsize > 1:
            return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=self.g)
        return self.normal(*shape, dtype=torch.bfloat16).to(dtype)

    def uniform(self, lo, hi, *shape):
        return torch.empty(shape, device="cuda").uniform_(lo, hi, generator=self.g)

    def perm(self, n):
        return torch.randperm(n, device="cuda", generator=self.g)

    def deal(self, values):
        v = torch.tensor(values, dtype=torch.int64, device="cuda")
        return v[self.perm(len(values))]


def _table(d, rows, lens, S, M, P, page):
    """Pages dealt at random to the given rows: block_table [S, M], ref_count [P], seq_lens [S]."""
    table = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
    count = (lens + page - 1) // page
    first = torch.cumsum(count, 0) - count
    j = torch.arange(M, device="cuda")
    held = j < count[:, None]
    at = torch.where(held, first[:, None] + j, 0)
    pages = d.perm(P)
    table[rows] = torch.where(held, pages[at], -1).to(torch.int32)
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    ref[pages[:int(count.sum())]] = 1
    seq = torch.zeros(S, dtype=torch.int32, device="cuda")
    seq[rows] = lens.to(torch.int32)
    return table, ref, seq


def prepare(case, seed):
    c, d = case, _Draw(seed)
    s = {"case": c}
    if c["kind"] in ("attend", "append"):
        B, page, Hkv, D = c["B"], c["page"], c["Hkv"], c["D"]
        live = B - c["pad"]
        cache = DTYPES[c["cache"]]
        new = d.deal(_lengths(live, c["lo"], c["hi"]))
        if c["kind"] == "append":       # what is there already: up to a page and a half
            lens = new + d.deal([i % (page + page // 2 + 1) for i in range(live)])
        else:
            lens = new
        S = B + 3
        M = _pages(int(lens.max()), page) + 1
        P = int(((lens + page - 1) // page).sum()) + 7
        rows = d.perm(S)[:live]
        table, ref, seq = _table(d, rows, lens, S, M, P, page)
        slots = torch.full((B,), -1, dtype=torch.int32, device="cuda")
        slots[d.perm(B)[:live].sort().values] = rows.to(torch.int32)
        shape = (P, page, Hkv, D) if c.get("layout") != "heads" else (P, Hkv, page, D)
        k, v = d.normal(*shape, dtype=cache), d.normal(*shape, dtype=cache)
        if c.get("layout") == "heads":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        s.update(table=table, seq=seq, slots=slots, k_cache=k, v_cache=v, k_scale=None,
                 v_scale=None)
        if c["cache"] == "e4m3":
            low, high = (0.5, 1.5) if c["kind"] == "attend" else (0.01, 0.03)
            s.update(k_scale=d.uniform(low, high, Hkv), v_scale=d.uniform(low, high, Hkv))
        if c["kind"] == "attend":
            s["q"] = d.normal(B, c["T"], c["Hq"], D, dtype=DTYPES[c["dtype"]])
        else:
            by_row = torch.zeros(S + 1, dtype=torch.int64, device="cuda")
            by_row[rows] = new
            n = by_row[slots.long()]             # padding (-1) reads the last entry, zero
            off = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
            off[1:] = torch.cumsum(n, 0)
            N = int(off[-1])
            # keys and values as a projection leaves them: side by side in one row
            kv = d.normal(N, 2 * Hkv, D, dtype=DTYPES[c["dtype"]])
            s.update(offsets=off, k=kv[:, :Hkv], v=kv[:, Hkv:])
        return s
    if c["kind"] == "branch":
        page, n, fan = c["page"], c["parents"], c["fan"]
        lens = d.deal(_lengths(n, c["lo"], c["hi"]))
        S = n * (fan + 1) + 5
        M = _pages(c["hi"] + c["grow"], page) + 1
        P = int(((lens + page - 1) // page).sum()) + n * fan * (2 + _pages(c["grow"], page)) + 9
        slots = d.perm(S)
        parents, children = slots[:n], slots[n:n * (fan + 1)]
        s["table"], s["ref"], s["seq"] = _table(d, parents, lens, S, M, P, page)
        s["parents"] = parents.repeat_interleave(fan).to(torch.int32)
        s["children"] = children.to(torch.int32)
        s["rows"] = s["children"]
        s["lens"] = (lens.repeat_interleave(fan) + c["grow"]).to(torch.int32)
        s["pools"] = [d.normal(P, page, c["Hkv"], c["D"], dtype=torch.bfloat16)
                      for _ in range(2 * c["layers"])]
        s["states"] = [d.normal(S, c["Hv"], c["Dv"], 128) for _ in range(c["states"])] + \
            [d.normal(S, c["conv"], 3, dtype=torch.bfloat16) for _ in range(c["states"])]
        return s
    if c["kind"] == "turnover":
        page, n = c["page"], c["rows"]
        out, new = (d.deal(_lengths(n, c["lo"], c["hi"])) for _ in range(2))
        S, M = 2 * n + 3, _pages(c["hi"], page) + 1
        P = int(((out + page - 1) // page).sum()) * 5 // 4 + 40
        rows = d.perm(S)
        s["table"], s["ref"], s["seq"] = _table(d, rows[:n], out, S, M, P, page)
        s["rows"] = rows[:2 * n].to(torch.int32)
        zero = torch.zeros(n, dtype=torch.int64, device="cuda")
        s["lens"] = torch.cat([zero, new]).to(torch.int32)
        s["back"] = torch.cat([out, zero]).to(torch.int32)
        return s
    page, n, P = c["page"], c["rows"], c["P"]
    U = int(P * c["used"])
    n = min(n, U)
    count = torch.full((n,), U // n, dtype=torch.int64, device="cuda")
    count[:U - (U // n) * n] += 1
    lens = count * page - d.deal([i % page for i in range(n)])
    S, M = n + 3, U // n + 2
    rows = d.perm(S)[:n]
    s["table"], s["ref"], s["seq"] = _table(d, rows, lens, S, M, P, page)
    s["table0"], s["ref0"] = s["table"].clone(), s["ref"].clone()
    s["pools"] = [d.normal(P, page, c["Hkv"], c["D"], dtype=torch.bfloat16)
                  for _ in range(2 * c["layers"])]
    return s


# ---------------------------------------------------------------- plain forms
def _attend(s):
    c = s["case"]
    B, T, Hq, Hkv, D, page = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"], c["page"]
    slots, q = s["slots"].long(), s["q"]
    table = s["table"][slots.clamp(min=0)].long()                      # [B, M]
    length = torch.where(slots >= 0, s["seq"][slots.clamp(min=0)], 0)[:, None]
    L = table.shape[1] * page
    def rows(cache, scale):                                            # [B, Hkv, L, D]
        x = cache[table.clamp(min=0)].float()
        x = x.reshape(B, L, Hkv, D).transpose(1, 2)
        return x if scale is None else x * scale[:, None, None]
    at = torch.arange(L, device=q.device)
    pos = length - T + torch.arange(T, device=q.device)                # [B, T]
    seen = (at <= pos[..., None]) & (at < length[..., None])           # [B, T, L]
    if c["window"] > 0:
        seen = seen & (at > pos[..., None] - c["window"])
    seen = seen[:, None, :, None, :]                                   # [B, 1, T, 1, L]
    qh = q.float().reshape(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4)
    x = qh.reshape(B, Hkv, -1, D) @ rows(s["k_cache"], s["k_scale"]).transpose(2, 3)
    x = x.reshape(B, Hkv, T, Hq // Hkv, L) / math.sqrt(D)
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    held = torch.where(seen.any(2)[:, :, 0, :, None], rows(s["v_cache"], s["v_scale"]), 0.0)
    y = p.reshape(B, Hkv, -1, L) @ held
    y = y.reshape(B, Hkv, T, Hq // Hkv, D) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)[..., 0]
    back = lambda z: z.transpose(1, 2).reshape(B, T, Hq, *z.shape[4:])  # noqa: E731
    return back(y).to(q.dtype), back(lse)


def _append(s):
    c = s["case"]
    page, N = c["page"], s["k"].shape[0]
    off = s["offsets"].long()
    i = torch.arange(N, device=off.device)
    b = torch.searchsorted(off, i, right=True) - 1
    slot = s["slots"].long()[b]
    pos = s["seq"].long()[slot] - (off[b + 1] - i)
    at = s["table"].long()[slot, pos // page]
    def write(cache, x, scale):
        x = x.float() if scale is None else \
            (x.float() / scale[:, None]).clamp(-448.0, 448.0)
        cache[at, pos % page] = x.to(cache.dtype)
        return cache
    return write(s["k_cache"], s["k"], s["k_scale"]), write(s["v_cache"], s["v"], s["v_scale"])


def _count(ref, pages, held, by):
    """ref += by at every held page."""
    at = torch.where(held, pages.long(), ref.shape[0])
    more = torch.cat([ref, ref.new_zeros(1)])
    more.scatter_add_(0, at.reshape(-1), torch.full_like(at, by, dtype=ref.dtype).reshape(-1))
    ref.copy_(more[:-1])


def _fork(table, ref, seq, parents, children, page, states):
    p, ch = parents.long(), children.long()
    j = torch.arange(table.shape[1], device=table.device)
    _count(ref, table[ch], j < ((seq[ch] + page - 1) // page)[:, None], -1)
    held = j < ((seq[p] + page - 1) // page)[:, None]
    _count(ref, table[p], held, 1)
    table[ch] = torch.where(held, table[p], -1)
    seq[ch] = seq[p]
    return [x.index_copy_(0, ch, x[p]) for x in states]


def _resize(table, ref, seq, rows, lens, page, pools):
    r = rows.long()
    j = torch.arange(table.shape[1], device=table.device)
    t, old = table[r], seq[r]
    had, want = (old + page - 1) // page, (lens + page - 1) // page
    gone = (j >= want[:, None]) & (j < had[:, None])
    _count(ref, t, gone, -1)
    t = torch.where(gone, -1, t)
    last = t.gather(1, (had - 1).clamp(min=0)[:, None].long())[:, 0].long()
    part = (lens > old) & (old % page != 0)
    copied = part & (ref[last.clamp(min=0)] > 1)
    need = (want - had).clamp(min=0) + copied
    upto = torch.cumsum(need, 0)
    free = torch.argsort((ref > 0).to(torch.uint8), stable=True)
    ok = (need == 0) | (upto <= (ref <= 0).sum())
    copied = copied & ok
    first = upto - need
    fresh = (j >= (had - copied.to(had.dtype))[:, None]) & (j < want[:, None]) & ok[:, None] & \
        (lens > old)[:, None]
    at = first[:, None] + j - (had - copied.to(had.dtype))[:, None]
    t = torch.where(fresh, free[torch.where(fresh, at, 0)].to(torch.int32), t)
    _count(ref, t, fresh, 1)
    _count(ref, last, copied, -1)
    table[r] = t
    seq[r] = torch.where(ok, lens, old)
    which = copied.nonzero()[:, 0]
    src, dst = last[which], free[first[which]]
    return [x.index_copy_(0, dst, x[src]) for x in pools]


def _compact(table, ref, seq, page, pools):
    used = ref > 0
    U = used.sum()
    i = torch.arange(ref.shape[0], device=ref.device)
    src, dst = (used & (i >= U)).nonzero()[:, 0], (~used & (i < U)).nonzero()[:, 0]
    to = torch.where(used, i, -1).to(torch.int32)
    to[src] = dst.to(torch.int32)
    held = torch.arange(table.shape[1], device=ref.device) < ((seq + page - 1) // page)[:, None]
    table.copy_(torch.where(held, to[table.long().clamp(min=0)], table))
    ref[dst] = ref[src]
    ref[src] = 0
    return to, [x.index_copy_(0, dst, x[src]) for x in pools]


def run(s):
    c = s["case"]
    if own:
        import gated_deltanet_state_gdn_b200 as gdn
    if c["kind"] == "attend":
        if own:
            return gdn.gdn_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["seq"],
                                      s["slots"], window=c["window"], k_scale=s["k_scale"],
                                      v_scale=s["v_scale"], return_lse=True)
        return _attend(s)
    if c["kind"] == "append":
        if own:
            return gdn.gdn_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"],
                                     s["seq"], s["slots"], s["offsets"], k_scale=s["k_scale"],
                                     v_scale=s["v_scale"])
        return _append(s)
    table, ref, seq, page = s["table"], s["ref"], s["seq"], c["page"]
    if c["kind"] == "branch":
        # a pass finds the children as the last one left them: their pages are given back first
        if own:
            gdn.gdn_page_fork(table, ref, seq, s["parents"], s["children"], page, s["states"])
            gdn.gdn_page_resize(table, ref, seq, s["rows"], s["lens"], page, s["pools"])
        else:
            _fork(table, ref, seq, s["parents"], s["children"], page, s["states"])
            _resize(table, ref, seq, s["rows"], s["lens"], page, s["pools"])
        return table, ref, seq, s["pools"], s["states"]
    if c["kind"] == "turnover":
        if own:
            gdn.gdn_page_resize(table, ref, seq, s["rows"], s["lens"], page)
            gdn.gdn_page_resize(table, ref, seq, s["rows"], s["back"], page)
        else:
            _resize(table, ref, seq, s["rows"], s["lens"], page, [])
            _resize(table, ref, seq, s["rows"], s["back"], page, [])
        return table, ref, seq
    # pages in order leave nothing to move: every pass starts from the fragmented tables again
    # (the moved pages' old places still hold their contents)
    table.copy_(s["table0"])
    ref.copy_(s["ref0"])
    if own:
        to = gdn.gdn_page_compact(table, ref, seq, page, s["pools"])
    else:
        to, _ = _compact(table, ref, seq, page, s["pools"])
    return table, ref, to, s["pools"]


def work(case):
    c = case
    if c["kind"] == "attend":
        live, T, D = c["B"] - c["pad"], c["T"], c["D"]
        lens = _lengths(live, c["lo"], c["hi"])
        most = c["window"] + T - 1 if c["window"] > 0 else 1 << 62
        keys = sum(min(n, most) for n in lens)
        q = live * T * c["Hq"] * D
        pairs = sum(max(0, min(n - T + 1 + t, c["window"] or n)) for n in lens for t in range(T))
        return {"bytes": keys * c["Hkv"] * D * 2 * SIZE[c["cache"]] + 2 * q * SIZE[c["dtype"]] +
                live * T * c["Hq"] * 4 + 4 * sum(_pages(min(n, most), c["page"]) for n in lens),
                "flops": 4 * D * c["Hq"] * pairs}
    if c["kind"] == "append":
        N = sum(_lengths(c["B"] - c["pad"], c["lo"], c["hi"]))
        return {"bytes": 2 * N * c["Hkv"] * c["D"] * (SIZE[c["dtype"]] + SIZE[c["cache"]]),
                "flops": 2 * N * c["Hkv"] * c["D"] if c["cache"] == "e4m3" else 0}
    if c["kind"] == "branch":
        lens = _lengths(c["parents"], c["lo"], c["hi"])
        n = c["parents"] * c["fan"]
        copied = c["fan"] * sum(1 for x in lens if x % c["page"])
        row = c["Hv"] * c["Dv"] * 128 * 4 + c["conv"] * 3 * 2
        pages = c["fan"] * sum(_pages(x, c["page"]) for x in lens)
        return {"bytes": 2 * n * c["states"] * row +
                2 * copied * 2 * c["layers"] * c["page"] * c["Hkv"] * c["D"] * 2 + 16 * pages,
                "flops": 0}
    if c["kind"] == "turnover":
        pages = sum(_pages(x, c["page"]) for x in _lengths(c["rows"], c["lo"], c["hi"]))
        # each page is given back and handed out, in each direction: its table entry and its
        # count are read and written
        return {"bytes": 2 * 2 * pages * 16 + 2 * 2 * c["rows"] * 16, "flops": 0}
    U = int(c["P"] * c["used"])
    moved = U * (c["P"] - U) // c["P"]
    return {"bytes": 2 * moved * 2 * c["layers"] * c["page"] * c["Hkv"] * c["D"] * 2 +
            4 * 4 * U + 2 * 4 * c["P"], "flops": 0}


# ---------------------------------------------------------------- 64 bits
def _to_e4m3(x):
    """The nearest number of 1 + 4 + 3 bits, ties to the even one, 448 at most, in 64 bits."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(a / step) * step


def exact(case, seed):
    c = case
    if c["kind"] not in ("attend", "append"):
        return None            # copies of values and whole numbers: nothing is computed
    s = prepare(case, seed)
    page = c["page"]
    if c["kind"] == "append":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        off, slots, seq = s["offsets"].tolist(), s["slots"].tolist(), s["seq"].tolist()
        for b in range(c["B"]):
            n = off[b + 1] - off[b]
            if n == 0:
                continue
            pos = torch.arange(seq[slots[b]] - n, seq[slots[b]], device="cuda")
            at = s["table"][slots[b]].long()[torch.div(pos, page, rounding_mode="floor")]
            for cache, x, scale in ((k, s["k"], s["k_scale"]), (v, s["v"], s["v_scale"])):
                x = x[off[b]:off[b + 1]].double()
                if scale is not None:
                    x = _to_e4m3(x / scale.double()[None, :, None])
                cache[at, torch.remainder(pos, page)] = x
        return k, v
    B, T, Hq, Hkv, D = c["B"], c["T"], c["Hq"], c["Hkv"], c["D"]
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    slots, seq = s["slots"].tolist(), s["seq"].tolist()
    for b in range(B):
        n = seq[slots[b]] if slots[b] >= 0 else 0
        if n == 0:
            continue
        pages = s["table"][slots[b], :_pages(n, page)].long()
        k, v = (x[pages].reshape(-1, Hkv, D)[:n].double() for x in (s["k_cache"], s["v_cache"]))
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"].double()[:, None], v * s["v_scale"].double()[:, None]
        for t in range(T):
            hi = n - T + t + 1                     # positions [lo, hi) are seen
            lo = max(0, hi - c["window"]) if c["window"] > 0 else 0
            if hi <= lo:
                continue
            q = s["q"][b, t].double().reshape(Hkv, Hq // Hkv, D)
            x = torch.einsum("hgd,lhd->hgl", q, k[lo:hi]) / D ** 0.5
            lse[b, t] = torch.logsumexp(x, -1).reshape(-1)
            out[b, t] = torch.einsum("hgl,lhd->hgd", torch.softmax(x, -1),
                                     v[lo:hi]).reshape(Hq, D)
    return out, lse
