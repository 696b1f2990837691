"""Plain models of the paged cache in 64 bits, and its cases (not collected: no test_ prefix)."""
import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float8_e4m3fn: 2.0 ** -4}


def pages_of(n, page):
    return -(-n // page)


class Case:
    """A cache with rows of the given lengths on shuffled pages, and B requests over them."""

    def __init__(self, seed, lens, *, T=1, Hq=4, H=2, D=64, page=16, dtype=torch.bfloat16,
                 cache=None, layout="tokens", pad=(), extra_pages=3, fill=None, device="cuda",
                 scales=True, width=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.T, self.Hq, self.H, self.D, self.page = list(lens), T, Hq, H, D, page
        self.dtype, self.cache = dtype, cache or dtype
        R = len(lens)
        self.rows = R + 2
        self.width = width or max([pages_of(n, page) for n in lens] + [1]) + 1
        need = sum(pages_of(n, page) for n in lens)
        self.P = need + extra_pages
        order = torch.randperm(self.P, generator=g).tolist()
        perm = torch.randperm(self.rows, generator=g).tolist()
        table = torch.full((self.rows, self.width), -1, dtype=torch.int32)
        seq = torch.zeros(self.rows, dtype=torch.int32)
        ref = torch.zeros(self.P, dtype=torch.int32)
        at = 0
        slots = []
        for i, n in enumerate(lens):
            for j in range(pages_of(n, page)):
                table[perm[i], j] = order[at]
                ref[order[at]] = 1
                at += 1
            seq[perm[i]] = n
            slots.append(-1 if i in pad else perm[i])
        shape = (self.P, page, H, D) if layout == "tokens" else (self.P, H, page, D)

        def values(*shape, to=self.dtype):
            x = torch.randn(*shape, generator=g)
            return x.to(torch.bfloat16).to(to) if to == torch.float8_e4m3fn else x.to(to)

        self.k, self.v = values(*shape, to=self.cache), values(*shape, to=self.cache)
        if layout == "heads":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.q = values(R, T, Hq, D)
        self.k_scale = self.v_scale = None
        if self.cache == torch.float8_e4m3fn and scales:
            self.k_scale = torch.rand(H, generator=g) + 0.5
            self.v_scale = torch.rand(H, generator=g) + 0.5
        self.table, self.seq, self.ref = table, seq, ref
        self.slots = torch.tensor(slots, dtype=torch.int32)
        self.device = device

    def to(self, t):
        if t is None:
            return None
        # (a transposed cache keeps its layout)
        return t.to(self.device) if t.is_contiguous() else t.transpose(1, 2).to(self.device).transpose(1, 2)

    def attend(self, gdn, **kw):
        kw.setdefault("return_lse", True)
        return gdn.gdn_paged_attn(self.to(self.q), self.to(self.k), self.to(self.v),
                                  self.to(self.table), self.to(self.seq), self.to(self.slots),
                                  k_scale=self.to(self.k_scale), v_scale=self.to(self.v_scale), **kw)


def wide(t):
    return t.detach().to("cpu", torch.float32).double().numpy()


def attend(c, *, scale=None, window=0, num_pages=None):
    """out, lse, and what their errors are measured against: per row, sum_j w_j |v_j| and the
    largest error of a score that float32 products and sums may make."""
    B, T, Hq, H, D, page = len(c.slots), c.T, c.Hq, c.H, c.D, c.page
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    k, v, q = wide(c.k), wide(c.v), wide(c.q)
    if c.k_scale is not None:
        k = k * wide(c.k_scale)[:, None]
        v = v * wide(c.v_scale)[:, None]
    table, seq, slots = c.table.numpy(), c.seq.numpy(), c.slots.numpy()
    out = np.zeros((B, T, Hq, D))
    lse = np.full((B, T, Hq), -np.inf)
    size = np.zeros((B, T, Hq, D))
    dx = np.zeros((B, T, Hq))
    count = np.zeros((B, T, Hq))
    for b in range(B):
        if slots[b] < 0 or slots[b] >= c.rows:
            continue
        n = int(min(max(seq[slots[b]], 0), c.width * page))
        for t in range(T):
            pos = n - T + t
            js = [j for j in range(max(0, pos - window + 1) if window else 0, pos + 1)
                  if 0 <= table[slots[b], j // page] < c.P]
            if not js:
                continue
            at = [(table[slots[b], j // page], j % page) for j in js]
            pg, of = np.array(at).T
            for h in range(Hq):
                kk, vv = k[pg, of, h // (Hq // H)], v[pg, of, h // (Hq // H)]
                x = scale * (kk @ q[b, t, h])
                m = x.max()
                if m == -np.inf:
                    continue
                w = np.exp(x - m)
                lse[b, t, h] = m + np.log(w.sum())
                w = w / w.sum()
                out[b, t, h] = w @ vv
                size[b, t, h] = w @ np.abs(vv)
                # a sum of D products in float32, each step rounded or cut (2^-23), then scaled
                dx[b, t, h] = ((D + 4) * 2.0 ** -23 * abs(scale) * (np.abs(kk) @ np.abs(q[b, t, h])).max()
                               + 2.0 ** -22 * np.abs(x).max())
                count[b, t, h] = len(js)
    return out, lse, size, dx, count


def check_attend(c, got, want, *, dtype=None):
    """Every element within the bound of its own arithmetic.

    The weights are exp of scores that are off by dx, by an exp2 good to 2^-21, rounded to the
    16-bit type of the product (half a step); numerator and denominator are sums of `count`
    terms in float32.  The output is rounded once."""
    out, lse = wide(got[0]), wide(got[1])
    ro, rl, size, dx, count = want
    p_step = HALF_STEP[torch.float16 if c.cache == torch.float8_e4m3fn else c.cache]
    f32 = 2 * (dx + 2.0 ** -21 + (count + 8) * 2.0 ** -23)
    lim = HALF_STEP[c.dtype] * np.abs(ro) * 1.01 + (p_step * 1.01 + f32)[..., None] * size + 1e-7
    err = np.abs(out - ro)
    assert np.isfinite(out).all()
    worst = np.unravel_index((err - lim).argmax(), err.shape)
    assert (err <= lim).all(), f"out {worst}: off {err[worst]:.3e}, limit {lim[worst]:.3e}"
    assert (np.isneginf(lse) == np.isneginf(rl)).all()
    fine = np.isfinite(rl)
    assert np.isfinite(lse[fine]).all()
    el = np.abs(lse[fine] - rl[fine])
    assert (el <= f32[fine] + 2.0 ** -22 * np.abs(rl[fine]) + 1e-7).all()
    assert (out[~fine] == 0).all()


class Tables:
    """The page table as plain lists, and what the calls say they do to it, one row at a time."""

    def __init__(self, table, ref, seq, page):
        self.t, self.ref, self.seq = table.tolist(), ref.tolist(), seq.tolist()
        self.page, self.P, self.width = page, len(self.ref), len(self.t[0])
        self.status = 0

    def ok_page(self, p):
        if 0 <= p < self.P:
            return True
        self.status |= 16
        return False

    def resize(self, rows, lens, pools=()):
        cap, page = self.width * self.page, self.page
        todo = []
        for r, n in zip(rows, lens):
            if r < 0:
                continue
            if r >= len(self.t):
                self.status |= 1
            elif list(rows).count(r) > 1:
                self.status |= 64
            elif not (0 <= n <= cap and 0 <= self.seq[r] <= cap):
                self.status |= 32
            else:
                todo.append((r, n))
        for r, n in todo:
            for j in range(pages_of(n, page), pages_of(self.seq[r], page)):
                if self.ok_page(self.t[r][j]):
                    self.ref[self.t[r][j]] -= 1
                self.t[r][j] = -1
        free = [p for p in range(self.P) if self.ref[p] <= 0]
        seen = list(self.ref)
        given, copies = [], []
        short = False
        for r, n in todo:
            old = self.seq[r]
            had, want = pages_of(old, page), pages_of(n, page)
            copied = False
            if n > old and old % page:
                last = self.t[r][had - 1]
                if not self.ok_page(last):
                    continue
                copied = seen[last] > 1
            need = max(want - had, 0) + copied
            if need and (short or need > len(free)):
                short = True
                self.status |= 128
                continue
            mine, free = free[:need], free[need:]
            if copied:
                copies.append((self.t[r][had - 1], mine[0]))
                self.ref[self.t[r][had - 1]] -= 1
                self.t[r][had - 1] = mine[0]
                self.ref[mine[0]] = 1
                mine = mine[1:]
            for j, p in zip(range(had, want), mine):
                self.t[r][j] = p
                self.ref[p] = 1
            self.seq[r] = n
        for x in pools:
            for s, d in copies:
                x[d] = x[s]

    def fork(self, parents, children, pools=()):
        cap, page = self.width * self.page, self.page
        pairs = [(p, c) for p, c in zip(parents, children) if p >= 0 and c >= 0]
        good = []
        for i, (p, c) in enumerate(pairs):
            if p >= len(self.t) or c >= len(self.t):
                self.status |= 1
                continue
            others = pairs[:i] + pairs[i + 1:]
            if p == c or any(c in o or o[1] == p for o in others):
                self.status |= 64
            elif not 0 <= self.seq[p] <= cap:
                self.status |= 32
            else:
                good.append((p, c))
        for p, c in good:
            if 0 <= self.seq[c] <= cap:
                for j in range(pages_of(self.seq[c], page)):
                    if self.ok_page(self.t[c][j]):
                        self.ref[self.t[c][j]] -= 1
                    self.t[c][j] = -1
            else:
                self.status |= 32
            for j in range(pages_of(self.seq[p], page)):
                if self.ok_page(self.t[p][j]):
                    self.ref[self.t[p][j]] += 1
                self.t[c][j] = self.t[p][j]
            self.seq[c] = self.seq[p]
            for x in pools:
                x[c] = x[p]

    def compact(self, pools=()):
        used = [p for p in range(self.P) if self.ref[p] > 0]
        U = len(used)
        src = [p for p in used if p >= U]
        dst = [p for p in range(U) if self.ref[p] <= 0]
        to = [p if self.ref[p] > 0 else -1 for p in range(self.P)]
        for s, d in zip(src, dst):
            to[s] = d
            self.ref[d], self.ref[s] = self.ref[s], 0
            for x in pools:
                x[d] = x[s]
        for r, row in enumerate(self.t):
            if not 0 <= self.seq[r] <= self.width * self.page:
                self.status |= 32
                continue
            for j in range(pages_of(self.seq[r], self.page)):
                if 0 <= row[j] < self.P and to[row[j]] >= 0:
                    row[j] = to[row[j]]
                else:
                    self.status |= 16
        return to

    def same(self, table, ref, seq):
        assert seq.tolist() == self.seq
        assert ref.tolist() == self.ref
        assert table.tolist() == self.t
