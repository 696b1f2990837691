"""Steps of a hybrid model, one recurrent and one softmax layer: gdn_conv1d and gdn_decode beside
gdn_page_resize, gdn_kv_append and gdn_paged_attn, every layer naming a request by the same int32
slot; forks copy the decode pool and the conv windows along with the pages.

Conv windows are compared bit for bit and conv outputs within the bound of test_gpu_conv1d; decode
with the float64 oracle over the call's own inputs (bf16 activations: relative L2 <= 2e-2); attention
with a softmax in 64 bits over the tokens each request has: weights and outputs are rounded once to
bf16 (half a step of 2^-8) or, over e4m3, weights once to fp16; the rest is fp32."""
import math

import numpy as np
import pytest
import torch

from _util import TOL_BF16, assert_out_close, assert_states_close, f64

pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
SLOTS, PAGE, PAGES = 9, 16, 60
H, HV, DK, DV, K = 4, 4, 128, 64, 4             # of the recurrent layer
HKV, HQ, D = 2, 8, 128                          # of the softmax layer
CHANNELS = 2 * H * DK + HV * DV


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_state_gdn_b200 as g
    g.lib()
    return g


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Hybrid:
    def __init__(self, gdn, oracle, cache, heads_padded):
        self.gdn, self.oracle, self.cache = gdn, oracle, cache
        self.g = torch.Generator(device="cuda").manual_seed(4)
        new = self.new
        # the decode pool as part of a larger allocation: slots further apart than their states
        # are large, with `heads_padded` heads too
        self.base = new(SLOTS, HV + 1, DV + (DV if heads_padded else 0), DK)
        self.pool = self.base[:, :HV, :DV]
        self.windows = new(SLOTS, CHANNELS, K - 1).to(BF16)
        self.weight, self.A_log, self.dt_bias = new(CHANNELS, K).to(BF16), new(HV), new(HV)
        self.k, self.v = (torch.full((PAGES, PAGE, HKV, D), math.nan, device="cuda").to(cache) for _ in range(2))
        self.scale = {} if cache == BF16 else dict(k_scale=torch.tensor([0.03, 0.05], device="cuda"),
                                                   v_scale=torch.tensor([0.04, 0.02], device="cuda"))
        self.table = torch.full((SLOTS, 6), -1, dtype=torch.int32, device="cuda")
        self.ref, self.seq, self.status = ints([0] * PAGES), ints([0] * SLOTS), ints([0])
        self.states, self.win = f64(self.pool), f64(self.windows)       # the models
        self.have = {s: [] for s in range(SLOTS)}
        self.padding = self.base.clone()

    def new(self, *shape):
        return torch.randn(*shape, device="cuda", generator=self.g)

    def inputs(self, n):
        b = lambda *s: self.new(*s).to(BF16)  # noqa: E731
        return dict(x=b(n, CHANNELS), a=b(n, 1, HV), b=b(n, 1, 1, HV), q=b(n, 1, HQ, D), kn=b(n, 1, HKV, D),
                    vn=b(n, 1, HKV, D))

    def pools(self):
        """The slot-indexed arrays: of a pool with padded heads, its heads."""
        dense = self.pool.stride(1) == DV * DK
        return ([self.pool] if dense else list(self.pool.unbind(1))) + [self.windows]

    def stored(self, x, name):
        if self.cache == BF16:
            return x.double()
        s = self.scale[name][:, None]
        return ((x.float() / s).clamp(-448, 448).to(E4M3).float() * s).double()

    def step(self, live, i):
        """One token of each live slot through both layers; the outputs, checked."""
        gdn, n = self.gdn, len(live)
        slots, offsets = ints(live), ints(list(range(n + 1)))
        st = dict(dev_status=self.status)
        y, _ = gdn.gdn_conv1d(i["x"], self.weight, self.windows, slots, offsets, **st)
        q = y[:, :H * DK].reshape(n, 1, H, DK)
        k = y[:, H * DK:2 * H * DK].reshape(n, 1, 1, H, DK)
        v = y[:, 2 * H * DK:].reshape(n, 1, 1, HV, DV)
        o, _ = gdn.gdn_decode(q, k, v, self.pool, slots, self.A_log, i["a"], self.dt_bias, i["b"], **st)
        gdn.gdn_page_resize(self.table, self.ref, self.seq, slots, ints([len(self.have[s]) + 1 for s in live]),
                            PAGE, [self.k, self.v], **st)
        gdn.gdn_kv_append(i["kn"], i["vn"], self.k, self.v, self.table, self.seq, slots, **st, **self.scale)
        out, lse = gdn.gdn_paged_attn(i["q"], self.k, self.v, self.table, self.seq, slots, return_lse=True, **st,
                                      **self.scale)

        w64 = f64(self.weight)
        before = self.win
        ry, self.win = self.oracle.conv1d(f64(i["x"]), w64, before, np.array(live), offsets.cpu().numpy())
        size, _ = self.oracle.conv1d(np.abs(f64(i["x"])), np.abs(w64), np.abs(before), np.array(live),
                                     offsets.cpu().numpy())
        assert (np.abs(f64(y) - ry) <= 2.0 ** -8 * np.abs(ry) + 8 * K * 2.0 ** -24 * size + 1e-30).all()
        np.testing.assert_array_equal(f64(self.windows), self.win)
        ro, self.states = self.oracle.decode(f64(q), f64(k), f64(v), self.states, np.array(live, dtype=np.int32),
                                             f64(self.A_log), f64(i["a"]), f64(self.dt_bias), f64(i["b"]))
        assert_out_close(f64(o), ro, TOL_BF16)
        assert_states_close(f64(self.pool), self.states, TOL_BF16)
        for b, s in enumerate(live):
            self.have[s] = self.have[s] + [(self.stored(i["kn"][b, 0], "k_scale"),
                                            self.stored(i["vn"][b, 0], "v_scale"))]
            kk, vv = (torch.stack([t[j] for t in self.have[s]]) for j in (0, 1))
            x = torch.einsum("hgd,lhd->hgl", i["q"][b, 0].double().reshape(HKV, -1, D), kk) / math.sqrt(D)
            w = torch.softmax(x, -1)
            want = torch.einsum("hgl,lhd->hgd", w, vv).reshape(HQ, D)
            size = torch.einsum("hgl,lhd->hgd", w, vv.abs()).reshape(HQ, D)
            weight = 2.0 ** -8 if self.cache == BF16 else 2.0 ** -11
            lim = 2.0 ** -8 * 1.01 * want.abs() + (weight * 1.01 + 2.0 ** -14) * size
            assert ((out[b, 0].double() - want).abs() <= lim).all(), s
            assert ((lse[b, 0].double() - torch.logsumexp(x, -1).reshape(-1)).abs() < 2.0 ** -14).all(), s
        return o, out

    def fork(self, parents, children):
        self.gdn.gdn_page_fork(self.table, self.ref, self.seq, ints(parents), ints(children), PAGE, self.pools(),
                               dev_status=self.status)
        for p, c in zip(parents, children):
            self.states[c], self.win[c], self.have[c] = self.states[p], self.win[p], list(self.have[p])
            assert torch.equal(self.pool[c], self.pool[p]) and torch.equal(self.windows[c], self.windows[p])


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("heads_padded", [False, True])
def test_forked_requests_go_on_in_every_layer(gdn, oracle_mod, cache, heads_padded):
    m = Hybrid(gdn, oracle_mod, cache, heads_padded)
    live = [5, 0, 7]
    for _ in range(20):                             # past the first page
        m.step(live, m.inputs(3))
    m.fork([5, 5, 0], [2, 8, 4])
    live = [5, 0, 7, 2, 8, 4]
    i = m.inputs(6)                                 # children get what their parents get: the same results
    for t in i.values():
        t[3], t[4], t[5] = t[0], t[0], t[1]
    o, out = m.step(live, i)
    assert torch.equal(o[3], o[0]) and torch.equal(o[4], o[0]) and torch.equal(o[5], o[1])
    for child, parent in ((3, 0), (4, 0), (5, 1)):  # (cut elsewhere, the parts may join to another rounding)
        assert ((out[child] - out[parent]).abs().float() <= 2.0 ** -7 * out[parent].abs().float() + 2.0 ** -14).all()
    for _ in range(3):                              # then each goes its own way
        m.step(live, m.inputs(6))
    gdn.gdn_page_compact(m.table, m.ref, m.seq, PAGE, [m.k, m.v], dev_status=m.status)
    m.fork([7], [0])                                # a child that held pages and states
    for _ in range(2):
        m.step([0, 7, 4], m.inputs(3))
    # slots that nobody used and the space between the states are as they were
    assert torch.equal(m.base[[1, 3, 6]], m.padding[[1, 3, 6]])
    assert torch.equal(m.base[:, HV:], m.padding[:, HV:]) and torch.equal(m.base[:, :, DV:], m.padding[:, :, DV:])
    assert int(m.status.item()) == 0
    # [5], [2] and [8] share their first page; all hold the pages of their lengths
    held = {}
    for s in range(SLOTS):
        for p in m.table[s, :-(-len(m.have[s]) // PAGE)].tolist():
            held[p] = held.get(p, 0) + 1
    assert [held.get(p, 0) for p in range(PAGES)] == m.ref.tolist() and max(held.values()) == 3
