"""GPU parity of gdn_paged_attn and gdn_kv_append with plain models in 64 bits (the bounds of
the comparisons are derived in _paged.check_attend)."""
import math

import numpy as np
import pytest
import torch

from _paged import HALF_STEP, Case, attend, check_attend, pages_of, wide

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_state_gdn_b200 as g
    g.lib()
    return g


def run(gdn, c, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    plain = {k: v for k, v in kw.items() if k in ("scale", "window")}
    got = c.attend(gdn, dev_status=st, **kw)
    torch.cuda.synchronize()
    check_attend(c, got, attend(c, **plain))
    return got, int(st.item())


LENS = [1, 0, 15, 16, 17, 63, 64, 65, 130, 200]


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, F16), (BF16, E4M3), (F16, E4M3)])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 128, 192, 256])
def test_head_dims_and_types(gdn, dtype, cache, D):
    c = Case(D, LENS, D=D, dtype=dtype, cache=cache)
    assert run(gdn, c)[1] == 0


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,H,T", [(1, 1, 1), (16, 1, 1), (15, 3, 2), (8, 1, 3), (8, 2, 16),
                                    (16, 1, 3), (16, 1, 9), (6, 6, 5)])
def test_groups_and_tokens(gdn, cache, D, Hq, H, T):
    # rows a head from 1 to 144: one to four warps over rows, one unit a head and several, and
    # requests with fewer positions than tokens
    c = Case(Hq + T, [1, 2, 0, 40, 129], T=T, Hq=Hq, H=H, D=D, cache=cache)
    assert run(gdn, c)[1] == 0


@pytest.mark.parametrize("page", [1, 3, 16, 24, 100, 272])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_pages_and_layouts(gdn, page, layout, cache):
    c = Case(page, [1, page, page + 1, 3 * page - 1, 290], page=page, layout=layout, cache=cache, T=2)
    assert run(gdn, c)[1] == 0


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("window", [1, 2, 5, 64, 100, 1000])
@pytest.mark.parametrize("cache", [F16, E4M3])
def test_windows(gdn, T, window, cache):
    c = Case(window, [1, 3, 64, 100, 101, 333], T=T, dtype=F16, cache=cache)
    assert run(gdn, c, window=window)[1] == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[20000], [1, 9000, 3], [70] * 700, [0] * 5 + [5000] + [1] * 300],
                         ids=["one", "three", "many", "skewed"])
def test_split_and_join(gdn, D, lens):
    # one request over all blocks; units over two; hundreds of whole ones, more rows of the batch
    # than a block keeps at hand, empty ones among them
    c = Case(len(lens), lens, D=D, Hq=2, H=1, page=32)
    assert run(gdn, c)[1] == 0


def test_scales_of_all_signs(gdn):
    for scale in (0.0, -0.3, 5.0):
        c = Case(3, LENS, T=2)
        run(gdn, c, scale=scale)


def test_padding_and_given_outputs(gdn):
    c = Case(4, [5, 40, 0, 7], pad=(1, 3), T=2)
    (o, l), _ = run(gdn, c)
    assert (o[[1, 3]] == 0).all() and (l[[1, 3]] == -math.inf).all()
    out = torch.full((4, 2, 4, 64), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((4, 2, 4), 9.0, device="cuda")
    o2, l2 = c.attend(gdn, out=out, lse=lse)
    assert o2 is out and l2 is lse
    live = [0, 2]
    assert torch.equal(o2[live], o[live]) and torch.equal(l2[live], l[live])
    assert (o2[[1, 3]] == 7).all() and (l2[[1, 3]] == 9).all()
    out.fill_(7.0)
    assert torch.equal(c.attend(gdn, out=out, return_lse=False), o2)
    o3, l3 = c.attend(gdn, lse=lse.fill_(9.0))
    assert torch.equal(o3, o) and (l3[[1, 3]] == 9).all() and torch.equal(l3[live], l[live])
    o4, l4 = c.attend(gdn, out=out)
    assert torch.equal(o4, o2) and torch.equal(l4, l)


def test_without_slots(gdn):
    c = Case(5, [5, 40, 17])
    order = [int(s) for s in c.slots]
    want = c.attend(gdn)
    c.table, c.seq = c.table[order], c.seq[order]
    table, seq = c.to(c.table), c.to(c.seq)
    got = gdn.gdn_paged_attn(c.to(c.q), c.to(c.k), c.to(c.v), table, seq, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_bad_rows_lengths_and_pages(gdn):
    c = Case(6, [40, 40, 40, 40, 40])
    s = [int(x) for x in c.slots]
    c.table[s[0], 1] = -1           # positions 16..31 are on no page
    c.table[s[1], 0] = c.P          # nor 0..15
    c.seq[s[2]] = c.width * c.page + 5
    c.table[s[2], 3] = -7
    c.seq[s[3]] = -2
    c.slots[4] = c.rows
    _, st = run(gdn, c)
    assert st == gdn.GDN_DEV_BAD_PAGE | gdn.GDN_DEV_BAD_LENGTH | gdn.GDN_DEV_BAD_SLOT


@pytest.mark.parametrize("cache", [BF16, F16, E4M3])
@pytest.mark.parametrize("window", [0, 3])
def test_unseen_positions_never_reach_the_output(gdn, cache, window):
    # infinities and NaN past the length, on other pages, ahead of the window, and in the later
    # tokens, which the earlier tokens of the same request do not see
    dtype = F16 if cache == F16 else BF16
    c = Case(7, [37, 16, 3], T=4, D=128, dtype=dtype, cache=cache)
    clean = attend(c, window=window)
    fine = c.attend(gdn, window=window)
    used = torch.zeros(c.P, c.page, dtype=torch.bool)
    for i, n in enumerate(c.lens):
        row = c.table[int(c.slots[i])]
        for j in range(n):
            used[int(row[j // c.page]), j % c.page] = True
    for x in (c.k, c.v):
        f = x.float()
        f[~used] = math.nan
        if window:                  # token 0 of the first request sees from 37 - 4 - window + 1 on
            row = c.table[int(c.slots[0])]
            for j in range(37 - 4 - window + 1):
                f[int(row[j // c.page]), j % c.page] = math.nan
        row = c.table[int(c.slots[0])]
        f[int(row[36 // c.page]), 36 % c.page] = math.nan if cache == E4M3 else math.inf
        f[int(row[35 // c.page]), 35 % c.page, :, 5::7] = math.nan
        x.copy_(f.to(cache))
    got = c.attend(gdn, window=window)
    for a, b in zip(got, fine):
        assert torch.equal(a[1:], b[1:]) and torch.equal(a[0, :2], b[0, :2])
        assert not torch.isfinite(a[0, 3]).all(-1).any() or a.dim() == 3
    check_attend(c, [g[1:] for g in got], [w[1:] for w in clean])
    # tokens that do see them: NaN everywhere a NaN is weighed
    assert torch.isnan(got[0][0, 2, :, 5::7]).all() and torch.isnan(got[0][0, 3]).all()


def test_infinite_scores(gdn):
    c = Case(8, [20, 20])
    row = c.table[int(c.slots[0])]
    c.k[int(row[0]), 3] = 0
    c.k[int(row[0]), 3, :, 0] = math.inf          # one key of score +-inf (by q's sign)
    c.q[0, :, :, 0] = -1.0
    (o, l) = c.attend(gdn)
    want = attend(c)
    check_attend(c, (o, l), want)                 # weight zero
    c.q[0, :, :, 0] = 1.0
    o, l = c.attend(gdn)
    assert torch.isnan(o[0]).all() and torch.isfinite(o[1]).all()
    c.k[...] = 0
    c.k[..., 0] = -math.inf                       # every score -inf: nothing is weighed
    o, l = c.attend(gdn)
    assert (o[0] == 0).all() and (l[0] == -math.inf).all()


def test_large_and_tiny_queries_over_8_bits(gdn):
    # rows of q are scaled by powers of two on their way to fp16: any magnitude of bf16 stands
    for power in (-100, -20, 0, 20, 60):
        c = Case(9, [40, 7], T=2, D=64, cache=E4M3)
        c.q = (c.q.float() * 2.0 ** power).to(BF16)
        run(gdn, c, scale=2.0 ** -power / 8)


def test_packed_and_strided_queries(gdn):
    c = Case(10, [40, 7, 100], T=3)
    want = c.attend(gdn)
    packed = torch.randn(3, 3, 10, 64, device="cuda", dtype=BF16)
    packed[:, :, 2:6] = c.to(c.q)
    c.q = packed[:, :, 2:6]
    c.to = lambda t: t.cuda() if t is not None and not t.is_cuda else t
    got = c.attend(gdn)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    c.q = packed.transpose(1, 2).contiguous().transpose(1, 2)[:, :, 2:6]    # heads outside tokens
    assert all(torch.equal(a, b) for a, b in zip(c.attend(gdn), want))


def test_one_result_every_time(gdn):
    c = Case(11, [3000, 1, 700], T=2, D=128)
    a = c.attend(gdn)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, c.attend(gdn)))


def test_offsets_past_32_bits(gdn):
    """A cache of more than 2^32 bytes: pages at its far end."""
    P, page, H, D = 70000, 64, 8, 64
    k = torch.zeros(P, page, H, D, dtype=BF16, device="cuda")
    v = torch.zeros(P, page, H, D, dtype=BF16, device="cuda")
    assert k.numel() * 2 > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(1)
    last = torch.randn(3, page, H, D, generator=g, device="cuda").to(BF16)
    k[-3:], v[-3:] = last, -last
    table = torch.tensor([[P - 1, P - 3, P - 2]], dtype=torch.int32, device="cuda")
    seq = torch.tensor([150], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, 8, D, generator=g, device="cuda").to(BF16)
    o = gdn.gdn_paged_attn(q, k, v, table, seq)
    small = gdn.gdn_paged_attn(q, last, -last, torch.tensor([[2, 0, 1]], dtype=torch.int32, device="cuda"), seq)
    assert torch.equal(o, small) and o.abs().max() > 0
    new = torch.randn(1, H, D, generator=g, device="cuda").to(BF16)
    gdn.gdn_kv_append(new, new, k, v, table, seq, torch.tensor([0], dtype=torch.int32, device="cuda"))
    assert torch.equal(k[P - 2, 149 - 128], new[0])
    assert int((k[:-3] != 0).sum()) == 0


# ---------------------------------------------------------------- append
def e4m3(x):
    """The nearest number of the type, ties to even, 448 at most (numpy, 64 bits)."""
    a = np.minimum(np.abs(x), 448.0)
    step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.sign(x) * np.round(a / step) * step


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (F16, F16), (BF16, E4M3), (F16, E4M3)])
@pytest.mark.parametrize("H,D,page,layout", [(2, 64, 16, "tokens"), (3, 80, 7, "heads"),
                                             (1, 256, 1, "tokens"), (8, 128, 64, "heads")])
def test_append_ragged(gdn, dtype, cache, H, D, page, layout):
    counts = [1, 0, 5, 33, 2, 40]
    had = [0, 4, 3, 16, 70, 9]
    c = Case(D + page, [a + b for a, b in zip(counts, had)], H=H, Hq=H, D=D, page=page, dtype=dtype,
             cache=cache, layout=layout, pad=(4,))
    g = torch.Generator().manual_seed(page)
    N = sum(counts) + 5
    kv = torch.randn(N, 2 * H, D, generator=g).to(dtype)
    off = torch.tensor(np.concatenate([[2], 2 + np.cumsum(counts)]), dtype=torch.int32)
    packed = kv.cuda()
    kc, vc = c.to(c.k).clone(memory_format=torch.preserve_format), c.to(c.v).clone(memory_format=torch.preserve_format)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = gdn.gdn_kv_append(packed[:, :H], packed[:, H:], kc, vc, c.to(c.table), c.to(c.seq), c.to(c.slots),
                          off.cuda(), k_scale=c.to(c.k_scale), v_scale=c.to(c.v_scale), dev_status=st)
    assert r[0] is kc and r[1] is vc and int(st.item()) == 0
    for got, start, x, scale in ((kc, c.k, kv[:, :H], c.k_scale), (vc, c.v, kv[:, H:], c.v_scale)):
        want = wide(start).copy()
        for b, n in enumerate(counts):
            if b == 4:
                continue
            row = c.table[int(c.slots[b])].tolist()
            for i in range(n):
                pos = had[b] + i
                y = wide(x[int(off[b]) + i])
                if cache == E4M3:
                    # the quotient in float32, as the call says
                    y = e4m3((y.astype(np.float32) / scale.numpy()[:, None]).astype(np.float64))
                want[row[pos // page], pos % page] = y
        np.testing.assert_array_equal(wide(got), want)


def test_append_uniform_and_without_slots(gdn):
    c = Case(21, [5, 9, 17], H=2, Hq=2)
    c.table, c.seq = c.table[[int(s) for s in c.slots]], c.seq[[int(s) for s in c.slots]]
    new = torch.randn(3, 4, 2, 64, device="cuda").to(BF16)
    k, v = c.to(c.k), c.to(c.v)
    gdn.gdn_kv_append(new, -new, k, v, c.to(c.table), c.to(c.seq))
    for b, n in enumerate([5, 9, 17]):
        for t in range(4):
            j = n - 4 + t
            p = int(c.table[b, j // 16])
            assert torch.equal(k[p, j % 16], new[b, t]) and torch.equal(v[p, j % 16], -new[b, t])


def test_append_saturates_and_keeps_nan(gdn):
    x = torch.tensor([500.0, -1e4, math.inf, -math.inf, math.nan, 448.0, 464.0, 0.001] * 2, dtype=BF16)
    new = x.reshape(1, 1, 16).cuda()
    k, v = (torch.zeros(1, 4, 1, 16, dtype=E4M3, device="cuda") for _ in range(2))
    gdn.gdn_kv_append(new, new, k, v, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                      torch.ones(1, dtype=torch.int32, device="cuda"))
    got = k.float().cpu()[0, 0, 0, :8].tolist()
    assert got[:4] == [448, -448, 448, -448] and math.isnan(got[4]) and got[5:7] == [448, 448]
    assert got[7] == 2.0 ** -9 * round(float(x[7]) * 2 ** 9)      # a subnormal: steps of 2^-9


def test_append_skips_and_tells(gdn):
    c = Case(22, [20, 20, 20, 20], H=2, Hq=2)
    s = [int(x) for x in c.slots]
    c.table[s[0], 1] = c.P + 3
    c.seq[s[1]] = 1                   # three new tokens at positions -2, -1, 0
    c.slots[2] = c.rows + 1
    c.seq[s[3]] = c.width * c.page + 2
    new = torch.randn(4, 3, 2, 64, device="cuda").to(BF16)
    k, v = c.to(c.k), c.to(c.v)
    k0 = k.clone()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_append(new, new, k, v, c.to(c.table), c.to(c.seq), c.to(c.slots), dev_status=st)
    assert int(st.item()) == gdn.GDN_DEV_BAD_PAGE | gdn.GDN_DEV_BAD_SLOT | gdn.GDN_DEV_BAD_LENGTH
    k0[int(c.table[s[1], 0]), 0] = new[1, 2]
    last = c.width * c.page - 1       # position of the only new token of row 3 inside its width
    if 0 <= int(c.table[s[3], last // 16]) < c.P:
        k0[int(c.table[s[3], last // 16]), last % 16] = new[3, 0]
    assert torch.equal(k, k0)


# ---------------------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3), (BF16, BF16)])
@pytest.mark.parametrize("nats", [12, 18, 26])
def test_a_dominant_token_of_no_value(gdn, dtype, cache, nats):
    """The first token outweighs each other one by e^nats and its value is zero: the output is the
    others' weighted mean.  In fp16 products a weight of w times the largest is off by half a step
    of fp16 (2^-11 of it), or by 2^-40 of the largest where w is below 2^-29."""
    B, n, D = 300, 1024, 64                 # a unit a block: the tokens share a running maximum
    c = Case(nats, [n] * B, Hq=1, H=1, D=D, dtype=dtype, cache=cache, page=64)
    c.k = (c.k.float() / 16).to(cache)      # scores of the others: below 1
    c.v = (c.v.float().abs() * 16 + 100).to(cache)
    if c.v_scale is not None:
        c.v_scale = c.v_scale * 2.0 ** (nats - 4)
    elif dtype == BF16:
        c.v = (c.v.float() * 2.0 ** nats).to(cache)
    for b in range(B):
        q, p = c.q[b, 0, 0].double(), int(c.table[int(c.slots[b]), 0])
        scale = 1.0 if c.k_scale is None else float(c.k_scale[0])
        c.k[p, 0, 0] = (q * (nats * math.sqrt(D) / float(q @ q) / scale)).to(cache)
        c.v[p, 0, 0] = 0
    want = attend(c)
    got = c.attend(gdn)
    if cache != BF16:
        # the largest weight is one of `total`; what lies below 2^-29 of it adds 2^-40 of it each
        v = wide(c.v).max() * (1.0 if c.v_scale is None else float(c.v_scale[0]))
        low = n * 2.0 ** -40 * v / HALF_STEP[F16] / 1.01
        want = (want[0], want[1], want[2] + low, *want[3:])
    assert (want[0] > 0).all()
    check_attend(c, got, want)


@pytest.mark.parametrize("dtype,cache", [(F16, F16), (BF16, E4M3), (BF16, BF16)])
def test_scores_of_any_size(gdn, dtype, cache):
    """A token alone has weight one whatever its score: up to where scores in fp32 come in steps of
    2^9 (a weight and the output are rounded once each)."""
    c = Case(34, [1] * 40, Hq=2, H=2, dtype=dtype, cache=cache, scales=False)
    rows = [int(c.table[int(s), 0]) for s in c.slots]
    v = torch.stack([c.v[p, 0] for p in rows]).double()[:, None]
    for power in range(0, 34):
        out, lse = c.attend(gdn, scale=2.0 ** power)
        x = torch.einsum("bthd,bhd->bth", c.q.double(), torch.stack([c.k[p, 0] for p in rows]).double())
        half = HALF_STEP[BF16 if cache == BF16 else F16] + HALF_STEP[dtype]
        assert ((out.cpu().double() - v).abs() <= 1.01 * half * v.abs() + 2.0 ** -25).all(), power
        bound = 2.0 ** power * 68 * 2.0 ** -23 * 64 * 16     # |q| |k| below 4 each
        assert ((lse.cpu().double() - x * 2.0 ** power).abs() <= bound + 1e-6).all(), power


@pytest.mark.parametrize("size", [1e-35, 1e-20, 1e20, 1e31])
@pytest.mark.parametrize("lens", [[300] * 4, [20000]], ids=["whole", "joined"])
def test_value_scales_of_any_size(gdn, size, lens):
    """A power of two more in the scale is one more in the output.  (Its digits are the same where it
    is a normal number.  Below 2^-126 bf16 has steps of 2^-133: o1 is off by 2^-9 of itself, here
    less than 2^-135, and the output by half a step.  The sums may be taken out another power of two:
    log2 of them, below 32, is off by an ulp, 2^-19, and its sum with the maximum by half of one.)"""
    c = Case(36, lens, T=2, cache=E4M3)
    (o1, l1), _ = run(gdn, c)
    power = 2.0 ** round(math.log2(size))
    c.v_scale = c.v_scale * power
    o2, l2 = c.attend(gdn)
    assert (l1 - l2).abs().max() <= 2.0 ** -17 and o2.abs().max() > 0
    want, got = o1.double() * power, o2.double()
    normal = want.abs() >= 2.0 ** -126
    assert torch.equal(got[normal], want[normal]) and ((got - want).abs()[~normal] <= 2.0 ** -133).all()


@pytest.mark.parametrize("lens", [[300] * 4, [20000]], ids=["whole", "joined"])
def test_large_values_do_not_pass_the_range_on_the_way(gdn, lens):
    """Values of one sign near the end of the range: their weighted sum, before it is divided by the
    sum of the weights, would be past it."""
    c = Case(37, lens, T=2, cache=E4M3)
    c.v = (c.v.float().abs() + 1).to(E4M3)
    (o1, l1), _ = run(gdn, c)
    c.v_scale = c.v_scale * 2.0 ** 115
    o2, l2 = c.attend(gdn)
    assert (l1 - l2).abs().max() <= 2.0 ** -17 and torch.equal(o2.double(), o1.double() * 2.0 ** 115)


def test_given_lse_alone_keeps_its_padding_rows(gdn):
    c = Case(31, [5, 40, 0, 7], pad=(1, 3), T=2)
    want, wl = c.attend(gdn)
    lse = torch.full((4, 2, 4), 9.0, device="cuda")
    out, got = c.attend(gdn, lse=lse, return_lse=False)
    live = [0, 2]
    assert got is lse and torch.equal(out, want) and torch.equal(lse[live], wl[live])
    assert (lse[[1, 3]] == 9).all()


def bytes_of(x, scale):
    """The e4m3 bytes of x / scale (the quotient in float32), the sign of a zero among them."""
    with np.errstate(divide="ignore", over="ignore", under="ignore"):
        y = np.float32(x) / np.float32(scale)
    a = np.abs(e4m3(y.astype(np.float64)))
    ex = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    code = np.where(a < 2.0 ** -6, a * 2 ** 9, (ex + 7) * 8 + (a / 2.0 ** ex - 1) * 8)
    return (code.astype(np.int64) + 128 * np.signbit(y)).astype(np.uint8)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("scale", [None, 1.0, 0.7, -0.7, 3e-3, -250.0, 1e-38, -1e-38, 1e37])
def test_append_rounds_to_the_same_bytes(gdn, dtype, scale):
    """Every byte, zeros of both signs and numbers that become zero among them."""
    g = torch.Generator().manual_seed(3)
    n, H, D, page = 40, 2, 64, 16
    x = torch.randn(n, H, D, generator=g) * 2.0 ** torch.randint(-16, 9, (n, H, D), generator=g)
    x = (x * abs(scale or 1.0)).to(dtype)
    x[0, :, :8] = torch.tensor([-0.0, 0.0, -1e-7, 1e-7, -2.0 ** -24, 2.0 ** -24, -3.0, 3.0]).to(dtype)
    k, v = (torch.zeros(3, page, H, D, dtype=E4M3, device="cuda") for _ in range(2))
    table = torch.tensor([[1, 0, 2]], dtype=torch.int32, device="cuda")
    sc = None if scale is None else torch.full((H,), scale, device="cuda")
    gdn.gdn_kv_append(x.cuda(), (-x).cuda(), k, v, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                      torch.tensor([0], dtype=torch.int32, device="cuda"), k_scale=sc, v_scale=sc)
    for got, y in ((k, x), (v, -x)):
        got = got.view(torch.uint8)[[1, 0, 2]].reshape(-1, H, D)[:n].cpu().numpy()
        np.testing.assert_array_equal(got, bytes_of(wide(y), scale or 1.0))


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float64])
def test_other_default_types(gdn, default):
    """What a call makes is of the types that it says, whatever torch's default type is."""
    c = Case(35, [5, 40, 0, 7], pad=(1,), T=2)
    want, wl = c.attend(gdn)
    out, lse = torch.empty_like(want), torch.empty_like(wl)
    torch.set_default_dtype(default)
    try:
        got = [c.attend(gdn), c.attend(gdn, out=out.zero_()), c.attend(gdn, lse=lse.fill_(-math.inf))]
    finally:
        torch.set_default_dtype(torch.float32)
    for o, x in got:
        assert o.dtype == BF16 and x.dtype == torch.float32
        assert torch.equal(o, want) and torch.equal(x, wl)


def test_windows_past_32_bits(gdn):
    c = Case(32, [70, 40, 300], T=2)
    want = c.attend(gdn)
    for window in (1 << 30, (1 << 31) - 1, 1 << 31, (1 << 32) + 5, 1 << 70):
        assert all(torch.equal(a, b) for a, b in zip(c.attend(gdn, window=window), want)), window


def test_append_refuses_other_numbers_of_requests(gdn):
    """k [B, T, heads, D] and slots [B]: tokens are not dealt out anew to another number of slots."""
    c = Case(33, [20, 20, 20, 20], H=2, Hq=2)
    new = torch.randn(2, 4, 2, 64, device="cuda").to(BF16)
    k, v = c.to(c.k), c.to(c.v)
    k0, v0 = k.clone(), v.clone()
    args = c.to(c.table), c.to(c.seq), c.to(c.slots)
    with pytest.raises(ValueError, match="requests"):
        gdn.gdn_kv_append(new, new, k, v, *args)
    assert torch.equal(k, k0) and torch.equal(v, v0)
    # packed tokens, and with offsets any grouping, are not such
    gdn.gdn_kv_append(new.reshape(8, 2, 64), new.reshape(8, 2, 64), k, v, *args)
    k1, v1 = k0.clone(), v0.clone()
    gdn.gdn_kv_append(new.reshape(1, 8, 2, 64), new.reshape(1, 8, 2, 64), k1, v1, *args)
    assert torch.equal(k, k1) and torch.equal(v, v1) and not torch.equal(k, k0)
    k1, v1 = k0.clone(), v0.clone()
    off = torch.tensor([0, 2, 4, 6, 8], dtype=torch.int32, device="cuda")
    gdn.gdn_kv_append(new, new, k1, v1, *args, off)
    assert torch.equal(k, k1) and torch.equal(v, v1)


@pytest.mark.parametrize("B", [5, 40, 300, 1023, 1024, 2500])
@pytest.mark.parametrize("tail", ["zeros", "past", "short"])
def test_append_offsets_with_a_tail(gdn, B, tail):
    """A list of offsets of fixed size of which only the first entries are in use: those behind fall
    back to zero, or stand past N (both are empty requests), or N goes further than the last."""
    live, T, H, D, page = max(2, B // 3), 2, 2, 64, 16
    g = torch.Generator().manual_seed(B)
    counts = torch.randint(0, 4, (live,), generator=g)
    n = int(counts.sum())
    off = torch.zeros(B + 1, dtype=torch.int64)
    off[1:live + 1] = torch.cumsum(counts, 0)
    N = n + 70
    off[live + 1:] = {"zeros": 0, "past": N + 5, "short": n}[tail]
    if tail == "past":              # the last live request ends where the tokens do
        counts[-1] += N - n
        off[live] = N
    seq = torch.zeros(B, dtype=torch.int32)
    seq[:live] = counts + 3
    width = pages_of(int(seq.max()), page)
    table = torch.arange(B * width, dtype=torch.int32).reshape(B, width)
    slots = torch.randperm(B, generator=g).to(torch.int32)
    by_slot = torch.empty_like(seq)
    by_slot[slots.long()] = seq
    kv = torch.randn(N, 2 * H, D, generator=g).to(BF16)
    k, v = (torch.zeros(B * width, page, H, D, dtype=BF16, device="cuda") for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    packed = kv.cuda()
    gdn.gdn_kv_append(packed[:, :H], packed[:, H:], k, v, table.cuda(), by_slot.cuda(), slots.cuda(),
                      off.to(torch.int32).cuda(), dev_status=st)
    wk, wv = (torch.zeros(B * width, page, H, D, dtype=BF16) for _ in range(2))
    at = 0
    for b in range(live):
        for i in range(int(counts[b])):
            p = int(table[int(slots[b]), (3 + i) // page])
            wk[p, (3 + i) % page], wv[p, (3 + i) % page] = kv[at, :H], kv[at, H:]
            at += 1
    assert torch.equal(k.cpu(), wk) and torch.equal(v.cpu(), wv) and int(st.item()) == 0
