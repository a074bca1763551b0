"""Paged key/value operators at the edges of what their description allows: bounds out of order, rows that see
nothing, values that are not finite, windows that hide nothing, keys far below a row's largest score."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def csa():
    from fp4_sparse_attention_pack_b200 import _build
    _build.build()
    import fp4_sparse_attention_pack_b200 as m
    return m


BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
TYPES = [(BF, BF), (HF, HF), (BF, E4), (HF, E4)]


def make(csa, old, new, H, hk, dim, dtype, cache, **kw):
    from .kv_case import Case
    return Case(csa, old, new, H, hk, dim, dtype, cache, **kw)


def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32)


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 200, 2 ** 30 + 77, 2 ** 30, 1 << 20])
@pytest.mark.parametrize("new,H,hk", [([8, 1, 5, 8, 3, 8], 2, 2),        # at most 16 rows to a kv head
                                      ([8, 1, 5, 8, 3, 8], 8, 2),        # 32
                                      ([8, 300, 5, 70, 1, 130], 6, 2)])  # chunks
def test_windows_that_hide_nothing(csa, dtype, cache, window, new, H, hk):
    """With tokens that stand before the cache's start, and a count that is read as 0, among sequences that are good."""
    c = make(csa, [9, 100, 700, 64, 0, 3000], new, H, hk, 128, dtype, cache, seed=21)
    c.hold_all()
    c.n_tokens[0] = 5    # 8 new over 5 held
    c.n_tokens[3] = -9   # read as empty
    want, wlse = c.attend(0.09)
    torch.cuda.synchronize()
    assert c.status[0].item() == csa.DEVERR_COUNT
    out, lse = c.attend(0.09, window)
    torch.cuda.synchronize()
    c.check(out, lse, 0.09, seqs=[0, 1, 2, 4, 5])
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    r = sum(new[:3])
    assert (out[r:r + new[3]] == 0).all() and torch.isneginf(lse[r:r + new[3]]).all()


@pytest.mark.parametrize("how", ["start", "held", "alias"])
@pytest.mark.parametrize("by", [1, 50])
@pytest.mark.parametrize("cu,total,max_new", [
    ([0, 10, 5, 20, 30], 30, 15),       # the second sequence's bounds decrease; rows 5 to 9 are the first's and the third's
    ([0, 12, 4, 9, 9, 14], 14, 12),
    ([0, 100, 5, 12], 12, 12),          # a bound beyond the rows
    ([-3, 4, 2, 12, 11, 1, 6], 12, 10),
    ([0, 3, 9, 9, 12], 12, 6),          # in order
    ([20, 1, 20, 1, 20], 20, 20),
])
def test_append_takes_each_sequence_by_its_own_bounds(csa, how, by, cu, total, max_new):
    """A sequence whose bounds are in order gets its rows, whatever the bounds of the others are."""
    cu, total, max_new, B = [x * by for x in cu], total * by, max_new * by, len(cu) - 1
    c = make(csa, [3 + 40 * b for b in range(B)], [max_new] * B, 2, 2, 64, BF, BF, seed=22)
    start = c.n_tokens.clone()
    c.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(total, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    wk, wv, wn = c.k_pages.clone(), c.v_pages.clone(), start.tolist()
    offends = False
    for b in range(B):
        lo, hi = cu[b], cu[b + 1]
        if not 0 <= lo <= hi <= total or hi - lo > max_new:
            offends = True
            continue
        at = torch.arange(wn[b], wn[b] + hi - lo, device="cuda")
        for pool, x in ((wk, k), (wv, v)):
            pool.permute(0, 2, 1, 3)[c.table[b, at // 64].long(), at % 64] = x[lo:hi]
        wn[b] += hi - lo
    csa.kv_append(c.desc, k, v, c.cu, max_new, start={"start": start, "held": None, "alias": c.n_tokens}[how])
    torch.cuda.synchronize()
    assert c.status[0].item() == (csa.DEVERR_COUNT if offends else 0)
    assert c.n_tokens.tolist() == wn
    assert torch.equal(bits(c.k_pages), bits(wk)) and torch.equal(bits(c.v_pages), bits(wv))


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [[1, 1], [4, 2], [8, 3], [30, 5], [200, 140]])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_infinite_queries(csa, dtype, cache, dim, new, value):
    """A channel of a query is infinite: its scores are infinities of both signs, so the row is NaN, and only the row."""
    c = make(csa, [150, 90], new, 8, 2, dim, dtype, cache, seed=23)
    c.hold_all()
    good, glse = c.attend(0.1)
    c.q[0, 3, 5] = value
    c.q[new[0], 6] = value
    out, lse = c.attend(0.1)
    torch.cuda.synchronize()
    keep = torch.ones(c.total, 8, dtype=torch.bool, device="cuda")
    for t, h in ((0, 3), (new[0], 6)):
        assert out[t, h].isnan().all() and lse[t, h].isnan()
        keep[t, h] = False
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], glse[keep])
    c.n_tokens[0] = new[0] - 1  # the first token sees no key
    out, lse = c.attend(0.1)
    torch.cuda.synchronize()
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,H,hk", [([6, 3], 8, 8), ([6, 3], 8, 2), ([40, 8], 8, 2), ([300, 4], 4, 2)])
def test_rows_that_see_no_key_are_zero(csa, dtype, cache, dim, new, H, hk):
    """More tokens than are held, and a value that is NaN where only later tokens see it."""
    c = make(csa, [0, 0], new, H, hk, dim, dtype, cache, seed=24)
    held = [2, 3]
    c.n_tokens.copy_(torch.tensor(held, dtype=torch.int32))
    c.v_pages[c.table[0, 0].long(), :, 1, 7] = torch.full((), math.nan, device="cuda").to(cache)
    out, lse = c.attend(0.2)
    torch.cuda.synchronize()
    for lo, m, n in ((0, new[0], held[0]), (new[0], new[1], held[1])):
        assert (out[lo:lo + m - n] == 0).all() and torch.isneginf(lse[lo:lo + m - n]).all()
        assert lse[lo + m - n:lo + m].isfinite().all()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("old,new,H,hk,window", [
    ([70, 200], [4, 3], 8, 4, 0),        # at most 16 rows to a kv head
    ([126, 9000, 60], [4, 4, 3], 8, 2, 0),
    ([5000, 64], [8, 5], 8, 2, 0),       # 32; a long sequence over many CTAs
    ([3000, 90], [5, 4], 6, 2, 100),
    ([900, 120], [16, 9], 8, 2, 0),      # one tile of the chunk kernel
    ([300, 40], [150, 70], 8, 4, 0),     # two
    ([300, 40], [150, 70], 6, 2, 50),
    ([900], [300], 2, 2, 0),
    ([20000], [70], 16, 2, 10000),
])
def test_values_that_are_not_finite_reach_the_tokens_that_see_them(csa, dtype, cache, dim, old, new, H, hk, window):
    """A key that only later tokens see, or only earlier ones through a window, in the same call: its NaN or infinity is
    no part of the others' sums."""
    c = make(csa, old, new, H, hk, dim, dtype, cache, seed=25)
    c.hold_all()
    scale = dim ** -0.5
    good, glse = c.attend(scale, window)
    want = good.clone()
    g, row = H // hk, 0
    for b, (o, m) in enumerate(zip(old, new)):
        at = torch.arange(o, o + m, device="cuda")
        places = [(o + m - 1, 3, math.inf), (o + m // 2, 4, math.nan), (o + 1, 5, -math.inf), (o + m - 1, 6, math.nan)]
        if window:
            places += [(max(0, o - window + 2), 7, math.inf), (max(0, o + m // 2 - window + 1), 8, math.nan)]
        for j, ch, x in places:
            if cache == E4:
                x = math.nan
            c.v_pages[c.table[b, j // 64].long(), hk - 1, j % 64, ch] = torch.full((), x, device="cuda").to(cache)
            see = (at >= j) & ((at < j + window) if window else at >= 0)
            want[row:row + m, H - g:, ch] = torch.where(see[:, None], x, want[row:row + m, H - g:, ch])
        row += m
    out, lse = c.attend(scale, window)
    torch.cuda.synchronize()
    assert torch.equal(lse, glse)
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.nan_to_num(nan=5.0), want.nan_to_num(nan=5.0))


def far_keys(csa, old, new, H, hk, dim, dtype, cache, nats, step):
    """One key of 16 has a score above all others by `nats`, and a value of 0: the others make the whole result.
    Each of their probabilities is rounded once, and off by at most `step` times the largest one besides."""
    c = make(csa, old, new, H, hk, dim, dtype, cache, seed=26)
    c.hold_all()
    c.q.fill_(1.0)
    n = old[0] + new[0]
    at = torch.arange(n, device="cuda")
    sink = at % 16 == 5
    k = torch.where(sink, 1.0, 0.0)[:, None, None].expand(n, hk, dim)
    v = torch.rand(n, hk, dim, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") * 192 + 256
    v = torch.where(sink[:, None, None], 0.0, v)
    for pool, x in ((c.k_pages, k), (c.v_pages, v)):
        pool.permute(0, 2, 1, 3)[c.table[0, at // 64].long(), at % 64] = x.to(cache)
    v = v.to(cache).double()
    out, lse = c.attend(nats / dim)
    torch.cuda.synchronize()
    pos = torch.arange(old[0], n, device="cuda")[:, None]
    s = torch.where(at <= pos, torch.where(sink, float(np.float32(nats / dim)) * dim, 0.0).double(), -math.inf)
    p = torch.softmax(s, -1)                                            # [tokens][keys]
    want = torch.einsum("tj,jhd->thd", p, v).repeat_interleave(H // hk, 1)
    sums = torch.einsum("tj,jhd->thd", (at <= pos).double(), v).repeat_interleave(H // hk, 1)
    # scores are exact in fp32 but for scale log2 e and its product (2^-22 of nats each), exp2 and the polynomial 2^-18
    eps = 2 * nats * 2.0 ** -21 + 2.0 ** -18 + (n / 8 + 64) * 2.0 ** -24
    u_p, u_o = 2.0 ** -8 if cache == BF else 2.0 ** -11, 2.0 ** -8 if dtype == BF else 2.0 ** -11
    err = (u_p + eps) * want + step * p.amax(-1)[:, None, None] * sums
    bound = err + u_o * (want + err) + 2.0 ** -25
    d = (out.double() - want).abs()
    assert (d <= bound).all(), (d / bound).max()
    l = torch.logsumexp(s, -1)[:, None]
    assert ((lse.double() - l).abs() <= eps + 2.0 ** -23 * l.abs()).all()


# (over E4M3 pages, calls of at most 32 rows to a kv head split their probabilities otherwise)
@pytest.mark.parametrize("dtype,cache,old,new,H,hk", [
    (dtype, cache, *size) for dtype, cache in TYPES
    for size in (([3990], [1], 8, 2), ([3990], [4], 8, 4), ([2000], [20], 8, 2), ([1500], [300], 2, 2))
    if cache != E4 or size[1][0] * size[2] // size[3] > 32])
@pytest.mark.parametrize("nats", [12.0, 17.5, 18.4])
def test_keys_far_below_the_largest_score(csa, dtype, cache, nats, old, new, H, hk):
    """Probabilities of 2^-17 to 2^-26.5 of a row's largest one.  In fp16 the largest lies at 2^7 or above, so half a
    step of its subnormals is 2^-32 of it (bf16 has none here)."""
    far_keys(csa, old, new, H, hk, 128, dtype, cache, nats, 2.0 ** -32)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nats", [10.0, 14.5, 15.7, 16.3])
@pytest.mark.parametrize("old,new,H,hk", [([3990], [1], 8, 2), ([3990], [4], 8, 2), ([2000], [8], 8, 2)])
def test_keys_far_below_the_largest_score_over_codes(csa, dtype, dim, nats, old, new, H, hk):
    """The last of three E4M3 terms is a multiple of 2^-19 and the largest probability 2^4 or more: half a step is 2^-24
    of it."""
    far_keys(csa, old, new, H, hk, dim, dtype, E4, nats, 2.0 ** -24)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("H", [16, 32])
def test_small_channels_of_a_query_over_codes(csa, dtype, dim, H):
    """A channel is kept to 2^-27 of the row's largest one: rows whose channels are all one small value, so that what its
    terms lose adds up."""
    rows = 10 * 128  # 2^-14 .. 2^-23 times 1 + i / 128
    B = rows // H
    c = make(csa, [3] * B, [1] * B, H, 1, dim, dtype, E4, seed=27)
    c.hold_all()
    i = torch.arange(rows, device="cuda")
    small = (1 + (i % 128).double() / 128) * 2.0 ** (-14 - (i // 128)).double()
    q = small[:, None].repeat(1, dim)
    q[:, 0] = 1.0
    c.q.copy_(q.view(B, H, dim).to(dtype))
    q = c.q.double()
    keys = torch.tensor([1.0, 0.5, -1.0, 0.75], device="cuda")[:, None].repeat(1, dim)
    keys[:, 0] = 0.0
    for j in range(4):
        c.k_pages[c.table[:, 0].long(), 0, j] = keys[j].to(E4)
    scale = 2.0 ** 11
    out, lse = c.attend(scale)
    torch.cuda.synchronize()
    s = scale * torch.einsum("thc,jc->thj", q, keys.double())
    want = torch.logsumexp(s, -1)
    # each score is off by 2^-27 a channel; products and sums are exact in fp32 but for 2^-24 of their size, as is exp2
    bound = scale * dim * 2.0 ** -27 + 2.0 ** -21 * (1 + s.abs().amax(-1))
    d = (lse.double() - want).abs()
    assert (d <= bound).all(), (d / bound).max()


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("old,new", [([1000, 300], [1, 2]), ([1000, 300], [30, 5]), ([1000, 300], [200, 140]), ([9000], [300])])
def test_scores_that_are_all_minus_infinity(csa, dtype, cache, dim, old, new):
    """Every score of a row is -infinity: zeros and lse -infinity (NaN over E4M3 pages in calls of at most 32 rows)."""
    c = make(csa, old, new, 8, 2, dim, dtype, cache, seed=28)
    c.hold_all()
    n = old[0] + new[0]
    at = torch.arange(n, device="cuda")
    c.k_pages.permute(0, 2, 1, 3)[c.table[0, at // 64].long(), at % 64, :, 0] = torch.ones(n, 2, device="cuda").to(cache)
    c.v_pages.permute(0, 2, 1, 3)[c.table[0, at // 64].long(), at % 64] = torch.full((n, 2, dim), 300.0, device="cuda").to(cache)
    good, glse = c.attend(0.1)
    c.q[0, 3, 0] = -math.inf
    c.q[new[0] - 1, 6, 0] = -math.inf
    out, lse = c.attend(0.1)
    torch.cuda.synchronize()
    keep = torch.ones(c.total, 8, dtype=torch.bool, device="cuda")
    for t, h in ((0, 3), (new[0] - 1, 6)):
        if cache == E4 and max(new) * 4 <= 32:
            assert out[t, h].isnan().all() and lse[t, h].isnan()
        else:
            assert (out[t, h] == 0).all() and torch.isneginf(lse[t, h])
        keep[t, h] = False
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], glse[keep])
