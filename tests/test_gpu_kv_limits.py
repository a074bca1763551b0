"""Paged key/value operators at their limits: many sequences, long pools, values that are not finite, explicit
streams, refused tensors."""
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


def make(csa, old, new, H, hk, dim, dtype, cache, **kw):
    from .kv_case import Case
    return Case(csa, old, new, H, hk, dim, dtype, cache, **kw)


def plain(c, scale, window=0):
    """The definition in fp64 on the GPU: (out, lse, sum of p |v|, sum of |v| that is seen), rows of all sequences."""
    g, n_tok = c.H // c.kv_heads, c.n_tokens.tolist()
    out = torch.zeros(c.used, c.H, c.dim, dtype=torch.float64, device="cuda")
    mag, vsum, lse = torch.zeros_like(out), torch.zeros_like(out), torch.zeros(c.used, c.H, dtype=torch.float64, device="cuda")
    row = 0
    for b, m in enumerate(c.new):
        n = n_tok[b]
        if m == 0:
            continue
        at = torch.arange(n, device="cuda")
        pages = c.table[b, at // 64].long()
        k, v = (p.permute(0, 2, 1, 3)[pages, at % 64].double() for p in (c.k_pages, c.v_pages))
        pos = torch.arange(n - m, n, device="cuda")[:, None]
        seen = (at <= pos) & (at > pos - window if window else at >= 0)
        for h in range(c.kv_heads):
            q = c.q[row:row + m, h * g:(h + 1) * g].double()
            s = torch.where(seen[:, None], q @ k[:, h].t() * scale, -math.inf)
            p = torch.softmax(s, -1)
            out[row:row + m, h * g:(h + 1) * g] = p @ v[:, h]
            mag[row:row + m, h * g:(h + 1) * g] = p @ v[:, h].abs()
            vsum[row:row + m, h * g:(h + 1) * g] = (seen.double() @ v[:, h].abs())[:, None]
            lse[row:row + m, h * g:(h + 1) * g] = torch.logsumexp(s, -1)
        row += m
    return out, lse, mag, vsum


def close(c, got, lse, scale, window=0, s_max=64.0):
    """u_p is the rounding of the probabilities; scores are below s_max, so fp32 products of `dim` terms, their sums and
    exp2 leave at most 2 s_max dim 2^-24 in the exponent; the polynomial of a quarter of them 2^-18.  A probability of
    fp16 is a multiple of 2^-24 with a row's largest at 1 or more, one of three E4M3 terms a multiple of 2^-17 with the
    largest at 2^4 or more, so each is off by up to half of that on top: 2^-25 or 2^-22 of the largest, which is no more
    than their sum."""
    want, l, mag, vsum = plain(c, scale, window)
    eps = 2 * s_max * c.dim * 2.0 ** -24 + 2.0 ** -18
    u_p = 2.0 ** -8 if c.cache_dtype == BF else 2.0 ** -11
    u_o = 2.0 ** -8 if c.dtype == BF else 2.0 ** -11
    p_err = (u_p + eps) * mag + {BF: 0.0, HF: 2.0 ** -25, E4: 2.0 ** -22}[c.cache_dtype] * vsum
    bound = p_err + u_o * (want.abs() + p_err) + 2.0 ** -25
    d = (got[:c.used].double() - want).abs()
    assert (d <= bound).all(), (d - bound).max()
    assert ((lse[:c.used].double() - l).abs() <= eps + 2.0 ** -23 * l.abs()).all()


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, E4), (BF, E4)])
@pytest.mark.parametrize("seed,B,most_new,most_old,g,hk,window", [
    (1, 37, 60, 900, 4, 2, 0), (2, 5, 700, 3000, 5, 1, 0), (3, 64, 9, 700, 16, 1, 100), (4, 23, 300, 300, 3, 4, 0),
    (5, 150, 3, 2000, 5, 2, 0), (6, 11, 130, 1500, 1, 8, 70), (7, 3, 40, 20000, 8, 1, 0)])
def test_ragged_batches(csa, seed, B, most_new, most_old, g, hk, window, dtype, cache):
    """Many items of unequal cost, which the cuts between the CTAs divide everywhere."""
    r = np.random.default_rng(seed)
    new = [int(x) for x in r.integers(0, most_new + 1, B)]
    old = [int(x) for x in r.integers(0, most_old + 1, B) // r.integers(1, 9, B)]
    new[0] = max(new[0], 1)
    c = make(csa, old, new, g * hk, hk, 64, dtype, cache, seed=seed)
    c.hold_all()
    out, lse = c.attend(0.125, window)
    torch.cuda.synchronize()
    assert c.status[0].item() == 0
    close(c, out, lse, 0.125, window)
    again, lse2 = c.attend(0.125, window)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # the joins' order is fixed


@pytest.mark.parametrize("new", [1, 20])
def test_the_largest_batch(csa, new):
    B = 1024
    c = make(csa, [(7 * i) % 200 for i in range(B)], [new if i % 3 else 0 for i in range(B)], 4, 1, 64, BF, BF, seed=1)
    c.hold_all()
    out, lse = c.attend(0.125)
    torch.cuda.synchronize()
    assert c.status[0].item() == 0
    close(c, out, lse, 0.125)


@pytest.mark.parametrize("H,hk", [(128, 1), (128, 2), (96, 1)])
@pytest.mark.parametrize("new", [1, 3, 50])
def test_many_heads_to_a_group(csa, H, hk, new):
    c = make(csa, [300, 0, 77], [new, new, 0], H, hk, 128, BF, BF, seed=2)
    c.hold_all()
    out, lse = c.attend(128 ** -0.5)
    torch.cuda.synchronize()
    close(c, out, lse, 128 ** -0.5)


@pytest.mark.parametrize("cache,kv_heads", [(BF, 8), (E4, 16)])
@pytest.mark.parametrize("new", [1, 150])
def test_pools_beyond_32_bits(csa, cache, kv_heads, new):
    """Pages whose elements lie behind 2^32: the sequence takes the first and the last ones of the pool."""
    dim, pages = 128, 66000  # 2^32 elements are 65,536 pages of 8 heads
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free memory")
    kp = torch.empty(pages, kv_heads, 64, dim, dtype=cache, device="cuda")
    vp = torch.empty_like(kp)
    n, H = 400, 2 * kv_heads
    ids = [pages - 1, 0, pages - 2, pages // 2, pages - 300, 5, pages - 7]
    kp[ids] = torch.full((), float("nan"), device="cuda").to(cache)
    vp[ids] = kp[ids]
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    n_tokens, status = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    d = csa.kv_cache(kp, vp, table, n_tokens, status)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(n, kv_heads, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
    csa.kv_append(d, k, v, torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    q = torch.randn(new, H, dim, generator=g, device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty(new, H, device="cuda")
    ws = torch.empty(csa.kv_attn_workspace(d, new, new, H), dtype=torch.uint8, device="cuda")
    csa.kv_attn(d, q, torch.tensor([0, new], dtype=torch.int32, device="cuda"), new, 0.09, out, ws, lse=lse)
    torch.cuda.synchronize()
    assert status[0].item() == 0 and n_tokens[0].item() == n
    at = torch.arange(n, device="cuda")
    for pool, x in ((kp, k), (vp, v)):
        assert torch.equal(pool[torch.tensor(ids, device="cuda")[at // 64], :, at % 64].float(), x.to(cache).float())

    class C:
        pass
    c = C()
    c.H, c.kv_heads, c.dim, c.dtype, c.cache_dtype, c.used, c.new = H, kv_heads, dim, BF, cache, new, [new]
    c.n_tokens, c.table, c.q = n_tokens, torch.arange(len(ids), device="cuda")[None], q
    c.k_pages, c.v_pages = kp[ids], vp[ids]
    close(c, out, lse, 0.09)


@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("new", [[1, 1], [60, 3], [200, 140]])
def test_what_is_not_finite_stays_in_its_rows(csa, cache, new):
    c = make(csa, [150, 90], new, 8, 2, 128, BF, cache, seed=4)
    c.hold_all()
    good, glse = c.attend(0.1)
    c.q[0, 3] = float("nan")            # a query: its row only
    out, lse = c.attend(0.1)
    torch.cuda.synchronize()
    assert out[0, 3].isnan().all() and lse[0, 3].isnan()
    keep = torch.ones(c.total, 8, dtype=torch.bool, device="cuda")
    keep[0, 3] = False
    assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], glse[keep])
    c.q[0, 3] = 0.5
    nan = torch.full((128,), float("nan"), device="cuda").to(cache)
    c.k_pages[c.table[1, 0].long(), 1, 5] = nan  # a key: the rows of its sequence and kv head that see it (all)
    out, lse = c.attend(0.1)
    torch.cuda.synchronize()
    lo = new[0]
    assert out[lo:, 4:].isnan().all() and lse[lo:, 4:].isnan().all()
    assert torch.equal(out[lo:, :4], good[lo:, :4]) and torch.equal(out[1:lo], good[1:lo])


@pytest.mark.parametrize("new", [[1, 0], [5, 40]])
def test_explicit_streams(csa, new):
    """The calls go to the stream that is given, not to the current one."""
    c = make(csa, [100, 64], new, 4, 2, 64, BF, BF, seed=6)
    s = torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(7)
    k, v = (torch.randn(c.total, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    r = csa.rotary(torch.linspace(1, 0.01, 32, device="cuda"), 64)
    pos = torch.arange(c.total, dtype=torch.int32, device="cuda")[None]
    x, y = torch.randn(c.total, 4, 64, generator=g, device="cuda"), torch.empty(c.total, 4, 64, device="cuda")
    torch.cuda.synchronize()
    csa.kv_append(c.desc, k, v, c.cu, c.max_new, start=c.n_tokens.clone(), rotary=r, pos=pos, stream=s)
    csa.rotate(r, x, pos, y, stream=s)
    ws = torch.empty(csa.kv_attn_workspace(c.desc, c.total, c.max_new, 4), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(c.q), torch.empty(c.total, 4, device="cuda")
    csa.kv_attn(c.desc, c.q, c.cu, c.max_new, 0.125, out, ws, lse=lse, stream=s)
    s.synchronize()
    close(c, out, lse, 0.125)
    back = torch.empty_like(x)
    csa.rotate(r, y, pos, back, inverse=True)
    # two rotations in fp32: each value is off by a few roundings of the pair's length
    length = (x[..., :32] ** 2 + x[..., 32:] ** 2).sqrt().repeat(1, 1, 2)
    assert ((back - x).abs() <= 16 * 2.0 ** -24 * length).all()


def test_tensors_that_are_refused(csa):
    c = make(csa, [10], [2], 4, 2, 64, BF, BF)
    out, lse = torch.empty_like(c.q), torch.empty(2, 4, device="cuda")
    ws = torch.empty(csa.kv_attn_workspace(c.desc, 2, 2, 4), dtype=torch.uint8, device="cuda")
    good = dict(cache=c.desc, q=c.q, cu=c.cu, max_new=2, scale=0.1, out=out, ws=ws, lse=lse, window=0)
    csa.kv_attn(**good)
    for what, bad in [("q", c.q.cpu()), ("q", c.q.float()), ("q", c.q[:, :, :32]), ("q", c.q[0]), ("out", out.half()),
                      ("out", out[:1]), ("cu", c.cu.long()), ("cu", c.cu[:1]), ("cu", c.cu.cpu()), ("lse", lse.double()),
                      ("lse", lse.t()), ("ws", ws.cpu()), ("ws", ws[::2])]:
        with pytest.raises((ValueError, csa.Csa2Error)):
            csa.kv_attn(**{**good, what: bad})
    for what, bad in [("q", None), ("cache", 3), ("scale", "x"), ("max_new", 0.5), ("cache", csa.csa2_heads())]:
        with pytest.raises((TypeError, ValueError)):
            csa.kv_attn(**{**good, what: bad})
    with pytest.raises(csa.Csa2Error):
        csa.kv_attn(**{**good, "ws": ws[:64]})
    with pytest.raises(csa.Csa2Error):
        csa.kv_attn(**{**good, "out": c.q})
    r = csa.rotary(torch.ones(16, device="cuda"), 32)
    pos = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    for args in [(c.q, pos[:, :1], out), (c.q, pos.long(), out), (c.q, pos, out[:1]), (c.q.transpose(1, 2), pos, out), (c.q, pos, None)]:
        with pytest.raises((TypeError, ValueError)):
            csa.rotate(r, *args)
    k = torch.zeros(2, 2, 64, dtype=BF, device="cuda")
    for kw in [dict(k=k.half()), dict(v=k[:1]), dict(k=k[:, :1]), dict(start=c.cu), dict(pos=pos), dict(rotary=c.desc)]:
        with pytest.raises((TypeError, ValueError)):
            csa.kv_append(**{**dict(cache=c.desc, k=k, v=k, cu=c.cu, max_new=2), **kw})
    torch.cuda.synchronize()
    assert c.status[0].item() == 0


def test_sizes_beyond_32_bits_are_refused(csa):
    """Broadcast tensors can have them without the memory; nothing is written."""
    c = make(csa, [10], [1], 4, 2, 64, BF, BF)
    k, cu = torch.ones(1, 2, 64, dtype=BF, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    before, count = c.k_pages.clone(), c.n_tokens.clone()
    many = k.expand((1 << 32) + 1, 2, 64)
    with pytest.raises(ValueError):
        csa.kv_append(c.desc, many, many, cu, 1)
    x = torch.ones(1, 1, 64, dtype=BF, device="cuda")
    wide = x.expand(1, (1 << 32) + 1, 64)
    with pytest.raises(ValueError):
        csa.rotate(csa.rotary(torch.ones(16, device="cuda"), 32), wide, torch.zeros(1, 1, dtype=torch.int32, device="cuda"), wide)
    torch.cuda.synchronize()
    assert torch.equal(c.k_pages.view(torch.int16), before.view(torch.int16)) and torch.equal(c.n_tokens, count)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("old,new,H,hk,window", [
    ([9000, 100, 5, 63, 0], [4, 3, 0, 2, 4], 8, 1, 0),     # 32 rows, a long sequence over many CTAs
    ([127, 128, 255, 256, 383, 0], [1] * 6, 20, 1, 0),     # 20 rows, one to four blocks
    ([124, 252, 60], [4, 4, 4], 16, 2, 0),                 # the new tokens end a page, a block
    ([3000, 500, 90], [3, 2, 1], 20, 2, 100),              # 30 rows through a window
    ([700, 64], [2, 1], 16, 2, 0),                         # 16 rows
    ([5000, 1], [1, 1], 5, 1, 64),
])
def test_codes_read_by_the_tensor_cores(csa, dtype, dim, old, new, H, hk, window):
    """E4M3 pages with at most 32 rows to a kv head."""
    c = make(csa, old, new, H, hk, dim, dtype, E4, seed=H + dim)
    c.hold_all()
    for scale in (dim ** -0.5, 1.0):  # the second: scores to +-50, one key takes nearly all
        out, lse = c.attend(scale, window)
        torch.cuda.synchronize()
        assert c.status[0].item() == 0
        close(c, out, lse, scale, window, s_max=128.0)
