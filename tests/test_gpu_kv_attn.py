"""Attention of new tokens over a paged key/value cache against the fp64 oracle."""
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


BF, HF, E4 = "bfloat16", "float16", "float8_e4m3fn"


def make(csa, old, new, H, hk, dim, dtype, cache, **kw):
    from .kv_case import Case
    return Case(csa, old, new, H, hk, dim, getattr(torch, dtype), getattr(torch, cache), **kw)


TYPES = [(BF, BF), (HF, HF), (BF, E4), (HF, E4)]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("old,new,H,hk", [
    ([0], [1], 1, 1),                          # the first token of all
    ([62, 63, 64, 0, 127], [1, 1, 1, 1, 1], 8, 2),   # around a page's end
    ([1000, 3, 517], [1, 1, 1], 16, 1),
    ([700, 0, 64, 129], [4, 2, 0, 3], 12, 4),  # drafts; one sequence brings nothing
    ([300], [37], 5, 1),                       # odd group
    ([0, 200], [130, 65], 14, 2),              # prompts across tiles
    ([0, 1], [257, 300], 2, 2),
    ([1500], [400], 8, 1),
])
def test_chunks(csa, dtype, cache, dim, old, new, H, hk):
    c = make(csa, old, new, H, hk, dim, dtype, cache, seed=len(old) * 100 + H)
    c.hold_all()
    out, lse = c.attend(0.125)
    torch.cuda.synchronize()
    assert c.status[0].item() == 0
    c.check(out, lse, 0.125)


@pytest.mark.parametrize("dtype,cache", [(BF, BF), (HF, E4)])
@pytest.mark.parametrize("window", [1, 2, 64, 100, 128, 5000])
@pytest.mark.parametrize("old,new,H,hk", [([500, 63, 0], [1, 1, 1], 8, 2), ([333, 0, 64], [150, 70, 1], 6, 2)])
def test_windows(csa, dtype, cache, window, old, new, H, hk):
    c = make(csa, old, new, H, hk, 128, dtype, cache, seed=window)
    c.hold_all()
    out, lse = c.attend(0.09, window)
    torch.cuda.synchronize()
    c.check(out, lse, 0.09, window)


@pytest.mark.parametrize("old,new,H,hk", [([9000, 4097, 20000], [1, 1, 1], 8, 2), ([6000], [4], 8, 1), ([5000, 3000], [16, 9], 8, 2),
                                          ([4000], [300], 4, 1)])
@pytest.mark.parametrize("cache", [BF, E4])
def test_long_sequences(csa, old, new, H, hk, cache):
    c = make(csa, old, new, H, hk, 128, BF, cache, seed=7)
    c.hold_all()
    out, lse = c.attend(128 ** -0.5)
    torch.cuda.synchronize()
    c.check(out, lse, 128 ** -0.5)


@pytest.mark.parametrize("H,hk", [(8, 8), (8, 1), (64, 2), (128, 128), (7, 1)])
def test_tokens_that_see_no_key(csa, H, hk):
    """More new tokens than the cache holds: the first ones stand before its start."""
    c = make(csa, [0, 0, 0], [5, 3, 40], H, hk, 64, BF, BF, seed=3)
    c.n_tokens.copy_(torch.tensor([2, 0, 1], dtype=torch.int32))
    out, lse = c.attend(0.2)
    torch.cuda.synchronize()
    c.check(out, lse, 0.2)
    assert (out[5:8] == 0).all() and torch.isneginf(lse[5:8]).all()
    assert (out[:3] == 0).all() and (out[8:47] == 0).all()


@pytest.mark.parametrize("new", [[1, 1], [3, 0], [90, 140]])
def test_rows_behind_the_last_sequence_stay(csa, new):
    c = make(csa, [100, 30], new, 8, 2, 128, BF, BF, seed=5, tail_rows=37)
    c.hold_all()
    out, lse = c.attend(0.1)
    torch.cuda.synchronize()
    c.check(out, lse, 0.1)
    assert (out[c.used:] == 777.0).all() and (lse[c.used:] == 777.0).all()


@pytest.mark.parametrize("new,H", [([1, 2], 6), ([80, 70], 6)])
def test_strides(csa, new, H):
    """q and out inside wider rows, and with the heads outermost; no lse."""
    c = make(csa, [50, 70], new, H, 2, 64, HF, HF, seed=6)
    c.hold_all()
    wide = torch.zeros(c.total, H + 3, 64 + 8, dtype=torch.float16, device="cuda")
    qv = wide[:, 2:2 + H, 8:]
    qv.copy_(c.q)
    outer = torch.zeros(H, c.total, 64, dtype=torch.float16, device="cuda")
    ov = outer.transpose(0, 1)
    c.attend(0.15, q=qv, out=ov, lse=None)
    torch.cuda.synchronize()
    c.check(ov, None, 0.15)
    wide2 = torch.full((c.total, 2 * H, 64), 5.0, dtype=torch.float16, device="cuda")
    c.attend(0.15, q=qv, out=wide2[:, :H], lse=None)
    torch.cuda.synchronize()
    assert torch.equal(wide2[:, :H], ov) and (wide2[:, H:] == 5.0).all()


@pytest.mark.parametrize("new", [[1, 1], [100, 3]])
@pytest.mark.parametrize("cache", [BF, E4])
def test_queries_of_any_magnitude(csa, new, cache):
    for q_scale, scale in ((2.0 ** 60, 2.0 ** -62), (2.0 ** -60, 2.0 ** 58), (1e4, 1e-5)):
        c = make(csa, [200, 10], new, 4, 2, 128, BF, cache, seed=8, q_scale=q_scale)
        c.hold_all()
        out, lse = c.attend(scale)
        torch.cuda.synchronize()
        c.check(out, lse, scale)


@pytest.mark.parametrize("new", [[1], [2], [60], [200]])
def test_peaked_and_growing_scores(csa, new):
    """Scores that grow along the sequence move the running maximum again and again; one key takes all."""
    c = make(csa, [900], new, 4, 2, 128, BF, BF, seed=9)
    n = 900 + new[0]
    ramp = torch.linspace(-3, 3, n, device="cuda")
    at = torch.arange(n, device="cuda")
    c.k_pages.permute(0, 2, 1, 3)[c.table[0, at // 64].long(), at % 64] = ramp[:, None, None].expand(n, 2, 128).to(torch.bfloat16)
    c.q.fill_(1.0)
    c.hold_all()
    for sign in (1.0, -1.0):
        q = (c.q * sign).contiguous()
        out, lse = c.attend(0.5, q=q)
        torch.cuda.synchronize()
        c.check(out, lse, 0.5, q=q)


@pytest.mark.parametrize("new", [[1, 1, 1], [70, 3, 200]])
@pytest.mark.parametrize("cache", [BF, E4])
def test_page_outside_the_pool_is_left_out(csa, new, cache):
    c = make(csa, [400, 300, 130], new, 4, 2, 128, BF, cache, seed=10)
    c.hold_all()
    good = c.table.clone()
    c.table[1, 2] = c.num_pages + 5
    c.table[1, 0] = -1
    out, lse = c.attend(0.1)
    torch.cuda.synchronize()
    assert c.status[0].item() == csa.DEVERR_PAGE
    c.check(out, lse, 0.1, seqs=[0, 2])
    # the same sequence with the bad pages' keys absent
    from .kv_case import host
    n = 300 + new[1]
    keep = np.array([j for j in range(n) if j // 64 not in (0, 2)])
    kp, vp, qh, tb = host(c.k_pages), host(c.v_pages), host(c.q), good.cpu().numpy()
    r0 = new[0]
    for h in range(4):
        k = kp[tb[1, keep // 64], h // 2, keep % 64]
        v = vp[tb[1, keep // 64], h // 2, keep % 64]
        for i in range(new[1]):
            see = keep <= 300 + i
            s = 0.1 * (k[see] @ qh[r0 + i, h])
            p = np.exp(s - s.max())
            o = p / p.sum() @ v[see]
            got = out[r0 + i, h].double().cpu().numpy()
            assert np.abs(got - o).max() <= 2.0 ** -7 * np.abs(v).max()


@pytest.mark.parametrize("new", [[1, 1], [90, 20]])
def test_counts_outside_the_cache(csa, new):
    c = make(csa, [100, 64], new, 4, 1, 64, BF, BF, seed=11)
    c.hold_all()
    c.n_tokens[1] = -9  # read as empty
    out, lse = c.attend(0.1)
    torch.cuda.synchronize()
    assert c.status[0].item() == csa.DEVERR_COUNT
    c.check(out, lse, 0.1, seqs=[0])
    assert (out[new[0]:] == 0).all() and torch.isneginf(lse[new[0]:]).all()


def test_bad_bounds_leave_the_sequence_out(csa):
    c = make(csa, [100, 64, 10], [4, 4, 4], 4, 1, 64, BF, BF, seed=12)
    c.hold_all()
    c.cu.copy_(torch.tensor([0, 4, 2, 12], dtype=torch.int32))  # decreasing; the last brings 10 with a bound of 4
    out, lse = c.attend(0.1, max_new=4)
    torch.cuda.synchronize()
    assert c.status[0].item() == csa.DEVERR_COUNT
    assert (out[4:] == 777.0).all()
    c.check(out, lse, 0.1, seqs=[0])
    for bad in ([0, 4, 8, 13], [-1, 4, 8, 12]):
        c.status.zero_()
        c.cu.copy_(torch.tensor(bad, dtype=torch.int32))
        c.attend(0.1)
        torch.cuda.synchronize()
        assert c.status[0].item() == csa.DEVERR_COUNT


@pytest.mark.parametrize("new,steps", [([1, 1], 4), ([40, 30], 2)])
def test_captured_and_replayed_with_growing_counts(csa, new, steps):
    """A graph of one call serves later steps: counts, pages and queries are read when it runs."""
    c = make(csa, [300 + 70, 20 + 70], new, 8, 2, 128, BF, BF, seed=13)
    c.hold_all()
    full = c.n_tokens.clone()
    s = torch.cuda.Stream()
    out, lse = torch.empty_like(c.q), torch.empty(c.total, 8, device="cuda")
    ws = torch.empty(max(16, csa.kv_attn_workspace(c.desc, c.total, c.max_new, 8)), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        csa.kv_attn(c.desc, c.q, c.cu, c.max_new, 0.1, out, ws, lse=lse)
    for i in range(steps):
        c.n_tokens.copy_(full - 70 + 70 * (i + 1) // steps)
        c.q.normal_()
        out.fill_(777.0)
        g.replay()
        torch.cuda.synchronize()
        c.check(out, lse, 0.1)


def test_two_streams_at_once(csa):
    cs = [make(csa, [3000, 200], n, 8, 2, 128, BF, BF, seed=14 + i) for i, n in enumerate(([1, 1], [200, 90]))]
    streams = [torch.cuda.Stream() for _ in cs]
    for c in cs:
        c.hold_all()
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for c, s, outs in zip(cs, streams, got):
            with torch.cuda.stream(s):  # the outputs and the workspace are filled on it as well
                outs.append(c.attend(0.1))
    torch.cuda.synchronize()
    for c, outs in zip(cs, got):
        for o, l in outs:
            c.check(o, l, 0.1)
            assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])  # and the same every time
