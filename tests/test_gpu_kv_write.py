"""Rotary positions and the append to a paged key/value cache against the fp64 oracle, and a run of the three operators."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kv as okv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def csa():
    from fp4_sparse_attention_pack_b200 import _build
    _build.build()
    import fp4_sparse_attention_pack_b200 as m
    return m


def spec(csa, rot, offset, neighbours, n_axes):
    from .kv_case import axis_of, inv_freq
    f, axis = inv_freq(rot), axis_of(rot, n_axes)
    return csa.rotary(f, rot, offset=offset, neighbours=neighbours, n_axes=n_axes, axis=axis), f.cpu().numpy(), axis


def bound(x, y, dtype, rot, offset, neighbours):
    """The output's rounding, and the fp32 rotation: an angle off by 2^-26 turns (1e-7 rad), sine and cosine by 2 ulp,
    three roundings: under 5e-7 of |a| + |b|, which is at most the row's largest two magnitudes."""
    from .kv_case import TINY, U
    part = np.abs(x[..., offset:offset + rot]).max(-1, keepdims=True)
    return U[dtype] * (np.abs(y) + 1e-6 * part) + 1e-6 * part + TINY[dtype]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tokens,heads,dim,rot,offset", [(1, 1, 64, 64, 0), (3, 5, 128, 32, 96), (700, 3, 128, 128, 0),
                                                         (65, 64, 512, 64, 448), (9, 1, 512, 256, 8), (33, 2, 24, 16, 8)])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotate(csa, dtype, tokens, heads, dim, rot, offset, neighbours, inverse):
    n_axes = 3 if tokens % 2 else 1
    r, f, axis = spec(csa, rot, offset, neighbours, n_axes)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, heads, dim, generator=g, device="cuda").to(dtype)
    pos = torch.randint(-5, 1 << 20, (n_axes, tokens), generator=g, device="cuda", dtype=torch.int32)
    out = torch.empty_like(x)
    csa.rotate(r, x, pos, out, inverse=inverse)
    xh = x.double().cpu().numpy()
    y = okv.rotate(xh, pos.cpu().numpy(), f, rot, offset, neighbours, axis, inverse)
    got = out.double().cpu().numpy()
    assert (np.abs(got - y) <= bound(xh, y, dtype, rot, offset, neighbours)).all()
    same = np.ones(dim, bool)
    same[offset:offset + rot] = False
    assert np.array_equal(got[..., same], xh[..., same])
    again = x.clone()
    csa.rotate(r, again, pos, again, inverse=inverse)  # in place
    assert torch.equal(again, out)


def test_rotate_strides_and_empty(csa):
    r, f, axis = spec(csa, 32, 0, False, 1)
    x = torch.randn(40, 6, 72, device="cuda").bfloat16()
    pos = torch.arange(40, dtype=torch.int32, device="cuda")[None]
    want = torch.empty(40, 4, 64, device="cuda", dtype=torch.bfloat16)
    csa.rotate(r, x[:, 1:5, 8:].contiguous(), pos, want)
    out = torch.zeros(4, 40, 64, device="cuda", dtype=torch.bfloat16)
    csa.rotate(r, x[:, 1:5, 8:], pos, out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), want)
    one = x[:1, :1, 8:].expand(40, 4, 64)  # one row for every token and head
    csa.rotate(r, one, pos, want)
    y = okv.rotate(one.double().cpu().numpy(), pos.cpu().numpy(), f, 32, 0, False, axis)
    assert np.abs(want.double().cpu().numpy() - y).max() <= 2.0 ** -8 * np.abs(y).max() + 1e-5
    csa.rotate(r, x[:0, :4, :64], pos[:, :0].contiguous(), want[:0])


def test_inverse_is_the_gradient(csa):
    """<grad_y, J dx> == <J^T grad_y, dx> in fp32, and J's action against a difference of two rotations."""
    r, f, axis = spec(csa, 64, 0, True, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x, dx, gy = (torch.randn(50, 4, 64, generator=g, device="cuda") for _ in range(3))
    pos = torch.randint(0, 5000, (3, 50), generator=g, device="cuda", dtype=torch.int32)

    def rot(t, inverse=False):
        o = torch.empty_like(t)
        csa.rotate(r, t, pos, o, inverse=inverse)
        return o.double()

    gx = rot(gy, True)
    jdx = rot(dx)
    a, b = (gy.double() * jdx).sum(), (gx * dx.double()).sum()
    scale = gy.double().norm() * dx.double().norm()
    assert abs(a - b) <= 1e-6 * scale
    diff = rot(x + dx) - rot(x - dx)
    assert (diff / 2 - jdx).abs().max() <= 4e-6 * (x.abs().max() + dx.abs().max()).double()


@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                         (torch.bfloat16, torch.float8_e4m3fn), (torch.float16, torch.float8_e4m3fn)])
@pytest.mark.parametrize("old,new,hk,dim,rot,offset,neighbours,n_axes", [
    ([0], [1], 1, 64, 0, 0, False, 1),
    ([63, 64, 0, 130], [1, 1, 1, 1], 8, 128, 128, 0, False, 1),
    ([10, 0, 64, 7], [70, 0, 130, 1], 3, 64, 32, 32, True, 3),
    ([500], [700], 2, 128, 64, 64, False, 3),
    ([5] * 300, [1] * 300, 1, 64, 64, 0, False, 1),
])
def test_append(csa, dtype, cache, old, new, hk, dim, rot, offset, neighbours, n_axes):
    from .kv_case import Case, U, TINY, host
    c = Case(csa, old, new, hk, hk, dim, dtype, cache, seed=sum(new), tail_rows=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(c.total, hk, dim, generator=g, device="cuda").to(dtype) * 3 for _ in range(2))
    k[0, 0, 0], v[0, 0, 1] = 600.0, -1000.0  # beyond E4M3
    before = [host(c.k_pages), host(c.v_pages)]
    tb = c.table.cpu().numpy()
    r = pos = None
    if rot:
        r, f, axis = spec(csa, rot, offset, neighbours, n_axes)
        pos = torch.randint(0, 100000, (n_axes, c.total), generator=g, device="cuda", dtype=torch.int32)
    start = c.n_tokens.clone()
    results = []
    for how in ("start", "held", "alias"):
        c.n_tokens.copy_(start)
        csa.kv_append(c.desc, k, v, c.cu, c.max_new, start={"start": start, "held": None, "alias": c.n_tokens}[how], rotary=r, pos=pos)
        torch.cuda.synchronize()
        assert c.status[0].item() == 0
        assert c.n_tokens.tolist() == [o + n for o, n in zip(old, new)]
        results.append((c.k_pages.view(torch.uint8).clone(), c.v_pages.view(torch.uint8).clone()))
    for a in results[1:]:
        assert torch.equal(a[0], results[0][0]) and torch.equal(a[1], results[0][1])
    kh, vh = host(k), host(v)
    ky = okv.rotate(kh, pos.cpu().numpy(), f, rot, offset, neighbours, axis) if rot else kh
    big = 448.0 if cache == torch.float8_e4m3fn else np.inf
    row = 0
    want = [b.copy() for b in before]
    err = [np.zeros_like(b) for b in before]
    for b, (o, n) in enumerate(zip(old, new)):
        for w, e, y, x in ((want[0], err[0], ky, kh), (want[1], err[1], vh, vh)):
            y = np.clip(y, -big, big)
            part = np.abs(x).max(-1, keepdims=True)
            okv.append(w, tb, b, o, y[row:row + n])
            okv.append(e, tb, b, o, (U[cache] * (np.abs(y) + 1e-6 * part) + 1e-6 * part * bool(rot) + TINY[cache])[row:row + n])
        row += n
    for got, w, e in zip((host(c.k_pages), host(c.v_pages)), want, err):
        same = (got == w) | (np.isnan(got) & np.isnan(w))
        assert (same | (np.abs(got - w) <= e)).all()


def test_positions_count_the_slots_by_default(csa):
    from .kv_case import Case
    c = Case(csa, [70, 3], [40, 20], 2, 2, 128, torch.bfloat16, torch.bfloat16, seed=2)
    r, f, axis = spec(csa, 128, 0, False, 1)
    k = torch.randn(60, 2, 128, device="cuda").bfloat16()
    csa.kv_append(c.desc, k, k, c.cu, 40, rotary=r)
    a = c.k_pages.view(torch.int16).clone()
    c.n_tokens.copy_(torch.tensor([70, 3], dtype=torch.int32))
    pos = torch.cat([torch.arange(70, 110), torch.arange(3, 23)]).int().cuda()[None].contiguous()
    csa.kv_append(c.desc, k, k, c.cu, 40, rotary=r, pos=pos)
    torch.cuda.synchronize()
    assert torch.equal(a, c.k_pages.view(torch.int16))


@pytest.mark.parametrize("explicit", [True, False])
def test_sequences_that_do_not_fit_stay(csa, explicit):
    from .kv_case import Case
    c = Case(csa, [60, 100, 5], [10, 10, 10], 2, 2, 64, torch.float16, torch.float16, seed=3)
    cap = c.max_pages * 64
    held = torch.tensor([60, cap - 9, -4 if explicit else 5], dtype=torch.int32, device="cuda")
    c.n_tokens.copy_(held)
    kb = c.k_pages.view(torch.int16).clone()
    k = torch.randn(30, 2, 64, device="cuda").half()
    csa.kv_append(c.desc, k, k, c.cu, 10, start=held if explicit else None)
    torch.cuda.synchronize()
    assert c.status[0].item() == csa.DEVERR_CAPACITY
    assert c.n_tokens.tolist() == [70, cap - 9, -4 if explicit else 15]
    tb = c.table.cpu()
    for p in tb[1][tb[1] >= 0].tolist():
        assert torch.equal(c.k_pages[p].view(torch.int16), kb[p])
    c.status.zero_()
    c.n_tokens.copy_(torch.tensor([60, 100, 5], dtype=torch.int32))
    csa.kv_append(c.desc, k, k, c.cu, 9)  # every sequence brings more than the bound
    torch.cuda.synchronize()
    assert c.status[0].item() == csa.DEVERR_COUNT and c.n_tokens.tolist() == [60, 100, 5]


def test_page_outside_the_pool_is_skipped(csa):
    from .kv_case import Case
    c = Case(csa, [60, 10], [70, 5], 1, 1, 64, torch.float16, torch.float16, seed=3)
    lost = int(c.table[0, 1])
    c.table[0, 1] = c.num_pages
    kb = c.k_pages.view(torch.int16).clone()
    k = torch.randn(75, 1, 64, device="cuda").half()
    csa.kv_append(c.desc, k, k, c.cu, 70)
    torch.cuda.synchronize()
    assert c.status[0].item() == csa.DEVERR_PAGE and c.n_tokens.tolist() == [130, 15]
    assert torch.equal(c.k_pages[lost].view(torch.int16), kb[lost])
    assert torch.equal(c.k_pages[int(c.table[0, 0]), 0, 60:], k[:4, 0]) and torch.equal(c.k_pages[int(c.table[0, 2]), 0, :2], k[68:70, 0])
    assert torch.equal(c.v_pages[int(c.table[1, 0]), 0, 10:15], k[70:, 0])


@pytest.mark.parametrize("cache", [torch.bfloat16, torch.float8_e4m3fn])
def test_a_prompt_in_chunks_then_tokens(csa, cache):
    """Rotate, append and attend as a layer does: a prompt in two chunks, single tokens, drafts of which some are taken
    back; against one attention in fp64 over everything."""
    from .kv_case import host
    B, H, hk, dim = 2, 8, 2, 128
    chunks = [[150, 90], [70, 0], [1, 1], [1, 1], [4, 3], [1, 1]]
    take_back = {4: [2, 3]}  # drafts rejected after step 4
    pages = 6
    g = torch.Generator(device="cuda").manual_seed(5)
    kp = torch.zeros(B * pages, hk, 64, dim, device="cuda").to(cache)
    vp = kp.clone()
    table = torch.randperm(B * pages, generator=torch.Generator().manual_seed(1)).int().view(B, pages).cuda()
    n_tokens, status = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    cd = csa.kv_cache(kp, vp, table, n_tokens, status)
    r, f, axis = spec(csa, 64, 0, False, 1)
    held = [0, 0]
    keys = [np.zeros((0, hk, dim)) for _ in range(B)]
    vals = [np.zeros((0, hk, dim)) for _ in range(B)]
    for step, new in enumerate(chunks):
        total, mx = sum(new), max(new)
        q = torch.randn(total, H, dim, generator=g, device="cuda").bfloat16()
        k, v = (torch.randn(total, hk, dim, generator=g, device="cuda").bfloat16() for _ in range(2))
        cu = torch.tensor([0, new[0], total], dtype=torch.int32, device="cuda")
        start = torch.tensor(held, dtype=torch.int32, device="cuda")
        pos = torch.cat([torch.arange(h, h + n) for h, n in zip(held, new)]).int().cuda()[None].contiguous()
        qr = torch.empty_like(q)
        csa.rotate(r, q, pos, qr)
        csa.kv_append(cd, k, v, cu, mx, start=start, rotary=r)
        ws = torch.empty(max(16, csa.kv_attn_workspace(cd, total, mx, H)), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        csa.kv_attn(cd, qr, cu, mx, dim ** -0.5, out, ws)
        torch.cuda.synchronize()
        assert status[0].item() == 0
        ph = pos.cpu().numpy()
        qh, kh = okv.rotate(host(q), ph, f, 64), okv.rotate(host(k), ph, f, 64)
        row = 0
        for b, n in enumerate(new):
            keys[b] = np.concatenate([keys[b][:held[b]], kh[row:row + n]])
            vals[b] = np.concatenate([vals[b][:held[b]], host(v)[row:row + n]])
            held[b] += n
            for h in range(hk):
                o, _, mag = okv.attention(qh[row:row + n, h * 4:h * 4 + 4], keys[b][:, h], vals[b][:, h], held[b], dim ** -0.5)
                got = host(out)[row:row + n, h * 4:h * 4 + 4]
                # rounded q and k change a score by |q||k| scale u, v is rounded, p is rounded, the output is rounded
                u = 2.0 ** -8 if cache == torch.bfloat16 else 2.0 ** -4
                s_err = 128 ** -0.5 * np.abs(qh[row:row + n, h * 4:h * 4 + 4]) @ np.abs(keys[b][:, h]).T * (2.0 ** -8 + u)
                tol = (2 * s_err.max() + u + 2.0 ** -8) * mag + 2.0 ** -8 * np.abs(o) if n else 0
                assert (np.abs(got - o) <= tol).all()
            row += n
        for b, back in enumerate(take_back.get(step, [0, 0])):
            held[b] -= back
