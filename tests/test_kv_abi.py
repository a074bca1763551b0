"""Argument checks of the paged key/value cache operators (no GPU: nothing reaches a kernel), and the oracle's own pins."""
import ctypes

import numpy as np
import pytest

from oracle import kv as okv

OK, INVALID, ALIGN, UNSUPPORTED, CUDA, WORKSPACE = 0, -1, -2, -3, -4, -6


@pytest.fixture(scope="module")
def capi():
    from fp4_sparse_attention_pack_b200 import _build
    _build.build()
    import fp4_sparse_attention_pack_b200 as m
    return m


def heads(m, p=64, ts=1024, hs=128):
    return m.csa2_heads(p, ts, hs)


def cache(m, **kw):
    a = dict(k_pages=16, v_pages=32, page_table=48, n_tokens=64, status=80, batch=2, max_pages=4, num_pages=9, kv_heads=2,
             head_dim=128, dtype=0)
    a.update(kw)
    return m.csa2_kv_cache(*a.values())


def rot(m, axis=None, **kw):
    a = dict(inv_freq=16, axis=None, rot_dim=64, rot_offset=0, neighbours=0, n_axes=1)
    a.update(kw)
    r = m.csa2_rotary(*a.values())
    if axis is not None:
        r.axis = (ctypes.c_uint8 * len(axis))(*axis)
    return r


@pytest.mark.parametrize("why,rc,kw", [
    ("dtype", INVALID, dict(dtype=3)), ("tokens", INVALID, dict(n=-1)), ("heads", INVALID, dict(h=0)),
    ("head_dim", INVALID, dict(d=12)), ("head_dim", INVALID, dict(d=1024)), ("inverse", INVALID, dict(inverse=2)),
    ("rot_dim", INVALID, dict(r=dict(rot_dim=8))), ("rot_dim", INVALID, dict(r=dict(rot_dim=24))),
    ("rot beyond the head", INVALID, dict(r=dict(rot_dim=64, rot_offset=72))), ("offset", INVALID, dict(r=dict(rot_offset=4))),
    ("axes", INVALID, dict(r=dict(n_axes=4))), ("axis", INVALID, dict(r=dict(axis=[0] * 31 + [1]))),
    ("neighbours", INVALID, dict(r=dict(neighbours=2))), ("inv_freq", INVALID, dict(r=dict(inv_freq=None))),
    ("inv_freq", ALIGN, dict(r=dict(inv_freq=20))), ("pos", INVALID, dict(pos=None)), ("pos", ALIGN, dict(pos=20)),
    ("x", INVALID, dict(x=dict(p=None))), ("x", ALIGN, dict(x=dict(p=24))), ("x stride", ALIGN, dict(x=dict(ts=1028))),
    ("x stride", INVALID, dict(x=dict(ts=-1024))), ("y rows meet", INVALID, dict(y=dict(p=128, hs=64))),
    ("y rows meet", INVALID, dict(y=dict(p=128, ts=256, hs=256))), ("in place, other strides", INVALID, dict(y=dict(ts=2048))),
    ("tokens", UNSUPPORTED, dict(n=1 << 31)),
])
def test_rotate_refusals(capi, why, rc, kw):
    r = rot(capi, **kw.get("r", {}))
    x, y = heads(capi, **kw.get("x", {})), heads(capi, **kw.get("y", {}))
    args = (ctypes.byref(r), ctypes.byref(x), ctypes.byref(y), kw.get("dtype", 0), kw.get("n", 4), kw.get("h", 8),
            kw.get("d", 128), kw.get("pos", 16), kw.get("inverse", 0), None)
    assert capi.lib().csa2_rotate(*args) == rc, why


def test_rotate_nothing_to_do(capi):
    r, x = rot(capi), heads(capi, p=None)
    assert capi.lib().csa2_rotate(ctypes.byref(r), ctypes.byref(x), ctypes.byref(x), 0, 0, 1, 128, None, 0, None) == OK
    assert capi.lib().csa2_rotate(None, ctypes.byref(x), ctypes.byref(x), 0, 0, 1, 128, None, 0, None) == INVALID


CACHES = [("pools", INVALID, dict(k_pages=None)), ("status", INVALID, dict(status=None)), ("batch", INVALID, dict(batch=0)),
          ("pages", INVALID, dict(max_pages=0)), ("heads", INVALID, dict(kv_heads=0)), ("dtype", INVALID, dict(dtype=3)),
          ("dim", UNSUPPORTED, dict(head_dim=96)), ("batch", UNSUPPORTED, dict(batch=1025)),
          ("capacity", UNSUPPORTED, dict(max_pages=1 << 25)), ("rows", UNSUPPORTED, dict(num_pages=1 << 24, kv_heads=2)),
          ("table", ALIGN, dict(page_table=52))]


@pytest.mark.parametrize("why,rc,kw", [(w, r, dict(c=c)) for w, r, c in CACHES] + [
    ("fp16 into bf16", INVALID, dict(dtype=2)), ("fp32", INVALID, dict(dtype=1)), ("total", INVALID, dict(total=-1)),
    ("max_new", INVALID, dict(max_new=-1)), ("cu", INVALID, dict(cu=None)), ("cu", ALIGN, dict(cu=20)),
    ("start", ALIGN, dict(start=20)), ("start meets n_tokens", INVALID, dict(start=48, c=dict(n_tokens=64, page_table=160, batch=5))),
    ("k", INVALID, dict(k=dict(p=None))), ("k", ALIGN, dict(k=dict(hs=132))), ("positions without a rotation", INVALID, dict(pos=16)),
    ("rotation", INVALID, dict(r=dict(rot_offset=72))), ("total", UNSUPPORTED, dict(total=(1 << 30) + 1)),
])
def test_append_refusals(capi, why, rc, kw):
    c, k = cache(capi, **kw.get("c", {})), heads(capi, **kw.get("k", {}))
    r = rot(capi, **kw["r"]) if "r" in kw else None
    args = (ctypes.byref(c), ctypes.byref(k), ctypes.byref(k), kw.get("dtype", 0), kw.get("cu", 16), kw.get("total", 4),
            kw.get("max_new", 4), kw.get("start"), ctypes.byref(r) if r else None, kw.get("pos"), None)
    assert capi.lib().csa2_kv_append(*args) == rc, why


@pytest.mark.parametrize("why,rc,kw", [(w, r, dict(c=c)) for w, r, c in CACHES] + [
    ("fp16 over bf16", INVALID, dict(dtype=2)), ("fp32", INVALID, dict(dtype=1)), ("heads", INVALID, dict(H=7)),
    ("heads", INVALID, dict(H=0)), ("heads", INVALID, dict(H=130)), ("scale", INVALID, dict(scale=0.0)),
    ("scale", INVALID, dict(scale=float("nan"))), ("scale", INVALID, dict(scale=float("inf"))), ("window", INVALID, dict(window=-1)),
    ("out is q", INVALID, dict(o=dict(p=64))), ("out rows meet", INVALID, dict(o=dict(p=128, ts=64))), ("cu", INVALID, dict(cu=None)),
    ("lse", ALIGN, dict(lse=20)), ("ws", ALIGN, dict(ws=20)), ("q", ALIGN, dict(q=dict(p=72))), ("q", INVALID, dict(q=dict(p=None))),
    ("total", UNSUPPORTED, dict(total=(1 << 30) + 1)),
])
def test_attn_refusals(capi, why, rc, kw):
    c, q, o = cache(capi, **kw.get("c", {})), heads(capi, **kw.get("q", {})), heads(capi, **{"p": 1 << 20, **kw.get("o", {})})
    args = (ctypes.byref(c), ctypes.byref(q), kw.get("H", 8), kw.get("dtype", 0), kw.get("cu", 16), kw.get("total", 4),
            kw.get("max_new", 4), kw.get("scale", 0.1), kw.get("window", 0), ctypes.byref(o), kw.get("lse"), kw.get("ws", 16), 0, None)
    assert capi.lib().csa2_kv_attn(*args) == rc, why


def test_injected_fault_comes_after_the_checks(capi, monkeypatch):
    monkeypatch.setenv("CSA2_INJECT_FAULT", "csa2_rotate,csa2_kv_append")
    r, x, c = rot(capi), heads(capi), cache(capi)
    assert capi.lib().csa2_rotate(ctypes.byref(r), ctypes.byref(x), ctypes.byref(x), 0, 4, 8, 128, 16, 0, None) == CUDA
    assert capi.lib().csa2_rotate(ctypes.byref(r), ctypes.byref(x), ctypes.byref(x), 9, 4, 8, 128, 16, 0, None) == INVALID
    assert capi.lib().csa2_kv_append(ctypes.byref(c), ctypes.byref(x), ctypes.byref(x), 0, 16, 4, 4, None, None, None, None) == CUDA


def test_binding_refuses_host_tensors(capi):
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        capi.rotary(torch.ones(32), 64)
    with pytest.raises(ValueError):
        capi.rotate(rot(capi), t, torch.zeros(1, 4, dtype=torch.int32), t)
    with pytest.raises(ValueError):
        capi.kv_cache(torch.zeros(3, 2, 64, 64).half(), torch.zeros(3, 2, 64, 64).half(), torch.zeros(1, 2).int(),
                      torch.zeros(1).int(), torch.zeros(4).int())
    with pytest.raises(ValueError):
        capi.kv_attn(cache(capi), t.half(), torch.zeros(3).int(), 1, 0.1, t.half(), None)


def test_oracle_rotation_keeps_relative_positions():
    rng = np.random.default_rng(0)
    f = 10000.0 ** (-np.arange(16) / 16.0)
    q, k = rng.normal(size=(2, 1, 1, 32))
    dots = [float((okv.rotate(q, np.array([[p + 5]]), f, 32, neighbours=n) * okv.rotate(k, np.array([[p]]), f, 32, neighbours=n)).sum())
            for n in (False, True) for p in (0, 10, 1000)]
    assert np.allclose(dots[:3], dots[0], atol=1e-12) and np.allclose(dots[3:], dots[3], atol=1e-12)
    x = rng.normal(size=(3, 2, 40))
    pos = rng.integers(0, 1000, size=(2, 3))
    y = okv.rotate(x, pos, f[:8], 16, 8, True, [0, 1] * 4)
    assert np.allclose(okv.rotate(y, pos, f[:8], 16, 8, True, [0, 1] * 4, inverse=True), x, atol=1e-14)
    assert np.array_equal(y[..., :8], x[..., :8]) and np.array_equal(y[..., 24:], x[..., 24:])
    # the second pair (channels 10, 11) turns by the second axis
    z = (x[..., 10] + 1j * x[..., 11]) * np.exp(1j * pos[1] * f[1])[:, None]
    assert np.allclose(y[..., 10] + 1j * y[..., 11], z, atol=1e-14)


def test_oracle_attention_against_a_masked_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(5, 2, 8)), rng.normal(size=(3, 8)), rng.normal(size=(3, 8))
    for window in (0, 2):
        o, lse, _ = okv.attention(q, k, v, 3, 0.3, window)
        at = np.arange(5) - 2
        j = np.arange(3)
        see = (j <= at[:, None]) & ((j > at[:, None] - window) if window else True)
        s = np.where(see[:, None], 0.3 * np.einsum("igc,jc->igj", q, k), -np.inf)
        with np.errstate(divide="ignore"):
            want = np.log(np.exp(s).sum(-1))
        assert np.allclose(lse, want)
        p = np.exp(s - np.where(np.isinf(want), 0, want)[..., None])
        assert np.allclose(o, p @ v)
