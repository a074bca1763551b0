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
