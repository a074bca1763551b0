"""Numbers that the Python calls of the paged key/value operators refuse (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

import fp4_sparse_attention_pack_b200 as csa


@pytest.mark.parametrize("what,kw", [("axis", dict(n_axes=3, axis=[0] * 15 + [256])), ("axis", dict(n_axes=3, axis=[-255] + [0] * 15)),
                                     ("axis", dict(axis=[1] * 16)), ("offset", dict(offset=1 << 32)), ("n_axes", dict(n_axes=(1 << 32) + 1))])
def test_rotary_refuses_numbers_that_it_would_cut(what, kw):
    with pytest.raises(ValueError, match=what):
        csa.rotary(torch.ones(16), 32, **kw)


@pytest.mark.parametrize("sizes", [((1 << 32) + 4, 4, 8), (4, (1 << 32) + 4, 8), (4, 4, (1 << 32) + 8)])
def test_workspace_refuses_numbers_that_it_would_cut(sizes):
    c = csa.csa2_kv_cache(16, 32, 48, 64, 80, 2, 4, 9, 2, 128, 0)
    with pytest.raises(ValueError):
        csa.kv_attn_workspace(c, *sizes)
