"""Sizes that one route of tree_attention does not serve are refused on the host (no GPU)."""
import ctypes

import pytest

from test_abi import A, L, fake_ptr  # noqa: F401  (L is a fixture)
from test_kv_plain import batch, cache

PAGES = 1 << 20                                   # with 2 heads and pages of 1,024 tokens 2^31 rows


@pytest.mark.parametrize("kw,heads,tree,want", [
    (dict(), 8, 9, 2), (dict(head_dim=64), 8, 9, 2), (dict(num_pages=PAGES + 7), 2, 64, 2),
    # one page less, fewer query rows, other formats and head_dim 256: on to the workspace, which is missing here
    (dict(num_pages=PAGES - 1), 8, 9, 4), (dict(), 8, 8, 4), (dict(head_dim=256), 8, 9, 4),
    (dict(format=1, k_scales=A, v_scales=A), 8, 9, 4), (dict(format=2, k_scales=A, v_scales=A), 8, 9, 4),
])
@fake_ptr
def test_rows_beyond_a_tma_coordinate(L, kw, heads, tree, want):
    f = dict(format=0, num_pages=PAGES, page_size=1024, kv_heads=2, k_scales=None, v_scales=None)
    c, b = cache(**{**f, **kw}), batch()
    args = (A, heads * 256, heads, tree, A, 1.0, A, None, None, 0, None)
    assert L.tree_attention(ctypes.byref(c), ctypes.byref(b), *args) == want
