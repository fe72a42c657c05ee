"""The plain 64-bit cache forms that the GPU tests compare with, pinned by
hand-worked values and library conversions, and the refusals of the cache and
attention entry points (no GPU)."""
import ctypes

import numpy as np
import pytest

import kv_util as U
import oracle as O
from test_abi import A, L, fake_ptr  # noqa: F401  (L is a fixture)


def test_e4m3_table_matches_the_oracle():
    ref = O.e4m3_array(np.arange(128, dtype=np.uint8))
    assert np.array_equal(U.E4M3, ref, equal_nan=True)


def test_fp8_by_hand():
    # max 3.5 = 448 * 2^-7: s = -7 + 15; 3.5 -> 448 (code 0x7E), -0.875 -> -112 (0xEE), a tie below
    x = np.zeros(64)
    x[:4] = [3.5, -0.875, 3.5 * 0.75, 0.0]         # 336 lies between 320 (0x7A) and 352 (0x7B): the even code
    codes, s = U.quantise(x[None], "fp8", 1.0)
    assert s[0] == 8 and list(codes[0, :4]) == [0x7E, 0xEE, 0x7A, 0x00]
    x[0] = 3.515625                                 # the next bf16 above: one step up
    assert U.quantise(x[None], "fp8", 1.0)[1][0] == 9
    assert U.quantise(np.zeros((1, 64)), "fp8", 1.0)[1][0] == 1
    assert U.quantise(np.full((1, 64), 1e30), "fp8", 1.0)[1][0] == 22
    got = U.values(codes, s, "fp8", 2.0)
    assert list(got[0, :4]) == [7.0, -1.75, 5.0, 0.0]


def test_nvfp4_by_hand():
    x = np.zeros(64)
    x[:6] = [6.0, 0.25, 0.75, 2.5, -5.0, -0.3]     # scale 1: ties to 0, 1.0, 2.0, -4.0
    codes, s = U.quantise(x[None], "nvfp4", 1.0)
    assert s.shape == (1, 4) and list(s[0]) == [0x38, 0, 0, 0]
    assert list(codes[0, :3]) == [7 | 0 << 4, 2 | 4 << 4, 14 | 9 << 4]
    assert list(U.values(codes, s, "nvfp4", 1.0)[0, :6]) == [6.0, 0.0, 1.0, 2.0, -4.0, -0.5]
    x[3] = np.nan
    assert U.quantise(x[None], "nvfp4", 1.0)[1][0, 0] == 0x7F


def test_codes_match_library_conversions():
    torch = pytest.importorskip("torch")
    r = np.random.default_rng(0)
    x = O.round_bf16(r.standard_normal((200, 64)) * 10 ** r.uniform(-3, 3, (200, 1)))
    codes, s = U.quantise(x, "fp8", 1.0)
    y = torch.from_numpy(x * 2.0 ** (15.0 - s)[:, None]).float().clamp(-448, 448).to(torch.float8_e4m3fn)
    assert np.array_equal(y.view(torch.uint8).numpy(), codes)


def test_attention_of_one_key_is_its_value():
    q, k, v = np.ones((2, 2, 64)), np.ones((3, 1, 64)), np.arange(3 * 64.0).reshape(3, 1, 64)
    seen = np.array([[True, False, False], [False, False, False]])
    out, lse, _, _ = U.attention(q, k, v, seen, 0.5)
    assert np.array_equal(out[0, 0], v[0, 0]) and lse[0, 0] == 32.0
    assert not out[1].any() and np.all(lse[1] == -np.inf)


# ------------------------------------------------------------------ refusals
def cache(**kw):
    from bit_quantized_weight_gb300 import QgKvCache
    f = dict(format=1, num_pages=4, page_size=16, kv_heads=2, head_dim=128, k=A, v=A, k_scales=A, v_scales=A,
             k_gscale=1.0, v_gscale=1.0)
    f.update(kw)
    return QgKvCache(**f)


def batch(**kw):
    from bit_quantized_weight_gb300 import QgKvBatch
    f = dict(page_table=A, seq_lens=A, token_start=A, n_seqs=2, max_pages=2, n_tokens=4)
    f.update(kw)
    return QgKvBatch(**f)


def calls(L, c, b):
    c, b = ctypes.byref(c), ctypes.byref(b)
    return [L.kv_cache_append(c, b, A, 256, A, 256, None), L.kv_cache_read(c, b, A, A, 0, None),
            L.kv_cache_accept(c, b, A, A, A, None),
            L.tree_attention(c, b, A, 512, 4, 4, A, 1.0, A, None, A, 1 << 30, None)]


@pytest.mark.parametrize("kw,want", [
    (dict(format=3), 1), (dict(format=-1), 1), (dict(num_pages=0), 1), (dict(page_size=8), 1),
    (dict(page_size=24), 1), (dict(page_size=2048), 1), (dict(kv_heads=0), 1), (dict(kv_heads=1025), 1),
    (dict(head_dim=0), 1), (dict(head_dim=96), 2), (dict(head_dim=512), 2), (dict(k=None), 1),
    (dict(v=None), 1), (dict(k_scales=None), 1), (dict(v_scales=None), 1), (dict(format=0), 1),
    (dict(k=A + 8), 3), (dict(v_scales=A + 4), 3), (dict(k_gscale=0.0), 1), (dict(v_gscale=-1.0), 1),
    (dict(k_gscale=float("inf")), 1), (dict(v_gscale=float("nan")), 1),
])
@fake_ptr
def test_every_call_rejects_a_bad_cache(L, kw, want):
    assert calls(L, cache(**kw), batch()) == [want] * 4


@pytest.mark.parametrize("kw,want", [
    (dict(n_seqs=-1), 1), (dict(n_seqs=1025), 1), (dict(max_pages=0), 1), (dict(n_tokens=-1), 1),
    (dict(n_tokens=(1 << 24) + 1), 1), (dict(page_table=None), 1), (dict(seq_lens=None), 1),
    (dict(token_start=None), 1), (dict(page_table=A + 4), 3), (dict(seq_lens=A + 4), 3),
    (dict(token_start=A + 8), 3),
])
@fake_ptr
def test_every_call_rejects_a_bad_batch(L, kw, want):
    assert calls(L, cache(), batch(**kw)) == [want] * 4


@fake_ptr
def test_calls_without_rows_do_nothing(L):
    b = batch(page_table=None, seq_lens=None, token_start=None, n_seqs=0, n_tokens=0)
    assert calls(L, cache(), b) == [0] * 4
    c, b = ctypes.byref(cache()), ctypes.byref(batch(n_tokens=0))
    assert L.kv_cache_append(c, b, None, 0, None, 0, None) == 0
    assert L.tree_attention(c, b, None, 0, 4, 4, None, 1.0, None, None, None, 0, None) == 0


@fake_ptr
def test_append_and_read_arguments(L):
    c, b = ctypes.byref(cache()), ctypes.byref(batch())
    assert L.kv_cache_append(None, b, A, 256, A, 256, None) == 1
    assert L.kv_cache_append(c, None, A, 256, A, 256, None) == 1
    assert L.kv_cache_append(c, b, None, 256, A, 256, None) == 1
    assert L.kv_cache_append(c, b, A, 255, A, 256, None) == 1
    assert L.kv_cache_append(c, b, A, 260, A, 256, None) == 3
    assert L.kv_cache_append(c, b, A, 256, A + 2, 256, None) == 3
    assert L.kv_cache_read(c, b, A, None, 0, None) == 1
    assert L.kv_cache_read(c, b, A, A, 2, None) == 1
    assert L.kv_cache_read(c, b, A + 4, A, 1, None) == 3
    assert L.kv_cache_accept(c, b, None, A, A, None) == 1
    assert L.kv_cache_accept(c, b, A, None, A, None) == 1
    assert L.kv_cache_accept(c, b, A, A, A + 4, None) == 3


@fake_ptr
def test_tree_attention_arguments(L):
    c, b = ctypes.byref(cache()), ctypes.byref(batch())
    ok = dict(q=A, qs=512, heads=4, tree=4, mask=A, scale=1.0, out=A, lse=A, ws=A, n=1 << 30)

    def call(**kw):
        a = {**ok, **kw}
        return L.tree_attention(c, b, a["q"], a["qs"], a["heads"], a["tree"], a["mask"], a["scale"], a["out"],
                                a["lse"], a["ws"], a["n"], None)

    for kw, want in [(dict(q=None), 1), (dict(out=None), 1), (dict(heads=3), 1), (dict(heads=0), 1),
                     (dict(heads=2 * 129), 1), (dict(tree=0), 1), (dict(tree=65), 1), (dict(qs=504), 1),
                     (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(qs=516), 3),
                     (dict(q=A + 2), 3), (dict(out=A + 8), 3), (dict(mask=A + 8), 3), (dict(lse=A + 4), 3),
                     (dict(ws=None), 4), (dict(n=0), 4), (dict(ws=A + 16), 3)]:
        assert call(**kw) == want, kw
    n = ctypes.c_size_t(0)
    assert L.tree_attention_workspace_size(c, 4, 4, ctypes.byref(n)) == 0 and n.value > 0
    assert L.tree_attention_workspace_size(c, 4, 65, ctypes.byref(n)) == 1
    assert L.tree_attention_workspace_size(c, 5, 4, ctypes.byref(n)) == 1
    assert L.tree_attention_workspace_size(c, 4, 4, None) == 1
    bad = cache(head_dim=80)
    assert L.tree_attention_workspace_size(ctypes.byref(bad), 4, 4, ctypes.byref(n)) == 2


def test_binding_refuses_host_tensors_and_unknown_formats():
    torch = pytest.importorskip("torch")
    import bit_quantized_weight_gb300 as q
    k = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.KVCache("bf16", k, k)
    with pytest.raises(ValueError):
        q.KVCache("int3", k, k)
    with pytest.raises(ValueError):
        q.KVBatch(torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                  torch.zeros(2, dtype=torch.int32), 1)
