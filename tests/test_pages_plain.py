"""The plain forms of the page calls and of beam search's selection, pinned by
hand-worked cases, and the refusals of their entry points (no GPU)."""
import ctypes

import numpy as np
import pytest

import pages_util as PU
from test_abi import A, L, fake_ptr  # noqa: F401  (L is a fixture)
from test_kv_plain import cache


# ------------------------------------------------------------------ plain forms
def three_rows():
    """Pages of 16: row 0 has 20 tokens on 4, 2; row 1 shares page 4 and has 33 on 4, 7, 1; row 2 has none."""
    P = PU.Pages(3, 4, 10, 16)
    P.table[0, :2], P.table[1, :3] = [4, 2], [4, 7, 1]
    P.lens[:2], P.held[:2] = [20, 33], [2, 3]
    P.refs[[4, 2, 7, 1]] = [2, 1, 1, 1]
    return P


def test_fork_by_hand():
    P = three_rows()
    assert P.fork([1, 1, 0]) is False
    assert P.lens.tolist() == [33, 33, 20] and P.held.tolist() == [3, 3, 2]
    assert P.table[0, :3].tolist() == P.table[1, :3].tolist() == [4, 7, 1] and P.table[2, :2].tolist() == [4, 2]
    assert P.refs.tolist() == [0, 2, 1, 0, 3, 0, 0, 2, 0, 0]
    assert P.fork([-1, -1, -1]) is False and not P.refs.any() and not P.held.any()
    assert three_rows().fork([0, 3, 0]) is True


def test_reserve_by_hand():
    P = three_rows()
    P.fork([0, 0, 1])                                        # page 2 (4 tokens) is shared by rows 0 and 1
    moves, left, bad = P.reserve([1, 13, 0])                 # both write it: row 0 keeps it, row 1 gets 0 and then 3
    assert not bad and moves == [(2, 0, 4, 0)] and left == 4      # free: 5 6 8 9
    assert P.table[0, :2].tolist() == [4, 2] and P.table[1, :3].tolist() == [4, 0, 3] and P.held.tolist() == [2, 3, 3]
    assert P.refs.tolist() == [1, 1, 1, 1, 3, 0, 0, 1, 0, 0]
    P.refs[5] = 1                                            # and one that a holder outside the table takes
    before = P.table.copy(), P.refs.copy(), P.held.copy()
    assert P.reserve([44, 44, 31]) == ([], -1, False)        # two, one and one more: nothing changes
    assert all(np.array_equal(a, b) for a, b in zip(before, (P.table, P.refs, P.held)))
    assert P.reserve([44, 44, 0]) == ([], 0, False) and P.held.tolist() == [4, 4, 3]


def test_compact_by_hand():
    P = three_rows()
    moves, where, live, bad = P.compact(10)                  # in use: 1 2 4 7; holes below 4: 0 3; 7 -> 0, 4 -> 3
    assert not bad and live == 4 and moves == [(7, 0, 16, 0), (4, 3, 16, 0)]
    assert where.tolist() == [-1, 1, 2, -1, 3, -1, -1, 0, -1, -1]
    assert P.table[0, :2].tolist() == [3, 2] and P.table[1, :3].tolist() == [3, 0, 1]
    assert P.refs.tolist() == [1, 1, 1, 2, 0, 0, 0, 0, 0, 0]


def test_selection_by_hand():
    """Two beams with the scores 0 and ln(1/2): candidates 1/4, 1/4, 1/2 and (1/2) (1/8, 3/4, 1/8)."""
    x = np.log(np.array([[1.0, 1, 2], [1, 6, 1]]))
    scores = np.log(np.array([[1.0, 0.5]]))
    f = lambda v: np.log(np.array([v]))
    good = (f([0.5, 0.375, 0.25, 0.25]), [[2, 1, 0, 1]], [[0, 1, 0, 0]], [[0, 1, 0, 1]])
    PU.check_selection(x, scores, None, 1, 0, [np.array(t) for t in good], 4)
    for i, wrong in ((0, f([0.5, 0.375, 0.25, 0.26])), (1, [[2, 1, 1, 0]]), (2, [[0, 0, 0, 0]]), (3, [[0, 0, 0, 1]])):
        got = [np.array(t) for t in good]
        got[i] = np.array(wrong)
        with pytest.raises(AssertionError):
            PU.check_selection(x, scores, None, 1, 0, got, 4)


# ------------------------------------------------------------------ refusals
def pages(**kw):
    from bit_quantized_weight_gb300 import QgKvPages
    f = dict(page_table=A, seq_lens=A, n_pages=A, refs=A, n_seqs=2, max_pages=2, num_pages=4, page_size=16)
    f.update(kw)
    return QgKvPages(**f)


def moves(**kw):
    from bit_quantized_weight_gb300 import QgKvMoves
    f = dict(list=A, count=A, capacity=4)
    f.update(kw)
    return QgKvMoves(**f)


def page_calls(L, p, m):
    p, m = ctypes.byref(p), ctypes.byref(m)
    return [L.kv_pages_fork(p, A, None), L.kv_pages_reserve(p, A, m, A, None), L.kv_pages_compact(p, m, A, A, None)]


@pytest.mark.parametrize("kw,want", [
    (dict(n_seqs=-1), 1), (dict(n_seqs=1025), 1), (dict(max_pages=0), 1), (dict(num_pages=0), 1), (dict(page_size=8), 1),
    (dict(page_size=24), 1), (dict(page_size=2048), 1), (dict(num_pages=(1 << 22) + 1), 2), (dict(page_table=None), 1),
    (dict(seq_lens=None), 1), (dict(n_pages=None), 1), (dict(refs=None), 1), (dict(page_table=A + 4), 3),
    (dict(seq_lens=A + 8), 3), (dict(n_pages=A + 4), 3), (dict(refs=A + 12), 3),
])
@fake_ptr
def test_every_call_rejects_a_bad_record(L, kw, want):
    assert page_calls(L, pages(**kw), moves()) == [want] * 3


@pytest.mark.parametrize("kw,want", [
    (dict(list=None), 1), (dict(count=None), 1), (dict(capacity=0), 1), (dict(capacity=(1 << 22) + 1), 1),
    (dict(list=A + 8), 3), (dict(count=A + 4), 3),
])
@fake_ptr
def test_every_call_rejects_a_bad_list(L, kw, want):
    assert page_calls(L, pages(), moves(**kw))[1:] == [want] * 2
    assert L.kv_pages_copy(ctypes.byref(cache()), ctypes.byref(moves(**kw)), None) == want


@fake_ptr
def test_page_call_arguments(L):
    p, m, c = ctypes.byref(pages()), ctypes.byref(moves()), ctypes.byref(cache())
    assert L.kv_pages_fork(None, A, None) == 1 and L.kv_pages_fork(p, None, None) == 1
    assert L.kv_pages_fork(p, A + 4, None) == 3
    assert L.kv_pages_fork(ctypes.byref(pages(n_seqs=0, page_table=None, seq_lens=None, n_pages=None)), None, None) == 0
    assert L.kv_pages_reserve(None, A, m, A, None) == 1 and L.kv_pages_reserve(p, None, m, A, None) == 1
    assert L.kv_pages_reserve(p, A, None, A, None) == 1
    assert L.kv_pages_reserve(p, A, ctypes.byref(moves(capacity=1)), A, None) == 1        # fewer than sequences
    assert L.kv_pages_reserve(p, A + 4, m, A, None) == 3 and L.kv_pages_reserve(p, A, m, A + 4, None) == 3
    assert L.kv_pages_compact(None, m, A, A, None) == 1 and L.kv_pages_compact(p, None, A, A, None) == 1
    assert L.kv_pages_compact(p, m, None, A, None) == 1
    assert L.kv_pages_compact(p, m, A + 4, A, None) == 3 and L.kv_pages_compact(p, m, A, A + 4, None) == 3
    assert L.kv_pages_copy(None, m, None) == 1 and L.kv_pages_copy(c, None, None) == 1


@pytest.mark.parametrize("kw,want", [
    (dict(format=3), 1), (dict(num_pages=0), 1), (dict(page_size=24), 1), (dict(kv_heads=0), 1), (dict(head_dim=96), 2),
    (dict(k=None), 1), (dict(v_scales=None), 1), (dict(k=A + 8), 3), (dict(v=A + 4), 3), (dict(k_scales=A + 4), 3),
    (dict(k_gscale=0.0), 1), (dict(v_gscale=float("nan")), 1),
])
@fake_ptr
def test_copy_rejects_a_bad_cache(L, kw, want):
    assert L.kv_pages_copy(ctypes.byref(cache(**kw)), ctypes.byref(moves()), None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(lanes=-1), 1), (dict(beams=0), 1), (dict(beams=65), 1), (dict(lanes=8193), 1), (dict(vocab=0), 1),
    (dict(vocab=(1 << 24) + 1, stride=1 << 25), 1), (dict(n_out=0), 1), (dict(n_out=65), 1), (dict(dtype=2), 1),
    (dict(dtype=-1), 1), (dict(stride=999), 1), (dict(stride=(1 << 40) + 1), 1), (dict(eos=-2), 1), (dict(eos=1000), 1),
    (dict(pad=-1), 1), (dict(pad=1000), 1), (dict(logits=None), 1), (dict(scores=None), 1), (dict(out_scores=None), 1),
    (dict(out_tokens=None), 1), (dict(out_parents=None), 1), (dict(logits=A + 8), 3), (dict(scores=A + 4), 3),
    (dict(finished=A + 1), 3), (dict(out_scores=A + 4), 3), (dict(out_tokens=A + 8), 3), (dict(out_parents=A + 4), 3),
    (dict(out_finished=A + 2), 3), (dict(workspace=None), 4), (dict(nbytes=64), 4), (dict(workspace=A + 16), 3),
    (dict(out_scores=0x300000, n_out=9), 1), (dict(out_finished=0x400000, n_out=9), 1), (dict(lanes=0, logits=None), 0),
])
@fake_ptr
def test_beam_select_arguments(L, kw, want):
    a = dict(logits=A, dtype=0, stride=1000, lanes=2, beams=8, vocab=1000, scores=0x300000, finished=0x400000, eos=-1, pad=0,
             n_out=8, out_scores=A, out_tokens=A, out_parents=A, out_finished=A, workspace=A, nbytes=1 << 30)
    a.update(kw)
    assert L.beam_select(a["logits"], a["dtype"], a["stride"], a["lanes"], a["beams"], a["vocab"], a["scores"], a["finished"],
                         a["eos"], a["pad"], a["n_out"], a["out_scores"], a["out_tokens"], a["out_parents"],
                         a["out_finished"], a["workspace"], a["nbytes"], None) == want


@fake_ptr
def test_beam_workspace_sizes(L):
    n = ctypes.c_size_t(0)
    for args in ((-1, 8, 1000, 8), (1, 0, 1000, 8), (1, 65, 1000, 8), (2000, 64, 1000, 8), (1, 8, 0, 8), (1, 8, 1000, 65)):
        assert L.beam_select_workspace_size(*args, ctypes.byref(n)) == 1
    assert L.beam_select_workspace_size(1, 8, 1000, 8, None) == 1
    assert L.beam_select_workspace_size(0, 8, 1000, 8, ctypes.byref(n)) == 0
    assert L.beam_select_workspace_size(1024, 64, 1 << 24, 64, ctypes.byref(n)) == 0 and n.value > 1 << 32


def test_records_refuse_tensors_of_the_host():
    torch = pytest.importorskip("torch")
    import bit_quantized_weight_gb300 as q
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        q.KVPages(torch.zeros((4, 2), dtype=torch.int32), i, i, i, 16)
    with pytest.raises(ValueError):
        q.KVMoves(torch.zeros((4, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    x, s, t = torch.zeros((4, 9)), torch.zeros((1, 4)), torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        q.beam_select(x, s, s.clone(), t, t.clone())
