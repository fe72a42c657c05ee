"""The page calls at their limits (GPU): pools that run out, waits that run
out, and sizes on both sides of each rule that picks a kernel."""
import numpy as np
import pytest

import pages_util as PU
from test_gpu_pages import do_compact, do_fork, do_reserve, i32, parts_of, random_cache, status

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("bit_quantized_weight_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield
    assert q.qg_last_device_status() == q.QG_OK


# ------------------------------------------------------------------ pools that run out
@pytest.mark.parametrize("pool", [3, 20000])
def test_a_reserve_that_finds_too_few_pages_is_heard_of(pool):
    """By n_free, or by the status word where there is none; in a replayed graph too."""
    P = PU.Pages(4, 8, pool, 16)
    P.refs[3:] = 1
    rec, moves, left, new = P.device(torch, q), q.KVMoves.empty(4), i32([7]), i32(np.ones(4))
    q.kv_pages_reserve(rec, new, moves)
    status(True)
    q.kv_pages_reserve(rec, new, moves, n_free=left)
    status(False)
    assert int(left) == -1 and int(moves.count) == 0
    P.same(rec)
    g, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=stream):
        q.kv_pages_reserve(rec, new, moves)
    g.replay()
    status(True)
    P.same(rec)
    new[3] = 0                                               # three pages suffice
    g.replay()
    status(False)
    P.reserve([1, 1, 1, 0])
    P.same(rec)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_what_is_appended_without_a_page_is_left_out_and_recorded(fmt):
    """Three of four rows write a token each; the fourth has no page, and then none has one for its next page."""
    r = np.random.default_rng(41)
    rec, moves, left = q.KVPages.empty(4, 3, 3, 16), q.KVMoves.empty(4), i32([7])
    cache = random_cache(r, fmt, 3, 16, 2, 64)
    batch = q.KVBatch(rec.page_table, rec.seq_lens, i32(np.arange(5)), 4)
    x = torch.randn((4, 2, 64), device="cuda").bfloat16()
    before = [t.clone() for t in parts_of(cache)]
    q.kv_pages_reserve(rec, i32(np.ones(4)), moves, n_free=left)
    assert int(left) == -1
    q.kv_cache_append(cache, batch, x, x)                    # against the rule: no row has a page
    status(True)
    assert all(torch.equal(a, b) for a, b in zip(parts_of(cache), before))
    q.kv_pages_reserve(rec, i32([16, 16, 16, 0]), moves, n_free=left)
    assert int(left) == 0
    q.kv_cache_append(cache, batch, x, x)                    # the fourth row has none
    status(True)
    rec.seq_lens.add_(torch.tensor([16, 16, 16, 0], dtype=torch.int32, device="cuda"))
    before = [t.clone() for t in parts_of(cache)]
    q.kv_pages_reserve(rec, i32([1, 1, 1, 0]), moves, n_free=left)
    assert int(left) == -3
    q.kv_cache_append(cache, batch, x, x)                    # nor have the others for their 17th token
    status(True)
    assert all(torch.equal(a, b) for a, b in zip(parts_of(cache), before))


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("fmt,page,moves,tokens", [("bf16", 64, 5, 64), ("fp8", 256, 700, 256), ("fp8", 256, 40, 200), ("nvfp4", 64, 1, 64)])
def test_a_copy_whose_wait_runs_out_reports_it_and_the_next_is_clean(fmt, page, moves, tokens):
    """Whole pages and long runs of part-filled ones, a stage of the ring and many."""
    r = np.random.default_rng(42)
    c = random_cache(r, fmt, 2 * moves, page, 4, 128)
    ids = r.permutation(2 * moves)
    lst = q.KVMoves(i32(np.stack([ids[:moves], ids[moves:], np.full(moves, tokens), np.zeros(moves, int)], 1)), i32([moves]))
    want = [t.clone() for t in parts_of(c)]
    src, dst = (torch.from_numpy(x).cuda() for x in (ids[:moves], ids[moves:]))
    for w in want:
        w[dst, :, :tokens] = w[src, :, :tokens]
    q.qg_debug_set_wait(20_000_000, True)
    try:
        q.kv_pages_copy(c, lst)
        assert q.qg_last_device_status() == q.QG_ERR_DEVICE_TIMEOUT
    finally:
        q.qg_debug_set_wait(0, False)
    q.kv_pages_copy(c, lst)
    status(False)
    assert all(torch.equal(a, b) for a, b in zip(parts_of(c), want))


# ------------------------------------------------------------------ the kernels' borders
@pytest.mark.parametrize("rows,wide", [(1, 64), (1, 65), (1, 512), (1, 513), (8, 65), (8, 128), (8, 129), (8, 257), (15, 300), (16, 65), (16, 511), (16, 512),
                                       (16, 513), (17, 65), (17, 512)])
def test_fork_at_the_border_of_the_kernel_for_few_rows(rows, wide):
    """Rows of every length up to the whole width that change places: a block
    that read a length after it was replaced would keep, drop or count columns
    of another row. Shared and lone pages; rows that end, and parents and
    entries that do not exist."""
    r = np.random.default_rng(rows * 1000 + wide)
    P = PU.Pages(rows, wide, rows * wide + 9, 16)

    def fill():
        order = list(r.permutation(P.pool))
        P.refs[:] = 0
        for b in range(rows):
            k = wide if b == rows - 1 else int(r.integers(0, wide + 1))
            share = min(k, int(P.held[b - 1]), int(r.integers(0, wide + 1))) if b else 0
            P.table[b] = -7
            P.table[b, :share] = P.table[b - 1, :share]
            P.table[b, share:k] = [order.pop() for _ in range(k - share)]
            P.held[b] = k
            P.lens[b] = max(0, k * 16 - int(r.integers(0, 40)))
            for e in P.table[b, :k]:
                P.refs[e] += 1
        return P.device(torch, q)

    for parent in (np.arange(rows)[::-1], np.roll(np.arange(rows), 1), r.permutation(rows), r.integers(0, rows, rows), r.integers(-1, rows, rows),
                   np.full(rows, -1), np.full(rows, rows - 1), r.choice([-2, rows, 2 ** 31 - 1, 0], rows)):
        rec = fill()
        do_fork(P, rec, parent.astype(np.int32))
        do_fork(P, rec, r.integers(0, rows, rows).astype(np.int32))
        assert (P.counts() == P.refs).all()
    fill()
    for e in P.table[0, :P.held[0]]:
        P.refs[e] -= 1
    P.table[0, :P.held[0]] = r.choice([-1, P.pool, -2 ** 31], P.held[0])      # entries outside the pool
    P.lens[rows // 2] = 2 ** 30 + 1                          # and a row that does not fit
    rec = P.device(torch, q)
    do_fork(P, rec, np.roll(np.arange(rows), 1).astype(np.int32))


@pytest.mark.parametrize("pool", [16383, 16384, 16385])
def test_pools_at_the_border_between_one_block_and_a_cluster(pool):
    r = np.random.default_rng(pool)
    P = PU.random_pages(r, 40, 300, pool, 16, fill=0.5)
    P.refs[[0, pool - 1]] += 1
    rec = P.device(torch, q)
    do_reserve(P, rec, r.choice([0, 1, 17, 160], 40))
    do_fork(P, rec, r.integers(-1, 40, 40).astype(np.int32))
    do_reserve(P, rec, r.integers(0, 3, 40))
    do_compact(P, rec, 100)
    do_compact(P, rec, pool)
    free = int((P.refs == 0).sum())
    P.refs[P.refs == 0] = 1                                  # none is left, and then the last one
    rec = P.device(torch, q)
    do_reserve(P, rec, np.full(40, 40))
    assert free > 1
    P.refs[pool - 1] = 0
    one = np.zeros(40, int)
    one[int(np.argmin(P.held))] = int(P.held.min() * 16 - P.lens[np.argmin(P.held)]) + 1
    rec = P.device(torch, q)
    do_reserve(P, rec, one)
    do_reserve(P, rec, one)
