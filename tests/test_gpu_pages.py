"""The page calls (GPU): fork, reserve and compact against the plain forms of
pages_util, whole numbers compared exactly; copies compared byte for byte."""
import numpy as np
import pytest

import kv_util as U
import oracle as O
import pages_util as PU
from gpu_util import guarded, to_dev

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


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def status(bad):
    assert q.qg_last_device_status() == (q.QG_ERR_INVALID_ARG if bad else q.QG_OK)


# (rows, table columns, pages of the pool, page size)
SIZES = [(1, 1, 1, 16), (1, 9, 40, 16), (8, 33, 200, 64), (3, 64, 33, 48), (17, 31, 1000, 16), (64, 130, 5000, 32),
         (200, 40, 9001, 16), (1024, 12, 20000, 16), (5, 3000, 40000, 1024)]


def do_fork(P, rec, parent):
    bad = P.fork(parent)
    q.kv_pages_fork(rec, i32(parent))
    status(bad)
    P.same(rec)


def do_reserve(P, rec, new):
    moves = q.KVMoves(torch.full((P.n + 3, 4), -5, dtype=torch.int32, device="cuda"), i32([-1]))
    left = i32([99])
    want, free, bad = P.reserve(new)
    q.kv_pages_reserve(rec, i32(new), moves, n_free=left)
    status(bad)
    P.same(rec)
    assert int(moves.count) == len(want) and int(left) == free
    got = moves.list.cpu().numpy()
    assert got[:len(want)].tolist() == [list(m) for m in want] and (got[len(want):] == -5).all()
    return moves


def do_compact(P, rec, capacity):
    moves = q.KVMoves(torch.full((capacity, 4), -5, dtype=torch.int32, device="cuda"), i32([-1]))
    where, live = torch.full((P.pool,), -9, dtype=torch.int32, device="cuda"), i32([-1])
    want, m, L, bad = P.compact(capacity)
    q.kv_pages_compact(rec, moves, where, n_live=live)
    status(bad)
    P.same(rec)
    assert int(moves.count) == len(want) and int(live) == L
    assert np.array_equal(where.cpu().numpy(), m)
    got = moves.list.cpu().numpy()
    assert got[:len(want)].tolist() == [list(x) for x in want] and (got[len(want):] == -5).all()
    return moves


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("seed", [0, 1])
def test_fork_is_the_definition(sizes, seed):
    r = np.random.default_rng(seed)
    P = PU.random_pages(r, *sizes)
    rec = P.device(torch, q)
    n = P.n
    for parent in (np.arange(n), r.permutation(n), r.integers(0, n, n), r.integers(-1, n, n), np.full(n, -1),
                   np.zeros(n)):
        do_fork(P, rec, parent.astype(np.int32))


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("seed", [0, 1])
def test_reserve_is_the_definition(sizes, seed):
    r = np.random.default_rng(seed)
    P = PU.random_pages(r, *sizes)
    rec = P.device(torch, q)
    n, page = P.n, P.page
    do_reserve(P, rec, np.ones(n))
    do_fork(P, rec, r.integers(0, n, n).astype(np.int32))
    do_reserve(P, rec, r.integers(0, 2, n))
    do_fork(P, rec, r.integers(0, n, n).astype(np.int32))
    do_reserve(P, rec, r.choice([0, 1, page - 1, page, page + 1, 3 * page], n))
    do_reserve(P, rec, r.choice([1, 2 * page], n))          # some is held ahead by now
    do_reserve(P, rec, np.full(n, max(1, (P.wide - int(P.held.max())) * page // 2)))   # and where it does not fit
    do_reserve(P, rec, np.ones(n))


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("capacity", [1, 7, 40000])
def test_compact_is_the_definition(sizes, capacity):
    r = np.random.default_rng(5)
    P = PU.random_pages(r, *sizes)
    rec = P.device(torch, q)
    do_compact(P, rec, capacity)
    do_compact(P, rec, capacity)
    do_fork(P, rec, np.where(r.random(P.n) < 0.5, -1, np.arange(P.n)).astype(np.int32))
    do_compact(P, rec, capacity)
    if capacity == 40000:
        live = int((P.refs != 0).sum())
        assert (P.refs[:live] != 0).all()


@pytest.mark.parametrize("pool", [8191, 8192, 8193, 32768, 262145, 1 << 22])
def test_large_pools(pool):
    """Few rows over a large pool, in use but for a few pages at its ends."""
    r = np.random.default_rng(6)
    P = PU.Pages(4, 8, pool, 16)
    P.refs[:] = 1
    P.refs[[3, pool // 2, pool - 70, pool - 2, pool - 1]] = 0
    rec = P.device(torch, q)
    do_reserve(P, rec, [16, 0, 33, 0])
    do_reserve(P, rec, [16, 0, 33, 100])                    # three too few: nothing changes
    P.refs[r.integers(10, pool // 3, 100)] = 0
    rec = P.device(torch, q)
    do_compact(P, rec, 64)
    do_compact(P, rec, 1000)


def test_a_shared_last_page_is_kept_by_the_lowest_where_all_write():
    P = PU.Pages(4, 4, 16, 16)
    P.table[:, 0], P.lens[:], P.held[:] = 9, 5, 1
    P.refs[9] = 4
    rec = P.device(torch, q)
    do_reserve(P, rec, [1, 1, 1, 1])
    assert P.table[:, 0].tolist() == [9, 0, 1, 2] and P.refs[9] == 1
    P.table[:, 0] = 9
    P.refs[:] = 0
    P.refs[9] = 4
    rec = P.device(torch, q)
    do_reserve(P, rec, [0, 1, 1, 1])                        # row 0 keeps reading it
    assert P.table[:, 0].tolist() == [9, 0, 1, 2]
    P.table[:, 0], P.refs[:] = 9, 0
    P.refs[9] = 5                                           # and so does a holder outside the table
    rec = P.device(torch, q)
    do_reserve(P, rec, [1, 1, 1, 1])
    assert P.table[:, 0].tolist() == [0, 1, 2, 3] and P.refs[9] == 1


def test_many_part_filled_pages_at_once():
    """1,024 rows whose last pages are shared by two, three and many rows, page numbers that collide when hashed."""
    n = 1024
    P = PU.Pages(n, 2, 1 << 15, 16)
    tail = np.where(np.arange(n) < 400, (np.arange(n) // 2) * 64, np.where(np.arange(n) < 900, 20000 + np.arange(n) // 3, 31000))
    P.table[:, 0], P.lens[:], P.held[:] = tail, 1 + np.arange(n) % 15, 1
    P.refs += np.bincount(tail, minlength=P.pool).astype(np.int32)
    rec = P.device(torch, q)
    do_reserve(P, rec, np.ones(n))
    do_reserve(P, rec, np.full(n, 16))


def test_rows_that_do_not_fit_are_left_out_and_recorded():
    def state():
        r = np.random.default_rng(8)
        P = PU.random_pages(r, 12, 20, 300, 16, fill=0.5)
        for b in range(12):                                  # all with a part-filled page of their own
            if P.held[b] == 0 or P.lens[b] % 16 == 0:
                free = int(np.nonzero(P.refs == 0)[0][-1])
                P.table[b, P.held[b]] = free
                P.refs[free] += 1
                P.held[b] += 1
                P.lens[b] = P.held[b] * 16 - 3
        return P

    for what in ("len", "long", "held", "wide", "entry", "parent", "ahead", "free"):
        P = state()
        if what == "len":
            P.lens[3] = -1
        elif what == "long":
            P.lens[3] = 2 ** 31 - 1
        elif what == "held":
            P.held[3] = -4
        elif what == "wide":
            P.held[3] = 21
        elif what == "entry":
            P.table[3, P.held[3] - 1] = 300
            P.table[5, P.held[5] - 1] = -1
        elif what == "ahead":                                # a page behind the last one's that another row has too
            P.lens[3] = max(1, (P.held[3] - 1) * 16 - 2)
            P.refs[P.table[3, P.held[3] - 1]] += 1
        elif what == "free":
            P.refs[P.table[3, P.held[3] - 1]] = 0
        rec = P.device(torch, q)
        if what in ("ahead", "free"):
            do_reserve(P, rec, np.full(12, 17))
            continue
        do_reserve(P, rec, np.ones(12))
        do_compact(P, rec, 50)
        parent = np.array([3, 1, 2, 3, 4, 5, 3, 7, 5, 9, -1, 0], np.int32)
        if what == "parent":
            parent[[2, 6]] = 12, -2
        do_fork(P, rec, parent)
    P = state()
    rec = P.device(torch, q)
    do_reserve(P, rec, [1, -1, 1, 20 * 16, 1, 2 ** 31 - 1] + [0] * 6)


def test_nothing_to_do():
    rec = q.KVPages.empty(0, 4, 100, 16)
    moves, left = q.KVMoves.empty(1), i32([7])
    q.kv_pages_fork(rec, i32([]))
    q.kv_pages_reserve(rec, i32([]), moves, n_free=left)
    assert int(left) == 100 and int(moves.count) == 0
    rec = q.KVPages.empty(3, 4, 100, 16)
    where, live = torch.zeros(100, dtype=torch.int32, device="cuda"), i32([7])
    q.kv_pages_compact(rec, q.KVMoves.empty(5), where, n_live=live)
    assert int(live) == 0 and bool((where == -1).all())
    q.kv_pages_reserve(rec, i32([0, 0, 0]), q.KVMoves.empty(3))
    q.kv_pages_copy(q.KVCache.empty("bf16", 2, 16, 1, 64), q.KVMoves.empty(3))
    assert int(rec.refs.sum()) == 0


# ------------------------------------------------------------------ copies
def random_cache(r, fmt, pages, page, heads, dim):
    c = q.KVCache.empty(fmt, pages, page, heads, dim)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        if t is not None:
            raw = torch.from_numpy(r.integers(0, 256, t.numel() * t.element_size(), dtype=np.uint8)).cuda()
            t.view(torch.uint8).view(-1).copy_(raw)
    return c


def parts_of(c):
    return [t.view(torch.int16) if t.dtype is torch.bfloat16 else t for t in (c.k, c.v, c.k_scales, c.v_scales) if t is not None]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("page,heads,dim", [(16, 1, 64), (48, 3, 64), (64, 4, 128), (64, 8, 256), (1024, 2, 128), (16, 33, 128)])
def test_copy_moves_the_tokens_and_nothing_else(fmt, page, heads, dim):
    r = np.random.default_rng(11)
    pages = 40
    c = random_cache(r, fmt, pages, page, heads, dim)
    ids = r.permutation(pages)
    n = 19
    tokens = [0, 1, 2, 3, 4, 15, 16, page - 1, page, page] + list(r.integers(0, page + 1, n - 10))
    moves = np.stack([ids[:n], ids[n:2 * n], np.minimum(tokens, page), np.zeros(n, int)], 1)
    want = [t.clone() for t in parts_of(c)]
    for src, dst, t, _ in moves.tolist():
        for w in want:
            w[dst, :, :t] = w[src, :, :t]
    lst = i32(np.concatenate([moves, np.full((4, 4), 1)]))   # entries behind the count do not matter
    q.kv_pages_copy(c, q.KVMoves(lst, i32([n])))
    status(False)
    assert all(torch.equal(a, b) for a, b in zip(parts_of(c), want))


@pytest.mark.parametrize("entry", [(-1, 2, 4), (2, 8, 4), (8, 2, 4), (2, -3, 4), (1, 2, -1), (1, 2, 17), (2 ** 31 - 1, 2, 4)])
def test_moves_that_do_not_fit_are_left_out_and_recorded(entry):
    r = np.random.default_rng(12)
    c = random_cache(r, "fp8", 8, 16, 2, 64)
    want = [t.clone() for t in parts_of(c)]
    for w in want:
        w[5, :, :7] = w[0, :, :7]
    q.kv_pages_copy(c, q.KVMoves(i32([entry + (0,), (0, 5, 7, 0)]), i32([2])))
    status(True)
    assert all(torch.equal(a, b) for a, b in zip(parts_of(c), want))
    for count in (-1, 3, 2 ** 31 - 1):
        q.kv_pages_copy(c, q.KVMoves(i32([(0, 5, 7, 0), (0, 6, 7, 0)]), i32([count])))
        status(True)
        assert all(torch.equal(a, b) for a, b in zip(parts_of(c), want))


def test_copy_beyond_32_bits():
    pages, page, heads, dim = 4200, 256, 8, 256
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("needs 12 GB of device memory")
    k = torch.zeros((pages, heads, page, dim), dtype=torch.bfloat16, device="cuda")
    k[pages - 1].normal_()
    c = q.KVCache("bf16", k, torch.zeros_like(k))
    q.kv_pages_copy(c, q.KVMoves(i32([(pages - 1, 0, page, 0), (pages - 2, 1, 9, 0)]), i32([2])))
    assert torch.equal(k[0], k[pages - 1])
    k[5].normal_()
    q.kv_pages_copy(c, q.KVMoves(i32([(5, pages - 2, 9, 0)]), i32([1])))
    assert torch.equal(k[pages - 2, :, :9], k[5, :, :9]) and float(k[pages - 2, :, 9:].abs().max()) == 0.0


def test_guard_bands_stay_untouched():
    P = PU.random_pages(np.random.default_rng(13), 9, 10, 77, 16)
    parts, checks = [], []
    for x in (P.table, P.lens, P.held, P.refs):
        t, c = guarded(x.shape, torch.int32)
        t.copy_(torch.from_numpy(x))
        parts.append(t)
        checks.append(c)
    rec = q.KVPages(*parts, 16)
    lst, c1 = guarded((9, 4), torch.int32)
    count, c2 = guarded((1,), torch.int32)
    left, c3 = guarded((1,), torch.int32)
    where, c4 = guarded((77,), torch.int32)
    moves = q.KVMoves(lst, count)
    q.kv_pages_reserve(rec, i32(np.ones(9)), moves, n_free=left)
    q.kv_pages_fork(rec, i32([0, 0, 1, 1, 4, -1, 6, 7, 7]))
    q.kv_pages_compact(rec, moves, where, n_live=left)
    torch.cuda.synchronize()
    status(False)
    for c in checks + [c1, c2, c3, c4]:
        c()


# ------------------------------------------------------------------ together
def test_calls_replay_from_a_graph():
    """fork, reserve and copy captured once: every replay reads the parents of
    that step and changes the same tensors."""
    r = np.random.default_rng(14)
    P = PU.random_pages(r, 8, 40, 400, 16, fill=0.3)
    rec = P.device(torch, q)
    cache = random_cache(r, "fp8", 400, 16, 2, 64)
    parent, new, moves, left = i32(np.arange(8)), i32(np.ones(8)), q.KVMoves.empty(8), i32([0])
    stream = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    saved = [t.clone() for t in (rec.page_table, rec.seq_lens, rec.n_pages, rec.refs)]
    with torch.cuda.stream(stream):
        q.kv_pages_fork(rec, parent)                         # outside the capture first
    torch.cuda.synchronize()
    for t, s in zip((rec.page_table, rec.seq_lens, rec.n_pages, rec.refs), saved):
        t.copy_(s)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        q.kv_pages_fork(rec, parent)
        q.kv_pages_reserve(rec, new, moves, n_free=left)
        q.kv_pages_copy(cache, moves)
        rec.seq_lens.add_(new)
    for _ in range(40):
        p = r.integers(-1, 8, 8).astype(np.int32)
        if r.random() < 0.7:
            p = r.integers(0, 8, 8).astype(np.int32)
        parent.copy_(torch.from_numpy(p))
        want = [t.clone() for t in parts_of(cache)]
        g.replay()
        P.fork(p)
        made, free, bad = P.reserve(np.ones(8))
        assert not bad and free >= 0
        P.lens += 1
        P.same(rec)
        assert int(left) == free and moves.list.cpu().numpy()[:len(made)].tolist() == [list(m) for m in made]
        for src, dst, t, _ in made:
            for w in want:
                w[dst, :, :t] = w[src, :, :t]
        assert all(torch.equal(a, b) for a, b in zip(parts_of(cache), want))
        assert (P.counts() <= P.refs).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_beams_keep_their_own_history(fmt):
    """40 steps of eight beams in two layers: after random forks, every beam's
    cache reads back as the history of the tokens it wrote and inherited; a
    compaction in between changes no beam's history."""
    r = np.random.default_rng(15)
    n, page, heads, dim, pool = 8, 16, 2, 64, 120
    rec = q.KVPages.empty(n, 12, pool, page)
    layers = [random_cache(r, fmt, pool, page, heads, dim) for _ in range(2)]
    moves, big, where = q.KVMoves.empty(n), q.KVMoves.empty(pool), torch.zeros(pool, dtype=torch.int32, device="cuda")
    left, start = i32([0]), i32(np.arange(n + 1))
    new = torch.ones(n, dtype=torch.int32, device="cuda")
    batch = q.KVBatch(rec.page_table, rec.seq_lens, start, n)
    history = [[[] for _ in range(n)] for _ in layers]       # per layer and beam: values as they were stored
    for step in range(40):
        parent = (np.arange(n) if step % 3 == 0 else r.integers(0, n, n)).astype(np.int32)
        q.kv_pages_fork(rec, i32(parent))
        q.kv_pages_reserve(rec, new, moves, n_free=left)
        assert int(left) >= 0
        for layer, c in enumerate(layers):
            q.kv_pages_copy(c, moves)
            x = O.round_bf16(r.standard_normal((n, heads, dim)))
            d = to_dev(O.bf16_bits(x))
            q.kv_cache_append(c, batch, d, d)
            stored = U.values(*U.quantise(x, fmt, 1.0), fmt, 1.0)
            history[layer] = [history[layer][int(p)] + [stored[i]] for i, p in enumerate(parent)]
        rec.seq_lens.add_(1)
        if step % 11 == 7:
            q.kv_pages_compact(rec, big, where)
            for c in layers:
                q.kv_pages_copy(c, big)
            live = int((rec.refs != 0).sum())
            assert bool((rec.refs[:live] != 0).all())
        if step % 5 == 4:
            length = step + 1
            whole = q.KVBatch(rec.page_table, i32(np.zeros(n)), i32(np.arange(n + 1) * length), n * length)
            for layer, c in enumerate(layers):
                outs = [torch.empty((n * length, heads, dim), dtype=torch.float32, device="cuda") for _ in range(2)]
                q.kv_cache_read(c, whole, *outs)
                want = np.stack([np.stack(h) for h in history[layer]]).reshape(n * length, heads, dim)
                for o in outs:
                    assert np.array_equal(o.cpu().numpy(), want.astype(np.float32)), (step, layer)
    status(False)
    refs = torch.zeros(pool, dtype=torch.int64, device="cuda")
    for b in range(n):
        refs.index_add_(0, rec.page_table[b, :int(rec.n_pages[b])].long(), torch.ones(int(rec.n_pages[b]), dtype=torch.int64, device="cuda"))
    assert torch.equal(refs.int(), rec.refs)
    q.kv_pages_fork(rec, i32(np.full(n, -1)))
    assert int(rec.refs.sum()) == 0 and int(rec.n_pages.sum()) == 0


@pytest.mark.parametrize("fmt,page,heads,dim", [("bf16", 64, 8, 128), ("bf16", 256, 3, 256), ("fp8", 48, 5, 64), ("nvfp4", 16, 4, 128),
                                                ("fp8", 1024, 2, 256), ("nvfp4", 64, 1, 64)])
def test_long_lists_of_moves(fmt, page, heads, dim):
    """Lists whose capacity is many pages: whole pages, part-filled ones, none; short lists in them; entries that do not fit."""
    r = np.random.default_rng(16)
    row = {"bf16": 2 * dim, "fp8": dim, "nvfp4": dim // 2}[fmt]
    n = max(3, 70 * 2 ** 20 // (2 * page * heads * row))
    pages = min(2 * n + 1, 3000)
    n_used = (pages - 1) // 2
    c = random_cache(r, fmt, pages, page, heads, dim)
    for count, mode in ((n_used, "whole"), (n_used, "mixed"), (1, "whole"), (0, "whole"), (min(n_used, 37), "bad")):
        ids = r.permutation(pages)
        tokens = np.full(n_used, page)
        if mode != "whole":
            tokens = np.where(r.random(n_used) < 0.5, page, r.integers(0, page + 1, n_used))
        moves = np.zeros((max(n, n_used), 4), np.int64)
        moves[:n_used, 0], moves[:n_used, 1], moves[:n_used, 2] = ids[:n_used], ids[n_used:2 * n_used], tokens
        if mode == "bad":
            moves[3, 0], moves[5, 1], moves[7, 2], moves[9, 2] = pages, -1, page + 1, -1
        want = [t.clone() for t in parts_of(c)]
        src, dst, t = (torch.from_numpy(moves[:count, i]).cuda() for i in range(3))
        ok = (src >= 0) & (src < pages) & (dst >= 0) & (dst < pages) & (t >= 0) & (t <= page)
        src, dst, t = src[ok], dst[ok], t[ok]
        inside = torch.arange(page, device="cuda")[None] < t[:, None]
        for w in want:
            keep = inside.view(len(t), 1, page, *[1] * (w.dim() - 3))
            w[dst] = torch.where(keep, w[src], w[dst])
        q.kv_pages_copy(c, q.KVMoves(i32(moves), i32([count])))
        status(mode == "bad")
        assert all(torch.equal(a, b) for a, b in zip(parts_of(c), want)), mode
    for count in (-1, max(n, n_used) + 1):
        q.kv_pages_copy(c, q.KVMoves(i32(moves), i32([count])))
        status(True)
        assert all(torch.equal(a, b) for a, b in zip(parts_of(c), want))


def test_many_rows_share_and_part():
    """Prompts of 1 to 40 rows whose beams go on from each other or from another prompt, pages in runs of every length."""
    r = np.random.default_rng(17)
    for n, wide, page in ((1000, 21, 16), (97, 70, 48), (33, 9, 64), (1024, 3, 1024)):
        P = PU.Pages(n, wide, n * wide + 5, page)
        order, b = list(r.permutation(P.pool)), 0
        while b < n:
            rows = min(n - b, int(r.integers(1, 41)))
            shared = [order.pop() for _ in range(int(r.integers(0, wide)))]
            for i in range(b, b + rows):
                own = [order.pop() for _ in range(int(r.integers(0, wide - len(shared) + 1)))] if len(order) > n * 2 else []
                P.table[i, :len(shared)], P.table[i, len(shared):len(shared) + len(own)] = shared, own
                P.held[i] = len(shared) + len(own)
                P.lens[i] = max(0, int(P.held[i]) * page - int(r.integers(0, page)))
                for e in shared + own:
                    P.refs[e] += 1
            b += rows
        rec = P.device(torch, q)
        for _ in range(3):
            near = np.clip(np.arange(n) + r.integers(-3, 4, n), 0, n - 1)
            do_fork(P, rec, np.where(r.random(n) < 0.1, -1, near).astype(np.int32))
        assert (P.counts() == P.refs).all()
        do_reserve(P, rec, r.integers(0, 3, n))
        do_compact(P, rec, 1 << 20)


@pytest.mark.parametrize("sizes", [(64, 300, 9000, 16), (64, 4096, 200000, 16), (64, 4097, 200000, 16), (65, 300, 9000, 16), (1, 4096, 5000, 16),
                                   (127, 9, 900, 32), (128, 9, 900, 32), (129, 17, 2000, 32)])
def test_fork_at_the_borders_of_its_kernels(sizes):
    r = np.random.default_rng(18)
    P = PU.random_pages(r, *sizes)
    rec = P.device(torch, q)
    for _ in range(3):
        do_fork(P, rec, r.integers(-1, P.n, P.n).astype(np.int32))
    P.table[0, :max(1, P.held[0])], P.held[0], P.lens[0] = -1, max(1, P.held[0]), 1        # entries outside the pool
    rec = P.device(torch, q)
    do_fork(P, rec, np.zeros(P.n, np.int32))


def test_long_lists_beyond_32_bits():
    """As test_copy_beyond_32_bits, with a list long enough for the bulk copies."""
    pages, page, heads, dim = 4200, 256, 8, 256
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("needs 12 GB of device memory")
    k = torch.zeros((pages, heads, page, dim), dtype=torch.bfloat16, device="cuda")
    k[pages - 70:].normal_()
    c = q.KVCache("bf16", k, torch.zeros_like(k))
    moves = [(pages - 1 - i, i, page if i % 3 else 9, 0) for i in range(64)]
    q.kv_pages_copy(c, q.KVMoves(i32(moves), i32([64])))
    for src, dst, n, _ in moves:
        assert torch.equal(k[dst, :, :n], k[src, :, :n]) and not k[dst, :, n:].any()


def test_page_calls_on_a_stream_of_their_own_and_what_the_binding_refuses():
    r = np.random.default_rng(19)
    P = PU.random_pages(r, 9, 40, 400, 16, fill=0.3)
    rec = P.device(torch, q)
    parent, new = r.integers(0, 9, 9).astype(np.int32), np.ones(9)
    dp, dn, moves, where = i32(parent), i32(new), q.KVMoves.empty(9), torch.zeros(400, dtype=torch.int32, device="cuda")
    big, cache, side = q.KVMoves.empty(400), random_cache(r, "fp8", 400, 16, 1, 64), torch.cuda.Stream()
    want = [t.clone() for t in parts_of(cache)]
    torch.cuda.synchronize()
    q.kv_pages_fork(rec, dp, stream=side)
    q.kv_pages_reserve(rec, dn, moves, stream=side)
    q.kv_pages_copy(cache, moves, stream=side)
    q.kv_pages_compact(rec, big, where, stream=side)
    q.kv_pages_copy(cache, big, stream=side)
    side.synchronize()
    P.fork(parent)
    made = P.reserve(new)[0]
    made += P.compact(400)[0]
    P.same(rec)
    for src, dst, t, _ in made:
        for w in want:
            w[dst, :, :t] = w[src, :, :t]
    assert all(torch.equal(a, b) for a, b in zip(parts_of(cache), want))
    for f in (lambda: q.kv_pages_fork(rec, dp[:8]), lambda: q.kv_pages_fork(rec, dp.long()), lambda: q.kv_pages_fork(rec, dp.cpu()),
              lambda: q.kv_pages_reserve(rec, dn.view(3, 3), moves), lambda: q.kv_pages_reserve(rec, dn, moves, n_free=dn),
              lambda: q.kv_pages_compact(rec, big, where[:399]), lambda: q.kv_pages_compact(rec, big, where, n_live=where),
              lambda: q.KVPages(rec.page_table[:8], rec.seq_lens, rec.n_pages, rec.refs, 16),
              lambda: q.KVPages(rec.page_table, rec.seq_lens.long(), rec.n_pages, rec.refs, 16),
              lambda: q.KVPages(rec.page_table[:, ::2], rec.seq_lens, rec.n_pages, rec.refs, 16),
              lambda: q.KVMoves(where, dn[:1]), lambda: q.KVMoves(big.list, dn), lambda: q.KVMoves(big.list[:, :3], dn[:1])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: q.kv_pages_reserve(rec, dn, q.KVMoves.empty(8)), lambda: q.kv_pages_fork(q.KVPages(*vars_of(rec), 24), dp),
              lambda: q.kv_pages_fork(rec, i32(np.zeros(10))[1:])):
        with pytest.raises(q.QGemvError):
            f()
    P.same(rec)


def vars_of(rec):
    return rec.page_table, rec.seq_lens, rec.n_pages, rec.refs
