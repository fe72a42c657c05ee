"""tree_attention (GPU) against the plain 64-bit form, with the bounds that
kv_util.attention_bounds derives, and the run of the cache's operators together
as a decode step uses them."""
import numpy as np
import pytest

import kv_util as U
import oracle as O
from checks import check_bf16
from gpu_util import bits16, guarded, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("bit_quantized_weight_gb300")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    q.qg_debug_set_wait(0, False)
    yield
    assert q.qg_last_device_status() == q.QG_OK


FMTS = ("bf16", "fp8", "nvfp4")


def seen_matrix(masks, first, t, length):
    bits = [(int(masks[first + i]) & (2 ** 64 - 1)) for i in range(t)]
    seen = np.ones((t, length + t), bool)
    for i in range(t):
        seen[i, length:] = [bool(bits[i] >> j & 1) for j in range(t)]
    return seen


def workspace(cache, heads, tree):
    return torch.empty(q.tree_attention_workspace_size(cache, heads, tree), dtype=torch.uint8, device="cuda")


def check(P, x, masks, scale, out, lse, rows=None):
    """out [total][Hq][D] (device bf16) and lse against the oracle, sequence by sequence."""
    got, got_lse = bits16(out), None if lse is None else lse.cpu().numpy().astype(np.float64)
    for b, (n, t) in enumerate(zip(P.lens, P.counts)):
        if t == 0 or (rows is not None and b not in rows):
            continue
        first = int(P.start[b])
        k, v = P.stored(0, b, 0, n + t), P.stored(1, b, 0, n + t)
        seen = seen_matrix(masks, first, t, n)
        ref, ref_lse, a, ds = U.attention(x[first:first + t], k, v, seen, scale)
        B, Bl = U.attention_bounds(a, ds, ref_lse, n + t, P.dim, P.fmt)
        check_bf16(got[first:first + t], ref, B, f"sequence {b}")
        if lse is not None:
            g = got_lse[first:first + t]
            empty = ~np.isfinite(ref_lse)
            assert np.array_equal(g[empty], ref_lse[empty])
            off = np.abs(g[~empty] - ref_lse[~empty])
            assert (off <= Bl[~empty]).all(), np.max(off / Bl[~empty])


def attend(P, group, masks=None, scale=None, tree=None, seed=20, qstd=1.0, with_lse=True):
    r = np.random.default_rng(seed)
    heads = group * P.heads
    x = O.round_bf16(r.standard_normal((P.total, heads, P.dim)) * qstd)
    cache, batch = P.device(torch, q)
    tree = tree or max(P.counts + [1])
    out, guard = guarded((P.total, heads, P.dim), torch.bfloat16)
    lse = torch.full((P.total, heads), 5.0, device="cuda") if with_lse else None
    md = None if masks is None else torch.from_numpy(masks).cuda()
    ws, ws_guard = guarded((q.tree_attention_workspace_size(cache, heads, tree),), torch.uint8)
    q.tree_attention(cache, batch, to_dev(O.bf16_bits(x)), out, tree, tree_mask=md, scale=scale, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    guard()
    ws_guard()
    assert q.qg_last_device_status() == q.QG_OK
    if masks is None:
        masks = [(1 << (i + 1)) - 1 for t in P.counts for i in range(t)]
    check(P, x, masks, P.dim ** -0.5 if scale is None else scale, out, lse)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,page,heads,group,lens,counts", [
    (128, 64, 1, 1, [0], [1]),                                # one key
    (128, 64, 4, 12, [1000], [1]),                            # a decode step
    (64, 16, 2, 4, [0, 15, 16, 17], [1, 1, 1, 1]),            # lengths around a page's end
    (128, 48, 2, 8, [31, 33, 0, 127, 128], [1, 2, 3, 0, 5]),  # ragged, an empty sequence
    (256, 32, 2, 5, [100, 7], [3, 2]),
    (128, 16, 1, 16, [513], [16]),
    (128, 128, 2, 7, [300, 40], [7, 33]),
    (64, 64, 1, 8, [129, 5], [64, 63]),                       # the largest trees
    (128, 32, 2, 12, [255], [20]),
    (256, 16, 1, 12, [60], [13]),
    (128, 64, 1, 32, [200, 3], [1, 1]),                       # many query heads
    (64, 256, 1, 128, [77], [2]),
    (128, 1024, 3, 3, [1100], [2]),
])
def test_trees_and_steps(fmt, dim, page, heads, group, lens, counts):
    P = U.Paged(21, fmt, dim, page, heads, lens, counts, kg=1.0 if fmt == "bf16" else 0.8, vg=1.0 if fmt == "bf16" else 1.3)
    attend(P, group, U.ancestor_masks(np.random.default_rng(22), counts))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,group,lens,counts", [
    (128, 12, [9001], [1]), (64, 4, [6000, 30, 2500], [2, 1, 9]), (256, 6, [3001], [2]), (128, 8, [4100], [24]),
])
def test_long_contexts_split_over_the_gpu(fmt, dim, group, lens, counts):
    P = U.Paged(23, fmt, dim, 64, 1, lens, counts)
    attend(P, group, U.ancestor_masks(np.random.default_rng(24), counts), qstd=2.0)


@pytest.mark.parametrize("fmt", FMTS)
def test_many_ragged_sequences(fmt):
    r = np.random.default_rng(25)
    lens, counts = [int(v) for v in r.integers(0, 400, 70)], [int(v) for v in r.integers(0, 4, 70)]
    P = U.Paged(26, fmt, 64, 16, 2, lens, counts)
    attend(P, 3, U.ancestor_masks(r, counts), tree=4)


@pytest.mark.parametrize("group,tree", [(1, 2), (20, 2)])
def test_as_many_sequences_as_a_call_takes(group, tree):
    """1,024 sequences, every seventh without tokens of its own."""
    r = np.random.default_rng(51)
    lens = [int(v) for v in r.integers(0, 40, 1024)]
    counts = [0 if b % 7 == 0 else 1 + b % tree for b in range(1024)]
    P = U.Paged(52, "fp8", 64, 16, 1, lens, counts)
    attend(P, group, U.ancestor_masks(r, counts), tree=tree)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,group,tree,lens,counts", [
    (128, 12, 64, [300, 0, 65, 700, 1], [1, 3, 20, 0, 64]),   # a plan for 768 rows, units of 12 to 768
    (64, 8, 33, [1000, 200], [1, 17]),                        # 264 rows planned, 8 and 136 there
    (128, 16, 8, [64, 63, 1], [1, 8, 2]),
    (128, 4, 8, [500, 9], [1, 2]),                            # 32 rows planned
])
def test_a_larger_max_tree_than_there_are_tokens(fmt, dim, group, tree, lens, counts):
    P = U.Paged(56, fmt, dim, 32, 2, lens, counts)
    attend(P, group, U.ancestor_masks(np.random.default_rng(57), counts), tree=tree)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group", [2, 20])
def test_lengths_around_every_tile(fmt, group):
    """Contexts that end just before, at and after each step and tile of 16, 32, 64, 128 and 256 keys."""
    lens = [n + d for n in (16, 32, 64, 128, 192, 256, 512) for d in (-3, -2, -1, 0, 1)]
    P = U.Paged(53, fmt, 64, 16, 1, lens, [2] * len(lens))
    attend(P, group, U.ancestor_masks(np.random.default_rng(54), P.counts))


def test_chain_without_a_mask_and_without_lse():
    P = U.Paged(27, "fp8", 128, 64, 2, [50, 0], [5, 64])
    attend(P, 4, None, with_lse=False)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group,t", [(4, 4), (8, 8), (8, 33)])
def test_rows_that_see_nothing(fmt, group, t):
    """Masks that leave rows empty (no context) or see only some drafts, bits
    beyond the sequence's tokens set."""
    P = U.Paged(28, fmt, 128, 16, 1, [0, 40], [t, t])
    masks = U.ancestor_masks(np.random.default_rng(29), [t, t])
    masks[1] = 0
    masks[2] = np.uint64(1 << 63).view(np.int64) if t < 64 else 0   # only a token that does not exist
    masks[t + 1] = 0
    masks[t + 3] |= np.uint64(1 << 63 | 1 << 62).view(np.int64)
    attend(P, group, masks)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group,t,n", [(2, 6, 37), (8, 12, 150), (8, 40, 64)])
def test_nan_and_infinity_in_unseen_places(fmt, group, t, n):
    """A draft whose keys and values are not finite reaches only the rows that
    see it: nobody here, though other rows of the same tile see its neighbours."""
    P = U.Paged(30, fmt, 128, 32, 2, [n, 5], [t, t])
    masks = U.ancestor_masks(np.random.default_rng(31), [t, t])
    for bad in (2, t - 1):
        masks[:] = masks & ~np.int64(1 << bad)
        for b in (0, 1):
            pg, off = P.at(b, P.lens[b] + bad, 1)
            for kv in (0, 1):
                codes, scales = P.parts[kv]
                if fmt == "bf16":
                    codes[pg, :, off] = [0x7F80, 0xFF80, 0x7FC0, 0x7F80] * (128 // 4)
                elif fmt == "fp8":
                    codes[pg, :, off] = 0x7F
                    scales[pg, :, off] = 255
                else:
                    scales[pg, :, off] = 0x7F
    attend(P, group, masks)


@pytest.mark.parametrize("fmt", ("bf16", "fp8"))
@pytest.mark.parametrize("group,n", [(2, 70), (5, 70), (12, 70), (12, 0), (40, 200)])
def test_nan_reaches_the_rows_that_see_it(fmt, group, n):
    """A draft with a NaN value: rows that see it get NaN there, others do not."""
    t = 5
    P = U.Paged(32, fmt, 64, 16, 1, [n], [t])
    masks = U.ancestor_masks(np.random.default_rng(33), [t])
    masks[:] = masks & ~np.int64(4)
    masks[3] |= 4
    pg, off = P.at(0, n + 2, 1)
    P.parts[1][0][pg, :, off, 7] = 0x7FC0 if fmt == "bf16" else 0x7F
    x = O.round_bf16(np.random.default_rng(34).standard_normal((t, group, 64)))
    cache, batch = P.device(torch, q)
    out = torch.empty((t, group, 64), dtype=torch.bfloat16, device="cuda")
    q.tree_attention(cache, batch, to_dev(O.bf16_bits(x)), out, t, tree_mask=torch.from_numpy(masks).cuda(),
                     workspace=workspace(cache, group, t))
    nan = torch.isnan(out).cpu().numpy()
    want = np.zeros_like(nan)
    want[3, :, 7] = True
    assert np.array_equal(nan, want)


def test_an_infinite_value_reaches_the_rows_that_see_it():
    for group in (2, 12):
        P = U.Paged(50, "bf16", 128, 16, 1, [33], [3])
        pg, off = P.at(0, 34, 1)
        P.parts[1][0][pg, :, off, 100] = 0xFF80                 # -infinity in draft 1
        masks = np.array([1, 3, 5], np.int64)
        cache, batch = P.device(torch, q)
        x = torch.randn((3, group, 128), device="cuda").to(torch.bfloat16)
        out = torch.empty_like(x)
        q.tree_attention(cache, batch, x, out, 3, tree_mask=torch.from_numpy(masks).cuda(),
                         workspace=workspace(cache, group, 3))
        got = out.float().cpu().numpy()
        assert (got[1, :, 100] == -np.inf).all()
        got[1, :, 100] = 0
        assert np.isfinite(got).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group", [2, 4, 12, 40])
@pytest.mark.parametrize("qstd,scale", [(30.0, None), (0.0, None), (1e-3, 1000.0), (1e18, 1e-18), (1.0, 0.0), (3.0, -0.5)])
def test_sharp_flat_and_wide_range_scores(fmt, group, qstd, scale):
    P = U.Paged(35, fmt, 128, 64, 1, [700], [6])
    attend(P, group, U.ancestor_masks(np.random.default_rng(36), [6]), scale=scale, qstd=qstd)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group,t", [(4, 2), (12, 8)])
def test_maxima_that_rise_and_fall_along_the_context(fmt, group, t):
    """Keys grow towards the end, then towards the start: every running
    maximum is replaced often, and values differ by orders of magnitude."""
    for order in (1, -1):
        P = U.Paged(37, fmt, 64, 16, 1, [600], [t])
        r = np.random.default_rng(38)
        ramp = np.linspace(0.01, 6.0, 600)[::order, None, None]
        pg, off = P.at(0, 0, 600)
        for kv in (0, 1):
            x = O.round_bf16(r.standard_normal((600, 1, 64)) * (ramp if kv == 0 else 10.0 ** (2 * np.sin(ramp * 3))))
            codes, scales = U.quantise(x, fmt, 1.0)
            P.parts[kv][0][pg, :, off] = codes
            if scales is not None:
                P.parts[kv][1][pg, :, off] = scales
        attend(P, group, U.ancestor_masks(r, [t]), qstd=2.0)


def test_strided_queries_and_rows_behind_the_last_sequence():
    P = U.Paged(39, "fp8", 128, 64, 2, [90, 10], [3, 2])
    cache, _ = P.device(torch, q)
    batch = P.batch(torch, q, n_tokens=9)
    r = np.random.default_rng(40)
    wide = O.round_bf16(r.standard_normal((9, 12, 128)))
    d = to_dev(O.bf16_bits(wide))
    out = torch.full((9, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((9, 8), 7.0, device="cuda")
    masks = U.ancestor_masks(r, [3, 2])
    m9 = np.concatenate([masks, np.full(4, -1, np.int64)])
    q.tree_attention(cache, batch, d[:, 2:10], out, 3, tree_mask=torch.from_numpy(m9).cuda(), lse=lse,
                     workspace=workspace(cache, 8, 3))
    check(P, wide[:5, 2:10], masks, 128 ** -0.5, out[:5], lse[:5])
    assert (out[5:] == 7.0).all() and (lse[5:] == 7.0).all()


@pytest.mark.parametrize("group", [2, 12])
def test_bad_device_data_is_left_out_and_recorded(group):
    lens, counts = [30, 30, 30, 30, 30], [4, 4, 4, 9, 4]
    P = U.Paged(41, "nvfp4", 64, 16, 2, lens, counts)
    cache, batch = P.device(torch, q)
    batch.seq_lens[1] = -5
    batch.seq_lens[2] = P.max_pages * 16 - 3
    r = np.random.default_rng(42)                            # sequence 3: more than max_tree tokens
    heads = 2 * group
    x = O.round_bf16(r.standard_normal((P.total, heads, 64)))
    masks = U.ancestor_masks(r, counts)
    out = torch.full((P.total, heads, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    q.tree_attention(cache, batch, to_dev(O.bf16_bits(x)), out, 8, tree_mask=torch.from_numpy(masks).cuda(),
                     workspace=workspace(cache, heads, 8))
    assert q.qg_last_device_status() == q.QG_ERR_INVALID_ARG
    check(P, x, masks, 0.125, out, None, rows=(0, 4))
    assert (out[4:21] == 7.0).all()
    # a page outside the cache: its keys are not seen
    cache, batch = P.device(torch, q)
    batch.page_table[0, 1] = -1
    batch.page_table[4, 0] = 1 << 30
    q.tree_attention(cache, batch, to_dev(O.bf16_bits(x)), out, 9, tree_mask=torch.from_numpy(masks).cuda(),
                     workspace=workspace(cache, heads, 9))
    assert q.qg_last_device_status() == q.QG_ERR_INVALID_ARG
    got = bits16(out)
    for b, gone in ((0, slice(16, 32)), (4, slice(0, 16))):
        first = int(P.start[b])
        k, v = np.zeros((34, 2, 64)), np.zeros((34, 2, 64))
        keep = [p for p in range(34) if not gone.start <= p < gone.stop]
        for p in keep:
            k[p], v[p] = P.stored(0, b, p, 1)[0], P.stored(1, b, p, 1)[0]
        seen = seen_matrix(masks, first, 4, 30)
        seen[:, gone] = False
        ref, lse, a, ds = U.attention(x[first:first + 4], k, v, seen, 0.125)
        B, _ = U.attention_bounds(a, ds, lse, 34, 64, P.fmt)
        check_bf16(got[first:first + 4], ref, B, f"sequence {b}")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group,t", [(12, 1), (12, 8)])
def test_same_bits_every_time_and_for_other_batches(fmt, group, t):
    """Two runs give the same bits, and nothing left in the workspace matters."""
    P = U.Paged(43, fmt, 128, 64, 2, [2000, 333], [t, t])
    cache, batch = P.device(torch, q)
    x = torch.randn((P.total, 2 * group, 128), device="cuda").to(torch.bfloat16)
    ws = workspace(cache, 2 * group, t)
    outs = []
    for fill in (0, 255, 127):
        ws.fill_(fill)
        out = torch.empty_like(x)
        lse = torch.empty((P.total, 2 * group), device="cuda")
        q.tree_attention(cache, batch, x, out, t, lse=lse, workspace=ws)
        outs.append((out, lse))
    for out, lse in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("fmt", FMTS)
def test_a_speculative_step_end_to_end(fmt):
    """Append a step's drafts from a fused projection, attend, accept a path,
    append the next step at the new lengths and attend again; the cache at the
    end equals one that held the accepted tokens from the start."""
    heads, group, dim, page = 2, 6, 128, 16
    lens, counts = [45, 0, 130], [6, 6, 6]
    P = U.Paged(44, fmt, dim, page, heads, lens, [12] * 3)   # pages for two steps
    P.counts, P.start, P.total = counts, np.array([0, 6, 12, 18], np.int32), 18
    cache, batch = P.device(torch, q)
    r = np.random.default_rng(45)
    hq = heads * group
    ws = workspace(cache, hq, 6)
    path = torch.from_numpy(np.tile(np.array([0, 2, 5, 0, 0, 0], np.int32), 3)).cuda()
    kept = torch.tensor([3, 1, 2], dtype=torch.int32, device="cuda")
    for step in range(2):
        qkv = O.round_bf16(r.standard_normal((18, hq + 2 * heads, dim)))
        d = to_dev(O.bf16_bits(qkv))
        masks = U.ancestor_masks(r, counts)
        out = torch.empty((18, hq, dim), dtype=torch.bfloat16, device="cuda")
        lse = torch.empty((18, hq), device="cuda")
        q.kv_cache_append(cache, batch, d[:, hq:hq + heads], d[:, hq + heads:])
        q.tree_attention(cache, batch, d[:, :hq], out, 6, tree_mask=torch.from_numpy(masks).cuda(), lse=lse, workspace=ws)
        for b in range(3):
            for kv, lo in ((0, hq), (1, hq + heads)):
                codes, scales = U.quantise(qkv[6 * b:6 * b + 6, lo:lo + heads], fmt, 1.0)
                pg, off = P.at(b, P.lens[b], 6)
                P.parts[kv][0][pg, :, off] = codes
                if scales is not None:
                    P.parts[kv][1][pg, :, off] = scales
        check(P, qkv[:, :hq], masks, dim ** -0.5, out, lse)
        q.kv_cache_accept(cache, batch, path, kept, new_lens=batch.seq_lens)
        for b, n in enumerate((3, 1, 2)):
            pg, off = P.at(b, P.lens[b], 6)
            tp, to = P.at(b, P.lens[b], n)
            for part in P.parts:
                for a in part:
                    if a is not None:
                        a[tp, :, to] = a[pg, :, off][[0, 2, 5][:n]]
            P.lens[b] += n
        assert batch.seq_lens.cpu().tolist() == P.lens
    total = sum(P.lens)
    rb = q.KVBatch(batch.page_table, torch.zeros(3, dtype=torch.int32, device="cuda"),
                   torch.tensor(np.concatenate(([0], np.cumsum(P.lens))), dtype=torch.int32, device="cuda"), total)
    k_out = torch.empty((total, heads, dim), dtype=torch.float32, device="cuda")
    v_out = torch.empty_like(k_out)
    q.kv_cache_read(cache, rb, k_out, v_out)
    for kv, got in ((0, k_out), (1, v_out)):
        want = np.concatenate([P.stored(kv, b, 0, n) for b, n in enumerate(P.lens)])
        assert np.array_equal(got.cpu().numpy(), want.astype(np.float32))


@pytest.mark.parametrize("group,t", [(6, 1), (12, 6)])
def test_captured_step_replays_with_new_lengths(group, t):
    """One graph of append, attend and accept, replayed: lengths are device
    data, two graphs share one workspace in turn, and an eager call between
    replays changes nothing."""
    fmt, heads, dim = "fp8", 2, 128
    P = U.Paged(46, fmt, dim, 64, heads, [700, 20], [t * 4] * 2)
    P.counts, P.start, P.total = [t, t], np.array([0, t, 2 * t], np.int32), 2 * t
    cache, batch = P.device(torch, q)
    twin, twin_batch = P.device(torch, q)
    hq = heads * group
    x = torch.zeros((2 * t, hq + 2 * heads, dim), dtype=torch.bfloat16, device="cuda")
    ws = workspace(cache, hq, t)
    path = torch.arange(t, dtype=torch.int32, device="cuda").repeat(2)
    kept = torch.full((2,), t, dtype=torch.int32, device="cuda")

    def step(c, b, out, lse):
        q.kv_cache_append(c, b, x[:, hq:hq + heads], x[:, hq + heads:])
        q.tree_attention(c, b, x[:, :hq], out, t, lse=lse, workspace=ws)
        q.kv_cache_accept(c, b, path, kept, new_lens=b.seq_lens)

    out, lse = torch.empty((2 * t, hq, dim), dtype=torch.bfloat16, device="cuda"), torch.empty((2 * t, hq), device="cuda")
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    side = torch.cuda.Stream()
    graphs = []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step(cache, batch, out, lse)
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        x.copy_(torch.randn(x.shape, device="cuda"))
        graphs[i % 2].replay()
        step(twin, twin_batch, out2, lse2)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)
        assert torch.equal(batch.seq_lens, twin_batch.seq_lens)
    assert torch.equal(cache.k, twin.k) and torch.equal(cache.v_scales, twin.v_scales)


def test_two_streams_with_their_own_workspaces():
    P = U.Paged(47, "nvfp4", 128, 64, 2, [3000, 100], [2, 2])
    cache, batch = P.device(torch, q)
    x = torch.randn((4, 16, 128), device="cuda").to(torch.bfloat16)
    ref = torch.empty_like(x)
    q.tree_attention(cache, batch, x, ref, 2, workspace=workspace(cache, 16, 2))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, spaces = [torch.empty_like(x) for _ in range(2)], [workspace(cache, 16, 2) for _ in range(2)]
    for _ in range(20):
        for s, o, w in zip(streams, outs, spaces):
            q.tree_attention(cache, batch, x, o, 2, workspace=w, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, ref)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,lanes,tokens,group,t", [
    (128, 1, 65536, 12, 16), (128, 8, 8192, 8, 64), (64, 1, 65536, 12, 16), (128, 1, 65536, 12, 7),
    (128, 2, 30001, 12, 1), (256, 1, 20000, 4, 4)])
def test_calls_back_to_back_give_what_they_give_alone(fmt, dim, lanes, tokens, group, t):
    """Calls that run one right behind the other (their tiles all in the L2
    cache, the next kernel waiting for the last) against calls that the host
    waits for."""
    r = np.random.default_rng(53)
    heads, page = 4, 64
    need = (tokens + t + page - 1) // page
    shape = (lanes * need, heads, page, dim)

    def store(seed):
        x = torch.from_numpy(np.random.default_rng(seed).integers(0, 256, shape, dtype=np.uint8))
        if fmt == "bf16":
            return x.cuda().to(torch.bfloat16).sub_(128).div_(64), None
        if fmt == "fp8":
            return (x & 0xBF).cuda(), torch.from_numpy(r.integers(10, 16, shape[:3], dtype=np.uint8)).cuda()
        codes = x[..., :dim // 2].contiguous()
        return codes.cuda(), torch.from_numpy(r.integers(0x30, 0x40, shape[:3] + (dim // 16,), dtype=np.uint8)).cuda()

    (k, ks), (v, vs) = store(1), store(2)
    cache = q.KVCache(fmt, k, v, ks, vs)
    table = torch.from_numpy(r.permutation(lanes * need).astype(np.int32).reshape(lanes, need)).cuda()
    batch = q.KVBatch(table, torch.full((lanes,), tokens, dtype=torch.int32, device="cuda"),
                      torch.arange(0, lanes * t + 1, t, dtype=torch.int32, device="cuda"), lanes * t)
    xs = [torch.randn((lanes * t, heads * group, dim), device="cuda").to(torch.bfloat16) for _ in range(2)]
    spaces = [workspace(cache, heads * group, t) for _ in range(2)]
    outs = [torch.empty_like(xs[i % 2]) for i in range(8)]
    for i in range(2):
        q.tree_attention(cache, batch, xs[i], outs[i], t, workspace=spaces[i])
        torch.cuda.synchronize()
    assert torch.isfinite(outs[0]).all()
    for _ in range(4):
        for i in range(2, 8):
            q.tree_attention(cache, batch, xs[i % 2], outs[i], t, workspace=spaces[i % 2])
        torch.cuda.synchronize()
        for i in range(2, 8):
            assert torch.equal(outs[i], outs[i % 2]), i
            outs[i].zero_()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("t", [6, 16])
def test_bounded_waits_report_a_timeout_and_recover(fmt, t):
    """The tensor-core kernel's key tiles are never announced: the call ends
    with QG_ERR_DEVICE_TIMEOUT, and a clean one right after is right."""
    P = U.Paged(49, fmt, 128, 64, 1, [900], [t])
    masks = U.ancestor_masks(np.random.default_rng(50), [t])
    x = O.round_bf16(np.random.default_rng(55).standard_normal((t, 12, 128)))
    cache, batch = P.device(torch, q)
    d, out, ws = to_dev(O.bf16_bits(x)), torch.empty((t, 12, 128), dtype=torch.bfloat16, device="cuda"), workspace(cache, 12, t)
    md = torch.from_numpy(masks).cuda()
    q.qg_debug_set_wait(20_000_000, True)
    try:
        q.tree_attention(cache, batch, d, out, t, tree_mask=md, workspace=ws)
        assert q.qg_last_device_status() == q.QG_ERR_DEVICE_TIMEOUT
    finally:
        q.qg_debug_set_wait(0, False)
    q.tree_attention(cache, batch, d, out, t, tree_mask=md, workspace=ws)
    assert q.qg_last_device_status() == q.QG_OK
    check(P, x, masks, 128 ** -0.5, out, None)


def test_refusals():
    P = U.Paged(48, "fp8", 64, 16, 2, [5], [2])
    cache, batch = P.device(torch, q)
    x = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, ws = torch.empty_like(x), workspace(cache, 4, 2)
    with pytest.raises(q.QGemvError) as e:
        q.tree_attention(cache, batch, x, out, 2)
    assert e.value.status == q.QG_ERR_WORKSPACE
    with pytest.raises(q.QGemvError):
        q.tree_attention(cache, batch, x, out, 65, workspace=ws)
    with pytest.raises(q.QGemvError):
        q.tree_attention(cache, batch, torch.zeros((2, 3, 64), dtype=torch.bfloat16, device="cuda"),
                         torch.empty((2, 3, 64), dtype=torch.bfloat16, device="cuda"), 2, workspace=ws)
    for bad in (dict(out=out.float()), dict(lse=torch.empty((2, 3), device="cuda")),
                dict(tree_mask=torch.zeros(3, dtype=torch.int64, device="cuda")),
                dict(tree_mask=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        kw = dict(out=out, workspace=ws)
        kw.update(bad)
        with pytest.raises(ValueError):
            q.tree_attention(cache, batch, x, kw.pop("out"), 2, **kw)
    with pytest.raises(ValueError):
        q.tree_attention(cache, batch, x.transpose(0, 1), out, 2, workspace=ws)
    assert q.qg_last_device_status() == q.QG_OK
