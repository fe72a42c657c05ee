"""tree_attention (GPU) where inputs are not finite, scores are far beyond the
exponential's range, or a row sees a single key: against the plain 64-bit form,
on every route (16, 32, 128 and 256 rows per unit, split over the GPU or not,
joined by four warps per row or by one)."""
import numpy as np
import pytest

import kv_util as U
import oracle as O
from checks import check_bf16
from gpu_util import bits16, to_dev

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


def chains(counts):
    return np.array([(1 << (i + 1)) - 1 for t in counts for i in range(t)], dtype=np.uint64).view(np.int64)


def own_only(counts):
    return np.array([1 << i for t in counts for i in range(t)], dtype=np.uint64).view(np.int64)


def attend(P, x, masks, scale=None, change=None):
    """(out as 64-bit values, its bits, lse) of queries x [total][Hq][D]; change(batch) edits the device batch."""
    cache, batch = P.device(torch, q)
    if change:
        change(batch)
    bits = O.bf16_bits(np.where(np.isnan(x), 0.0, x))
    bits[np.isnan(x)] = 0x7FC0
    heads, tree = x.shape[1], max(P.counts)
    out = torch.zeros((P.total, heads, P.dim), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((P.total, heads), device="cuda")
    ws = torch.empty(q.tree_attention_workspace_size(cache, heads, tree), dtype=torch.uint8, device="cuda")
    q.tree_attention(cache, batch, to_dev(bits), out, tree, tree_mask=torch.from_numpy(masks).cuda(), scale=scale,
                     lse=lse, workspace=ws)
    torch.cuda.synchronize()
    got = bits16(out)
    return O.bf16_array(got), got, lse.cpu().numpy().astype(np.float64)


def seen_by(P, b, masks):
    n, t, first = P.lens[b], P.counts[b], int(P.start[b])
    seen = np.ones((t, n + t), bool)
    for i in range(t):
        seen[i, n:] = [bool(int(masks[first + i]) >> j & 1) for j in range(t)]
    return seen


def check_rows(P, x, masks, got, lse, ok, scale=None):
    """The rows ok [total][Hq] against the oracle."""
    scale = P.dim ** -0.5 if scale is None else scale
    for b, (n, t) in enumerate(zip(P.lens, P.counts)):
        rows = slice(int(P.start[b]), int(P.start[b]) + t)
        if not ok[rows].any():
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            ref, ref_lse, a, ds = U.attention(x[rows], P.stored(0, b, 0, n + t), P.stored(1, b, 0, n + t),
                                              seen_by(P, b, masks), scale)
        B, Bl = U.attention_bounds(a, ds, ref_lse, n + t, P.dim, P.fmt)
        check_bf16(got[rows][ok[rows]], ref[ok[rows]], B[ok[rows]], f"sequence {b}")
        off = np.abs(lse[rows] - ref_lse)[ok[rows]]
        assert (off <= Bl[ok[rows]]).all(), np.max(off / Bl[ok[rows]])


# (group, tokens per sequence, sequences, heads): 12 and 24 rows per unit, 72, 192, and calls of 2,560 and 2,592 rows
ROUTES = [(12, 1, 1, 2), (12, 2, 1, 2), (12, 6, 1, 2), (12, 16, 1, 1), (4, 4, 40, 4), (12, 6, 9, 4)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [9, 1300])
@pytest.mark.parametrize("group,t,lanes,heads", ROUTES)
def test_a_nan_query_gives_nan(fmt, n, group, t, lanes, heads):
    """A row of q that holds a NaN is NaN in out and lse, whether its keys were
    read by one CTA or by many; the other rows are as ever."""
    counts = [t] * lanes
    P = U.Paged(71, fmt, 64, 64, heads, [n] * lanes, counts)
    r = np.random.default_rng(72)
    masks = U.ancestor_masks(r, counts)
    x = O.round_bf16(r.standard_normal((P.total, group * heads, 64)))
    bad = np.zeros(x.shape[:2], bool)
    bad[::2, 1::3] = True
    x[bad, 17] = np.nan
    got, bits, lse = attend(P, x, masks)
    assert np.isnan(got[bad]).all() and np.isnan(lse[bad]).all()
    assert np.isfinite(got[~bad]).all() and np.isfinite(lse[~bad]).all()
    few = ~bad
    few[2 * t:] = False                                          # two sequences by the oracle
    check_rows(P, np.nan_to_num(x), masks, bits, lse, few)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [0, 40, 4096])
@pytest.mark.parametrize("group,t,lanes,heads", ROUTES)
def test_a_nan_key_gives_nan_to_the_rows_that_see_it(fmt, n, group, t, lanes, heads):
    """The key is the only one that its row sees in the last part of the unit
    (4,096 positions end with a step, and each draft sees itself alone)."""
    if n * lanes > 100000:
        n = 1024
    counts = [t] * lanes
    P = U.Paged(73, fmt, 64, 64, heads, [n] * lanes, counts)
    masks = own_only(counts)
    j = t - 1
    for b in range(lanes):
        pg, off = P.at(b, n + j, 1)
        codes, scales = P.parts[0]
        if fmt == "nvfp4":
            scales[pg, :, off] = 0x7F
        else:
            codes[pg, :, off, 5] = 0x7FC0 if fmt == "bf16" else 0x7F
    x = O.round_bf16(np.random.default_rng(74).standard_normal((P.total, group * heads, 64)))
    got, bits, lse = attend(P, x, masks)
    bad = np.zeros(x.shape[:2], bool)
    bad[P.start[1:] - 1] = True
    assert np.isnan(got[bad]).all() and np.isnan(lse[bad]).all()
    assert np.isfinite(got[~bad]).all() and np.isfinite(lse[~bad]).all()


@pytest.mark.parametrize("fmt", ("bf16", "fp8"))
@pytest.mark.parametrize("n", [128, 1024])
@pytest.mark.parametrize("group,t,lanes,heads", ROUTES)
def test_an_odd_value_arrives_however_small_its_weight(fmt, n, group, t, lanes, heads):
    """The last draft's value is infinite (FP8: NaN) and its weight is 2^-500 of
    the row's largest: the output that it belongs to is not finite, the others
    are. (At 128 positions the draft's part is a warp's only one in the join.)"""
    counts = [t] * lanes
    P = U.Paged(75, fmt, 64, 64, heads, [n] * lanes, counts)
    for b in range(lanes):
        for p, v in ((5, 4.0), (n + t - 1, -4.0)):
            codes, scales = U.quantise(np.full((1, heads, 64), v), fmt, 1.0)
            pg, off = P.at(b, p, 1)
            P.parts[0][0][pg, :, off] = codes
            if scales is not None:
                P.parts[0][1][pg, :, off] = scales
        P.parts[1][0][pg, :, off, 9] = 0x7F80 if fmt == "bf16" else 0x7F
    masks = own_only(counts)
    x = np.full((P.total, group * heads, 64), 6.0)               # scores 192 and -192, times log2(e)
    got, bits, lse = attend(P, x, masks)
    last = P.start[1:] - 1
    assert not np.isfinite(got[last][:, :, 9]).any()
    got[last, :, 9] = 0.0
    assert np.isfinite(got).all() and np.isfinite(lse).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 16, 45, 70, 640])
@pytest.mark.parametrize("back", [1, 2, 15, 33])
@pytest.mark.parametrize("dim,group,t", [(64, 2, 3), (128, 3, 5), (128, 8, 3), (64, 12, 5), (128, 40, 5), (256, 12, 3)])
def test_odd_values_of_the_context_reach_every_row(fmt, n, back, dim, group, t):
    """A value `back` positions before the drafts is NaN (and in bf16 another is
    infinite): every row sees the context, so every row has it."""
    if back > n:
        pytest.skip("no such position")
    P = U.Paged(76, fmt, dim, 16, 1, [n], [t])
    pg, off = P.at(0, n - back, 1)
    codes, scales = P.parts[1]
    want = np.zeros(dim, bool)
    if fmt == "nvfp4":
        scales[pg, :, off, 2] = 0x7F
        want[32:48] = True
    else:
        codes[pg, :, off, 7] = 0x7FC0 if fmt == "bf16" else 0x7F
        want[7] = True
    if fmt == "bf16":
        codes[pg, :, off, 11] = 0xFF80
    masks = U.ancestor_masks(np.random.default_rng(77), [t])
    masks[-1] = 0                                                # sees the context alone
    x = O.round_bf16(np.random.default_rng(78).standard_normal((t, group, dim)))
    got, _, lse = attend(P, x, masks)
    assert np.isnan(got[:, :, want]).all()
    if fmt == "bf16":
        assert (got[:, :, 11] == -np.inf).all()
        want[11] = True
    assert np.isfinite(got[:, :, ~want]).all() and np.isfinite(lse).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group", [2, 8, 12, 40])
def test_an_odd_value_beside_a_page_outside_the_cache(fmt, group):
    """A page of 16 keys lies outside the cache: its neighbours' NaN still
    reaches every row, and nothing of the page does."""
    P = U.Paged(79, fmt, 64, 16, 1, [200], [3])
    pg, off = P.at(0, 70, 1)                                     # page 4; page 5 shares a block of 32 keys with it
    codes, scales = P.parts[1]
    want = np.zeros(64, bool)
    if fmt == "nvfp4":
        scales[pg, :, off, 1] = 0x7F
        want[16:32] = True
    else:
        codes[pg, :, off, 20] = 0x7FC0 if fmt == "bf16" else 0x7F
        want[20] = True
    x = O.round_bf16(np.random.default_rng(80).standard_normal((3, group, 64)))

    def change(batch):
        batch.page_table[0, 5] = -1

    got, _, lse = attend(P, x, chains([3]), change=change)
    assert q.qg_last_device_status() == q.QG_ERR_INVALID_ARG
    assert np.isnan(got[:, :, want]).all()
    assert np.isfinite(got[:, :, ~want]).all() and np.isfinite(lse).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", [1e8, 1e9, 4e9, 1e12, 1e20])
@pytest.mark.parametrize("group,t,n", [(2, 3, 700), (12, 2, 700), (12, 6, 700), (12, 6, 5000), (40, 6, 700)])
def test_scores_far_beyond_the_exponentials_range(fmt, size, group, t, n):
    """Scores of about `size`: neighbours lie so far apart that each row's output
    is the value of its largest key, unless two are closer than the error of a
    32-bit score allows to tell (few rows). A score is off by at most
    ds (D + 10) 2^-22, as in kv_util.attention_bounds, the weight of the largest
    by half a step of its 16-bit type and 2^-20 for the sum and the exponential."""
    dim, g = 64, 1.0 if fmt == "bf16" else 4.0
    P = U.Paged(81, fmt, dim, 64, 1, [n], [t], kg=g, vg=g, std=1e3)
    r = np.random.default_rng(83)
    x = O.round_bf16(r.standard_normal((t, group, dim)) * size / 1e3)
    masks = U.ancestor_masks(r, [t])
    got, bits, lse = attend(P, x, masks)
    assert np.isfinite(got).all() and np.isfinite(lse).all()
    k, v = P.stored(0, 0, 0, n + t)[:, 0], P.stored(1, 0, 0, n + t)[:, 0]
    seen = seen_by(P, 0, masks)
    told = 0
    for i in range(t):
        keys = np.nonzero(seen[i])[0]
        for h in range(group):
            s = k[keys] @ x[i, h] * dim ** -0.5
            err = (np.abs(k[keys]) @ np.abs(x[i, h])).max() * dim ** -0.5 * (dim + 10) * 2.0 ** -22
            assert abs(lse[i, h] - s.max()) <= err + 2.0 ** -20 * abs(s.max()) + 20
            order = np.argsort(s)
            if s[order[-1]] - s[order[-2]] <= 2 * err + 40:
                continue
            told += 1
            ref = v[keys[order[-1]]]
            check_bf16(bits[i, h], ref, np.abs(ref) * (2.0 ** (-8 if fmt == "bf16" else -11) + 2.0 ** -20) + 1e-15)
    assert told > t * group // 2


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group,t", [(2, 1), (24, 1), (40, 1), (128, 2)])
def test_a_maximum_that_grows_by_eight_where_scores_are_whole(fmt, group, t):
    """Base-2 scores B + 8 in the first half of the context and B + 16 behind it,
    B = 2^24 or a little more, exact in 32 bits but without a bit to spare: the
    weights of the second half are 2^8 times those of the first, and no sum of a
    maximum and a small number is exact. Scores are exact here (scale = ln 2 in 32
    bits makes the factor 1), so only the weights' rounding is left of the bound."""
    dim, heads, lanes, n = 64, 4, 8, 6000
    if group * t > 32:
        lanes, n = 5, 4000
    P = U.Paged(84, fmt, dim, 64, heads, [n] * lanes, [t] * lanes)
    r = np.random.default_rng(85)
    for b in range(lanes):
        k = np.zeros((n + t, heads, dim))
        k[:, :, 0] = 66.0 if fmt == "nvfp4" else 64.0            # 6 times an E4M3 scale
        k[:, :, 16] = np.where(np.arange(n + t) < n // 2, 4.0, 8.0)[:, None]
        k[:, :, 17] = 12.0
        v = r.standard_normal((n + t, heads, dim)) * 100.0
        v[:, :, 0] = 300.0                                       # FP8: the same scale for every token, and it is 1
        v = np.clip(v, -300.0, 300.0)
        pg, off = P.at(b, 0, n + t)
        for kv, y in ((0, k), (1, O.round_bf16(v))):
            codes, scales = U.quantise(y, fmt, 1.0)
            P.parts[kv][0][pg, :, off] = codes
            if scales is not None:
                P.parts[kv][1][pg, :, off] = scales
        assert np.array_equal(P.stored(0, b, 0, n + t), k)
    x = np.zeros((P.total, heads * group, dim))
    x[:, :, 0], x[:, :, 16] = 2.0 ** 18, 2.0
    masks = chains(P.counts)
    scale = float(np.float32(np.log(2.0)))
    got, bits, lse = attend(P, x, masks, scale=scale)
    assert np.isfinite(got).all() and np.isfinite(lse).all()
    for b in range(lanes):
        rows = slice(int(P.start[b]), int(P.start[b]) + t)
        ref, ref_lse, a, _ = U.attention(x[rows, ::group], P.stored(0, b, 0, n + t), P.stored(1, b, 0, n + t),
                                         seen_by(P, b, masks), scale)
        B, _ = U.attention_bounds(a, np.zeros(ref_lse.shape), ref_lse, n + t, dim, fmt)
        # ln 2 is off by 2^-25: 8 of them in a ratio of weights
        B = B + a[0] * 2.0 ** -20
        for h in range(group):
            check_bf16(bits[rows, h::group], ref, B, f"sequence {b}")
            assert (np.abs(lse[rows, h::group] - ref_lse) <= 2.0 ** -20 * np.abs(ref_lse)).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,group,t", [(64, 2, 5), (128, 1, 1), (128, 4, 7), (64, 40, 2), (128, 12, 6), (128, 12, 20),
                                         (256, 8, 6)])
def test_a_row_that_sees_one_key_is_its_value(fmt, dim, group, t):
    """The one weight and the sum that divides are the same power of two, so the
    value comes back bit for bit (codes times scales are bf16 numbers here)."""
    P = U.Paged(86, fmt, dim, 16, 2, [0, 0], [t, t])
    masks = own_only(P.counts)
    x = O.round_bf16(np.random.default_rng(87).standard_normal((P.total, 2 * group, dim)))
    _, bits, _ = attend(P, x, masks)
    for b in range(2):
        v = P.stored(1, b, 0, t)
        assert np.array_equal(O.round_bf16(v), v)
        rows = slice(int(P.start[b]), int(P.start[b]) + t)
        assert np.array_equal(O.bf16_array(bits[rows]), np.repeat(v, group, axis=1))


@pytest.mark.parametrize("n", [9, 1300])
@pytest.mark.parametrize("left", [0, 1])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,t,lanes,heads", ROUTES)
def test_scores_of_minus_infinity(n, left, dim, group, t, lanes, heads):
    """Keys whose scores are -infinity have no weight: rows that see no others
    get zeros and -infinity, rows that see one other key get its value."""
    lanes = min(lanes, 9 if dim == 256 else lanes)
    P = U.Paged(88, "bf16", dim, 64, heads, [n] * lanes, [t] * lanes)
    for b in range(lanes):
        pg, off = P.at(b, 0, n + t)
        keep = P.parts[0][0][pg[1], :, off[1], 3].copy()
        P.parts[0][0][pg, :, off, 3] = 0xFF80
        if left:
            P.parts[0][0][pg[1], :, off[1], 3] = keep
    x = O.round_bf16(np.random.default_rng(89).standard_normal((P.total, group * heads, dim)))
    x[:, :, 3] = 2.0
    got, _, lse = attend(P, x, chains(P.counts))
    for b in range(lanes):
        rows = slice(int(P.start[b]), int(P.start[b]) + t)
        if not left:
            assert not got[rows].any() and (lse[rows] == -np.inf).all()
            continue
        v = np.repeat(P.stored(1, b, 1, 1), group, axis=1)
        assert np.array_equal(got[rows], np.repeat(v, t, axis=0)) and np.isfinite(lse[rows]).all()
