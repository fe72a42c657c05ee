"""The paged cache (GPU): append, read and accept against the plain 64-bit
forms of kv_util. Codes, scales and moved rows are compared bit for bit, values
read back exactly (one fp32 rounding of an exact product, then bf16)."""
import numpy as np
import pytest

import kv_util as U
import oracle as O
from gpu_util import bits16, to_dev

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


FMTS = ("bf16", "fp8", "nvfp4")


def same_part(got, want):
    return np.array_equal(got[0], want[0]) and (want[1] is None or np.array_equal(got[1], want[1]))


def write(P, kv, b, first, x):
    """x [n][heads][dim] quantised into the host copy."""
    pg, off = P.at(b, first, len(x))
    codes, scales = U.quantise(x, P.fmt, P.g[kv])
    P.parts[kv][0][pg, :, off] = codes
    if scales is not None:
        P.parts[kv][1][pg, :, off] = scales


def spread(r, shape):
    """bf16 values over many magnitudes, zero rows and single-value rows among them."""
    x = r.standard_normal(shape) * 10 ** r.uniform(-6, 5, shape[:-1] + (1,))
    x[r.random(shape[:-1]) < 0.1] = 0.0
    x[r.random(shape) < 0.05] = 0.0
    return O.round_bf16(x)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,heads,page,lens,counts,g", [
    (128, 4, 64, [0], [1], 1.0),
    (64, 1, 16, [5, 0, 31], [3, 17, 1], 0.75),
    (128, 3, 48, [47, 48, 0, 100], [1, 0, 49, 2], 1.0),
    (256, 2, 32, [7] * 40, [2] * 40, 3.0),
    (128, 2, 256, [0, 1000], [700, 4], 0.0625),
])
def test_append_is_the_definition(fmt, dim, heads, page, lens, counts, g):
    P = U.Paged(1, fmt, dim, page, heads, lens, counts, kg=g, vg=2 * g)
    cache, batch = P.device(torch, q)
    r = np.random.default_rng(2)
    # rows lie apart, as columns of a wider projection
    wide = spread(r, (P.total, heads * 2 + 3, dim))
    w = to_dev(O.bf16_bits(wide))
    q.kv_cache_append(cache, batch, w[:, 1:1 + heads], w[:, 2 + heads:2 + 2 * heads])
    for b in range(len(lens)):
        rows = slice(P.start[b], P.start[b + 1])
        write(P, 0, b, lens[b], wide[rows, 1:1 + heads])
        write(P, 1, b, lens[b], wide[rows, 2 + heads:2 + 2 * heads])
    for kv in (0, 1):
        assert same_part(P.host_part(cache, kv), P.parts[kv])


@pytest.mark.parametrize("fmt", FMTS)
def test_append_ties_and_bounds(fmt):
    """Every rounding border: multiples of a half step around the codes, for
    each scale; values at and next to 448 * 2^s and 6 * scale."""
    dim, heads = 64, 1
    m = np.arange(128, 256)
    rows = []
    for top in (256, 255, 254, 224, 225, 223, 192, 168, 128, 129):
        for e in (-20, -14, -3, 0, 5, 9):
            x = np.zeros(64)
            x[0] = top * 2.0 ** e
            x[1:] = np.tile(m, 1)[::2][:63] * 2.0 ** (e - (np.arange(63) % 9)) * np.where(np.arange(63) % 2, 1, -1)
            x[16], x[32], x[48] = x[0] / 2, x[0] / 4, x[0] / 8
            rows.append(x)
    x = O.round_bf16(np.array(rows))[:, None, :]
    P = U.Paged(3, fmt, dim, 16, heads, [0], [len(rows)])
    cache, batch = P.device(torch, q)
    d = to_dev(O.bf16_bits(x))
    q.kv_cache_append(cache, batch, d, d)
    write(P, 0, 0, 0, x)
    write(P, 1, 0, 0, x)
    for kv in (0, 1):
        assert same_part(P.host_part(cache, kv), P.parts[kv])


@pytest.mark.parametrize("fmt", ("fp8", "nvfp4"))
def test_append_infinities_and_nan(fmt):
    x = np.zeros((6, 1, 64))
    x[0, 0, :] = np.linspace(-3, 3, 64)
    x[0, 0, 3] = np.inf
    x[1, 0, :] = 1.0
    x[1, 0, 40] = np.nan
    x[2, 0, :] = -np.inf
    x[3, 0, :] = np.nan
    x[4, 0, :] = O.bf16_array(np.full(64, 0x7F7F, np.uint16))
    x[5, 0, :] = O.bf16_array(np.arange(64, dtype=np.uint16))      # subnormal bf16
    x = np.where(np.isfinite(x), O.round_bf16(np.nan_to_num(x, posinf=0, neginf=0)), x)
    P = U.Paged(4, fmt, 64, 16, 1, [0], [6])
    cache, batch = P.device(torch, q)
    bits = O.bf16_bits(np.where(np.isnan(x), 0.0, x))
    bits[np.isnan(x)] = 0x7FC0
    d = to_dev(bits)
    q.kv_cache_append(cache, batch, d, d)
    k_out = torch.empty((6, 1, 64), dtype=torch.float32, device="cuda")
    v_out = torch.empty_like(k_out)
    q.kv_cache_read(cache, batch, k_out, v_out)
    codes, scales = U.quantise(x, fmt, 1.0)
    assert np.array_equal(k_out.cpu().numpy().astype(np.float64), U.values(codes, scales, fmt, 1.0), equal_nan=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,heads,page,lens,counts", [
    (128, 4, 64, [0], [1]),
    (64, 1, 16, [5, 0, 31], [3, 17, 1]),
    (256, 3, 48, [47, 48, 0, 100], [1, 0, 49, 2]),
    (128, 2, 256, [0, 1000], [1500, 4]),
    (64, 5, 16, list(range(70)), [1] * 70),
])
def test_read_is_the_stored_values(fmt, dim, heads, page, lens, counts):
    P = U.Paged(5, fmt, dim, page, heads, lens, counts, kg=0.3, vg=1.7)
    cache, batch = P.device(torch, q)
    want = [np.concatenate([P.stored(kv, b, n, t) for b, (n, t) in enumerate(zip(lens, counts))]) for kv in (0, 1)]
    for dt in (torch.float32, torch.bfloat16):
        outs = [torch.full((P.total, heads, dim), 7.0, dtype=dt, device="cuda") for _ in range(2)]
        q.kv_cache_read(cache, batch, *outs)
        for got, ref in zip(outs, want):
            # code * scale is exact, g enters with one fp32 rounding
            f32 = ref.astype(np.float32)
            if dt == torch.float32:
                assert np.array_equal(got.cpu().numpy(), f32)
            else:
                assert np.array_equal(bits16(got), O.bf16_bits(f32.astype(np.float64)))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,heads,page,lens,counts,kept", [
    (128, 4, 64, [100], [8], [3]),
    (64, 1, 16, [5, 0, 31, 9], [3, 17, 1, 4], [0, 17, 1, 2]),
    (256, 3, 48, [47, 48, 0], [64, 1, 64], [33, 1, 64]),
    (128, 8, 16, [3] * 33, [5] * 33, [2] * 33),
    (64, 2, 32, [11, 0], [300, 70], [150, 70]),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_accept_moves_the_path(fmt, dim, heads, page, lens, counts, kept, in_place):
    P = U.Paged(6, fmt, dim, page, heads, lens, counts)
    cache, batch = P.device(torch, q)
    r = np.random.default_rng(7)
    path = np.full(P.total, 99, np.int32)
    for b, (t, n) in enumerate(zip(counts, kept)):
        path[P.start[b]:P.start[b] + n] = np.sort(r.choice(t, n, replace=False))
    want_lens = np.array(lens) + kept
    for b, n in enumerate(kept):
        chosen = path[P.start[b]:P.start[b] + n]
        for part in P.parts:
            pg, off = P.at(b, lens[b], counts[b])
            tp, to = P.at(b, lens[b], n)
            for a in part:
                if a is not None:
                    a[tp, :, to] = a[pg, :, off][chosen]
    new_lens = batch.seq_lens if in_place else torch.full((len(lens),), -1, dtype=torch.int32, device="cuda")
    q.kv_cache_accept(cache, batch, torch.from_numpy(path).cuda(),
                      torch.tensor(kept, dtype=torch.int32, device="cuda"), new_lens)
    for kv in (0, 1):
        assert same_part(P.host_part(cache, kv), P.parts[kv])
    assert np.array_equal(new_lens.cpu().numpy(), want_lens)


def test_accept_refuses_a_bad_path_whole():
    lens, counts = [10, 10, 10, 10, 10], [6] * 5
    P = U.Paged(8, "fp8", 64, 16, 2, lens, counts)
    cache, batch = P.device(torch, q)
    path = np.tile(np.array([0, 2, 4, 0, 0, 0], np.int32), 5)
    path[6:9] = [0, 0, 4]           # below its index, not ascending
    path[12:15] = [0, 2, 6]         # beyond the sequence's tokens
    path[18:21] = [0, -2, 4]
    kept = torch.tensor([3, 3, 3, 3, 7], dtype=torch.int32, device="cuda")   # more than there are
    new = torch.zeros(5, dtype=torch.int32, device="cuda")
    q.kv_cache_accept(cache, batch, torch.from_numpy(path).cuda(), kept, new)
    assert q.qg_last_device_status() == q.QG_ERR_INVALID_ARG
    assert new.cpu().tolist() == [13, 10, 10, 10, 10]
    for part in P.parts:
        pg, off = P.at(0, 10, 6)
        tp, to = P.at(0, 10, 3)
        for a in part:
            a[tp, :, to] = a[pg, :, off][[0, 2, 4]]
    for kv in (0, 1):
        assert same_part(P.host_part(cache, kv), P.parts[kv])


def test_bad_device_data_is_left_out_and_recorded():
    """Sequences and pages that do not fit: the others are served, nothing
    else is written, rows behind the last sequence stay as they were."""
    lens, counts = [3, 20, 5, 40, 2], [2, 2, 2, 2, 2]
    P = U.Paged(9, "nvfp4", 64, 16, 1, lens, counts)
    cache, batch = P.device(torch, q)
    big = P.batch(torch, q, n_tokens=13)                     # three rows behind the last sequence
    big.seq_lens[1] = -1
    big.seq_lens[3] = P.max_pages * 16 - 1                   # one position too many
    big.page_table[4, 0] = P.pages                           # page outside the cache
    x = O.round_bf16(np.random.default_rng(10).standard_normal((13, 1, 64)))
    d = to_dev(O.bf16_bits(x))
    q.kv_cache_append(cache, big, d, d)
    assert q.qg_last_device_status() == q.QG_ERR_INVALID_ARG
    for b in (0, 2):
        for kv in (0, 1):
            write(P, kv, b, lens[b], x[2 * b:2 * b + 2])
    for kv in (0, 1):
        assert same_part(P.host_part(cache, kv), P.parts[kv])
    outs = [torch.full((13, 1, 64), 7.0, dtype=torch.float32, device="cuda") for _ in range(2)]
    q.kv_cache_read(cache, big, *outs)
    assert q.qg_last_device_status() == q.QG_ERR_INVALID_ARG
    for kv in (0, 1):
        got = outs[kv].cpu().numpy()
        for b in (0, 2):
            assert np.array_equal(got[2 * b:2 * b + 2], P.stored(kv, b, lens[b], 2).astype(np.float32))
        assert (got[[2, 3, 6, 7, 10, 11, 12]] == 7.0).all() and (got[8:10] == 0.0).all()


@pytest.mark.parametrize("starts", [[0, 4, 2, 6], [-1, 2, 4, 6], [0, 2, 4, 1 << 30], [6, 4, 2, 0]])
def test_bad_token_starts_touch_nothing_outside(starts):
    P = U.Paged(11, "fp8", 64, 16, 1, [1, 2, 3], [2, 2, 2])
    cache, batch = P.device(torch, q)
    batch.token_start.copy_(torch.tensor(starts, dtype=torch.int32))
    d = to_dev(O.bf16_bits(O.round_bf16(np.random.default_rng(12).standard_normal((6, 1, 64)))))
    q.kv_cache_append(cache, batch, d, d)
    assert q.qg_last_device_status() == q.QG_ERR_INVALID_ARG
    outs = [torch.zeros((6, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q.kv_cache_read(cache, batch, *outs)
    assert q.qg_last_device_status() == q.QG_ERR_INVALID_ARG
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    q.kv_cache_accept(cache, batch, torch.zeros(6, dtype=torch.int32, device="cuda"),
                      torch.ones(3, dtype=torch.int32, device="cuda"), new)
    assert q.qg_last_device_status() == q.QG_ERR_INVALID_ARG


def test_pool_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes: the last pages hold what is appended to them."""
    pages, page, heads, dim = 4200, 256, 8, 256
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("needs 12 GB of device memory")
    k = torch.empty((pages, heads, page, dim), dtype=torch.bfloat16, device="cuda")
    cache = q.KVCache("bf16", k, torch.empty_like(k))
    assert k.numel() * 2 > 2 ** 32
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    n = 2 * page + 5
    batch = q.KVBatch(table, torch.zeros(1, dtype=torch.int32, device="cuda"),
                      torch.tensor([0, n], dtype=torch.int32, device="cuda"), n)
    x = torch.randn((n, heads, dim), device="cuda").to(torch.bfloat16)
    y = torch.randn((n, heads, dim), device="cuda").to(torch.bfloat16)
    q.kv_cache_append(cache, batch, x, y)
    assert torch.equal(k[pages - 1, :, 3], x[3]) and torch.equal(cache.v[pages - 2, :, 4], y[2 * page + 4])
    a, b = torch.empty_like(x), torch.empty_like(x)
    q.kv_cache_read(cache, batch, a, b)
    assert torch.equal(a, x) and torch.equal(b, y)
    # and what attention reads there
    qq = torch.zeros((1, heads, dim), dtype=torch.bfloat16, device="cuda")
    one = q.KVBatch(table, torch.tensor([n - 1], dtype=torch.int32, device="cuda"),
                    torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1)
    out = torch.empty_like(qq)
    ws = torch.empty(q.tree_attention_workspace_size(cache, heads, 1), dtype=torch.uint8, device="cuda")
    q.tree_attention(cache, one, qq, out, 1, workspace=ws)
    mean = y.double().mean(0)
    assert (out[0].double() - mean).abs().max() < 2.0 ** -8 * mean.abs().max() + 2.0 ** -8


def test_guard_bands_stay_untouched():
    from gpu_util import guarded
    P = U.Paged(13, "fp8", 64, 16, 3, [9, 0], [3, 5])
    cache, batch = P.device(torch, q)
    k_out, c1 = guarded((8, 3, 64), torch.float32)
    v_out, c2 = guarded((8, 3, 64), torch.float32)
    q.kv_cache_read(cache, batch, k_out, v_out)
    kc, c3 = guarded(tuple(cache.k.shape), torch.uint8)
    ks, c4 = guarded(tuple(cache.k_scales.shape), torch.uint8)
    other = q.KVCache("fp8", kc, cache.v, ks, cache.v_scales)
    x = torch.randn((8, 3, 64), device="cuda").to(torch.bfloat16)
    q.kv_cache_append(other, batch, x, x)
    torch.cuda.synchronize()
    for c in (c1, c2, c3, c4):
        c()
