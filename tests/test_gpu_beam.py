"""beam_select (GPU) against every candidate in 64 bits (pages_util)."""
import numpy as np
import pytest

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


def call(x, dtype, scores, n_out, finished=None, eos=-1, pad=0, apart=0, workspace=None):
    """x float64 [rows][vocab] (values of dtype); the outputs as numpy."""
    rows, V = x.shape
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    wide = torch.full((rows, V + apart), float("nan"), dtype=dt, device="cuda")
    wide[:, :V] = torch.from_numpy(x).cuda().to(dt)
    L, B = scores.shape
    s = torch.from_numpy(scores.astype(np.float32)).cuda()
    f = None if finished is None else torch.from_numpy(finished).cuda()
    out = (torch.full((L, n_out), 7.0, device="cuda"), torch.full((L, n_out), -3, dtype=torch.int32, device="cuda"),
           torch.full((L, n_out), -3, dtype=torch.int32, device="cuda"), torch.ones((L, n_out), dtype=torch.bool, device="cuda"))
    if workspace is None:
        workspace = torch.full((q.beam_select_workspace_size(L, B, V, n_out),), 0xFF, dtype=torch.uint8, device="cuda")
    q.beam_select(wide[:, :V], s, *out, finished=f, eos=eos, pad=pad, workspace=workspace)
    return [t.cpu().numpy() for t in out]


def logits(r, rows, V, dtype, spread=2.5):
    x = r.standard_normal((rows, V)) * spread
    x[r.integers(0, rows, rows * 3), r.integers(0, V, rows * 3)] += 8.0
    return O.round_bf16(x) if dtype == "bf16" else x.astype(np.float32).astype(np.float64)


def check(x, dtype, scores, n_out, finished=None, eos=-1, pad=0, apart=0, bad=False):
    got = call(x, dtype, scores, n_out, finished, eos, pad, apart)
    assert q.qg_last_device_status() == (q.QG_ERR_INVALID_ARG if bad else q.QG_OK)
    PU.check_selection(x, scores.astype(np.float32), finished, eos, pad, got, n_out)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lanes,beams,vocab,n_out,apart", [
    (1, 1, 1, 1, 0), (1, 1, 1, 64, 0), (2, 3, 2, 4, 0), (3, 1, 7, 5, 0), (1, 4, 8, 40, 3), (1, 2, 9, 2, 1), (2, 2, 31, 64, 0),
    (1, 8, 300, 8, 0), (5, 3, 1000, 6, 5), (1, 1, 8191, 64, 0), (1, 2, 8192, 33, 0), (1, 2, 8193, 32, 7),
    (2, 4, 50001, 8, 0), (1, 8, 65536, 8, 0), (4, 4, 100003, 8, 0), (1, 64, 5000, 64, 0), (37, 16, 700, 16, 2),
    (700, 1, 50, 3, 0), (1, 1, 262144, 1, 0), (1, 3, 300007, 64, 13),
])
def test_selection_is_the_best_of_all_candidates(dtype, lanes, beams, vocab, n_out, apart):
    r = np.random.default_rng(vocab + n_out)
    x = logits(r, lanes * beams, vocab, dtype)
    scores = -10 * r.random((lanes, beams))
    check(x, dtype, scores, n_out, apart=apart, eos=vocab // 2, pad=vocab - 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n_out", [1, 6, 32, 33, 64])
def test_orders_that_fill_every_list(dtype, n_out):
    """Logits that rise, fall, are all alike, or alike but for a few: the lists
    of best tokens overflow, or hold ties only."""
    V = 20000
    t = np.arange(V)
    rows = [t / 100.0, -t / 100.0, np.zeros(V), np.where(t % 5000 == 17, 1.0, 0.0), (t // 64) / 50.0, np.where(t < V - 3, 0.0, 1.0)]
    x = np.stack(rows)
    x = O.round_bf16(x) if dtype == "bf16" else x.astype(np.float32).astype(np.float64)
    for r in range(len(rows)):
        check(x[r:r + 1], dtype, np.zeros((1, 1)), n_out)
    check(x, dtype, np.zeros((2, 3)), n_out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masked_logits(dtype):
    """Rows and stretches of -infinity, of the type's lowest value, and next to it."""
    r = np.random.default_rng(3)
    V = 9001
    low = -float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).max)
    x = logits(r, 8, V, dtype)
    x[0] = -np.inf
    x[1, :] = low
    x[2, 5:] = -np.inf
    x[3, 8:] = low
    x[4, :8500] = -np.inf
    x[5, ::2] = low
    x[6] = -np.inf
    x[6, 8999] = 3.0
    x[7, :] = low
    x[7, 100] = -low                                         # one token has all the weight
    for n_out in (1, 7, 64):
        check(x, dtype, -np.arange(8.0).reshape(2, 4), n_out)
        check(x, dtype, -np.arange(8.0).reshape(8, 1), n_out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("what", ["nan", "-nan", "inf", "score nan", "score inf"])
def test_rows_without_a_sum_are_left_out_and_recorded(dtype, what):
    r = np.random.default_rng(4)
    x, scores = logits(r, 6, 12345, dtype), -r.random((2, 3))
    if what.startswith("score"):
        scores[0, 1] = float(what.split()[1])
    else:
        x[1, 12344 if what == "nan" else 77] = {"nan": np.nan, "-nan": -np.nan, "inf": np.inf}[what]
    got = check(x, dtype, scores, 8, bad=True)
    assert not (got[2] == 1).any()


def test_infinities_in_rows_that_do_not_count_do_not_matter():
    r = np.random.default_rng(5)
    x, scores = logits(r, 6, 5000, "bf16"), -r.random((2, 3))
    x[1], x[5] = np.nan, np.inf
    scores[0, 1] = -np.inf
    finished = np.zeros((2, 3), bool)
    finished[1, 2] = True
    check(x, "bf16", scores, 5, finished=finished, pad=9)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_finished_dead_and_missing_candidates(dtype):
    r = np.random.default_rng(6)
    V = 3
    x = logits(r, 12, V, dtype)
    scores = -5 * r.random((3, 4))
    finished = np.zeros((3, 4), bool)
    finished[0] = True                                       # four candidates of the lane in all
    finished[1, 1] = True
    scores[1, 3] = -np.inf
    scores[2] = -np.inf                                      # none at all
    finished[2, 0] = True                                    # finished and dead
    for n_out in (1, 4, 5, 17):
        check(x, dtype, scores, n_out, finished=finished, eos=1, pad=2)


def test_ties_between_rows_go_to_the_lower_row_whatever_its_alignment():
    """Equal rows get equal sums: an odd vocabulary puts each at another alignment."""
    for dtype, V in (("bf16", 9001), ("fp32", 8195), ("bf16", 50007)):
        one = logits(np.random.default_rng(7), 1, V, dtype)
        got = check(np.repeat(one, 8, 0), dtype, np.full((1, 8), -1.25), 24)
        for o in range(24):
            assert got[2][0, o] == o % 8
        assert (got[0][0].reshape(3, 8) == got[0][0].reshape(3, 8)[:, :1]).all()


def test_scores_far_apart_and_equal():
    r = np.random.default_rng(8)
    x = logits(r, 4, 1000, "fp32")
    check(x, "fp32", np.array([[0.0, -1e30, -3e38, -50.0]]), 64)
    check(np.zeros((4, 16)), "fp32", np.zeros((1, 4)), 64)
    check(-np.zeros((1, 16)) * np.where(np.arange(16) % 2, 1.0, -1.0), "fp32", np.zeros((1, 1)), 16)   # zeros of both signs


def test_same_bits_every_time_and_in_place():
    r = np.random.default_rng(9)
    x = logits(r, 32, 30011, "bf16")
    scores = -r.random((4, 8))
    first = call(x, "bf16", scores, 8)
    for _ in range(5):
        assert all(np.array_equal(a, b) for a, b in zip(first, call(x, "bf16", scores, 8)))
    d = to_dev(O.bf16_bits(x))
    s = torch.from_numpy(scores.astype(np.float32)).cuda()
    f = torch.zeros((4, 8), dtype=torch.bool, device="cuda")
    t, p = (torch.zeros((4, 8), dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.empty(q.beam_select_workspace_size(4, 8, 30011, 8), dtype=torch.uint8, device="cuda")
    q.beam_select(d, s, s, t, p, f, finished=f, workspace=ws)
    for got, want in zip((s, t, p, f), first):
        assert np.array_equal(got.cpu().numpy(), want)
    with pytest.raises(q.QGemvError):
        big = torch.empty((4, 9), device="cuda")
        q.beam_select(d, s, big[:, :8].contiguous(), t, p, f, finished=f, workspace=ws[:64])


def test_guard_bands_stay_untouched():
    r = np.random.default_rng(10)
    x, scores = logits(r, 6, 4099, "fp32"), -r.random((2, 3))
    s, c0 = guarded((2, 3), torch.float32)
    s.copy_(torch.from_numpy(scores))
    d, c1 = guarded((6, 4099), torch.float32)
    d.copy_(torch.from_numpy(x))
    outs = [guarded((2, 5), t) for t in (torch.float32, torch.int32, torch.int32, torch.uint8)]
    need = q.beam_select_workspace_size(2, 3, 4099, 5)
    ws, c2 = guarded((need,), torch.uint8)
    q.beam_select(d, s, *(o for o, _ in outs), workspace=ws)
    torch.cuda.synchronize()
    for c in [c0, c1, c2] + [c for _, c in outs]:
        c()
    PU.check_selection(x, scores.astype(np.float32), None, -1, 0, [o.cpu().numpy() for o, _ in outs], 5)


def test_streams_and_graphs():
    """A call on a stream of its own, and two captured calls that share a workspace."""
    r = np.random.default_rng(11)
    xs = [logits(r, 8, 20011, "bf16") for _ in range(3)]
    scores = -r.random((1, 8))
    want = [call(x, "bf16", scores, 8) for x in xs]
    d = torch.empty((8, 20011), dtype=torch.bfloat16, device="cuda")
    s0 = torch.from_numpy(scores.astype(np.float32)).cuda()
    ws = torch.empty(q.beam_select_workspace_size(1, 8, 20011, 8), dtype=torch.uint8, device="cuda")
    outs = [(torch.zeros((1, 8), device="cuda"), *(torch.zeros((1, 8), dtype=torch.int32, device="cuda") for _ in range(2)),
             torch.zeros((1, 8), dtype=torch.bool, device="cuda")) for _ in range(2)]
    side = torch.cuda.Stream()
    d.copy_(to_dev(O.bf16_bits(xs[0])))
    torch.cuda.synchronize()
    q.beam_select(d, s0, *outs[0], workspace=ws, stream=side)
    torch.cuda.synchronize()
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(outs[0], want[0]))
    graphs = []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            q.beam_select(d, s0, *out, workspace=ws)
        graphs.append(g)
    for i, x in enumerate(xs):
        d.copy_(to_dev(O.bf16_bits(x)))
        for g, out in zip(graphs, outs):
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(out, want[i]))


def test_offsets_beyond_32_bits():
    """Rows far apart: the last ones start behind 2^32 bytes."""
    if torch.cuda.mem_get_info()[0] < 12 * 2 ** 30:
        pytest.skip("needs 12 GB of device memory")
    rows, V, stride = 24, 1001, 100_000_003
    flat = torch.zeros((rows - 1) * stride + V, dtype=torch.bfloat16, device="cuda")
    d = flat.as_strided((rows, V), (stride, 1))
    x = logits(np.random.default_rng(12), rows, V, "bf16")
    d.copy_(torch.from_numpy(x).to(torch.bfloat16))
    scores = -np.random.default_rng(13).random((3, 8))
    out = [torch.zeros((3, 8), device="cuda"), *(torch.zeros((3, 8), dtype=torch.int32, device="cuda") for _ in range(2)),
           torch.zeros((3, 8), dtype=torch.bool, device="cuda")]
    ws = torch.empty(q.beam_select_workspace_size(3, 8, V, 8), dtype=torch.uint8, device="cuda")
    q.beam_select(d, torch.from_numpy(scores.astype(np.float32)).cuda(), *out, workspace=ws)
    PU.check_selection(x, scores.astype(np.float32), None, -1, 0, [o.cpu().numpy() for o in out], 8)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lanes,beams,vocab,n_out,apart", [
    (5, 8, 40001, 8, 0), (700, 2, 4097, 5, 3), (9, 64, 12288, 64, 0), (153, 4, 8199, 33, 1), (3, 5, 400000, 12, 5), (2, 1, 5000011, 16, 0),
    (1300, 1, 8192, 8, 8),
])
def test_selection_over_many_logits(dtype, lanes, beams, vocab, n_out, apart):
    """Calls whose blocks take parts of rows one after another, some of them skipped."""
    r = np.random.default_rng(vocab)
    x = logits(r, lanes * beams, vocab, dtype)
    scores = -10 * r.random((lanes, beams))
    scores[r.random((lanes, beams)) < 0.1] = -np.inf
    check(x, dtype, scores, n_out, finished=r.random((lanes, beams)) < 0.2, apart=apart, eos=vocab // 2, pad=vocab - 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n_out", [1, 33, 64])
def test_orders_that_fill_every_list_of_many_logits(dtype, n_out):
    V, copies = 60001, 16
    t = np.arange(V)
    rows = [t / 400.0, -t / 400.0, np.zeros(V), np.where(t % 5000 == 17, 1.0, 0.0), (t // 64) / 50.0, np.where(t < V - 3, 0.0, 1.0)]
    x = np.stack(rows)
    x = O.round_bf16(x) if dtype == "bf16" else x.astype(np.float32).astype(np.float64)
    got = check(np.repeat(x, copies, 0), dtype, np.zeros((6, copies)), n_out)
    # rows of a lane are equal and so are their sums, whatever their alignment: by logit, then row, then token
    for lane in range(6):
        best = np.lexsort((t, -x[lane]))[:n_out]
        order = sorted((-x[lane, k], row, k) for k in best for row in range(copies))[:n_out]
        assert got[1][lane].tolist() == [k for _, _, k in order]
        assert got[2][lane].tolist() == [lane * copies + row for _, row, _ in order]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_logits_masked_and_without_a_sum(dtype):
    r = np.random.default_rng(21)
    V, low = 50003, -float(torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).max)
    x, scores = logits(r, 128, V, dtype), -r.random((16, 8))
    x[3] = -np.inf
    x[4, :40000], x[5, 40000:], x[6] = -np.inf, -np.inf, low
    x[7, ::2], x[8, 5:] = low, low
    check(x, dtype, scores, 9)
    x[60, V - 1], x[61, 0], x[62, 30000], scores[9, 1] = np.nan, np.inf, -np.nan, np.inf
    got = check(x, dtype, scores, 9, bad=True)
    assert not np.isin(got[2], [60, 61, 62, 73]).any()


def test_many_logits_give_the_same_bits_every_time():
    r = np.random.default_rng(22)
    x, scores = logits(r, 160, 40011, "fp32"), -r.random((20, 8))
    first = call(x, "fp32", scores, 8)
    for _ in range(5):
        assert all(np.array_equal(a, b) for a, b in zip(first, call(x, "fp32", scores, 8)))


@pytest.mark.parametrize("lanes,beams,vocab,n_out", [(400, 64, 40, 64), (5000, 3, 7, 4), (1, 1, 1 << 24, 4), (1, 64, 70001, 64)])
def test_sizes_at_the_limits(lanes, beams, vocab, n_out):
    r = np.random.default_rng(23)
    x = logits(r, lanes * beams, vocab, "bf16")
    x[-1, -1] = 40.0                                         # the last token of the last row
    check(x, "bf16", -3 * r.random((lanes, beams)), n_out, eos=vocab - 1)


def test_a_row_of_the_largest_call():
    """65,536 rows; the first and the last are looked at."""
    x = torch.zeros((65536, 5), dtype=torch.float32, device="cuda")
    x[0], x[-1] = torch.tensor([0.0, 3, 1, 2, -1]).cuda(), torch.tensor([5.0, 3, 1, 9, -1]).cuda()
    s, out = torch.zeros((65536, 1), device="cuda"), [torch.empty((65536, 3), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    q.beam_select(x, s, *out, workspace=torch.empty(q.beam_select_workspace_size(65536, 1, 5, 3), dtype=torch.uint8, device="cuda"))
    assert out[1][0].tolist() == [1, 3, 2] and out[1][-1].tolist() == [3, 0, 1] and out[1][7].tolist() == [0, 1, 2]
    assert bool((out[2] == torch.arange(65536, device="cuda")[:, None]).all())


def test_what_the_binding_refuses_and_takes():
    x, s = torch.zeros((8, 33), device="cuda"), torch.zeros((2, 4), device="cuda")
    o, t, p = (torch.zeros((2, 4), dtype=d, device="cuda") for d in (torch.float32, torch.int32, torch.int32))
    f, ws = torch.zeros((2, 4), dtype=torch.bool, device="cuda"), torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    ok = dict(logits=x, scores=s, out_scores=o, out_tokens=t, out_parents=p, out_finished=f, finished=f.clone(), workspace=ws)
    for bad in (dict(logits=x.cpu()), dict(logits=x.half()), dict(logits=x[:7]), dict(logits=x.view(-1)), dict(logits=x.t().contiguous().t()),
                dict(scores=s.cpu()), dict(scores=s.double()), dict(scores=s.t().contiguous().t()), dict(scores=s.view(-1)),
                dict(out_scores=o[:1]), dict(out_scores=o.half()), dict(out_tokens=t.long()), dict(out_tokens=t[:, :3]),
                dict(out_parents=p.cpu()), dict(out_parents=p.view(4, 2)), dict(out_finished=f.int()), dict(out_finished=f[:1]),
                dict(finished=f.float()), dict(finished=f.view(-1)), dict(finished=f.cpu()), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            q.beam_select(**{**ok, **bad})
    for bad in (dict(workspace=None), dict(workspace=ws[:8]), dict(eos=33), dict(pad=-1), dict(logits=x.view(-1)[1:].as_strided((8, 32), (32, 1)))):
        with pytest.raises(q.QGemvError):
            q.beam_select(**{**ok, **bad})
    q.beam_select(**{**ok, "out_finished": None, "finished": None})
    q.beam_select(**{**ok, "out_finished": None, "finished": torch.full((2, 4), 2, dtype=torch.uint8, device="cuda"), "pad": 9})
    assert bool((t == 9).all()) and p.tolist() == [[0, 1, 2, 3], [4, 5, 6, 7]]
