"""beam_select (GPU) where its bounds could fail it."""
import numpy as np
import pytest

import pages_util as PU

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


def graph_us(f, calls=4):
    """Microseconds of a call in a replayed graph, the best of ten replays."""
    stream, g, times = torch.cuda.Stream(), torch.cuda.CUDAGraph(), []
    with torch.cuda.stream(stream):
        f()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        for _ in range(calls):
            f()
    for _ in range(12):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1000 / calls)
    return min(times[2:])


def test_the_second_bound_does_not_lose_the_first():
    """64 beams with the same twelve likely tokens, next to each other, of which
    few lanes see one: a bound from the lanes' best tokens alone lies among the
    unlikely ones, more than the join can list, and it reads all pieces again
    for each of 64 outputs (43 times the time that tokens in different places
    take). One pass more, with bounds that hold, costs less than the whole
    call: twice is allowed for it, and once more for the noise of a shared GPU."""
    r = np.random.default_rng(51)
    B, V, N, us = 64, 50257, 64, []
    scores = -r.random((1, B)).astype(np.float32)
    for places in (lambda: np.arange(12), lambda: r.choice(V, 12, replace=False)):
        x = r.standard_normal((B, V)).astype(np.float32)
        for row in x:
            row[places()] = 12 + 4 * r.random(12)
        d, s = torch.from_numpy(x).cuda(), torch.from_numpy(scores).cuda()
        out = [torch.zeros((1, N), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32, torch.bool)]
        ws = torch.empty(q.beam_select_workspace_size(1, B, V, N), dtype=torch.uint8, device="cuda")
        us.append(graph_us(lambda: q.beam_select(d, s, *out, workspace=ws)))
        PU.check_selection(x, scores, None, -1, 0, [t.cpu().numpy() for t in out], N)
    assert us[0] <= 3 * us[1], us


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,step", [(4096, 4096, 1), (40, 300007, 7500)])
def test_sums_of_equal_terms_are_exact_but_for_the_logarithm(dtype, rows, vocab, step):
    """Row r has 1 + r step zeros, the rest -infinity: every exponential is 2^0
    = 1 or 0 and every partial sum a whole number below 2^24, so that a score is
    -ln(1 + r step) but for the logarithm (2^-23) and the rounding of the score."""
    count = 1 + step * torch.arange(rows, device="cuda")
    x = torch.where(torch.arange(vocab, device="cuda") < count[:, None], 0.0, -np.inf).to(dtype)
    out = [torch.zeros((rows, 1), dtype=t, device="cuda") for t in (torch.float32, torch.int32, torch.int32)]
    ws = torch.empty(q.beam_select_workspace_size(rows, 1, vocab, 1), dtype=torch.uint8, device="cuda")
    q.beam_select(x, torch.zeros((rows, 1), device="cuda"), *out, workspace=ws)
    want = -np.log(count.cpu().numpy().astype(np.float64))
    assert (np.abs(out[0][:, 0].cpu().numpy() - want) <= 2.0 ** -23 + 2.0 ** -24 * np.abs(want)).all()
    assert not out[1].any() and torch.equal(out[2][:, 0], torch.arange(rows, dtype=torch.int32, device="cuda"))
