"""The sign of zero in what kv_cache_append writes (GPU): codes are compared bit
for bit with the plain forms of kv_util, on every way that a quotient takes."""
import numpy as np
import pytest

import kv_util as U
import oracle as O
from gpu_util import to_dev

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


@pytest.mark.parametrize("fmt", ("bf16", "fp8", "nvfp4"))
@pytest.mark.parametrize("g", [1.0, 0.75, 3.0, 1e-30])
@pytest.mark.parametrize("dim,tokens", [(64, 7), (128, 33), (256, 5), (128, 9000)])
def test_negative_zeros_keep_their_sign(fmt, g, dim, tokens):
    """Zeros of either sign among values of every size, rows of zeros alone, and
    values so small that their codes are zeros."""
    r = np.random.default_rng(61)
    size = 10.0 ** r.uniform(-4, 4, (tokens, 2, 1))
    size[1::5] = 10.0 ** r.uniform(-32, -19, size[1::5].shape)   # beyond what a reciprocal is used for
    x = r.standard_normal((tokens, 2, dim)) * size
    x[r.random(x.shape) < 0.1] *= 1e-8
    x[r.random(x.shape) < 0.2] = 0.0
    x[3::4, 1] = 0.0
    x = O.round_bf16(np.where((x == 0) & (r.random(x.shape) < 0.5), -0.0, x))
    assert (np.signbit(x) & (x == 0)).any()
    P = U.Paged(62, fmt, dim, 16, 2, [3], [tokens], kg=g, vg=2 * g)
    cache, batch = P.device(torch, q)
    d = to_dev(O.bf16_bits(x))
    q.kv_cache_append(cache, batch, d, d)
    pg, off = P.at(0, 3, tokens)
    for kv in (0, 1):
        codes, scales = U.quantise(x, fmt, P.g[kv])
        P.parts[kv][0][pg, :, off] = codes
        if scales is not None:
            P.parts[kv][1][pg, :, off] = scales
        got = P.host_part(cache, kv)
        assert np.array_equal(got[0], P.parts[kv][0])
        assert scales is None or np.array_equal(got[1], P.parts[kv][1])
