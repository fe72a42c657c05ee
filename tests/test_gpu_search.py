"""Beam search as a decode loop runs it (GPU): projections, cache, attention,
selection and pages of a small model, eager and as a replayed graph."""
import numpy as np
import pytest

import pages_util as PU
import synth
from gpu_util import nvfp4_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("bit_quantized_weight_gb300")

BEAMS, VOCAB, HIDDEN, HEADS, KV, DIM, PAGE = 8, 1008, 256, 4, 2, 64, 16
EOS, PAD = 77, 5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    yield
    assert q.qg_last_device_status() == q.QG_OK


class Model:
    """One layer: attention over the cache, its output added to the token's row, and the logits."""

    def __init__(self, fmt, pool):
        r = np.random.default_rng(31)
        self.qkv = nvfp4_dev(synth.nvfp4_weights(31, "search.qkv", (HEADS + 2 * KV) * DIM, HIDDEN, 0.1))
        self.head = nvfp4_dev(synth.nvfp4_weights(32, "search.head", VOCAB, HIDDEN, 0.05))
        self.embed = torch.from_numpy(r.standard_normal((VOCAB, HIDDEN))).cuda().bfloat16()
        self.rec = q.KVPages.empty(BEAMS, 12, pool, PAGE)
        self.cache = q.KVCache.empty(fmt, pool, PAGE, KV, DIM)
        self.batch = q.KVBatch(self.rec.page_table, self.rec.seq_lens, torch.arange(BEAMS + 1, dtype=torch.int32, device="cuda"), BEAMS)
        self.moves, self.left = q.KVMoves.empty(BEAMS), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.one = torch.ones(BEAMS, dtype=torch.int32, device="cuda")
        self.token = torch.zeros(BEAMS, dtype=torch.int32, device="cuda")
        self.x = torch.empty((BEAMS, HIDDEN), dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty((BEAMS, (HEADS + 2 * KV) * DIM), dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty((BEAMS, HEADS, DIM), dtype=torch.bfloat16, device="cuda")
        self.logits = torch.empty((BEAMS, VOCAB), dtype=torch.float32, device="cuda")
        self.ws = torch.empty(q.tree_attention_workspace_size(self.cache, HEADS, 1), dtype=torch.uint8, device="cuda")

    def step(self):
        """Logits of the next token after self.token, which the cache holds from now on."""
        torch.index_select(self.embed, 0, self.token, out=self.x)
        q.kv_pages_reserve(self.rec, self.one, self.moves, n_free=self.left)
        q.kv_pages_copy(self.cache, self.moves)
        q.qgemv_nvfp4(self.qkv["codes"], self.qkv["scales"], self.qkv["g"], self.x, self.y)
        heads = self.y.view(BEAMS, HEADS + 2 * KV, DIM)
        q.kv_cache_append(self.cache, self.batch, heads[:, HEADS:HEADS + KV], heads[:, HEADS + KV:])
        q.tree_attention(self.cache, self.batch, heads[:, :HEADS], self.out, 1, workspace=self.ws)
        self.rec.seq_lens.add_(1)
        self.x.add_(self.out.view(BEAMS, HIDDEN))
        q.qgemv_nvfp4(self.head["codes"], self.head["scales"], self.head["g"], self.x, self.logits)


class Search(Model):
    def __init__(self, fmt, pool):
        super().__init__(fmt, pool)
        self.scores = torch.full((1, BEAMS), -np.inf, device="cuda")
        self.scores[0, 0] = 0.0
        self.finished = torch.zeros((1, BEAMS), dtype=torch.bool, device="cuda")
        self.tokens, self.parents = (torch.zeros((1, BEAMS), dtype=torch.int32, device="cuda") for _ in range(2))
        self.select_ws = torch.empty(q.beam_select_workspace_size(1, BEAMS, VOCAB, BEAMS), dtype=torch.uint8, device="cuda")

    def step(self):
        super().step()
        q.beam_select(self.logits, self.scores, self.scores, self.tokens, self.parents, self.finished, finished=self.finished,
                      eos=EOS, pad=PAD, workspace=self.select_ws)
        q.kv_pages_fork(self.rec, self.parents.view(-1))
        self.token.copy_(self.tokens.view(-1))


def state(s):
    return [t.cpu().numpy().copy() for t in (s.scores, s.tokens, s.parents, s.finished)]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_search_keeps_the_best_and_their_histories(fmt):
    """60 steps. Each selection is the best of that step's logits; afterwards,
    every beam's tokens fed alone through sequences that share no page give the
    score that the search kept for it: each step adds one selection's bound and
    two roundings of the score (to fp32, and of the sum it is made from)."""
    s, steps = Search(fmt, 90), 60
    history, bound = [[] for _ in range(BEAMS)], np.zeros(BEAMS)
    for _ in range(steps):
        before = state(s)
        s.step()
        after = state(s)
        x = s.logits.cpu().numpy().astype(np.float64)
        PU.check_selection(x, before[0], before[3], EOS, PAD, after, BEAMS)
        assert int(s.left) >= 0
        p = after[2][0]
        bound = bound[p] + np.where(before[3][0][p], 0.0, PU.sum_bound(x)[p] + 2.0 ** -23 * np.abs(after[0][0]))
        history = [history[int(p[i])] + [(int(after[1][0, i]), bool(before[3][0, p[i]]))] for i in range(BEAMS)]
    final = state(s)[0][0]
    assert (s.rec.refs > 1).any() or len({tuple(h) for h in history}) == BEAMS
    alone, want = Model(fmt, 90), np.zeros(BEAMS)
    for k in range(steps):
        alone.step()
        z = alone.logits.cpu().numpy().astype(np.float64)
        z -= PU.log_sums(z)[:, None]
        token = [h[k][0] for h in history]
        want += [0.0 if h[k][1] else z[i, t] for i, (h, t) in enumerate(zip(history, token))]
        alone.token.copy_(torch.tensor(token, dtype=torch.int32))
    assert int((alone.rec.refs > 1).sum()) == 0
    assert (np.abs(final - want) <= bound).all(), (final - want, bound)
    q.kv_pages_fork(s.rec, torch.full((BEAMS,), -1, dtype=torch.int32, device="cuda"))
    assert not s.rec.refs.any() and not s.rec.n_pages.any()


def test_a_captured_step_searches_as_eager_ones_do():
    eager, s = Search("fp8", 90), Search("fp8", 90)
    warm = Search("fp8", 90)
    stream, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        warm.step()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        s.step()
    for _ in range(50):
        eager.step()
        g.replay()
        for a, b in zip((eager.scores, eager.tokens, eager.parents, eager.finished, eager.logits, *vars_of(eager.rec)),
                        (s.scores, s.tokens, s.parents, s.finished, s.logits, *vars_of(s.rec))):
            assert torch.equal(a, b)


def vars_of(rec):
    return rec.page_table, rec.seq_lens, rec.n_pages, rec.refs


def test_compaction_between_steps_changes_no_beam():
    a, b = Search("nvfp4", 90), Search("nvfp4", 90)
    list_, where = q.KVMoves.empty(90), torch.zeros(90, dtype=torch.int32, device="cuda")
    taken = torch.arange(0, 40, 2, device="cuda")
    b.rec.refs[taken] = 1                                    # pages of a prefix store, given back later
    for k in range(40):
        if k == 20:
            b.rec.refs[taken] = 0
        if k % 7 == 3:
            q.kv_pages_compact(b.rec, list_, where)
            q.kv_pages_copy(b.cache, list_)
            taken = where[taken].long() if k < 20 else taken
        a.step(), b.step()
        assert torch.equal(a.scores, b.scores) and torch.equal(a.tokens, b.tokens) and torch.equal(a.logits, b.logits)
    live = int((b.rec.refs != 0).sum())
    assert live == int((a.rec.refs != 0).sum())
