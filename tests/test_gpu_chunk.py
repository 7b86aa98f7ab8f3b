"""Attention of a chunk and the weights of cached rows (include/mla_chunk.h) on
the GPU against the float64 oracle, within bounds derived from the arithmetic
(oracle/chunk.py)."""
import numpy as np
import pytest

from chunk_testlib import Paged, f64, put
from mla_testlib import LSE_TOL, REL_L2, ensure_built
from oracle import chunk as C
from oracle import layer as L

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SCALE = 1.0 / 16.0


@pytest.fixture(scope="module")
def m():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import head_latent_attention_paged_gb300 as mod
    return mod


class Case:
    """New tokens and lengths [(n, T)] of each request, and the device's buffers."""

    def __init__(self, m, requests, heads, page, kv, causal=True, seed=0, lead=0, pad=0, spread=1.0, **kw):
        rng = np.random.default_rng(seed)
        self.m, self.heads, self.causal = m, heads, causal
        self.new = np.array([r[0] for r in requests], dtype=np.int64)
        self.paged = Paged(rng, [r[1] for r in requests], page, kv, **kw)
        self.starts = (lead + np.concatenate([[0], np.cumsum(self.new)])).astype(np.int32)
        self.tokens = int(self.starts[-1]) + pad
        q = rng.standard_normal((self.tokens, heads, 576), dtype=np.float32) * spread
        q[..., :512] *= 0.61
        self.q = torch.from_numpy(q).to(torch.bfloat16).cuda()
        self.problem = self.paged.problem(m, heads, causal=int(causal), sm_scale=SCALE)
        self.lens, self.table = put(self.paged.lens, np.int32), put(self.paged.table)
        self.starts_gpu = put(self.starts)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.make_plan()
        self.o = torch.full((max(self.tokens, 1), heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((max(self.tokens, 1), heads), 7.0, device="cuda")

    def make_plan(self, **kw):
        self.plan = self.m.mla_chunk_make_plan(self.problem, self.tokens,
                                               context_tokens=int(self.paged.lens.sum()), **kw)
        # nothing is read from a workspace that the call has not written
        self.workspace = torch.full((int(self.plan.workspace_bytes),), 0xFF, dtype=torch.uint8, device="cuda")

    def attend(self, stream=None):
        self.m.mla_chunk_attend(self.plan, self.q, self.starts_gpu, self.paged.cache, self.table, self.lens,
                                self.workspace, self.o, self.lse, status=self.status, stream=stream)

    def weigh(self, lse, out, into=None, stream=None):
        self.m.mla_cache_weights(self.plan, self.q, lse, self.starts_gpu, self.paged.cache, self.table, self.lens,
                                 self.workspace, out, weights_in=into, status=self.status, stream=stream)

    def queries(self, b):
        return f64(self.q[self.starts[b]:self.starts[b + 1]])

    def check_attention(self, status=0):
        torch.cuda.synchronize()
        assert int(self.status) == status
        o, lse = f64(self.o), f64(self.lse)
        for b, n in enumerate(self.new):
            part = slice(self.starts[b], self.starts[b + 1])
            ro, to, rl, tl = C.attend(self.queries(b), self.paged.rows(b), SCALE, self.causal)
            blind = np.isneginf(rl)
            assert np.all(np.isneginf(lse[part][blind])) and np.all(o[part][blind] == 0)
            assert np.all(np.abs(lse[part][~blind] - rl[~blind]) <= tl[~blind]), b
            L.assert_rounded(o[part], ro, to, "bf16", f"o of request {b}")
            if n and not blind.all():
                assert np.linalg.norm(o[part] - ro) <= REL_L2 * np.linalg.norm(ro)
                assert np.abs(lse[part][~blind] - rl[~blind]).max() <= LSE_TOL
        # what belongs to no request is as it was
        rest = np.ones(len(o), dtype=bool)
        rest[self.starts[0]:self.starts[-1]] = False
        assert np.all(o[rest] == 7.0) and np.all(lse[rest] == 7.0)


MIXED = [(5, 705), (0, 40), (1, 64), (130, 130), (7, 3), (1, 1), (0, 0), (2, 129)]
CASES = [  # requests (new, cached), heads, page
    ([(1, 1)], 1, 16),
    ([(1, 127), (1, 128), (1, 129), (1, 0)], 3, 64),
    (MIXED, 4, 64),
    (MIXED, 7, 16),
    (MIXED, 20, 32),
    ([(33, 1000)], 20, 128),
    ([(1, 2000), (2, 129), (64, 64)], 32, 32),
    ([(3, 300)], 128, 64),
    ([(1, 9000)], 20, 64),
    ([(700, 1500)], 20, 64),
    ([(64, 64), (13, 1024), (65, 4096)], 16, 128),
]


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("requests,heads,page", CASES)
def test_attention(m, requests, heads, page, kv):
    case = Case(m, requests, heads, page, kv, lead=2, pad=3)
    case.attend()
    case.check_attention()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_attention_not_causal(m, kv):
    case = Case(m, MIXED, 5, 64, kv, causal=False)
    case.attend()
    case.check_attention()


@pytest.mark.parametrize("sm_count", [1, 2, 7, 40, 152, 400])
def test_attention_does_not_depend_on_the_split(m, sm_count):
    case = Case(m, [(3, 3000), (40, 500), (1, 777)], 20, 64, "bf16", seed=4)
    case.make_plan(sm_count=sm_count)
    case.attend()
    case.check_attention()


def test_attention_of_many_requests(m):
    rng = np.random.default_rng(8)
    requests = [(int(n), int(n + c)) for n, c in zip(rng.integers(0, 9, 301), rng.integers(0, 200, 301))]
    case = Case(m, requests, 8, 16, "bf16", seed=8)
    case.attend()
    case.check_attention()


@pytest.mark.parametrize("spread", [8.0, 60.0])
def test_attention_of_steep_scores(m, spread):
    """Scores of hundreds: the running maximum grows again and again."""
    case = Case(m, [(20, 1500), (3, 400)], 20, 64, "bf16", seed=2, spread=spread)
    case.attend()
    case.check_attention()


def _weights(case, b, lse):
    part = slice(case.starts[b], case.starts[b + 1])
    return C.weights(case.queries(b), lse[part], case.paged.rows(b), SCALE, case.causal)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("requests,heads,page", CASES)
def test_weights(m, requests, heads, page, kv):
    case = Case(m, requests, heads, page, kv, seed=1)
    case.attend()
    lens = case.paged.lens
    width = int(lens.max()) + 5
    before = torch.rand(len(lens), width, device="cuda")
    for into in (None, before):
        out = torch.full((len(lens), width), 9.0, device="cuda")
        case.weigh(case.lse, out, into)
        torch.cuda.synchronize()
        assert int(case.status) == 0
        got, lse = f64(out), f64(case.lse)
        for b, n in enumerate(lens):
            w, t = _weights(case, b, lse)
            base = 0.0 if into is None else f64(before[b, :n])
            assert np.all(np.abs(got[b, :n] - base - w) <= t + 2 * C.U * (w + base)), b
            assert np.all(got[b, n:] == 9.0)
            if into is None and case.new[b] and n >= case.new[b]:   # every query gives one in all
                assert abs(got[b, :n].sum() - case.new[b] * heads) <= 1e-3 * case.new[b] * heads
    # in place, and the same bits again
    twice = before.clone()
    case.weigh(case.lse, twice, twice)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        assert torch.equal(twice[b, :n], out[b, :n]) and torch.equal(twice[b, n:], before[b, n:])


def test_weights_of_a_short_stride(m):
    """Slots from the stride on are neither read nor written."""
    case = Case(m, [(3, 300), (2, 90)], 4, 16, "bf16")
    case.attend()
    whole, part = torch.zeros(2, 300, device="cuda"), torch.full((2 * 100 + 7,), 9.0, device="cuda")
    case.weigh(case.lse, whole)
    case.m.mla_cache_weights(case.plan, case.q, case.lse, case.starts_gpu, case.paged.cache, case.table, case.lens,
                             case.workspace, part, stride=100)
    got = part[:200].view(2, 100)
    assert torch.equal(got[0], whole[0, :100]) and torch.equal(got[1, :90], whole[1, :90])
    assert torch.all(got[1, 90:] == 9.0) and torch.all(part[200:] == 9.0)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_page_outside_the_pool_is_masked(m, kv):
    case = Case(m, [(9, 500), (4, 200)], 6, 64, kv, seed=5)
    bad = case.paged.table.copy()
    bad[0, 2], bad[1, 0] = case.paged.num_pages, -1
    case.table.copy_(torch.from_numpy(bad))
    case.attend()
    torch.cuda.synchronize()
    assert int(case.status) == m.MLA_STATUS_BAD_PAGE
    o, lse = f64(case.o), f64(case.lse)
    out = torch.zeros(2, 500, device="cuda")
    case.weigh(case.lse, out)
    for b, page in ((0, 2), (1, 0)):
        part = slice(case.starts[b], case.starts[b + 1])
        rows, q = case.paged.rows(b), case.queries(b)
        live = np.ones(len(rows), dtype=bool)
        live[page * 64:(page + 1) * 64] = False
        for j, n in enumerate(C.seen(len(rows), len(q))):
            ro, to, rl, tl = C.attend(q[j:j + 1], rows[:n][live[:n]], SCALE, causal=False)
            assert np.all(np.abs(lse[part][j] - rl[0]) <= tl[0])
            L.assert_rounded(o[part][j], ro[0], to[0], "bf16")
        got = f64(out[b])
        assert np.all(got[:len(rows)][~live] == 0)
        w, t = C.weights(q, lse[part], rows, SCALE)
        assert np.all(np.abs(got[:len(rows)] - w)[live] <= (t + 2 * C.U * w)[live])


def test_starts_and_lengths_out_of_range_are_reported(m):
    case = Case(m, [(4, 100), (6, 50)], 4, 64, "bf16", seed=6)
    most = case.paged.max_pages * 64
    case.starts_gpu.copy_(torch.tensor([-3, 4, 1 << 30]))
    case.lens.copy_(torch.tensor([100, -5]))
    case.attend()
    torch.cuda.synchronize()
    assert int(case.status) == m.MLA_STATUS_BAD_INDEX and most >= 100
    ro, to, rl, tl = C.attend(case.queries(0), case.paged.rows(0), SCALE)
    L.assert_rounded(f64(case.o[:4]), ro, to, "bf16")
    assert torch.all(case.o[4:] == 0) and torch.all(torch.isinf(case.lse[4:]))


def test_fewer_expanded_rows_than_there_are(m):
    """A quantised cache's rows behind context_tokens are masked out."""
    case = Case(m, [(2, 90), (3, 200)], 4, 64, "fp8", seed=7)
    case.plan = m.mla_chunk_make_plan(case.problem, case.tokens, context_tokens=190)
    case.attend()
    torch.cuda.synchronize()
    assert int(case.status) == m.MLA_STATUS_BAD_INDEX
    ro, to, rl, tl = C.attend(case.queries(0), case.paged.rows(0), SCALE)
    L.assert_rounded(f64(case.o[:2]), ro, to, "bf16")
    ro, to, rl, tl = C.attend(case.queries(1), case.paged.rows(1)[:100], SCALE, causal=False)
    L.assert_rounded(f64(case.o[2:5]), ro, to, "bf16")
