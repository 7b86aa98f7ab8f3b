"""Eviction from the paged cache (include/mla_chunk.h) on the GPU: which rows
are kept, where they go, and that every other byte stays, exactly."""
import numpy as np
import pytest

from chunk_testlib import ROW, Paged, put
from mla_testlib import ensure_built
from oracle import chunk as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import head_latent_attention_paged_gb300 as mod
    return mod


def _raw(paged):
    return paged.cache.cpu().numpy().view(np.uint8).reshape(paged.num_pages * paged.page, ROW[paged.kv])


def _run(m, paged, w, pos, budget, sinks=0, recent=0, in_place=False, status=0):
    """One eviction, compared with the oracle; returns the outputs."""
    B, S = w.shape
    plan = m.mla_evict_make_plan(paged.problem(m), budget, sinks, recent)
    ws = torch.full((max(16, int(plan.workspace_bytes)),), 0xFF, dtype=torch.uint8, device="cuda")
    lens, wg, pg, table = put(paged.lens, np.int32), put(w), put(pos), put(paged.table)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = _raw(paged).copy()
    if in_place:
        outs = [lens, wg, pg]
        fill_w, fill_p = w, pos
    else:
        outs = [torch.full_like(lens, -9), torch.full_like(wg, -9.0), torch.full_like(pg, -9)]
        fill_w, fill_p = np.full_like(w, -9.0), np.full_like(pos, -9)
    m.mla_cache_evict(plan, paged.cache, table, lens, wg, pg, ws, *outs, status=word)
    torch.cuda.synchronize()
    assert int(word) == status
    want, want_w, want_p, left = before.copy(), fill_w.copy(), fill_p.copy(), []
    for b, n in enumerate(paged.lens):
        kept, origin = C.evict(w[b, :n], pos[b, :n], budget, sinks, recent)
        left.append(kept)
        want_w[b, :kept], want_p[b, :kept] = w[b, origin], pos[b, origin]
        want_w[b, kept:n], want_p[b, kept:n] = 0.0, -1
        want[paged.slots[b][:kept]] = before[paged.slots[b][origin]]
    got_l, got_w, got_p = (t.cpu().numpy() for t in outs)
    assert got_l.tolist() == left
    assert np.array_equal(got_w.view(np.uint32), want_w.view(np.uint32))
    assert np.array_equal(got_p, want_p)
    assert np.array_equal(_raw(paged), want)
    return outs


def _weights(rng, B, S):
    w = np.exp(1.5 * rng.standard_normal((B, S), dtype=np.float32))
    w[w < 0.4] = 0.0                                   # many equal ones
    return w


CASES = [  # lengths, budget, sinks, recent
    ([1], 1, 0, 0),
    ([2], 1, 0, 0),
    ([2], 1, 0, 1),
    ([300], 128, 1, 17),
    ([0, 5, 127, 128, 129, 1000], 128, 4, 32),
    ([1000, 1023, 1025, 2049, 64], 1, 0, 0),
    ([5000], 4999, 0, 3),
    ([5000], 37, 50, 2),                               # more protected than the budget holds
    ([4160] * 5, 4096, 4, 256),
    ([70000], 4096, 4, 64),
    ([9000], 100, 0, 2**31 - 1),                       # all of them recent: the lowest slots
    (list(range(1, 140)), 50, 2, 8),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kv,page", [("bf16", 64), ("fp8", 16), ("fp4", 128), ("fp8", 64), ("bf16", 32)])
@pytest.mark.parametrize("lens,budget,sinks,recent", CASES)
def test_evict(m, lens, budget, sinks, recent, kv, page, in_place):
    rng = np.random.default_rng(len(lens) + budget)
    paged = Paged(rng, lens, page, kv)
    S = max(lens) + 3
    w = _weights(rng, len(lens), S)
    pos = np.broadcast_to(np.arange(S, dtype=np.int32), w.shape).copy()
    _run(m, paged, w, pos, budget, sinks, recent, in_place)


def test_evict_again_and_again(m):
    """Slots out of order from earlier evictions, rows appended behind them."""
    rng = np.random.default_rng(3)
    paged = Paged(rng, [700, 900, 650], 64, "fp8")
    w = _weights(rng, 3, 960)
    pos = np.broadcast_to(np.arange(960, dtype=np.int32), w.shape).copy()
    newest = np.array([699, 899, 649])
    for budget, more in ((600, 40), (600, 13), (580, 0), (580, 1)):
        outs = _run(m, paged, w, pos, budget, 4, 30, in_place=True)
        left, w, pos = (t.cpu().numpy() for t in outs)
        for b in range(3):                              # new tokens behind the kept ones
            n = left[b]
            w[b, n:n + more] = rng.random(more)
            pos[b, n:n + more] = newest[b] + 1 + np.arange(more)
            newest[b] += more
        paged.lens = left + more
        paged.raw = _raw(paged).copy()


def test_special_weights(m):
    """NaN least, -0 as 0, infinities, negative and subnormal weights."""
    rng = np.random.default_rng(5)
    paged = Paged(rng, [400], 16, "bf16")
    special = np.array([np.nan, -0.0, 0.0, np.inf, -np.inf, -1.0, 1e-42, -1e-42, -np.nan, 3e38], dtype=np.float32)
    w = np.tile(special, 40)[None]
    pos = np.arange(400, dtype=np.int32)[None]
    for budget in (1, 39, 41, 80, 81, 160, 200, 279, 320, 321, 399):
        paged = Paged(np.random.default_rng(5), [400], 16, "bf16")
        _run(m, paged, w, pos.copy(), budget, 0, 1)


def test_a_page_outside_the_pool_moves_nothing(m):
    rng = np.random.default_rng(6)
    paged = Paged(rng, [640], 64, "bf16")
    w = np.zeros((1, 640), dtype=np.float32)
    w[0, 320:] = 1.0                                   # the second half moves into the first
    pos = np.arange(640, dtype=np.int32)[None]
    table = paged.table.copy()
    table[0, 1], table[0, 7] = -1, paged.num_pages     # a page written to, and one read from
    plan = m.mla_evict_make_plan(paged.problem(m), 320)
    ws = torch.zeros(int(plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = _raw(paged).copy()
    m.mla_cache_evict(plan, paged.cache, put(table), put([640], np.int32), put(w), put(pos), ws,
                      torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, 640, device="cuda"),
                      torch.zeros(1, 640, dtype=torch.int32, device="cuda"), status=word)
    torch.cuda.synchronize()
    assert int(word) == m.MLA_STATUS_BAD_PAGE
    want = before.copy()
    for i in range(5):
        if i not in (1, 2):                            # page 1 cannot be written, page 2's rows are page 7's
            want[paged.slots[0][i * 64:(i + 1) * 64]] = before[paged.slots[0][(i + 5) * 64:(i + 6) * 64]]
    assert np.array_equal(_raw(paged), want)


def test_lengths_out_of_range_are_reported(m):
    rng = np.random.default_rng(7)
    paged = Paged(rng, [128, 128], 64, "bf16")
    plan = m.mla_evict_make_plan(paged.problem(m), 100)
    ws = torch.zeros(int(plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    word, left = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    w, pos = torch.rand(2, 120, device="cuda"), torch.arange(120, dtype=torch.int32, device="cuda").repeat(2, 1)
    m.mla_cache_evict(plan, paged.cache, put(paged.table), put([1 << 30, -7], np.int32), w, pos, ws, left, status=word)
    torch.cuda.synchronize()
    assert int(word) == m.MLA_STATUS_BAD_INDEX and left.tolist() == [100, 0]
