"""What include/mla_chunk.h allows beyond one call after another on small caches:
streams, graphs, shared pages, caches past 32-bit offsets, garbage in padding,
clusters without room for every slot's key."""
import numpy as np
import pytest

from chunk_testlib import ROW, Paged, f64, kind, put
from mla_testlib import ensure_built
from oracle import chunk as C
from oracle import layer as L
from test_gpu_chunk import SCALE, Case
from test_gpu_evict import _run, _weights

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import head_latent_attention_paged_gb300 as mod
    return mod


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_garbage_in_padding_reaches_nothing(m, kv):
    """Queries that belong to no request may be NaN; so may the lse of others' rows."""
    case = Case(m, [(3, 90), (70, 300), (1, 64)], 20, 64, kv, lead=5, pad=4)
    case.q[:5] = float("nan")
    case.q[-4:] = float("nan")
    case.attend()
    case.check_attention()
    case.lse[:5] = float("nan")
    case.lse[-4:] = float("nan")
    out = torch.full((3, 300), 9.0, device="cuda")
    case.weigh(case.lse, out)
    torch.cuda.synchronize()
    lse = f64(case.lse)
    for b, n in enumerate(case.paged.lens):
        part = slice(case.starts[b], case.starts[b + 1])
        w, t = C.weights(case.queries(b), lse[part], case.paged.rows(b), SCALE)
        assert np.all(np.abs(f64(out[b, :n]) - w) <= t + 2 * C.U * w) and torch.all(out[b, n:] == 9.0)


def test_a_query_that_saw_nothing_gives_nothing(m):
    case = Case(m, [(9, 4), (5, 0), (2, 200)], 7, 16, "bf16")
    case.attend()
    case.check_attention()
    assert torch.all(torch.isneginf(case.lse[:5]))
    out = torch.zeros(3, 200, device="cuda")
    case.weigh(case.lse, out)
    torch.cuda.synchronize()
    assert abs(float(out[0].sum()) - 4 * 7) < 1e-3 and float(out[1].abs().sum()) == 0


@pytest.mark.parametrize("sm_count", [2, 9, 152])
@pytest.mark.parametrize("kv", ["bf16", "fp4"])
def test_long_runs_of_rows_that_see_nothing(m, kv, sm_count):
    """More row tiles without any tile, one after another, than are handed on at once."""
    case = Case(m, [(40, 0), (300, 5), (12, 200), (200, 0), (90, 31)], 16, 32, kv, lead=1, pad=2)
    case.make_plan(sm_count=sm_count)
    case.attend()
    case.check_attention()


def test_requests_that_share_pages(m):
    """A prefix that several requests have in common is read in place."""
    case = Case(m, [(4, 200), (6, 200)], 8, 64, "bf16", seed=3)
    case.paged.table[1, :2] = case.paged.table[0, :2]
    case.paged.slots[1][:128] = case.paged.slots[0][:128]
    case.table.copy_(torch.from_numpy(case.paged.table))
    case.attend()
    case.check_attention()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_caches_past_32_bit_offsets(m, kv):
    """Rows whose byte offsets are beyond 2^32 (and 2^33 for bf16's values)."""
    page, slots = 64, {"bf16": 1 << 22, "fp8": 1 << 23, "fp4": 15 << 20}[kv]
    case = Case(m, [(3, 500), (20, 129)], 4, page, kv, seed=11)
    paged = case.paged
    pool = torch.zeros(slots * ROW[kv] // 2, dtype=torch.int16, device="cuda")
    tail = put(paged.raw.view(np.uint8).reshape(-1)).view(torch.int16)
    pool[-tail.numel():] = tail
    shift = slots // page - paged.num_pages
    paged.cache, paged.num_pages = pool, slots // page
    live = paged.table != 0x40000000
    paged.table[live] += shift
    case.table.copy_(torch.from_numpy(paged.table))
    case.problem = paged.problem(m, 4, sm_scale=SCALE)
    case.make_plan()
    case.attend()
    case.check_attention()
    out = torch.zeros(2, 500, device="cuda")
    case.weigh(case.lse, out)
    assert abs(float(out.sum()) - 23 * 4) < 1e-2
    # and an eviction moves them there
    plan = m.mla_evict_make_plan(case.problem, 100)
    ws = torch.zeros(int(plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    pos = torch.arange(500, dtype=torch.int32, device="cuda").repeat(2, 1)
    w = f64(out).astype(np.float32)
    m.mla_cache_evict(plan, pool, case.table, case.lens, out, pos, ws)
    torch.cuda.synchronize()
    got = pool[-tail.numel():].view(torch.uint8).cpu().numpy().reshape(-1, ROW[kv])
    raw = paged.raw.view(np.uint8).reshape(-1, ROW[kv])
    for b, n in enumerate((500, 129)):
        _, origin = C.evict(w[b, :n], np.arange(n), 100)
        assert np.array_equal(got[paged.slots[b][:100]], raw[paged.slots[b][origin]])
    assert int(pool[:-tail.numel()].abs().max()) == 0


def test_two_streams_at_once(m):
    """Calls on workspaces of their own overlap."""
    cases = [Case(m, [(200, 1500), (5, 900)], 20, 64, kv, seed=s) for s, kv in enumerate(("bf16", "fp8", "bf16"))]
    outs = [torch.zeros(2, 1500, device="cuda") for _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for case, out, stream in zip(cases, outs, streams):
            case.attend(stream)
            case.weigh(case.lse, out, stream=stream)
    torch.cuda.synchronize()
    for case, out in zip(cases, outs):
        case.check_attention()
        assert abs(float(out.sum()) - 205 * 20) < 1.0


def test_two_graphs_on_one_workspace(m):
    """Captured once each, replayed in turn on one stream, on new inputs."""
    a = Case(m, [(40, 600), (3, 300)], 20, 64, "fp8", seed=1)
    b = Case(m, [(7, 1000), (90, 400)], 20, 64, "fp8", seed=2)
    size = max(a.workspace.numel(), b.workspace.numel())
    a.workspace = b.workspace = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(2, 1000, device="cuda") for _ in range(2)]
    graphs = []
    for case, out in ((a, outs[0]), (b, outs[1])):
        case.attend()
        case.weigh(case.lse, out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            stream = torch.cuda.current_stream()
            case.attend(stream)
            case.weigh(case.lse, out, stream=stream)
        graphs.append(g)
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for case, out in ((a, outs[0]), (b, outs[1])):
            case.q.normal_(generator=gen).mul_(0.7)
            case.o.fill_(7.0)
            case.lse.fill_(7.0)
            out.zero_()
        for _ in range(2):
            for g in graphs:
                g.replay()
        for case, out in ((a, outs[0]), (b, outs[1])):
            case.check_attention()
            assert abs(float(out.sum()) - case.new.sum() * 20) < 0.5


def test_equal_calls_give_equal_bits(m):
    case = Case(m, [(100, 3000), (1, 5000), (33, 700)], 20, 64, "bf16", seed=9)
    got = []
    for _ in range(3):
        case.attend()
        out = torch.zeros(3, 5000, device="cuda")
        case.weigh(case.lse, out)
        torch.cuda.synchronize()
        got.append((case.o.clone(), case.lse.clone(), out))
    for o, lse, out in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(lse, got[0][1]) and torch.equal(out, got[0][2])


def test_no_tokens_still_copies_weights(m):
    """A step without any query: weights_out = weights_in."""
    paged = Paged(np.random.default_rng(0), [70, 0, 5], 16, "bf16")
    plan = m.mla_chunk_make_plan(paged.problem(m, 4), 0)
    ws = torch.zeros(int(plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    before, out = torch.rand(3, 80, device="cuda"), torch.full((3, 80), 9.0, device="cuda")
    m.mla_cache_weights(plan, None, None, put(np.zeros(4), np.int32), paged.cache, put(paged.table),
                        put(paged.lens, np.int32), ws, out, weights_in=before)
    torch.cuda.synchronize()
    for b, n in enumerate((70, 0, 5)):
        assert torch.equal(out[b, :n], before[b, :n]) and torch.all(out[b, n:] == 9.0)


def test_a_call_in_place_of_an_earlier_kernels_output(m):
    """Inputs that a kernel ahead on the stream writes are waited for."""
    case = Case(m, [(50, 800)], 20, 64, "bf16", seed=4)
    case.attend()
    torch.cuda.synchronize()
    want = case.o.clone()
    q = case.q.clone()
    for _ in range(5):
        case.q.zero_()
        case.o.zero_()
        torch.cuda._sleep(200000)
        case.q.copy_(q)
        case.attend()
        assert torch.equal(case.o, want)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_more_slots_than_keys_fit(m, in_place):
    """Slots beyond those whose keys a cluster keeps in shared memory."""
    rng = np.random.default_rng(12)
    paged = Paged(rng, [420000], 128, "fp4")
    w = _weights(rng, 1, 420000)
    pos = rng.permutation(420000).astype(np.int32)[None]
    _run(m, paged, w, pos, 100000, 4, 1000, in_place)


def test_evict_of_many_requests(m):
    rng = np.random.default_rng(13)
    lens = rng.integers(0, 200, 400)
    paged = Paged(rng, lens, 16, "fp4")
    w = _weights(rng, 400, 201)
    pos = np.broadcast_to(np.arange(201, dtype=np.int32), w.shape).copy()
    _run(m, paged, w, pos, 60, 2, 9)


def test_evict_in_a_graph(m):
    """Captured with outputs in place: replayed on a cache that has grown again."""
    rng = np.random.default_rng(14)
    paged = Paged(rng, [300, 200], 64, "bf16")
    plan = m.mla_evict_make_plan(paged.problem(m), 128, 4, 16)
    ws = torch.zeros(int(plan.workspace_bytes), dtype=torch.uint8, device="cuda")
    lens, table = put(paged.lens, np.int32), put(paged.table)
    w, pos = torch.rand(2, 300, device="cuda"), torch.arange(300, dtype=torch.int32, device="cuda").repeat(2, 1)
    cache, keep = paged.cache, paged.cache.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.mla_cache_evict(plan, cache, table, lens, w, pos, ws, stream=torch.cuda.current_stream())
    for n in ((300, 200), (129, 128), (5, 299)):
        weights = rng.random((2, 300), dtype=np.float32)
        n = np.minimum(n, paged.lens)
        cache.copy_(keep)
        lens.copy_(torch.from_numpy(n.astype(np.int32)))
        w.copy_(torch.from_numpy(weights))
        pos.copy_(torch.arange(300, dtype=torch.int32).repeat(2, 1))
        g.replay()
        torch.cuda.synchronize()
        got = cache.view(-1, 576).cpu().numpy()
        for b in range(2):
            kept, origin = C.evict(weights[b, :n[b]], np.arange(n[b]), 128, 4, 16)
            assert int(lens[b]) == kept
            assert np.array_equal(got[paged.slots[b][:kept]], paged.raw.view(np.int16)[paged.slots[b][origin]])
            assert np.array_equal(pos[b, :kept].cpu().numpy(), origin)
