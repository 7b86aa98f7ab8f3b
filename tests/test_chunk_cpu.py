"""The operators of include/mla_chunk.h without a GPU: plans, refusals before any
CUDA call, and the oracle against independent forms."""
import ctypes

import numpy as np
import pytest

from oracle import chunk as C


@pytest.fixture(scope="module")
def m():
    from head_latent_attention_paged_gb300 import _build
    _build.build()
    import head_latent_attention_paged_gb300 as mod
    mod.load()
    return mod


def _problem(m, batch=4, heads=20, page=64, num_pages=100, max_pages=30, **kw):
    return m.make_problem(batch, 1, heads, page, num_pages, max_pages, **kw)


def _code(m, fn, *args, **kw):
    with pytest.raises(m.MlaError) as e:
        fn(*args, **kw)
    return e.value.code


# ---------------------------------------------------------------- plans
def test_chunk_plan(m):
    p = m.mla_chunk_make_plan(_problem(m), 1000)
    assert p.tokens == 1000 and p.clusters == 76 and p.context_tokens == 0
    offsets = [p.ws_partial_o, p.ws_partial_lse, p.ws_segments, p.ws_starts, p.ws_rows, p.workspace_bytes]
    assert offsets == sorted(offsets) and all(x % 256 == 0 for x in offsets)
    assert p.ws_partial_lse >= 152 * 128 * 512 * 4 and p.ws_starts - p.ws_segments >= 152 * 16
    q = m.mla_chunk_make_plan(_problem(m, kv_dtype=m.MLA_KV_FP8_E4M3_E8M0), 1000, context_tokens=777)
    assert q.workspace_bytes - q.ws_rows >= (777 + 4 * 31) * 1152 and q.ws_rows - q.ws_starts >= 5 * 8
    # a bf16 cache is read in place: nothing is set aside for its rows
    assert m.mla_chunk_make_plan(_problem(m), 1000, context_tokens=777).workspace_bytes == p.workspace_bytes
    assert m.mla_chunk_make_plan(_problem(m), 0, sm_count=1).clusters == 1


@pytest.mark.parametrize("change,code", [
    (dict(heads=0), -1), (dict(heads=129), -2), (dict(batch=-1), -1), (dict(page=48), -2), (dict(num_pages=0), -1),
    (dict(topk_width=128), -2), (dict(causal=2), -1), (dict(sm_scale=0.0), -1), (dict(sm_scale=float("nan")), -1),
    (dict(kv_lora_rank=256), -2), (dict(kv_dtype=3), -2), (dict(max_pages=1 << 26), -2)])
def test_chunk_plan_refuses_problems(m, change, code):
    assert _code(m, m.mla_chunk_make_plan, _problem(m, **change), 10) == code


def test_chunk_plan_refuses_sizes(m):
    fp8 = _problem(m, kv_dtype=m.MLA_KV_FP8_E4M3_E8M0)
    assert _code(m, m.mla_chunk_make_plan, _problem(m), -1) == m.MLA_ERR_INVALID_ARGUMENT
    assert _code(m, m.mla_chunk_make_plan, _problem(m), 10, sm_count=0) == m.MLA_ERR_INVALID_ARGUMENT
    assert _code(m, m.mla_chunk_make_plan, fp8, 10, context_tokens=-1) == m.MLA_ERR_INVALID_ARGUMENT
    assert _code(m, m.mla_chunk_make_plan, _problem(m, heads=128), 1 << 24) == m.MLA_ERR_UNSUPPORTED
    assert _code(m, m.mla_chunk_make_plan, fp8, 10, context_tokens=1 << 31) == m.MLA_ERR_UNSUPPORTED
    assert m.load().mla_chunk_make_plan(None, 1, 0, 152, None, None) == m.MLA_ERR_INVALID_ARGUMENT


def test_evict_plan(m):
    p = m.mla_evict_make_plan(_problem(m), 100, 4, 8)     # 1920 slots a request
    assert p.most_moves == 100 and p.workspace_bytes >= 4 * 4 + 4 * 100 * 8
    assert m.mla_evict_make_plan(_problem(m), 1900).most_moves == 20
    assert m.mla_evict_make_plan(_problem(m), 5000).most_moves == 0
    for bad in (dict(budget=0), dict(budget=1, sinks=-1), dict(budget=1, recent=-1)):
        assert _code(m, m.mla_evict_make_plan, _problem(m), **bad) == m.MLA_ERR_INVALID_ARGUMENT
    assert _code(m, m.mla_evict_make_plan, _problem(m, page=8), 1) == m.MLA_ERR_UNSUPPORTED


# ---------------------------------------------------------------- refusals
# addresses that no call may reach: every case is refused by its arguments
A = [0x7F0000000000 + (i << 32) for i in range(16)]


def _attend(m, **kw):
    plan = kw.pop("plan", None) or m.mla_chunk_make_plan(_problem(m), 10)
    a = dict(q=A[0], starts=A[1], cache=A[2], table=A[3], lens=A[4], ws=A[5], o=A[6], lse=A[7], status=None,
             size=plan.workspace_bytes)
    a.update(kw)
    m.mla_chunk_attend(plan, a["q"], a["starts"], a["cache"], a["table"], a["lens"], a["ws"], a["o"], a["lse"],
                       status=a["status"], workspace_bytes=a["size"])


def _weigh(m, **kw):
    plan = kw.pop("plan", None) or m.mla_chunk_make_plan(_problem(m), 10)
    a = dict(q=A[0], starts=A[1], cache=A[2], table=A[3], lens=A[4], ws=A[5], out=A[6], lse=A[7], into=A[8],
             status=None, size=plan.workspace_bytes, stride=100)
    a.update(kw)
    m.mla_cache_weights(plan, a["q"], a["lse"], a["starts"], a["cache"], a["table"], a["lens"], a["ws"], a["out"],
                        weights_in=a["into"], stride=a["stride"], status=a["status"], workspace_bytes=a["size"])


def _evict(m, **kw):
    plan = kw.pop("plan", None) or m.mla_evict_make_plan(_problem(m), 50)
    a = dict(cache=A[0], table=A[1], lens=A[2], w=A[3], pos=A[4], ws=A[5], lo=A[6], wo=A[7], po=A[8], status=None,
             size=plan.workspace_bytes, stride=100)
    a.update(kw)
    m.mla_cache_evict(plan, a["cache"], a["table"], a["lens"], a["w"], a["pos"], a["ws"], a["lo"], a["wo"], a["po"],
                      stride=a["stride"], status=a["status"], workspace_bytes=a["size"])


@pytest.mark.parametrize("call,names", [(_attend, "q starts cache table lens ws o lse"),
                                        (_weigh, "q starts cache table lens ws out lse"),
                                        (_evict, "cache table lens w pos ws")])
def test_missing_and_misaligned_pointers(m, call, names):
    for name in names.split():
        assert _code(m, call, m, **{name: 0}) == m.MLA_ERR_INVALID_ARGUMENT, name
        assert _code(m, call, m, **{name: A[9] + 2}) == m.MLA_ERR_MISALIGNED, name
    for name in {_attend: ("q", "cache", "ws", "o"), _weigh: ("q", "cache", "ws"), _evict: ("cache", "ws")}[call]:
        assert _code(m, call, m, **{name: A[9] + 4}) == m.MLA_ERR_MISALIGNED, name
    if call is _attend:
        assert _code(m, call, m, o=A[9] + 16) == m.MLA_ERR_MISALIGNED
    assert _code(m, call, m, status=A[9] + 2) == m.MLA_ERR_MISALIGNED
    assert _code(m, call, m, size=100) == m.MLA_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("call,cls", [(_attend, "MlaChunkPlan"), (_weigh, "MlaChunkPlan"), (_evict, "MlaEvictPlan")])
def test_a_plan_that_was_not_made(m, call, cls):
    plan = getattr(m, cls)()
    plan.problem = _problem(m)
    assert _code(m, call, m, plan=plan, size=1 << 40) == m.MLA_ERR_INVALID_ARGUMENT


def test_weights_refusals(m):
    for bad in (dict(stride=0), dict(stride=-5), dict(stride=1 << 62)):
        assert _code(m, _weigh, m, **bad) == m.MLA_ERR_INVALID_ARGUMENT
    assert _code(m, _weigh, m, into=A[6] + 4) == m.MLA_ERR_INVALID_ARGUMENT       # shifted by one
    assert _code(m, _weigh, m, into=A[6] + 4 * 399) == m.MLA_ERR_INVALID_ARGUMENT  # the last element


def test_evict_refusals(m):
    for bad in (dict(stride=0), dict(stride=1 << 62)):
        assert _code(m, _evict, m, **bad) == m.MLA_ERR_INVALID_ARGUMENT
    # outputs on other arrays, and shifted on their own
    for bad in (dict(wo=A[4]), dict(po=A[3]), dict(lo=A[3]), dict(wo=A[3] + 4), dict(po=A[4] + 4 * 399),
                dict(wo=A[0] + 64), dict(lo=A[1]), dict(ws=A[0]), dict(ws=A[2]), dict(wo=A[8]), dict(status=A[5])):
        assert _code(m, _evict, m, **bad) == m.MLA_ERR_INVALID_ARGUMENT, bad


def test_nothing_to_do_needs_no_gpu(m):
    """No tokens, or no requests: nothing is launched."""
    _attend(m, plan=m.mla_chunk_make_plan(_problem(m), 0))
    _attend(m, plan=m.mla_chunk_make_plan(_problem(m, batch=0), 5))
    _weigh(m, plan=m.mla_chunk_make_plan(_problem(m, batch=0), 5))
    plan = m.mla_evict_make_plan(_problem(m, batch=0), 5)
    _evict(m, plan=plan, size=1 << 20)


def test_structures_have_the_headers_sizes(m):
    assert ctypes.sizeof(m.MlaChunkPlan) == ctypes.sizeof(m.MlaProblem) + 8 + 8 + 8 + 6 * 8
    assert ctypes.sizeof(m.MlaEvictPlan) == ctypes.sizeof(m.MlaProblem) + 16 + 4 * 8


# ---------------------------------------------------------------- the oracle
def test_oracle_attention_against_a_mask():
    rng = np.random.default_rng(0)
    q, rows = rng.standard_normal((5, 3, 576)) / 4, rng.standard_normal((9, 576))
    s = np.einsum("jhd,td->jht", q, rows) / 16
    hidden = np.arange(9)[None] > np.arange(5)[:, None] + 4
    s = np.where(hidden[:, None], -np.inf, s)
    p = np.exp(s - s.max(-1, keepdims=True))
    o, _, lse, _ = C.attend(q, rows, 1 / 16)
    assert np.allclose(o, np.einsum("jht,td->jhd", p / p.sum(-1, keepdims=True), rows[:, :512]), atol=1e-12)
    w, _ = C.weights(q, lse, rows, 1 / 16)
    assert np.allclose(w, (p / p.sum(-1, keepdims=True)).sum((0, 1)), atol=1e-12) and np.isclose(w.sum(), 15)
    # more new tokens than rows: the first see nothing
    o, _, lse, _ = C.attend(q, rows[:2], 1 / 16)
    assert np.all(np.isneginf(lse[:3])) and np.all(o[:3] == 0) and np.all(np.isfinite(lse[3:]))
    assert C.weights(q, lse, rows[:2], 1 / 16)[0].sum() == pytest.approx(6)


def test_oracle_eviction_by_hand():
    w = np.array([1, 5, 5, 2, 0, 5, 3, 0], dtype=np.float32)
    pos = np.arange(8)
    assert C.evict(w, pos, 3)[1].tolist() == [5, 1, 2]            # three fives, slot 0 free
    assert C.evict(w, pos, 3, recent=1)[1].tolist() == [7, 1, 2]  # the newest before a five
    assert C.evict(w, pos, 2, sinks=1, recent=1)[1].tolist() == [0, 7]
    assert C.evict(w, pos[::-1], 2, sinks=1)[1].tolist() == [7, 1]   # position 0 stands in slot 7
    assert C.evict(w, pos, 1, sinks=3)[1].tolist() == [0]
    assert C.evict(w, pos, 8) [0] == 8 and C.evict(w[:0], pos[:0], 4)[0] == 0
    w[3] = np.nan
    assert C.evict(w, pos, 7)[1].tolist() == [0, 1, 2, 7, 4, 5, 6]
