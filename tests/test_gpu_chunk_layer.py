"""The chunk operators together, as runner.AttentionLayer runs them: prompts
prefilled in chunks, decode steps, the cache evicted by the weights that both
left, and decoding over what is left.  Attention and weights are checked against
the oracle on the values that entered them; a chunk's output against that of the
decode step, token by token."""
import numpy as np
import pytest

from chunk_testlib import f64, put
from mla_testlib import LSE_TOL, REL_L2, ensure_built
from oracle import chunk as C
from oracle import layer as L
from test_gpu_attention_layer import HIDDEN, _cached, _layer

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import head_latent_attention_paged_gb300 as mod
    return mod


def _tracked(m, heads, batch, q_len, kind, kv, page=64, max_pages=6):
    """test_gpu_attention_layer's layer, and one of the same weights that tracks."""
    from head_latent_attention_paged_gb300.runner import AttentionLayer
    g = torch.Generator(device="cuda").manual_seed(5)
    one, _, _ = _layer(m, g, heads, batch, q_len, kind, "pairs", "none", page=page, max_pages=max_pages)
    names = ("hidden_norm", "w_qkv_a", "q_norm", "kv_norm", "w_q_b", "w_uk", "w_uv", "w_o")
    two = AttentionLayer(**{n: getattr(one, n) for n in names}, batch=batch, q_len=q_len, page_size=page,
                         num_pages=one.problem.num_pages, max_pages=max_pages, rope=one.rope, kv_dtype=kind,
                         eps=one.eps, track=True)
    return one, two


def _close(a, b):
    """The chunk's form of an output and the decode step's: both round the queries, the
    weights and the projection to bf16, the chunk its o_lat as well (2^-9 each on
    average, below 0.01 together), and a library product may round a value the other
    way for another number of rows, which moves one in some hundred codes of a
    quantised cache by a step (2^-3, 2^-1: below 0.01)."""
    a, b = f64(a), f64(b)
    assert np.linalg.norm(a - b) <= 2e-2 * np.linalg.norm(b)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("heads,batch,page", [(4, 3, 64), (20, 4, 16)])
def test_prefill_evict_decode(m, kv, heads, batch, page):
    kind = {"bf16": m.MLA_KV_BF16, "fp8": m.MLA_KV_FP8_E4M3_E8M0, "fp4": m.MLA_KV_FP4_E2M1_E8M0}[kv]
    max_pages = 384 // page
    plain, layer = _tracked(m, heads, batch, 1, kind, kv, page, max_pages)
    rng = np.random.default_rng(5)
    g = torch.Generator(device="cuda").manual_seed(6)
    table = rng.permutation(layer.problem.num_pages)[:batch * max_pages].reshape(batch, max_pages).astype(np.int32)
    bt = put(table)
    total = np.array([150, 97, 200, 1][:batch])
    hidden = [torch.randn(n, HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16) for n in total]

    # the prompts: two chunks, the second of uneven parts and with padding
    done = np.zeros(batch, dtype=np.int64)
    outs = [[] for _ in range(batch)]
    S = max_pages * page
    for part in (np.minimum(total, 64), total - np.minimum(total, 64)):
        starts = np.concatenate([[0], np.cumsum(part)]).astype(np.int32)
        pad = 3
        x = torch.cat([hidden[b][done[b]:done[b] + part[b]] for b in range(batch)]
                      + [torch.full((pad, HIDDEN), 1.0, device="cuda", dtype=torch.bfloat16)])
        req = np.concatenate([np.repeat(np.arange(batch), part), np.zeros(pad)]).astype(np.int32)
        pos = np.concatenate([done[b] + np.arange(part[b]) for b in range(batch)] + [np.full(pad, -1)]).astype(np.int32)
        done = done + part
        out, same = layer.prefill(x, None, put(pos), put(req), put(starts), bt, put(done, np.int32))
        assert same is x
        for b in range(batch):
            outs[b].append(out[starts[b]:starts[b + 1]])
    torch.cuda.synchronize()
    assert layer.status() == 0

    # the same tokens one by one through the decode step
    for k in range(int(total.max())):
        live = k < total
        x = torch.stack([hidden[b][k] if live[b] else torch.zeros(HIDDEN, device="cuda", dtype=torch.bfloat16)
                         for b in range(batch)])
        step, _ = plain.decode(x, None, put(np.where(live, k, -1), np.int32), bt,
                               put(np.where(live, k + 1, 0), np.int32))
        if k in (0, 1, 63, 64, 65, 96, 149, 199):
            for b in np.flatnonzero(live):
                _close(torch.cat(outs[b])[k], step[b])
    # every query gave each of its heads' weight away, one in all
    w = f64(layer.weights)
    assert np.allclose(w[:, :S].sum(1), total * heads, rtol=1e-3)
    where = layer.slot_positions.cpu().numpy()
    for b in range(batch):
        assert np.array_equal(where[b, :S], np.where(np.arange(S) < total[b], np.arange(S), -1))

    # cut to 90 rows, and go on decoding behind them
    before, budget = _cached(layer, kv), 90
    lens = put(total, np.int32)
    layer.evict(budget, bt, lens, sinks=2, recent=10)
    torch.cuda.synchronize()
    left = lens.cpu().numpy()
    assert left.tolist() == np.minimum(total, budget).tolist()
    w_after, where = f64(layer.weights), layer.slot_positions.cpu().numpy()
    after = _cached(layer, kv)
    for b in range(batch):
        n = total[b]
        kept, origin = C.evict(w[b, :n].astype(np.float32), np.arange(n), budget, 2, 10)
        slots = table[b, np.arange(n) // page] * page + np.arange(n) % page
        assert np.array_equal(w_after[b, :kept], w[b, origin]) and np.all(w_after[b, kept:S] == 0)
        assert np.array_equal(where[b, :kept], origin) and np.all(where[b, kept:S] == -1)
        assert np.array_equal(after[slots[:kept]], before[slots[origin]])
    for k in range(3):
        x = torch.randn(batch, HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16)
        weights = f64(layer.weights)
        slots, lens = left.copy(), put(left + 1, np.int32)
        layer.decode(x, None, put(total + k, np.int32), bt, lens, slots=put(slots, np.int32))
        torch.cuda.synchronize()
        assert layer.status() == 0
        left = left + 1
        q_hat = layer.workspace[int(layer.plan.ws_q_hat):][:batch * heads * 1152].view(torch.bfloat16)
        q_hat = f64(q_hat).reshape(batch, heads, 576)
        cached, o_lat, lse, weights_now = _cached(layer, kv), f64(layer.o_lat), f64(layer.lse), f64(layer.weights)
        for b in range(batch):
            rows = cached[table[b, np.arange(left[b]) // page] * page + np.arange(left[b]) % page]
            ro, _, rl, _ = C.attend(q_hat[b][None], rows, 1 / 16)
            assert np.linalg.norm(o_lat[b] - ro[0]) <= REL_L2 * np.linalg.norm(ro[0])
            assert np.abs(lse[b] - rl[0]).max() <= LSE_TOL
            rw, tw = C.weights(q_hat[b][None], lse[b][None], rows, 1 / 16)
            got = weights_now[b, :left[b]] - weights[b, :left[b]]
            assert np.all(np.abs(got - rw) <= tw + 4 * C.U * weights_now[b, :left[b]])
        where = layer.slot_positions.cpu().numpy()
        assert np.array_equal(where[np.arange(batch), slots], total + k)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_slots_are_positions_without_an_eviction(m, kv):
    """The key turned ahead of the append is that of a row cached at its position, to
    a rounding to bf16."""
    kind = {"bf16": m.MLA_KV_BF16, "fp8": m.MLA_KV_FP8_E4M3_E8M0}[kv]
    one, two = _tracked(m, 4, 2, 2, kind, kv)
    g = torch.Generator(device="cuda").manual_seed(8)
    bt = put(np.arange(12).reshape(2, 6), np.int32)
    x = torch.randn(4, HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16)
    pos, lens = put([0, 1, 0, 1], np.int32), put([2, 2], np.int32)
    a = one.decode(x, None, pos, bt, lens)[0].clone()
    b = two.decode(x, None, pos, bt, lens, slots=pos)[0]
    _close(a, b)
    if kv == "bf16":                        # the bf16 rows differ by no rounding at all
        assert torch.equal(one.cache, two.cache)


def test_residual(m):
    """hidden and residual: the sum that the norm gives, and its output."""
    one, two = _tracked(m, 4, 2, 1, m.MLA_KV_BF16, "bf16")
    g = torch.Generator(device="cuda").manual_seed(4)
    x, residual = (torch.randn(9, HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    x = (x * 4).round() / 4                 # sums that bf16 holds: the norm's input is the same either way
    residual = (residual * 4).round() / 4
    args = (put([0, 1, 2, 3, 4, 0, 1, 2, 3], np.int32), put([0] * 5 + [1] * 4, np.int32), put([0, 5, 9], np.int32),
            put(np.arange(12).reshape(2, 6), np.int32), put([5, 4], np.int32))
    out, summed = one.prefill(x, residual, *args)
    want, _ = two.prefill(x + residual, None, *args)
    assert torch.equal(summed, x + residual) and torch.equal(out, want)


def test_captured_prefill_and_eviction(m):
    """Captured once and replayed on other inputs: the results of eager calls."""
    _, eager = _tracked(m, 4, 2, 1, m.MLA_KV_FP8_E4M3_E8M0, "fp8")
    _, graphed = _tracked(m, 4, 2, 1, m.MLA_KV_FP8_E4M3_E8M0, "fp8")
    g = torch.Generator(device="cuda").manual_seed(9)
    bt = put(np.arange(12).reshape(2, 6), np.int32)
    x = torch.randn(150, HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16)

    def inputs(part):
        pos = np.concatenate([np.arange(part[0]), np.arange(part[1]), np.full(150 - sum(part), -1)])
        req = np.repeat([0, 1, 0], [part[0], part[1], 150 - sum(part)])
        return [put(a, np.int32) for a in (pos, req, [0, part[0], sum(part)], part)]

    def go(layer, pos, req, starts, lens):
        out, _ = layer.prefill(x, None, pos, req, starts, bt, lens)
        layer.evict(40, bt, lens, sinks=1, recent=4)
        return out

    static = inputs((70, 80))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(graphed, *[t.clone() for t in static])        # loads what is loaded once
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go(graphed, *static)
    for part in ((33, 100), (1, 149), (0, 130)):
        for layer in (eager, graphed):
            layer.weights.zero_()
            layer.slot_positions.fill_(-1)
            layer.cache.zero_()
        for t, v in zip(static, inputs(part)):
            t.copy_(v)
        graph.replay()
        lens = inputs(part)
        want = go(eager, *lens)
        torch.cuda.synchronize()
        assert torch.equal(out[:sum(part)], want[:sum(part)])
        assert torch.equal(static[3], lens[3])
        assert torch.equal(graphed.weights, eager.weights) and torch.equal(graphed.cache, eager.cache)
        assert torch.equal(graphed.slot_positions, eager.slot_positions)


def test_layer_refusals(m):
    plain, layer = _tracked(m, 4, 2, 1, m.MLA_KV_BF16, "bf16")
    bt, lens = put(np.arange(12).reshape(2, 6), np.int32), put([3, 4], np.int32)
    x = torch.zeros(7, HIDDEN, dtype=torch.bfloat16, device="cuda")
    pos, req, starts = put(np.arange(7), np.int32), put(np.zeros(7), np.int32), put([0, 3, 7], np.int32)
    with pytest.raises(ValueError):
        plain.evict(5, bt, lens)
    for bad in (dict(positions=pos.long()), dict(requests=req[:6]), dict(query_starts=starts[:2]),
                dict(seq_lens=lens.cpu()), dict(block_table=bt[:1]), dict(hidden=x[:6]), dict(residual=x.float()),
                dict(slots=pos[:5])):
        a = dict(hidden=x, residual=None, positions=pos, requests=req, query_starts=starts, block_table=bt, seq_lens=lens)
        a.update(bad)
        with pytest.raises(ValueError):
            layer.prefill(**a)
    with pytest.raises(ValueError):
        layer.evict(5, bt, lens.long())
    with pytest.raises(m.MlaError):
        layer.evict(0, bt, lens)
