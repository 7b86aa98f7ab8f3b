"""What a tracking runner.AttentionLayer notes of the tokens it caches, and what
eviction makes of it, where tokens are padding, out of range, or written again."""
import numpy as np
import pytest

from chunk_testlib import f64, put
from mla_testlib import ensure_built
from test_gpu_attention_layer import HIDDEN
from test_gpu_chunk_layer import _tracked

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import head_latent_attention_paged_gb300 as mod
    return mod


def _states(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16)


def _table(batch=2, max_pages=6):
    return put(np.arange(batch * max_pages).reshape(batch, max_pages), np.int32)


def test_requests_outside_the_batch_are_reported(m):
    """As by a layer that does not track: a status bit, and nothing written."""
    _, layer = _tracked(m, 4, 2, 1, m.MLA_KV_BF16, "bf16")
    bt, lens = _table(), put([4, 3], np.int32)
    layer.prefill(_states(7, 1), None, put([0, 1, 2, 3, 0, 1, 2], np.int32), put([0] * 4 + [1] * 3, np.int32),
                  put([0, 4, 7], np.int32), bt, lens)
    torch.cuda.synchronize()
    assert layer.status() == 0
    cache, weights, positions = layer.cache.clone(), layer.weights.clone(), layer.slot_positions.clone()
    bad = put([-1, 2, 1 << 30, -5], np.int32)
    layer.prompt(_states(4, 2), put([0, 1, 2, 3], np.int32), bad, bt)
    torch.cuda.synchronize()
    assert layer.status() == m.MLA_STATUS_BAD_INDEX
    assert torch.equal(layer.cache, cache)
    slots = 6 * 64
    assert torch.equal(layer.weights[:, :slots], weights[:, :slots])
    assert torch.equal(layer.slot_positions[:, :slots], positions[:, :slots])


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_padding_with_slots_leaves_the_cache(m, kv):
    """Slots of a padded batch filled up with zeros: no row of slot 0 is lost."""
    kind = {"bf16": m.MLA_KV_BF16, "fp8": m.MLA_KV_FP8_E4M3_E8M0, "fp4": m.MLA_KV_FP4_E2M1_E8M0}[kv]
    _, layer = _tracked(m, 4, 2, 1, kind, kv)
    bt = _table()
    layer.prefill(_states(7, 1), None, put([0, 1, 2, 3, 0, 1, 2], np.int32), put([0] * 4 + [1] * 3, np.int32),
                  put([0, 4, 7], np.int32), bt, put([4, 3], np.int32))
    cache, weights, positions = layer.cache.clone(), layer.weights.clone(), layer.slot_positions.clone()
    # both requests padded in a step, and a chunk of padding alone
    layer.decode(_states(2, 2), None, put([-1, -1], np.int32), bt, put([0, 0], np.int32), slots=put([0, 0], np.int32))
    layer.prefill(_states(3, 3), None, put([-1] * 3, np.int32), put([0, 1, 1], np.int32), put([0, 0, 0], np.int32), bt,
                  put([4, 3], np.int32), slots=put([0, 0, 2], np.int32))
    torch.cuda.synchronize()
    assert layer.status() == 0
    slots = 6 * 64
    assert torch.equal(layer.cache, cache) and torch.equal(layer.weights[:, :slots], weights[:, :slots])
    assert torch.equal(layer.slot_positions[:, :slots], positions[:, :slots])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_rejected_drafts_weight_is_not_its_slots_next_tokens(m, kv):
    """Two drafts a step, the second rejected: its slot is decoded again and holds what the
    new tokens' queries give alone, as where its weight has been cleared by hand."""
    kind = {"bf16": m.MLA_KV_BF16, "fp8": m.MLA_KV_FP8_E4M3_E8M0}[kv]
    layers = [_tracked(m, 4, 2, 2, kind, kv)[1] for _ in range(2)]
    bt = _table()

    def step(layer, seed, first):
        layer.decode(_states(4, seed), None, put([first, first + 1] * 2, np.int32), bt, put([first + 2] * 2, np.int32))
        torch.cuda.synchronize()
        return f64(layer.weights)

    for layer in layers:
        step(layer, 5, 0)
        rejected = step(layer, 6, 2)                   # tokens 2 and 3; 3 is rejected
        assert np.all(rejected[:, 3] > 0)
    layers[1].weights[:, 3] = 0
    after = [step(layer, 7, 3) for layer in layers]    # 3 again, and 4
    assert np.array_equal(after[0], after[1])
    # a query gives each head's weight away, one in all.  Scores are sums of 576 products
    # in 32 bits, off by 576 * 2^-23 of their magnitudes' sum at most, which is below 15 here
    # (|q . row| / 16 with values of order one), and lse by as much again: 2e-3 of a weight
    given = (after[0][:, :3] - rejected[:, :3]).sum(1) + after[0][:, 3] + after[0][:, 4]
    assert np.allclose(given, 2 * 4, rtol=2e-3, atol=0)
    assert layers[0].slot_positions[:, :5].tolist() == [[0, 1, 2, 3, 4]] * 2 and layers[0].status() == 0


def test_a_draft_rejected_in_a_graph(m):
    """The same from a captured step, replayed on positions that go back."""
    _, eager = _tracked(m, 4, 2, 2, m.MLA_KV_BF16, "bf16")
    _, graphed = _tracked(m, 4, 2, 2, m.MLA_KV_BF16, "bf16")
    bt = _table()
    static = [_states(4, 0), put([0, 1] * 2, np.int32), put([2, 2], np.int32)]

    def go(layer, hidden, positions, lens):
        return layer.decode(hidden, None, positions, bt, lens)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(graphed, *static)                           # loads what is loaded once
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = go(graphed, *static)
    for layer in (eager, graphed):
        for request in range(2):
            layer.forget(request)
    for seed, first in enumerate((0, 2, 3, 3, 5)):
        args = [_states(4, seed), put([first, first + 1] * 2, np.int32), put([first + 2] * 2, np.int32)]
        for t, v in zip(static, args):
            t.copy_(v)
        graph.replay()
        want = go(eager, *args)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(graphed.weights, eager.weights)
        assert torch.equal(graphed.slot_positions, eager.slot_positions)
    assert eager.status() == graphed.status() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_requests_that_share_a_prefix(m, kv):
    """Four requests over one prompt's pages, more rows between them than the pool holds:
    outputs and weights are those of requests with pages of their own."""
    from head_latent_attention_paged_gb300.runner import AttentionLayer
    kind = {"bf16": m.MLA_KV_BF16, "fp8": m.MLA_KV_FP8_E4M3_E8M0, "fp4": m.MLA_KV_FP4_E2M1_E8M0}[kv]
    B, page, prefix = 4, 16, 6
    one, apart = _tracked(m, 4, B, 1, kind, kv, page, 8)
    names = ("hidden_norm", "w_qkv_a", "q_norm", "kv_norm", "w_q_b", "w_uk", "w_uv", "w_o")
    shared = AttentionLayer(**{n: getattr(one, n) for n in names}, batch=B, page_size=page, num_pages=prefix + B,
                            max_pages=8, rope=one.rope, kv_dtype=kind, eps=one.eps, track=True)
    own = np.arange(B * 8).reshape(B, 8)
    common = np.concatenate([np.broadcast_to(np.arange(prefix), (B, prefix)), prefix + np.arange(B)[:, None],
                             np.zeros((B, 1), dtype=np.int64)], axis=1)
    own, common = put(own, np.int32), put(common, np.int32)
    # the prompt, cached once; the same bytes in every request's pages
    n = prefix * page
    shared.prefill(_states(n, 1), None, put(np.arange(n), np.int32), put(np.zeros(n), np.int32),
                   put([0, n, n, n, n], np.int32), common, put([n, 0, 0, 0], np.int32))
    for b in range(B):
        apart.cache[own[b, :prefix].long()] = shared.cache[:prefix]
    for layer in (shared, apart):
        layer.weights.zero_()
    # a turn of five tokens each, and a step
    five = 5 * B
    args = (_states(five, 2), None, put(np.tile(n + np.arange(5), B), np.int32), put(np.repeat(np.arange(B), 5), np.int32),
            put(np.arange(0, five + 1, 5), np.int32))
    lens = put([n + 5] * B, np.int32)
    outs = [layer.prefill(*args, bt, lens)[0] for layer, bt in ((shared, common), (apart, own))]
    torch.cuda.synchronize()
    assert shared.status() == apart.status() == 0 and B * (n + 5) > shared.problem.num_pages * page
    assert torch.equal(outs[0], outs[1]) and torch.equal(shared.weights, apart.weights)
    # a query gives each head's weight away, one in all (and see the bound above)
    assert np.allclose(f64(shared.weights).sum(1), 5 * 4, rtol=2e-3, atol=0)
    step = (_states(B, 3), None, put([n + 5] * B, np.int32))
    outs = [layer.decode(*step, bt, lens + 1)[0].clone() for layer, bt in ((shared, common), (apart, own))]
    torch.cuda.synchronize()
    assert shared.status() == apart.status() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(shared.weights, apart.weights)
