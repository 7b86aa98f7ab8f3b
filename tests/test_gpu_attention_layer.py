"""The layer operators together, as runner.AttentionLayer runs them: a prompt
cached in chunks, then decode steps.  Every stage is checked on the values that
entered it (norms, rotation and cache rows against oracle.layer, the attention
against the oracle's decompressed form), so the roundings in between do not
enter the tolerances."""
import numpy as np
import pytest

import oracle as O
from oracle import layer as L
from mla_testlib import ATOL_MAX, LSE_TOL, REL_L2, ensure_built

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HIDDEN, Q_RANK, EPS = 320, 768, 1e-6


@pytest.fixture(scope="module")
def m():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import head_latent_attention_paged_gb300 as mod
    return mod


def _f64(t):
    return t.detach().cpu().double().numpy()


def _layer(m, g, heads, batch, q_len, kv, layout, scaling, page=64, max_pages=6):
    from head_latent_attention_paged_gb300.runner import AttentionLayer
    from test_layer_cpu import _plan_args

    def w(*shape, fan_in=None):
        x = torch.randn(*shape, generator=g, device="cuda") / (fan_in or shape[0]) ** 0.5
        return x.to(torch.bfloat16)

    a = _plan_args(m, scaling)
    plan = m.mla_rope_plan(layout=m.MLA_ROPE_HALVES if layout == "halves" else m.MLA_ROPE_INTERLEAVED, **a)
    freq, amplitude = L.rope_frequencies(64, 1e6, scaling, a.get("factor", 1.0), a.get("original_positions", 0),
                                         a.get("fast_rotations", 0), a.get("slow_rotations", 0))
    norm = lambda n: (1 + 0.1 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    layer = AttentionLayer(hidden_norm=norm(HIDDEN), w_qkv_a=w(HIDDEN, Q_RANK + 576), q_norm=norm(Q_RANK),
                           kv_norm=norm(512), w_q_b=w(Q_RANK, heads * 256), w_uk=w(heads, 512, 192, fan_in=512),
                           w_uv=w(heads, 512, 256, fan_in=512), w_o=w(heads * 256, HIDDEN), batch=batch,
                           q_len=q_len, page_size=page, num_pages=batch * max_pages + 2, max_pages=max_pages,
                           rope=plan, kv_dtype=kv, eps=EPS)
    return layer, freq, float(np.float32(amplitude))


def _cached(layer, kv):
    """The pool's rows as float64, from its bytes."""
    raw = layer.cache.cpu().numpy()
    slots = np.arange(raw.shape[0] * layer.problem.page_size)
    return L.gather_rows(raw.view(np.uint16) if kv == "bf16" else raw, slots, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("heads,batch,q_len,layout,scaling", [(4, 3, 1, "pairs", "none"), (20, 5, 2, "halves", "yarn")])
def test_prompt_then_decode(m, kv, heads, batch, q_len, layout, scaling):
    kind = {"bf16": m.MLA_KV_BF16, "fp8": m.MLA_KV_FP8_E4M3_E8M0, "fp4": m.MLA_KV_FP4_E2M1_E8M0}[kv]
    g = torch.Generator(device="cuda").manual_seed(3)
    rng = np.random.default_rng(3)
    layer, freq, amplitude = _layer(m, g, heads, batch, q_len, kind, layout, scaling)
    P, max_pages = layer.problem.page_size, layer.problem.max_pages_per_seq
    table = rng.permutation(layer.problem.num_pages)[:batch * max_pages].reshape(batch, max_pages).astype(np.int32)
    bt = torch.from_numpy(table).cuda()
    lens = rng.integers(1, max_pages * P - 2 * q_len, batch)
    lens[0] = 0                                           # a request without a prompt
    lens[1] = P                                           # one that ends with its page
    # the prompts in two chunks, tokens of all requests shuffled
    req = np.repeat(np.arange(batch), lens).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    order = rng.permutation(len(req))
    req, pos = req[order], pos[order]
    hidden = torch.randn(len(req), HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16)
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    for part in (slice(0, len(req) // 3), slice(len(req) // 3, None)):
        layer.prompt(hidden[part], put(pos[part]), put(req[part]), bt)
    slots = L.slots_of(pos, req, table, P, layer.problem.num_pages)
    rows = layer.context(put(pos), put(req), bt)
    assert np.array_equal(_f64(rows), _cached(layer, kv)[slots])
    # the prompt's rows from the layer's own projection of its normed input
    _, x, t = L.rms_norm(_f64(hidden), weight=_f64(layer.hidden_norm), eps=np.float32(EPS))
    xg = torch.empty_like(hidden)
    m.mla_rms_norm(m.make_norm_problem(len(req), HIDDEN, eps=EPS), hidden, layer.hidden_norm, xg)
    L.assert_rounded(_f64(xg), x, t, "bf16", "prompt norm")

    residual = torch.randn(layer.rows, HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16)
    for step in range(2):
        new = torch.randn(layer.rows, HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16)
        positions = (lens[:, None] + np.arange(q_len)).astype(np.int32).reshape(-1)
        lens = lens + q_len
        before = residual.clone()
        out, res = layer.decode(new, residual, put(positions), bt, put(lens.astype(np.int32)))
        torch.cuda.synchronize()
        assert layer.status() == 0
        h, x, t = L.rms_norm(_f64(new), _f64(before), _f64(layer.hidden_norm), np.float32(EPS))
        L.assert_rounded(_f64(res), h, np.abs(h) * L.U, "bf16", "residual")
        L.assert_rounded(_f64(layer.x), x, t, "bf16", "hidden norm")
        qkv = _f64(layer.qkv_a)
        _, q_a, t = L.rms_norm(qkv[:, :Q_RANK], weight=_f64(layer.q_norm), eps=np.float32(EPS))
        L.assert_rounded(_f64(layer.q_a), q_a, t, "bf16", "query latent")
        request = np.repeat(np.arange(batch), q_len)
        slots = L.slots_of(positions, request, table, P, layer.problem.num_pages)
        y, t = L.row_values(qkv[:, Q_RANK:], positions, _f64(layer.kv_norm), np.float32(EPS), freq, amplitude, layout)
        raw = layer.cache.view(-1, {"bf16": 1152, "fp8": 594, "fp4": 324}[kv])[put(slots)].cpu().numpy()
        if kv == "bf16":
            raw = (raw.view(np.uint16).astype(np.uint32) << 16).view(np.float32)
        L.assert_cache_rows(raw, y, t, kv, "new rows")
        # the rotated queries, from the same product before the rotation
        q0 = _f64(torch.matmul(layer.q_a, layer.w_q_b).view(layer.rows, heads, 256))
        q = _f64(layer.q)
        yq, tq = L.rope(q0[..., 192:], positions, freq, amplitude, layout)
        assert np.array_equal(q[..., :192], q0[..., :192])
        L.assert_rounded(q[..., 192:], yq, tq, "bf16", "queries")
        # the attention over the cache as it stands
        cached, w_uk, w_uv = _cached(layer, kv), _f64(layer.w_uk), _f64(layer.w_uv)
        o, lse = _f64(layer.o), _f64(layer.lse)
        for r in range(layer.rows):
            b, j = divmod(r, q_len)
            vis = np.arange(lens[b] - q_len + j + 1)
            at = L.slots_of(vis, np.full(len(vis), b), table, P, layer.problem.num_pages)
            c, kr = cached[at, :512], cached[at, 512:]
            ref, _, _ = O.attend_non_absorbed(q[r, :, :192], q[r, :, 192:], w_uk, w_uv, c, kr, 1.0 / 16.0)
            q_lat = O.round_to_bf16(O.absorb_query(q[r, :, :192], w_uk))
            _, ref_lse, _ = O.attend_absorbed(q_lat, q[r, :, 192:], w_uv, c, kr, 1.0 / 16.0)
            assert np.linalg.norm(o[r] - ref) <= REL_L2 * np.linalg.norm(ref)
            assert np.abs(o[r] - ref).max() <= ATOL_MAX * max(1.0, np.abs(ref).max())
            assert np.abs(lse[r] - ref_lse).max() <= LSE_TOL
        product = torch.matmul(layer.o.view(layer.rows, -1), layer.w_o)
        assert torch.equal(out, product)
        residual = res.clone()


def test_decode_step_in_a_graph_and_a_padded_batch(m):
    """The step captured and replayed on new inputs gives the eager step's
    bits; a padded request (length 0, position -1) writes nothing and gives
    zeros.  The other requests' attention is then split over other CTAs (the
    work split goes by all lengths), and splits agree to the rounding of the
    probabilities: 2e-3 of the latent output, 5e-4 of the lse, the bounds of the
    split tests."""
    g = torch.Generator(device="cuda").manual_seed(8)
    layer, _, _ = _layer(m, g, 8, 4, 1, m.MLA_KV_FP8_E4M3_E8M0, "pairs", "none")
    bt = torch.arange(4 * 6, dtype=torch.int32, device="cuda").view(4, 6)
    pos = torch.tensor([5, 64, 17, 200], dtype=torch.int32, device="cuda")
    lens = pos + 1
    for r in range(4):
        n = int(pos[r])
        layer.prompt(torch.randn(n, HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16),
                     torch.arange(n, dtype=torch.int32, device="cuda"),
                     torch.full((n,), r, dtype=torch.int32, device="cuda"), bt)
    hidden, residual = (torch.randn(4, HIDDEN, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cache = layer.cache.clone()
    want = [t.clone() for t in layer.decode(hidden, residual, pos, bt, lens)]
    after, lat, lse = layer.cache.clone(), _f64(layer.o_lat), _f64(layer.lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    h, r, p, n = (t.clone() for t in (hidden, residual, pos, lens))
    h.zero_()
    with torch.cuda.stream(side):
        layer.decode(h, r, p, bt, n)                     # warm-up of the library products
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out, res = layer.decode(h, r, p, bt, n)
    torch.cuda.synchronize()
    layer.cache.copy_(cache)
    h.copy_(hidden)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(res, want[1]) and torch.equal(layer.cache, after)
    layer.cache.copy_(cache)                             # request 2 becomes padding
    p[2], n[2] = -1, 0
    graph.replay()
    torch.cuda.synchronize()
    for r in (0, 1, 3):
        assert np.linalg.norm(_f64(layer.o_lat)[r] - lat[r]) <= 2e-3 * np.linalg.norm(lat[r])
        assert np.abs(_f64(layer.lse)[r] - lse[r]).max() <= 5e-4
    assert bool((out[2] == 0).all()) and bool((layer.lse[2] == -float("inf")).all())
    assert layer.status() == 0
    with pytest.raises(ValueError):                      # shapes and types that the kernels cannot see
        layer.decode(hidden.float(), None, pos, bt, lens)
    with pytest.raises(ValueError):
        layer.decode(hidden, None, pos.long(), bt, lens)
    with pytest.raises(ValueError):
        layer.prompt(hidden, pos, pos[:3], bt)
    page = int(bt[2, 0])
    assert torch.equal(layer.cache[page], cache[page])
