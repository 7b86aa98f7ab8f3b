"""The layer operators (include/mla_layer.h) on the GPU where their documented
results are hardest to keep: the ends of the 32-bit range, exact quotients,
infinities and signed zeros, calls so large that a warp takes many tokens."""
import numpy as np
import pytest

from oracle import fp8 as F8
from oracle import layer as L
from mla_testlib import ensure_built
from test_gpu_layer import _Norm, _Pool, _dt, _f64, _rand

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import head_latent_attention_paged_gb300 as mod
    return mod


# Widths of each kernel: a few lanes, a warp, a block for a row, on 16-byte
# boundaries (shift 0) and off them.
FORMS = [(3, 64, 0), (3, 64, 1), (600, 100, 0), (600, 130, 1), (3, 4096, 0), (520, 2048, 0), (520, 2881, 0),
         (2, 32768, 0), (2, 32768, 1)]


@pytest.mark.parametrize("out", ["same", "mx", "row"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,shift", FORMS)
def test_norm_over_the_range_of_32_bits(m, kind, out, rows, cols, shift):
    """Finite rows whose squares leave the range of 32 bits at either end are
    normed like any other, with no eps and with one; a row of zeros without an
    eps is NaN (0 / 0).  Rows of both ends in one call, ordinary ones between."""
    rng = np.random.default_rng(1)
    for eps in (0.0, 1e-6, 2.0 ** -140):
        n = _Norm(m, rng, rows, cols, kind, out, residual=True, shift=shift, eps=eps)
        scale = torch.tensor([2.0 ** -115, 2.0 ** 110, 1.0, 2.0 ** -70, 2.0 ** 60, 2.0 ** 45, 2.0 ** -55],
                             device="cuda").repeat(rows // 7 + 1)[:rows, None]
        n.x.copy_((n.x.float() * scale).to(_dt(kind)))
        n.residual.copy_((n.residual.float() * scale).to(_dt(kind)))
        n.run()
        keep = torch.arange(min(rows, 14))
        n.check_rows(keep, f"{kind} {out} {rows}x{cols} eps {eps}")
    n = _Norm(m, rng, rows, cols, kind, out, residual=False, shift=shift, eps=0.0)
    n.x[1] = 0.0
    n.run()
    got = n.out if out == "same" else torch.from_numpy(F8.e4m3_to_f64(n.out.cpu().numpy()))
    assert bool(got[1].isnan().all()) and not bool(got[0].isnan().any())


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_append_over_the_range_of_32_bits(m, kv):
    """The append's latent norm over the same range."""
    rng = np.random.default_rng(2)
    for eps in (0.0, 1e-6):
        pool = _Pool(m, rng, kv, 64, 1, 1)
        rows = _rand(rng, (28, 576), "bf16")
        scale = torch.tensor([2.0 ** -115, 2.0 ** 110, 1.0, 2.0 ** -70, 2.0 ** 60, 2.0 ** 45, 2.0 ** -55],
                             device="cuda").repeat(4)[:, None]
        rows[:, :512] = (rows[:, :512].float() * scale).to(torch.bfloat16)
        weight = _rand(rng, (512,), "bf16")
        pos = torch.arange(28, dtype=torch.int32, device="cuda")
        m.mla_cache_append_tokens(pool.problem, 28, rows, pos, pool.bt, pool.dev, norm_weight=weight, norm_eps=eps)
        y, t = L.row_values(_f64(rows), np.arange(28), _f64(weight), np.float32(eps))
        L.assert_cache_rows(pool.rows(pool.slots(np.arange(28), np.zeros(28, dtype=int))), y, t, kv, f"eps {eps}")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,shift", [(2, 64, 0), (2, 128, 1), (700, 256, 0), (2, 4096, 0), (2, 4096, 1),
                                             (515, 2048, 0), (515, 512, 1)])
def test_norm_row_scales_are_quotients(m, kind, rows, cols, shift):
    """scale = amax / 448 and code = e4m3(y / scale), both quotients rounded
    once to 32 bits: rows of +-1 without an eps have y = +-weight exactly, the
    weights lie on and beside the codes' midpoints."""
    rng = np.random.default_rng(cols + shift)
    codes = np.arange(0, 126)
    mid = (F8.e4m3_to_f64(codes) + F8.e4m3_to_f64(codes + 1)) / 2
    for _ in range(8):
        n = _Norm(m, rng, rows, cols, kind, "row", residual=False, shift=shift, eps=0.0)
        top = np.exp2(rng.uniform(-3, 6)) if kind == "f16" else np.exp2(rng.uniform(-60, 90))
        w = torch.from_numpy(top * rng.uniform(-1, 1, cols)).to(_dt(kind))
        w[0] = top
        scale = np.float32(float(w.abs().max().to(torch.float32))) / np.float32(448)
        beside = (mid[rng.integers(0, len(mid), cols // 2)] * float(scale)).astype(np.float32)
        beside = beside.view(np.int32) + rng.integers(-2, 3, cols // 2).astype(np.int32)
        w[cols // 2:] = torch.from_numpy(beside.view(np.float32)).to(_dt(kind)).clamp(max=float(w[0]))
        n.weight = w.cuda()
        n.x.copy_(torch.from_numpy(rng.choice([-1.0, 1.0], (rows, cols))))
        n.run()
        y = (n.x.double() * n.weight.double()).cpu().numpy().astype(np.float32)
        assert np.array_equal(n.scales.cpu().numpy(), np.broadcast_to(scale, rows))
        want = F8._round_to_e4m3((y / scale).astype(np.float64))
        assert np.array_equal(F8.e4m3_to_f64(n.out.cpu().numpy()), want)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,shift", [(5, 64, 0), (5, 96, 1), (600, 1024, 0), (600, 1030, 1)])
def test_norm_of_an_infinite_value_with_row_scales(m, kind, rows, cols, shift):
    """An infinite weight makes its values and their rows' scales infinite: the
    others' codes are their quotients by it, 0, and its own NaN."""
    n = _Norm(m, np.random.default_rng(6), rows, cols, kind, "row", residual=False, shift=shift)
    n.weight[5] = float("inf")
    n.run()
    code = F8.e4m3_to_f64(n.out.cpu().numpy())
    assert bool(n.scales.isposinf().all()) and np.isnan(code[:, 5]).all()
    assert (np.delete(code, 5, axis=1) == 0).all()


@pytest.mark.parametrize("out", ["same", "mx", "row"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,shift", [(5, 64, 0), (5, 96, 1), (600, 1024, 0), (600, 1030, 1)])
def test_norm_signs_of_zeros(m, kind, out, rows, cols, shift):
    """A zero keeps its sign through the product with the weight, except where
    a whole group (with group scales) is zero: its codes are 0."""
    rng = np.random.default_rng(4)
    n = _Norm(m, rng, rows, cols, kind, out, residual=False, shift=shift)
    n.x[:, 3:9] = -0.0
    n.x[:, 12:17] = 0.0
    n.x[:, 32:64] = -0.0
    n.weight[::2] = n.weight[::2].abs()
    n.weight[1::2] = -n.weight[1::2].abs()
    n.run()
    n_neg = torch.signbit(n.x) ^ torch.signbit(n.weight)
    got = torch.signbit(n.out) if out == "same" else n.out >= 0x80
    cols_of = list(range(3, 9)) + list(range(12, 17)) + ([] if out == "mx" else list(range(32, 64)))
    assert torch.equal(got[:, cols_of], n_neg[:, cols_of])
    if out == "mx":
        assert int(n.out[:, 32:64].max()) == 0 and int(n.scales[:, 1].max()) == 0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,shift", [(5, 64, 0), (5, 96, 1), (600, 1024, 0), (600, 1030, 1)])
def test_norm_of_an_infinite_weight_with_group_scales(m, kind, rows, cols, shift):
    """NaN or the largest code under the weight, in its own group alone."""
    rng = np.random.default_rng(6)
    n = _Norm(m, rng, rows, cols, kind, "mx", residual=False, shift=shift)
    n.weight[5], n.weight[6] = float("inf"), float("-inf")
    n.run()
    code = F8.e4m3_to_f64(n.out.cpu().numpy())
    assert (np.isnan(code[:, 5:7]) | (np.abs(code[:, 5:7]) == 448)).all()
    assert not np.isnan(np.delete(code, [5, 6], axis=1)).any()
    _, y, t = n.reference()
    L.assert_quantised(code[:, 32:], n.scales[:, 1:].cpu().numpy().astype(np.int64) - 127, y[:, 32:], t[:, 32:], 32,
                       "e4m3")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["token", "head"])
def test_rope_between_columns_of_one_buffer(m, kind, order):
    """Heads turned out of one column range of a wide buffer into another,
    token by token or head by head: they share no element."""
    rng = np.random.default_rng(7)
    tokens, heads, D = 37, 5, 64
    outer, inner = (tokens, heads) if order == "token" else (heads, tokens)
    buf = _rand(rng, (outer, 2 * inner * D + 64), kind)
    x = buf[:, :inner * D].unflatten(1, (inner, D))
    out = buf[:, inner * D:2 * inner * D].unflatten(1, (inner, D))
    if order == "head":
        x, out = x.transpose(0, 1), out.transpose(0, 1)
    before = buf.clone()
    x64 = _f64(x)
    pos = rng.integers(0, 4096, tokens).astype(np.int32)
    pr = m.make_rope_problem(tokens, heads, D, 0, 0 if kind == "bf16" else 2, 0, x.stride(0), x.stride(1),
                             out.stride(0), out.stride(1))
    m.mla_rope(pr, m.mla_rope_plan(), x, torch.from_numpy(pos).cuda(), out)
    freq, _ = L.rope_frequencies(64)
    y, t = L.rope(x64, pos, freq)
    L.assert_rounded(_f64(out), y, t, kind)
    assert torch.equal(buf[:, :inner * D], before[:, :inner * D])
    assert torch.equal(buf[:, 2 * inner * D:], before[:, 2 * inner * D:])
    with pytest.raises(m.MlaError) as e:     # half a head earlier: some of x's elements
        m.mla_rope(pr, m.mla_rope_plan(), x, torch.from_numpy(pos).cuda(), buf.flatten()[inner * D - D // 2:])
    assert e.value.code == m.MLA_ERR_INVALID_ARGUMENT


# ---------------------------------------------------------------- streams
@pytest.mark.parametrize("captured", [False, True])
def test_a_call_waits_for_another_streams_work(m, captured):
    """Calls start while their predecessor on the stream still runs; a long one
    on another stream, waited for by an event in between, is waited for all the
    same, before its output is read and before its input is written: eager, and
    as a captured graph's fork and join."""
    rng = np.random.default_rng(14)
    tokens, heads, dim = 40000, 32, 128
    x = _rand(rng, (tokens, heads, dim), "bf16")
    turned, small = torch.empty_like(x), _rand(rng, (64, 512), "bf16")
    small_out, out = torch.empty_like(small), torch.empty(tokens, heads * dim, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    plan, rp = m.mla_rope_plan(rope_dim=dim), m.make_rope_problem(tokens, heads, dim)
    np_small, np_big = m.make_norm_problem(64, 512), m.make_norm_problem(tokens, heads * dim)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        two.wait_stream(one)
        m.mla_rope(rp, plan, x, pos, turned, stream=two)             # long, x to turned
        m.mla_rms_norm(np_small, small, None, small_out, stream=one)
        one.wait_stream(two)
        m.mla_rms_norm(np_big, turned, None, out, stream=one)        # reads turned
        m.mla_rms_norm(np_big, out, None, x, stream=one)             # writes x

    def alone():
        m.mla_rope(rp, plan, x, pos, turned)
        m.mla_rms_norm(np_big, turned, None, out)
        m.mla_rms_norm(np_big, out, None, x)

    first = x.clone()
    want = []
    for _ in range(3):
        alone()
        want.append((out.clone(), x.clone()))
    torch.cuda.synchronize()
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=one):
            step()
        torch.cuda.synchronize()
    for _ in range(4):
        x.copy_(first)
        turned.zero_()
        torch.cuda.synchronize()
        for w_out, w_x in want:
            if captured:
                graph.replay()
                torch.cuda.synchronize()
            else:
                step()
                torch.cuda.synchronize()
            assert torch.equal(out, w_out) and torch.equal(x, w_x)


# ---------------------------------------------------------------- many tokens
@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("tokens,requests,full", [(9731, 5, True), (20011, 7, False), (40009, 3, True), (45003, 4, False),
                                                  (30000, 6, True)])
def test_many_tokens_of_a_warp(m, kv, tokens, requests, full):
    """Prompt-sized calls, where a warp takes several tokens one after another:
    tokens of no position and of no slot lie between the others, and a last
    warp has fewer.  Every row written is compared with the oracle, every
    other one with what it held; the gather returns the cache's values.  30,000
    tokens go without a list of requests, in equal shares."""
    rng = np.random.default_rng(tokens)
    page, share = 64, tokens // requests
    in_order = tokens % requests == 0
    max_pages = -(-(share if in_order else tokens // (requests - 1)) // page) + 1
    pool = _Pool(m, rng, kv, page, requests, max_pages)
    cap = max_pages * page
    if in_order:
        req = np.repeat(np.arange(requests), share).astype(np.int32)
        pos = np.concatenate([rng.permutation(cap)[:share] for _ in range(requests)]).astype(np.int32)
    else:
        pick = rng.choice(requests * cap, tokens, replace=False)
        req, pos = (pick // cap).astype(np.int32), (pick % cap).astype(np.int32)
    pool.table[1, 1], pool.table[requests - 1, 0] = pool.num_pages + 3, -7
    pool.bt = torch.from_numpy(pool.table).cuda()
    kind = rng.integers(0, 12, tokens)
    pos[kind == 0] = -1
    pos[kind == 1] = cap + rng.integers(0, 9, int((kind == 1).sum()))
    if not in_order:
        req[kind == 2] = requests
        req[kind == 3] = -1
    pos[:9] = -1                                          # a warp's tokens, all of them
    stride = 584
    wide = _rand(rng, (tokens, stride), "bf16")
    rows = wide[:, 8:]
    weight = _rand(rng, (512,), "bf16") if full else None
    plan = m.mla_rope_plan(layout=m.MLA_ROPE_HALVES if requests == 3 else m.MLA_ROPE_INTERLEAVED) if full else None
    freq = L.rope_frequencies(64)[0] if full else None
    positions, of = torch.from_numpy(pos).cuda(), None if in_order else torch.from_numpy(req).cuda()
    m.mla_cache_append_tokens(pool.problem, tokens, rows, positions, pool.bt, pool.dev, requests=of, row_stride=stride,
                              norm_weight=weight, rope=plan, status=pool.status)
    slots = pool.slots(pos, req)
    live = slots >= 0
    bits = m.MLA_STATUS_BAD_INDEX | m.MLA_STATUS_BAD_PAGE
    assert int(pool.status) == bits
    y, t = L.row_values(_f64(rows)[live], pos[live], None if weight is None else _f64(weight), np.float32(1e-6), freq, 1.0,
                        "halves" if requests == 3 else "pairs")
    L.assert_cache_rows(pool.rows(slots[live]), y, t, kv)
    pool.check_untouched(slots[live])
    pool.status.zero_()
    out = torch.full((tokens, 640), 7.0, dtype=torch.bfloat16, device="cuda")
    m.mla_cache_gather(pool.problem, tokens, pool.dev, positions, pool.bt, out, requests=of, out_stride=640,
                       status=pool.status)
    assert int(pool.status) == bits
    want = np.full((tokens, 640), 7.0)
    want[slots == -2, :576] = 0.0
    want[live, :576] = L.gather_rows(pool.dev.cpu().numpy(), slots[live], kv)
    assert np.array_equal(_f64(out), want)
