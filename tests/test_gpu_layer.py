"""The operators that feed the decode (include/mla_layer.h) on the GPU against
the float64 oracle: every output lies between the roundings of y - t and y + t,
t the derived bound on the 32-bit arithmetic (oracle/layer.py)."""
import numpy as np
import pytest

from oracle import cache_append as CA
from oracle import fp4 as F4
from oracle import fp8 as F8
from oracle import layer as L
from mla_testlib import ensure_built
from test_layer_cpu import _plan_args

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"bf16": "bfloat16", "f16": "float16", "f32": "float32"}


@pytest.fixture(scope="module")
def m():
    ensure_built()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import head_latent_attention_paged_gb300 as mod
    return mod


def _dt(kind):
    return getattr(torch, DT[kind])


def _f64(t):
    return t.detach().cpu().double().numpy()


def _rand(rng, shape, kind, spread=0.0):
    x = rng.standard_normal(shape) * np.exp2(rng.uniform(-spread, spread, shape))
    return torch.from_numpy(x).to(_dt(kind)).cuda()


# ---------------------------------------------------------------- norm
class _Norm:
    """Buffers of one norm call, with a guard behind every row and output."""

    def __init__(self, m, rng, rows, cols, kind, out, residual, weight=True, pad=0, shift=0, eps=1e-6):
        dt, self.m, self.kind, self.fmt, self.rows, self.cols = _dt(kind), m, kind, out, rows, cols
        s = cols + pad
        self.eps = eps

        def wide(n, fill=None):
            base = _rand(rng, (n * s + shift,), kind, 2.0) if fill is None else torch.full(
                (n * s + shift,), fill, dtype=dt, device="cuda")
            return base, base[shift:].view(n, s)[:, :cols]

        self.x = wide(rows)[1]
        self.residual = wide(rows)[1] if residual else None
        self.weight = _rand(rng, (cols,), kind) if weight else None
        self.ro_base, self.ro = wide(rows, 7.0) if residual else (None, None)
        code = {"same": m.MLA_NORM_OUT_SAME, "mx": m.MLA_NORM_OUT_E4M3_E8M0, "row": m.MLA_NORM_OUT_E4M3_ROW}[out]
        self.scales = None
        if out == "same":
            self.out_base, self.out = wide(rows, 7.0)
        else:
            self.out_base = torch.full((rows * s + shift,), 0x55, dtype=torch.uint8, device="cuda")
            self.out = self.out_base[shift:].view(rows, s)[:, :cols]
            self.scales = (torch.full((rows, (cols + 31) // 32), 0x55, dtype=torch.uint8, device="cuda")
                           if out == "mx" else torch.full((rows,), 7.0, device="cuda"))
        self.problem = m.make_norm_problem(rows, cols, {"bf16": 0, "f16": 1, "f32": 2}[kind], code, eps,
                                           x_stride=s, residual_stride=s, residual_out_stride=s, out_stride=s)

    def run(self, stream=None):
        self.m.mla_rms_norm(self.problem, self.x, self.weight, self.out, residual=self.residual,
                            residual_out=self.ro, scales=self.scales, stream=stream)

    def reference(self):
        return L.rms_norm(_f64(self.x), None if self.residual is None else _f64(self.residual),
                          None if self.weight is None else _f64(self.weight), np.float32(self.eps))

    def check_rows(self, keep, label=""):
        """Check some of the rows, and the guards of all."""
        names = ("x", "residual", "ro", "out", "scales")
        whole = {k: getattr(self, k) for k in names}
        for k, v in whole.items():
            setattr(self, k, None if v is None else v[keep])
        bases, self.out_base, self.ro_base = (self.out_base, self.ro_base), None, None
        self.check(label=label)
        for k, v in whole.items():
            setattr(self, k, v)
        self.out_base, self.ro_base = bases
        self.check_guards(label)

    def check(self, ref=None, label=""):
        h, y, t = ref or self.reference()
        if self.ro is not None:
            L.assert_rounded(_f64(self.ro), h, np.abs(h) * L.U, self.kind, f"{label} h")
        if self.fmt == "same":
            L.assert_rounded(_f64(self.out), y, t, self.kind, label)
        elif self.fmt == "mx":
            L.assert_quantised(F8.e4m3_to_f64(self.out.cpu().numpy()),
                               self.scales.cpu().numpy().astype(np.int64) - 127, y, t, 32, "e4m3", label)
        else:
            s = _f64(self.scales)[:, None]
            amax = np.maximum(np.abs(y).max(-1, keepdims=True) / 448.0, 2.0 ** -126)
            assert (np.abs(s - amax) <= t.max(-1, keepdims=True) / 448.0 + 2 * L.U * amax).all(), label
            # the scale's reciprocal and the product: one rounding each
            v, tv = y / s, t / s + 3 * L.U * np.abs(y / s)
            code = F8.e4m3_to_f64(self.out.cpu().numpy())
            ok = (code >= F8._round_to_e4m3(v - tv)) & (code <= F8._round_to_e4m3(v + tv))
            assert ok.all(), (label, int((~ok).sum()))
        self.check_guards(label)

    def check_guards(self, label=""):
        for base, view in ((self.out_base, self.out), (self.ro_base, self.ro)):
            if base is None:
                continue
            fill = 0x55 if base.dtype == torch.uint8 else 7.0
            view.fill_(fill)
            assert bool((base == fill).all()), f"{label}: elements behind the rows were written"


COLS = [1, 2, 7, 8, 31, 32, 33, 64, 127, 250, 256, 512, 768, 1000, 1344, 2048, 2881, 4096, 5120,
        8184, 8192, 10000, 16384, 20001, 32768]


@pytest.mark.parametrize("out", ["same", "mx", "row"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_norm_widths(m, kind, out):
    """Every width packed, with a residual: rows on and off 16-byte
    boundaries, whole and broken groups, from one element to the limit."""
    rng = np.random.default_rng(11)
    for cols in COLS:
        for rows in (1, 5):
            n = _Norm(m, rng, rows, cols, kind, out, residual=True)
            n.run()
            n.check(label=f"{kind} {out} {rows}x{cols}")


@pytest.mark.parametrize("out", ["same", "mx", "row"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_norm_widths_of_many_rows(m, kind, out):
    """The variants that many rows take, at each one's widths."""
    rng = np.random.default_rng(13)
    for cols in (40, 100, 130, 257, 512, 768, 1000, 1030, 2048, 2881, 4096, 4100, 8191, 8192, 10001, 16384, 20001,
                 32767, 32768):
        rows = 515
        n = _Norm(m, rng, rows, cols, kind, out, residual=True)
        n.run()
        n.check_rows(torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, 254, 511, 512, 513, 514]), f"{kind} {out} {cols}")


@pytest.mark.parametrize("out", ["same", "mx", "row"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,shift,residual,weight", [
    (3, 768, 576, 0, False, True), (130, 512, 8, 0, True, False), (3, 512, 4, 0, True, True),
    (9, 768, 576, 8, True, True), (4, 640, 0, 1, True, True), (7, 96, 3, 2, False, False),
    (700, 64, 0, 0, True, True), (2, 2048, 1, 0, True, True), (1000, 2050, 0, 0, False, True),
    (33, 4095, 1, 0, True, True),
])
def test_norm_strides(m, kind, out, rows, cols, pad, shift, residual, weight):
    """Slices of wider rows and shifted buffers: nothing behind a row or in
    front of the buffer's slice is written."""
    n = _Norm(m, np.random.default_rng(5), rows, cols, kind, out, residual, weight, pad, shift)
    n.run()
    n.check()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(37, 96), (37, 777), (600, 777), (37, 4096), (3, 2881), (520, 2881)])
@pytest.mark.parametrize("which", ["out=x", "ro=residual", "ro=x", "out=x ro=residual", "out=residual"])
def test_norm_in_place(m, kind, rows, cols, which):
    n = _Norm(m, np.random.default_rng(6), rows, cols, kind, "same", True)
    ref = n.reference()
    if "out=x" in which:
        n.out_base, n.out = n.x, n.x
    if "out=residual" in which:
        n.out_base = n.out = n.residual
        n.ro = n.ro_base = None
    if "ro=residual" in which:
        n.ro_base, n.ro = n.residual, n.residual
    if "ro=x" in which:
        n.ro_base, n.ro = n.x, n.x
    n.run()
    n.check(ref)


def test_norm_columns_of_one_buffer(m):
    """Input and output as two column ranges of one wide buffer."""
    rng = np.random.default_rng(3)
    buf = _rand(rng, (50, 1344), "bf16")
    before = buf.clone()
    x, out = buf[:, :640], buf[:, 640:1280]
    _, y, t = L.rms_norm(_f64(x))
    m.mla_rms_norm(m.make_norm_problem(50, 640, x_stride=1344, out_stride=1344), x, None, out)
    L.assert_rounded(_f64(out), y, t, "bf16")
    assert torch.equal(buf[:, :640], before[:, :640]) and torch.equal(buf[:, 1280:], before[:, 1280:])


@pytest.mark.parametrize("out", ["same", "mx", "row"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cols", [64, 100, 4096])
def test_norm_special_rows(m, kind, out, cols):
    """Rows of zeros, of the smallest and of large values, one with a NaN and
    one with an infinity: finite rows are right, the others stay in their
    own rows."""
    rng = np.random.default_rng(8)
    n = _Norm(m, rng, 8, cols, kind, out, residual=False)
    tiny, big = (6e-8, 6e4) if kind == "f16" else (1e-38, 1e17)
    n.x[0] = 0.0
    n.x[1] = tiny
    n.x[2] *= big / 60 if kind == "f16" else big
    n.x[4, 3] = float("nan")
    n.x[6, cols - 1] = float("-inf")
    n.weight[5] = 0.0
    n.run()
    torch.cuda.synchronize()
    keep = [0, 1, 2, 3, 5, 7]
    h, y, t = n.reference()
    code = None if out == "same" else F8.e4m3_to_f64(n.out.cpu().numpy())
    if out == "same":
        assert bool(n.out[4].isnan().all())
        assert bool(n.out[6, cols - 1].isnan()) and bool((n.out[6, :cols - 1] == 0).all())
    else:
        assert np.isnan(code[4]).all() and np.isnan(code[6, cols - 1])
        if out == "row":
            assert bool(n.scales[[4, 6]].isnan().all())
        else:                            # a NaN does not enter its group's scale
            assert (code[6, :cols - 1] == 0).all() and bool((n.scales[[4, 6]] == 0).all())
    if out == "row":                     # an all-zero row: the smallest scale, zero codes
        assert float(n.scales[0]) == 2.0 ** -126 and (code[0] == 0).all()
    sub = _Norm(m, rng, 6, cols, kind, out, residual=False)
    sub.out_base = sub.out = n.out[keep]
    sub.scales = None if n.scales is None else n.scales[keep]
    sub.check((h[keep], y[keep], t[keep]))


def test_norm_many_rows_past_32_bits_of_offset(m):
    """More than 2^32 bytes of input: the last rows are read where they are."""
    rows, cols = 1 << 20, 2304
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = _rand(np.random.default_rng(2), (7, cols), "bf16")
    x[-7:] = tail
    out = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
    m.mla_rms_norm(m.make_norm_problem(rows, cols, out_format=m.MLA_NORM_OUT_E4M3_E8M0), x, None, out, scales=scales)
    _, y, t = L.rms_norm(_f64(tail))
    L.assert_quantised(F8.e4m3_to_f64(out[-7:].cpu().numpy()), scales[-7:].cpu().numpy().astype(np.int64) - 127,
                       y, t, 32, "e4m3")
    assert int(out[:-7].max()) == 0 and int(scales[:-7].max()) == 0


# ---------------------------------------------------------------- rope
def _rope_case(m, rng, tokens, heads, head_dim, offset, dim, layout, kind, scaling, in_place, transposed,
               longest=131072, order="token", pad=0, shift=0, positions=None):
    a = _plan_args(m, scaling)
    plan = m.mla_rope_plan(rope_dim=dim, layout=m.MLA_ROPE_HALVES if layout == "halves" else m.MLA_ROPE_INTERLEAVED, **a)
    freq, amplitude = L.rope_frequencies(dim, 1e6, scaling, a.get("factor", 1.0), a.get("original_positions", 0),
                                         a.get("fast_rotations", 0), a.get("slow_rotations", 0))
    D = head_dim + pad
    shape = (tokens, heads, D) if order == "token" else (heads, tokens, D)

    def make(fill=None):
        n = tokens * heads * D + shift
        base = _rand(rng, (n,), kind) if fill is None else torch.full((n,), fill, dtype=_dt(kind), device="cuda")
        v = base[shift:].view(shape)[..., :head_dim]
        return base, v if order == "token" else v.transpose(0, 1)

    _, x = make()
    base, out = (None, x) if in_place else make(7.0)
    if positions is None:
        positions = rng.integers(0, longest, tokens).astype(np.int32)
        positions[::7] = -1 if tokens > 3 else positions[::7]
    pos = torch.from_numpy(positions).cuda()
    before, x64 = out.clone(), _f64(x)
    pr = m.make_rope_problem(tokens, heads, head_dim, offset, {"bf16": 0, "f16": 1, "f32": 2}[kind],
                             int(transposed), x.stride(0), x.stride(1), out.stride(0), out.stride(1))
    m.mla_rope(pr, plan, x, pos, None if in_place else out)
    y, t = L.rope(x64[..., offset:offset + dim], np.maximum(positions, 0), freq, float(np.float32(amplitude)),
                  layout, transposed)
    live, got = positions >= 0, _f64(out)
    L.assert_rounded(got[live][..., offset:offset + dim], y[live], t[live], kind)
    rest = np.r_[0:offset, offset + dim:head_dim]
    assert np.array_equal(got[live][..., rest], x64[live][..., rest])
    assert torch.equal(out[torch.from_numpy(~live).cuda()], before[torch.from_numpy(~live).cuda()])
    if base is not None:
        out.fill_(7.0)
        assert bool((base == 7.0).all()), "elements outside the heads were written"
    if not in_place:
        assert np.array_equal(_f64(x), x64)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("tokens,heads,head_dim,offset,dim", [
    (1, 1, 64, 0, 64), (9, 20, 256, 192, 64), (130, 3, 128, 0, 128), (5, 7, 96, 72, 24), (4, 2, 40, 3, 6),
    (17, 64, 192, 128, 64), (3, 5, 2, 0, 2), (6, 1, 256, 0, 256), (33, 12, 80, 0, 80), (2, 200, 64, 32, 32),
    (600, 20, 256, 192, 64),
])
def test_rope_shapes(m, kind, layout, in_place, tokens, heads, head_dim, offset, dim):
    _rope_case(m, np.random.default_rng(tokens), tokens, heads, head_dim, offset, dim, layout, kind, "none",
               in_place, False)


@pytest.mark.parametrize("scaling", ["linear", "parts", "yarn"])
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_rope_scalings(m, scaling, transposed, layout):
    _rope_case(m, np.random.default_rng(1), 40, 5, 128, 64, 64, layout, "f32", scaling, True, transposed, 1 << 20)


@pytest.mark.parametrize("order,pad,shift", [("head", 0, 0), ("token", 8, 0), ("token", 3, 0), ("head", 8, 8),
                                             ("token", 0, 1), ("head", 5, 3)])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rope_strides(m, order, pad, shift, in_place, kind):
    _rope_case(m, np.random.default_rng(2), 11, 6, 128, 64, 64, "pairs", kind, "none", in_place, False,
               order=order, pad=pad, shift=shift)


def test_rope_far_positions(m):
    """Up to the last 32-bit position: the angle's fraction of a turn is kept."""
    pos = np.array([0, 1, 2, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, 131071, -2 ** 31], dtype=np.int32)
    for layout in ("pairs", "halves"):
        _rope_case(m, np.random.default_rng(4), len(pos), 4, 64, 0, 64, layout, "f32", "none", True, False,
                   positions=pos)


def test_rope_of_a_broadcast_input(m):
    """One key turned for every head of an output: a head stride of 0 on the
    input, whose elements are read again for each head."""
    rng = np.random.default_rng(9)
    x, pos = _rand(rng, (30, 80), "bf16"), rng.integers(0, 5000, 30).astype(np.int32)
    out = torch.zeros(30, 7, 80, dtype=torch.bfloat16, device="cuda")
    pr = m.make_rope_problem(30, 7, 80, rope_offset=16, x_token_stride=80, x_head_stride=0, out_token_stride=560,
                             out_head_stride=80)
    m.mla_rope(pr, m.mla_rope_plan(), x, torch.from_numpy(pos).cuda(), out)
    freq, _ = L.rope_frequencies(64)
    y, t = L.rope(_f64(x)[:, 16:], pos, freq)
    for h in range(7):
        assert torch.equal(out[:, h, :16], x[:, :16])
        L.assert_rounded(_f64(out)[:, h, 16:], y, t, "bf16")


def test_rope_past_32_bits_of_offset(m):
    """Heads of more than 2^32 bytes, in place: the last tokens are turned
    where they are, the others as their positions say (-1: not at all)."""
    tokens, heads, head_dim = (1 << 17) + 3, 64, 256
    x = torch.zeros(tokens, heads, head_dim, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(10)
    x[-5:] = _rand(rng, (5, heads, head_dim), "bf16")
    x[7] = 1.0
    before = _f64(x[-5:])
    pos = torch.full((tokens,), -1, dtype=torch.int32, device="cuda")
    pos[-5:] = torch.tensor([0, 5, 77, -1, 100000], dtype=torch.int32)
    m.mla_rope(m.make_rope_problem(tokens, heads, head_dim, rope_offset=192), m.mla_rope_plan(), x, pos)
    freq, _ = L.rope_frequencies(64)
    y, t = L.rope(before[..., 192:], [0, 5, 77, 0, 100000], freq)
    y[3], t[3] = before[3, :, 192:], 0.0
    got = _f64(x[-5:])
    L.assert_rounded(got[..., 192:], y, t, "bf16")
    assert np.array_equal(got[..., :192], before[..., :192])
    assert bool((x[7] == 1.0).all()) and bool((x[8:-5] == 0).all())


def test_rope_gradient(m):
    """The transposed map is the gradient: <R x, g> = <x, R^T g> for every pair
    of random vectors (the sums' own error bound), and it matches central
    differences of a weighted sum of R x (a linear map: any step is exact but
    for rounding; step 1)."""
    rng = np.random.default_rng(5)
    tokens, heads, dim = 12, 3, 64
    plan = m.mla_rope_plan(scaling=m.MLA_ROPE_SCALING_YARN, factor=8.0, original_positions=4096)
    pos = torch.from_numpy(rng.integers(0, 100000, tokens).astype(np.int32)).cuda()
    x, g = (_rand(rng, (tokens, heads, dim), "f32") for _ in range(2))

    def turned(v, transposed):
        out = torch.empty_like(v)
        m.mla_rope(m.make_rope_problem(tokens, heads, dim, dtype=m.MLA_DTYPE_F32, transposed=transposed), plan, v,
                   pos, out)
        return out

    gx = turned(g, 1)
    a, b = (turned(x, 0).double() * g.double()).sum(-1), (x.double() * gx.double()).sum(-1)
    # each of the 64 products is off by at most 8 U A (|a| + |b|) |g|
    bound = 8 * L.U * 1.3 * 4 * (x.double().norm(dim=-1) * g.double().norm(dim=-1))
    assert bool(((a - b).abs() <= bound).all())
    for i in (0, 1, 31, 63):
        d = torch.zeros_like(x)
        d[..., i] = 1.0
        num = ((turned(x + d, 0).double() - turned(x - d, 0).double()) * g.double()).sum(-1) / 2
        slack = 2 * 8 * L.U * 1.3 * 4 * (x.double().norm(dim=-1) + 1) * g.double().norm(dim=-1)
        assert bool(((num - gx[..., i].double()).abs() <= slack).all())


# ---------------------------------------------------------------- cache rows
class _Pool:
    """A paged pool with a shuffled block table and a pattern in every byte."""

    def __init__(self, m, rng, kv, page, requests, max_pages, pool=None, spare=3):
        self.m, self.kv, self.page, self.B, self.max_pages = m, kv, page, requests, max_pages
        self.num_pages = pool or requests * max_pages + spare
        self.table = rng.permutation(self.num_pages)[:requests * max_pages].reshape(requests, max_pages).astype(np.int32)
        self.row_bytes = {"bf16": 1152, "fp8": 594, "fp4": 324}[kv]
        self.host = rng.integers(0, 256, (self.num_pages * page, self.row_bytes), dtype=np.uint8)
        if kv == "bf16":
            bits = self.host.view(np.uint16)
            bits[(bits & 0x7F80) == 0x7F80] = 0          # no NaN or infinity
        self.dev = torch.from_numpy(self.host.copy()).cuda()
        self.bt = torch.from_numpy(self.table).cuda()
        self.problem = m.make_problem(requests, 1, 1, page, self.num_pages, max_pages, kv_dtype={"bf16": 0, "fp8": 1, "fp4": 2}[kv])
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def slots(self, positions, requests):
        return L.slots_of(positions, requests, self.table, self.page, self.num_pages)

    def rows(self, slots):
        raw = self.dev[torch.from_numpy(slots).cuda()].cpu().numpy()
        if self.kv != "bf16":
            return raw
        return (raw.view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)

    def check_untouched(self, written):
        keep = np.ones(len(self.host), dtype=bool)
        keep[written] = False
        assert np.array_equal(self.dev.cpu().numpy()[keep], self.host[keep]), "another slot was written"


def _tokens(rng, pool, tokens):
    """Distinct (request, position) pairs in any order, some -1."""
    cap = pool.max_pages * pool.page
    pick = rng.choice(pool.B * cap, tokens, replace=False)
    requests, positions = (pick // cap).astype(np.int32), (pick % cap).astype(np.int32)
    if tokens > 3:
        positions[rng.integers(0, tokens, tokens // 5)] = -1
    return requests, positions


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("tokens,requests,norm,layout,scaling,stride", [
    (1, 1, True, "pairs", "none", 576), (5, 3, False, "halves", "none", 584), (67, 4, True, "halves", "yarn", 1344),
    (300, 2, True, "pairs", "parts", 1344), (129, 5, False, None, None, 576), (130, 5, True, None, None, 576),
    (64, 3, False, "pairs", "linear", 640),
])
def test_append_tokens(m, kv, page, tokens, requests, norm, layout, scaling, stride):
    rng = np.random.default_rng(tokens + page)
    pool = _Pool(m, rng, kv, page, requests, max(1, -(-400 // page)))
    req, pos = _tokens(rng, pool, tokens)
    wide = _rand(rng, (tokens, stride), "bf16", 3.0)
    rows = wide[:, stride - 576:]
    weight = _rand(rng, (512,), "bf16") if norm else None
    plan = freq = None
    amplitude = 1.0
    if layout:
        a = _plan_args(m, scaling)
        plan = m.mla_rope_plan(layout=m.MLA_ROPE_HALVES if layout == "halves" else m.MLA_ROPE_INTERLEAVED, **a)
        freq, amplitude = L.rope_frequencies(64, 1e6, scaling, a.get("factor", 1.0), a.get("original_positions", 0),
                                             a.get("fast_rotations", 0), a.get("slow_rotations", 0))
    m.mla_cache_append_tokens(pool.problem, tokens, rows, torch.from_numpy(pos).cuda(), pool.bt, pool.dev,
                              requests=torch.from_numpy(req).cuda(), row_stride=stride, norm_weight=weight,
                              norm_eps=1e-5, rope=plan, status=pool.status)
    live = pos >= 0
    slots = pool.slots(pos, req)
    y, t = L.row_values(_f64(rows)[live], pos[live], None if weight is None else _f64(weight), np.float32(1e-5), freq,
                        float(np.float32(amplitude)), layout or "pairs")
    L.assert_cache_rows(pool.rows(slots[live]), y, t, kv)
    pool.check_untouched(slots[live])
    assert int(pool.status) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("q", [1, 3])
def test_append_tokens_agrees_with_the_one_token_append(m, kv, q):
    """Without norm and rope: the bytes of mla_cache_append and of the oracle,
    for rows at the quantisers' edges; requests by their order."""
    from test_gpu_append import _special_rows
    rng = np.random.default_rng(9)
    B, page = 6, 64
    pool = _Pool(m, rng, kv, page, B, 2)
    rows = np.concatenate([_special_rows(rng, B) for _ in range(q)])
    pos = rng.permuted(np.tile(np.arange(2 * page), (B, 1)), axis=1)[:, :q].astype(np.int32)
    m.mla_cache_append_tokens(pool.problem, B * q, torch.from_numpy(rows.view(np.int16)).cuda(),
                              torch.from_numpy(pos).cuda(), pool.bt, pool.dev, status=pool.status)
    old = torch.from_numpy(pool.host.copy()).cuda()
    want = pool.host.view(np.uint16).reshape(-1, page, 576) if kv == "bf16" else pool.host.reshape(pool.num_pages, -1)
    for j in range(q):
        mine = rows.reshape(B, q, 576)[:, j]
        m.mla_cache_append(pool.problem, torch.from_numpy(np.ascontiguousarray(mine).view(np.int16)).cuda(),
                           torch.from_numpy(np.ascontiguousarray(pos[:, j])).cuda(), pool.bt, old)
        want = CA.append_rows(want, mine, pos[:, j], pool.table, page, kv)
    assert torch.equal(pool.dev, old)
    assert np.array_equal(pool.dev.cpu().numpy().reshape(-1), want.view(np.uint8).reshape(-1))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_append_tokens_keeps_nan(m, kv):
    """A NaN is stored as one (code in FP8, the group's scale in FP4), in its
    own row; a norm spreads it over the row's latent."""
    rng = np.random.default_rng(12)
    pool = _Pool(m, rng, kv, 64, 1, 1)
    rows = _rand(rng, (4, 576), "bf16")
    rows[1, 100] = float("nan")
    rows[2, 570] = float("nan")
    rows[3, 32:64] = float("nan")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    for norm in (False, True):
        weight = torch.ones(512, dtype=torch.bfloat16, device="cuda") if norm else None
        m.mla_cache_append_tokens(pool.problem, 4, rows, pos, pool.bt, pool.dev, norm_weight=weight)
        out = torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda")
        m.mla_cache_gather(pool.problem, 4, pool.dev, pos, pool.bt, out)
        nan = out.isnan().cpu().numpy()
        want = np.zeros((4, 576), dtype=bool)
        group = 16 if kv == "fp4" else 1
        for r, cs in ((1, [100]), (2, [570]), (3, range(32, 64))):
            for c in cs:
                want[r, c // group * group:c // group * group + group] = True
        if norm:
            want[[1, 3], :512] = True
        assert np.array_equal(nan, want)


def _all_codes(rng, kv, slots):
    """Rows with every code and scale byte, NaN and extreme scales among them."""
    raw = rng.integers(0, 256, (slots, {"bf16": 1152, "fp8": 594, "fp4": 324}[kv]), dtype=np.uint8)
    if kv != "bf16":
        n = 576 if kv == "fp8" else 288
        raw[1, n:], raw[2, n:], raw[3, n:], raw[4, n:] = 0, 1, 254, 255
        raw[5:8, n:] = rng.integers(0, 12, raw[5:8, n:].shape)
    return raw


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("tokens,requests,stride", [(1, 1, 576), (37, 3, 640), (500, 2, 576), (260, 4, 1152)])
def test_gather_bits(m, kv, page, tokens, requests, stride):
    """Every value exact (code * 2^(scale - 127) rounded to bf16); rows of
    negative positions and columns behind a row as they were."""
    rng = np.random.default_rng(page + tokens)
    pool = _Pool(m, rng, kv, page, requests, max(1, -(-400 // page)))
    pool.host = _all_codes(rng, kv, len(pool.host))
    pool.dev = torch.from_numpy(pool.host).cuda()
    req, pos = _tokens(rng, pool, tokens)
    out = torch.full((tokens, stride), 7.0, dtype=torch.bfloat16, device="cuda")
    m.mla_cache_gather(pool.problem, tokens, pool.dev, torch.from_numpy(pos).cuda(), pool.bt, out,
                       requests=torch.from_numpy(req).cuda(), out_stride=stride, status=pool.status)
    got, live = _f64(out), pos >= 0
    want = np.full((tokens, stride), 7.0)
    want[live, :576] = L.gather_rows(pool.host, pool.slots(pos, req)[live], kv)
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(np.signbit(got[live]) | np.isnan(got[live]), np.signbit(want[live]) | np.isnan(want[live]))
    assert int(pool.status) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_tokens_without_a_slot(m, kv):
    """Bad requests, positions and pages: reported, not written, gathered as
    zeros; the rows beside them are right."""
    rng = np.random.default_rng(21)
    pool = _Pool(m, rng, kv, 32, 3, 4)
    pool.table[1, 2] = pool.num_pages
    pool.table[2, 0] = -1
    pool.bt = torch.from_numpy(pool.table).cuda()
    req = np.array([0, 3, -1, 0, 1, 2, 1, 0, 2**31 - 1], dtype=np.int32)
    pos = np.array([5, 1, 2, 4 * 32, 70, 3, 0, 127, 2**31 - 1], dtype=np.int32)
    ok = np.array([1, 0, 0, 0, 0, 0, 1, 1, 0], dtype=bool)
    rows = _rand(rng, (len(req), 576), "bf16")
    put = [torch.from_numpy(a).cuda() for a in (req, pos)]
    m.mla_cache_append_tokens(pool.problem, len(req), rows, put[1], pool.bt, pool.dev, requests=put[0], status=pool.status)
    assert int(pool.status) == m.MLA_STATUS_BAD_INDEX | m.MLA_STATUS_BAD_PAGE
    slots = pool.slots(pos, req)
    assert np.array_equal(slots >= 0, ok)
    L.assert_cache_rows(pool.rows(slots[ok]), _f64(rows)[ok], np.zeros((ok.sum(), 576)), kv)
    pool.check_untouched(slots[ok])
    out = torch.full((len(req), 576), 7.0, dtype=torch.bfloat16, device="cuda")
    for status, bits in ((pool.status, m.MLA_STATUS_BAD_INDEX | m.MLA_STATUS_BAD_PAGE), (None, 0)):
        pool.status.zero_()
        m.mla_cache_gather(pool.problem, len(req), pool.dev, put[1], pool.bt, out, requests=put[0], status=status)
        assert int(pool.status) == bits
        assert bool((out[torch.from_numpy(~ok).cuda()] == 0).all())
        assert np.array_equal(_f64(out)[ok], L.gather_rows(pool.dev.cpu().numpy(), slots[ok], kv))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_rows_past_32_bits_of_offset(m, kv):
    """A pool of more than 2^32 bytes: rows at its end are written and read."""
    row = {"bf16": 1152, "fp8": 594, "fp4": 324}[kv]
    page, pages = 128, (1 << 32) // (row * 128) + 40
    dev = torch.zeros(pages, page * row, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[pages - 1, pages - 2, 0]], dtype=torch.int32, device="cuda")
    pr = m.make_problem(1, 1, 1, page, pages, 3, kv_dtype={"bf16": 0, "fp8": 1, "fp4": 2}[kv])
    rng = np.random.default_rng(1)
    rows = _rand(rng, (3 * page, 576), "bf16")
    pos = torch.arange(3 * page, dtype=torch.int32, device="cuda")
    m.mla_cache_append_tokens(pr, 3 * page, rows, pos, table, dev)
    raw = torch.cat([dev[-1:], dev[-2:-1], dev[:1]]).view(3 * page, row).cpu().numpy()
    y = _f64(rows)
    got = raw if kv != "bf16" else (raw.view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    L.assert_cache_rows(got, y, np.zeros_like(y), kv)
    assert int(dev[1:-2].max()) == 0
    out = torch.empty_like(rows)
    m.mla_cache_gather(pr, 3 * page, dev, pos, table, out)
    assert np.array_equal(_f64(out), L.gather_rows(raw, np.arange(3 * page), kv))


# ---------------------------------------------------------------- streams and graphs
def test_addresses_in_place_of_tensors(m):
    """The calls take device addresses and stream handles as well."""
    rng = np.random.default_rng(31)
    stream = torch.cuda.Stream()
    n = _Norm(m, rng, 9, 96, "bf16", "row", True)
    pool = _Pool(m, rng, "fp4", 32, 3, 2)
    rows, q = _rand(rng, (6, 576), "bf16"), _rand(rng, (6, 2, 64), "bf16")
    pos = torch.tensor([0, 33, 5, 6, 63, 1], dtype=torch.int32, device="cuda")
    out, q0 = torch.zeros_like(rows), _f64(q)
    torch.cuda.synchronize()
    st = stream.cuda_stream
    m.mla_rms_norm(n.problem, n.x.data_ptr(), n.weight.data_ptr(), n.out.data_ptr(), residual=n.residual.data_ptr(),
                   residual_out=n.ro.data_ptr(), scales=n.scales.data_ptr(), stream=st)
    m.mla_rope(m.make_rope_problem(6, 2, 64), m.mla_rope_plan(), q.data_ptr(), pos.data_ptr(), stream=st)
    m.mla_cache_append_tokens(pool.problem, 6, rows.data_ptr(), pos.data_ptr(), pool.bt.data_ptr(), pool.dev.data_ptr(),
                              status=pool.status.data_ptr(), stream=st)
    m.mla_cache_gather(pool.problem, 6, pool.dev.data_ptr(), pos.data_ptr(), pool.bt.data_ptr(), out.data_ptr(), stream=st)
    torch.cuda.synchronize()
    n.check()
    freq, _ = L.rope_frequencies(64)
    y, t = L.rope(q0, pos.cpu().numpy(), freq)
    L.assert_rounded(_f64(q), y, t, "bf16")
    slots = pool.slots(pos.cpu().numpy(), np.repeat(np.arange(3), 2))
    L.assert_cache_rows(pool.rows(slots), _f64(rows), np.zeros((6, 576)), "fp4")
    assert np.array_equal(_f64(out), L.gather_rows(pool.dev.cpu().numpy(), slots, "fp4"))


def test_calls_on_streams_and_in_a_graph(m):
    """The four operators on a side stream, two sets of buffers at a time on
    two streams, and captured and replayed on new inputs: the same bits."""
    rng = np.random.default_rng(30)
    sets = []
    for k in range(2):
        pool = _Pool(m, rng, "fp8", 64, 3, 4)
        sets.append(dict(norm=_Norm(m, rng, 60, 768, "bf16", "mx", True), q=_rand(rng, (60, 4, 256), "bf16"), pool=pool,
                         rows=_rand(rng, (60, 576), "bf16"), w=_rand(rng, (512,), "bf16"),
                         pos=torch.from_numpy(np.tile(rng.permutation(256)[:20], 3).astype(np.int32)).cuda(),
                         out=torch.empty(60, 576, dtype=torch.bfloat16, device="cuda")))
    plan, rp = m.mla_rope_plan(), m.make_rope_problem(60, 4, 256, rope_offset=192)

    def step(s, stream):
        s["norm"].run(stream)
        m.mla_rope(rp, plan, s["q"], s["pos"], stream=stream)
        m.mla_cache_append_tokens(s["pool"].problem, 60, s["rows"], s["pos"], s["pool"].bt, s["pool"].dev,
                                  norm_weight=s["w"], rope=plan, stream=stream)
        m.mla_cache_gather(s["pool"].problem, 60, s["pool"].dev, s["pos"], s["pool"].bt, s["out"], stream=stream)

    def results(s):
        return [t.clone() for t in (s["norm"].out, s["norm"].scales, s["norm"].ro, s["q"], s["pool"].dev, s["out"])]

    start = [s["q"].clone() for s in sets]
    for s in sets:
        step(s, None)
    torch.cuda.synchronize()
    want = [results(s) for s in sets]
    for s, q in zip(sets, start):
        s["q"].copy_(q)
        s["out"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for s, st in zip(sets, streams):
        step(s, st)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(results(s), w))
    g = torch.cuda.CUDAGraph()
    sets[0]["q"].copy_(start[0])
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=streams[0]):
        step(sets[0], streams[0])
    for name in ("rows", "pos", "w"):                    # new inputs in the captured buffers
        sets[0][name].copy_(sets[1][name])
    sets[0]["q"].copy_(start[1])
    for name in ("x", "residual", "weight"):
        getattr(sets[0]["norm"], name).copy_(getattr(sets[1]["norm"], name))
    g.replay()
    torch.cuda.synchronize()
    got = results(sets[0])
    for i in (0, 1, 2, 3, 5):
        assert torch.equal(got[i], want[1][i])
