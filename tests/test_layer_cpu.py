"""The operators that feed the decode (include/mla_layer.h) on the CPU: what
they refuse before any CUDA call, the rotary plan's table, and the oracle that
the GPU tests compare with against hand-worked values."""
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import fp4 as F4
from oracle import fp8 as F8
from oracle import layer as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20          # an aligned address that no refused call reads
B, C, D, E = (A * k for k in (1 << 10, 2 << 10, 3 << 10, 5 << 10))
INVALID, UNSUPPORTED, MISALIGNED = -1, -2, -3


@pytest.fixture(scope="module")
def m():
    from head_latent_attention_paged_gb300 import _build
    _build.build()
    import head_latent_attention_paged_gb300 as mod
    mod.load()
    return mod


def _refused(m, code, call, *a, **kw):
    with pytest.raises(m.MlaError) as e:
        call(*a, **kw)
    assert e.value.code == code, e.value.code


# ---------------------------------------------------------------- norm
@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(cols=32769), UNSUPPORTED),
    (dict(dtype=3), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(out_format=3), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(x_stride=63), INVALID), (dict(out_stride=63), INVALID), (dict(x_stride=2 ** 62), INVALID),
    (dict(residual_stride=63), INVALID), (dict(residual_out_stride=63), INVALID),
])
def test_norm_refuses_problems(m, kw, code):
    pr = m.make_norm_problem(**dict(dict(rows=4, cols=64), **kw))
    _refused(m, code, m.mla_rms_norm, pr, A, B, C, residual=D, residual_out=E)


def test_norm_refuses_pointers(m):
    pr = m.make_norm_problem(4, 64)
    norm = m.mla_rms_norm
    _refused(m, INVALID, norm, pr, None, None, A)
    _refused(m, INVALID, norm, pr, A, None, None)
    _refused(m, INVALID, norm, pr, A, None, B, residual_out=C)           # a sum without a residual
    _refused(m, INVALID, norm, pr, A, None, B, scales=C)                 # scales of a 16-bit output
    _refused(m, MISALIGNED, norm, pr, A + 1, None, B)
    _refused(m, MISALIGNED, norm, pr, A, B + 1, C)
    for fmt in (m.MLA_NORM_OUT_E4M3_E8M0, m.MLA_NORM_OUT_E4M3_ROW):
        q = m.make_norm_problem(4, 64, out_format=fmt)
        _refused(m, INVALID, norm, q, A, None, B)                        # no scales
        _refused(m, INVALID, norm, q, A, None, A, scales=C)              # codes on the input
        _refused(m, INVALID, norm, q, A, None, B, scales=B + 64)         # scales among the codes
    _refused(m, MISALIGNED, norm, m.make_norm_problem(4, 64, out_format=m.MLA_NORM_OUT_E4M3_ROW),
             A, None, B, scales=C + 2)
    q = m.make_norm_problem(4, 64, out_format=m.MLA_NORM_OUT_E4M3_E8M0, scale_stride=1)
    _refused(m, INVALID, norm, q, A, None, B, scales=C)
    # overlaps: shifted, with another stride, two outputs on one buffer
    _refused(m, INVALID, norm, pr, A, None, A + 2)
    _refused(m, INVALID, norm, m.make_norm_problem(4, 64, x_stride=128), A, None, A)
    _refused(m, INVALID, norm, pr, A, None, B, residual=C, residual_out=B)
    _refused(m, INVALID, norm, pr, A, None, B, residual=C, residual_out=C + 128)
    _refused(m, INVALID, norm, pr, A, B, B + 64)


def test_norm_of_no_rows_needs_no_buffers(m):
    m.mla_rms_norm(m.make_norm_problem(0, 64), None, None, None)


# ---------------------------------------------------------------- rope plan
def _plan_args(m, scaling):
    return dict(none=dict(), linear=dict(scaling=m.MLA_ROPE_SCALING_LINEAR, factor=4.0),
                parts=dict(scaling=m.MLA_ROPE_SCALING_PARTS, factor=8.0, original_positions=8192,
                           fast_rotations=4.0, slow_rotations=1.0),
                yarn=dict(scaling=m.MLA_ROPE_SCALING_YARN, factor=16.0, original_positions=4096,
                          fast_rotations=32.0, slow_rotations=1.0))[scaling]


@pytest.mark.parametrize("scaling", ["none", "linear", "parts", "yarn"])
@pytest.mark.parametrize("dim,theta", [(64, 1e6), (2, 1e4), (128, 1e4), (256, 5e5), (80, 1e6)])
def test_rope_plan_table(m, scaling, dim, theta):
    """turns[i] 2^-64 of a turn per position, within the rounding of a 53-bit
    frequency (a few units, from the power, the blend and the division), and
    the products with far positions the angle's fraction of a turn."""
    a = _plan_args(m, scaling)
    plan = m.mla_rope_plan(rope_dim=dim, theta=theta, **a)
    freq, amplitude = L.rope_frequencies(dim, theta, scaling, a.get("factor", 1.0),
                                         a.get("original_positions", 0), a.get("fast_rotations", 0),
                                         a.get("slow_rotations", 0))
    assert abs(plan.amplitude - amplitude) <= amplitude * L.U
    for i in range(dim // 2):
        turns = freq[i] / (2 * math.pi) * 2.0 ** 64
        assert abs(plan.turns[i] - turns) <= 8 * turns * 2.0 ** -53 + 1
    for pos in (0, 1, 131071, 2 ** 31 - 1):
        phase = (plan.turns[0] * pos) % 2 ** 64 / 2.0 ** 64
        want = math.fmod(pos * freq[0] / (2 * math.pi), 1.0)
        off = abs(phase - want)
        assert min(off, 1 - off) <= 16 * (pos + 1) * freq[0] / 6 * 2.0 ** -53


def test_rope_amplitude_and_fast_frequencies(m):
    assert m.mla_rope_plan(amplitude=0.5).amplitude == 0.5
    assert m.mla_rope_plan(scaling=m.MLA_ROPE_SCALING_YARN, factor=0.5, original_positions=64).amplitude == 1.0
    # positions stretched so far that a pair turns more than once per position
    plan = m.mla_rope_plan(scaling=m.MLA_ROPE_SCALING_LINEAR, factor=0.1)
    turn = 10.0 / (2 * math.pi)
    assert abs(plan.turns[0] / 2.0 ** 64 - (turn - 1.0)) < 1e-15


@pytest.mark.parametrize("kw,code", [
    (dict(layout=2), UNSUPPORTED), (dict(rope_dim=0), UNSUPPORTED), (dict(rope_dim=63), UNSUPPORTED),
    (dict(rope_dim=258), UNSUPPORTED), (dict(scaling=4), UNSUPPORTED), (dict(scaling=-1), UNSUPPORTED),
    (dict(theta=1.0), INVALID), (dict(theta=float("inf")), INVALID), (dict(theta=float("nan")), INVALID),
    (dict(amplitude=-1.0), INVALID), (dict(amplitude=float("nan")), INVALID), (dict(amplitude=1e300), INVALID),
    (dict(scaling=1, factor=0.0), INVALID), (dict(scaling=1, factor=float("nan")), INVALID),
    (dict(scaling=1, factor=5e-324), INVALID),                           # no finite frequency
    (dict(scaling=2, factor=2.0), INVALID),                              # no original length
    (dict(scaling=3, factor=2.0, original_positions=64, fast_rotations=1.0), INVALID),
    (dict(scaling=2, factor=2.0, original_positions=64, slow_rotations=0.0), INVALID),
])
def test_rope_plan_refuses(m, kw, code):
    _refused(m, code, m.mla_rope_plan, **kw)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), INVALID), (dict(num_heads=0), INVALID), (dict(head_dim=63), INVALID),
    (dict(rope_offset=-1), INVALID), (dict(rope_offset=193), INVALID), (dict(dtype=3), UNSUPPORTED),
    (dict(transposed=2), INVALID), (dict(x_token_stride=-1), INVALID),
    (dict(out_token_stride=0), INVALID), (dict(out_head_stride=255), INVALID),
    (dict(out_token_stride=1024, out_head_stride=300), INVALID), (dict(x_head_stride=2 ** 62), INVALID),
])
def test_rope_refuses_problems(m, kw, code):
    pr = m.make_rope_problem(**dict(dict(tokens=3, num_heads=4, head_dim=256), **kw))
    _refused(m, code, m.mla_rope, pr, m.mla_rope_plan(), A, B, C)


def test_rope_refuses_pointers(m):
    plan, pr = m.mla_rope_plan(), m.make_rope_problem(3, 4, 256)
    _refused(m, INVALID, m.mla_rope, pr, m.MlaRopePlan(), A, B)          # a plan nobody made
    _refused(m, INVALID, m.mla_rope, pr, plan, None, B)
    _refused(m, INVALID, m.mla_rope, pr, plan, A, None)
    _refused(m, MISALIGNED, m.mla_rope, pr, plan, A + 1, B)
    _refused(m, MISALIGNED, m.mla_rope, pr, plan, A, B + 2)
    _refused(m, INVALID, m.mla_rope, pr, plan, A, B, A + 512)            # neither in place nor apart
    _refused(m, INVALID, m.mla_rope, m.make_rope_problem(3, 4, 256, out_token_stride=2048), plan, A, B)
    _refused(m, INVALID, m.mla_rope, pr, plan, A, A + 1024)              # positions among the heads
    m.mla_rope(m.make_rope_problem(0, 4, 256), plan, None, None)


# ---------------------------------------------------------------- cache rows
def _cache(m, **kw):
    return m.make_problem(**dict(dict(batch=4, q_len=1, num_heads=1, page_size=64, num_pages=100,
                                      max_pages_per_seq=30), **kw))


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=48), UNSUPPORTED), (dict(kv_dtype=3), UNSUPPORTED), (dict(num_pages=0), INVALID),
    (dict(batch=-1), INVALID), (dict(kv_lora_rank=256), UNSUPPORTED), (dict(rope_dim=32), UNSUPPORTED),
    (dict(num_pages=2 ** 26), UNSUPPORTED),
])
def test_cache_calls_refuse_problems(m, kw, code):
    pr = _cache(m, **kw)
    _refused(m, code, m.mla_cache_append_tokens, pr, 8, A, B, C, D, requests=E)
    _refused(m, code, m.mla_cache_gather, pr, 8, D, B, C, A, requests=E)


def test_cache_calls_refuse_arguments(m):
    pr = _cache(m)
    far = 1 << 40        # past the pool

    def append(tokens=8, rows=far, positions=A, table=B, kv=D, **kw):
        m.mla_cache_append_tokens(pr, tokens, rows, positions, table, kv, **kw)

    def gather(tokens=8, rows=far, positions=A, table=B, kv=D, row_stride=576, **kw):
        m.mla_cache_gather(pr, tokens, kv, positions, table, rows, out_stride=row_stride, **kw)

    for call in (append, gather):
        _refused(m, INVALID, call, tokens=-1)
        for name in ("rows", "positions", "table", "kv"):
            _refused(m, INVALID, call, **{name: None})
        _refused(m, INVALID, call, tokens=9)                             # not the same number for each
        _refused(m, INVALID, call, row_stride=568)
        _refused(m, INVALID, call, row_stride=2 ** 61)
        _refused(m, MISALIGNED, call, row_stride=580)
        _refused(m, MISALIGNED, call, rows=far + 8)
        _refused(m, MISALIGNED, call, kv=D + 8)
        for name in ("positions", "table", "requests", "status"):
            _refused(m, MISALIGNED, call, **{name: A + 2})
        _refused(m, INVALID, call, rows=D + 1152)                        # inside the pool
        call(tokens=0, rows=None, positions=None, table=None, kv=None)
    _refused(m, MISALIGNED, append, norm_weight=C + 2)
    _refused(m, INVALID, append, norm_weight=C, norm_eps=-1.0)
    _refused(m, INVALID, append, norm_weight=C, norm_eps=float("nan"))
    _refused(m, INVALID, append, rope=m.MlaRopePlan())
    _refused(m, UNSUPPORTED, append, rope=m.mla_rope_plan(rope_dim=32))
    empty = _cache(m, batch=0)
    _refused(m, INVALID, m.mla_cache_gather, empty, 8, D, A, B, far)     # no request to share tokens


# ---------------------------------------------------------------- the oracle itself
def test_oracle_rounding_against_numpy():
    rng = np.random.default_rng(0)
    x = rng.standard_normal(4000) * 10.0 ** rng.uniform(-9, 5, 4000)
    assert np.array_equal(L.round_to(x, "f16"), x.astype(np.float16).astype(np.float64))
    x = rng.standard_normal(4000) * 10.0 ** rng.uniform(-44, 38, 4000)
    assert np.array_equal(L.round_to(x, "f32"), x.astype(np.float32).astype(np.float64))
    assert L.round_to(1 + 2.0 ** -8, "bf16") == 1.0 and L.round_to(1 + 3 * 2.0 ** -8, "bf16") == 1 + 2.0 ** -6


def test_oracle_quantisers_agree_with_the_cache_encoders():
    rng = np.random.default_rng(1)
    x = L.round_to(rng.standard_normal((50, 576)) * 10.0 ** rng.uniform(-3, 3, (50, 1)), "bf16")
    zero = np.zeros_like(x)
    for enc, kv in ((F8, "fp8"), (F4, "fp4")):
        raw = enc.quantize_rows(x)
        L.assert_cache_rows(raw, x, zero, kv)
        raw[7, 3] ^= 0x40                       # a planted mistake is seen
        with pytest.raises(AssertionError):
            L.assert_cache_rows(raw, x, zero, kv)


def test_oracle_rope_by_hand():
    """Quarter turns of unit vectors, both layouts, and the transposed map."""
    freq = np.array([math.pi / 2, math.pi])
    x = np.array([[1.0, 2.0, 3.0, 4.0]])
    y, _ = L.rope(x, [1], freq)
    assert np.allclose(y, [[-2, 1, -3, -4]])
    y, _ = L.rope(x, [1], freq, layout="halves")
    assert np.allclose(y, [[-3, -2, 1, -4]])
    y, _ = L.rope(x, [1], freq, amplitude=2.0, transposed=True)
    assert np.allclose(y, [[4, -2, -6, -8]])


def test_plain_c_consumer_of_the_layer_header(m, tmp_path):
    """A C99 program includes the header, links the library and makes a rotary plan."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no gcc")
    src = tmp_path / "layer.c"
    src.write_text('#include <stdio.h>\n#include "mla_layer.h"\n'
                   "int main(void) {\n"
                   "  mla_rope_config c = {MLA_ROPE_HALVES, 64, MLA_ROPE_SCALING_NONE, 0, 1e6, 1.0, 0, 0, 0};\n"
                   "  mla_rope_plan plan;\n"
                   "  if (mla_rope_make_plan(&c, &plan) != MLA_OK) return 1;\n"
                   "  if (mla_rms_norm(0, 0, 0, 0, 0, 0, 0, 0) != MLA_ERR_INVALID_ARGUMENT) return 2;\n"
                   '  printf("%g\\n", (double)plan.amplitude);\n  return 0;\n}\n')
    exe = tmp_path / "layer"
    lib = os.path.dirname(m.LIB_PATH)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe), m.LIB_PATH, f"-Wl,-rpath,{lib}"], check=True)
    assert subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.strip() == "1"
