"""The rotary plan's table against the frequencies in 60 decimal digits: the
bound that include/mla_layer.h states on an angle."""
import decimal
from decimal import Decimal as D

import pytest

PI = D("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module")
def m():
    from head_latent_attention_paged_gb300 import _build
    _build.build()
    import head_latent_attention_paged_gb300 as mod
    mod.load()
    return mod


@pytest.mark.parametrize("dim,theta", [(64, 1e6), (256, 5e5), (2, 1e4), (80, 1.5), (128, 1e300)])
@pytest.mark.parametrize("factor", [1.0, 4.0, 40.0, 0.75, 0.1, 1e-3, 1e-6, 3e-9])
def test_turns_of_scaled_frequencies(m, dim, theta, factor):
    with decimal.localcontext() as c:
        c.prec = 60
        for scaling in (m.MLA_ROPE_SCALING_NONE, m.MLA_ROPE_SCALING_LINEAR, m.MLA_ROPE_SCALING_PARTS):
            plan = m.mla_rope_plan(rope_dim=dim, theta=theta, scaling=scaling, factor=factor, original_positions=4096,
                                   fast_rotations=4.0, slow_rotations=1.0)
            bound = D(2) ** -52 * (1 if scaling == m.MLA_ROPE_SCALING_NONE else max(1, 1 / D(factor)))
            f, step = D(1), D(theta) ** (D(-2) / D(dim))
            for i in range(dim // 2):
                w = D(1)
                if scaling == m.MLA_ROPE_SCALING_LINEAR:
                    w = D(0)
                elif scaling == m.MLA_ROPE_SCALING_PARTS:
                    w = min(D(1), max(D(0), (4096 * f / (2 * PI) - 1) / 3))
                g = w * f + (1 - w) * f / D(factor)
                off = (g / (2 * PI) - D(plan.turns[i]) / D(2) ** 64) % 1
                assert min(abs(off), 1 - abs(off)) < bound, (i, scaling)
                f *= step
