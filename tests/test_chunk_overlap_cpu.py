"""Outputs of the chunk operators that stand on inputs, on the workspace or on each other:
refused, as the kernels read while others of their blocks write."""
import pytest

from test_chunk_cpu import A, _attend, _code, _problem, _weigh, m  # noqa: F401

# 10 tokens of 20 heads, 4 requests, 100 pages of 64 rows; addresses as in test_chunk_cpu
ROWS = 10 * 20


def _attend_overlaps(ws):
    return [dict(o=A[0]), dict(o=A[0] + ROWS * 1152 - 32), dict(lse=A[0] + 64), dict(o=A[2] + 100 * 64 * 1152 - 32),
            dict(lse=A[1]), dict(lse=A[1] + 16), dict(o=A[3]), dict(lse=A[4] + 12), dict(o=A[5]), dict(lse=A[5] + ws - 4),
            dict(lse=A[6]), dict(lse=A[6] + ROWS * 1024 - 4), dict(o=A[7]), dict(status=A[6] + 8), dict(status=A[7]),
            dict(status=A[4]), dict(status=A[5]), dict(ws=A[0]), dict(ws=A[2] + 1024), dict(ws=A[4]), dict(ws=A[3])]


def _weigh_overlaps(ws):
    return [dict(out=A[0]), dict(out=A[0] + ROWS * 1152 - 4), dict(out=A[7]), dict(out=A[7] + ROWS * 4 - 4), dict(out=A[1] + 16),
            dict(out=A[2] + 8), dict(out=A[3]), dict(out=A[4] + 12), dict(out=A[5] + ws - 4), dict(status=A[6]),
            dict(status=A[6] + 4 * 399), dict(status=A[8]), dict(status=A[7]), dict(ws=A[0]), dict(ws=A[7]), dict(ws=A[8]),
            dict(ws=A[2] + 1024)]


@pytest.mark.parametrize("call,overlaps", [(_attend, _attend_overlaps), (_weigh, _weigh_overlaps)])
def test_outputs_stand_alone(m, call, overlaps):  # noqa: F811
    plan = m.mla_chunk_make_plan(_problem(m), 10)
    for bad in overlaps(int(plan.workspace_bytes)):
        assert _code(m, call, m, plan=plan, **bad) == m.MLA_ERR_INVALID_ARGUMENT, bad
