"""The plain form of the distillation loss where a share is far below what fp32 holds: its gradient against differences,
and against the values that the formulas give by hand."""

import numpy as np
import pytest

import distill_ref as R


@pytest.mark.parametrize("part", range(4))
@pytest.mark.parametrize("gap", [95.0, 150.0, 600.0])
@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
def test_gradient_against_differences(kind, gap, part):
    rng = np.random.default_rng(1)
    V, k = 8, 3
    x, ids, values, tail = rng.normal(size=(1, V)), np.array([[1, 4, 6]]), rng.normal(size=(1, k)), rng.normal(size=1)
    others = [v for v in range(V) if v not in ids[0]]
    if part == 0:
        x[0, 4] -= gap
    elif part == 1:
        x[0, others] -= gap
    elif part == 2:
        values[0, 0] -= gap
    else:
        tail -= gap
    args = dict(ids=ids, values=values, tail=tail, kind=kind, mix=0.3)
    g, h = R.distill(x, **args)["grad"][0], 1e-4
    for v in range(V):
        d = np.zeros_like(x)
        d[0, v] = h
        num = (R.distill(x + d, **args)["kd"][0] - R.distill(x - d, **args)["kd"][0]) / (2 * h)
        # third derivatives stay below the divergence (gap at most); its 2^-52 over the step
        assert abs(num - g[v]) <= gap * h * h + gap * 2.0 ** -51 / h


def test_values_by_hand():
    """Two listed entries and no rest: p = (1/2, 1/2), the student's second one 150 below."""
    x, ids = np.array([[0.0, -150.0, -np.inf]]), np.array([[0, 1]])
    got = R.distill(x, ids, np.zeros((1, 2)), np.array([-np.inf]))
    assert abs(got["kd"][0] - (75.0 - np.log(2.0))) < 1e-12 and np.allclose(got["grad"][0], [0.5, -0.5, 0.0], atol=1e-15)
    # the rest's gradient is the teacher's rest shared by the student's entries, whatever the gap
    x = np.array([[0.0, -300.0, -300.0 + np.log(3.0)]])
    got = R.distill(x, np.array([[0]]), np.zeros((1, 1)), np.zeros(1))
    assert np.allclose(got["grad"][0], [0.5, -0.125, -0.375], atol=1e-15)
