"""Scores over Q4 rows whose queries have a large common part, or one large dimension, that the keys take out again: the
same however many tokens a call has, and so whichever kernel computes them.

Tolerances.  A query's value is held as two binary16 halves, 2^-23 of itself off at most; the errors of a row's products are
independent, so that a score is off by scale |k| 2^-23 / sqrt(3) times the query's size (its common part and three standard
deviations), root mean square, and sums of the products in fp32, the plain form's among them, by about as much.  Scores
here are of usual size and softmax weights nearly even, so that outputs are as far off relative to their norm as the
weights relative to themselves.  Twice this without the root of three, and 2e-6 for all that does not grow with the query
(the usual 4e-6 is for a single output)."""
import pytest
import torch

import test_gpu_q4 as q4
from test_gpu_q4 import m  # noqa: F401

pytestmark = pytest.mark.gpu


def even_keys(rows, w, seed):
    """Codes u and 16 - u of 1 .. 15, side by side: a block's values add up to zero."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.randint(1, 16, (rows.shape[0], w // 2), generator=g, device="cuda", dtype=torch.uint8)
    rows[:, :w // 2] = u | ((16 - u) << 4)


@pytest.mark.parametrize("common", [0, 1, 10, -10, 100, 1000])
@pytest.mark.parametrize("new", [1, 2, 3, 5, 8, 40])
@pytest.mark.parametrize("geom", [(16, 8, 128, 128), (14, 2, 64, 64), (8, 1, 64, 64), (3, 3, 128, 128)])
def test_queries_with_a_common_part(m, geom, new, common):
    b = q4.Batch(geom, [new] * 4, [1500] * 4, True, block=64, seed=1)
    even_keys(b.k, b.w, 3)
    b.q += common
    got, err = b.run(m)
    assert err == 0
    ref = b.ref()
    size = float(q4.value(b.k[:64], b.w).square().mean().sqrt()) * geom[3] ** 0.5
    tol = 2 * b.scale * size * 2.0 ** -23 * (abs(common) + 3) + 2e-6
    assert float((got.double() - ref).norm() / ref.norm()) <= tol


@pytest.mark.parametrize("times", [10, 100])
@pytest.mark.parametrize("new", [1, 3, 8, 40])
@pytest.mark.parametrize("geom", [(16, 8, 128, 128), (14, 2, 64, 64)])
def test_queries_with_one_large_dimension(m, geom, new, times):
    """What is below 2^-20 of a block's largest product is cut off where few rows are computed: a block of 32 products in
    its four steps, up to 15 times the largest of the query times the scale, by twice 2^-20 of that at most."""
    b = q4.Batch(geom, [new] * 4, [1500] * 4, True, block=64, seed=2)
    b.q.view(-1, geom[2])[:, 5] *= times
    b.scale /= times / 10
    got, err = b.run(m)
    assert err == 0
    ref = b.ref()
    d = float(q4.value(b.k[:64], b.w).abs().max()) / 8
    cut = 2 * 4 * 2.0 ** -20 * 15 * float(b.q.abs().max()) * d * b.scale
    # a score off by `cut` changes a weight by as much of itself, an output by that times its distance from the values
    assert float((got.double() - ref).abs().max()) <= cut * float(q4.value(b.v[:64], b.w).abs().max()) + q4.ATOL
