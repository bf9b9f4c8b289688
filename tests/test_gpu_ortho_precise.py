"""Orthogonalised updates of 22-bit products, tightly enough that products of 11
bits, or one of the three left out, would show; and lists that bring every size
of tile."""
import math

import pytest
import torch

import matrix_oracle as R
import mixed_precision_optimizer_mta_amd as M
from test_gpu_ortho import matrix, on_gpu
from test_gpu_ortho_steps import PER_STEP, by_two, one_by_one

pytestmark = pytest.mark.gpu


def most(rows, want):
    """Of a float32 result.  The first X, of norm 1, is rounded to 22 bits (a
    uniform error of up to 2^-23 of each element), and that error grows by no
    more than small singular values do; beside it the 8e-7 that later steps'
    roundings and float32 sums are documented to come to."""
    return 2.0 ** -23 / 3 ** 0.5 * math.prod(abs(r[0]) for r in rows) / \
        want.norm().item() + 8e-7


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6])
@pytest.mark.parametrize("rows,cols", [(130, 3001), (2500, 200), (257, 130)])
def test_steps(rows, cols, steps):
    """Small tiles, sums cut along k, two steps as one product."""
    x = matrix(rows, cols, "f32", steps)
    co = PER_STEP[:steps]
    want = R.orthogonal(x, co)
    limit = most(co, want)
    rough = min(R.off(f(x, 1, co), want) for f in (by_two, one_by_one))
    assert limit < rough / 5
    y = M.orthogonalize(on_gpu(x), steps=steps, coefficients=co, precise=True)
    assert R.off(y, want) <= limit


# What the host takes at 256 compute units: next and last are the products over
# all columns, times those of symmetric matrices.
LISTS = {
    # more than forty matrices: sums cut, times in 64 and next alone in 128 for
    # the last five; 128 by twos and 256 for the others
    "45 of 769x701": [(769, 701)] * 44 + [(701, 769)],
    "all 128 by twos": [(1601, 1603), (1603, 1601), (1601, 1601)],
    "128 alone, next by twos": [(2049, 2051)],
    "times 128, next 256": [(3001, 3003)],
    "all 256, two steps at once": [(1667, 1601)] * 4 + [(1601, 1667)] * 4,
    "times 256, next 128": [(515, 517)] * 20 + [(517, 515)] * 20,
    "many columns, next 256": [(2303, 769)] * 6 + [(769, 2303)] * 6,
}


@pytest.mark.parametrize("dtype,precise", [("f32", True), ("bf16", False)])
@pytest.mark.parametrize("name", list(LISTS))
def test_tiles(name, dtype, precise):
    xs = [matrix(r, c, dtype, i, pad=i % 2) for i, (r, c) in
          enumerate(LISTS[name])]
    xs = [on_gpu(x) for x in xs]
    ys = M.orthogonalize(xs, precise=precise, dtype=torch.float32)
    for x, y in zip(xs, ys):
        want = R.orthogonal(x)
        # (products of 11 bits: up to 1.1e-3, as documented, and 2e-4 at least)
        limit = most([R.COEF] * 5, want)
        assert R.off(y, want) <= (limit if precise else 1.1e-3)
        assert limit < 2e-4 / 5


@pytest.mark.parametrize("name", ["128 alone, next by twos",
                                  "all 256, two steps at once"])
def test_float16_results(name):
    xs = [on_gpu(matrix(r, c, "f16", i)) for i, (r, c) in
          enumerate(LISTS[name])]
    for x, y in zip(xs, M.orthogonalize(xs)):
        want = R.orthogonal(x)
        # (elements are about 1 / sqrt(rows): all but a few above 2^-14)
        assert R.off(y, want) <= most([R.COEF] * 5, want) + \
            R.half_step(torch.float16)
