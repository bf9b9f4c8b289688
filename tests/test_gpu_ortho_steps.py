"""Orthogonalised updates whose steps are taken two at a time, whose sums are cut
along k or whose products take the smallest tiles, against the float64
definition."""
import pytest
import torch

import matrix_oracle as R
import mixed_precision_optimizer_mta_amd as M
from test_gpu_ortho import matrix, on_gpu

pytestmark = pytest.mark.gpu

# one for each step: no two alike, and no singular value above 2
PER_STEP = [(3.4445, -4.7750, 2.0315), (3.2, -4.0, 1.7), (2.9, -3.6, 1.6),
            (3.0, -3.8, 1.7), (2.2, -2.0, 0.8), (1.875, -1.25, 0.375)]


def times(p, q, e0, e1, e2, planes):
    """e0 P Q + e1 P + e2 of two symmetric matrices with their diagonals apart;
    what is off the result's is kept in float16 values."""
    d, e = torch.diag(p.diagonal()), torch.diag(q.diagonal())
    o, n = p - d, q - e
    y = e0 * (o @ n + d @ n + o @ e + d @ e) + e1 * p + e2 * torch.eye(
        p.shape[0], dtype=torch.float64)
    diag = torch.diag(y.diagonal())
    return R._kept(y - diag, 512, planes) + diag


def by_two(x, planes, rows):
    """The documented roundings where two steps are one product."""
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + R.EPS)
    blocks = [rows[k:k + 2] for k in range(0, len(rows), 2)]
    for n, block in enumerate(blocks):
        whole, part = R._kept(x, 8192, 2), R._kept(x, 8192, planes)
        s = part @ part.t()
        diag = torch.diag(s.diagonal())
        s = R._kept(s - diag, 512, planes) + diag
        a, b, c = block[0]
        y, rest = times(s, s, c, b, a, planes), a
        if len(block) > 1:
            a, b, c = block[1]
            t = times(s, y, 1, 0, 0, planes)
            s = times(t, y, 1, 0, 0, planes)
            t = times(s, s, c, b, a, planes)
            y, rest = times(t, y, 1, 0, 0, planes), rest * a
        diag = y.diagonal()[:, None]
        left = whole - R._kept(x, 8192, 1)
        late = planes == 2 or n + 2 >= len(blocks)
        x = diag * (whole - left) + (diag if late else rest) * left + \
            (y - torch.diag(y.diagonal())) @ part
    return x.t() if tall else x


def one_by_one(x, planes, rows):
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + R.EPS)
    for k, (a, b, c) in enumerate(rows):
        whole, part = R._kept(x, 8192, 2), R._kept(x, 8192, planes)
        s = part @ part.t()
        diag = torch.diag(s.diagonal())
        s = R._kept(s - diag, 512, planes) + diag
        y = times(s, s, c, b, a, planes)
        diag = y.diagonal()[:, None]
        left = whole - R._kept(x, 8192, 1)
        late = planes == 2 or k + 2 >= len(rows)
        x = diag * (whole - left) + (diag if late else a) * left + \
            (y - torch.diag(y.diagonal())) @ part
    return x.t() if tall else x


def check(x, y, rows, precise, grows=30):
    """Which way is taken depends on what is quicker: the rougher of the two, a
    quarter more for what the order of additions brings about, and the float32
    sums of an addition for every sixteen values of k, half a step each, of
    either sign, times what an error grows by."""
    want = R.orthogonal(x, rows)
    planes = 2 if precise else 1
    rough = max(R.off(f(x, planes, rows), want) for f in (by_two, one_by_one))
    k = 3 * (max(x.shape) // 16 + 3)
    sums = (3 * len(rows) * k) ** 0.5 * 2.0 ** -24 * grows
    assert R.off(y, want) <= 1.25 * rough + R.half_step(y.dtype) + sums


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6])
@pytest.mark.parametrize("rows,cols", [(130, 3001), (2500, 200)])
def test_steps(rows, cols, steps, precise):
    """Few rows and many columns: two steps are one product there."""
    x = matrix(rows, cols, "f32", steps)
    co = PER_STEP[:steps]
    y = M.orthogonalize(on_gpu(x), steps=steps, coefficients=co,
                        precise=precise)
    check(x, y, co, precise)


@pytest.mark.parametrize("precise", [False, True])
def test_a_list_of_different_lengths(precise):
    """Sums cut along k where a part of the shorter ones is empty."""
    shapes = [(70, 5000), (90, 100), (200, 65), (66, 66), (100, 1)]
    xs = [matrix(r, c, "f32", i) for i, (r, c) in enumerate(shapes)]
    ys = M.orthogonalize([on_gpu(x) for x in xs], coefficients=PER_STEP[:5],
                         precise=precise)
    for x, y in zip(xs, ys):
        check(x, y, PER_STEP[:5], precise)


@pytest.mark.parametrize("precise", [False, True])
def test_two_steps_that_grow_too_much_for_one_product(precise):
    """5 T5(x) and 6 T5(x / 5), T5 = 16 x^5 - 20 x^3 + 5 x: slopes 25 and 6, and
    150 for both."""
    co = [(25.0, -100.0, 80.0), (6.0, -0.96, 1.2 * 16 / 625)]
    x = matrix(130, 3000, "f32", 3)
    y = M.orthogonalize(on_gpu(x), steps=2, coefficients=co, precise=precise)
    want = R.orthogonal(x, co)
    rough = R.off(one_by_one(x, 2 if precise else 1, co), want)
    assert y.isfinite().all()
    # (slopes of the polynomials themselves: up to 25 in each step)
    assert R.off(y, want) <= 1.25 * rough + 2.0 ** -24 + \
        3 * (3 * 190) ** 0.5 * 2.0 ** -24 * 25 * 25


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("rows,cols,rank", [(16, 64, 3), (64, 700, 5),
                                            (33, 2000, 1), (130, 3000, 20),
                                            (300, 256, 40)])
def test_most_steps_of_matrices_without_full_rank(rows, cols, rank, precise):
    """Ten steps raise what rounding leaves of the other directions to any size,
    but singular values stay where the polynomial has them, below 1.21.  Those
    of up to 64 rows are right beyond that: 2^-52 of the Gram matrix comes to
    2^-16, beside 1, of what multiplies directions of up to 2^-26 + 18."""
    g = torch.Generator().manual_seed(rank)
    x = torch.randn(rows, rank, generator=g) @ torch.randn(rank, cols,
                                                           generator=g)
    y = M.orthogonalize(x.cuda(), steps=10, precise=precise)
    assert y.isfinite().all()
    assert torch.linalg.matrix_norm(y.double().cpu(), 2) <= 1.25
    if rows <= 64:
        assert R.off(y, R.orthogonal(x, steps=10)) <= 2.0 ** -22 + 2.0 ** -24


def test_replays():
    """Captured steps by twos and in parts, replayed on new values with eager
    work between."""
    xs = [on_gpu(matrix(r, c, "bf16", i))
          for i, (r, c) in enumerate([(130, 3000), (70, 900), (30, 40)])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        M.orthogonalize(xs)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ys = M.orthogonalize(xs)
    for k in range(3):
        for x in xs:
            x.copy_(torch.randn(x.shape, generator=torch.Generator()
                                .manual_seed(k)))
        graph.replay()
        torch.cuda.synchronize()
        got = [y.clone() for y in ys]
        for g, want in zip(got, M.orthogonalize(xs)):
            assert torch.equal(g, want)
