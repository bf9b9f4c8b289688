"""Orthogonalised updates of matrices whose norm is far below eps: X begins far
below 1 and its digits are those of any other."""
import pytest
import torch

import matrix_oracle as R
import mixed_precision_optimizer_mta_amd as M
from test_gpu_ortho import matrix, on_gpu
from test_gpu_ortho_steps import PER_STEP

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("part", [1e-3, 1e-6, 1e-12, 1e-30])
@pytest.mark.parametrize("rows,cols", [(40, 70), (130, 257), (257, 130),
                                       (130, 3001)])
def test_far_below_eps(rows, cols, part, precise):
    x = matrix(rows, cols, "f32", rows)
    eps = x.norm().item() / part
    y = M.orthogonalize(on_gpu(x), eps=eps, precise=precise)
    want = R.orthogonal(x, eps=eps)
    # Five steps of X in 22 bits, of diagonals and sums in float32, and the
    # result's own rounding; beside them, where X grows to a size at which A
    # counts, 2.5e-3 of the products of 11 bits or 1e-5 of those of 22, as
    # documented.
    most = 5 * (2.0 ** -22 + 4 * 2.0 ** -24) + 2.0 ** -24
    if part > 1e-5:
        most += 1e-5 if precise else 2.5e-3
    assert R.off(y, want) <= most


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("part", [2.0 ** -18, 1e-3, 0.3])
def test_ten_steps_from_below(part, precise):
    """Singular values that begin far below 1 and grow by up to 3.4445^10."""
    g = torch.Generator().manual_seed(5)
    x = torch.linalg.qr(torch.randn(300, 130, generator=g))[0].t().contiguous()
    eps = x.double().norm().item() * (1 / part - 1)
    y = M.orthogonalize(on_gpu(x), steps=10, eps=eps, precise=precise)
    want = R.orthogonal(x, steps=10, eps=eps)
    # All singular values are alike.  An error grows by the polynomial's slope,
    # up to 3.4445 for small ones as they do themselves, below 1.6 (its steepest
    # descent) for those near 1, which the six steps after 0.3 / sqrt(130) are:
    # 1.6^6 = 17 times ten steps' 2^-22 and sums of 2^-20 stay below 1e-4, and
    # 17 times the 5e-4 of products of 11 bits below 1e-2.
    most = 1e-4 if precise else 1e-2
    assert R.off(y, want) <= most


def test_per_step_and_weights():
    """Coefficients that differ by step, two steps at once, and the weights of
    an optimizer."""
    x = matrix(130, 3001, "f32", 9)
    eps = x.norm().item() * 1e9
    y = M.orthogonalize(on_gpu(x), steps=6, coefficients=PER_STEP, eps=eps,
                        precise=True)
    assert R.off(y, R.orthogonal(x, PER_STEP, eps=eps)) <= \
        6 * (2.0 ** -22 + 4 * 2.0 ** -24) + 2.0 ** -24
    for shape in ((130, 257), (257, 130)):
        p = torch.nn.Parameter(torch.zeros(*shape, device="cuda"))
        u = matrix(*shape, "f32", 1)
        p.grad = on_gpu(u).contiguous()
        opt = M.MtaOptimizer([p], kind="muon", lr=1.0, momentum=0.0,
                             nesterov=False, ns_eps=u.norm().item() * 1e9,
                             update_scale=1.0)
        opt.step()
        want = -R.orthogonal(u, eps=u.norm().item() * 1e9)
        assert R.off(p, want) <= 5 * (2.0 ** -22 + 4 * 2.0 ** -24) + \
            2.0 ** -23


def test_a_list_of_loud_and_faint():
    """Each as it is alone, to the bit."""
    xs = [on_gpu(matrix(r, c, "f32", i, size=s)) for i, (r, c, s) in enumerate(
        [(130, 257, 1.0), (130, 257, 1e-12), (257, 130, 1e-20), (40, 50, 1e-9),
         (300, 300, 1e-3), (100, 120, 0.0)])]
    for x, y in zip(xs, M.orthogonalize(xs)):
        assert y.isfinite().all()
        assert torch.equal(M.orthogonalize(x), y)


@pytest.mark.parametrize("eps", [0.0, 1e-160, 2.3e-308, 5e-324])
def test_zeros(eps):
    """However small eps is."""
    g = torch.ones(300, 200, device="cuda")
    for shape in ((20, 30), (1, 1), (130, 257), (257, 130)):
        z = torch.zeros(*shape, device="cuda")
        one, other = M.orthogonalize([z, g], eps=eps)
        assert torch.equal(one, z) and other.isfinite().all()
        faint = torch.zeros(*shape, device="cuda")
        faint[0, 0] = 1e-45            # the smallest there is
        y = M.orthogonalize(faint, eps=eps)
        want = R.orthogonal(torch.ones(1, 1), eps=0.0)
        assert abs(y[0, 0].item() - want.item()) <= 1e-5
        y[0, 0] = 0.0
        assert not y.any()
