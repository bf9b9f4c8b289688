"""Rows of the linear cross entropy whose logits or weights leave the range of
finite numbers: what becomes of them, and that the others do not notice."""
import pytest
import torch

import matrix_oracle as R
import mixed_precision_optimizer_mta_amd as M
from test_gpu_linear_loss import case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,vocab,h,w", [
    ("f32", 5, 1e30, -1e30), ("bf16", 5, 1e30, -1e30),
    ("bf16", 700, 1e30, -1e30),
    # 16-bit elements: logits of -infinity from a weight of it, and logits whose
    # multiple of log2(e) is none
    ("f16", 5, 1.0, -float("inf")), ("f16", 700, 1.0, -float("inf")),
    ("bf16", 5, 1.0, -3e38)])
def test_no_logit_that_is_a_number(dtype, vocab, h, w):
    """log softmax of nothing but -infinity is NaN, in loss, logp and
    gradients."""
    dt = R.DTYPES[dtype]
    hidden = torch.zeros(3, 8, dtype=dt, device="cuda")
    hidden[:, 0] = h
    weight = torch.zeros(vocab, 8, dtype=dt, device="cuda")
    weight[:, 0] = w
    t = torch.tensor([0, vocab - 1, -100], device="cuda")
    r = M.linear_cross_entropy_grad(hidden, weight, t)
    assert r.loss.isnan() and r.logp[:2].isnan().all() and r.logp[2] == 0
    assert r.dhidden[:2].isnan().all() and not r.dhidden[2].any()
    assert r.dweight.isnan().any()
    f = M.linear_cross_entropy_forward(hidden, weight, t)
    assert f.loss.isnan() and f.logp[:2].isnan().all()


@pytest.mark.parametrize("vocab", [50, 700])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_row_beside_it(dtype, vocab):
    """Only one row's logits are all -infinity: sixteen products of the lowest
    number with 1 or more."""
    d = case(30, vocab, 16, dtype, 1, masked=0.0)
    w = d["w"].abs() + 1
    want = M.linear_cross_entropy_grad(d["h"], w, d["t"])
    h = d["h"].clone()
    h[4] = torch.finfo(h.dtype).min
    r = M.linear_cross_entropy_grad(h, w, d["t"])
    rest = torch.arange(30) != 4
    assert r.logp[4].isnan() and r.loss.isnan()
    assert r.dhidden[4].isnan().all()
    assert torch.equal(r.logp[rest], want.logp[rest])
    assert torch.equal(r.dhidden[rest], want.dhidden[rest])


def test_logits_far_below_a_row_s_others():
    """A tile of the vocabulary whose logits are all beyond -2^127 / log2(e)
    adds nothing to a row whose other logits are ordinary."""
    for vocab in (257, 513, 700):
        h = torch.ones(4, 8, dtype=torch.bfloat16, device="cuda")
        w = torch.zeros(vocab, 8, dtype=torch.bfloat16, device="cuda")
        w[:5, 0] = torch.arange(5)
        w[128:, 0] = -3e38
        t = torch.tensor([0, 3, 4, 1], device="cuda")
        r = M.linear_cross_entropy_grad(h, w, t)
        z = torch.zeros(128, dtype=torch.float64)
        z[:5] = torch.arange(5)
        lp = torch.log_softmax(z, 0)[t.cpu()]
        # the sum of 128 exponentials, and the argument's and value's roundings
        assert torch.allclose(r.logp.cpu().double(), lp, rtol=0, atol=64 *
                              2.0 ** -24)
        assert r.dhidden.isfinite().all() and r.dweight.isfinite().all()


@pytest.mark.parametrize("rows", [30, 1500])
@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_an_infinite_weight(dtype, rows):
    """The row's own gradient is no number; the others' are what they are."""
    d = case(rows, 300, 64, dtype, 2)
    on = (d["t"] != -100).nonzero()[:, 0]
    wt = torch.rand(rows, generator=torch.Generator().manual_seed(1)).cuda()
    wt[on[0]] = 0.75                       # the largest stays the largest
    wt.clamp_max_(0.75)
    want = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"], weights=wt)
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    for bad in (float("inf"), -float("inf"), float("nan")):
        w2 = wt.clone()
        w2[on[3]] = bad
        rest[on[3]] = False
        r = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"], weights=w2)
        assert not r.dhidden[on[3]].isfinite().any()
        assert not r.dweight.isfinite().any()
        assert torch.equal(r.logp, want.logp)
        assert torch.equal(r.dhidden[rest], want.dhidden[rest])
        f = M.linear_cross_entropy_forward(d["h"], d["w"], d["t"], weights=w2)
        dh, _ = M.linear_cross_entropy_backward(d["h"], d["w"], d["t"],
                                                f.saved, need_weight=False)
        assert torch.equal(dh[rest], want.dhidden[rest])
    # no finite weight at all: no NaN where the product with it has none
    w2 = torch.full_like(wt, float("inf"))
    r = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"], weights=w2)
    assert r.loss == float("inf")
    assert not r.dhidden[on].isfinite().any()
    assert not r.dhidden[d["t"] == -100].any()


@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_small_weights_under_a_large_scale(dtype):
    """Weights that are no normal numbers times 2^-14, and a factor that makes
    up for them: dw as of ordinary ones, to the bit but for the weights' own
    digits (2^-126 times 0.7 keeps 23 of 24, a rounding of 2^-24 of each)."""
    d = case(90, 300, 64, dtype, 3)
    wt = 0.5 + torch.rand(90, generator=torch.Generator().manual_seed(2))
    wt = wt.cuda()
    to = torch.empty(300, 64, device="cuda")

    def dw(weights, scale):
        return M.linear_cross_entropy_grad(
            d["h"], d["w"], d["t"], weights=weights, grad_scale=torch.tensor(
                [scale], device="cuda"), out_weight=to).dweight.double()

    want = dw(wt, 1.0)
    got = dw(wt * 2.0 ** -126, 2.0 ** 126)
    # dz's own rounding may turn out the other way: half a step of either
    assert (got - want).norm() <= 4 * (R.half_step(R.DTYPES[dtype]) +
                                       2.0 ** -23) * want.norm()
    for tiny, large in ((2.0 ** -120, 2.0 ** 120), (2.0 ** 100, 2.0 ** -100)):
        assert torch.equal(dw(wt * tiny, large), want)
