"""The clipped policy loss on the GPU against its float64 definition, and the
run that ends in it: a loss-scaled training step of an output layer."""
import numpy as np
import pytest
import torch

import mixed_precision_optimizer_mta_amd as M
from mixed_precision_optimizer_mta_amd import _binding as B
import ops_oracle as R

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def case(rows, vocab, dtype, seed=0, pad=0, masked=0.2, kl=True):
    """Inputs with ratios on both sides of the clip and none within 1e-3 of
    its border."""
    g = gen(seed)
    z = torch.randn(rows, vocab + pad, generator=g) * 2
    a = torch.randint(vocab, (rows,), generator=g)
    z[torch.arange(rows), a] += 6 * torch.rand(rows, generator=g)
    z = z.to(R.DTYPES[dtype])
    logp = torch.log_softmax(z[:, :vocab].double(), 1).gather(
        1, a[:, None])[:, 0]
    ratio = torch.tensor([0.5, 0.797, 0.803, 0.95, 1.0, 1.1, 1.297, 1.303,
                          2.0]).double()[torch.randint(9, (rows,),
                                                       generator=g)]
    d = {"z": z.cuda()[:, :vocab], "a": a.cuda(),
         "old": (logp - ratio.log()).float().cuda(),
         "adv": torch.randn(rows, generator=g).cuda(),
         "w": ((torch.rand(rows, generator=g) >= masked) *
               (0.5 + torch.rand(rows, generator=g)) / rows).cuda(),
         "ref": (logp + 0.3 * torch.randn(rows, generator=g)).float().cuda()
         if kl else None}
    d["kw"] = dict(clip_low=0.2, clip_high=0.3, kl_coef=0.1 if kl else 0.0)
    return d


def call(fn, d, **more):
    return fn(d["z"], d["a"], d["old"], d["adv"], weights=d["w"],
              ref_logp=d["ref"], **d["kw"], **more)


def oracle(d):
    f = lambda t: None if t is None else R.to64(t)  # noqa: E731
    return R.policy(f(d["z"]), d["a"].cpu().numpy(), f(d["old"]), f(d["adv"]),
                    f(d["w"]), f(d["ref"]), d["kw"]["clip_low"],
                    d["kw"]["clip_high"], d["kw"]["kl_coef"])


# A row's sum of exponentials: each is off by a step of the hardware's 2^x and
# |z - max| log2(e) 2^-24 of its argument's rounding (weighted with itself:
# below 2^-22), the float32 additions by 2^-24 each: at most 64 of a lane (or
# vocab / 1024 of a streamed row, and as many rescalings), 6 across a wave.
def sum_error(vocab):
    n = 64 if vocab <= 65536 else 3 * vocab / 1024
    return (n + 16) * 2.0 ** -24


def check(d, r, scale=1.0):
    z = R.to64(d["z"])
    rows, vocab = z.shape
    w = R.to64(d["w"])
    stats, logp, grad = oracle(d)
    e = sum_error(vocab)
    got = R.to64(r.logp)
    assert (np.abs(got - logp) <= e + 2.0 ** -24 * np.abs(logp)).all()
    ratio = np.exp(logp - R.to64(d["old"]))
    adv = R.to64(d["adv"])
    k = np.abs(ratio * adv)
    b = d["kw"]["kl_coef"]
    if d["ref"] is not None:
        k = k + b * np.exp(R.to64(d["ref"]) - logp) + b
    # logp's error times the terms' slopes, and a float32 rounding of the sum
    slack = 2 * e * (np.abs(w) * (k + 1)).sum()
    assert (np.abs(R.to64(r.stats) - stats) <= slack + 2.0 ** -24 *
            np.abs(stats)).all()
    if r.dlogits is None:
        return
    dt = r.dlogits.dtype
    want = scale * grad
    top = z.max(1, keepdims=True)
    p = np.exp(z - top - np.log(np.exp(z - top).sum(1, keepdims=True)))
    # the coefficient c is off by logp's error times k, p by its exponent's
    # argument and the sum's error, and each product by a rounding
    c = scale * np.abs(w)[:, None] * k[:, None]
    perr = p * (e + 2.0 ** -20 + (top - z) * 2.0 ** -23)
    one = np.zeros_like(z)
    one[np.arange(rows), d["a"].cpu().numpy()] = 1.0
    bound = c * (2 * perr + (2 * e + 2.0 ** -20) * np.abs(one - p)) + \
        R.half_step(dt) * np.abs(want)
    # 1 - p of the action is expm1 of logp, off by logp's error
    bound = bound + one * c * 2 * e
    if dt == torch.float16:
        bound = bound + 2.0 ** -25
    err = np.abs(R.to64(r.dlogits) - want)
    assert (err <= bound).all()
    assert (R.to64(r.dlogits)[w == 0] == 0).all()


VOCABS = [1, 2, 7, 8, 9, 511, 513, 4096, 4097, 6000, 16384, 16385, 50257,
          65536, 65537, 70001, 131072]


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("vocab", VOCABS)
def test_loss_and_gradient(vocab, dtype):
    rows = 9 if vocab < 20000 else 5
    d = case(rows, vocab, dtype, vocab)
    r = call(M.policy_loss_grad, d, grad_scale=torch.full((1,), 512.0).cuda())
    check(d, r, 512.0)
    f = call(M.policy_loss_forward, d)
    check(d, f)
    assert torch.equal(f.stats, r.stats) and torch.equal(f.logp, r.logp)
    g = M.policy_loss_backward(d["z"], d["a"], f.saved,
                               grad_scale=torch.full((1,), 512.0).cuda())
    check(d, r._replace(dlogits=g), 512.0)
    again = call(M.policy_loss_grad, d,
                 grad_scale=torch.full((1,), 512.0).cuda())
    assert torch.equal(again.dlogits, r.dlogits)
    assert torch.equal(again.stats, r.stats)


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("rows,vocab,pad", [
    (1, 300, 0), (2, 300, 1), (3, 1000, 3), (4, 5000, 7), (2049, 40, 0),
    (9000, 17, 2), (2100, 5001, 0), (33, 20011, 5)])
def test_row_counts_and_padded_rows(rows, vocab, pad, dtype):
    d = case(rows, vocab, dtype, rows, pad, masked=0.5, kl=rows % 2 == 0)
    check(d, call(M.policy_loss_grad, d))


def test_every_row_masked_and_no_rows():
    d = case(6, 900, "bf16", masked=2.0)
    d["z"].fill_(float("nan"))
    r = call(M.policy_loss_grad, d)
    assert (r.stats == 0).all() and (r.logp == 0).all()
    assert (r.dlogits == 0).all()
    f = call(M.policy_loss_forward, d)
    assert (M.policy_loss_backward(d["z"], d["a"], f.saved) == 0).all()
    e = torch.zeros(0, 50).cuda()
    n = torch.zeros(0).cuda()
    r = M.policy_loss_grad(e, n.long(), n, n)
    assert (r.stats == 0).all() and r.dlogits.shape == (0, 50)
    f = M.policy_loss_forward(e, n.long(), n, n)
    assert M.policy_loss_backward(e, n.long(), f.saved).shape == (0, 50)


def test_masked_rows_hold_anything():
    d = case(8, 5000, "f32", 3, masked=0.0)
    want = call(M.policy_loss_grad, d)
    e = {k: v.clone() if isinstance(v, torch.Tensor) else v
         for k, v in d.items()}
    for k in (1, 6):
        d["w"][k] = e["w"][k] = 0.0
    clean = call(M.policy_loss_grad, d)
    for k, bad in ((1, float("nan")), (6, float("inf"))):
        e["z"][k] = bad
        e["old"][k] = bad
        e["adv"][k] = bad
        e["ref"][k] = bad
        e["a"][k] = 1 << 40
    got = call(M.policy_loss_grad, e)
    for a, b in zip(got[:2] + got[3:], clean[:2] + clean[3:]):
        assert torch.equal(a, b)
    assert torch.equal(got.dlogits[0], want.dlogits[0])


@pytest.mark.parametrize("vocab", [100, 9000, 50000, 70000])
@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_masked_vocabulary_entries(vocab, dtype):
    # -inf logits and the type's lowest value have probability 0
    d = case(4, vocab, dtype, 1, masked=0.0)
    a = d["a"].cpu()
    keep = d["z"][torch.arange(4), a].clone()
    d["z"][:, ::3] = -float("inf")
    d["z"][1, 1::2] = torch.finfo(d["z"].dtype).min
    d["z"][2, :] = -float("inf")           # the action alone is left
    d["z"][torch.arange(4), a] = keep
    z = d["z"].double().cpu()
    lp = torch.log_softmax(z, 1).gather(1, a[:, None])[:, 0]
    d["old"] = (lp - 0.05).float().cuda()
    d["ref"] = (lp + 0.1).float().cuda()
    r = call(M.policy_loss_grad, d)
    with np.errstate(invalid="ignore"):
        stats, logp, grad = oracle(d)
    assert np.isfinite(grad).all()
    assert (np.abs(R.to64(r.logp) - logp) <= sum_error(vocab) +
            2.0 ** -24 * np.abs(logp)).all()
    g = R.to64(r.dlogits)
    assert (g[grad == 0] == 0).all() and np.isfinite(g).all()
    # coefficients are below 1: roundings as in check()
    assert (np.abs(g - grad) <= 2 * R.half_step(r.dlogits.dtype) *
            np.abs(grad) + 4 * sum_error(vocab) + 2.0 ** -25).all()
    f = call(M.policy_loss_forward, d)
    b = M.policy_loss_backward(d["z"], d["a"], f.saved)
    assert (np.abs(R.to64(b) - grad) <= 2 * R.half_step(b.dtype) *
            np.abs(grad) + 4 * sum_error(vocab) + 2.0 ** -25).all()


@pytest.mark.parametrize("vocab", [60, 9000, 70000])
def test_not_finite_rows_stay_apart(vocab):
    d = case(6, vocab, "bf16", 2, masked=0.0)
    clean = call(M.policy_loss_grad, d)
    d["z"][1, 3] = float("nan")
    d["z"][2, 5] = float("inf")
    d["z"][3] = -float("inf")
    d["a"][4] = vocab
    d["a"][5] = -1
    r = call(M.policy_loss_grad, d)
    f = call(M.policy_loss_forward, d)
    b = M.policy_loss_backward(d["z"], d["a"], f.saved)
    for g in (r.dlogits, b):
        assert torch.isnan(g[1:]).any(1).all()
        assert torch.isfinite(g[0]).all()
    assert torch.equal(r.dlogits[0], clean.dlogits[0])
    assert torch.isnan(r.logp[1:]).all() and torch.isnan(r.stats[0])


def confident(vocab, dtype, gaps=(12.0, 16.0, 20.0, 25.0)):
    """One row for each gap by which the action's logit passes the others',
    which are normal and end in -25, no clipping, no KL term: (inputs, 1 - p,
    logp, ratio), in float64 from sums without the action's term."""
    rows = len(gaps)
    g = gen(vocab)
    z = torch.randn(rows, vocab, generator=g).clamp(-3, 3)
    a = torch.randint(vocab, (rows,), generator=g)
    a[0], a[-1] = 0, vocab - 1           # the ends of a row among them
    z[torch.arange(rows), a] = torch.tensor(gaps)
    z = z.to(R.DTYPES[dtype])
    z64 = R.to64(z)
    others = np.exp(z64 - z64.max(1, keepdims=True))
    others[np.arange(rows), a.numpy()] = 0.0
    rest = others.sum(1)
    logp = -np.log1p(rest)
    old = torch.from_numpy(logp).float()
    adv = torch.tensor([1.0, -2.0, 3.0, -0.5][:rows])
    d = {"z": z.cuda(), "a": a.cuda(), "old": old.cuda(), "adv": adv.cuda(),
         "w": torch.full((rows,), 1.0 / rows).cuda(), "ref": None,
         "kw": dict(clip_low=0.2, clip_high=0.2, kl_coef=0.0)}
    return d, rest / (1 + rest), logp, np.exp(logp - R.to64(old))


# Relative error of a sum of exponentials of arguments to -30: an argument's
# difference, its product with log2(e) and that constant are roundings of half
# a step each, 2.5 * 2^-24 * 30, and the sum and 2^x as in sum_error.
def rest_error(vocab):
    return sum_error(vocab) + 75 * 2.0 ** -24


CONFIDENT = [2, 40, 700, 4096, 9001, 50257, 65537, 131072]


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("vocab", CONFIDENT)
def test_confident_rows_keep_the_digits_of_the_rest(vocab, dtype):
    """Where p of the action nears 1, its gradient is -c (1 - p) and logp is
    ln p: both have as many digits as the sum of the other entries."""
    d, rest, logp, ratio = confident(vocab, dtype)
    e = rest_error(vocab)
    r = call(M.policy_loss_grad, d, grad_scale=torch.full((1,), 64.0).cuda())
    got = R.to64(r.logp)
    assert (np.abs(got - logp) <= (e + 2.0 ** -23) * np.abs(logp)).all()
    want = -64.0 / len(rest) * R.to64(d["adv"]) * ratio * rest
    g = R.to64(r.dlogits)[np.arange(len(rest)), d["a"].cpu().numpy()]
    # ratio is off by logp's error (below e), c and its product by roundings
    bound = (2 * e + 2.0 ** -21 + R.half_step(r.dlogits.dtype)) * np.abs(want)
    if dtype == "f16":
        bound = bound + 2.0 ** -25
    assert (np.abs(g - want) <= bound).all()


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("vocab", CONFIDENT)
def test_confident_rows_have_the_same_gradient_in_two_calls(vocab, dtype):
    d, rest, _, ratio = confident(vocab, dtype)
    scale = torch.full((1,), 64.0).cuda()
    f = call(M.policy_loss_forward, d)
    g = M.policy_loss_backward(d["z"], d["a"], f.saved, grad_scale=scale)
    at = np.arange(len(rest)), d["a"].cpu().numpy()
    want = -64.0 / len(rest) * R.to64(d["adv"]) * ratio * rest
    bound = (2 * rest_error(vocab) + 2.0 ** -21 +
             R.half_step(g.dtype)) * np.abs(want)
    if dtype == "f16":
        bound = bound + 2.0 ** -25
    assert (np.abs(R.to64(g)[at] - want) <= bound).all()
    z = d["z"].clone().requires_grad_()
    loss, _ = M.policy_loss(z, d["a"], d["old"], d["adv"], d["w"])
    (loss * 64.0).backward()
    assert torch.equal(z.grad, g)
    assert torch.equal(g, call(M.policy_loss_grad, d,
                               grad_scale=scale).dlogits)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_small_ratios_keep_their_digits(dtype):
    """A token of which the old policy was far surer: r = exp(logp - old) down
    to 1e-35, unclipped for a positive advantage, in the loss (one row a call)
    and in its gradient."""
    vocab = 300
    for k, gap in enumerate((5.0, 20.0, 25.0, 30.0, 40.0, 60.0, 80.0)):
        d = case(1, vocab, dtype, k, masked=0.0, kl=False)
        z = R.to64(d["z"])
        a = d["a"].item()
        top = z.max()
        logp = z[0, a] - top - np.log(np.exp(z - top).sum())
        d["old"] = torch.full((1,), logp + gap).cuda()
        d["w"], d["adv"] = torch.ones(1).cuda(), torch.full((1,), 1.5).cuda()
        ratio = np.exp(logp - R.to64(d["old"])[0])
        r = call(M.policy_loss_grad, d)
        e = 2 * sum_error(vocab) + 2.0 ** -20
        assert abs(r.stats[0].item() + 1.5 * ratio) <= e * 1.5 * ratio
        p = np.exp(z[0] - top) / np.exp(z[0] - top).sum()
        one = np.zeros(vocab)
        one[a] = 1.0
        want = -1.5 * ratio * (one - p)
        # 2^-126: below it a result has fewer digits than float32's 24
        assert (np.abs(R.to64(r.dlogits)[0] - want) <=
                (2 * e + R.half_step(d["z"].dtype)) * np.abs(want) +
                2.0 ** -133).all()
    for gap, r0 in ((740.0, 0.0), (800.0, 0.0), (float("inf"), 0.0)):
        d["old"] = torch.full((1,), logp + gap).cuda()
        r = call(M.policy_loss_grad, d)
        assert r.stats[0] == r0 and (r.dlogits == 0).all()


def test_large_logits_keep_their_differences():
    for dtype in ("f32", "bf16"):
        for base in (1e4, -1e6, 1e30):
            z = torch.full((1, 5000), base).to(R.DTYPES[dtype]).cuda()
            one = torch.zeros(1).cuda()
            r = M.policy_loss_grad(z, one.long(), one - float(np.log(5000)),
                                   one + 1)
            assert abs(r.logp.item() + np.log(5000)) <= sum_error(5000)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("base", [1e4, -1e6, 1e30, -1e38])
def test_large_logits_reach_the_backward(base, dtype):
    """Equal logits of any size: p is 1 / vocab for each, in both forms."""
    n = 5000
    z = torch.full((2, n), base).to(R.DTYPES[dtype]).cuda()
    z[1, 7] = -float("inf")
    a = torch.tensor([0, n - 1]).cuda()
    one = torch.ones(2).cuda()
    args = (z, a, -torch.tensor([n, n - 1.0]).log().cuda(), one)
    f = M.policy_loss_forward(*args)
    got = M.policy_loss_backward(z, a, f.saved)
    for g in (got, M.policy_loss_grad(*args).dlogits):
        g = R.to64(g)
        for t, m in ((0, n), (1, n - 1)):
            want = np.full(n, 0.5 / m)
            want[a[t].item()] = 0.5 / m - 0.5
            if t == 1:
                want[7] = 0.0
            # p is off by its sum's error, the ratio by logp's and old's
            # rounding (below 2^-21), each product by a rounding
            bound = np.abs(want) * (2 * sum_error(n) + 2.0 ** -19 +
                                    R.half_step(z.dtype))
            assert (np.abs(g[t] - want) <= bound).all()


def test_no_kl_term_ignores_the_reference():
    d = case(4, 300, "f32", 6, masked=0.0)
    d["kw"]["kl_coef"] = 0.0
    want = call(M.policy_loss_grad, {**d, "ref": None})
    d["ref"][1] = float("inf")
    got = call(M.policy_loss_grad, d)
    assert torch.equal(got.dlogits, want.dlogits)
    assert got.stats[0] == want.stats[0] and got.stats[1] == float("inf")


def test_default_weights_and_the_border():
    z = torch.zeros(4, 8).cuda()
    a = torch.arange(4).cuda()
    lp = float(-np.log(8))
    adv = torch.tensor([1.0, -1.0, 0.0, 2.0]).cuda()
    old = torch.full((4,), lp).cuda()
    r = M.policy_loss_grad(z, a, old, adv)
    assert abs(r.stats[0].item() + 0.5) <= 2.0 ** -20
    assert r.stats[1] == 0 and r.stats[2] == 0
    p = 1 / 8
    want = -(adv.cpu().double() / 4)[:, None] * (
        torch.eye(4, 8).double() - p)
    assert (r.dlogits.cpu().double() - want).abs().max() <= 2.0 ** -20
    # no clip at all: a ratio of exactly 1 is on both borders, and active
    r0 = M.policy_loss_grad(z, a, r.logp, adv, clip_low=0.0, clip_high=0.0)
    act = r0.stats[2].item()
    assert act in (0.0, 0.25, 0.5, 0.75)


@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_a_ratio_on_the_border_is_not_clipped(dtype):
    """vocab 1: logp is 0, so with old_logp 0 the ratio is exactly 1, which
    with no room to either side is both borders.  The slope is then that of
    the unclipped term, for either sign of the advantage."""
    z = torch.tensor([[3.0], [-2.0], [0.0], [1e4]]).to(R.DTYPES[dtype]).cuda()
    zero = torch.zeros(4).cuda()
    adv = torch.tensor([1.0, -1.0, 0.5, -2.0]).cuda()
    w = torch.tensor([1.0, 2.0, 4.0, 8.0]).cuda()
    r = M.policy_loss_forward(z, zero.long(), zero, adv, weights=w,
                              clip_low=0.0, clip_high=0.0)
    assert (r.logp == 0).all()
    assert r.stats.tolist() == [-(adv * w).sum().item(), 0.0, 0.0]
    coef = r.saved.view(4, 4)[:, 2]
    assert torch.equal(coef, -adv * w)
    # a step past the border on the side that the sign clips
    old = torch.tensor([-1.0, 1.0, -1.0, 1.0]).cuda() * 2.0 ** -20
    r = M.policy_loss_forward(z, zero.long(), old, adv, weights=w,
                              clip_low=0.0, clip_high=0.0)
    assert r.stats[2] == w.sum() and (r.saved.view(4, 4)[:, 2] == 0).all()
    # and on the other
    r = M.policy_loss_forward(z, zero.long(), -old, adv, weights=w,
                              clip_low=0.0, clip_high=0.0)
    assert r.stats[2] == 0 and (r.saved.view(4, 4)[:, 2] != 0).all()


def test_gradient_is_the_losses_difference():
    d = case(3, 40, "f32", 11, masked=0.0)
    g = R.to64(call(M.policy_loss_grad, d).dlogits)
    z = R.to64(d["z"])
    h = 1e-5
    f = lambda t: None if t is None else R.to64(t)  # noqa: E731

    def loss(zz):
        return R.policy(zz, d["a"].cpu().numpy(), f(d["old"]), f(d["adv"]),
                        f(d["w"]), f(d["ref"]), 0.2, 0.3, 0.1)[0][0]

    for t in range(3):
        for j in range(0, 40, 3):
            up, dn = z.copy(), z.copy()
            up[t, j] += h
            dn[t, j] -= h
            num = (loss(up) - loss(dn)) / (2 * h)
            # h^2 of the third derivative, 1e-16 / h of the difference, and
            # the float32 gradient's own error, of coefficients below 3
            assert abs(g[t, j] - num) <= 1e-9 + 3 * sum_error(40)


@pytest.mark.parametrize("vocab", [77, 9001, 50257, 66001])
def test_in_place(vocab):
    for dtype in R.DTYPES:
        d = case(5, vocab, dtype, 4, pad=1)
        want = call(M.policy_loss_grad, d).dlogits.clone()
        f = call(M.policy_loss_forward, d)
        keep = d["z"].clone()
        r = call(M.policy_loss_grad, d, out=d["z"])
        assert r.dlogits.data_ptr() == d["z"].data_ptr()
        assert torch.equal(d["z"], want)
        two = M.policy_loss_backward(keep, d["a"], f.saved)
        M.policy_loss_backward(keep, d["a"], f.saved, out=keep)
        assert torch.equal(keep, two)


def test_nothing_outside_the_gradient_is_written():
    d = case(7, 1003, "bf16", 6)
    wide = torch.full((9, 1010), 5.0, dtype=torch.bfloat16).cuda()
    out = wide[1:8, 3:1006]
    r = call(M.policy_loss_grad, d, out=out)
    assert torch.equal(out, call(M.policy_loss_grad, d).dlogits)
    assert r.dlogits is out
    for edge in (wide[0], wide[8], wide[:, :3], wide[:, 1006:]):
        assert (edge == 5).all()


def test_offsets_past_32_bits():
    rows, vocab = 86000, 50257           # 4.3e9 logits
    z = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    d = case(3, vocab, "bf16", 8, masked=0.0)
    at = torch.tensor([0, 43000, 85999]).cuda()
    z[at] = d["z"]
    full = lambda v: torch.zeros(rows, dtype=v.dtype,  # noqa: E731
                                 device="cuda").index_copy_(0, at, v)
    big = {"z": z, "kw": d["kw"]}
    for k in ("a", "old", "adv", "w", "ref"):
        big[k] = full(d[k])
    want = call(M.policy_loss_grad, d)
    r = call(M.policy_loss_grad, big, out=z)
    assert torch.equal(z[at], want.dlogits)
    assert torch.equal(r.logp[at], want.logp)
    assert (z[1000] == 0).all() and (z[85998] == 0).all()


def test_refusals_of_tensors():
    d = case(4, 100, "bf16")
    bad = [("a", d["a"].int()), ("a", d["a"][:3]), ("old", d["old"].double()),
           ("adv", d["adv"].cpu()), ("w", d["w"].half()),
           ("ref", torch.zeros(8).cuda()[::2]), ("z", d["z"].t())]
    for k, v in bad:
        with pytest.raises(ValueError):
            call(M.policy_loss_grad, {**d, k: v})
    with pytest.raises(TypeError):
        call(M.policy_loss_grad, {**d, "z": d["z"].double()})
    with pytest.raises(M.MtaError):
        call(M.policy_loss_grad, {**d, "ref": None})
    with pytest.raises(M.MtaError):
        call(M.policy_loss_grad, {**d, "kw": dict(clip_low=2.0)})
    with pytest.raises(ValueError):
        call(M.policy_loss_grad, d, out=torch.zeros(4, 100).cuda())
    with pytest.raises(ValueError):
        call(M.policy_loss_grad, d, grad_scale=torch.ones(2).cuda())
    f = call(M.policy_loss_forward, d)
    with pytest.raises(ValueError):
        M.policy_loss_backward(d["z"][:2], d["a"][:2], f.saved)


def test_values_of_another_order_of_rows_are_refused():
    d = case(15, 100, "bf16")
    want = call(M.policy_loss_grad, d)
    d["z"] = d["z"].reshape(3, 5, 100)
    for k in ("old", "adv", "w", "ref"):
        d[k] = d[k].reshape(3, 5)
    got = call(M.policy_loss_grad, {**d, "w": d["w"].reshape(15)})
    assert torch.equal(got.dlogits.reshape(15, 100), want.dlogits)
    f = call(M.policy_loss_forward, d)
    for k in ("a", "old", "adv", "w", "ref"):
        bad = {**d, k: d[k].reshape(5, 3)}
        for fn in (M.policy_loss_grad, M.policy_loss_forward):
            with pytest.raises(ValueError):
                call(fn, bad)
    with pytest.raises(ValueError):
        M.policy_loss_backward(d["z"], d["a"].reshape(5, 3), f.saved)


def test_captured_calls_replay_on_new_inputs():
    d = case(50, 5003, "bf16")
    scale = torch.full((1,), 4.0).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(M.policy_loss_grad, d, grad_scale=scale)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = call(M.policy_loss_grad, d, grad_scale=scale)
        f = call(M.policy_loss_forward, d)
        b = M.policy_loss_backward(d["z"], d["a"], f.saved, grad_scale=scale)
    for seed in range(4):
        e = case(50, 5003, "bf16", 30 + seed)
        for k in ("z", "a", "old", "adv", "w", "ref"):
            d[k].copy_(e[k])
        scale.fill_(2.0 ** seed)
        graph.replay()
        torch.cuda.synchronize()
        want = call(M.policy_loss_grad, e, grad_scale=scale)
        assert torch.equal(r.dlogits, want.dlogits)
        assert torch.equal(r.stats, want.stats)
        assert torch.equal(r.logp, want.logp)
        assert torch.equal(f.stats, want.stats)
        check(e, want._replace(dlogits=b), 2.0 ** seed)


def test_autograd():
    d = case(6, 700, "f16", 5)
    z = d["z"].clone().requires_grad_()
    loss, logp = M.policy_loss(z, d["a"], d["old"], d["adv"], d["w"],
                               d["ref"], 0.2, 0.3, 0.1)
    assert not logp.requires_grad
    loss *= 1024.0
    logp *= 1.0
    loss.backward()
    check(d, M.PolicyLoss(call(M.policy_loss_forward, d).stats, logp, None,
                          z.grad), 1024.0)


@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_autograd_takes_the_shifted_logits_of_a_batch(dtype):
    """logits[:, :-1] against tokens[:, 1:], and logits of [vocab, ...] order:
    the gradients of contiguous copies, in their places."""
    z = (torch.randn(3, 9, 300, generator=gen(1)) * 2).to(
        R.DTYPES[dtype]).cuda()
    tokens = torch.randint(300, (3, 9), generator=gen(2)).cuda()
    v = [torch.randn(3, 9, generator=gen(3 + k)).cuda() for k in range(3)]
    v[0] -= 6.0                            # (old log-probabilities)
    v[2] -= 6.0
    w = torch.rand(3, 9, generator=gen(9)).cuda()

    def loss(t, *args):
        out, logp = M.policy_loss(t, *args, 0.2, 0.3, 0.1)
        assert logp.shape == (3, 8)
        (out * 32.0).backward()
        return out.detach(), logp

    args = [t[:, 1:] for t in (tokens, v[0], v[1], w, v[2])]
    flat = [t.contiguous() for t in args]
    x = z[:, :-1].contiguous().requires_grad_()
    want = loss(x, *flat)
    y = z.clone().requires_grad_()
    got = loss(y[:, :-1], *args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(y.grad[:, :-1], x.grad) and (y.grad[:, -1] == 0).all()
    t = z[:, :-1].permute(2, 0, 1).contiguous().requires_grad_()
    got = loss(t.permute(1, 2, 0), *args)
    assert torch.equal(got[0], want[0])
    assert torch.equal(t.grad.permute(1, 2, 0), x.grad)


def test_a_graph_refuses_logits_overwritten_since():
    d = case(6, 700, "bf16", 6)
    z = d["z"].clone().requires_grad_()
    y = z * 1.0
    loss, _ = M.policy_loss(y, d["a"], d["old"], d["adv"])
    call(M.policy_loss_grad, {**d, "z": y.detach()}, out=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        loss.backward()
    with torch.inference_mode():
        t = d["z"].clone()
        r = call(M.policy_loss_grad, {**d, "z": t}, out=t)
    assert torch.equal(r.dlogits, call(M.policy_loss_grad, d).dlogits)


def test_a_loss_scaled_step_of_an_output_layer():
    """Hidden states kept in 8 bits, float16 logits and their gradient times
    the device's loss scale, the weight gradient from the checkpoint, one
    joint clip and one step: against the same step in float64."""
    rows, width, vocab = 96, 64, 1000
    h = (torch.randn(rows, width, generator=gen(1))).half().cuda()
    w = torch.nn.Parameter((torch.randn(vocab, width, generator=gen(2)) *
                            0.1).cuda())
    opt = M.MtaOptimizer([w], kind="sgd", lr=0.5, max_norm=1.0,
                         loss_scale=4096.0)
    w0 = R.to64(w)
    z = h.matmul(w.detach().half().t())
    a = torch.randint(vocab, (rows,), generator=gen(3)).cuda()
    f = M.policy_loss_forward(z, a, torch.zeros(rows).cuda(),
                              torch.zeros(rows).cuda())
    old = f.logp + 0.05 * torch.randn(rows, generator=gen(4)).cuda()
    adv = torch.randn(rows, generator=gen(5)).cuda()
    ck = M.ckpt_pack(h)
    r = M.policy_loss_grad(z, a, old, adv, ref_logp=f.logp, kl_coef=0.1,
                           grad_scale=opt.loss_scale, out=z.clone())
    w.grad = torch.zeros_like(w)
    M.ckpt_wgrad(ck, r.dlogits, bias=False, out=w.grad, accumulate=True)
    opt.step()
    stats, logp, dz = R.policy(R.to64(z), a.cpu().numpy(), R.to64(old),
                               R.to64(adv), np.full(rows, 1 / rows),
                               R.to64(f.logp), 0.2, 0.2, 0.1)
    kept = R.to64(ck.unpack())
    g = dz.T @ kept
    norm = np.sqrt((g * g).sum())
    coef = min(1.0, 1.0 / (norm + 1e-6))
    want = w0 - 0.5 * coef * g
    # dlogits is rounded to float16 (half a step 2^-11, and 2^-25 / 4096 below
    # its normal range); sums and the clip add a few float32 steps
    mass = (np.abs(dz) * 2.0 ** -10 + 2.0 ** -37).T @ np.abs(kept)
    err = np.abs(R.to64(w) - want)
    assert (err <= 0.5 * coef * mass * (1 + 1 / max(norm, 1e-3)) +
            2.0 ** -23 * np.abs(w0) + 2.0 ** -12 * np.abs(g) * coef).all()
    assert abs(opt.last_norm.item() - norm) <= 2.0 ** -10 * norm
    assert opt.amp.read()["step"] == 1
    # an overflowing logit is seen: the step is skipped, the scale backs off
    z[3, 5] = float("inf")
    r = M.policy_loss_grad(z, a, old, adv, grad_scale=opt.loss_scale)
    M.ckpt_wgrad(ck, r.dlogits, bias=False, out=w.grad)
    before = w.detach().clone()
    opt.step()
    assert torch.equal(w.detach(), before)
    assert opt.amp.read()["scale"] == 2048.0
