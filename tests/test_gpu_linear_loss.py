"""The cross entropy of a linear output layer on the GPU against its float64
definition."""
import pytest
import torch

import matrix_oracle as R
import mixed_precision_optimizer_mta_amd as M

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def case(rows, vocab, width, dtype, seed=0, pad=(0, 0), masked=0.2):
    """Hidden states that raise their target's logit by 0 to 10."""
    g = gen(seed)
    dt = R.DTYPES[dtype]
    w = torch.randn(vocab, width + pad[1], generator=g) * 0.3
    t = torch.randint(vocab, (rows,), generator=g)
    h = torch.randn(rows, width + pad[0], generator=g)
    at = w[t, :width]
    h[:, :width] += at * (10 * torch.rand(rows, 1, generator=g) /
                          at.square().sum(1, keepdim=True).clamp_min(0.1))
    off = torch.rand(rows, generator=g) < masked
    off[:1] = False
    return {"h": h.to(dt).cuda()[:, :width], "w": w.to(dt).cuda()[:, :width],
            "t": torch.where(off, -100, t).cuda()}


def near(y, want, most):
    bad = (y.double() - want).abs() > most
    assert y.shape == want.shape and not bad.any(), (
        int(bad.sum()), float(((y.double() - want).abs() / most).max()))


def check(d, r, scale=1.0, weights=None):
    e = R.linear_loss(d["h"], d["w"], d["t"], weights, scale=scale)
    near(r.loss, e["loss"], e["loss_off"])
    near(r.logp, e["logp"], e["logp_off"])
    if r.dhidden is not None:
        near(r.dhidden, e["dh"], e["dh_off"])
    if r.dweight is not None:
        near(r.dweight, e["dw"], e["dw_off"] + e["dw"].abs() *
             R.half_step(r.dweight.dtype) +
             (2.0 ** -25 if r.dweight.dtype == torch.float16 else 0.0))
    return e


SIZES = [(1, 1, 1), (1, 2, 8), (2, 63, 64), (63, 257, 100), (64, 64, 63),
         (65, 1000, 257), (300, 129, 128), (5, 5003, 65), (129, 300, 1),
         (1000, 2, 64)]


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("rows,vocab,width", SIZES)
def test_loss_and_gradients(rows, vocab, width, dtype):
    d = case(rows, vocab, width, dtype, rows + vocab)
    r = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"])
    check(d, r)
    f = M.linear_cross_entropy_forward(d["h"], d["w"], d["t"])
    assert torch.equal(f.loss, r.loss) and torch.equal(f.logp, r.logp)
    dh, dw = M.linear_cross_entropy_backward(d["h"], d["w"], d["t"], f.saved)
    assert torch.equal(dh, r.dhidden) and torch.equal(dw, r.dweight)
    assert not r.dhidden[d["t"] == -100].any()


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("pad", [(3, 0), (0, 5), (1, 1), (64, 64), (8, 24)])
def test_strides_and_alignment(pad, dtype):
    d = case(70, 333, 128, dtype, 3, pad)
    check(d, M.linear_cross_entropy_grad(d["h"], d["w"], d["t"]))
    # off 16 bytes, too
    h = torch.empty(70 * 128 + 1, dtype=d["h"].dtype, device="cuda")[1:]
    w = torch.empty(333 * 128 + 1, dtype=d["h"].dtype, device="cuda")[1:]
    e = {"h": h.view(70, 128).copy_(d["h"]),
         "w": w.view(333, 128).copy_(d["w"]), "t": d["t"]}
    a = M.linear_cross_entropy_grad(e["h"], e["w"], e["t"])
    b = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"])
    assert all(torch.equal(getattr(a, k), getattr(b, k))
               for k in ("loss", "logp", "dhidden", "dweight"))


@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_pieces_of_the_vocabulary(dtype):
    """More of dz than is kept at a time, and sums over parts."""
    rows = 4000 if dtype != "f32" else 1400
    d = case(rows, 70001, 64, dtype, 7)
    check(d, M.linear_cross_entropy_grad(d["h"], d["w"], d["t"]))


def test_large_tiles():
    d = case(5000, 9000, 512, "bf16", 8)
    check(d, M.linear_cross_entropy_grad(d["h"], d["w"], d["t"]))


@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_weights_and_scale(dtype):
    d = case(90, 400, 72, dtype, 4)
    g = gen(5)
    wt = torch.rand(90, generator=g) * 3 - 0.5
    wt[::7] = 0.0
    wt[3] = 1e-6
    wt = wt.cuda()
    scale = torch.tensor([4096.0], device="cuda")
    check(d, M.linear_cross_entropy_grad(d["h"], d["w"], d["t"], weights=wt,
                                         grad_scale=scale), 4096.0, wt)


@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_rows_that_are_left_out_are_not_read(dtype):
    d = case(100, 300, 64, dtype, 6)
    want = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"])
    off = d["t"] == -100
    h = d["h"].clone()
    h[off] = float("nan")
    h[off.nonzero()[0, 0]] = float("inf")
    for t, wt, ig in ((d["t"], None, -100),
                      (torch.where(off, 10 ** 12, d["t"]), None, 10 ** 12),
                      (torch.where(off, -5, d["t"]),
                       (~off).float() / (~off).sum(), -100)):
        r = M.linear_cross_entropy_grad(h, d["w"], t, weights=wt,
                                        ignore_index=ig)
        assert torch.equal(r.logp, want.logp)
        assert torch.equal(r.dhidden, want.dhidden)
        assert torch.equal(r.dweight, want.dweight)
        assert torch.equal(r.loss, want.loss)


def test_nothing_left():
    d = case(30, 50, 16, "bf16")
    t = torch.full_like(d["t"], -100)
    r = M.linear_cross_entropy_grad(d["h"], d["w"], t)
    assert r.loss == 0 and not r.logp.any()
    assert not r.dhidden.any() and not r.dweight.any()
    r = M.linear_cross_entropy_grad(d["h"][:0], d["w"], t[:0])
    assert r.loss == 0 and r.dhidden.shape == (0, 16)
    assert not r.dweight.any()
    w = torch.ones(50, 16, device="cuda")
    M.linear_cross_entropy_grad(d["h"][:0], d["w"], t[:0], out_weight=w,
                                accumulate=True)
    assert (w == 1).all()


@pytest.mark.parametrize("bad", [-1, 50, 2 ** 40, -2 ** 40])
def test_a_target_out_of_range(bad):
    d = case(30, 50, 16, "f32", masked=0.0)
    want = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"])
    t = d["t"].clone()
    t[7] = bad
    r = M.linear_cross_entropy_grad(d["h"], d["w"], t)
    rest = torch.arange(30) != 7
    assert r.loss.isnan() and r.logp[7].isnan() and r.dhidden[7].isnan().all()
    assert r.dweight.isnan().all()
    assert torch.equal(r.logp[rest], want.logp[rest])
    assert torch.equal(r.dhidden[rest], want.dhidden[rest])


def test_what_is_not_finite():
    d = case(30, 50, 16, "bf16", masked=0.0)
    h = d["h"].clone()
    h[4, 2] = float("nan")
    r = M.linear_cross_entropy_grad(h, d["w"], d["t"])
    assert r.logp[4].isnan() and r.loss.isnan()
    rest = torch.arange(30) != 4
    assert r.dhidden[4].isnan().all() and r.dhidden[rest].isfinite().all()
    # a row's largest possible gap: probability 1 and 0, no NaN
    big = torch.zeros(2, 16, dtype=torch.float32, device="cuda")
    w = torch.zeros(5, 16, device="cuda")
    big[:, 0] = 1e30
    w[1, 0], w[2, 0] = 1e8, -1e8
    t = torch.tensor([1, 2], device="cuda")
    r = M.linear_cross_entropy_grad(big, w, t)
    assert r.logp[0] == 0 and r.logp[1].item() == pytest.approx(-2e38)
    assert r.dweight.isfinite().all()


def test_probability_near_one_keeps_its_digits():
    h = torch.zeros(1, 8, device="cuda")
    h[0, 0] = 1.0
    w = torch.zeros(3, 8, device="cuda")
    w[1, 0] = 30.0
    r = M.linear_cross_entropy_grad(h, w, torch.tensor([1], device="cuda"))
    e = 2 * torch.tensor(-30.0, dtype=torch.float64).exp()
    rest = e / (1 + e)
    assert r.logp.item() == pytest.approx(-torch.log1p(e).item(), rel=1e-6)
    assert r.dweight[1, 0].item() == pytest.approx(-rest.item(), rel=1e-6)


@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_given_outputs(dtype):
    d = case(65, 200, 50, dtype, 9)
    dt = R.DTYPES[dtype]
    want = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"])
    wide = torch.full((67, 61), 7.0, dtype=dt, device="cuda")
    old = torch.randn(200, 53, generator=gen(1)).cuda()
    acc = old.clone()
    r = M.linear_cross_entropy_grad(
        d["h"], d["w"], d["t"], out=wide[1:66, 3:53],
        out_weight=acc[:, 2:52], accumulate=True)
    assert r.dhidden.data_ptr() == wide[1, 3:].data_ptr()
    assert torch.equal(wide[1:66, 3:53], want.dhidden)
    wide[1:66, 3:53] = 7.0
    assert (wide == 7.0).all()
    full = M.linear_cross_entropy_grad(
        d["h"], d["w"], d["t"], out_weight=torch.empty(200, 50,
                                                       device="cuda")).dweight
    assert torch.equal(full.to(dt), want.dweight)
    assert torch.equal(acc[:, 2:52], old[:, 2:52] + full)
    assert torch.equal(acc[:, :2], old[:, :2]) and torch.equal(
        acc[:, 52:], old[:, 52:])
    f = M.linear_cross_entropy_forward(d["h"], d["w"], d["t"])
    dh, none = M.linear_cross_entropy_backward(d["h"], d["w"], d["t"], f.saved,
                                               need_weight=False)
    assert none is None and torch.equal(dh, want.dhidden)
    none, dw = M.linear_cross_entropy_backward(d["h"], d["w"], d["t"], f.saved,
                                               need_hidden=False)
    assert none is None and torch.equal(dw, want.dweight)


@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_autograd(dtype):
    d = case(24, 150, 40, dtype, 2)
    h = d["h"].view(2, 12, 40).clone().requires_grad_()
    w = d["w"].clone().requires_grad_()
    t = d["t"].view(2, 12)
    loss, logp = M.linear_cross_entropy(h, w, t)
    assert logp.shape == (2, 12) and not logp.requires_grad
    (loss * 64.0).backward()
    r = M.LinearLoss(loss.detach(), logp.view(-1), None, h.grad.view(24, 40),
                     w.grad)
    check(d, r, 64.0)
    # any strides: a transposed weight, the shifted rows of a batch
    h2 = d["h"].view(2, 12, 40).clone().requires_grad_()
    w2 = d["w"].t().contiguous().requires_grad_()
    a, _ = M.linear_cross_entropy(h2[:, :-1], w2.t(), t[:, 1:])
    b, _ = M.linear_cross_entropy(h2[:, :-1].contiguous(),
                                  w2.t().contiguous(), t[:, 1:].contiguous())
    ga = torch.autograd.grad(a, (h2, w2))
    gb = torch.autograd.grad(b, (h2, w2))
    assert torch.equal(a, b)
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))


def test_gradients_against_differences():
    d = case(6, 30, 12, "f32", 11, masked=0.0)
    r = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"])
    g = gen(3)
    for name, grad in (("h", r.dhidden), ("w", r.dweight)):
        v = torch.randn(d[name].shape, generator=g).cuda()
        step = 2.0 ** -7
        up, down = [M.linear_cross_entropy_forward(
            **{"hidden": d["h"], "weight": d["w"], "targets": d["t"],
               **{{"h": "hidden", "w": "weight"}[name]: d[name] + s * v}}).loss
            for s in (step, -step)]
        slope = ((up - down) / (2 * step)).item()
        # third derivatives below 10 of |v|^3, and the losses' roundings
        most = 10 * step ** 2 * v.norm().item() ** 3 / 6 + 4 * 2.0 ** -24 / step
        assert abs(slope - (grad * v).sum().item()) <= most


def test_a_float32_weight_under_16_bits_and_what_needs_no_gradient():
    d = case(24, 150, 64, "bf16", 2)
    w = d["w"].float().requires_grad_()
    loss, _ = M.linear_cross_entropy(d["h"], w, d["t"])
    loss.backward()
    want = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"])
    assert w.grad.dtype == torch.float32
    assert torch.equal(w.grad, want.dweight.float())
    h = d["h"].clone().requires_grad_()
    M.linear_cross_entropy(h, d["w"], d["t"])[0].backward()
    assert torch.equal(h.grad, want.dhidden)


def test_streams_and_graph():
    d = case(200, 1000, 96, "bf16", 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"])
    s.synchronize()
    check(d, got)
    scale = torch.ones(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"],
                                        grad_scale=scale)
        f = M.linear_cross_entropy_forward(d["h"], d["w"], d["t"])
        b = M.linear_cross_entropy_backward(d["h"], d["w"], d["t"], f.saved,
                                            grad_scale=scale)
    for seed in range(4):
        e = case(200, 1000, 96, "bf16", 20 + seed)
        for k in d:
            d[k].copy_(e[k])
        scale.fill_(2.0 ** seed)
        graph.replay()
        torch.cuda.synchronize()
        want = M.linear_cross_entropy_grad(e["h"], e["w"], e["t"],
                                           grad_scale=scale)
        for k in ("loss", "logp", "dhidden", "dweight"):
            assert torch.equal(getattr(r, k), getattr(want, k)), k
        assert torch.equal(f.loss, want.loss)
        assert torch.equal(b[0], want.dhidden)
        assert torch.equal(b[1], want.dweight)


def test_given_outputs_count_as_written():
    d = case(8, 20, 16, "f32")
    x = d["h"].clone().requires_grad_()
    y = x * 1.0
    z = y * y
    M.linear_cross_entropy_grad(d["h"], d["w"], d["t"], out=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        z.sum().backward()


def test_a_weight_past_32_bits_of_offset():
    """4.4 GB of weights; targets in their last rows."""
    vocab, width, rows = 1_100_003, 2048, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.empty(vocab, width, dtype=torch.bfloat16, device="cuda")
    w.normal_(0, 0.02, generator=g)
    h = torch.randn(rows, width, generator=g, device="cuda").bfloat16()
    t = torch.arange(vocab - 16, vocab, 2, device="cuda")
    f = M.linear_cross_entropy_forward(h, w, t)
    z = torch.cat([h.double() @ w[lo:lo + 100_000].double().t().contiguous()
                   for lo in range(0, vocab, 100_000)], 1)
    lp = torch.log_softmax(z, 1)
    # sums of 2048 products of 0.8 x 0.02 each and of 8600 tiles
    near(f.logp, lp.gather(1, t[:, None])[:, 0],
         torch.full((rows,), (2048 // 16 + 16) * 2.0 ** -24 * 40 +
                    9000 * 2.0 ** -24, device="cuda").double())
    dh, dw = M.linear_cross_entropy_backward(h, w, t, f.saved)
    last = torch.arange(vocab - 16, vocab, device="cuda")
    p = lp[:, last].exp()
    p[torch.arange(rows), torch.arange(0, 16, 2)] -= 1
    want = (p / rows).t().contiguous() @ h.double()
    assert R.off(dw[last], want) <= 2 * 2.0 ** -8
    full = torch.zeros(rows, width, dtype=torch.float64, device="cuda")
    for lo in range(0, vocab, 100_000):
        full += lp[:, lo:lo + 100_000].exp() @ w[lo:lo + 100_000].double()
    full = (full - w[t].double()) / rows
    assert R.off(dh, full) <= 2 * 2.0 ** -8


def test_the_workspace_is_checked():
    from mixed_precision_optimizer_mta_amd import _binding as B
    d = case(20, 50, 64, "bf16")
    loss = torch.empty(1, device="cuda")
    a = B.mta_linear_loss_args(
        h=d["h"].data_ptr(), w=d["w"].data_ptr(), targets=d["t"].data_ptr(),
        loss=loss.data_ptr(), rows=20, vocab=50, width=64, ldh=64, ldw=64,
        ignore_index=-100, type=B.MTA_BF16, dw_type=B.MTA_BF16, lddh=64,
        lddw=64)
    need = B.mta_linear_loss_workspace(a)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for at, size, code in ((None, need, -1), (ws.data_ptr(), need - 1, -1),
                           (ws.data_ptr() + 128, need, -2),
                           (d["h"].data_ptr() // 256 * 256, need, -1)):
        a.workspace, a.workspace_bytes = at, size
        with pytest.raises(M.MtaError) as e:
            B.mta_linear_loss(a)
        assert e.value.code == code
