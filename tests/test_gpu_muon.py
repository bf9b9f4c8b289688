"""MtaOptimizer's kind "muon": against its float64 definition step by step,
beside groups of other kinds, and the training step that ends in it."""
import pytest
import torch

import matrix_oracle as R
import mixed_precision_optimizer_mta_amd as M

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


SHAPES = [(40, 70), (70, 40), (64, 64), (8, 3, 3, 3), (130, 257)]


def params(dtype=torch.float32, seed=0):
    g = gen(seed)
    return [torch.nn.Parameter((torch.randn(*s, generator=g) * 0.02).to(
        dtype).cuda()) for s in SHAPES]


def set_grads(ps, seed):
    g = gen(100 + seed)
    for p in ps:
        x = (torch.randn(p.shape, generator=g) * 1e-3).to(p.dtype).cuda()
        if p.grad is None:
            p.grad = x
        else:
            p.grad.copy_(x)


def scale_of(rows, cols, kind):
    if kind == "spectral":
        return max(1.0, rows / cols) ** 0.5
    return 0.2 * max(rows, cols) ** 0.5 if kind == "rms" else kind


class Plain:
    """The rule in float64, on the CPU."""

    def __init__(self, ps, lr, wd, mu, nesterov, scale):
        self.w = [p.detach().cpu().double().flatten(1) for p in ps]
        self.m = [torch.zeros_like(w) for w in self.w]
        self.o = lr, wd, mu, nesterov, scale

    def step(self, gs, coef=1.0):
        lr, wd, mu, nesterov, scale = self.o
        for i, g in enumerate(gs):
            g = g.detach().cpu().double().flatten(1) * coef
            self.m[i] = self.m[i] * mu + g
            u = g + mu * self.m[i] if nesterov else self.m[i]
            s = scale_of(*u.shape, scale)
            self.w[i] = self.w[i] * (1 - lr * wd) - \
                lr * s * R.orthogonal(u)


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("scale", ["spectral", "rms", 0.5])
def test_float32(scale, nesterov):
    ps = params()
    opt = M.MtaOptimizer(ps, kind="muon", lr=0.02, weight_decay=0.1,
                         momentum=0.9, nesterov=nesterov, update_scale=scale)
    plain = Plain(ps, 0.02, 0.1, 0.9, nesterov, scale)
    start = [w.clone() for w in plain.w]
    for k in range(3):
        set_grads(ps, k)
        plain.step([p.grad for p in ps])
        opt.step()
    for p, w, w0, m in zip(ps, plain.w, start, plain.m):
        y = p.detach().cpu().double().flatten(1)
        # 1e-5 of the way gone (a result's error, as for orthogonalize), and
        # two roundings of the weights a step
        most = 1e-5 * (w - w0).norm() + 6 * 2.0 ** -24 * w.norm()
        assert (y - w).norm() <= most
        assert R.off(opt.state[p]["momentum_buffer"].flatten(1), m) <= 1e-6


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_master_weights(dtype):
    ps = params(dtype)
    opt = M.MtaOptimizer(ps, kind="muon", lr=0.02, momentum=0.9,
                         master_weights=True)
    plain = Plain(ps, 0.02, 0.0, 0.9, True, "spectral")
    start = [w.clone() for w in plain.w]
    for k in range(2):
        set_grads(ps, k)
        plain.step([p.grad for p in ps])
        opt.step()
    for p, w, w0 in zip(ps, plain.w, start):
        master = opt.state[p]["master_weight"]
        assert torch.equal(p.detach(), master.to(dtype))
        # 1.5e-3 of the way (products of 11 bits)
        assert (master.cpu().double().flatten(1) - w).norm() <= \
            1.5e-3 * (w - w0).norm()


def test_beside_another_kind_under_one_clip():
    """Matrices by muon, the rest by AdamW, one joint norm: the rest exactly as
    in an AdamW optimizer that is given that coefficient."""
    g = gen(5)
    mats = params()
    vecs = [torch.nn.Parameter(torch.randn(n, generator=g).cuda())
            for n in (70, 513)]
    twin = [torch.nn.Parameter(v.detach().clone()) for v in vecs]
    opt = M.MtaOptimizer(
        [{"params": mats, "kind": "muon", "lr": 0.02, "momentum": 0.95,
          "weight_decay": 0.01}, {"params": vecs}],
        kind="adamw", lr=1e-3, weight_decay=0.1, max_norm=0.05)
    alone = M.MtaOptimizer(twin, kind="adamw", lr=1e-3, weight_decay=0.1)
    plain = Plain(mats, 0.02, 0.01, 0.95, True, "spectral")
    start = [w.clone() for w in plain.w]
    for k in range(3):
        set_grads(mats + vecs, k)
        norm = sum(p.grad.double().square().sum() for p in mats + vecs).sqrt()
        coef = min(1.0, 0.05 / (norm.item() + 1e-6))
        gs = [p.grad.clone() for p in mats]
        opt.step()
        assert opt.last_norm.item() == pytest.approx(norm.item(), rel=1e-6)
        c = opt.last_coef.item()
        assert c == pytest.approx(coef, rel=1e-5)
        plain.step(gs, c)
        for t, v in zip(twin, vecs):
            t.grad = v.grad * opt.last_coef
        alone.step()
    for t, v in zip(twin, vecs):
        assert torch.equal(t, v)
    for p, w, w0 in zip(mats, plain.w, start):
        assert (p.detach().cpu().double().flatten(1) - w).norm() <= \
            1e-5 * (w - w0).norm() + 6 * 2.0 ** -24 * w.norm()


def test_loss_scale_skips_and_zeroes():
    ps = params(torch.float16)
    opt = M.MtaOptimizer(ps, kind="muon", lr=0.02, momentum=0.9,
                         master_weights=True, loss_scale=256.0, zero_grad=True)
    set_grads(ps, 0)
    opt.step()
    before = [(opt.state[p]["master_weight"].clone(),
               opt.state[p]["momentum_buffer"].clone()) for p in ps]
    assert not any(p.grad.any() for p in ps)
    set_grads(ps, 1)
    ps[1].grad[0, 0] = float("inf")
    opt.step()
    for p, (w, m) in zip(ps, before):
        assert torch.equal(opt.state[p]["master_weight"], w)
        assert torch.equal(opt.state[p]["momentum_buffer"], m)
        assert not p.grad.any()
    assert opt.amp.read()["scale"] == 128.0
    # the first step, unscaled (in float16 the small gradients would not hold)
    twin = params(torch.float16)
    set_grads(twin, 0)
    plain = Plain(twin, 0.02, 0.0, 0.9, True, "spectral")
    start = [w.clone() for w in plain.w]
    plain.step([p.grad.double() / 256.0 for p in twin])
    for (y, _), w, w0 in zip(before, plain.w, start):
        assert (y.cpu().double().flatten(1) - w).norm() <= \
            1.5e-3 * (w - w0).norm()


def test_captured_steps():
    ps, twin = params(), params()
    for x in (ps, twin):
        set_grads(x, 0)
    a, b = [M.MtaOptimizer(x, kind="muon", lr=0.02, momentum=0.9,
                           weight_decay=0.1, max_norm=0.1, capturable=True)
            for x in (ps, twin)]
    a.step()
    b.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for k in range(1, 5):
        set_grads(ps, k)
        set_grads(twin, k)
        graph.replay()
        b.step()
        torch.cuda.synchronize()
        for p, q in zip(ps, twin):
            assert torch.equal(p, q)
    assert a.amp.read()["step"] == 5


def test_state_dict_round_trip():
    def make(ps):
        return M.MtaOptimizer([{"params": ps[:3], "kind": "muon", "lr": 0.02,
                                "momentum": 0.9}, {"params": ps[3:]}],
                              kind="adamw", lr=1e-3)

    ps = params()
    opt = make(ps)
    for k in range(2):
        set_grads(ps, k)
        opt.step()
    twin = [torch.nn.Parameter(p.detach().clone()) for p in ps]
    other = make(twin)
    other.load_state_dict(opt.state_dict())
    for k in range(2, 4):
        for x, o in ((ps, opt), (twin, other)):
            set_grads(x, k)
            o.step()
    assert all(torch.equal(p, q) for p, q in zip(ps, twin))
    assert opt.state_dict()["state"][0]["step"] == 4


def test_moved_and_missing_gradients():
    ps, twin = params(), params()
    opt, ref = [M.MtaOptimizer(x, kind="muon", lr=0.02, momentum=0.9)
                for x in (ps, twin)]
    for k in range(3):
        for x in (ps, twin):
            set_grads(x, k)
        ps[0].grad = ps[0].grad.clone()
        ps[2].grad = twin[2].grad = None
        opt.step()
        ref.step()
        assert all(torch.equal(p, q) for p, q in zip(ps, twin))


def test_a_training_step():
    """A small language model's step: activations kept in 8 bits, the output
    layer's loss without logits times the device's loss scale, matrices by
    muon and the rest by AdamW: gradients and new weights against float64."""
    vocab, width, rows = 500, 64, 96
    g = gen(1)
    emb = torch.nn.Parameter((torch.randn(vocab, width, generator=g)).cuda())
    w1 = torch.nn.Parameter((torch.randn(128, width, generator=g) *
                             0.1).cuda())
    b1 = torch.nn.Parameter(torch.zeros(128).cuda())
    w2 = torch.nn.Parameter((torch.randn(width, 128, generator=g) *
                             0.1).cuda())
    head = torch.nn.Parameter((torch.randn(vocab, width, generator=g) *
                               0.2).cuda())
    tokens = torch.randint(vocab, (rows,), generator=g).cuda()
    targets = torch.randint(vocab, (rows,), generator=g).cuda()
    targets[::9] = -100
    opt = M.MtaOptimizer(
        [{"params": [w1, w2], "kind": "muon", "lr": 0.02, "momentum": 0.95},
         {"params": [emb, b1, head]}], kind="adamw", lr=1e-3,
        loss_scale=1024.0, max_norm=1.0)
    start = [p.detach().cpu().double() for p in (w1, w2)]
    x = emb[tokens]
    h = M.checkpointed_act(M.checkpointed_linear(x, w1, b1), "gelu")
    y = x + M.checkpointed_linear(h, w2)
    loss, logp = M.linear_cross_entropy(y, head, targets)
    (loss * opt.loss_scale).backward()

    e = [p.detach().cpu().double().requires_grad_()
         for p in (emb, w1, b1, w2, head)]
    ex = e[0][tokens.cpu()]
    eh = torch.nn.functional.gelu(ex @ e[1].t() + e[2])
    z = (ex + eh @ e[3].t()) @ e[4].t()
    want = torch.nn.functional.cross_entropy(z, targets.cpu())
    want.backward()
    assert loss.item() == pytest.approx(want.item(), rel=1e-5)
    assert logp[0].item() == 0.0
    for p, q in zip((emb, w1, b1, w2, head), e):
        # what is kept in 8 bits is off by at most 2^-4 of itself
        assert R.off(p.grad / 1024.0, q.grad) <= 2.0 ** -4
    assert R.off(head.grad / 1024.0, e[4].grad) <= 1e-4   # not through those
    gs = [p.grad.detach().cpu().double() for p in (w1, w2)]
    opt.step()
    c = opt.last_coef.item() / 1024.0
    for p, w0, gr in zip((w1, w2), start, gs):
        s = scale_of(*w0.shape, "spectral")
        step = 0.02 * s * R.orthogonal(gr * c * 1.95)
        assert R.off(p, w0 - step) <= 1e-5
