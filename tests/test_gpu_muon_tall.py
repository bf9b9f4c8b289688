"""MtaOptimizer's kind "muon" on tall matrices beyond the small ones' way, whose
weights are updated from X turned back, and on more matrices than a launch
takes."""
import pytest
import torch

import matrix_oracle as R
import mixed_precision_optimizer_mta_amd as M
from test_gpu_muon import Plain, gen

pytestmark = pytest.mark.gpu

SHAPES = [(257, 130), (130, 257), (300, 65), (129, 9, 9), (1601, 70)]


def params(shapes, dtype=torch.float32, seed=0):
    g = gen(seed)
    return [torch.nn.Parameter((torch.randn(*s, generator=g) * 0.02).to(
        dtype).cuda()) for s in shapes]


def set_grads(ps, seed):
    g = gen(100 + seed)
    for p in ps:
        x = (torch.randn(p.shape, generator=g) * 1e-3).to(p.dtype).cuda()
        if p.grad is None:
            p.grad = x
        else:
            p.grad.copy_(x)


def way(opt, plain, ps, steps, part, **kw):
    """Some steps of both; each weight within `part` of the way gone and two
    roundings of itself a step."""
    start = [w.clone() for w in plain.w]
    for k in range(steps):
        set_grads(ps, k)
        plain.step([p.grad for p in ps])
        opt.step()
    for p, w, w0 in zip(ps, plain.w, start):
        y = opt.master(p).detach().cpu().double().flatten(1)
        assert (y - w).norm() <= part * (w - w0).norm() + \
            2 * steps * 2.0 ** -24 * w.norm()
        assert torch.equal(p.detach(), opt.master(p).to(p.dtype))


@pytest.mark.parametrize("scale", ["spectral", "rms"])
def test_float32(scale):
    ps = params(SHAPES)
    opt = M.MtaOptimizer(ps, kind="muon", lr=0.02, weight_decay=0.1,
                         momentum=0.9, update_scale=scale)
    plain = Plain(ps, 0.02, 0.1, 0.9, True, scale)
    way(opt, plain, ps, 3, 1e-5)
    for p, m in zip(ps, plain.m):
        assert R.off(opt.state[p]["momentum_buffer"].flatten(1), m) <= 1e-6


@pytest.mark.parametrize("precise,part", [(None, 1.5e-3), (True, 1e-5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_master_weights_and_a_skipped_step(dtype, precise, part):
    ps = params(SHAPES, dtype)
    opt = M.MtaOptimizer(ps, kind="muon", lr=0.02, master_weights=True,
                         loss_scale=1.0, ns_precise=precise)
    plain = Plain(ps, 0.02, 0.0, 0.95, True, "spectral")
    way(opt, plain, ps, 2, part)
    before = [(p.detach().clone(), opt.master(p).clone(),
               opt.state[p]["momentum_buffer"].clone()) for p in ps]
    set_grads(ps, 7)
    ps[0].grad[200, 100] = float("nan")
    opt.step()
    for p, (w16, w, m) in zip(ps, before):
        assert torch.equal(p.detach(), w16)
        assert torch.equal(opt.master(p), w)
        assert torch.equal(opt.state[p]["momentum_buffer"], m)


def test_more_matrices_than_a_launch_takes():
    shapes = [(257, 130), (66, 130), (40, 70), (130, 66)] * 23
    ps = params(shapes)
    opt = M.MtaOptimizer(ps, kind="muon", lr=0.02, momentum=0.9)
    way(opt, Plain(ps, 0.02, 0.0, 0.9, True, "spectral"), ps, 2, 1e-5)
