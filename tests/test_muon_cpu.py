"""MtaOptimizer's kind "muon" without a GPU: what its constructor refuses."""
import pytest
import torch

import mixed_precision_optimizer_mta_amd as M


def p(*shape):
    return torch.nn.Parameter(torch.zeros(*shape))


def test_matrices_alone():
    M.MtaOptimizer([p(3, 4), p(3, 4, 5)], kind="muon")
    with pytest.raises(ValueError, match="two or more"):
        M.MtaOptimizer([p(3, 4), p(3)], kind="muon")
    with pytest.raises(ValueError, match="two or more"):
        M.MtaOptimizer([{"params": [p(3)], "kind": "muon"}])
    opt = M.MtaOptimizer([{"params": [p(3, 3)], "kind": "muon"},
                          {"params": [p(3)]}], kind="adamw")
    with pytest.raises(ValueError, match="two or more"):
        opt.add_param_group({"params": [p(3)], "kind": "muon"})
    assert len(opt.param_groups) == 2
    opt.add_param_group({"params": [p(4, 3)], "kind": "muon"})


def test_a_groups_kind():
    with pytest.raises(ValueError, match="own kind"):
        M.MtaOptimizer([{"params": [p(3, 3)], "kind": "sgd"}], kind="adamw")
    M.MtaOptimizer([{"params": [p(3, 3)], "kind": "sgd"}], kind="sgd")


@pytest.mark.parametrize("kw", [
    dict(update_scale="other"), dict(update_scale=float("nan")),
    dict(ns_steps=0), dict(ns_steps=17), dict(ns_coefficients=(1.0, 2.0)),
    dict(packed_moments=True)])
def test_bad_options(kw):
    with pytest.raises(ValueError):
        M.MtaOptimizer([p(3, 3)], kind="muon", **kw)


def test_needs_gradients_on_the_gpu():
    w = p(3, 3)
    opt = M.MtaOptimizer([w], kind="muon")
    opt.step()                              # none has a gradient
    w.grad = torch.zeros(3, 3)
    with pytest.raises(TypeError):
        opt.step()
