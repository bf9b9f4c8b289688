"""Options and checkpoints of MtaOptimizer's groups of kind "muon", without a
GPU."""
import pytest
import torch

import mixed_precision_optimizer_mta_amd as M


def p(*shape):
    return torch.nn.Parameter(torch.zeros(*shape))


def momenta(opt):
    return [g["momentum"] for g in opt.param_groups]


def test_momentum_by_default():
    """That of muon_update, unless the optimizer or the group has one."""
    groups = [{"params": [p(3, 3)], "kind": "muon"}, {"params": [p(3)]},
              {"params": [p(2, 2)], "kind": "muon", "momentum": 0.5}]

    def new(**kw):
        return M.MtaOptimizer([dict(g) for g in groups], **kw)

    assert momenta(M.MtaOptimizer([p(3, 3)], kind="muon")) == [0.95]
    assert momenta(M.MtaOptimizer([p(3, 3)], kind="muon", momentum=0.0)) == \
        [0.0]
    assert momenta(new()) == [0.95, 0.0, 0.5]
    assert momenta(new(momentum=0.0)) == [0.0, 0.0, 0.5]
    assert momenta(new(kind="momentum", momentum=0.9)) == [0.9, 0.9, 0.5]
    opt = new()
    opt.add_param_group({"params": [p(4, 3)], "kind": "muon"})
    opt.add_param_group({"params": [p(4)]})
    assert momenta(opt) == [0.95, 0.0, 0.5, 0.95, 0.0]
    for kind in ("adamw", "adam", "sgd", "momentum"):
        assert momenta(M.MtaOptimizer([p(3)], kind=kind)) == [0.0]


def test_a_checkpoint_keeps_the_kind():
    """Groups of an optimizer of kind "muon" loaded into one of another kind,
    whose groups have it as their own: the rule they were saved under."""
    a = M.MtaOptimizer([p(3, 3)], kind="muon", lr=0.02)
    a.add_param_group({"params": [p(2, 2)]})
    sd = a.state_dict()
    assert [g["kind"] for g in sd["param_groups"]] == ["muon", "muon"]
    b = M.MtaOptimizer([{"params": [p(3, 3)], "kind": "muon"},
                        {"params": [p(2, 2)], "kind": "muon"}], kind="adamw")
    b.load_state_dict(sd)
    assert [b._kind(g) for g in b.param_groups] == ["muon", "muon"]
    assert b.param_groups[0]["lr"] == 0.02
    # other kinds' groups are as they were
    assert "kind" not in M.MtaOptimizer([p(3)], kind="adamw").param_groups[0]


def test_a_group_is_a_dict():
    opt = M.MtaOptimizer([p(3, 3)], kind="muon")
    with pytest.raises(TypeError):
        opt.add_param_group([p(2, 2)])
