"""The cross entropy of a linear output layer where its sums are parted, its rows
are many or its tiles few, against the float64 definition."""
import pytest
import torch

import matrix_oracle as R
import mixed_precision_optimizer_mta_amd as M
from test_gpu_linear_loss import case, check, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("rows,vocab,width,masked", [
    (70000, 40, 24, 0.5),      # more rows than one pass of the first kernel
    (70000, 40, 24, 0.999),    # a few of many
    (3, 30001, 200, 0.0),      # dh in parts
    (3001, 70, 200, 0.3),      # dw in parts
    (130, 1030, 520, 0.1)])
def test_shapes(rows, vocab, width, masked, dtype):
    d = case(rows, vocab, width, dtype, rows, masked=masked)
    check(d, M.linear_cross_entropy_grad(d["h"], d["w"], d["t"]))


@pytest.mark.parametrize("to", list(R.DTYPES))
@pytest.mark.parametrize("rows,vocab,width", [(3001, 70, 200),
                                              (1400, 70001, 64)])
def test_added_to_what_is_there(rows, vocab, width, to):
    """dw in parts, and in pieces of the vocabulary."""
    d = case(rows, vocab, width, "bf16", 5)
    dt = R.DTYPES[to]
    old = torch.randn(vocab, width + 3, generator=torch.Generator()
                      .manual_seed(1)).to(dt).cuda()
    dw = old.clone()
    M.linear_cross_entropy_grad(d["h"], d["w"], d["t"],
                                out_weight=dw[:, :width], accumulate=True)
    e = R.linear_loss(d["h"], d["w"], d["t"])
    want = e["dw"] + old[:, :width].double()
    # the addition's own rounding to float32 and the result's
    near(dw[:, :width], want, e["dw_off"] + want.abs() * (
        R.half_step(dt) * 1.001 + 2.0 ** -24) +
        (2.0 ** -25 if dt == torch.float16 else 0.0))
    assert torch.equal(dw[:, width:], old[:, width:])


def test_one_gradient_alone():
    """Each in a plan of its own."""
    d = case(500, 3000, 130, "bf16", 6)
    f = M.linear_cross_entropy_forward(d["h"], d["w"], d["t"])
    e = R.linear_loss(d["h"], d["w"], d["t"])
    dh, none = M.linear_cross_entropy_backward(
        d["h"], d["w"], d["t"], f.saved, need_weight=False)
    assert none is None
    near(dh, e["dh"], e["dh_off"])
    none, dw = M.linear_cross_entropy_backward(
        d["h"], d["w"], d["t"], f.saved, need_hidden=False)
    assert none is None
    near(dw, e["dw"], e["dw_off"] + e["dw"].abs() * 2.0 ** -8)


def test_replays():
    """A captured call over new values, with eager work between, a mask that
    leaves other rows each time, and once none."""
    d = case(300, 2000, 96, "bf16", 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        M.linear_cross_entropy_grad(d["h"], d["w"], d["t"])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"])
    for k, masked in enumerate((0.5, 1.0, 0.0)):
        new = case(300, 2000, 96, "bf16", 20 + k, masked=masked)
        for name in ("h", "w", "t"):
            d[name].copy_(new[name])
        if masked == 1.0:
            d["t"].fill_(-100)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (r.loss, r.logp, r.dhidden, r.dweight)]
        want = M.linear_cross_entropy_grad(d["h"], d["w"], d["t"])
        for g, w in zip(got, (want.loss, want.logp, want.dhidden,
                              want.dweight)):
            assert torch.equal(g, w)
