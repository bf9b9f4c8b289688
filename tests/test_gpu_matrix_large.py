"""Offsets past 32 bits: a matrix, hidden states and their gradients of more than
2^31 elements."""
import pytest
import torch

import matrix_oracle as R
import mixed_precision_optimizer_mta_amd as M
from test_gpu_linear_loss import case, near
from test_gpu_ortho import matrix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tall", [False, True])
def test_a_matrix(tall):
    """Zeros but for its last columns, whose result is theirs alone."""
    rows, cols, wide = 2080, 1 << 20, 300
    y = matrix(rows, wide, "bf16", 1)
    x = torch.zeros((cols, rows) if tall else (rows, cols),
                    dtype=torch.bfloat16, device="cuda")
    at = x[-wide:].t() if tall else x[:, -wide:]
    at.copy_(y)
    got = M.orthogonalize(x)
    del x, at
    far = got[-wide:].t() if tall else got[:, -wide:]
    # 1.1e-3 as documented, and the result's rounding
    assert R.off(far, R.orthogonal(y)) <= 1.1e-3 + 2.0 ** -8
    rest = got[:-wide] if tall else got[:, :-wide]
    assert not rest.any()


def test_hidden_states():
    """512 rows 2048 times: the same mean and weight gradient, and each time the
    same rows' gradients, in pieces of the vocabulary."""
    times, width, vocab = 2048, 2056, 600
    d = case(512, vocab, width, "bf16", 3, masked=0.0)
    h = d["h"].repeat(times, 1)
    assert h.numel() > 1 << 31
    r = M.linear_cross_entropy_grad(h, d["w"], d["t"].repeat(times))
    del h
    e = R.linear_loss(d["h"], d["w"], d["t"])
    near(r.loss, e["loss"], e["loss_off"])
    logp = r.logp.view(times, 512)
    near(logp[0], e["logp"], e["logp_off"])
    assert torch.equal(logp[-1], logp[0])
    dh = r.dhidden.view(times, 512, width)
    near(dh[0].double() * times, e["dh"], e["dh_off"])
    assert torch.equal(dh[-1], dh[0]) and torch.equal(dh[times // 2], dh[0])
    # sums of 2^20 rows: an addition for every sixteen, half a step each of at
    # most the sum of magnitudes
    h, w = d["h"].double(), d["w"].double()
    z = torch.softmax(h @ w.t().contiguous(), 1)
    z[torch.arange(512), d["t"]] -= 1
    most = z.abs().t().contiguous() @ h.abs() / 512
    near(r.dweight, e["dw"], e["dw_off"] + e["dw"].abs() * 2.0 ** -8 +
         (2 ** 20 // 16) * 2.0 ** -24 * most)
