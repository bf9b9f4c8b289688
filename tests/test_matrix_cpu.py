"""The operators of include/mta_matrix.h without a GPU: exports, struct
layouts and the refusal of every bad argument before any device work."""
import ctypes
import os
import re

import pytest
import torch

import mixed_precision_optimizer_mta_amd as M
from mixed_precision_optimizer_mta_amd import _binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mta_matrix.h")


def test_library_exports_every_declared_operator():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mta_[a-z0-9_]+)\s*\(", text)))
    lib = ctypes.CDLL(B.LIB_PATH)
    for name in names:
        assert hasattr(lib, name), name
    assert sorted(B.MATRIX_EXPORTS) == names
    assert M.mta_matrix_version() == 1 == B.MATRIX_VERSION


def test_struct_layouts():
    assert ctypes.sizeof(B.mta_ortho_matrix) == 80
    assert ctypes.sizeof(B.mta_ortho_args) == 112
    assert ctypes.sizeof(B.mta_linear_loss_args) == 176


def _code(fn, *a):
    with pytest.raises(M.MtaError) as e:
        fn(*a)
    return e.value.code


G, MO, OUT, W, W16, WS = (k << 28 for k in range(1, 7))
GOOD = dict(g=G, m=MO, out=OUT, w=W, w16=W16, rows=40, cols=70, ldg=70,
            ldout=70, scale=1.0)


def ortho(entries=None, co=(3.4445, -4.7750, 2.0315), **kw):
    ms = [GOOD] if entries is None else entries
    table = (B.mta_ortho_matrix * max(1, len(ms)))(
        *[B.mta_ortho_matrix(**{**GOOD, **m}) for m in ms])
    steps = kw.get("steps", 5)
    flat = list(co) * max(1, min(steps, 16))
    args = B.mta_ortho_args(
        matrices=table, count=len(ms), workspace=WS,
        workspace_bytes=1 << 27,
        coefficients=(ctypes.c_double * len(flat))(*flat), eps=1e-7,
        momentum=0.95, lr=0.02, weight_decay=0.1, steps=5, type=B.MTA_BF16,
        out_type=B.MTA_BF16, copy_type=B.MTA_BF16, nesterov=1, precise=0)
    for k, v in kw.items():
        setattr(args, k, v)
    args._keep = table
    return args


@pytest.mark.parametrize("matrix,kw,code", [
    (dict(rows=-1), {}, -1),
    (dict(cols=-1), {}, -1),
    (dict(rows=(1 << 20) + 1), {}, -1),
    (dict(cols=(1 << 20) + 1), {}, -1),
    (dict(g=None), {}, -1),
    (dict(out=None, w=None, w16=None), {}, -1),
    (dict(w=None), {}, -1),                    # a copy without weights
    (dict(scale=float("nan")), {}, -1),
    (dict(scale=float("inf")), {}, -1),
    (dict(ldg=69), {}, -1),
    (dict(ldout=69), {}, -1),
    (dict(ldg=1 << 60), {}, -1),
    (dict(g=G + 1), {}, -2),
    (dict(out=OUT + 1), {}, -2),
    (dict(m=MO + 2), {}, -2),
    (dict(w=W + 2), {}, -2),
    (dict(w16=W16 + 1), {}, -2),
    (dict(g=G + 2), dict(type=B.MTA_F32), -2),
    (dict(out=G), {}, -1),                     # overlaps
    (dict(m=G + 64), {}, -1),
    (dict(w=MO), {}, -1),
    (dict(w16=W + 16), {}, -1),
    (dict(out=WS + 256), {}, -1),
    ({}, dict(type=3), -3),
    ({}, dict(out_type=-1), -3),
    ({}, dict(copy_type=B.MTA_F32), -3),
    ({}, dict(steps=0), -1),
    ({}, dict(steps=17), -1),
    ({}, dict(coefficients=None), -1),
    ({}, dict(co=(3.4445, -4.7750, float("nan"))), -1),
    ({}, dict(co=(9.0, 0.0, 0.0)), -1),        # grows to 9^5
    ({}, dict(co=(3.4445, 4.7750, 2.0315)), -1),
    ({}, dict(eps=-1e-9), -1),
    ({}, dict(eps=float("nan")), -1),
    ({}, dict(momentum=-0.1), -1),
    ({}, dict(momentum=float("inf")), -1),
    ({}, dict(lr=-1.0), -1),
    ({}, dict(lr=float("nan")), -1),
    ({}, dict(weight_decay=-1.0), -1),
    ({}, dict(nesterov=2), -1),
    ({}, dict(precise=2), -1),
    ({}, dict(d_coef=0x7000001), -2),
    ({}, dict(d_amp=0x7000004), -2),
    ({}, dict(d_coef=W + 4), -1),
    ({}, dict(workspace=None), -1),
    ({}, dict(workspace=WS + 128), -2),
    ({}, dict(workspace_bytes=1000), -1),
    ({}, dict(matrices=None), -1),
    ({}, dict(count=-1), -1),
])
def test_orthogonalize_refuses(matrix, kw, code):
    co = kw.pop("co") if "co" in kw else (3.4445, -4.7750, 2.0315)
    assert _code(B.mta_orthogonalize, ortho([matrix], co, **kw)) == code
    assert M.mta_last_error() != ""


def test_orthogonalize_refuses_what_only_small_values_reach():
    """Five steps and three more bring whatever begins above 1/512 to 1,
    where the last polynomial, 60 (x^2 - 1)^2, is 0; smaller ones come to
    0.447, where it makes 17 of them."""
    co = [(3.4445, -4.7750, 2.0315)] * 5 + [(1.875, -1.25, 0.375)] * 3 + \
        [(60.0, -120.0, 60.0)]
    flat = [v for row in co for v in row]
    x = [k / 512 for k in range(1, 513)]
    for a, b, c in co:
        x = [v * (a + b * v * v + c * v ** 4) for v in x]
        assert max(map(abs, x)) < 7
    args = ortho()
    args.steps, args.coefficients = 9, (ctypes.c_double * 27)(*flat)
    assert _code(B.mta_orthogonalize, args) == -1
    assert "coefficients" in M.mta_last_error()


@pytest.mark.parametrize("co,steps", [((3.4445, -4.7750, 2.0315), 11),
                                      ((5.0, -20.0, 16.0), 8)])
def test_orthogonalize_refuses_slopes_past_2_18(co, steps):
    """Ten usual steps, and seven of 16 x^5 - 20 x^3 + 5 x (whose values stay in
    [-1, 1]), come as far as the workspace, which is missing; one more does
    not."""
    for n, word in ((steps - 1, "workspace"), (steps, "coefficients")):
        args = ortho(workspace=None)
        args.steps = n
        args.coefficients = (ctypes.c_double * (3 * n))(*list(co) * n)
        assert _code(B.mta_orthogonalize, args) == -1
        assert word in M.mta_last_error()


def test_orthogonalize_refuses_shared_outputs_of_a_list():
    far = {k: GOOD[k] + (1 << 20) for k in ("g", "m", "out", "w", "w16")}
    assert _code(B.mta_orthogonalize,
                 ortho([{}, {**far, "out": OUT + 100}])) == -1
    assert "matrix" in M.mta_last_error() or "tensor" in M.mta_last_error()


def test_orthogonalize_workspace():
    def need(entries, **kw):
        return B.mta_orthogonalize_workspace(ortho(entries, **kw))

    small = need([{}])
    # two runs of 64 columns: their Gram matrices and the factor in float64
    assert small >= 3 * 48 * 48 * 8
    size = dict(rows=600, cols=700, ldg=700, ldout=700)
    one = need([size])
    # two X of two planes, A and B, 600 rows each
    assert one >= 600 * (704 * 2 * 2 * 2 + 640 * 2 * 2)
    assert small % 256 == 0 and one % 256 == 0
    assert need([size], precise=1) > one
    # forty matrices share a launch, the small ones another
    assert need([{}] * 40) == 40 * small == need([{}] * 81)
    many = need([size] * 40)
    assert 40 * 600 * (704 * 8 + 640 * 4) <= many == need([size] * 81)
    assert need([size] * 40 + [{}] * 40) == many
    # 4 GiB at a time, unless one matrix needs more
    big = dict(rows=8192, cols=8192)
    assert need([big]) < need([big] * 30) <= 1 << 32
    assert need([dict(rows=1 << 16, cols=1 << 16)]) > 1 << 32
    assert need([dict(rows=0)]) == 0
    assert _code(B.mta_orthogonalize_workspace, ortho([dict(rows=-1)])) == -1


def test_nothing_to_do_touches_no_device():
    B.mta_orthogonalize(ortho([]))
    B.mta_orthogonalize(ortho([dict(rows=0), dict(cols=0, g=None)],
                              workspace=None, workspace_bytes=0))


def test_python_refusals():
    x = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="GPU"):
        M.orthogonalize(x)
    with pytest.raises(ValueError, match="steps"):
        M.orthogonalize([], steps=0)
    with pytest.raises(ValueError, match="coefficients"):
        M.orthogonalize([], coefficients=(1.0, 2.0))
    with pytest.raises(ValueError, match="coefficients"):
        M.orthogonalize([], steps=3, coefficients=[(1.0, 2.0, 3.0)] * 2)
    with pytest.raises(ValueError, match="one momentum"):
        M.muon_update([x], [])
    with pytest.raises(ValueError, match="scale"):
        M.orthogonalize([x], scale=[1.0, 2.0])
    with pytest.raises(ValueError, match="out"):
        M.orthogonalize([x], out=[])


H, WT, T, WS2, SC, DH, DW, SV, LP, LO = (k << 28 for k in range(8, 18))


def linear(**kw):
    a = B.mta_linear_loss_args(
        h=H, w=WT, targets=T, weights=None, d_grad_scale=SC, dh=DH, dw=DW,
        saved=SV, logp=LP, loss=LO, workspace=WS2, workspace_bytes=1 << 27,
        rows=20, vocab=50, width=64, ldh=64, ldw=64, lddh=64, lddw=64,
        ignore_index=-100, type=B.MTA_BF16, dw_type=B.MTA_F32)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


REFUSED = [
    (dict(rows=-1), -1), (dict(rows=(1 << 30) + 1), -1),
    (dict(vocab=0), -1), (dict(vocab=(1 << 28) + 1), -1),
    (dict(width=0), -1), (dict(width=(1 << 20) + 1), -1),
    (dict(rows=1 << 30, vocab=1 << 28), -1),
    (dict(type=3), -3), (dict(dw_type=-1), -3),
    (dict(accumulate=2), -1), (dict(reserved=1), -1),
    (dict(h=None), -1), (dict(w=None), -1), (dict(targets=None), -1),
    (dict(ldh=63), -1), (dict(ldw=63), -1), (dict(lddh=63), -1),
    (dict(lddw=63), -1), (dict(ldw=1 << 60), -1),
    (dict(h=H + 1), -2), (dict(w=WT + 1), -2), (dict(dh=DH + 1), -2),
    (dict(dw=DW + 2), -2), (dict(targets=T + 4), -2),
    (dict(d_grad_scale=SC + 2), -2), (dict(saved=SV + 8), -2),
    (dict(dh=H), -1), (dict(dw=WT), -1), (dict(dw=DH + 64), -1),
    (dict(dh=T), -1), (dict(dw=SC), -1),
]


@pytest.mark.parametrize("kw,code", REFUSED + [
    (dict(loss=None), -1), (dict(loss=LO + 2), -2), (dict(logp=LP + 1), -2),
    (dict(weights=LP + 4), -1), (dict(weights=0x7000002), -2),
    (dict(logp=LO), -1), (dict(saved=H + 128), -1)])
def test_linear_loss_refuses(kw, code):
    assert _code(B.mta_linear_loss, linear(**kw)) == code
    assert M.mta_last_error() != ""


@pytest.mark.parametrize("kw,code", REFUSED + [
    (dict(saved=None), -1), (dict(dh=None, dw=None), -1),
    (dict(dh=SV), -1)])
def test_linear_loss_backward_refuses(kw, code):
    assert _code(B.mta_linear_loss_backward, linear(**kw)) == code


def test_linear_loss_workspace():
    def need(**kw):
        return B.mta_linear_loss_workspace(linear(**kw), 256)

    big = dict(rows=8192, vocab=50257, width=1600, ldh=1600, ldw=1600,
               lddh=1600, lddw=1600)
    loss = need(**big, dh=None, dw=None)
    both = need(**big)
    # no logits: 823 MB in 16 bits; a piece of dz is 256 MiB at most, the
    # hidden states' sums in 32 bits are 52 MB
    assert loss < 100 << 20 < both < 420 << 20
    # the vocabulary adds its tiles' partial sums alone
    more = need(**{**big, "vocab": 4 * 50257})
    assert more - both <= 8 * 8192 * (3 * 50257 // 128 + 1) + (300 << 20)
    # a weight that is not as the products want it is laid out again
    assert need(**{**big, "w": WT + 2}) >= both + 50257 * 1600 * 2
    assert need(rows=0) < 1 << 20
    assert _code(B.mta_linear_loss_workspace, linear(), -1) == -1
    assert _code(B.mta_linear_loss_workspace, linear(vocab=0), 256) == -1
    for rows, vocab, width in [(1, 1, 1), (3, 100000, 7), (70000, 2, 9),
                               (1 << 20, 1 << 10, 64)]:
        for cus in (1, 8, 256, 304):
            assert B.mta_linear_loss_workspace(
                linear(rows=rows, vocab=vocab, width=width, ldh=width,
                       ldw=width, lddh=width, lddw=width), cus) % 256 == 0


def test_linear_loss_python_refusals():
    h, w = torch.zeros(4, 8), torch.zeros(5, 8)
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        M.linear_cross_entropy_grad(h, w, t)
    with pytest.raises(TypeError, match="hidden"):
        M.linear_cross_entropy_forward(h.double(), w, t)
    with pytest.raises(ValueError, match="GPU"):
        M.linear_cross_entropy(h, w, t)
