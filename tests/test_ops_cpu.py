"""The operators of include/mta_ops.h without a GPU: exports, struct layouts
and the refusal of every bad argument before any device work."""
import ctypes
import os
import re

import pytest
import torch

import mixed_precision_optimizer_mta_amd as M
from mixed_precision_optimizer_mta_amd import _binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mta_ops.h")


def test_library_exports_every_declared_operator():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(mta_[a-z0-9_]+)\s*\(", text)))
    lib = ctypes.CDLL(B.LIB_PATH)
    for name in names:
        assert hasattr(lib, name), name
    assert sorted(B.OPS_EXPORTS) == names
    assert M.mta_ops_version() == 1 == B.OPS_VERSION


def test_struct_layouts():
    assert ctypes.sizeof(B.mta_ckpt_tensor) == 64
    assert ctypes.sizeof(B.mta_ckpt_wgrad_args) == 112
    assert ctypes.sizeof(B.mta_policy_args) == 168


def _code(fn, *a):
    with pytest.raises(M.MtaError) as e:
        fn(*a)
    return e.value.code


X, Y, Q, S = 0x1000000, 0x2000000, 0x3000000, 0x4000000
GOOD = (X, None, Q, S, 4, 40, 40, 40)


def _t(**kw):
    names = ["x", "y", "q", "scale", "rows", "cols", "ldx", "ldy"]
    return tuple(kw.get(n, v) for n, v in zip(names, GOOD))


@pytest.mark.parametrize("entry,type,act,code", [
    (GOOD, 3, 0, -3),
    (GOOD, 0, 5, -1),
    (GOOD, 0, -1, -1),
    (_t(rows=-1), 0, 0, -1),
    (_t(cols=-1), 0, 0, -1),
    (_t(x=None), 0, 0, -1),
    (_t(q=None), 0, 0, -1),
    (_t(scale=None), 0, 0, -1),
    (_t(ldx=39), 0, 0, -1),
    (_t(x=X + 2), 0, 0, -2),            # float32 off 4 bytes
    (_t(x=X + 1), 1, 0, -2),
    (_t(q=Q + 8), 0, 0, -2),            # codes off 16 bytes
    (_t(y=None), 0, 1, -1),             # an activation without its output
    (_t(y=Y, ldy=39), 0, 1, -1),
    (_t(y=Y + 1), 1, 1, -2),
    (_t(q=X), 0, 0, -1),                # codes over the input
    (_t(scale=Q + 255), 0, 0, -1),      # 4 x 64 bytes of codes
    (_t(y=X + 16), 0, 1, -1),           # output shifted into the input
    (_t(y=X, ldy=41), 0, 1, -1),        # in place at another pitch
    (_t(cols=(1 << 30) + 1, ldx=1 << 31), 0, 0, -1),
    (_t(rows=1 << 60, ldx=1 << 40), 0, 0, -1),
])
def test_pack_refuses(entry, type, act, code):
    assert _code(B.mta_ckpt_pack, [entry], type, act) == code
    assert M.mta_last_error() != ""


def test_lists_refuse_shared_outputs_and_name_the_tensor():
    other = _t(x=X + 0x100000, q=Q + 0x100000, scale=S + 0x100000)
    assert _code(B.mta_ckpt_pack, [GOOD, other, _t(x=X + 0x200000)], 0, 0) \
        == -1
    assert "tensor 0" in M.mta_last_error() and "tensor 2" in \
        M.mta_last_error()
    # a later tensor's input under an earlier one's codes
    assert _code(B.mta_ckpt_pack, [GOOD, _t(
        x=Q, q=Q + 0x100000, scale=S + 0x100000)], 0, 0) == -1


def test_column_slices_of_one_buffer_do_not_overlap():
    # two outputs side by side in rows of 80: refused only when they meet
    def two(second):
        return [_t(y=Y, ldy=80),
                _t(x=X + 0x100000, q=Q + 0x100000, scale=S + 0x100000,
                   y=second, ldy=80)]
    assert _code(B.mta_ckpt_pack, two(Y + 39 * 4), 0, 1) == -1
    # the good one passes every check and fails at the missing device, or
    # (with a GPU) is not run: its addresses are made up
    if not torch.cuda.is_available():
        assert _code(B.mta_ckpt_pack, two(Y + 40 * 4), 0, 1) == -5


@pytest.mark.parametrize("fn", [B.mta_ckpt_pack, B.mta_ckpt_act_backward])
def test_null_lists(fn):
    L = B.lib()
    raw = getattr(L, fn.__name__)
    assert raw(None, 1, 0, 1, None) == -1
    assert raw(None, -1, 0, 1, None) == -1
    assert raw(None, 0, 0, 1, None) == 0       # an empty list is no work
    assert L.mta_ckpt_unpack(None, 2, 0, None) == -1


def test_backward_and_unpack_refuse():
    assert _code(B.mta_ckpt_act_backward, [_t(y=Y)], 0, 0) == -1   # no act
    assert _code(B.mta_ckpt_act_backward, [_t()], 0, 1) == -1      # no dx
    assert _code(B.mta_ckpt_act_backward, [_t(x=None, y=Y)], 0, 1) == -1
    assert _code(B.mta_ckpt_unpack, [_t()], 0) == -1
    assert _code(B.mta_ckpt_unpack, [_t(y=Q)], 0) == -1
    assert _code(B.mta_ckpt_unpack, [_t(y=Y)], 7) == -3


def _w(**kw):
    d = dict(q=Q, scale=S, dy=X, dw=Y, db=0x5000000, workspace=None,
             workspace_bytes=0, tokens=10, fin=40, fout=50, lddy=50, lddw=40,
             type=1, gtype=0, accumulate=0, reserved=0)
    d.update(kw)
    return B.mta_ckpt_wgrad_args(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), -1), (dict(fin=-1), -1), (dict(fout=-1), -1),
    (dict(type=5), -3), (dict(gtype=5), -3), (dict(accumulate=2), -1),
    (dict(reserved=1), -1), (dict(dw=None), -1), (dict(dy=None), -1),
    (dict(q=None), -1), (dict(scale=None), -1), (dict(lddy=49), -1),
    (dict(lddw=39), -1), (dict(dy=X + 1), -2), (dict(dw=Y + 2), -2),
    (dict(db=0x5000002), -2), (dict(q=Q + 4), -2),
    (dict(workspace=0x6000008), -2), (dict(db=Y + 64), -1),
    (dict(dw=X), -1), (dict(dw=Q), -1),
    (dict(fin=1 << 31, lddw=1 << 31), -1),
    (dict(tokens=1 << 55, lddy=1 << 10), -1),
])
def test_wgrad_refuses(kw, code):
    assert _code(B.mta_ckpt_wgrad, _w(**kw)) == code


def test_wgrad_workspace_sizes():
    L = B.lib()
    assert L.mta_ckpt_wgrad(None, None) == -1
    assert L.mta_ckpt_wgrad_workspace(1, 1, 1, 1, 1, None) == -1
    for bad in ((-1, 1, 1, 1, 1), (1, -1, 1, 1, 1), (1, 1, 1, 9, 1),
                (1, 1, 1, 1, -1)):
        assert _code(B.mta_ckpt_wgrad_workspace, *bad) in (-1, -3)
    # no tokens, or few: one part, no workspace
    assert B.mta_ckpt_wgrad_workspace(0, 100, 100, 1, 256) == 0
    assert B.mta_ckpt_wgrad_workspace(5, 100, 100, 1, 256) == 0
    # many tokens for few tiles: parts of whole float32 results
    n = B.mta_ckpt_wgrad_workspace(1 << 16, 64, 64, 1, 256)
    assert n > 0 and n % 16 == 0 and n >= 2 * 64 * 64 * 4


def test_gradients_of_nothing_are_no_work():
    # fout 0: nothing to write
    B.mta_ckpt_wgrad(_w(fout=0, lddy=0))


def _p(**kw):
    d = dict(logits=X, actions=0x2000000, old_logp=0x2100000,
             advantages=0x2200000, weights=0x2300000, ref_logp=0x2400000,
             d_grad_scale=0x2500000, dlogits=0x8000000, saved=0x2600000,
             logp=0x2700000, stats=0x2800000, workspace=0x2900000,
             workspace_bytes=1 << 20, rows=4, vocab=100, ld=100, ldd=100,
             clip_low=0.2, clip_high=0.2, kl_coef=0.1, type=1, reserved=0)
    d.update(kw)
    return B.mta_policy_args(**d)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), -1), (dict(vocab=0), -1), (dict(vocab=1 << 29, ld=1 << 29, ldd=1 << 29), -1),
    (dict(type=3), -3), (dict(reserved=1), -1), (dict(clip_low=-0.1), -1),
    (dict(clip_low=1.1), -1), (dict(clip_low=float("nan")), -1),
    (dict(clip_high=-0.1), -1), (dict(clip_high=float("inf")), -1),
    (dict(kl_coef=-1.0), -1), (dict(kl_coef=float("nan")), -1),
    (dict(ref_logp=None), -1), (dict(stats=None), -1),
    (dict(logits=None), -1), (dict(actions=None), -1),
    (dict(old_logp=None), -1), (dict(advantages=None), -1),
    (dict(workspace=None), -1), (dict(workspace_bytes=95), -1),
    (dict(ld=99), -1), (dict(ldd=99), -1), (dict(logits=X + 1), -2),
    (dict(actions=0x2000004), -2), (dict(saved=0x2600004), -2),
    (dict(stats=0x2800002), -2), (dict(workspace=0x2900004), -2),
    (dict(weights=0x2300001), -2), (dict(logp=0x2700002), -2),
    (dict(d_grad_scale=0x2500001), -2), (dict(dlogits=X + 2), -1),
    (dict(dlogits=X, ldd=101), -1), (dict(logp=0x2400000), -1),
    (dict(stats=0x2700008), -1), (dict(rows=1 << 58, ld=1 << 20), -1),
])
def test_policy_refuses(kw, code):
    assert _code(B.mta_policy_loss, _p(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dlogits=None), -1), (dict(saved=None), -1),
    (dict(logits=None), -1), (dict(actions=None), -1), (dict(ldd=99), -1),
    (dict(saved=0x8000000), -1), (dict(type=-1), -3),
])
def test_policy_backward_refuses(kw, code):
    assert _code(B.mta_policy_loss_backward, _p(**kw)) == code


def test_policy_null_arguments():
    L = B.lib()
    assert L.mta_policy_loss(None, None) == -1
    assert L.mta_policy_loss_backward(None, None) == -1
    assert L.mta_policy_loss_workspace(1, None) == -1
    assert _code(B.mta_policy_loss_workspace, -1) == -1
    assert B.mta_policy_loss_workspace(0) == 0
    assert B.mta_policy_loss_workspace(1) == 24
    assert B.mta_policy_loss_workspace(4096) == 4096 * 24
    assert B.mta_policy_loss_workspace(4097) == (4097 + 4096) * 24
    assert _code(B.mta_policy_loss_workspace, 1 << 60) == -1


def test_tensors_off_the_gpu_are_refused():
    x = torch.zeros(4, 40)
    for fn in (lambda: M.ckpt_pack(x), lambda: M.ckpt_act(x, "relu"),
               lambda: M.checkpointed_act(x, "relu"),
               lambda: M.checkpointed_linear(x, torch.zeros(3, 40)),
               lambda: M.policy_loss_grad(x, torch.zeros(4).long(),
                                          torch.zeros(4), torch.zeros(4)),
               lambda: M.Checkpoint8(torch.zeros(4, 64).byte(),
                                     torch.zeros(4, 2).byte(), (4, 40))):
        with pytest.raises(ValueError):
            fn()
    with pytest.raises(TypeError):
        M.ckpt_pack(x.double())
    with pytest.raises(ValueError):
        M.ckpt_act(x, "swish")
    with pytest.raises(TypeError):
        M.Checkpoint8(torch.zeros(4, 64), torch.zeros(4, 2).byte(), (4, 40))
    assert M.ckpt_pack([]) == [] and M.ckpt_unpack([]) == []


def test_one_value_a_row_has_the_rows_shape():
    from mixed_precision_optimizer_mta_amd.policy import _vector

    def fits(shape, rows):
        t = torch.zeros(shape)
        try:
            assert _vector(t, torch.float32, rows, t.device, "x") is not None
            return True
        except ValueError as e:
            assert "one value a row" in str(e)
            return False

    for rows in ((3, 5), (1, 3, 5), (3, 1, 5)):
        for good in ((3, 5), (15,), (3, 5, 1), (1, 15)):
            assert fits(good, rows)
        for bad in ((5, 3), (3, 4), (14,), (15, 2), ()):
            assert not fits(bad, rows)
    assert fits((), ()) and fits((1,), ()) and fits((), (1,))
    assert fits((0,), (0, 5)) and fits((0, 5), (0, 5))
    assert not fits((2,), ()) and not fits((1,), (0,))
    t = torch.zeros(3, 5)
    for bad in (t.double(), torch.zeros(5, 3).t()):
        with pytest.raises(ValueError):
            _vector(bad, torch.float32, (3, 5), t.device, "x")
    assert _vector(None, torch.float32, (3, 5), t.device, "x") is None


def test_rows_of_a_view():
    from mixed_precision_optimizer_mta_amd.checkpoint import _as_rows
    x = torch.zeros(4, 6, 10)
    assert _as_rows(x, "x") == (24, 10, 10)
    assert _as_rows(x[:, :, :7], "x") == (24, 7, 10)
    assert _as_rows(x[:, 2], "x") == (4, 10, 60)
    assert _as_rows(x[:, 2:3, 1:], "x") == (4, 9, 60)
    assert _as_rows(x[1, 2], "x") == (1, 10, 10)
    assert _as_rows(x[:0], "x")[0] == 0
    for bad in (x[:, :4], x.transpose(0, 1), x.transpose(1, 2),
                torch.zeros(1, 10).expand(4, 10), torch.zeros(())):
        with pytest.raises(ValueError):
            _as_rows(bad, "x")
