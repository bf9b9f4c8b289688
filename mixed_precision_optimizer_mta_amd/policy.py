"""The clipped policy loss with a KL term, from the logits, over PyTorch
tensors: mta_policy_loss and mta_policy_loss_backward of include/mta_ops.h.

``policy_loss_grad`` is the loss and its gradient in one pass over the logits,
the gradient multiplied by a factor in device memory: the ``loss_scale`` of a
loss-scaled MtaOptimizer, so that a float16 gradient is scaled before it is
rounded and the optimizer's step divides the scale out again.
``policy_loss_forward`` and ``policy_loss_backward`` are the two halves, and
``policy_loss`` is both as an autograd function.
"""
import math
from collections import namedtuple

import torch

from . import _binding as B
from .checkpoint import (_as_rows, _check_type, _on_stream, _rows_or_copy,
                         _same_device, _written)
from .torch_list import _G

#: stats: float32 [3] on the device, (loss, sum w kl, sum of the weights of
#: clipped rows); logp: float32, one a row; saved: for policy_loss_backward;
#: dlogits: the gradient, or None
PolicyLoss = namedtuple("PolicyLoss", "stats logp saved dlogits")


def _one_a_row(shape, rows):
    """Whether a shape is that of the rows, dimensions of one aside, or flat in
    their order."""
    shape = [n for n in shape if n != 1]
    return shape == [n for n in rows if n != 1] or \
        shape == [n for n in (math.prod(rows),) if n != 1]


def _vector(t, dtype, rows, dev, what):
    """The address of one value a row, for logits of shape [*rows, vocab]."""
    if t is None:
        return None
    if t.dtype != dtype or t.device != dev or not t.is_contiguous() or (
            t.shape != rows and not _one_a_row(t.shape, rows)):
        raise ValueError(f"{what} is a contiguous {dtype} tensor of shape "
                         f"{list(rows)}, one value a row, on the logits' "
                         f"device, not {t.dtype} {list(t.shape)}")
    return t.data_ptr()


def _scalar(t, dev):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() != 1 or t.device != dev:
        raise ValueError("grad_scale is a one-element float32 tensor on the "
                         "logits' device")
    return t.data_ptr()


def _run(logits, actions, old_logp, advantages, weights, ref_logp, clip_low,
         clip_high, kl_coef, grad, save, grad_scale, out):
    _check_type(logits, "logits")
    rows, vocab, ld = _as_rows(logits, "logits")
    if vocab < 1:
        raise ValueError("logits needs a last dimension of at least 1")
    dev, lead = logits.device, logits.shape[:-1]
    f32 = torch.float32
    dlogits, ldd = None, vocab
    if grad:
        if out is None:
            dlogits = logits.new_empty(logits.shape)
        else:
            if out.shape != logits.shape or out.dtype != logits.dtype:
                raise ValueError("out has the logits' shape and dtype")
            _same_device(dev, out)
            dlogits, ldd = out, _as_rows(out, "out")[2]
    # partial sums, then stats; what is handed out apart from them has its
    # own storage
    need = B.mta_policy_loss_workspace(rows)
    buf = torch.empty(need // 4 + 3, dtype=f32, device=dev)
    logp = logits.new_empty(logits.shape[:-1], dtype=f32)
    saved = torch.empty(4 * rows, dtype=f32, device=dev) if save else None
    base = buf.data_ptr()
    args = B.mta_policy_args(
        logits.data_ptr(), _vector(actions, torch.int64, lead, dev, "actions"),
        _vector(old_logp, f32, lead, dev, "old_logp"),
        _vector(advantages, f32, lead, dev, "advantages"),
        _vector(weights, f32, lead, dev, "weights"),
        _vector(ref_logp, f32, lead, dev, "ref_logp"),
        _scalar(grad_scale, dev),
        None if dlogits is None else dlogits.data_ptr(),
        saved.data_ptr() if save else None, logp.data_ptr(), base + need, base,
        need, rows, vocab, ld, ldd,
        clip_low, clip_high, kl_coef, _G[logits.dtype], 0)
    _on_stream(dev.index, B.mta_policy_loss, args)
    _written(out)
    return PolicyLoss(buf[need // 4:], logp, saved, dlogits)


def policy_loss_grad(logits, actions, old_logp, advantages, weights=None,
                     ref_logp=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                     grad_scale=None, out=None):
    """The loss over the rows of logits [..., vocab] and its gradient in one
    pass: a PolicyLoss whose dlogits is *grad_scale times the gradient, in the
    logits' dtype, in `out` (which may be the logits themselves) or a new
    tensor.

    actions: int64; old_logp, advantages: float32; weights: float32 (default
    1 / rows each; a row of weight 0 is not read and has gradient 0); ref_logp:
    float32, needed for kl_coef > 0.  Each has one value a row, in the logits'
    shape [...] or flat in the rows' order."""
    return _run(logits, actions, old_logp, advantages, weights, ref_logp,
                clip_low, clip_high, kl_coef, True, False, grad_scale, out)


def policy_loss_forward(logits, actions, old_logp, advantages, weights=None,
                        ref_logp=None, clip_low=0.2, clip_high=0.2,
                        kl_coef=0.0):
    """The loss alone; ``saved`` serves policy_loss_backward."""
    return _run(logits, actions, old_logp, advantages, weights, ref_logp,
                clip_low, clip_high, kl_coef, False, True, None, None)


def policy_loss_backward(logits, actions, saved, grad_scale=None, out=None):
    """*grad_scale times the loss's gradient with respect to the logits, from
    what policy_loss_forward saved for the same logits and actions."""
    _check_type(logits, "logits")
    rows, vocab, ld = _as_rows(logits, "logits")
    dev, lead = logits.device, logits.shape[:-1]
    if saved.numel() != 4 * rows or saved.dtype != torch.float32 or \
            saved.device != dev or not saved.is_contiguous():
        raise ValueError("saved is that of a forward over the same rows")
    given = out
    if out is None:
        out = logits.new_empty(logits.shape)
    elif out.shape != logits.shape or out.dtype != logits.dtype:
        raise ValueError("out has the logits' shape and dtype")
    _same_device(dev, out)
    args = B.mta_policy_args(
        logits=logits.data_ptr(),
        actions=_vector(actions, torch.int64, lead, dev, "actions"),
        d_grad_scale=_scalar(grad_scale, dev), dlogits=out.data_ptr(),
        saved=saved.data_ptr(), rows=rows, vocab=vocab, ld=ld,
        ldd=_as_rows(out, "out")[2], type=_G[logits.dtype])
    _on_stream(dev.index, B.mta_policy_loss_backward, args)
    _written(given)
    return out


class _Policy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, actions, *args):
        r = policy_loss_forward(logits, actions, *args)
        ctx.save_for_backward(logits, actions, r.saved)
        ctx.mark_non_differentiable(r.logp)
        # (not a view: a caller may scale the loss in place)
        return r.stats[0].clone(), r.logp

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss, _):
        logits, actions, saved = ctx.saved_tensors
        d = policy_loss_backward(logits, actions, saved,
                                 grad_scale=dloss.float().reshape(1))
        return (d,) + (None,) * 8


def policy_loss(logits, actions, old_logp, advantages, weights=None,
                ref_logp=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0):
    """(loss, logp) with the loss differentiable with respect to the logits;
    the gradient of a scaled loss is scaled before it is rounded.  Tensors of
    any strides are taken: logits whose rows are not equally spaced, such as
    the logits[:, :-1] of a batch, are copied first."""
    def flat(t):
        return None if t is None else t.contiguous()

    return _Policy.apply(_rows_or_copy(logits), flat(actions), flat(old_logp),
                         flat(advantages), flat(weights), flat(ref_logp),
                         clip_low, clip_high, kl_coef)
