"""The cross entropy of a linear output layer over PyTorch tensors, from its
input and weight and without keeping the logits: mta_linear_loss and
mta_linear_loss_backward of include/mta_matrix.h.

``linear_cross_entropy_grad`` is the loss with the gradients of the hidden
states and of the weight in one call, both multiplied by a factor in device
memory: the ``loss_scale`` of a loss-scaled MtaOptimizer, which its step divides
out again.  ``linear_cross_entropy_forward`` and
``linear_cross_entropy_backward`` are the two halves, and
``linear_cross_entropy`` is both as an autograd function.

All of them may be captured into a HIP graph; as for the checkpoints' functions,
a backward pass is captured whole, together with its forward and with no graph
of an earlier eager forward over the same parameters still alive.
"""
from collections import namedtuple

import torch

from . import _binding as B
from .checkpoint import (_as_rows, _check_type, _on_stream, _rows_or_copy,
                         _same_device, _written)
from .policy import _scalar, _vector
from .torch_list import _G

#: loss: float32, no dimensions; logp: float32, one a row, 0 where a row is
#: left out; saved: for linear_cross_entropy_backward; dhidden and dweight: the
#: gradients, or None
LinearLoss = namedtuple("LinearLoss", "loss logp saved dhidden dweight")


def _weight(weight, hidden):
    _check_type(weight, "weight")
    if weight.dim() != 2 or weight.shape[0] < 1 or weight.shape[1] < 1 or \
            hidden.shape[-1] != weight.shape[1]:
        raise ValueError("weight is [vocabulary, width] and the last "
                         "dimension of hidden width, each at least 1")
    if weight.dtype != hidden.dtype:
        raise TypeError("hidden and weight share one dtype")
    return _as_rows(weight, "weight")


def _gradients(hidden, weight, need_h, need_w, out, out_weight, accumulate):
    """(dhidden, pitch, dweight, pitch): new tensors, or those given."""
    dh = dw = None
    ldh = ldw = weight.shape[1]
    if need_h:
        dh = torch.empty(hidden.shape, dtype=hidden.dtype,
                         device=hidden.device) if out is None else out
        if dh.shape != hidden.shape or dh.dtype != hidden.dtype:
            raise ValueError("out has hidden's shape and dtype")
        ldh = _as_rows(dh, "out")[2]
    elif out is not None:
        raise ValueError("out for a gradient that is not asked for")
    if accumulate and out_weight is None:
        raise ValueError("accumulate needs out_weight")
    if need_w:
        dw = torch.empty(weight.shape, dtype=weight.dtype,
                         device=weight.device) if out_weight is None else \
            out_weight
        if dw.shape != weight.shape or dw.dtype not in _G:
            raise ValueError("out_weight has weight's shape and is float32, "
                             "bfloat16 or float16")
        ldw = _as_rows(dw, "out_weight")[2]
    elif out_weight is not None:
        raise ValueError("out_weight for a gradient that is not asked for")
    _same_device(hidden.device, weight, dh, dw)
    return dh, max(ldh, weight.shape[1]), dw, max(ldw, weight.shape[1])


def _args(hidden, weight, targets, ignore_index, grad_scale, dh, lddh, dw,
          lddw, accumulate):
    _check_type(hidden, "hidden")
    rows, width, ldh = _as_rows(hidden, "hidden")
    vocab, _, ldw = _weight(weight, hidden)
    dev, lead = hidden.device, hidden.shape[:-1]
    return B.mta_linear_loss_args(
        h=hidden.data_ptr(), w=weight.data_ptr(),
        targets=_vector(targets, torch.int64, lead, dev, "targets"),
        d_grad_scale=_scalar(grad_scale, dev),
        dh=None if dh is None else dh.data_ptr(),
        dw=None if dw is None else dw.data_ptr(), rows=rows, vocab=vocab,
        width=width, ldh=ldh, ldw=ldw, lddh=lddh, lddw=lddw,
        ignore_index=ignore_index, type=_G[hidden.dtype],
        dw_type=_G[hidden.dtype if dw is None else dw.dtype],
        accumulate=int(bool(accumulate)), reserved=0)


def _run(call, args, dev):
    need = _on_stream(dev.index, lambda *a: B.mta_linear_loss_workspace(
        a[0]), args)
    # (the allocator's blocks lie at multiples of 512 bytes)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    args.workspace, args.workspace_bytes = ws.data_ptr(), need
    _on_stream(dev.index, call, args)


def _check(hidden, weight):
    _check_type(hidden, "hidden")
    if hidden.dim() == 0:
        raise ValueError("hidden needs at least one dimension")
    _weight(weight, hidden)


def _loss(hidden, weight, targets, weights, ignore_index, grad, save,
          grad_scale, out, out_weight, accumulate):
    _check(hidden, weight)
    dh, lddh, dw, lddw = _gradients(hidden, weight, grad, grad, out,
                                    out_weight, accumulate)
    dev, lead = hidden.device, hidden.shape[:-1]
    args = _args(hidden, weight, targets, ignore_index, grad_scale, dh, lddh,
                 dw, lddw, accumulate)
    f32 = torch.float32
    args.weights = _vector(weights, f32, lead, dev, "weights")
    loss = torch.empty((), dtype=f32, device=dev)
    logp = torch.empty(lead, dtype=f32, device=dev)
    saved = torch.empty(4 * args.rows, dtype=f32, device=dev) if save else None
    args.loss, args.logp = loss.data_ptr(), logp.data_ptr()
    args.saved = saved.data_ptr() if save else None
    _run(B.mta_linear_loss, args, dev)
    _written(out, out_weight)
    return LinearLoss(loss, logp, saved, dh, dw)


def linear_cross_entropy_grad(hidden, weight, targets, weights=None,
                              ignore_index=-100, grad_scale=None, out=None,
                              out_weight=None, accumulate=False):
    """The cross entropy of hidden [..., width] times weight [vocabulary,
    width] against targets (int64, [...]), summed with `weights` (float32,
    [...]; by default the mean over the rows with a target), and its gradients
    times *grad_scale.

    A row whose target is ignore_index or whose weight is 0 is not read; its
    logp is 0 and its gradient 0.  With float16, rows of unequal weights have the
    digits that are left beside the largest: what is below 2^-28 of it has fewer.
    dhidden is a new tensor or `out`; dweight a
    new one or `out_weight` (of any of the three dtypes), overwritten or, with
    accumulate, added to."""
    return _loss(hidden, weight, targets, weights, ignore_index, True, False,
                 grad_scale, out, out_weight, accumulate)


def linear_cross_entropy_forward(hidden, weight, targets, weights=None,
                                 ignore_index=-100):
    """The loss alone; ``saved`` serves linear_cross_entropy_backward."""
    return _loss(hidden, weight, targets, weights, ignore_index, False, True,
                 None, None, None, False)


def linear_cross_entropy_backward(hidden, weight, targets, saved,
                                  grad_scale=None, need_hidden=True,
                                  need_weight=True, out=None, out_weight=None,
                                  accumulate=False):
    """(dhidden, dweight), times *grad_scale, from what
    linear_cross_entropy_forward saved for the same hidden, weight and
    targets; None for one that is not needed."""
    _check(hidden, weight)
    if not need_hidden and not need_weight:
        return None, None
    rows = hidden.numel() // hidden.shape[-1]
    if saved.numel() != 4 * rows or saved.dtype != torch.float32 or \
            saved.device != hidden.device or not saved.is_contiguous():
        raise ValueError("saved is that of a forward over the same rows")
    dh, lddh, dw, lddw = _gradients(hidden, weight, need_hidden, need_weight,
                                    out, out_weight, accumulate)
    args = _args(hidden, weight, targets, 0, grad_scale, dh, lddh, dw, lddw,
                 accumulate)
    args.saved = saved.data_ptr()
    _run(B.mta_linear_loss_backward, args, hidden.device)
    _written(out, out_weight)
    return dh, dw


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, targets, weights, ignore_index):
        r = linear_cross_entropy_forward(hidden, weight, targets, weights,
                                         ignore_index)
        ctx.save_for_backward(hidden, weight, targets, r.saved)
        ctx.mark_non_differentiable(r.logp)
        return r.loss, r.logp

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss, _):
        hidden, weight, targets, saved = ctx.saved_tensors
        need_h, need_w = ctx.needs_input_grad[:2]
        dh, dw = linear_cross_entropy_backward(
            hidden, weight, targets, saved, dloss.float().reshape(1), need_h,
            need_w)
        return dh, dw, None, None, None


def linear_cross_entropy(hidden, weight, targets, weights=None,
                         ignore_index=-100):
    """(loss, logp) with the loss differentiable with respect to hidden and
    weight; the gradients of a scaled loss are scaled before they are rounded.
    Tensors of any strides are taken; a weight of another dtype (a float32
    master under 16-bit hidden states) is cast to hidden's, and its gradient
    back (linear_cross_entropy_grad writes one of float32).  There is no gradient for weights: those that require one are
    refused."""
    if weights is not None and weights.requires_grad and \
            torch.is_grad_enabled():
        raise ValueError("there is no gradient for weights: detach them")
    _check_type(hidden, "hidden")
    _check_type(weight, "weight")

    def flat(t):
        return None if t is None else t.contiguous()

    return _Linear.apply(_rows_or_copy(hidden),
                         _rows_or_copy(weight.to(hidden.dtype)), flat(targets),
                         flat(weights), ignore_index)
