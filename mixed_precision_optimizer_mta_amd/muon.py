"""Orthogonalised updates over PyTorch tensors: mta_orthogonalize of
include/mta_matrix.h.

``orthogonalize`` brings the singular values of a matrix, or of the matrices of
a list together (up to forty a launch), near 1 by Newton-Schulz steps; ``muon_update`` is that of
momenta that take their gradients in first (the update of the Muon rule).  An
MtaOptimizer applies it to the weights of its groups of kind "muon".

Marshalling only, as for the other operators: every call runs on the current
stream of its tensors' device and may be captured into a HIP graph.
"""
import ctypes

import torch

from . import _binding as B
from .checkpoint import (_as_rows, _check_type, _on_stream, _same_device,
                         _written)
from .torch_list import _G

#: the coefficients a, b, c of one Newton-Schulz step: a step's slope at 0 is
#: as large as it can be while singular values stay within about 0.3 of 1
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _coefficients(coefficients, steps):
    """A ctypes array of a, b, c for each step, from one triple or one a
    step."""
    steps = int(steps)
    if not 1 <= steps <= B.MTA_ORTHO_STEPS:
        raise ValueError(f"steps is in [1, {B.MTA_ORTHO_STEPS}], not {steps}")
    rows = list(coefficients)
    if len(rows) == 3 and not hasattr(rows[0], "__len__"):
        rows = [rows] * steps
    if len(rows) != steps or any(len(r) != 3 for r in rows):
        raise ValueError("coefficients is one (a, b, c), or one for each of "
                         f"the {steps} steps")
    flat = [float(x) for r in rows for x in r]
    return (ctypes.c_double * len(flat))(*flat)


def _matrix(t, what):
    """(rows, cols, pitch) of a matrix."""
    _check_type(t, what)
    if t.dim() != 2:
        raise ValueError(f"{what} is a matrix, not a tensor of "
                         f"{t.dim()} dimensions")
    return _as_rows(t, what)


def _scales(scale, count):
    if scale is None:
        return [1.0] * count
    if isinstance(scale, (int, float)):
        return [float(scale)] * count
    scales = [float(s) for s in scale]
    if len(scales) != count:
        raise ValueError("scale is one number, or one for each matrix")
    return scales


def table(entries):
    """The matrices of a call: entries (g, m, out, w, w16 as addresses, rows,
    cols, ldg, ldout, scale)."""
    return (B.mta_ortho_matrix * max(1, len(entries)))(
        *[B.mta_ortho_matrix(*e) for e in entries]), len(entries)


def run(matrices, dev, type, out_type, copy_type, coefficients, eps, momentum,
        nesterov, precise, lr=0.0, weight_decay=0.0, coef=None, amp=None):
    """One mta_orthogonalize over a table(), its workspace from PyTorch's
    allocator."""
    args = B.mta_ortho_args(
        matrices=matrices[0], count=matrices[1], coefficients=coefficients,
        d_coef=coef, d_amp=amp, eps=eps, momentum=momentum, lr=lr,
        weight_decay=weight_decay, steps=len(coefficients) // 3, type=type,
        out_type=out_type, copy_type=copy_type, nesterov=int(bool(nesterov)),
        precise=int(bool(precise)))
    need = B.mta_orthogonalize_workspace(args)
    # (the allocator's blocks lie at multiples of 512 bytes)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    args.workspace = ws.data_ptr() if need else None
    args.workspace_bytes = need
    _on_stream(dev.index, B.mta_orthogonalize, args)


def _results(xs, out, dtype):
    """New tensors of dtype, or the checked `out`, one for each matrix."""
    if out is None:
        return [torch.empty(x.shape, dtype=dtype or x.dtype, device=x.device)
                for x in xs]
    outs = [out] if isinstance(out, torch.Tensor) else list(out)
    if len(outs) != len(xs) or any(
            o.shape != x.shape for o, x in zip(outs, xs)):
        raise ValueError("out has one tensor of the shape of each matrix")
    if any(o.dtype != outs[0].dtype for o in outs) or (
            dtype is not None and outs and outs[0].dtype != dtype):
        raise TypeError("the tensors of out share one dtype")
    return outs


def _call(xs, moms, out, dtype, scale, steps, coefficients, eps, momentum,
          nesterov, precise):
    co = _coefficients(coefficients, steps)
    if not xs:
        return []
    dev, dt = xs[0].device, xs[0].dtype
    scales = _scales(scale, len(xs))
    outs = _results(xs, out, dtype)
    odt = outs[0].dtype
    if odt not in _G:
        raise TypeError("results are float32, bfloat16 or float16")
    entries = []
    for i, (x, o) in enumerate(zip(xs, outs)):
        rows, cols, ld = _matrix(x, "a matrix")
        if x.dtype != dt:
            raise TypeError("the matrices of a call share one dtype")
        _same_device(dev, x, o)
        m = None if moms is None else moms[i]
        if m is not None:
            _same_device(dev, m)
            if m.dtype != torch.float32 or m.shape != x.shape or \
                    not m.is_contiguous():
                raise ValueError("a momentum is a contiguous float32 tensor "
                                 "of its gradient's shape")
        entries.append((x.data_ptr(), None if m is None else m.data_ptr(),
                        o.data_ptr(), None, None, x.shape[0], x.shape[1],
                        ld, _matrix(o, "out")[2], scales[i]))
    if precise is None:
        precise = odt != torch.bfloat16
    run(table(entries), dev, _G[dt], _G[odt], B.MTA_BF16, co, eps, momentum,
        nesterov, precise)
    if out is not None:
        _written(*outs)
    if moms is not None:
        _written(*moms)
    return outs


def orthogonalize(x, steps=5, coefficients=COEFFICIENTS, eps=1e-7, scale=None,
                  dtype=None, precise=None, out=None):
    """The matrix x, or each matrix of a list (of one dtype), divided by its
    Frobenius norm + eps and taken through `steps` Newton-Schulz steps
    X = a X + (b A + c A A) X, A = X X^T (of the transpose where there are more
    rows than columns), times `scale` (one number, or one a matrix).

    coefficients: one (a, b, c), or one for each step; small singular values
    grow by the product of the a, which is at most 2^18 (ten of the default
    steps).  The results are new tensors of `dtype` (default: x's), or `out`.
    precise: products of 22 bits instead of float16's 11, at three times the
    work; by default for float32 and float16 results, whose digits are more
    than those of the 11."""
    if isinstance(x, torch.Tensor):
        return _call([x], None, out, dtype, scale, steps, coefficients, eps,
                     0.0, False, precise)[0]
    return _call(list(x), None, out, dtype, scale, steps, coefficients, eps,
                 0.0, False, precise)


def muon_update(grads, momenta, momentum=0.95, nesterov=True, steps=5,
                coefficients=COEFFICIENTS, eps=1e-7, scale=None, dtype=None,
                precise=None, out=None):
    """The momenta m (float32, in place) become momentum * m + g, and
    g + momentum * m (nesterov) or m comes back orthogonalised as in
    ``orthogonalize``, in `dtype` (default: the gradients').  One gradient and
    one momentum, or lists of them."""
    if isinstance(grads, torch.Tensor):
        return _call([grads], [momenta], out, dtype, scale, steps,
                     coefficients, eps, momentum, nesterov, precise)[0]
    grads, momenta = list(grads), list(momenta)
    if len(grads) != len(momenta):
        raise ValueError("one momentum for each gradient")
    return _call(grads, momenta, out, dtype, scale, steps, coefficients, eps,
                 momentum, nesterov, precise)
