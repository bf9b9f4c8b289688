"""Plain float64 forms of the operators of include/mta_matrix.h, and a form of
the Newton-Schulz steps with the documented roundings in otherwise exact
arithmetic, from which tolerances are taken.  They share no code with the
library."""
import math

import torch

COEF = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype):
    """A rounding's relative error."""
    return torch.finfo(dtype).eps / 2


def orthogonal(x, coef=COEF, steps=5, eps=EPS):
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + eps)
    rows = [coef] * steps if not hasattr(coef[0], "__len__") else coef
    for a, b, c in rows:
        s = x @ x.t()
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.t() if tall else x


def _kept(x, scale, planes):
    """x in one or two float16 values."""
    y = (x * scale).float()
    hi = y.half().double()
    lo = (y.double() - hi).half().double() if planes == 2 else 0.0
    return (hi + lo) / scale


def orthogonal_rounded(x, planes, coef=COEF, steps=5, eps=EPS):
    """The steps with X kept in two float16 values, products of `planes` of
    them and diagonals apart."""
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + eps)
    planes = 2 if x.shape[0] < 16 else planes
    for k in range(steps):
        a, b, c = coef
        whole, part = _kept(x, 8192, 2), _kept(x, 8192, planes)
        s = part @ part.t()
        d = s.diagonal().clone()
        o = _kept(s - torch.diag(d), 1024, planes)
        q = b * o + c * (o @ o + (d[:, None] + d) * o)
        e = b * d + c * (d * d + (o @ o).diagonal())
        q = _kept(q - torch.diag(q.diagonal()), 512, planes)
        x = a * whole + e[:, None] * (whole if planes == 2 or k + 2 >= steps
                                      else part) + q @ part
    return x.t() if tall else x


def off(y, want):
    """2-norm of the difference over the 2-norm of what is wanted."""
    y, want = y.detach().cpu().double(), want.detach().cpu().double()
    norm = want.norm().item()
    return (y - want).norm().item() / norm if norm else y.norm().item()
