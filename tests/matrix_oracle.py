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


def linear_loss(h, w, targets, weights=None, ignore=-100, scale=1.0):
    """A dict of float64 values on h's device: loss, logp, dh, dw and, for the
    16-bit (or three-fold) dz, how far each may be off."""
    dt = h.dtype
    h, w = h.double().clone(), w.double()
    rows, vocab, width = h.shape[0], w.shape[0], w.shape[1]
    on = targets != ignore
    if weights is not None:
        on &= weights != 0
    h[~on] = 0
    if weights is None:
        wt = on.double() / max(1, int(on.sum()))
    else:
        wt = torch.where(on, weights.double(), 0.0)
    at = torch.where(on, targets, 0)[:, None]
    z = h @ w.t().contiguous()
    lp = torch.log_softmax(z, 1)
    logp = torch.where(on, lp.gather(1, at)[:, 0], 0.0)
    p = lp.exp()
    rest = -torch.expm1(lp.gather(1, at))
    dz = p.scatter(1, at, -rest) * (wt * scale)[:, None]
    out = {"loss": -(wt * logp).sum(), "logp": logp, "dh": dz @ w,
           "dw": dz.t().contiguous() @ h}
    # Errors.  A sum of n products in float32: one addition for every sixteen
    # of them (six times as many for float32's pairs), each half a step of at
    # most the sum of magnitudes; what is left out of float32's nine products
    # is below 2^-23 of each.
    u = 2.0 ** -24
    runs = 6 if dt == torch.float32 else 1

    def sums(n, magnitudes):
        return (runs * (n // 16 + 8) + 8) * u * magnitudes

    ez = sums(width, h.abs() @ w.abs().t().contiguous())
    far = (z - z.amax(1, keepdim=True)).abs()
    # the logit's own, the exponential's argument and value, the row's sum (64
    # of a lane's columns, joined over tiles)
    rel = 2 * ez.amax(1, keepdim=True) + (2 * far + 16) * u + \
        (96 + vocab / 128) * u
    out["logp_off"] = rel.amax(1) + 4 * u * logp.abs() + 1e-12
    out["loss_off"] = (wt.abs() * out["logp_off"]).sum() + \
        u * out["loss"].abs() + 1e-12
    half = half_step(torch.float32 if dt == torch.float32 else dt)
    room = 2.0 ** -39 * wt.abs().max() * scale if dt == torch.float16 else 0.0
    ed = dz.abs() * (rel + half + 4 * u) + room
    ed[~on] = 0
    mine = half_step(dt)
    out["dh_off"] = ed @ w.abs() + sums(vocab + 64, dz.abs() @ w.abs()) + \
        mine * out["dh"].abs() + 1e-30
    out["dw_off"] = ed.t().contiguous() @ h.abs() + \
        sums(rows + 64, dz.abs().t().contiguous() @ h.abs()) + 1e-30
    if dt == torch.float16:  # results below 2^-14 have 2^-24 between them
        out["dh_off"] += 2.0 ** -25
    return out
