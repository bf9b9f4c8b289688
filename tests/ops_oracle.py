"""Plain float64 forms of the operators of include/mta_ops.h, in numpy, and the
conversions the tests share.  They state the definitions; they share no code
with the library."""
import math

import numpy as np
import torch

BLOCK = 32
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
MOST = {torch.float16: 1.875 * 2.0 ** 15, torch.bfloat16: 1.875 * 2.0 ** 127,
        torch.float32: 1.875 * 2.0 ** 127}


def half_step(dtype):
    """A rounding's relative error."""
    return torch.finfo(dtype).eps / 2


def _e4m3():
    v = np.empty(128)
    for c in range(127):
        e, m = c >> 3, c & 7
        v[c] = (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
    v[127] = np.nan
    return v


E4M3 = _e4m3()


def to64(t):
    return t.detach().cpu().double().numpy()


def pack(x):
    """(codes [rows, cols up to 32], scale bytes, kept values [rows, cols]) of
    a tensor, by the definition."""
    v = to64(x).reshape(-1, x.shape[-1])
    rows, cols = v.shape
    most = MOST[x.dtype]
    fine = np.isfinite(v)
    c = np.where(fine, np.clip(v, -most, most), np.nan)
    nb = -(-cols // BLOCK)
    p = np.zeros((rows, nb * BLOCK))
    p[:, :cols] = c
    p = p.reshape(rows, nb, BLOCK)
    top = np.max(np.where(np.isnan(p), 0.0, np.abs(p)), axis=2)
    k = np.full(top.shape, -117)
    for b in range(-117, 129):           # the smallest k that holds
        k = np.where(top > 448 * 2.0 ** b, b + 1, k)
    y = np.abs(p) / np.exp2(k[:, :, None].astype(float))
    # nearest code, ties to the even one: between neighbours lo <= y
    yy = np.where(np.isnan(y), 0.0, y)
    lo = np.searchsorted(E4M3[:127], yy, side="right") - 1
    hi = np.minimum(lo + 1, 126)
    dl, dh = yy - E4M3[lo], E4M3[hi] - yy
    code = np.where((dh < dl) | ((dh == dl) & (lo % 2 == 1)), hi, lo)
    code = np.where(np.isnan(p), 127, code)
    kept = E4M3[code] * np.exp2(k[:, :, None].astype(float))
    neg = np.signbit(p) & ~np.isnan(p)
    kept = np.where(neg, -kept, kept)
    code = np.where(neg, code + 128, code)
    return (code.reshape(rows, -1).astype(np.uint8),
            (k + 127).astype(np.uint8), kept.reshape(rows, -1)[:, :cols])


def kept(codes, scale, cols):
    """float64 values of codes and scales."""
    c = codes.astype(int)
    v = np.where(c > 127, -1.0, 1.0) * E4M3[c & 127]
    k = np.repeat(scale.astype(float) - 127, BLOCK, axis=1)
    return (v * np.exp2(k))[:, :cols]


_erf = np.vectorize(math.erf, otypes=[float])


def act(x, kind):
    """(value, slope) in float64."""
    with np.errstate(all="ignore"):
        if kind == "relu":
            return (np.where(x > 0, x, np.where(np.isnan(x), x, 0.0)),
                    np.where(x > 0, 1.0, np.where(np.isnan(x), x, 0.0)))
        if kind == "gelu":
            phi = 0.5 * (1 + _erf(x / math.sqrt(2)))
            d = np.exp(-x * x / 2) / math.sqrt(2 * math.pi)
            xd = np.where(d == 0, 0.0, x * d)
        else:
            if kind == "silu":
                u, du = x, np.ones_like(x)
            else:
                c = 2 * math.sqrt(2 / math.pi)
                u = c * (x + 0.044715 * x ** 3)
                du = c * (1 + 3 * 0.044715 * x * x)
            phi = 1 / (1 + np.exp(-u))
            t = phi * (1 - phi)
            xd = np.where(t == 0, 0.0, x * t * du)
        v = np.where(np.isneginf(x), 0.0, x * phi)
        return v, phi + xd


def policy(z, a, old, adv, w, ref, lo, hi, beta):
    """(stats, logp, dlogits) of the clipped policy loss in float64; rows of
    weight 0 are zero."""
    rows = z.shape[0]
    stats, logp, grad = np.zeros(3), np.zeros(rows), np.zeros(z.shape)
    for t in range(rows):
        if w[t] == 0:
            continue
        top = z[t].max()
        e = np.exp(z[t] - top)
        lse = top + math.log(e.sum())
        logp[t] = z[t, a[t]] - lse
        r = math.exp(logp[t] - old[t])
        cut = min(max(r, 1 - lo), 1 + hi)
        over = r * adv[t] > cut * adv[t]
        loss, slope, kl = -min(r * adv[t], cut * adv[t]), 0.0, 0.0
        if not over:
            slope = -r * adv[t]
        if ref is not None:
            d = ref[t] - logp[t]
            kl = math.expm1(d) - d
            loss += beta * kl
            slope -= beta * math.expm1(d)
        stats += w[t] * np.array([loss, kl, float(over)])
        one = np.zeros(z.shape[1])
        one[a[t]] = 1.0
        grad[t] = w[t] * slope * (one - e / e.sum())
    return stats, logp, grad
