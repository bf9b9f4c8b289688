"""8-bit activation checkpoints on the GPU against their float64 definition:
pack and unpack bit for bit, the activations and the weight gradient within
bounds counted from their roundings."""
import numpy as np
import pytest
import torch

import mixed_precision_optimizer_mta_amd as M
from mixed_precision_optimizer_mta_amd import _binding as B
import ops_oracle as R

pytestmark = pytest.mark.gpu
ACTS = ["relu", "silu", "gelu", "gelu_tanh"]
TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def activations(shape, dtype, seed=0, pad=0):
    """Normal values with loud channels, in rows padded by `pad`."""
    g = gen(seed)
    x = torch.randn(*shape[:-1], shape[-1] + pad, generator=g)
    x *= torch.where(torch.rand(shape[-1] + pad, generator=g) < 0.1, 30.0, 1.0)
    return x.to(dtype).cuda()[..., :shape[-1]]


def codes(ck):
    rows, nb = ck.rows, ck.blocks
    return (ck.q.cpu().numpy().reshape(rows, nb * 32),
            ck.scale.cpu().numpy().reshape(rows, nb))


def check_pack(x, ck):
    q, s, kept = R.pack(x)
    gq, gs = codes(ck)
    assert np.array_equal(gs, s)
    # a NaN keeps no sign
    assert np.array_equal(np.where(gq == 255, 127, gq), q)
    for dt in R.DTYPES.values():
        y = ck.unpack(dt)
        assert y.shape == x.shape and y.dtype == dt
        want = torch.from_numpy(kept)
        if dt == torch.float16:
            want = want.clamp(-65504, 65504)
        assert np.array_equal(R.to64(y).reshape(kept.shape),
                              want.to(dt).double().numpy(), equal_nan=True)


SHAPES = [(1, 1), (1, 31), (3, 32), (5, 33), (7, 64), (129, 97), (33, 1600),
          (2, 8197), (2, 3, 5, 40), (70, 7), (1030, 9), (1, 768), (768,)]


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_pack_is_the_definition(shape, dtype):
    x = activations(shape, R.DTYPES[dtype])
    check_pack(x, M.ckpt_pack(x))


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_pack_of_padded_rows_at_odd_addresses(dtype, pad):
    for cols in (1, 40, 65, 96):
        x = activations((37, cols + 1), R.DTYPES[dtype], cols, pad)[:, 1:]
        check_pack(x, M.ckpt_pack(x))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_16_bit_pattern(dtype):
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(R.DTYPES[dtype])
    # alone in its block, and beside a value that sets the scale
    alone = v.reshape(-1, 1).cuda()
    check_pack(alone, M.ckpt_pack(alone))
    for anchor in (448.0, 449.0, 3.5e-3, 2.0 ** -16):
        x = torch.full((65536 // 16, 32), anchor, dtype=v.dtype)
        x[:, :16] = v.reshape(-1, 16)
        check_pack(x.cuda(), M.ckpt_pack(x.cuda()))


def test_special_float32_values():
    big = torch.finfo(torch.float32).max
    rows = [[0.0] * 32, [-0.0] + [0.0] * 31, [2.0 ** -149] * 32,
            [2.0 ** -126, 2.0 ** -130] * 16, [big, 1.0] * 16,
            [float("nan")] * 32, [float("inf"), 1.0, -float("inf"), 3.0] * 8,
            [float("nan"), 448.0, 1e-3, -0.0] * 8, [448.0 * 2.0 ** -117] * 32,
            [np.nextafter(np.float32(448), np.float32(449))] * 32,
            [464.0, 1.0] * 16, [1.875 * 2.0 ** 127, 2.0 ** 100] * 16]
    for k in range(-40, 40, 7):          # ties of every code at a scale
        mid = (R.E4M3[:126] + R.E4M3[1:127]) / 2 * 2.0 ** k
        full = np.concatenate([mid, -mid])
        for i in range(0, 252, 31):
            r = np.full(32, 448 * 2.0 ** k)
            r[:len(full[i:i + 31])] = full[i:i + 31]
            rows.append(list(r))
    x = torch.tensor(np.array(rows), dtype=torch.float32).cuda()
    check_pack(x, M.ckpt_pack(x))


def test_lists_take_one_call_and_skip_empty_tensors():
    g = np.random.default_rng(3)
    xs = [activations((int(g.integers(0, 40)), int(g.integers(1, 200))),
                      torch.bfloat16, i) for i in range(70)]
    for x, ck in zip(xs, M.ckpt_pack(xs)):
        if x.numel():
            check_pack(x, ck)
    back = M.ckpt_unpack(M.ckpt_pack(xs))
    assert [b.shape for b in back] == [x.shape for x in xs]
    for shape in ((0, 5), (3, 0), (0,)):
        e = torch.zeros(shape, device="cuda")
        assert M.ckpt_pack(e).unpack().shape == e.shape


def test_nothing_outside_the_buffers_is_written():
    rows, cols = 9, 45
    x = activations((rows, cols), torch.bfloat16)
    q = torch.full((16 + rows * 64 + 16,), 0x55, dtype=torch.uint8).cuda()
    s = torch.full((16 + rows * 2 + 16,), 0x55, dtype=torch.uint8).cuda()
    y = torch.full((rows, 50), 7.0, dtype=torch.bfloat16).cuda()
    e = (x.data_ptr(), y[:, 3:].data_ptr(), q.data_ptr() + 16,
         s.data_ptr() + 16, rows, cols, cols, 50)
    B.mta_ckpt_pack([e], 1, 1)
    torch.cuda.synchronize()
    assert (q[:16] == 0x55).all() and (q[-16:] == 0x55).all()
    assert (s[:16] == 0x55).all() and (s[-16:] == 0x55).all()
    assert (y[:, :3] == 7).all() and (y[:, 3 + cols:] == 7).all()
    oq, osc, _ = R.pack(x)
    assert np.array_equal(q[16:-16].cpu().numpy().reshape(rows, 64), oq)
    assert np.array_equal(s[16:-16].cpu().numpy().reshape(rows, 2), osc)
    assert torch.equal(y[:, 3:3 + cols], x.clamp_min(0))


# Activation values and slopes are float32 expressions of at most a dozen
# operations (each half a step, 2^-24 relative), a 2^x and a reciprocal of the
# hardware's (a step each, 2^-23), whose error in the exponent, |u| 2^-23, is
# weighted with x u' s (1 - s): below 3 for all four.  16 * 2^-23 = 2^-19 of
# (1 + |x|) bounds their sum.  The result is rounded once more.
ACT = 2.0 ** -19


def act_inputs(dtype):
    # to every magnitude that its squares and cubes leave finite, and beyond
    x = torch.cat([torch.linspace(-12, 12, 3001),
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 60.0, -60.0, 100.0,
                                 -100.0, 3e4, -3e4, float("inf"),
                                 -float("inf"), float("nan")])])
    if dtype != torch.float16:
        x = torch.cat([x, torch.tensor([1e13, -1e13, 3e38, -3e38])])
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("act", ACTS)
def test_activation_values(act, dtype):
    dt = R.DTYPES[dtype]
    x = act_inputs(dt)
    y, ck = M.ckpt_act(x, act)
    check_pack(x, ck)
    x64 = R.to64(x)
    want = R.act(x64, act)[0]
    got = R.to64(y)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    bound = R.half_step(dt) * np.abs(want[fine]) + ACT * (
        1 + np.minimum(np.abs(x64[fine]), np.abs(want[fine]) + 1))
    assert (np.abs(got[fine] - want[fine]) <= bound).all()


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("act", ACTS)
def test_activation_backward(act, dtype):
    dt = R.DTYPES[dtype]
    x = act_inputs(dt)
    _, ck = M.ckpt_act(x, act)
    kept = R.to64(ck.unpack(torch.float32))
    dy = torch.randn(x.shape, generator=gen(5)).to(dt).cuda()
    got = R.to64(M.ckpt_act_backward(ck, dy, act))
    want = R.to64(dy) * R.act(kept, act)[1]
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    bound = R.half_step(dt) * np.abs(want) + 2 * ACT * np.abs(R.to64(dy))
    if dt == torch.float16:
        bound = bound + 2.0 ** -25
    assert (np.abs(got - want)[fine] <= bound[fine]).all()


# float32 activations have the digits of a float32.  With steps of 2^-24:
# e^-|u| is off by two, 1 + e, a quotient and a product by one each, so a
# sigmoid by four of itself and 1 - s too, s (1 - s) by nine.  gelu_tanh's u is
# off by six of itself (its constants and three operations), which its
# exponential multiplies with |u|; below 2^-126 an exponential has steps of
# 2^-149.
def test_float32_activations_keep_a_float32s_digits():
    x = torch.cat([torch.linspace(-86, 86, 4001), torch.linspace(-3, 3, 999),
                   torch.tensor([-90.0, -100.0, -104.0, 120.0])]).cuda()
    x64 = R.to64(x)
    u64 = 2 * np.sqrt(2 / np.pi) * (x64 + 0.044715 * x64 ** 3)
    for act, u, steps in (("silu", x64, 0.0), ("gelu_tanh", u64, 6.0)):
        y, ck = M.ckpt_act(x, act)
        with np.errstate(over="ignore"):
            e = np.exp(-np.abs(u))
            s = np.where(u < 0, e, 1.0) / (1 + e)
        err = (steps * np.minimum(np.abs(u), 110) + 8) * 2.0 ** -24
        bound = err * np.abs(x64 * s) + (np.abs(x64) + 1) * 2.0 ** -148
        assert (np.abs(R.to64(y) - x64 * s) <= bound).all(), act
    # the slopes, at values that are kept as they are
    k = torch.tensor([m * 2.0 ** p for p in range(-6, 7) for m in range(8, 16)])
    k = torch.cat([k, -k]).div_(8).reshape(-1, 1).cuda()
    k64 = R.to64(k)[:, 0]
    u64 = 2 * np.sqrt(2 / np.pi) * (k64 + 0.044715 * k64 ** 3)
    du64 = 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * k64 ** 2)
    for act, u, du, steps in (("silu", k64, 1.0, 0.0),
                              ("gelu_tanh", u64, du64, 6.0)):
        ck = M.ckpt_pack(k)
        assert np.array_equal(R.to64(ck.unpack())[:, 0], k64)
        got = R.to64(M.ckpt_act_backward(ck, torch.ones_like(k), act))[:, 0]
        with np.errstate(over="ignore"):
            e = np.exp(-np.abs(u))
        s, t = np.where(u < 0, e, 1.0) / (1 + e), e / (1 + e) ** 2
        err = (2 * steps * np.minimum(np.abs(u), 110) + 16) * 2.0 ** -24
        bound = err * (s + np.abs(k64 * t * du)) + \
            (1 + np.abs(k64 * du)) * 2.0 ** -147
        assert (np.abs(got - (s + k64 * t * du)) <= bound).all(), act


@pytest.mark.parametrize("act", ACTS)
def test_slope_is_the_values_difference(act):
    # away from relu's corner: central differences of the float64 value over
    # h = 2^-13 are off by h^2/6 times the third derivative (below 3)
    x = torch.linspace(-4, 4, 400).cuda() + 0.003
    ck = M.ckpt_pack(x)
    kept = R.to64(ck.unpack())
    h = 2.0 ** -13
    num = (R.act(kept + h, act)[0] - R.act(kept - h, act)[0]) / (2 * h)
    got = R.to64(M.ckpt_act_backward(ck, torch.ones_like(x), act))
    away = np.abs(kept) > h
    assert (np.abs(got - num)[away] <= 2 * ACT + h * h).all()


@pytest.mark.parametrize("shape,pad", [((5, 33), 3), ((130, 96), 0),
                                       ((2, 3, 70), 1), ((1, 1), 0)], ids=str)
@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_activation_shapes_strides_and_mixed_types(shape, pad, dtype):
    dt = R.DTYPES[dtype]
    x = activations(shape, torch.float32, 1, pad)
    y, ck = M.ckpt_act(x, "silu")
    check_pack(x, ck)
    assert y.shape == x.shape
    dy = activations(shape, dt, 2, pad)
    got = R.to64(M.ckpt_act_backward(ck, dy, "silu"))
    want = R.to64(dy) * R.act(R.to64(ck.unpack()), "silu")[1]
    assert (np.abs(got - want) <= R.half_step(dt) * np.abs(want) +
            2 * ACT * np.abs(R.to64(dy)) + 2.0 ** -25).all()


def test_activation_in_place():
    for dt in R.DTYPES.values():
        x = activations((67, 75), dt)
        y, ck = M.ckpt_act(x, "gelu")
        x2 = x.clone()
        ck2 = M.Checkpoint8.empty(x.shape, dt, x.device)
        B.mta_ckpt_pack([(x2.data_ptr(), x2.data_ptr(), ck2.q.data_ptr(),
                          ck2.scale.data_ptr(), 67, 75, 75, 75)], TYPE[dt], 3)
        assert torch.equal(x2, y) and torch.equal(ck2.q, ck.q)
        assert torch.equal(ck2.scale, ck.scale)
        dy = activations((67, 75), dt, 9)
        dx = M.ckpt_act_backward(ck, dy, "gelu")
        B.mta_ckpt_act_backward(
            [(dy.data_ptr(), dy.data_ptr(), ck.q.data_ptr(),
              ck.scale.data_ptr(), 67, 75, 75, 75)], TYPE[dt], 3)
        assert torch.equal(dx, dy)


def test_offsets_past_32_bits():
    # 4.3e9 elements; the last rows are those of a small tensor
    rows, cols = 1_350_000, 3200
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    tail = activations((50, cols), torch.bfloat16)
    x[-50:] = tail
    x[:50] = tail
    y, ck = M.ckpt_act(x, "relu")
    small = M.ckpt_pack(tail)
    for part in (ck.q.view(rows, cols)[-50:], ck.q.view(rows, cols)[:50]):
        assert torch.equal(part.reshape(-1), small.q)
    assert torch.equal(ck.scale.view(rows, -1)[-50:].reshape(-1), small.scale)
    assert torch.equal(y[-50:], tail.clamp_min(0))
    del y
    back = ck.unpack()
    assert torch.equal(back[-50:], small.unpack())
    assert torch.equal(back[rows // 2], torch.ones_like(back[0]))


# --------------------------------------------------------------------------
# weight gradient
# --------------------------------------------------------------------------

def wgrad_case(tokens, fin, fout, dtype, seed=0, pad=0):
    x = activations((tokens, fin), torch.float32, seed)
    ck = M.ckpt_pack(x)
    dy = torch.randn(tokens, fout + pad, generator=gen(seed + 1)).to(
        dtype).cuda()[:, :fout]
    kept = R.to64(ck.unpack()) if tokens and fin else np.zeros((tokens, fin))
    return ck, dy, kept


def check_wgrad(dw, db, dy, kept, old_w=0.0, old_b=0.0):
    """Each of the products' float32 additions is off by half a step of the
    partial sum it makes, and no partial sum passes the sum of magnitudes: at
    most tokens + 64 (parts, waves, the old value) of them, 2^-24 each."""
    d = R.to64(dy)
    n = (d.shape[0] + 64) * 2.0 ** -24
    for got, want, mass in (
            (dw, old_w + d.T @ kept, np.abs(d).T @ np.abs(kept)),
            (db, old_b + d.sum(0), np.abs(d).sum(0))):
        if got is None:
            continue
        mass = mass + np.abs(old_w if got is dw else old_b)
        bound = n * mass + R.half_step(got.dtype) * np.abs(want)
        if got.dtype == torch.float16:
            bound = bound + 2.0 ** -25
        assert (np.abs(R.to64(got) - want) <= bound).all()


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("tokens,fin,fout", [
    (1, 1, 1), (1, 32, 8), (2, 33, 9), (31, 7, 130), (32, 128, 128),
    (33, 129, 127), (64, 257, 16), (100, 40, 300), (257, 96, 40),
    (1000, 130, 260), (4099, 65, 33), (640, 520, 516)])
def test_wgrad_shapes(tokens, fin, fout, dtype):
    ck, dy, kept = wgrad_case(tokens, fin, fout, R.DTYPES[dtype])
    dw, db = M.ckpt_wgrad(ck, dy)
    assert dw.shape == (fout, fin) and dw.dtype == torch.float32
    check_wgrad(dw, db, dy, kept)
    again = M.ckpt_wgrad(ck, dy)
    assert torch.equal(again[0], dw) and torch.equal(again[1], db)


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("tokens,fin,fout", [
    (9001, 520, 260), (20011, 129, 200), (20000, 40, 8), (2051, 1601, 1602),
    (2051, 1600, 1504)])
def test_wgrad_of_many_tokens_and_few_outputs(tokens, fin, fout, dtype):
    """Tiles cut along the tokens, and workgroups whose waves share them."""
    ck, dy, kept = wgrad_case(tokens, fin, fout, R.DTYPES[dtype])
    dw, db = M.ckpt_wgrad(ck, dy)
    check_wgrad(dw, db, dy, kept)
    again = M.ckpt_wgrad(ck, dy)
    assert torch.equal(again[0], dw) and torch.equal(again[1], db)
    old = torch.full_like(dw, 3.0), torch.full_like(db, -2.0)
    M.ckpt_wgrad(ck, dy, out=old[0], out_bias=old[1], accumulate=True)
    assert torch.equal(old[0], dw + 3.0) and torch.equal(old[1], db - 2.0)


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("tokens,fin,fout", [
    (1, 40, 24), (31, 130, 9), (33, 7, 130), (1000, 130, 260), (1024, 768, 640),
    (2051, 1601, 1602), (2051, 1600, 1504), (4099, 65, 33), (8193, 260, 1000),
    (9001, 520, 260), (20000, 40, 8), (20011, 129, 200), (33000, 33, 24)])
def test_wgrad_takes_every_token_once(tokens, fin, fout, dtype):
    """Sums of whole numbers below 2^24, exact in float32 in any order: a token
    that is left out, taken twice or paired with another's dy shows.  x has
    four significant bits, which its checkpoint keeps; dy as many as the sums
    leave room for, so that its second bfloat16 value is there where it can
    be.  x is taken at its size and at 2^-30 of it, where float16 holds none
    of it."""
    most = min(255 if dtype == "bf16" else 511, (1 << 24) // (15 * tokens) - 1)
    x = torch.randint(-15, 16, (tokens, fin), generator=gen(tokens)).float()
    dy = torch.randint(-most, most + 1, (tokens, fout), generator=gen(fin))
    dy = dy.to(R.DTYPES[dtype]).cuda()
    d = dy.double().cpu().numpy()
    want = torch.from_numpy(d.T @ x.double().numpy()).float().cuda()
    bias = torch.from_numpy(d.sum(0)).float().cuda()
    for scale in (1.0, 2.0 ** -30):
        ck = M.ckpt_pack((x * scale).cuda())
        dw, db = M.ckpt_wgrad(ck, dy)
        assert torch.equal(dw, want * scale) and torch.equal(db, bias)
        M.ckpt_wgrad(ck, dy, out=dw, out_bias=db, accumulate=True)
        assert torch.equal(dw, 2 * want * scale) and torch.equal(db, 2 * bias)


@pytest.mark.parametrize("gtype", list(R.DTYPES))
@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("tokens", [70, 3000])
def test_wgrad_accumulates_into_strided_gradients(tokens, dtype, gtype):
    fin, fout, gt = 75, 141, R.DTYPES[gtype]
    ck, dy, kept = wgrad_case(tokens, fin, fout, R.DTYPES[dtype], pad=3)
    wide = (torch.randn(fout, fin + 5, generator=gen(8)) * 50).to(gt).cuda()
    before = wide.clone()
    db = (torch.randn(fout, generator=gen(9)) * 50).to(gt).cuda()
    old_b = R.to64(db)
    got = M.ckpt_wgrad(ck, dy, out=wide[:, 2:2 + fin], out_bias=db,
                       accumulate=True)
    assert got[0].data_ptr() == wide[:, 2:].data_ptr() and got[1] is db
    check_wgrad(wide[:, 2:2 + fin], db, dy, kept,
                R.to64(before[:, 2:2 + fin]), old_b)
    assert torch.equal(wide[:, :2], before[:, :2])
    assert torch.equal(wide[:, 2 + fin:], before[:, 2 + fin:])


def test_wgrad_of_no_tokens_and_no_features():
    ck, dy, _ = wgrad_case(0, 40, 24, torch.bfloat16)
    dw, db = M.ckpt_wgrad(ck, dy)
    assert (dw == 0).all() and (db == 0).all()
    out, ob = torch.ones(24, 40).cuda(), torch.ones(24).cuda()
    M.ckpt_wgrad(ck, dy, out=out, out_bias=ob, accumulate=True)
    assert (out == 1).all() and (ob == 1).all()
    ck, dy, kept = wgrad_case(37, 0, 24, torch.float32)
    dw, db = M.ckpt_wgrad(ck, dy)
    assert dw.shape == (24, 0)
    check_wgrad(None, db, dy, kept)
    ck, dy, kept = wgrad_case(37, 24, 0, torch.float32)
    assert M.ckpt_wgrad(ck, dy)[0].shape == (0, 24)


def test_wgrad_without_bias_and_in_three_dimensions():
    x = activations((3, 50, 96), torch.bfloat16)
    dy = activations((3, 50, 40), torch.bfloat16, 4, pad=8)
    ck = M.ckpt_pack(x)
    dw, db = M.ckpt_wgrad(ck, dy, bias=False, dtype=torch.bfloat16)
    assert db is None and dw.dtype == torch.bfloat16
    check_wgrad(dw, None, dy.reshape(150, 40),
                R.to64(ck.unpack()).reshape(150, 96))


@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_not_finite_gradients_stay_in_their_row(dtype):
    ck, dy, kept = wgrad_case(130, 70, 60, R.DTYPES[dtype])
    dy[5, 7], dy[129, 40], dy[64, 59] = float("inf"), float("nan"), -float(
        "inf")
    dw, db = M.ckpt_wgrad(ck, dy)
    bad = [7, 40, 59]
    ok = [o for o in range(60) if o not in bad]
    assert not torch.isfinite(db[bad]).any()
    # every kept value of these tokens is nonzero, so no product is 0 * inf
    assert not torch.isfinite(dw[bad]).any()
    assert db[7] == float("inf") and db[59] == -float("inf")
    check_wgrad(dw[ok], db[ok], dy[:, ok], kept)


def test_infinite_activations_reach_the_gradient():
    x = activations((64, 96), torch.bfloat16)
    x[10, 33] = float("inf")
    ck = M.ckpt_pack(x)
    dy = activations((64, 16), torch.bfloat16, 2)
    dw, db = M.ckpt_wgrad(ck, dy)
    assert torch.isnan(dw[:, 33]).all() and torch.isfinite(db).all()
    assert torch.isfinite(dw[:, :33]).all() and torch.isfinite(
        dw[:, 34:]).all()


def test_float32_gradients_are_not_rounded_to_16_bits():
    # one token: each result is one product, off by float32 roundings alone
    ck, dy, kept = wgrad_case(1, 64, 64, torch.float32)
    dw, db = M.ckpt_wgrad(ck, dy)
    want = R.to64(dy).T @ kept
    assert (np.abs(R.to64(dw) - want) <= 3 * 2.0 ** -24 * np.abs(want)).all()
    assert torch.equal(db, dy[0])
    # and at both ends of the range
    for s in (1e-30, 1e30):
        dw = M.ckpt_wgrad(ck, dy * s)[0]
        want = R.to64(dy * s).T @ kept
        assert (np.abs(R.to64(dw) - want) <=
                3 * 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.parametrize("dtype,low", [("bf16", -133), ("f16", -24),
                                       ("f32", -149)])
def test_products_are_exact_to_the_ends_of_the_range(dtype, low):
    # one token: a result is one exact product, rounded to float32.  dy runs
    # over its type's powers of two, subnormal ones included, and the kept
    # values over scales of which the smallest is 2^-24 / 2^-9 (the last one
    # exact in float16) and a few beyond float16's range on either side
    dt = R.DTYPES[dtype]
    top = 15 if dtype == "f16" else 127
    dy = torch.tensor([[1.5 * 2.0 ** e for e in range(low + 1, top + 1)] +
                       [2.0 ** low, 0.0, -2.0 ** low]],
                      dtype=torch.float64).to(dt).cuda()
    for ks in (range(-15, 8), (-117, -60, -16, 8, 40), (-117,)):
        x = torch.zeros(1, 32 * len(ks))
        for j, k in enumerate(ks):
            x[0, 32 * j:32 * j + 32] = torch.tensor(
                [448.0 if i == 0 else (1 + i % 8) * 2.0 ** -9 if i < 9 else
                 float(i) for i in range(32)]) * 2.0 ** k
        ck = M.ckpt_pack(x.cuda())
        kept = R.to64(ck.unpack())
        dw, db = M.ckpt_wgrad(ck, dy)
        want = R.to64(dy).T @ kept
        err = np.abs(R.to64(dw) - want)
        fine = np.abs(want) < 2.0 ** 127
        bound = 3 * 2.0 ** -24 * np.abs(want) + 2.0 ** -149
        # a float32's third eight bits fall below 2^-133 from 2^-117 on: the
        # products lose what lies under bfloat16's smallest value
        if dtype == "f32":
            bound = bound + 2.0 ** -133 * np.abs(kept)
        assert (err <= bound)[fine].all(), (ks, err[fine].max())


def test_zero_blocks_do_not_cost_float16_its_products():
    # all-zero blocks (a relu's) beside ordinary ones, and tiny nonzero ones
    x = activations((200, 96), torch.float16, 3)
    x[:, 32:64] = 0
    dy = torch.randn(200, 40, generator=gen(4)).half().cuda()
    for tiny in (0.0, 1e-34):
        y = x.float()
        y[7, 40] = tiny
        ck = M.ckpt_pack(y)
        dw, db = M.ckpt_wgrad(ck, dy)
        check_wgrad(dw, db, dy, R.to64(ck.unpack()))


def takes_float16_products(ck, dy):
    """Whether a float16 dy's product found every kept value exact in float16:
    the answers stand at the end of the workspace."""
    tokens, fin, fout = ck.rows, ck.shape[-1], dy.shape[1]
    need = B.mta_ckpt_wgrad_workspace(tokens, fin, fout, 2)
    ws = torch.full((need,), 255, dtype=torch.uint8).cuda()
    dw = torch.empty(fout, fin).cuda()
    B.mta_ckpt_wgrad(B.mta_ckpt_wgrad_args(
        *ck.pointers(), dy.data_ptr(), dw.data_ptr(), None, ws.data_ptr(),
        need, tokens, fin, fout, fout, fin, 2, 0, 0, 0))
    n = min(-(-tokens * ck.blocks // 1024), 256)
    flags = ws[need - -(-4 * n // 16) * 16:][:4 * n].view(torch.int32).tolist()
    assert set(flags) <= {0, 1}
    check_wgrad(dw, None, dy, R.to64(ck.unpack(torch.float32)))
    return all(flags)


@pytest.mark.parametrize("fin", [1, 33, 768, 769, 1601])
def test_kept_float16_values_are_exact_in_float16(fin):
    dy = torch.randn(2047, 40, generator=gen(4)).half().cuda()
    for scale in (1.0, 1e-3, 1e-5, 3e-7, 3e4):
        x = torch.randn(2047, fin, generator=gen(fin)) * scale
        x.clamp_(-65504, 65504)
        x[::3] = 0.0
        ck = M.ckpt_pack(x.half().cuda())
        assert takes_float16_products(ck, dy), scale
    # one value of another type that float16 does not hold
    for tiny in (2.0 ** -25, 65536.0, 1.5 * 2.0 ** -24):
        y = torch.randn(2047, fin, generator=gen(fin))
        y[1023, fin - 1] = 0.0
        ck = M.ckpt_pack(y.half().float().cuda())
        assert takes_float16_products(ck, dy)
        y[1023, max(0, fin - 32):] = 0.0
        y[1023, fin - 1] = tiny
        ck = M.ckpt_pack(y.cuda())
        assert not takes_float16_products(ck, dy), tiny


def test_float16_products_at_every_scale_are_exact():
    # one token; blocks of scale 2^k with four-bit values that float16 holds,
    # most of them subnormal there, against every magnitude of dy
    dy = torch.tensor([[1.5 * 2.0 ** e for e in range(-23, 16)] +
                       [2.0 ** -24, 0.0, 2.0 ** -14 - 2.0 ** -24]],
                      dtype=torch.float64).half().cuda()
    ks = range(-32, -8)
    x = torch.zeros(1, 32 * len(ks))
    for j, k in enumerate(ks):
        v = [f * 2.0 ** (k + 8 - i) for f in (1.75, 1.125) for i in range(16)]
        x[0, 32 * j:32 * j + 32] = torch.tensor(
            [y if y * 2.0 ** 24 % 1 == 0 else 0.0 for y in v])
    ck = M.ckpt_pack(x.cuda())
    kept = R.to64(ck.unpack())
    assert (kept * 2.0 ** 24 % 1 == 0).all() and (kept[0, 32:] != 0).any()
    assert takes_float16_products(ck, dy)
    dw, _ = M.ckpt_wgrad(ck, dy, bias=False)
    # each result is one product of 4 and 11 significant bits, not below
    # float32's smallest normal: exact
    assert np.array_equal(R.to64(dw), R.to64(dy).T @ kept)


def test_wgrad_offsets_past_32_bits():
    # rows of dy 131,072 apart: the last start past 2^32 elements
    tokens, fin, fout, ld = 33000, 33, 24, 131072
    base = torch.zeros(tokens, ld, dtype=torch.bfloat16, device="cuda")
    ck, dy, kept = wgrad_case(tokens, fin, fout, torch.bfloat16)
    base[:, -fout:] = dy
    got = M.ckpt_wgrad(ck, base[:, -fout:])
    want = M.ckpt_wgrad(ck, dy)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_wgrad(got[0], got[1], dy, kept)


def test_refusals_of_tensors():
    ck, dy, _ = wgrad_case(10, 40, 24, torch.bfloat16)
    cases = [
        lambda: M.ckpt_wgrad(ck, dy[:5]),
        lambda: M.ckpt_wgrad(ck, dy.t()),
        lambda: M.ckpt_wgrad(ck, dy.cpu()),
        lambda: M.ckpt_wgrad(ck, dy, accumulate=True),
        lambda: M.ckpt_wgrad(ck, dy, out=torch.zeros(40, 24).cuda()),
        lambda: M.ckpt_wgrad(ck, dy, out=torch.zeros(24, 40).cuda(),
                             out_bias=torch.zeros(24).cuda().half()),
        lambda: M.ckpt_wgrad(ck, dy, bias=False,
                             out_bias=torch.zeros(24).cuda()),
        lambda: M.ckpt_act_backward(ck, dy, "relu"),
        lambda: M.Checkpoint8(ck.q, ck.scale, (11, 40)),
        lambda: M.Checkpoint8(ck.q, ck.scale.cpu(), (10, 40)),
    ]
    for c in cases:
        with pytest.raises(ValueError):
            c()
    for c in (lambda: M.ckpt_wgrad(ck, dy.double()),
              lambda: M.ckpt_wgrad(ck, dy, dtype=torch.float64),
              lambda: M.ckpt_pack([dy, dy.float()]),
              lambda: ck.unpack(torch.float64)):
        with pytest.raises(TypeError):
            c()
    # a workspace that is too small is refused by the library
    big = M.ckpt_pack(torch.zeros(4096, 32).cuda())
    need = B.mta_ckpt_wgrad_workspace(4096, 32, 24, 0)
    assert need > 0
    g = torch.zeros(4096, 24).cuda()
    w, ws = torch.zeros(24, 32).cuda(), torch.zeros(need).byte().cuda()
    with pytest.raises(M.MtaError):
        B.mta_ckpt_wgrad(B.mta_ckpt_wgrad_args(
            big.q.data_ptr(), big.scale.data_ptr(), g.data_ptr(),
            w.data_ptr(), None, ws.data_ptr(), need - 1, 4096, 32, 24, 24, 32,
            0, 0, 0, 0))


# --------------------------------------------------------------------------
# streams, graphs, autograd
# --------------------------------------------------------------------------

def test_a_side_stream_orders_its_own_work():
    x = activations((4000, 800), torch.bfloat16)
    want = M.ckpt_pack(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y = torch.zeros_like(x)
        for _ in range(20):          # the pack has to wait for the last add
            y += 0
        y += x
        got = M.ckpt_pack(y)
        dw, _ = M.ckpt_wgrad(got, y)
    s.synchronize()
    assert torch.equal(got.q, want.q) and torch.equal(got.scale, want.scale)
    assert torch.equal(dw, M.ckpt_wgrad(want, x)[0])


def test_captured_calls_replay_on_new_inputs():
    def work(x, dy, g):
        y, ck = M.ckpt_act(x, "gelu_tanh")
        dx = M.ckpt_act_backward(ck, dy, "gelu_tanh")
        M.ckpt_wgrad(ck, dy, bias=False, out=g, accumulate=True)
        return y, dx

    x, dy = (activations((3000, 96), torch.bfloat16, s) for s in (1, 2))
    g1, g2 = torch.zeros(96, 96).cuda(), torch.zeros(96, 96).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work(x, dy, g1.clone())
    torch.cuda.current_stream().wait_stream(s)
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dx = work(x, dy, g1)
    with torch.cuda.graph(other):       # a second graph with its own buffers
        y2, dx2 = work(x, dy, g2)
    g1.zero_()
    g2.zero_()
    want = torch.zeros_like(g1)
    for seed in range(4):
        x.copy_(activations((3000, 96), torch.bfloat16, 10 + seed))
        dy.copy_(activations((3000, 96), torch.bfloat16, 20 + seed))
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        ey, edx = work(x, dy, want)
        for a, b in ((y, ey), (dx, edx), (y2, ey), (dx2, edx), (g1, want),
                     (g2, want)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("wdtype", list(R.DTYPES))
def test_checkpointed_layers_have_the_formulas_gradients(wdtype):
    wt = R.DTYPES[wdtype]
    x = activations((6, 20, 64), torch.bfloat16).requires_grad_()
    w = (torch.randn(48, 64, generator=gen(3)) * 0.1).to(wt).cuda()
    b = torch.randn(48, generator=gen(4)).to(wt).cuda()
    w.requires_grad_(), b.requires_grad_()
    h = M.checkpointed_linear(x, w, b)
    a = M.checkpointed_act(h, "silu")
    da = torch.randn(a.shape, generator=gen(6)).bfloat16().cuda()
    a.backward(da)
    assert w.grad.dtype == wt and b.grad.dtype == wt
    kx = R.to64(M.ckpt_pack(x.detach()).unpack()).reshape(120, 64)
    kh = R.to64(M.ckpt_pack(h.detach()).unpack()).reshape(120, 48)
    dh = R.to64(da).reshape(120, 48) * R.act(kh, "silu")[1]
    # dh is rounded to bfloat16 on its way, half a step 2^-9 relative and
    # the activation's own bound; so its sums are off by that of their mass
    err = np.abs(dh) * 2.0 ** -8 + 2 * ACT * np.abs(R.to64(da).reshape(
        120, 48))
    n = 184 * 2.0 ** -24
    want = dh.T @ kx
    mass = np.abs(dh).T @ np.abs(kx)
    bound = err.T @ np.abs(kx) + n * mass + 2.0 * R.half_step(wt) * np.abs(
        want)
    assert (np.abs(R.to64(w.grad) - want) <= bound).all()
    bound = err.sum(0) + n * np.abs(dh).sum(0) + 2 * R.half_step(
        wt) * np.abs(dh.sum(0))
    assert (np.abs(R.to64(b.grad) - dh.sum(0)) <= bound).all()
    # x's gradient is the plain product of the rounded dh
    assert x.grad.shape == x.shape and torch.isfinite(x.grad).all()
    # expanded gradients (of a sum) are taken
    x2 = x.detach().requires_grad_()
    M.checkpointed_act(M.checkpointed_linear(x2, w, b), "relu").sum().backward()
    assert torch.isfinite(x2.grad).all()


@pytest.mark.parametrize("wdtype", list(R.DTYPES))
@pytest.mark.parametrize("xdtype", list(R.DTYPES))
def test_a_layers_input_gradient_is_the_product(xdtype, wdtype):
    xt, wt = R.DTYPES[xdtype], R.DTYPES[wdtype]
    x = activations((6, 20, 64), xt).requires_grad_()
    w = (torch.randn(48, 64, generator=gen(3)) * 0.1).to(wt).cuda()
    dy = torch.randn(6, 20, 48, generator=gen(4)).to(xt).cuda()
    y = M.checkpointed_linear(x, w.requires_grad_())
    y.backward(dy)
    w64, d64 = R.to64(w.detach().to(xt)), R.to64(dy)
    # 48 products, each addition off by half a step of the magnitudes' sum,
    # rounded once
    want, mass = d64 @ w64, np.abs(d64) @ np.abs(w64)
    bound = R.half_step(xt) * np.abs(want) + 50 * 2.0 ** -24 * mass
    if xt == torch.float16:
        bound = bound + 2.0 ** -25
    assert x.grad.dtype == xt
    assert (np.abs(R.to64(x.grad) - want) <= bound).all()


def test_layers_take_any_strides_and_parameter_types():
    x = activations((12, 40, 32), torch.bfloat16).transpose(0, 1)
    x.requires_grad_()
    w = torch.randn(8, 32, generator=gen(1)).bfloat16().cuda()
    b = torch.zeros(8, device="cuda")
    w.requires_grad_(), b.requires_grad_()
    y = M.checkpointed_act(M.checkpointed_linear(x, w, b).transpose(0, 1),
                           "gelu")
    assert y.shape == (12, 40, 8)
    y.sum().backward()
    assert x.grad.shape == x.shape and w.grad.dtype == torch.bfloat16
    assert b.grad.dtype == torch.float32
    # the same from contiguous tensors
    x2 = x.detach().contiguous().requires_grad_()
    w2, b2 = w.detach().clone().requires_grad_(), b.detach().clone()
    b2.requires_grad_()
    M.checkpointed_act(M.checkpointed_linear(x2, w2, b2), "gelu").sum(
    ).backward()
    # (the order of tokens in the sums is the same)
    assert torch.equal(w2.grad, w.grad) and torch.equal(b2.grad, b.grad)


def test_layers_skip_what_needs_no_gradient():
    x = activations((5, 32), torch.float32)
    w = torch.randn(8, 32).cuda()
    y = M.checkpointed_linear(x.requires_grad_(), w)
    y.sum().backward()
    assert torch.equal(x.grad, w.sum(0).expand(5, 32)) or torch.allclose(
        x.grad, w.sum(0).expand(5, 32), atol=32 * 2.0 ** -23)
    b = torch.zeros(8, device="cuda", requires_grad=True)
    M.checkpointed_linear(x.detach(), w, b).sum().backward()
    assert torch.equal(b.grad, torch.full((8,), 5.0).cuda())


def test_layers_without_gradients():
    x = activations((70, 512), torch.bfloat16)
    w = torch.nn.Parameter(torch.randn(96, 512).cuda())
    b = torch.nn.Parameter(torch.randn(96).cuda())
    want = M.checkpointed_linear(x, w, b)
    with torch.no_grad():
        y = M.checkpointed_linear(x, w, b)
        a = M.checkpointed_act(y, "gelu")
    assert want.requires_grad and not y.requires_grad and not a.requires_grad
    assert torch.equal(y, want)
    assert torch.equal(a, M.checkpointed_act(want, "gelu"))
    with torch.inference_mode():
        assert torch.equal(M.checkpointed_linear(x, w, b), want)
        assert torch.equal(M.checkpointed_act(y, "gelu"), a)


def test_a_backward_frees_the_checkpoints():
    # a saved tensor is freed by the backward that uses it (a second one then
    # refuses), and passes the hooks.  (The allocator's count right after a
    # backward says less: the gradients just dropped, 65536 + 98304 bytes of
    # this linear layer, may still be held by autograd's own thread.)
    x = activations((64, 512), torch.bfloat16).requires_grad_()
    w = torch.nn.Parameter(torch.randn(96, 512).bfloat16().cuda())
    sizes = []

    def pack(t):
        sizes.append((t.dtype, t.numel()))
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        act = M.checkpointed_act(x, "relu")
        lin = M.checkpointed_linear(x, w)
    kept = (torch.uint8, 64 * 512 * 33 // 32)
    assert sizes.count(kept) == 2
    assert all(s in (kept, (torch.bfloat16, 96 * 512)) for s in sizes)
    for y, inputs in ((act, [x]), (lin, [x, w])):
        want = torch.autograd.grad(y, inputs, torch.ones_like(y),
                                   retain_graph=True)
        got = torch.autograd.grad(y, inputs, torch.ones_like(y))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        with pytest.raises(RuntimeError, match="second time"):
            torch.autograd.grad(y, inputs, torch.ones_like(y))


def test_captured_layers_train_as_eager_ones():
    """Forward and backward of both layers in one graph, the gradients in the
    buffers that capture made, against eager passes after each replay."""
    def grads(x, dy, w1, b1, w2):
        y = M.checkpointed_linear(M.checkpointed_act(
            M.checkpointed_linear(x, w1, b1), "gelu"), w2)
        return torch.autograd.grad(y, [x, w1, b1, w2], dy)

    def leaves(seed):
        r = [(torch.randn(*s, generator=gen(seed + k)) * 0.2).bfloat16().cuda()
             for k, s in enumerate(((256, 128), (64, 128), (64,), (96, 64)))]
        return [t.requires_grad_() for t in r]

    p = leaves(1)
    dy = torch.randn(256, 96, generator=gen(9)).bfloat16().cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        grads(p[0], dy, *p[1:])
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = grads(p[0], dy, *p[1:])
    for seed in range(4):
        q = leaves(20 + 10 * seed)
        with torch.no_grad():
            for a, b in zip(p, q):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, grads(q[0], dy, *q[1:])):
            assert torch.equal(a, b)
