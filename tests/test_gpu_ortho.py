"""Orthogonalised updates on the GPU against their float64 definition."""
import pytest
import torch

import matrix_oracle as R
import mixed_precision_optimizer_mta_amd as M
from mixed_precision_optimizer_mta_amd import _binding as B

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def matrix(rows, cols, dtype, seed=0, pad=0, size=1e-3):
    """Normal entries, two directions that stand out, rows of cols + pad."""
    g = gen(seed)
    x = torch.randn(rows, cols + pad, generator=g)
    x += torch.randn(rows, 2, generator=g) @ torch.randn(
        2, cols + pad, generator=g)
    return (x * size).to(R.DTYPES[dtype])[:, :cols]


def on_gpu(x):
    """The same matrix with the same pitch on the GPU."""
    y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    return y.copy_(x)


def allowed(x, planes, out):
    """What the documented roundings come to, by carrying them out, a quarter
    more for the others that float32 sums bring about, and the result's own.
    Float32 sums: three additions for every sixteen values of k in each of
    three products of five steps, half a step each, errors of either sign (the
    root of their number), times the 30 that a step's error grows by at the
    smallest singular values here."""
    want = R.orthogonal(x)
    k = 3 * (max(x.shape) // 16 + 3)
    sums = 15 * k ** 0.5 * 2.0 ** -24 * 30
    return want, 1.25 * R.off(R.orthogonal_rounded(x, planes), want) + \
        R.half_step(out) + sums


SHAPES = [(1, 1), (1, 9), (9, 1), (2, 3), (16, 16), (3, 130), (65, 64),
          (129, 257), (300, 77), (128, 512), (255, 256)]


@pytest.mark.parametrize("dtype", list(R.DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_orthogonalize(rows, cols, dtype):
    x = matrix(rows, cols, dtype, rows * 1000 + cols, pad=3)
    y = M.orthogonalize(on_gpu(x))
    assert y.dtype == x.dtype and y.shape == x.shape
    want, most = allowed(x, 1 if dtype == "bf16" else 2, x.dtype)
    assert R.off(y, want) <= most


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("out", list(R.DTYPES))
@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_types_and_precision(dtype, out, precise):
    x = matrix(70, 200, dtype, 5)
    y = M.orthogonalize(on_gpu(x), dtype=R.DTYPES[out], precise=precise)
    assert y.dtype == R.DTYPES[out]
    want, most = allowed(x, 2 if precise else 1, y.dtype)
    assert R.off(y, want) <= most


def test_a_list_is_each_alone_and_a_transpose_is_the_transpose():
    shapes = [(40, 300), (300, 40), (16, 16), (129, 129), (1, 50), (0, 7),
              (7, 0), (256, 300)] + [(33, 65)] * 45
    xs = [matrix(r, c, "bf16", i).cuda() for i, (r, c) in enumerate(shapes)]
    ys = M.orthogonalize(xs)
    for x, y in zip(xs, ys):
        assert y.shape == x.shape
        assert torch.equal(M.orthogonalize(x), y)
        if x.shape[0] != x.shape[1]:           # (a square one is not turned)
            assert torch.equal(M.orthogonalize(x.t().contiguous()).t(), y)
    assert M.orthogonalize([]) == []


def test_many_tiles():
    """Lists whose products take the large tile, and mixed ones."""
    for shapes in ([(1600, 1600)] * 9, [(768, 2304)] * 9 + [(2304, 768)],
                   [(1601, 4000)] * 5 + [(777, 1333)] * 3 + [(64, 64)]):
        xs = [on_gpu(matrix(r, c, "bf16", i))
              for i, (r, c) in enumerate(shapes)]
        for x, y in zip(xs, M.orthogonalize(xs)):
            # 1.1e-3 as documented, and the result's rounding
            assert R.off(y, R.orthogonal(x)) <= 1.1e-3 + 2.0 ** -8


def test_scale_steps_coefficients_and_eps():
    x = matrix(50, 90, "f32", 3)
    g = on_gpu(x)
    one = M.orthogonalize(g)
    assert torch.equal(M.orthogonalize(g, scale=-0.5), one * -0.5)
    assert [torch.equal(y, s * one) for y, s in zip(
        M.orthogonalize([g, g], scale=[2, 4]), (2, 4))] == [True, True]
    per = [(1.875, -1.25, 0.375)] * 3 + [(1.5, -0.5, 0.0)] * 9
    y = M.orthogonalize(g, steps=12, coefficients=per)
    assert R.off(y, R.orthogonal(x, per)) <= 1e-5
    # twelve such steps end at singular values of 1
    assert R.off(y @ y.t(), torch.eye(50)) <= 1e-4
    assert R.off(M.orthogonalize(g, steps=1),
                 R.orthogonal(x, steps=1)) <= 1e-5
    assert R.off(M.orthogonalize(g, eps=1.0, steps=2),
                 R.orthogonal(x, eps=1.0, steps=2)) <= 1e-5
    z = torch.zeros(20, 30, device="cuda")
    assert not M.orthogonalize(z).any()
    assert not M.orthogonalize(z, eps=0.0).any()


@pytest.mark.parametrize("size", [1e-30, 1e30])
def test_sizes_beyond_float16(size):
    x = matrix(40, 60, "f32", 4, size=size)
    assert R.off(M.orthogonalize(on_gpu(x), eps=0.0),
                 R.orthogonal(x, eps=0.0)) <= 1e-5


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_matrix(bad):
    xs = [matrix(60, 90, "bf16", i).cuda() for i in range(3)]
    alone = M.orthogonalize(xs[0])
    xs[1][7, 11] = bad
    ys = M.orthogonalize(xs)
    assert torch.equal(ys[0], alone)
    assert ys[1].isnan().all()
    assert ys[2].isfinite().all()


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype", list(R.DTYPES))
def test_muon_update(dtype, nesterov):
    shapes = [(70, 200), (200, 70), (5, 1001)]
    gs = [matrix(r, c, dtype, i, pad=i) for i, (r, c) in enumerate(shapes)]
    ms = [matrix(r, c, "f32", 10 + i) for i, (r, c) in enumerate(shapes)]
    dg, dm = [on_gpu(g) for g in gs], [m.cuda() for m in ms]
    ys = M.muon_update(dg, dm, momentum=0.9, nesterov=nesterov)
    mu = torch.tensor(0.9, dtype=torch.float32)
    for g, m, y, new in zip(gs, ms, ys, dm):
        m = m * mu + g.float()                 # each operation rounded once
        assert torch.equal(new.cpu(), m)
        u = g.float() + mu * m if nesterov else m
        want, most = allowed(u, 1 if dtype == "bf16" else 2, g.dtype)
        assert y.dtype == g.dtype and R.off(y, want) <= most


def test_out_and_its_neighbours():
    x = matrix(37, 51, "bf16", 1).cuda()
    want = M.orthogonalize(x)
    wide = torch.full((39, 60), 7.0, dtype=torch.bfloat16, device="cuda")
    M.orthogonalize([x], out=[wide[1:38, 4:55]])
    assert torch.equal(wide[1:38, 4:55], want)
    wide[1:38, 4:55] = 7.0
    assert (wide == 7.0).all()
    flat = torch.full((51 * 37 + 2,), 7.0, device="cuda")
    out = flat[1:-1].view(51, 37)              # off 16 bytes, another type
    M.orthogonalize(x.t().contiguous(), out=out, precise=False)
    assert R.off(out.t(), want) <= 2.0 ** -8
    assert flat[0] == 7.0 and flat[-1] == 7.0


def test_out_counts_as_written():
    x = matrix(8, 8, "f32").cuda().requires_grad_()
    y = x * 1.0
    z = y * y
    M.orthogonalize(x.detach(), out=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        z.sum().backward()


def test_streams_and_graph():
    xs = [matrix(100, 200, "bf16", i).cuda() for i in range(3)]
    ms = [torch.zeros(100, 200, device="cuda") for _ in xs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = M.orthogonalize(xs)
    s.synchronize()
    for x, y in zip(xs, got):
        assert torch.equal(y, M.orthogonalize(x))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = M.muon_update(xs, ms)
        again = M.orthogonalize(xs[0])
    eager = [torch.zeros_like(m) for m in ms]
    for m in ms:
        m.zero_()
    for seed in range(4):
        for i, x in enumerate(xs):
            x.copy_(matrix(100, 200, "bf16", 10 * seed + i))
        graph.replay()
        torch.cuda.synchronize()
        want = M.muon_update(xs, eager)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(ms, eager))
        assert torch.equal(again, M.orthogonalize(xs[0]))


def test_clip_coefficient_loss_scale_and_weights():
    """The C entry's other inputs: a clip coefficient and a loss-scale state
    in device memory, and weights that take the step with their copy."""
    g = matrix(60, 100, "f16", 1)
    m0, w0 = matrix(60, 100, "f32", 2), matrix(60, 100, "f32", 3, size=0.02)
    coef = torch.tensor([0.25], device="cuda")
    for found in (0.0, 1.0):
        amp = M.AmpState(8.0)
        amp.write(8.0, 3, 0, found)
        m, w = m0.cuda(), w0.cuda()
        w16 = torch.full((60, 100), 9.0, dtype=torch.bfloat16, device="cuda")
        dg = on_gpu(g)
        from mixed_precision_optimizer_mta_amd import muon
        muon.run(muon.table([(dg.data_ptr(), m.data_ptr(), None, w.data_ptr(),
                              w16.data_ptr(), 60, 100, 100, 0, 0.5)]),
                 dg.device, B.MTA_F16, B.MTA_F32, B.MTA_BF16,
                 muon._coefficients(muon.COEFFICIENTS, 5), 1e-7, 0.95, True,
                 True, lr=0.02, weight_decay=0.1, coef=coef.data_ptr(),
                 amp=amp.ptr)
        if found:
            assert torch.equal(m.cpu(), m0) and torch.equal(w.cpu(), w0)
            assert (w16 == 9.0).all()
            continue
        ge = (g.float() * 0.125) * 0.25
        mu = torch.tensor(0.95)
        mn = m0 * mu + ge
        assert torch.equal(m.cpu(), mn)
        x = R.orthogonal(ge + mu * mn)
        want = w0.double() * (1 - 0.02 * 0.1) - 0.02 * 0.5 * x
        # roundings of w * decay and of the sum, and 1e-5 of the step
        most = 2.0 ** -23 + 1e-5 * (0.01 * x.norm() / want.norm()).item()
        assert R.off(w, want) <= most
        assert torch.equal(w16, w.bfloat16())
