"""GPU tests of the orthogonalised update against tests/block8_reference.py (fp64 products).

The bound of a result's error is that of block8_reference.orthogonalise (roundings to 11 bits in every step, carried on
by the steps behind them), plus the rounding of the result.  It is for the worst case, in which every rounding points the
same way; matrices whose result is known in closed form are held to much less.
"""
import numpy as np
import pytest
import torch

import block8_reference as ref
import token_dispatch_grouped_top_amd as mok

pytestmark = pytest.mark.gpu
COEF = mok.NEWTON_SCHULZ
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def workspace(n, rows, cols, fill=0xff):
    return torch.full((mok.mok_muon_workspace_size(n, rows, cols),), fill, dtype=torch.uint8, device="cuda")


def gradients(rng, n, rows, cols, size=1e-3):
    few = rng.normal(size=(n, rows, 2)) @ rng.normal(size=(n, 2, cols))
    return ((rng.normal(size=(n, rows, cols)) + few) * size).astype(np.float32)


def orth(x, dtype=torch.float32, steps=5, coef=COEF):
    n, rows, cols = x.shape
    out = torch.full((n * rows * cols + 8,), -7.0, dtype=torch.bfloat16, device="cuda")
    mok.mok_orthogonalise(dev(x, dtype), n, rows, cols, out, workspace(n, rows, cols), steps=steps, coefficients=coef)
    assert (host(out)[n * rows * cols:] == -7).all()
    return host(out)[:n * rows * cols].reshape(x.shape)


SIZES = [(1, 1, 1), (2, 1, 7), (3, 5, 1), (1, 64, 64), (2, 65, 130), (3, 130, 65), (1, 200, 333), (2, 300, 190),
         (1, 64, 1000), (1, 1000, 63), (5, 128, 128)]


@pytest.mark.parametrize("n,rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("steps", [1, 2, 5])
def test_orthogonalise(n, rows, cols, dtype, steps):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = dev(gradients(rng, n, rows, cols), dtype).float().cpu().numpy()
    got = orth(x, dtype, steps)
    for i in range(n):
        want, e = ref.orthogonalise(x[i], COEF, steps)
        assert np.linalg.norm(got[i] - want) <= e + 2.0 ** -8 * np.linalg.norm(want)
        # roundings point every way: what is left of them is a small part of the bound, of the size of bf16's own
        assert np.linalg.norm(got[i] - want) <= 2.0 ** -7 * np.linalg.norm(want)


@pytest.mark.parametrize("n,rows,cols", [(70, 256, 256), (2, 2048, 2112), (130, 200, 264)])
def test_orthogonalise_large_tiles(n, rows, cols):
    """Sizes that take the large tiles, against torch's fp64 products on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, rows, cols, generator=gen, device="cuda")
    out = torch.empty(n, rows, cols, dtype=torch.bfloat16, device="cuda")
    mok.mok_orthogonalise(x, n, rows, cols, out, workspace(n, rows, cols))
    a, b, c = COEF
    for i in range(0, n, max(1, n // 8)):
        y = x[i].double() / x[i].double().norm()
        for _ in range(5):
            g = y @ y.T.contiguous()
            y = a * y + (b * g + c * g @ g) @ y
        assert (out[i].double() - y).norm() <= 2.0 ** -7 * y.norm()


@pytest.mark.parametrize("rows,cols", [(48, 100), (100, 48), (256, 512)])
def test_equal_singular_values(rows, cols):
    """U V^T with all singular values equal to s: every step is the scalar polynomial p(s) = s (a + b g + c g^2), g = s^2,
    and so is what roundings to 11 bits (u) make of it, if they are the same for all of X, of G and of B: |p'(s)| times
    the error that X has, u g |b + 2 c g| s from G, u |b g + c g^2| s from B, u |p(s)| from the new X."""
    rng = np.random.default_rng(rows)
    k = min(rows, cols)
    q = np.linalg.qr(rng.normal(size=(rows, k)))[0] @ np.linalg.qr(rng.normal(size=(cols, k)))[0].T
    got = orth((q * 3.7)[None].astype(np.float32))[0]
    a, b, c = COEF
    s, u = k ** -0.5, 2.0 ** -11
    e = u * s
    for _ in range(5):
        e = abs(a + 3 * b * s ** 2 + 5 * c * s ** 4) * e + \
            u * s ** 3 * (abs(b + 2 * c * s * s) + abs(b + c * s * s))
        s = s * (a + s * s * (b + s * s * c))
        e += u * abs(s)
    assert np.linalg.norm(got - s * q) <= (e / abs(s) + 2.0 ** -8) * np.linalg.norm(s * q)
    # the diagonals' rounding is kept, and with it nearly all of that
    assert np.linalg.norm(got - s * q) <= 2.0 ** -8 * np.linalg.norm(s * q)


def test_special_matrices():
    """Zero stays zero, values that are not finite spoil their own matrix alone, and the size of the input does not
    matter, up to where its norm passes fp32's range."""
    rng = np.random.default_rng(0)
    x = gradients(rng, 6, 40, 70, 1.0)
    x[0] = 0
    x[1, 3, 4], x[2, 0, 0] = np.inf, np.nan
    x[3] *= np.float32(3e38) / np.abs(x[3]).max()
    x[4] = x[5] * np.float32(2.0 ** -100)
    got = orth(x)
    assert not got[0].any() and np.isnan(got[1]).all() and np.isnan(got[2]).all()
    assert np.array_equal(got[4], got[5])
    want = ref.orthogonalise(x[3], COEF, 5)[0]
    assert np.linalg.norm(got[3] - want) <= 2.0 ** -7 * np.linalg.norm(want)


def test_other_coefficients():
    rng = np.random.default_rng(1)
    x = gradients(rng, 1, 96, 160)
    coef = (1.875, -1.25, 0.375)
    got = orth(x, steps=16, coef=coef)[0]
    want, _ = ref.orthogonalise(x[0], coef, 16)
    assert np.linalg.norm(got - want) <= 2.0 ** -7 * np.linalg.norm(want)
    assert np.allclose(got @ got.T, np.eye(96), atol=0.02)


HYPER = dict(lr=2e-3, momentum=0.9, weight_decay=0.1, grad_scale=0.5, scale=3.0)


@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (2, 65, 130), (3, 130, 65), (1, 300, 190), (40, 256, 300)])
@pytest.mark.parametrize("grads", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("nesterov", [0, 1])
@pytest.mark.parametrize("copy", [False, True])
def test_muon_step(n, rows, cols, grads, nesterov, copy):
    rng = np.random.default_rng(rows + cols)
    g = dev(gradients(rng, n, rows, cols), grads)
    p0, m0 = rng.normal(size=(n, rows, cols)).astype(np.float32), gradients(rng, n, rows, cols, 1e-2)
    p, m = dev(p0), dev(m0)
    pb = torch.zeros(n, rows, cols, dtype=torch.bfloat16, device="cuda") if copy else None
    mok.mok_muon_step(p, g, m, n, rows, cols, workspace(n, rows, cols), nesterov=nesterov, p_bf16=pb, **HYPER)
    g64 = host(g) * HYPER["grad_scale"]
    m64 = HYPER["momentum"] * m0.astype(np.float64) + g64
    # momentum is rounded to fp32, g and the fused sum once each
    tol = U * (2 * np.abs(g64) + 2 * HYPER["momentum"] * np.abs(m0)) + U * np.abs(m64) + 1e-44
    assert np.all(np.abs(host(m) - m64) <= tol)
    v = g64 + HYPER["momentum"] * m64 if nesterov else m64
    h = HYPER
    for i in range(0, n, max(1, n // 4)):
        x, _ = ref.orthogonalise(v[i], COEF, 5)
        want = p0[i] * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * h["scale"] * x
        # three roundings of p, and the update's error as test_orthogonalise has it (its own result is not rounded)
        size = 4 * U * np.linalg.norm(p0[i]) + h["lr"] * h["scale"] * 2.0 ** -7 * np.linalg.norm(x)
        assert np.linalg.norm(host(p[i]) - want) <= size
    if copy:
        assert torch.equal(pb, p.bfloat16())


@pytest.mark.parametrize("n,rows,cols", [(12, 2040, 2176), (11, 2303, 2040)])
def test_largest_tiles(n, rows, cols):
    """Enough of the largest tiles for the chip in every product; the step and the update alone, against torch's fp64
    products on the GPU, with the tolerances of test_muon_step and test_orthogonalise."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    normal = lambda: torch.randn(n, rows, cols, generator=gen, device="cuda")  # noqa: E731
    g, p0, m0 = normal(), normal(), normal()
    p, m, pb = p0.clone(), m0.clone(), torch.zeros(n, rows, cols, dtype=torch.bfloat16, device="cuda")
    ws = workspace(n, rows, cols)
    mok.mok_muon_step(p, g, m, n, rows, cols, ws, nesterov=0, p_bf16=pb, **HYPER)
    out = torch.empty_like(pb)
    mok.mok_orthogonalise(m, n, rows, cols, out, ws)
    a, b, c = COEF
    h = HYPER
    assert torch.equal(pb, p.bfloat16())
    for i in range(n):
        v = m[i].double()
        assert (v - (h["momentum"] * m0[i].double() + h["grad_scale"] * g[i].double())).abs().max() <= 4 * U * 8
        y = v / v.norm()
        for _ in range(5):
            gram = y @ y.T.contiguous()
            y = a * y + (b * gram + c * gram @ gram) @ y
        assert (out[i].double() - y).norm() <= 2.0 ** -7 * y.norm()
        want = p0[i].double() * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * h["scale"] * y
        size = 4 * U * p0[i].double().norm() + h["lr"] * h["scale"] * 2.0 ** -7 * y.norm()
        assert (p[i].double() - want).norm() <= size


def test_muon_scalars():
    """lr and grad_scale from the device, and a step that is skipped."""
    rng = np.random.default_rng(7)
    n, rows, cols = 2, 70, 130
    g, p0, m0 = gradients(rng, n, rows, cols), rng.normal(size=(n, rows, cols)), gradients(rng, n, rows, cols)
    def step(scalars, **kw):
        p, m, ws = dev(p0, torch.float32), dev(m0), workspace(n, rows, cols)
        mok.mok_muon_step(p, dev(g), m, n, rows, cols, ws, scalars=scalars, **{**HYPER, **kw})
        return p, m
    numbers = torch.tensor([1e-2, 0.25, 0.0, 0.0], device="cuda")
    a, b = step(numbers), step(None, lr=float(np.float32(1e-2)), grad_scale=0.25)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    numbers.view(torch.int32)[3] = 1
    a = step(numbers)
    assert torch.equal(a[0], dev(p0, torch.float32)) and torch.equal(a[1], dev(m0))


@pytest.mark.parametrize("n,rows,cols", [(40, 256, 256), (20, 320, 300), (1, 384, 4160), (3, 1100, 900), (100, 40, 70)])
def test_repeats_are_equal(n, rows, cols):
    """The same call gives the same bits: with several workgroups on a CU, with K in pieces, in every tile size."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, rows, cols, generator=gen, device="cuda")
    ws, first = workspace(n, rows, cols), None
    for _ in range(6):
        out = torch.empty(n, rows, cols, dtype=torch.bfloat16, device="cuda")
        mok.mok_orthogonalise(x, n, rows, cols, out, ws)
        first = out if first is None else first
        assert torch.equal(out, first)
    y = x[n // 2].double() / x[n // 2].double().norm()
    for _ in range(5):
        g = y @ y.T.contiguous()
        y = COEF[0] * y + (COEF[1] * g + COEF[2] * g @ g) @ y
    assert (first[n // 2].double() - y).norm() <= 2.0 ** -7 * y.norm()
