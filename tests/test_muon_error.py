"""How far the orthogonalised update is off, as a function of the gradient's rank, of its shape and of the steps.

`fp16_form` is the update with X, G and B rounded to fp16 as the header says (a factor 2^8, the diagonals' remainders of G
and B kept) and everything else in 64 bits.  A rounding to fp16 is off by at most 2^-11 of the value, by 0.85 * 2^-12 in
the root mean square; X has norm 1 at the start, and a direction that the gradient lacks grows by `a` in each step, so the
first rounding alone comes out as 0.85 * 2^-12 a^steps of Frobenius norm.  X's later roundings are of its norm then, at
most a to the steps before, and add to that in squares: twice 2^-12 a^steps holds them, and G's and B's smaller ones.  Sums
over thousands of roundings that point every way differ by a few percent from one set to another: half as much again as
fp16_form's error is far from chance.
"""
import numpy as np
import pytest
import torch

import block8_reference as ref
import token_dispatch_grouped_top_amd as mok

COEF = mok.NEWTON_SCHULZ


def missing(steps, coef=COEF):
    """Bound of the error's norm that mok.h names."""
    return 2.0 ** -11 * coef[0] ** steps


def fp16_form(v, coef, steps):
    a, b, c = coef
    keep = lambda x: (x * 256).astype(np.float32).astype(np.float16).astype(np.float64) / 256  # noqa: E731
    x = np.asarray(v, np.float64)
    tall = x.shape[0] > x.shape[1]
    x = keep((x.T if tall else x) / np.linalg.norm(x))
    for i in range(steps):
        gram = x @ x.T
        g = keep(gram)
        d = np.diag(gram) - np.diag(g)
        p = b * (g + np.diag(d)) + c * (g @ g + d[:, None] * g + g * d)
        h = keep(p)
        x = a * x + h @ x + (np.diag(p) - np.diag(h))[:, None] * x
        x = keep(x) if i + 1 < steps else x
    return x.T if tall else x


def of_rank(rng, r, rows, cols):
    return (rng.normal(size=(rows, r)) @ rng.normal(size=(r, cols))).astype(np.float32)


RANKS = [(1, 256, 192), (4, 200, 333), (16, 192, 256), (64, 384, 520), (256, 768, 800)]


@pytest.mark.parametrize("r,rows,cols", RANKS)
@pytest.mark.parametrize("steps", [1, 3, 5, 6])
def test_form_of_low_rank(r, rows, cols, steps):
    v = of_rank(np.random.default_rng(r), r, rows, cols)
    want, _ = ref.orthogonalise(v, COEF, steps)
    off = np.linalg.norm(fp16_form(v, COEF, steps) - want)
    assert off <= missing(steps)
    assert off >= 0.35 * missing(steps)                # and it is no less: the gradient's rank is what decides
    if steps == 5:
        assert off / np.linalg.norm(want) <= 0.25 / r ** 0.5
        assert r > 64 or off / np.linalg.norm(want) > 0.01


@pytest.mark.parametrize("rows,cols", [(64, 512), (384, 1024), (520, 260)])
def test_form_of_full_rank(rows, cols):
    v = np.random.default_rng(rows).normal(size=(rows, cols))
    want, _ = ref.orthogonalise(v, COEF, 5)
    assert np.linalg.norm(fp16_form(v, COEF, 5) - want) <= 2.0 ** -10 * np.linalg.norm(want)


def update(v, coef, steps, bf16=False):
    """The library's update: of the step in fp32, from parameters of zero, or the one in bf16."""
    n, rows, cols = v.shape
    ws = torch.full((mok.mok_muon_workspace_size(n, rows, cols),), 0xff, dtype=torch.uint8, device="cuda")
    x = torch.from_numpy(np.ascontiguousarray(v)).cuda()
    out = torch.zeros(v.shape, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    if bf16:
        mok.mok_orthogonalise(x, n, rows, cols, out, ws, steps=steps, coefficients=coef)
    else:
        mok.mok_muon_step(out, x, torch.zeros_like(x), n, rows, cols, ws, lr=1.0, momentum=0.0, scale=-1.0, steps=steps,
                          coefficients=coef)
    return out.double().cpu().numpy()


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.gpu
@pytest.mark.parametrize("r,rows,cols", RANKS)
@pytest.mark.parametrize("steps", [1, 3, 5])
def test_low_rank(gpu, r, rows, cols, steps):
    rng = np.random.default_rng(r)
    v = np.stack([of_rank(rng, r, rows, cols) for _ in range(2)])
    got, rounded = update(v, COEF, steps), update(v, COEF, steps, bf16=True)
    for i in range(2):
        want, _ = ref.orthogonalise(v[i], COEF, steps)
        off = np.linalg.norm(got[i] - want)
        assert off <= missing(steps)
        assert off <= 1.5 * np.linalg.norm(fp16_form(v[i], COEF, steps) - want)
        assert np.linalg.norm(rounded[i] - want) <= missing(steps) + 2.0 ** -8 * np.linalg.norm(want)


@pytest.mark.gpu
@pytest.mark.parametrize("n,rows,cols", [(1, 64, 512), (2, 384, 1024), (1, 520, 260), (2, 190, 333), (1, 768, 1600)])
@pytest.mark.parametrize("few", [0, 2])
def test_full_rank(gpu, n, rows, cols, few):
    """What the step takes from the parameters, before any rounding to bf16; noise alone, and with directions in common."""
    rng = np.random.default_rng(rows)
    v = rng.normal(size=(n, rows, cols)).astype(np.float32)
    if few:
        v += np.stack([of_rank(rng, few, rows, cols) for _ in range(n)])
    got = update(v, COEF, 5)
    for i in range(n):
        want, _ = ref.orthogonalise(v[i], COEF, 5)
        off, size = np.linalg.norm(got[i] - want), np.linalg.norm(want)
        assert off <= 1.5 * np.linalg.norm(fp16_form(v[i], COEF, 5) - want)
        assert few or off <= 2.0 ** -10 * size


@pytest.mark.gpu
def test_full_rank_largest_tiles(gpu):
    """Enough of the largest tiles in every product; a matrix of each end and one between against 64 bits."""
    n, rows, cols = 12, 2040, 2176
    gen = torch.Generator(device="cuda").manual_seed(n)
    v = torch.randn(n, rows, cols, generator=gen, device="cuda")
    p, ws = torch.zeros_like(v), torch.empty(mok.mok_muon_workspace_size(n, rows, cols), dtype=torch.uint8, device="cuda")
    mok.mok_muon_step(p, v, torch.zeros_like(v), n, rows, cols, ws, lr=1.0, momentum=0.0, scale=-1.0)
    a, b, c = COEF
    for i in (0, 5, n - 1):
        x = v[i].double() / v[i].double().norm()
        for _ in range(5):
            g = x @ x.T.contiguous()
            x = a * x + (b * g + c * g @ g) @ x
        # near square: singular values down to a thousandth of the largest, which the steps do not bring to 1
        assert (p[i].double() - x).norm() <= 2.0 ** -9 * x.norm()
