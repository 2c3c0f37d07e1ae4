"""The orthogonalised update at the ends of its ranges.  Matrices with one value c in each row (and column) of the smaller
side have equal singular values: the update is s in those places, s the scalar polynomial's value, and zero elsewhere."""
import numpy as np
import pytest
import torch

import block8_reference as ref
import token_dispatch_grouped_top_amd as mok

pytestmark = pytest.mark.gpu
A, B, C = mok.NEWTON_SCHULZ


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.empty_cache()


def scalar(k, steps=5):
    """The value, and what X's roundings to 11 bits make of it: a step carries an error on by |p'(s)| and rounds its result
    (but the last); G's and B's roundings are kept beside them in fp32."""
    s, u = k ** -0.5, 2.0 ** -11
    e = u * s
    for i in range(steps):
        e *= abs(A + 3 * B * s ** 2 + 5 * C * s ** 4)
        s = s * (A + s * s * (B + s * s * C))
        e += u * abs(s) if i + 1 < steps else 2.0 ** -20 * abs(s)
    return s, e


@pytest.mark.parametrize("rows,cols", [(32768, 32768), (32768, 64), (1, 32768), (32768, 1), (100, 32705)])
def test_largest_sides(rows, cols):
    k = min(rows, cols)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    places = torch.randperm(max(rows, cols), generator=gen, device="cuda")[:k]
    at = (torch.arange(k, device="cuda"), places) if rows <= cols else (places, torch.arange(k, device="cuda"))
    sign = torch.randint(0, 2, (k,), generator=gen, device="cuda").float() * 2 - 1
    g = torch.zeros(rows, cols, device="cuda")
    g[at] = 3.7 * sign
    p, m = torch.zeros_like(g), torch.zeros_like(g)
    pb = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mok.mok_muon_workspace_size(1, rows, cols), dtype=torch.uint8, device="cuda")
    mok.mok_muon_step(p, g, m, 1, rows, cols, ws, lr=1.0, momentum=0.0, scale=-1.0, p_bf16=pb)
    assert torch.equal(m, g)
    want, tol = scalar(k)
    for got, step in ((p, 0.0), (pb, 2.0 ** -8)):
        assert ((got[at].float() * sign - want).abs() <= tol + step * (abs(want) + tol)).all()
        got[at] = 0
        assert not got.any()


def test_most_matrices():
    n, rows, cols = 65535, 2, 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, rows, cols, generator=gen, device="cuda")
    out = torch.empty(n, rows, cols, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(mok.mok_muon_workspace_size(n, rows, cols), dtype=torch.uint8, device="cuda")
    mok.mok_orthogonalise(x, n, rows, cols, out, ws)
    v = x.double()
    y = v / v.square().sum((1, 2), keepdim=True).sqrt()
    mul = lambda a, b: (a[:, :, :, None] * b[:, None]).sum(2)  # noqa: E731
    for _ in range(5):
        g = mul(y, y.mT)
        y = A * y + mul(B * g + C * mul(g, g), y)
    # the smaller singular value may be near zero: the bound of one that is (2^-11 a^5) beside bf16's rounding
    assert ((out.double() - y).square().sum((1, 2)).sqrt() <= 2.0 ** -11 * A ** 5 + 2.0 ** -8 * y.square().sum((1, 2)).sqrt()).all()
    # and for most it is not
    off = (out.double() - y).square().sum((1, 2)).sqrt() / y.square().sum((1, 2)).sqrt()
    assert off.median() <= 2.0 ** -8


def test_more_than_2_31_values():
    n, rows, cols = 130, 4096, 4160
    gen = torch.Generator(device="cuda").manual_seed(2)
    g = torch.empty(n, rows, cols, dtype=torch.bfloat16, device="cuda")
    for i in range(n):
        g[i] = torch.randn(rows, cols, generator=gen, device="cuda")
    p, m = (torch.zeros(n, rows, cols, device="cuda") for _ in range(2))
    ws = torch.empty(mok.mok_muon_workspace_size(n, rows, cols), dtype=torch.uint8, device="cuda")
    mok.mok_muon_step(p, g, m, n, rows, cols, ws, lr=1.0, momentum=0.0, scale=-1.0)
    del ws
    for i in (0, 70, n - 1):
        assert torch.equal(m[i], g[i].float())
        y = g[i].double() / g[i].double().norm()
        for _ in range(5):
            gram = y @ y.T.contiguous()
            y = A * y + (B * gram + C * gram @ gram) @ y
        # near square: test_muon_error.py, test_full_rank_largest_tiles
        assert (p[i].double() - y).norm() <= 2.0 ** -9 * y.norm()
