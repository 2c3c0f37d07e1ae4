"""What a training step with the block operands gives back, part by part and as a whole, against 64 bits: the operands made
through SwiGLU and its backward, the merged rows, the gates' and the tokens' gradients; and each expert's weight gradient,
gate and up apart, against the formula's and along directions of the formula's, which differences of the loss confirm.

Tolerances of the parts are roundings: half a step of a code (2^-4 of a value, 2^-10 of the scale below the normal
ones) and SwiGLU's fp32 ones (test_gpu_block8.py); n products added up in fp32 n + 2 times 2^-24 of their magnitudes'
sum; a result in bf16 2^-8 of it.

As a whole every E4M3 operand is off by half a step at random: 2^-4 / sqrt(3) at the most for a mantissa of 1, 2.7 % in the
root mean square over mantissas.  The down gradient meets two such operands, and h's two behind one of them, twice as
SwiGLU has it in both factors: sqrt(6) 2.7 % = 6.6 % of its norm; the gate and up gradient two of its own, two of da and
four of h: sqrt(8) 2.7 % = 7.6 %; the tokens' gradient the same.  Twice that is allowed, where a part that is missing is
all of it.
"""
import numpy as np
import pytest
import torch

import block8_reference as ref
from test_gpu_block8_step import E, H, I, T, Step, host, k

pytestmark = pytest.mark.gpu
OFF = 0.15


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def step_of(seed):
    s = Step(seed)
    weights = {n: w.double() for n, w in s.w.items()}
    s.run()
    torch.cuda.synchronize()
    return s, weights


def f64(t):
    return host(t.float()).astype(np.float64)


@pytest.mark.parametrize("seed", [1, 6])
def test_operands_through_swiglu(seed):
    s, _ = step_of(seed)
    counts, h, da = host(s.counts).tolist(), f64(s.h), f64(s.da)
    g = np.abs(h[:, :I])
    a = ref.swiglu(h)
    dh, size = ref.swiglu_backward(h, da)
    for o, x, slack in ((s.aq, a, np.abs(a) * (g + 8) * 2.0 ** -23),
                        (s.dhq, dh, size * (np.concatenate([g, g], 1) + 12) * 2.0 ** -23)):
        def near(codes, each, x, slack):
            assert np.all(np.abs(ref.values(codes) * each - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * each + 2 * slack)
        near(host(o.codes), np.repeat(f64(o.scales).T, 128, 1)[:, :o.W], x, slack)
        codes_t, scales_t, first = host(o.codes_t), f64(o.scales_t), 0
        for c, at in zip(counts, ref.starts(counts)):
            b = np.s_[at // 128:at // 128 + ref.blocks(c)]
            each = np.repeat(scales_t[b].T, 128, 1) if o is s.dhq else \
                np.repeat(np.repeat(scales_t[:, b], 128, 0)[:o.W], 128, 1)
            near(codes_t[:, at:at + c], each[:, :c], x[first:first + c].T, slack[first:first + c].T)
            assert not codes_t[:, at + c:at + 128 * ref.blocks(c)].any()
            first += c


@pytest.mark.parametrize("seed", [1, 6])
def test_rows_and_gates(seed):
    s, _ = step_of(seed)
    soa, gate, y, dx = host(s.soa).reshape(T, k), f64(s.gate), f64(s.y), f64(s.dx)
    dout = f64(s.dout)
    terms = gate[..., None] * y[soa]                    # [T][k][H]
    out = terms.sum(1)
    assert np.all(np.abs(f64(s.out) - out) <= 2.0 ** -8 * np.abs(out) + (k + 2) * 2.0 ** -24 * np.abs(terms).sum(1))
    terms = dout[:, None] * y[soa]
    assert np.all(np.abs(f64(s.dgate) - terms.sum(2)) <= (H + 2) * 2.0 ** -24 * np.abs(terms).sum(2))
    terms = dx[soa]
    tokens = terms.sum(1)
    assert np.all(np.abs(f64(s.dx_tokens) - tokens) <= 2.0 ** -8 * np.abs(tokens) + (k + 2) * 2.0 ** -24 * np.abs(terms).sum(1))


def layer(s, w, gradients=False):
    """The loss sum(out * dout) of the layer in 64 bits; or its gradients by the weights and the tokens."""
    x, dout, gate = s.x.double(), s.dout.double(), s.gate.double()
    loss, dx = 0.0, torch.zeros_like(x)
    dw = {n: torch.zeros_like(t) for n, t in w.items()}
    for j in range(k):
        for e in range(E):
            rows = (s.idx[:, j] == e).nonzero().flatten()
            h = x[rows] @ w["gu"][e].T.contiguous()
            g, u = h[:, :I], h[:, I:]
            sig = torch.sigmoid(g)
            a, dy = g * sig * u, gate[rows, j, None] * dout[rows]
            if not gradients:
                loss = loss + (a @ w["d"][e].T.contiguous() * dy).sum()
                continue
            da = dy @ w["d"][e]
            dh = torch.cat([da * u * sig * (1 + g * (1 - sig)), da * g * sig], 1)
            dw["d"][e] += dy.T.contiguous() @ a
            dw["gu"][e] += dh.T.contiguous() @ x[rows]
            dx[rows] += dh @ w["gu"][e]
    return (dw, dx) if gradients else loss


def regions():
    for e in range(E):
        yield "d", (e, slice(None))
        yield "gu", (e, slice(0, I))
        yield "gu", (e, slice(I, 2 * I))


@pytest.mark.parametrize("seed", [2, 7])
def test_gradients_of_each_part(seed):
    s, w = step_of(seed)
    dw, dx = layer(s, w, gradients=True)
    for n, at in regions():
        want, got = dw[n][at], s.dw[n][at].double()
        assert want.norm() > 0 and (got - want).norm() <= OFF * want.norm()
        direction = torch.zeros_like(w[n])
        direction[at] = want / want.norm()
        eps = 1e-4
        slope = (layer(s, {**w, n: w[n] + eps * direction}) - layer(s, {**w, n: w[n] - eps * direction})) / (2 * eps)
        assert abs(slope - want.norm()) <= 1e-5 * want.norm()
        assert abs((got * direction[at]).sum() - slope) <= OFF * slope
    assert (s.dx_tokens.double() - dx).norm() <= OFF * dx.norm()
