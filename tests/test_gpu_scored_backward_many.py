"""GPU tests of the scored route's backward where four tokens share a wave:
every width of a lane's share of the row, with masked and extreme logits.

Bounds as for few tokens: (4 |x| + 192) 2^-24 of the terms' magnitude, |x| at
most 104, from the roundings of the exponentials, the shares, the sum (a lane
adds at most 32 terms, then 4 levels) and the products, 2^-120 below the normal
numbers, and half a step of the type."""
import numpy as np
import pytest
import torch

import scored_reference as ref
import token_dispatch_grouped_top_amd as mok

pytestmark = pytest.mark.gpu
SPARSE, DENSE = 8193, 32771


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _logits(rng, T, E, kind):
    l = rng.normal(size=(T, E)).astype(np.float32) + np.float32(0.5) * rng.normal(size=E).astype(np.float32)
    if kind == "masks":
        l[:, rng.random(E) < 0.2] = -np.inf                       # experts switched off
        half = l[T // 2:]
        half[rng.random(half.shape) < 0.9] = np.nan               # hardly any left
        l[-1] = -np.inf                                           # a row with none
    elif kind == "extreme":
        l *= 200
        l[0] = np.finfo(np.float32).min                           # the lowest value of the type: all alike
        l[1, ::3] = np.inf
        l[1, 1::3] = -np.finfo(np.float32).max
        l[2] = -90 + rng.normal(size=E)                           # sigmoids below the normal numbers
    return l


def _check(E, k, score, renorm, dtype, kind, T, pad, scale):
    rng = np.random.default_rng(E * 10 + k + 2 * score + renorm)
    a = _logits(rng, T, E, kind)
    if dtype == torch.bfloat16:
        a = np.where(np.isfinite(a), np.clip(a, -3.38953139e38, 3.38953139e38), a)
    wide_in = torch.full((T, E + pad), 7.0, dtype=dtype, device="cuda")
    wide_in[:, :E] = torch.from_numpy(a).cuda()
    x = wide_in[:, :E]
    lv = x.double().cpu().numpy()
    picks = np.argsort(-ref.clean(lv), axis=1, kind="stable")[:, :k].astype(np.int32)   # of masked experts too
    picks[rng.random((T, k)) < 0.1] = -1
    picks[2] = -1                                                 # no pick at all
    if k > 1:
        picks[0, 1] = picks[0, 0]                                 # an expert twice
        picks[5:4000:7, k - 1] = picks[5:4000:7, 0]
    picks[1, 0] = E + 3                                           # out of range
    dg = rng.normal(size=(T, k)).astype(np.float32)
    dg[picks == -1] = np.nan                                      # not read into the result
    wide = torch.full((T, E + pad), 3.0, dtype=dtype, device="cuda")
    r = mok.mok_router_desc(n_experts=E, top_k=k, score=score, n_groups=1, top_groups=1, group_rule=0,
                            renorm=int(renorm), scale=scale)
    mok.mok_route_scored_backward(r, x, T, torch.from_numpy(picks).cuda(), torch.from_numpy(dg).cuda(), wide[:, :E])
    want, size = ref.route_backward(lv, score, picks, np.nan_to_num(dg), renorm, scale)
    c = ref.clean(lv)
    xm = np.minimum(np.abs(np.where(c > -np.inf, c, 0)).max(1, keepdims=True) * 2, 104.0)
    bar = (4 * xm + 192) * 2.0 ** -24 * size + 2.0 ** -120
    if dtype == torch.bfloat16:
        bar = bar + 2.0 ** -8 * (np.abs(want) + bar)
    err = np.abs(wide[:, :E].double().cpu().numpy() - want)
    assert np.all(err <= bar), float((err / bar).max())
    assert bool((wide[:, E:] == 3.0).all())                       # behind the rows: untouched


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["normal", "masks", "extreme"])
@pytest.mark.parametrize("E,k,pad", [(3, 2, 1), (64, 6, 0), (65, 8, 3), (128, 16, 8), (160, 6, 8), (256, 8, 0), (257, 5, 0),
                                     (384, 8, 4), (512, 12, 8)])
def test_dense(E, k, pad, kind, dtype):
    _check(E, k, ref.SOFTMAX, False, dtype, kind, DENSE, pad, 2.5)


@pytest.mark.parametrize("score,renorm", [(ref.SIGMOID, False), (ref.SIGMOID, True), (ref.SOFTMAX, True)])
@pytest.mark.parametrize("kind", ["masks", "extreme"])
@pytest.mark.parametrize("E,k,pad", [(3, 3, 1), (64, 16, 0), (201, 7, 3), (384, 8, 8), (512, 12, 0)])
def test_sparse(E, k, pad, kind, score, renorm):
    for dtype in (torch.float32, torch.bfloat16):
        _check(E, k, score, renorm, dtype, kind, SPARSE, pad, 1.0)
