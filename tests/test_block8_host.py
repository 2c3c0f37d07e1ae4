"""Host checks of the 8-bit block operands and of the orthogonalised update: refusals before any launch, sizes, and the
reference's own codes."""
import ctypes as C

import numpy as np
import pytest
import torch

import block8_reference as ref
import token_dispatch_grouped_top_amd as mok

L = mok._lib
OK, BAD, UNSUPPORTED, WORKSPACE = mok.MOK_OK, mok.MOK_ERR_INVALID_ARG, mok.MOK_ERR_UNSUPPORTED, mok.MOK_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


def _source(**kw):
    s = dict(op=0, type=1, x=16, ld=4096, d=None, ldd=0, ring_rows=0, reserved=0)
    s.update(kw)
    return mok.mok_block8_source(**s)


def _quantise(rows=4, W=128, offsets=16, n_local=2, codes=16, scales=16, codes_t=16, scales_t=16, t_scales=0, **kw):
    return L.mok_block8_quantise(C.byref(_source(**kw)), rows, W, offsets, n_local, codes, scales, codes_t, scales_t,
                                 t_scales, None)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(W=0), dict(W=96), dict(W=-64), dict(n_local=0), dict(n_local=257), dict(offsets=None),
    dict(offsets=18), dict(codes=None), dict(scales=None), dict(codes_t=None), dict(scales_t=None),
    dict(codes=None, scales=None, codes_t=None, scales_t=None), dict(codes=24), dict(codes_t=8), dict(scales=2),
    dict(scales_t=2), dict(t_scales=2), dict(t_scales=-1), dict(op=3), dict(op=-1), dict(type=2), dict(x=None),
    dict(x=17), dict(type=0, x=18), dict(ld=127), dict(op=1, ld=255), dict(op=2, ld=127, d=16, ldd=64),
    dict(op=2, d=16, ldd=63), dict(op=2, d=None, ldd=64), dict(op=2, d=17, ldd=64), dict(reserved=1),
    dict(ring_rows=-1), dict(ring_rows=4, op=1), dict(ring_rows=4, type=0)])
def test_quantise_refuses(bad):
    assert _quantise(**bad) == BAD


def test_quantise_limits():
    assert _quantise(rows=(1 << 31) - 1, W=64 * 4096, ld=1 << 20) == UNSUPPORTED
    assert L.mok_block8_quantise(None, 4, 128, 16, 2, 16, 16, 16, 16, 0, None) == BAD
    assert _quantise(rows=0, x=None) == OK
    assert _quantise(rows=0, x=None, n_local=1, offsets=None) == OK


@pytest.mark.parametrize("bad", [dict(w=None), dict(w=17), dict(type=2), dict(n=-1), dict(N=65), dict(K=0),
                                 dict(codes=None), dict(scales=None), dict(codes=8), dict(scales=2), dict(codes_t=None),
                                 dict(scales_t=None), dict(codes_t=8), dict(scales_t=6)])
def test_weights_refuse(bad):
    a = dict(w=16, type=1, n=2, N=128, K=192, codes=16, scales=16, codes_t=16, scales_t=16)
    a.update(bad)
    assert L.mok_block8_quantise_weights(*a.values(), None) == BAD


def test_weights_limits():
    assert L.mok_block8_quantise_weights(None, 0, 0, 64, 64, None, None, None, None, None) == OK
    assert L.mok_block8_quantise_weights(16, 0, 65536, 64, 64, 16, 16, None, None, None) == UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(a=None), dict(a=8), dict(sa=None), dict(sa=2), dict(rows=-1), dict(K=32),
                                 dict(offsets=None), dict(offsets=2), dict(n=0), dict(n=257), dict(w=None), dict(w=8),
                                 dict(sw=None), dict(sw=1), dict(N=0), dict(N=100), dict(out=None), dict(out=8),
                                 dict(type=3)])
def test_gemm_refuses(bad):
    a = dict(a=16, sa=16, rows=4, K=128, offsets=16, n=2, w=16, sw=16, N=64, out=16, type=1)
    a.update(bad)
    assert L.mok_block8_gemm(*a.values(), None) == BAD


def test_gemm_limits():
    call = lambda rows, K, N: L.mok_block8_gemm(16, 16, rows, K, 16, 2, 16, 16, N, 16, 1, None)  # noqa: E731
    assert call(4, (1 << 20) + 64, 64) == UNSUPPORTED
    assert call(4, 1 << 17, 1 << 15) == UNSUPPORTED
    assert call((1 << 31) - 1, 64, 1 << 16) == UNSUPPORTED
    assert L.mok_block8_gemm(None, None, 0, 64, None, 1, None, None, 64, None, 0, None) == OK


@pytest.mark.parametrize("bad", [dict(dy=None), dict(dy=8), dict(sdy=None), dict(sdy=2), dict(M=0), dict(M=96),
                                 dict(x=None), dict(x=8), dict(sx=None), dict(sx=2), dict(N=32), dict(rows=-1),
                                 dict(offsets=None), dict(offsets=2), dict(n=0), dict(n=257), dict(dw=None), dict(dw=4),
                                 dict(type=2), dict(add=2), dict(add=-1), dict(type=1, add=1)])
def test_wgrad_refuses(bad):
    a = dict(dy=16, sdy=16, M=64, x=16, sx=16, N=64, rows=4, offsets=16, n=2, dw=16, type=0, add=1)
    a.update(bad)
    assert L.mok_block8_wgrad(*a.values(), None) == BAD


def test_wgrad_limits():
    call = lambda M, N, rows, n: L.mok_block8_wgrad(16, 16, M, 16, 16, N, rows, 16, n, 16, 0, 0, None)  # noqa: E731
    assert call(64, 64, 1 << 24, 2) == UNSUPPORTED
    assert call(1 << 16, 1 << 16, 4, 256) == UNSUPPORTED


def test_slots():
    for rows in (0, 1, 127, 128, 129, 1000):
        for n in (1, 2, 7, 256):
            assert mok.mok_block8_slots(rows, n) == ref.slots(rows, n)
    assert mok.mok_block8_slots(-1, 1) == mok.mok_block8_slots(1, 0) == mok.mok_block8_slots(1, 257) == 0
    # whatever the rows' split, the experts' blocks fit
    rng = np.random.default_rng(0)
    for _ in range(300):
        n, rows = int(rng.integers(1, 20)), int(rng.integers(0, 700))
        counts = np.bincount(rng.integers(0, n, rows), minlength=n)
        assert ref.starts(counts)[-1] <= ref.slots(rows, n)
        ones = np.minimum(1, counts)
        assert ref.starts(ones)[-1] <= ref.slots(int(ones.sum()), n)


def _hyper(**kw):
    ns = dict(a=3.0, b=-4.0, c=2.0, steps=5)
    ns.update({k: kw.pop(k) for k in list(kw) if k in ns})
    h = dict(lr=1e-3, momentum=0.9, weight_decay=0.1, grad_scale=1.0, scale=1.0, nesterov=1, reserved=0)
    h.update(kw)
    return mok.mok_muon_hyper(*h.values(), mok.mok_newton_schulz(*ns.values()))


@pytest.mark.parametrize("bad", [dict(lr=NAN), dict(lr=INF), dict(momentum=1.0), dict(momentum=-0.1),
                                 dict(momentum=NAN), dict(weight_decay=INF), dict(grad_scale=NAN), dict(scale=INF),
                                 dict(nesterov=2), dict(reserved=1), dict(a=NAN), dict(b=INF), dict(c=NAN),
                                 dict(steps=0), dict(steps=33)])
def test_muon_refuses_numbers(bad):
    size = mok.mok_muon_workspace_size(2, 64, 96)
    call = lambda h: L.mok_muon_step(16, 16, 16, 1, 16, 2, 64, 96, C.byref(h), None, 256, size, None)  # noqa: E731
    assert call(_hyper(**bad)) == BAD


@pytest.mark.parametrize("bad", [dict(p=None), dict(p=2), dict(p_bf16=17), dict(grad=None), dict(grad=17), dict(type=2),
                                 dict(m=None), dict(m=6), dict(n=-1), dict(rows=0), dict(cols=0), dict(rows=32769),
                                 dict(cols=32769), dict(n=65536), dict(scalars=8), dict(ws=None), dict(ws=128)])
def test_muon_refuses_buffers(bad):
    a = dict(p=16, p_bf16=None, grad=16, type=1, m=16, n=2, rows=64, cols=96, h=C.byref(_hyper()), scalars=None, ws=256,
             size=1 << 40)
    a.update(bad)
    assert L.mok_muon_step(*a.values(), None) == BAD


def test_muon_workspace():
    assert mok.mok_muon_workspace_size(1, 0, 4) == mok.mok_muon_workspace_size(-1, 4, 4) == 0
    size = mok.mok_muon_workspace_size(3, 100, 70)
    assert size == mok.mok_muon_workspace_size(3, 70, 100) > 3 * 2 * (3 * 128 * 128)
    ns = mok.mok_newton_schulz(3.0, -4.0, 2.0, 5)
    orth = lambda **kw: L.mok_orthogonalise(*{**dict(x=16, type=0, n=3, rows=100, cols=70, ns=C.byref(ns), out=16,  # noqa: E731
                                                     ws=256, size=size), **kw}.values(), None)
    assert orth(size=size - 1) == WORKSPACE
    assert L.mok_muon_step(16, None, 16, 1, 16, 3, 100, 70, C.byref(_hyper()), None, 256, size - 1, None) == WORKSPACE
    for bad in (dict(x=None), dict(x=2), dict(out=None), dict(out=17), dict(ws=None), dict(ws=64), dict(type=5),
                dict(rows=0), dict(ns=None)):
        assert orth(**bad) == BAD
    assert orth(n=0, x=None, out=None, ws=None, size=0) == OK


def test_binding_refuses_without_a_gpu():
    if torch.cuda.is_available():
        pytest.skip("for a machine without a GPU")
    x = torch.zeros(4, 128)
    codes, scales = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 4)
    with pytest.raises(ValueError, match="not the current GPU"):
        mok.mok_block8_quantise(x, 4, 128, codes, scales)
    with pytest.raises(ValueError, match="float16"):
        mok.mok_block8_quantise(x.half(), 4, 128, codes, scales)
    with pytest.raises(ValueError, match="strides"):
        mok.mok_block8_quantise(x.T, 4, 128, codes, scales)
    with pytest.raises(ValueError, match="codes"):
        mok.mok_block8_quantise_weights(1 << 12, 1, 64, 128, x, scales)
    with pytest.raises(ValueError, match="out"):
        mok.mok_block8_gemm(16, 16, 4, 128, 16, 16, 64, codes)
    with pytest.raises(ValueError, match="dw"):
        mok.mok_block8_wgrad(16, 16, 64, 16, 16, 64, 4, codes)
    with pytest.raises(ValueError, match="out"):
        mok.mok_orthogonalise(16, 1, 4, 8, x, 256)
    with pytest.raises(ValueError, match="scalars"):
        mok.mok_muon_step(16, 16, 16, 1, 4, 8, None, 0.1, 0.9, 1.0, scalars=torch.zeros(3))


def test_reference_codes_are_torchs():
    """The reference's rounding against torch's conversion of every quotient of a grid and of random ones."""
    rng = np.random.default_rng(1)
    x = np.concatenate([np.linspace(-448, 448, 20001), rng.normal(size=5000) * 1e-2, ref._POS[:127],
                        (ref._POS[:126] + ref._POS[1:127]) / 2, [0.0, -0.0]]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(x, np.float32(1)), want)
