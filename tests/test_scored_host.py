"""Host checks of the scored route, its backward, the bias update and the
AdamW step: bad arguments are refused before any launch, and the plain forms
that the GPU tests compare with agree with differences and with their own
definitions."""
import ctypes as C

import numpy as np
import pytest
import torch

import scored_reference as ref
import token_dispatch_grouped_top_amd as mok

L = mok._lib
E_ARG, E_UNS, E_WS = mok.MOK_ERR_INVALID_ARG, mok.MOK_ERR_UNSUPPORTED, mok.MOK_ERR_WORKSPACE


def _router(**kw):
    d = dict(n_experts=32, top_k=4, score=mok.MOK_SCORE_SIGMOID, n_groups=8, top_groups=4,
             group_rule=mok.MOK_GROUP_TOP2, renorm=1, scale=2.5)
    d.update(kw)
    return mok.mok_router_desc(**d)


BAD_ROUTERS = [dict(n_experts=0), dict(n_experts=4097), dict(top_k=0), dict(top_k=33), dict(top_k=17),
               dict(n_groups=0), dict(n_groups=5), dict(n_groups=65, n_experts=65), dict(top_groups=0),
               dict(top_groups=9), dict(score=2), dict(score=-1), dict(group_rule=2), dict(renorm=2),
               dict(scale=float("nan")), dict(scale=float("inf"))]


@pytest.mark.parametrize("bad", BAD_ROUTERS)
def test_bad_router_refused(bad):
    r = _router(**bad)
    assert L.mok_route_scored(C.byref(r), 16, 0, 5000, None, 4, 16, 16, None, None) == E_ARG
    assert L.mok_route_scored_backward(C.byref(r), 16, 0, 5000, 4, 16, 16, 16, 5000, None) == E_ARG


def test_route_refusals():
    r = C.byref(_router())
    route, bwd = L.mok_route_scored, L.mok_route_scored_backward
    assert route(None, 16, 0, 32, None, 4, 16, 16, None, None) == E_ARG
    assert route(r, 16, 2, 32, None, 4, 16, 16, None, None) == E_ARG      # type
    assert route(r, 16, 0, 31, None, 4, 16, 16, None, None) == E_ARG      # ld < E
    assert route(r, 16, 0, 32, None, -1, 16, 16, None, None) == E_ARG
    assert route(r, None, 0, 32, None, 4, 16, 16, None, None) == E_ARG
    assert route(r, 16, 0, 32, None, 4, None, 16, None, None) == E_ARG
    assert route(r, 16, 0, 32, None, 4, 16, None, None, None) == E_ARG
    assert route(r, None, 0, 32, None, 0, None, None, None, None) == mok.MOK_OK   # no tokens
    assert route(r, 18, 0, 32, None, 4, 16, 16, None, None) == E_ARG      # fp32 at no multiple of 4
    assert route(r, 17, 1, 32, None, 4, 16, 16, None, None) == E_ARG      # bf16 at an odd address
    assert route(r, 16, 0, 32, 18, 4, 16, 16, None, None) == E_ARG
    assert route(r, 16, 0, 32, None, 4, 18, 16, None, None) == E_ARG
    assert route(r, 16, 0, 32, None, 4, 16, 18, None, None) == E_ARG
    assert route(r, 16, 0, 32, None, 4, 16, 16, 18, None) == E_ARG
    assert route(r, 16, 0, 32, None, 1 << 26, 16, 16, None, None) == E_UNS   # more threads than a launch has
    assert bwd(r, 16, 0, 32, 1 << 26, 16, 16, 16, 32, None) == E_UNS
    assert bwd(r, 18, 0, 32, 4, 16, 16, 16, 32, None) == E_ARG
    assert bwd(r, 16, 1, 32, 4, 16, 16, 17, 32, None) == E_ARG
    assert bwd(r, 16, 0, 32, 4, 16, 16, 16, 31, None) == E_ARG            # ldd < E
    assert bwd(r, 16, 0, 32, 4, None, 16, 16, 32, None) == E_ARG
    assert bwd(r, 16, 0, 32, 4, 16, None, 16, 32, None) == E_ARG
    assert bwd(r, 16, 0, 32, 4, 16, 16, None, 32, None) == E_ARG
    assert bwd(r, None, 0, 32, 0, None, None, None, 32, None) == mok.MOK_OK
    bias = L.mok_route_bias_update
    assert bias(16, 1, 0, 1e-3, 16, 0, None) == E_ARG
    assert bias(16, 1, 65537, 1e-3, 16, 0, None) == E_ARG
    assert bias(16, -1, 8, 1e-3, 16, 0, None) == E_ARG
    assert bias(16, 1, 8, float("nan"), 16, 0, None) == E_ARG
    assert bias(16, 1, 8, 1e-3, 16, 2, None) == E_ARG
    assert bias(None, 1, 8, 1e-3, 16, 0, None) == E_ARG
    assert bias(16, 1, 8, 1e-3, None, 0, None) == E_ARG
    assert bias(None, 0, 8, 1e-3, None, 0, None) == mok.MOK_OK
    assert bias(18, 1, 8, 1e-3, 16, 0, None) == E_ARG and bias(16, 1, 8, 1e-3, 18, 0, None) == E_ARG
    assert bias(16, 1 << 22, 8, 1e-3, 16, 0, None) == E_UNS


def test_forward_scored_refusals():
    d = mok.mok_layer_desc(hidden=256, inter=512, n_experts=32, top_k=4, expert_base=0, n_local=8)
    tok = mok.mok_tokens(1, 1, 16)
    call = L.mok_moe_forward_scored

    def go(desc=d, router=_router(), logits=16, kind=0, ld=32, T=4, idx=16, gate=16, ws_bytes=1 << 30):
        return call(C.byref(desc), C.byref(router), logits, kind, ld, None, T, idx, gate, None, C.byref(tok),
                    16, 16, C.byref(tok), 16, ws_bytes, None)
    assert go(router=_router(n_experts=64)) == E_ARG                       # not the layer's
    assert go(router=_router(top_k=2)) == E_ARG
    assert go(router=_router(top_groups=0)) == E_ARG
    assert go(logits=None) == E_ARG
    assert go(kind=3) == E_ARG
    assert go(logits=18) == E_ARG and go(idx=18) == E_ARG
    assert go(ld=31) == E_ARG
    assert go(idx=None) == E_ARG and go(gate=None) == E_ARG                # both or neither
    assert go(T=17) == E_ARG                                               # more tokens than rows
    assert go(ws_bytes=16) == E_WS
    assert call(None, C.byref(_router()), 16, 0, 32, None, 4, 16, 16, None, C.byref(tok), 16, 16,
                C.byref(tok), 16, 1 << 30, None) == E_ARG


def _tensor(**kw):
    d = dict(p=1 << 20, grad=2 << 20, m=3 << 20, v=4 << 20, n=64, lr_scale=1.0)
    d.update(kw)
    return mok.mok_adamw_tensor(**d)


def _build(tensors, table=64, size=1 << 20):
    a = (mok.mok_adamw_tensor * max(len(tensors), 1))(*tensors)
    return L.mok_adamw_build_table(a, len(tensors), table, size, C.byref(mok.mok_adamw_plan()), None)


@pytest.mark.parametrize("bad", [dict(n=-1), dict(grad_type=2), dict(state_format=2), dict(p=None), dict(grad=None),
                                 dict(m=None), dict(v=None), dict(state_format=1), dict(state_format=1, m_scale=64),
                                 dict(p=(1 << 20) + 2), dict(p_bf16=65), dict(grad=66), dict(grad=65, grad_type=1),
                                 dict(m=66), dict(v=66), dict(lr_scale=float("nan")), dict(weight_decay=float("inf"))])
def test_bad_adamw_tensor_refused(bad):
    assert _build([_tensor(**bad)]) == E_ARG
    assert _build([_tensor(p=9 << 20), _tensor(**bad)]) == E_ARG


def test_adamw_table_refusals():
    t = _tensor()
    assert _build([t, t]) == E_ARG                                         # the same tensor twice
    assert _build([t, _tensor(p=(1 << 20) + 64 * 4 - 4)]) == E_ARG         # overlapping parameters
    assert _build([_tensor(n=1 << 62)]) == E_UNS
    far = [_tensor(p=i << 50, n=6 << 30) for i in range(1, 4)]             # more units than a launch has
    assert _build(far) == E_UNS
    assert _build([t], table=None) == E_ARG
    assert _build([t], table=72) == E_ARG                                  # not 16-byte aligned
    need = mok.mok_adamw_table_size(1)
    assert need > 0 and mok.mok_adamw_table_size(3) > need and mok.mok_adamw_table_size(-1) == 0
    assert _build([t], size=need - 1) == E_WS
    a, plan = (mok.mok_adamw_tensor * 1)(t), mok.mok_adamw_plan()
    assert L.mok_adamw_build_table(None, 1, 64, 1 << 20, C.byref(plan), None) == E_ARG
    assert L.mok_adamw_build_table(a, -1, 64, 1 << 20, C.byref(plan), None) == E_ARG
    assert L.mok_adamw_build_table(a, 1, 64, 1 << 20, None, None) == E_ARG
    assert _build([]) == mok.MOK_OK
    assert _build([_tensor(n=0, p=None)]) == mok.MOK_OK                    # nothing to do


def test_adamw_step_refusals():
    def step(plan=dict(n_units=(1, 0), n_tensors=(1, 0), list=1), table=64, scalars=None, **kw):
        h = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, grad_scale=1.0, step=1)
        h.update(kw)
        p = mok.mok_adamw_plan((C.c_int64 * 2)(*plan.get("n_units", (0, 0))),
                               (C.c_int32 * 2)(*plan.get("n_tensors", (0, 0))), plan.get("list", 0))
        return L.mok_adamw_step(table, C.byref(p), C.byref(mok.mok_adamw_hyper(**h)),
                                scalars, None)
    for bad in (dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")),
                dict(eps=-1.0), dict(eps=float("inf")), dict(grad_scale=float("inf")), dict(step=0), dict(step=-3)):
        assert step(**bad) == E_ARG, bad
    assert step(scalars=8) == E_ARG                                        # not 16-byte aligned
    assert step(table=None) == E_ARG
    for plan in (dict(n_units=(-1, 0)), dict(n_units=(1, 0)), dict(n_units=(0, 1), n_tensors=(1, 0), list=1),
                 dict(n_units=(0, 1 << 24), n_tensors=(0, 1), list=1), dict(n_units=(1, 0), n_tensors=(-1, 0)),
                 dict(n_units=(1, 0), n_tensors=(2, 0), list=1), dict(n_units=(1, 1), n_tensors=(1, 1), list=1)):
        assert step(plan=plan) == E_ARG, plan
    assert step(plan={}, table=None) == mok.MOK_OK                         # an empty list
    assert L.mok_adamw_step(64, None, C.byref(mok.mok_adamw_hyper(step=1)), None, None) == E_ARG
    assert L.mok_adamw_step(64, C.byref(mok.mok_adamw_plan()), None, None, None) == E_ARG


def test_binding_refuses_wrong_tensors():
    r = _router()
    x, idx, gate = torch.zeros(4, 32), torch.zeros(4, 4, dtype=torch.int32), torch.zeros(4, 4)
    with pytest.raises(ValueError, match="logits.*current GPU"):
        mok.mok_route_scored(r, x, 4, idx, gate, stream=0)
    for bad in (x.double(), x[:3], x[:, :31], torch.zeros(32, 4).t()):
        with pytest.raises(ValueError, match="logits"):
            mok.mok_route_scored(r, bad, 4, idx, gate, stream=0)
    with pytest.raises(ValueError, match="topk_idx"):
        mok._buffer(idx.long(), "topk_idx", (torch.int32,), 16, 0)
    with pytest.raises(ValueError, match="topk_idx"):
        mok._buffer(idx, "topk_idx", (torch.int32,), 17, 0)
    with pytest.raises(ValueError, match="topk_idx"):
        mok._buffer(idx.t(), "topk_idx", (torch.int32,), 16, 0)
    with pytest.raises(ValueError, match="topk_idx.*current GPU"):
        mok._buffer(idx, "topk_idx", (torch.int32,), 16, 0)
    f = torch.zeros(64)
    for t in (dict(p=f, grad=f, m=f, v=f), dict(p=f.double(), grad=f, m=f, v=f),
              dict(p=f, grad=f.half(), m=f, v=f)):
        with pytest.raises(ValueError):
            mok.AdamwTensors([t])
    with pytest.raises(ValueError, match="scalars"):
        mok.mok_adamw_step(mok.AdamwTensors([]), 1e-3, 0.9, 0.95, 1e-8, 1, scalars=torch.zeros(3), stream=0)


# ------------------------------------------------- the plain forms themselves
@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_reference_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    l = rng.normal(size=(5, 12))
    picks, _, _ = ref.route(l, score, 4, renorm=renorm)
    picks[1, 3] = -1
    picks[2] = -1
    dg = rng.normal(size=picks.shape)
    got, size = ref.route_backward(l, score, picks, dg, renorm, 2.5)
    step = 1e-5
    for e in range(12):
        up, down = l.copy(), l.copy()
        up[:, e] += step
        down[:, e] -= step
        diff = ((ref.gates(up, score, picks, renorm, 2.5) - ref.gates(down, score, picks, renorm, 2.5)) * dg
                ).sum(1) / (2 * step)
        # central differences: error of order step^2 and of rounding 2^-53 / step
        assert np.all(np.abs(got[:, e] - diff) <= 1e-8)
    assert np.all(np.abs(got) <= size + 1e-15)
    assert np.all(got[2] == 0)


def test_random_bits_are_even_and_keep_the_mean():
    n = 1 << 16
    bm, br = ref.random_bits(np.arange(n), 3, 7, 11)
    for b in (bm, br):
        assert abs(b.mean() / 65536 - 0.5) < 6 / np.sqrt(12 * n)           # six deviations of the mean
        assert np.all(np.bincount(b >> 8, minlength=256) > n / 256 - 6 * np.sqrt(n / 256))
    assert abs(np.corrcoef(bm, br)[0, 1]) < 6 / np.sqrt(n)
    # a value between two codes: the mean of m and of r^2 over the elements is the value itself
    m = np.full(n, 3.3, np.float32)
    m[::32] = 440.0                                                        # fixes the scale
    s = ref.scale_byte(m)
    assert np.all(s == 127)
    got = ref.decode(ref.encode_m(m, bm, s), s)
    rest = np.arange(n) % 32 != 0
    assert abs(got[rest].mean() - float(np.float32(3.3))) < 6 * 0.125 / np.sqrt(n)       # quantum 1/4, deviation at most half
    got = ref.decode(ref.encode_r(m, br, s), s) ** 2
    assert abs(got[rest].mean() - float(np.float32(3.3)) ** 2) < 6 * 0.5 * (3.5 ** 2 - 3.25 ** 2) / np.sqrt(n)


def test_scale_is_the_smallest_without_saturation():
    x = np.zeros(32 * 5, np.float32)
    x[0], x[32], x[64], x[96] = 448.0, np.nextafter(np.float32(448), np.float32(500)), 1e-3, 3e38
    got = ref.scale_byte(x).astype(int) - 127
    assert got[0] == 0 and got[1] == 1 and got[4] == -127
    for value, e in zip((1e-3, 3e38), got[2:4]):
        assert value <= 448 * 2.0 ** e and value > 448 * 2.0 ** (e - 1)
