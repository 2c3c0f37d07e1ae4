"""GPU tests of the scored route, its backward, the bias update and the fused
layer that routes by it, against the 64-bit forms of tests/scored_reference.py.

Picks and load are equal, always.  Gates: fp32 evaluation of exp(x) with x the
distance to the row's largest logit or the logit itself (relative error |x|
2^-24 from rounding x or its product with log2 e, twice, and two steps of the
exponential), a sum (at most 12 levels and 64 terms in a row), a reciprocal and two products: in
all (2 |x| + 96) 2^-24 of the gate, where |x| is at most 104 (below that exp
is 0 in fp32), and 2^-126 below the normal numbers.  Gradients: the same
factors on each term of a value's sum, that is (4 |x| + 192) 2^-24 of the
terms' magnitude (two factors such as u and s), and half a step of the type.
"""
import numpy as np
import pytest
import torch

import scored_reference as ref
import token_dispatch_grouped_top_amd as mok
import workloads as W
from gpu_harness import SENTINEL, DeviceWorkload, to_host

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _router(E, k, score, G=1, top_groups=1, top2=False, renorm=False, scale=1.0):
    return mok.mok_router_desc(n_experts=E, top_k=k, score=score, n_groups=G, top_groups=top_groups,
                               group_rule=int(top2), renorm=int(renorm), scale=scale)


def _logits(rng, T, E, kind):
    l = rng.normal(size=(T, E)) + 0.5 * rng.normal(size=E)
    if kind == "ties":
        l = rng.integers(-1, 2, size=(T, E)).astype(float)
    elif kind == "masks":
        l[:, rng.random(E) < 0.2] = -np.inf           # experts switched off
        l[T // 2:][rng.random((T - T // 2, E)) < 0.9] = np.nan    # hardly any left
        l[-1] = -np.inf                                # a row with none
    elif kind == "extreme":
        l *= 200.0
        l[0] = np.finfo(np.float32).min                # the lowest value of the type: all alike
        if T > 1:
            l[1, ::3] = np.inf
            l[1, 1::3] = -np.finfo(np.float32).max
        if T > 2:
            l[2] = -90.0 + rng.normal(size=E)          # sigmoids below fp32's smallest normal number
    return l


def _tensor(a, dtype, pad):
    wide = torch.full((a.shape[0], a.shape[1] + pad), 7.0, dtype=torch.float64)
    wide[:, :a.shape[1]] = torch.from_numpy(a)
    wide = torch.clamp(wide, -3.38953139e38, 3.38953139e38).where(torch.isfinite(wide), wide) if dtype == torch.bfloat16 else wide
    return wide.to(dtype).cuda()[:, :a.shape[1]]


def _gate_bar(logits, gate):
    l = ref.clean(logits)
    x = np.minimum(np.abs(np.where(l > -np.inf, l, 0.0)).max(1, keepdims=True) * 2, 104.0)
    return (2 * x + 96) * 2.0 ** -24 * np.abs(gate) + 2.0 ** -126


ROUTES = [
    # E, k, G, top_groups, top2
    (8, 2, 1, 1, False), (1, 1, 1, 1, False), (7, 7, 1, 1, False), (33, 5, 1, 1, False), (64, 8, 8, 3, True),
    (160, 6, 8, 3, False), (256, 8, 8, 4, True), (384, 8, 1, 1, False), (65, 4, 5, 2, True), (63, 9, 21, 4, True),
    (60, 3, 60, 7, True), (1000, 32, 4, 2, False), (513, 12, 27, 9, True), (2048, 16, 64, 5, True), (4096, 32, 2, 1, False),
    (4095, 8, 3, 2, True), (4092, 6, 33, 5, True),
]


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("E,k,G,top_groups,top2", ROUTES)
def test_route_matches_reference(E, k, G, top_groups, top2, score):
    rng = np.random.default_rng(E * 100 + k + score)
    case = 0
    for kind in ("normal", "ties", "masks", "extreme"):
        for dtype in (torch.float32, torch.bfloat16):
            for with_bias in (False, True):
                case += 1
                T = (1, 3, 70, 129)[case % 4]
                renorm, scale, pad = bool(case // 2 % 2), (1.0, 2.5)[case % 2], (0, 5, 8)[case % 3]
                print(f"[route] E={E} k={k} G={G} score={score} {kind} {dtype} bias={with_bias} T={T}", flush=True)
                x = _tensor(_logits(rng, T, E, kind), dtype, pad)
                b = torch.from_numpy(rng.normal(size=E) * 0.1).float().cuda() if with_bias else None
                if kind == "ties" and with_bias:
                    b = torch.from_numpy(rng.integers(-1, 2, size=E) * 0.5).float().cuda()
                idx = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
                gate = torch.full((T, k), float("nan"), device="cuda")
                load = torch.full((E,), 5, dtype=torch.int32, device="cuda")
                mok.mok_route_scored(_router(E, k, score, G, top_groups, top2, renorm, scale), x, T, idx, gate,
                                     bias=b, load=load)
                lv = x.double().cpu().numpy()
                ri, rg, rl = ref.route(lv, score, k, None if b is None else b.cpu().numpy(), G, top_groups, top2,
                                       renorm, scale)
                assert np.array_equal(idx.cpu().numpy(), ri), (kind, dtype, with_bias)
                err = np.abs(gate.cpu().numpy().astype(np.float64) - rg)
                assert np.all(err <= _gate_bar(lv, rg)), (kind, dtype, with_bias, err.max())
                assert np.array_equal(load.cpu().numpy(), rl + 5)


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("E,k,G,top_groups,top2", [
    (8, 2, 1, 1, False), (3, 3, 1, 1, False), (160, 6, 8, 3, False), (256, 8, 8, 4, True), (384, 8, 1, 1, False),
    (65, 4, 5, 2, True), (512, 14, 16, 5, True), (201, 7, 3, 2, True), (96, 9, 12, 2, False), (130, 5, 2, 1, True)])
def test_route_of_many_tokens(E, k, G, top_groups, top2, score):
    """Four tokens share a wave."""
    rng = np.random.default_rng(E * 100 + k + score + 7)
    for case, kind in enumerate(("normal", "ties", "masks", "extreme", "normal", "extreme")):
        T = 2049 + 7 * case
        dtype = (torch.float32, torch.bfloat16)[case % 2]
        renorm, scale, pad = case in (0, 2, 5), (1.0, 2.5)[case % 2], (0, 5, 8)[case % 3]
        print(f"[route] E={E} k={k} G={G} score={score} {kind} {dtype} T={T}", flush=True)
        x = _tensor(_logits(rng, T, E, kind), dtype, pad)
        b = torch.from_numpy(rng.normal(size=E) * 0.1).float().cuda() if case < 4 else None
        idx = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
        gate = torch.full((T, k), float("nan"), device="cuda")
        load = torch.zeros(E, dtype=torch.int32, device="cuda")
        mok.mok_route_scored(_router(E, k, score, G, top_groups, top2, renorm, scale), x, T, idx, gate, bias=b, load=load)
        lv = x.double().cpu().numpy()
        ri, rg, rl = ref.route(lv, score, k, None if b is None else b.cpu().numpy(), G, top_groups, top2, renorm, scale)
        assert np.array_equal(idx.cpu().numpy(), ri), (kind, dtype)
        err = np.abs(gate.cpu().numpy().astype(np.float64) - rg)
        assert np.all(err <= _gate_bar(lv, rg)), (kind, dtype, err.max())
        assert np.array_equal(load.cpu().numpy(), rl)


@pytest.mark.parametrize("T", [70, 2100])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_buffers_at_any_element(T, dtype):
    """Logits, gradients and bias that begin one element behind an aligned address, rows that keep the alignment."""
    rng = np.random.default_rng(T)
    E, k = 64, 6
    r = _router(E, k, ref.SIGMOID, 4, 2, True, True, 2.5)
    r_dense = _router(E, k, ref.SOFTMAX)
    store = torch.from_numpy(rng.normal(size=(T, E + 8))).to(dtype).cuda()
    x, bias = store[:, 1:E + 1], (0.1 * torch.randn(E + 1, device="cuda"))[1:]
    idx = torch.full((T * k + 1,), 9, dtype=torch.int32, device="cuda")[1:]
    gate = torch.empty(T * k + 1, device="cuda")[1:]
    mok.mok_route_scored(r, x, T, idx, gate, bias=bias)
    lv = x.double().cpu().numpy()
    ri, rg, _ = ref.route(lv, ref.SIGMOID, k, bias.cpu().numpy(), 4, 2, True, True, 2.5)
    assert np.array_equal(idx.view(T, k).cpu().numpy(), ri)
    assert np.all(np.abs(gate.view(T, k).double().cpu().numpy() - rg) <= _gate_bar(lv, rg))
    dg = torch.randn(T * k + 1, device="cuda")[1:]
    for router, score, renorm, scale in ((r, ref.SIGMOID, True, 2.5), (r_dense, ref.SOFTMAX, False, 1.0)):
        out = torch.full((T, E + 8), 3.0, dtype=dtype, device="cuda")
        mok.mok_route_scored_backward(router, x, T, idx, dg, out[:, 1:E + 1])
        want, size = ref.route_backward(lv, score, ri, dg.view(T, k).double().cpu().numpy(), renorm, scale)
        bar = (4 * 10 + 192) * 2.0 ** -24 * size + 2.0 ** -120
        if dtype == torch.bfloat16:
            bar = bar + 2.0 ** -8 * (np.abs(want) + bar)
        assert np.all(np.abs(out[:, 1:E + 1].double().cpu().numpy() - want) <= bar)
        assert bool((out[:, 0] == 3.0).all()) and bool((out[:, E + 1:] == 3.0).all())


def test_two_streams_add_to_one_load():
    """Two calls at once on different streams, their loads counted into one buffer."""
    E, k, T = 96, 4, 3000
    r = _router(E, k, ref.SOFTMAX)
    load = torch.zeros(E, dtype=torch.int32, device="cuda")
    xs = [torch.randn(T, E, device="cuda") for _ in range(2)]
    outs = [(torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, x, (i, g) in zip(streams, xs, outs):
        mok.mok_route_scored(r, x, T, i, g, load=load, stream=s)
    torch.cuda.synchronize()
    want = sum(ref.route(x.double().cpu().numpy(), ref.SOFTMAX, k)[2] for x in xs)
    assert np.array_equal(load.cpu().numpy(), want)


def test_route_tells_close_scores_apart():
    """Scores that fp32 cannot order: neighbours of one fp32 step in the logits, a bias that brings two scores
    within 2^-40 of each other, and groups whose sums differ in the last bits."""
    rng = np.random.default_rng(5)
    T, E, k = 257, 64, 8
    base = rng.normal(size=(T, 1)).astype(np.float32) * 3
    l = np.repeat(base, E, 1)
    for t in range(T):                       # every expert a different number of steps above the base
        l[t] = (l[t].view(np.int32) + rng.permutation(E).astype(np.int32)).view(np.float32)
    for score in (ref.SOFTMAX, ref.SIGMOID):
        for G, tg in ((1, 1), (8, 3)):
            x = torch.from_numpy(np.tile(l, (9, 1))).cuda()      # the rows again: enough for four to a wave
            for bias in (np.zeros(E), rng.integers(-4, 5, E) * 2.0 ** -24):
                b = torch.from_numpy(bias).float().cuda()
                idx = torch.empty(9 * T, k, dtype=torch.int32, device="cuda")
                gate = torch.empty(9 * T, k, device="cuda")
                mok.mok_route_scored(_router(E, k, score, G, tg, True), x, 9 * T, idx, gate, bias=b)
                few, fewg = torch.empty_like(idx[:T]), torch.empty_like(gate[:T])
                mok.mok_route_scored(_router(E, k, score, G, tg, True), x[:T], T, few, fewg, bias=b)
                ri, _, _, gaps = ref.route_and_gaps(l, score, k, bias, G, tg, True)
                # Two sums of neighbours, such as p(1 + 3d) + p(1 + 4d) and p(1 + 2d) + p(1 + 5d), differ by p d^2
                # only, and d goes down to 2^-30 here: below fp64.  An evaluation in fp64 has an exponential (one
                # step), an addition, a division or product and a sum: less than 8 roundings, so two of them agree on
                # the order of values that are 2^-48 apart and on nothing less.
                clear = gaps >= 2.0 ** -48
                for got in (few, *idx.split(T)):
                    assert np.array_equal(got.cpu().numpy()[clear], ri[clear]), (score, G)
                assert clear.sum() > 3 * T // 4


@pytest.mark.parametrize("score", [ref.SOFTMAX, ref.SIGMOID])
@pytest.mark.parametrize("E,k", [(8, 2), (1, 1), (7, 7), (50, 16), (100, 5), (160, 6), (256, 8), (384, 8), (513, 12), (1000, 32),
                                 (2000, 4), (4096, 3)])
def test_backward_matches_reference(E, k, score):
    rng = np.random.default_rng(E * 10 + k + score)
    case = 0
    for kind in ("normal", "masks", "extreme"):
        for dtype in (torch.float32, torch.bfloat16):
            for renorm in (False, True):
                case += 1
                T = (1, 3, 70, 129, 2051, 2049)[case % 6]
                if E in (50, 100, 160) and kind == "normal":
                    T = 8193 if renorm or score == ref.SIGMOID else 32771       # four tokens share a wave
                scale, pad = (1.0, 2.5)[case % 2], (0, 5, 8)[case % 3]
                print(f"[bwd] E={E} k={k} score={score} {kind} {dtype} renorm={renorm} T={T}", flush=True)
                x = _tensor(_logits(rng, T, E, kind), dtype, pad)
                lv = x.double().cpu().numpy()
                picks, _, _ = ref.route(lv, score, k)
                picks[rng.random((T, k)) < 0.1] = -1
                if T > 2:
                    picks[2] = -1                              # no pick at all
                    if k > 1:
                        picks[0, 1] = picks[0, 0]              # an expert twice
                    picks[1, 0] = E + 3                        # out of range
                dg = rng.normal(size=(T, k)).astype(np.float32)
                dg[picks == -1] = np.nan                       # not read into the result
                wide = torch.full((T, E + pad), 3.0, dtype=dtype, device="cuda")
                dl = wide[:, :E]
                mok.mok_route_scored_backward(_router(E, k, score, renorm=renorm, scale=scale), x, T,
                                              torch.from_numpy(picks).cuda(), torch.from_numpy(dg).cuda(), dl)
                want, size = ref.route_backward(lv, score, picks, np.nan_to_num(dg), renorm, scale)
                xm = np.minimum(np.abs(np.where(ref.clean(lv) > -np.inf, ref.clean(lv), 0)).max(1, keepdims=True) * 2, 104.0)
                bar = (4 * xm + 192) * 2.0 ** -24 * size + 2.0 ** -120
                if dtype == torch.bfloat16:
                    bar = bar + 2.0 ** -8 * (np.abs(want) + bar)
                err = np.abs(dl.double().cpu().numpy() - want)
                assert np.all(err <= bar), (kind, dtype, renorm, float((err / bar).max()))
                assert bool((wide[:, E:] == 3.0).all())        # behind the rows: untouched


def test_backward_against_differences_of_the_gates():
    """The gradient of sum(dgate gate) over a perturbed logit, from the forward's own formula in 64 bits."""
    rng = np.random.default_rng(9)
    T, E, k = 6, 24, 4
    l = rng.normal(size=(T, E)).astype(np.float32)
    for score in (ref.SOFTMAX, ref.SIGMOID):
        for renorm in (False, True):
            x = torch.from_numpy(l).cuda()
            idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
            gate = torch.empty(T, k, device="cuda")
            r = _router(E, k, score, renorm=renorm, scale=1.5)
            mok.mok_route_scored(r, x, T, idx, gate)
            dg = torch.randn(T, k, device="cuda")
            dl = torch.empty(T, E, device="cuda")
            mok.mok_route_scored_backward(r, x, T, idx, dg, dl)
            picks, d64, eps = idx.cpu().numpy(), dg.double().cpu().numpy(), 1e-5
            for e in range(E):
                up, down = l.astype(np.float64), l.astype(np.float64)
                up[:, e] += eps
                down[:, e] -= eps
                diff = ((ref.gates(up, score, picks, renorm, 1.5) - ref.gates(down, score, picks, renorm, 1.5)) * d64).sum(1) / (2 * eps)
                assert np.all(np.abs(dl[:, e].cpu().numpy() - diff) <= 5e-5)   # (4 * 10 + 192) 2^-24 of terms below 3


@pytest.mark.parametrize("layers,E", [(1, 1), (1, 384), (3, 7), (60, 256), (2, 4097), (1, 65536)])
def test_bias_update(layers, E):
    rng = np.random.default_rng(E)
    load = rng.poisson(50, size=(layers, E)).astype(np.int32)
    load[0, : E // 2] = 2_000_000_000                       # sums and products past 32 bits
    load[-1] = 9 if layers > 1 else load[-1]                # balanced: no change
    bias = rng.normal(size=(layers, E)).astype(np.float32)
    for clear in (0, 1):
        dl, db = torch.from_numpy(load).cuda(), torch.from_numpy(bias).cuda()
        mok.mok_route_bias_update(dl, layers, E, 1e-2, db, clear_load=clear)
        l64 = load.astype(np.int64)
        step = np.sign(l64.sum(1, keepdims=True) - E * l64)
        want = bias + np.float32(1e-2) * step.astype(np.float32)
        assert np.array_equal(db.cpu().numpy(), want)
        assert np.array_equal(dl.cpu().numpy(), load * (1 - clear))


def test_route_many_rows_past_32_bit_offsets():
    """More than 2^32 logits: the last tokens' rows lie past what 32 bits address."""
    E, k, T = 256, 8, (1 << 24) + 77
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(200, E, device="cuda").bfloat16()
    x[-200:] = tail
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, k, device="cuda")
    load = torch.zeros(E, dtype=torch.int32, device="cuda")
    r = _router(E, k, ref.SIGMOID, 8, 4, True, True, 2.5)
    mok.mok_route_scored(r, x, T, idx, gate, load=load)
    ri, rg, _ = ref.route(tail.double().cpu().numpy(), ref.SIGMOID, k, None, 8, 4, True, True, 2.5)
    assert np.array_equal(idx[-200:].cpu().numpy(), ri)
    assert bool((idx[: T - 200] == torch.arange(k, device="cuda")).all())
    assert int(load.long().sum()) == T * k
    dg = torch.randn(T, k, device="cuda")
    mok.mok_route_scored_backward(r, x, T, idx, dg, x2 := torch.empty_like(x))
    want, size = ref.route_backward(tail.double().cpu().numpy(), ref.SIGMOID, ri, dg[-200:].double().cpu().numpy(), True, 2.5)
    bar = 300 * 2.0 ** -24 * size
    assert np.all(np.abs(x2[-200:].double().cpu().numpy() - want) <= bar + 2.0 ** -8 * (np.abs(want) + bar) + 1e-30)


def test_route_on_a_side_stream_and_replayed_from_a_graph():
    T, E, k = 300, 256, 8
    x = torch.randn(T, E, device="cuda")
    bias = 0.1 * torch.randn(E, device="cuda")
    r = _router(E, k, ref.SIGMOID, 8, 4, True, True, 2.5)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, k, device="cuda")
    load = torch.zeros(1, E, dtype=torch.int32, device="cuda")
    dg, dl = torch.randn(T, k, device="cuda"), torch.empty(T, E, device="cuda")

    def step():
        mok.mok_route_scored(r, x, T, idx, gate, bias=bias, load=load)
        mok.mok_route_scored_backward(r, x, T, idx, dg, dl)
        mok.mok_route_bias_update(load, 1, E, 1e-3, bias, clear_load=1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    bias0 = bias.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for replay in range(4):
        x.copy_(torch.randn(T, E, device="cuda"))
        bias.copy_(bias0)
        load.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (idx, gate, dl, bias)]
        bias.copy_(bias0)
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (idx, gate, dl, bias))), replay
        ri, _, rl = ref.route(x.double().cpu().numpy(), ref.SIGMOID, k, bias0.cpu().numpy(), 8, 4, True)
        assert np.array_equal(idx.cpu().numpy(), ri)
        want = bias0.cpu().numpy() + np.float32(1e-3) * np.sign(rl.sum() - E * rl).astype(np.float32)
        assert np.array_equal(bias.cpu().numpy(), want)


@pytest.mark.parametrize("T", [300, 2100])
@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("base,n_local", [(0, 16), (5, 8)])
def test_fused_layer_with_the_scored_route(mode, base, n_local, T):
    """mok_moe_forward_scored is mok_route_scored followed by mok_moe_forward_routed, bit for bit, with rows that
    pick fewer than k experts or none."""
    wl = W.logits_workload("scored", 31, T=T, H=256, I=128, E=16, k=4, x_std=1.0, w_std=0.02, expert_base=base,
                           n_local=n_local, n_partitions=3)
    dw = DeviceWorkload(wl)
    logits = dw.logits.clone()
    logits[::7, 3:] = -float("inf")
    logits[50:60] = float("nan")
    bias = 0.1 * torch.randn(16, device="cuda")
    r = _router(16, 4, ref.SIGMOID, 4, 2, True, True, 2.5)
    idx = torch.empty(T, 4, dtype=torch.int32, device="cuda")
    gate = torch.empty(T, 4, device="cuda")
    load = torch.zeros(16, dtype=torch.int32, device="cuda")
    mok.mok_route_scored(r, logits, T, idx, gate, bias=bias, load=load)
    d = dw.desc(mode=mode)
    ws = torch.empty(mok.mok_forward_workspace_size(d, T, 1), dtype=torch.uint8, device="cuda")
    want, got, inside = dw.outs[0], dw.new_out(), dw.new_out()
    mok.mok_moe_forward_routed(d, idx, gate, T, dw.x, dw.w_gu, dw.w_d, want, ws)
    assert mok.mok_device_status(ws) == 0
    idx2, gate2, load2 = torch.empty_like(idx), torch.empty_like(gate), torch.zeros_like(load)
    mok.mok_moe_forward_scored(d, r, logits, T, dw.x, dw.w_gu, dw.w_d, got, ws, bias=bias, topk_idx=idx2,
                               topk_gate=gate2, load=load2)
    assert mok.mok_device_status(ws) == 0
    mok.mok_moe_forward_scored(d, r, logits, T, dw.x, dw.w_gu, dw.w_d, inside, ws, bias=bias)
    assert mok.mok_device_status(ws) == 0
    assert torch.equal(idx, idx2) and torch.equal(gate, gate2) and torch.equal(load, load2)
    rows = dw.out_rows(want)
    assert np.array_equal(rows, dw.out_rows(got)) and np.array_equal(rows, dw.out_rows(inside))
    picks = idx.cpu().numpy()
    local = ((picks >= base) & (picks < base + n_local)).any(1)
    assert np.all(rows[~local] == SENTINEL) and not local[50:60].any() and not np.any(rows[local] == SENTINEL)


def test_one_training_step_of_the_share():
    """The calls of a training step in a row: scored route inside the layer, the layer's backward down to dgate,
    the route's backward, the bias update, the weight gradients and AdamW over experts and router."""
    wl = W.logits_workload("step", 32, T=256, H=256, I=128, E=16, k=4, x_std=1.0, w_std=0.02, n_partitions=2)
    dw = DeviceWorkload(wl)
    T, H, I, E, k = 256, 256, 128, 16, 4
    r = _router(E, k, ref.SIGMOID, 4, 2, True, True, 2.5)
    bias, load = torch.zeros(E, device="cuda"), torch.zeros(E, dtype=torch.int32, device="cuda")
    idx, gate = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    x = torch.cat(dw.x_parts).view(torch.bfloat16)
    w_router = 0.05 * torch.randn(E, H, device="cuda")
    logits = x.float() @ w_router.t()
    d = dw.desc()
    mok.mok_route_scored(r, logits, T, idx, gate, bias=bias, load=load)
    s = dw.schedule(idx)
    R = int(s["offsets"][-1])
    assert R == T * k
    ring = torch.zeros((R, H), dtype=torch.int16, device="cuda")
    mok.mok_dispatch_gather(dw.x, H, k, s["aos"], s["offsets"], E, 0, R, ring, None, R, mok.MOK_ACT_BF16)
    act, y = torch.zeros((R, I), dtype=torch.int16, device="cuda"), torch.zeros((R, H), dtype=torch.int16, device="cuda")
    mok.mok_expert_ffn(d, ring, None, R, s["offsets"], 0, R, dw.w_gu, dw.w_d, act, None, R, y, R)
    dout_t = torch.randn(T, H, device="cuda").bfloat16()
    dout = mok.Tokens([dout_t[:128], dout_t[128:]], 128)
    dy, dgate = torch.zeros((R, H), dtype=torch.int16, device="cuda"), torch.zeros(T, k, device="cuda")
    mok.mok_combine_backward(dout, y, R, s["aos"], s["offsets"], E, R, gate, k, H, dy, R, dgate)
    gu_b, d_b = mok.mok_packed_weights_bwd_size(d)
    gu_t, d_t = torch.empty(gu_b, dtype=torch.uint8, device="cuda"), torch.empty(d_b, dtype=torch.uint8, device="cuda")
    mok.mok_pack_weights_bwd(d, dw.w_gu, dw.w_d, gu_t, d_t)
    h, dh = (torch.zeros((R, 2 * I), dtype=torch.int16, device="cuda") for _ in range(2))
    dxs = torch.zeros((R, H), dtype=torch.int16, device="cuda")
    mok.mok_expert_ffn_backward(d, ring, R, dy, s["offsets"], 0, R, dw.w_gu, gu_t, d_t, h, dh, dxs, R)
    dwgu, dwd = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device="cuda"), torch.zeros((E, H, I), dtype=torch.bfloat16, device="cuda")
    wws = torch.empty(mok.mok_wgrad_workspace_size(d, R), dtype=torch.uint8, device="cuda")
    mok.mok_expert_wgrad(d, ring, R, act, R, dy, dh, R, s["offsets"], dwgu, dwd, wws)
    dlogits = torch.empty(T, E, device="cuda")
    mok.mok_route_scored_backward(r, logits, T, idx, dgate, dlogits)
    mok.mok_route_bias_update(load, 1, E, 1e-3, bias, clear_load=1)
    dw_router = dlogits.t() @ x.float()
    master = {"gu": dw.w_gu.view(torch.bfloat16).float(), "d": dw.w_d.view(torch.bfloat16).float(), "r": w_router}
    grads = {"gu": dwgu, "d": dwd, "r": dw_router}
    copies = {"gu": dw.w_gu.view(torch.bfloat16), "d": dw.w_d.view(torch.bfloat16), "r": None}
    before = {n: (master[n].double().cpu().numpy().ravel(), grads[n].double().cpu().numpy().ravel()) for n in master}
    old = mok.AdamwTensors([dict(p=master[n], grad=grads[n], p_bf16=copies[n], m=torch.zeros_like(master[n]),
                                 v=torch.zeros_like(master[n]), weight_decay=0.1) for n in master])
    mok.mok_adamw_step(old, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1)
    torch.cuda.synchronize()
    # the chain's ends: the routing's gradient from the device's own dgate, the first AdamW step from its own gradients
    want, size = ref.route_backward(logits.double().cpu().numpy(), ref.SIGMOID, to_host(idx), dgate.double().cpu().numpy(), True, 2.5)
    bar = 300 * 2.0 ** -24 * size + 1e-30
    assert np.all(np.abs(dlogits.double().cpu().numpy() - want) <= bar)
    assert bool((dgate != 0).any()) and bool((dlogits != 0).any())
    picked = np.bincount(to_host(idx).ravel(), minlength=E)
    assert np.array_equal(to_host(bias), np.float32(1e-3) * np.sign(picked.sum() - E * picked).astype(np.float32))
    assert int(load.abs().sum()) == 0
    hyper = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=1, grad_scale=1.0)
    for n in master:
        p0, g0 = before[n]
        p, _, _, _ = ref.adamw(p0, g0, 0 * p0, 0 * p0, hyper, weight_decay=0.1)
        got = master[n].double().cpu().numpy().ravel()
        # p keep and the update: 3 roundings of p, 16 of an update of at most lr (step 1: m / sqrt(v) is the sign)
        assert np.all(np.abs(got - p) <= 3 * 2.0 ** -24 * np.abs(p0) + 16 * 2.0 ** -24 * 1.1e-3), n
        if copies[n] is not None:
            assert torch.equal(copies[n], master[n].bfloat16())
