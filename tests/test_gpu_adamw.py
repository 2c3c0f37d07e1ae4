"""GPU tests of the AdamW step against the forms of tests/scored_reference.py.

8-bit states: codes and scales are equal to those from fp32 values formed by
the same operations, and lie within one quantum of the 64-bit state.  fp32:
m and v within three roundings of the magnitudes that are added; p within two
roundings of p and, of the update, 16 roundings (two for m / (r / sqrt(bc2) +
eps)'s operands each, one for every operation) plus what the error of m, seen
against |m|'s terms, makes of it.
"""
import numpy as np
import pytest
import torch

import scored_reference as ref
import token_dispatch_grouped_top_amd as mok

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=7, grad_scale=0.5)


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def _make(rng, n, states, grads, copy, offset=0):
    """Host arrays and device tensors of one tensor; offset: elements that the device views begin behind an allocation."""
    def dev(a, dtype):
        t = torch.zeros(n + offset, dtype=dtype, device="cuda")
        t[offset:] = torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()
        return t[offset:]
    t = dict(p=dev(rng.normal(size=n), torch.float32),
             grad=dev(rng.normal(size=n) * 1e-2, torch.bfloat16 if grads == "bf16" else torch.float32))
    m, r = (rng.normal(size=n) * 1e-2).astype(np.float32), (rng.random(n) * 1e-2).astype(np.float32)
    if n > 40:
        m[32:64], r[32:64] = 0, 0                    # a block of zeros
    if states == "8bit":
        b = np.full(n, 1 << 15)
        ms, rs = ref.scale_byte(m), ref.scale_byte(r)
        t["m"], t["v"] = dev(ref.encode_m(m, b, ms), torch.uint8), dev(ref.encode_r(r, b, rs), torch.uint8)
        t["m_scale"], t["v_scale"] = torch.from_numpy(ms).cuda(), torch.from_numpy(rs).cuda()
    else:
        t["m"], t["v"] = dev(m, torch.float32), dev(r * r, torch.float32)
    if copy:
        t["p_bf16"] = dev(np.zeros(n), torch.bfloat16)
    return t


def _host(t):
    return {k: (x.float() if x.dtype == torch.bfloat16 else x).cpu().numpy() for k, x in t.items()
            if isinstance(x, torch.Tensor)}


def _check(before, t, number, h, lr_scale=1.0, weight_decay=0.0, seed=0):
    n = len(before["p"])
    after = _host(t)
    coded = before["m"].dtype == np.uint8
    m0, v0 = before["m"], before["v"]
    if coded:
        m0, r0 = ref.decode(m0, before["m_scale"]), ref.decode(v0, before["v_scale"])
        v0 = (r0.astype(np.float32) * r0.astype(np.float32))
    _, m32, v32, r32 = ref.adamw(before["p"], before["grad"], m0, v0, h, lr_scale, weight_decay, np.float32)
    p, m, v, r = ref.adamw(before["p"], before["grad"], m0, v0, h, lr_scale, weight_decay)
    g = np.abs(before["grad"].astype(np.float64) * h["grad_scale"])
    em = 3 * U * (h["beta1"] * np.abs(m0) + (1 - h["beta1"]) * g) + 1e-44
    if coded:
        bm, br = ref.random_bits(np.arange(n), number, h["step"], seed)
        ms, rs = ref.scale_byte(m32), ref.scale_byte(r32)
        assert np.array_equal(after["m_scale"], ms) and np.array_equal(after["v_scale"], rs)
        assert np.array_equal(after["m"], ref.encode_m(m32, bm, ms))
        assert np.array_equal(after["v"], ref.encode_r(r32, br, rs))
        for code, scale, x in ((after["m"], ms, m), (after["v"], rs, r)):
            unit = np.exp2(ref.per_value(scale.astype(np.float64) - 127, n))
            quantum = np.maximum(np.abs(x) / 8, 2.0 ** -9 * unit)
            # v is held in fp32: below 2^-150 it rounds to 0, and r with it, which is then off by at most 2^-75
            assert np.all(np.abs(ref.decode(code, scale) - x) <= quantum * (1 + 1e-6) + 2.0 ** -75)
    else:
        assert np.all(np.abs(after["m"] - m) <= em)
        assert np.all(np.abs(after["v"] - v) <= 4 * U * v + 1e-44)
    rate = h["lr"] * lr_scale / (1 - h["beta1"] ** h["step"])
    denom = r / np.sqrt(1 - h["beta2"] ** h["step"]) + h["eps"]
    bar = 3 * U * np.abs(before["p"]) + rate * (16 * U * np.abs(m) + em) / denom + 1e-44
    assert np.all(np.abs(after["p"] - p) <= bar), float((np.abs(after["p"] - p) / bar).max())
    if "p_bf16" in after:
        assert torch.equal(t["p_bf16"], t["p"].bfloat16())


@pytest.mark.parametrize("states", ["f32", "8bit"])
@pytest.mark.parametrize("grads", ["f32", "bf16"])
def test_step_matches_reference(states, grads):
    rng = np.random.default_rng(1)
    for n in (1, 2, 3, 31, 32, 33, 64, 127, 1023, 4096, 4097, 8200, 40001):
        for copy in (False, True):
            for offset in (0, 1, 4):
                if states == "8bit" and n > 9000 and offset:
                    continue
                t = _make(rng, n, states, grads, copy, offset)
                before = _host(t)
                t["weight_decay"], t["lr_scale"] = 0.1, 0.25
                print(f"[adamw] {states} {grads} n={n} copy={copy} offset={offset}", flush=True)
                mok.mok_adamw_step(mok.AdamwTensors([t]), seed=9, **HYPER)
                _check(before, t, 0, HYPER, 0.25, 0.1, 9)


@pytest.mark.parametrize("device_scalars", [False, True])
def test_many_tensors_of_mixed_kinds(device_scalars):
    """More tensors than one launch takes, of both state formats, empty ones among them."""
    rng = np.random.default_rng(2)
    ts = []
    for i in range(120):
        t = _make(rng, int(rng.integers(1, 6000)), ("f32", "8bit")[i % 2], ("f32", "bf16")[i // 2 % 2], i % 3 == 0)
        t["weight_decay"] = 0.1 if i % 5 else 0.0
        ts.append(t)
    empty = {k: torch.empty(0, device="cuda") for k in ("p", "grad", "m", "v")}
    ts.insert(7, empty)
    before = [_host(t) for t in ts]
    scalars = None
    h = dict(HYPER)
    if device_scalars:
        scalars = torch.zeros(4, device="cuda")
        scalars[0], scalars[1] = 2e-3, 0.25
        scalars.view(torch.int32)[2] = 19
        h.update(lr=float(np.float32(2e-3)), grad_scale=0.25, step=19)
    mok.mok_adamw_step(mok.AdamwTensors(ts), scalars=scalars, seed=4, **HYPER)
    for i, t in enumerate(ts):
        if t is not empty:
            _check(before[i], t, i, h, 1.0, t["weight_decay"], 4)


def test_skip_leaves_everything():
    rng = np.random.default_rng(3)
    ts = [_make(rng, 5000, s, "bf16", True) for s in ("f32", "8bit")]
    before = [_host(t) for t in ts]
    lst = mok.AdamwTensors(ts)
    for step, skip in ((5, 1), (0, 0), (-2, 0)):
        scalars = torch.zeros(4, device="cuda")
        scalars[0] = scalars[1] = 1.0
        scalars.view(torch.int32)[2:] = torch.tensor([step, skip], dtype=torch.int32, device="cuda")
        mok.mok_adamw_step(lst, scalars=scalars, **HYPER)
        for b, t in zip(before, ts):
            a = _host(t)
            assert all(np.array_equal(a[k], b[k]) for k in b)


def test_values_that_are_not_finite():
    """A NaN or infinite gradient spoils its own element, not its block."""
    rng = np.random.default_rng(4)
    for states in ("f32", "8bit"):
        t = _make(rng, 300, states, "f32", False)
        t["grad"][5], t["grad"][70], t["grad"][71] = float("nan"), float("inf"), -float("inf")
        before = _host(t)
        mok.mok_adamw_step(mok.AdamwTensors([t]), seed=1, **HYPER)
        after = _host(t)
        bad = np.isin(np.arange(300), (5, 70, 71))
        if states == "8bit":
            assert np.all(after["m"][bad] == 0x7F) and np.all(after["v"][bad] == 0x7F)
            assert not np.any((after["m"][~bad] & 127) == 127) and not np.any((after["v"][~bad] & 127) == 127)
        else:
            assert np.all(~np.isfinite(after["m"][bad])) and np.all(np.isfinite(after["m"][~bad]))
        assert np.all(np.isfinite(after["p"][~bad])) and np.all(np.isnan(after["p"][bad]))
        assert np.all(after["p"][~bad] != before["p"][~bad])


def test_tiny_and_huge_gradients():
    """Blocks at both ends of the scales, a value far below its block's largest: r > 0 never becomes 0."""
    n = 96
    g = np.full(n, 1e-15)
    g[:32] = 1e-25
    g[0] = 0.0
    g[64:] = 1e15
    g[64] = 1e-6
    t = dict(p=torch.zeros(n, device="cuda"), grad=torch.from_numpy(g).float().cuda(),
             m=torch.zeros(n, dtype=torch.uint8, device="cuda"), v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
             m_scale=torch.zeros(3, dtype=torch.uint8, device="cuda"), v_scale=torch.zeros(3, dtype=torch.uint8, device="cuda"))
    before = _host(t)
    h = dict(HYPER, grad_scale=1.0)
    mok.mok_adamw_step(mok.AdamwTensors([t]), seed=3, **h)
    _check(before, t, 0, h, seed=3)
    v = t["v"].cpu().numpy()
    assert np.all(v[:32] == 0) and np.all(v[32:] > 0)       # (1e-25)^2 is 0 in fp32; 1e-15 and 1e-6 are not


def test_states_keep_their_mean_over_many_steps():
    """With beta2 = 0.999 a step moves r by a fraction of a quantum.  The states in 8 bits follow those in fp32: the
    mean over the elements of m and of v / E[g^2].  A rounding's deviation is at most half a quantum, a quarter of
    v at most in the square, in a step a share of at most |g^2 / v - 1| / 1000 of the elements moves by a quantum:
    the deviation of v stays below its own size, so the mean over 2^16 elements is within 6 / 256 of it."""
    n = 1 << 16
    torch.manual_seed(0)
    def state(dt):
        return torch.zeros(n, dtype=dt, device="cuda")
    a = dict(p=state(torch.float32), grad=state(torch.float32), m=state(torch.float32), v=state(torch.float32))
    b = dict(p=state(torch.float32), grad=a["grad"], m=state(torch.uint8), v=state(torch.uint8),
             m_scale=torch.zeros(n // 32, dtype=torch.uint8, device="cuda"), v_scale=torch.zeros(n // 32, dtype=torch.uint8, device="cuda"))
    lst = mok.AdamwTensors([a, b])
    for step in range(1, 301):
        size = 1.0 if step <= 100 else 2.0               # the gradients grow: v has to follow
        a["grad"].copy_(size * torch.randn(n, device="cuda") + 0.5)
        mok.mok_adamw_step(lst, lr=0.0, beta1=0.9, beta2=0.999, eps=1e-8, step=step, seed=5)
    host = _host(b)
    m, r = ref.decode(host["m"], host["m_scale"]), ref.decode(host["v"], host["v_scale"])
    am, av = a["m"].double().cpu().numpy(), a["v"].double().cpu().numpy()
    assert abs((r * r).mean() / av.mean() - 1) < 6 / 256
    assert abs(m.mean() - am.mean()) < 6 / 256 * np.abs(am).mean() * 2


def test_replayed_from_a_graph():
    """A captured step reads its learning rate and step number anew, on each replay."""
    rng = np.random.default_rng(6)
    ts = [_make(rng, 9001, s, "bf16", True) for s in ("f32", "8bit")]
    twin = [{k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in t.items()} for t in ts]
    scalars = torch.zeros(4, device="cuda")
    scalars[0], scalars[1] = 1e-3, 1.0
    lst, other = mok.AdamwTensors(ts), mok.AdamwTensors(twin)
    kw = dict(lr=0.0, beta1=0.9, beta2=0.99, eps=1e-8, step=1, seed=8, scalars=scalars)
    graph = torch.cuda.CUDAGraph()
    scalars.view(torch.int32)[2] = 0                     # the capture itself runs nothing
    with torch.cuda.graph(graph):
        mok.mok_adamw_step(lst, **kw)
    for step in range(1, 5):
        scalars[0] = 1e-3 / step
        scalars.view(torch.int32)[2] = step
        grad = torch.randn(9001, device="cuda").bfloat16()
        for t in (*ts, *twin):
            t["grad"].copy_(grad)
        graph.replay()
        torch.cuda.synchronize()
        mok.mok_adamw_step(other, **kw)
        torch.cuda.synchronize()
        for t, u in zip(ts, twin):
            assert all(torch.equal(t[k], u[k]) for k in t), step


def test_elements_past_32_bits():
    """One tensor of more than 2^32 elements: the last ones' offsets and random bits need all 64."""
    n = (1 << 32) + 4101
    tail = 9000
    t = dict(p=torch.zeros(n, device="cuda"), grad=torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
             m=torch.zeros(n, dtype=torch.uint8, device="cuda"), v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
             m_scale=torch.zeros((n + 31) // 32, dtype=torch.uint8, device="cuda"),
             v_scale=torch.zeros((n + 31) // 32, dtype=torch.uint8, device="cuda"))
    t["grad"][-tail:] = torch.randn(tail, device="cuda").bfloat16()
    begin = n - tail
    h = dict(HYPER, grad_scale=1.0)
    mok.mok_adamw_step(mok.AdamwTensors([t]), seed=2, **h)
    g = t["grad"][-tail:].float().cpu().numpy()
    z = np.zeros(tail)
    p, _, _, _ = ref.adamw(z, g, z, z, h)
    _, m32, v32, r32 = ref.adamw(z, g, z, z, h, dtype=np.float32)
    assert np.all(np.abs(t["p"][-tail:].cpu().numpy() - p) <= 40 * U * np.abs(p) + 1e-30)
    lead = -begin % 32                                   # blocks of 32 from the tensor's begin
    bm, br = ref.random_bits(begin + lead + np.arange(tail - lead, dtype=np.uint64), 0, h["step"], 2)
    ms, rs = ref.scale_byte(m32[lead:]), ref.scale_byte(r32[lead:])
    assert np.array_equal(t["m"][-tail + lead:].cpu().numpy(), ref.encode_m(m32[lead:], bm, ms))
    assert np.array_equal(t["v"][-tail + lead:].cpu().numpy(), ref.encode_r(r32[lead:], br, rs))
    assert float(t["p"][:begin].abs().max()) == 0.0
