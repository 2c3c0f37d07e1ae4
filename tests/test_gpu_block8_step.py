"""The 8-bit block operands and the Muon step as a training step of an expert share uses them, after the schedule and the
gather of the layer; captured and replayed, and on side streams.

The step's parts are compared with the same formulas in 64 bits on what the parts before them wrote, so each tolerance is
that of one part: products as in test_gpu_block8.py, the update by orthogonalised() below.
"""
import numpy as np
import pytest
import torch

import block8_reference as ref
import token_dispatch_grouped_top_amd as mok

pytestmark = pytest.mark.gpu
H, I, E, k, T = 256, 192, 6, 2, 300
BLOCKS, LINES = mok.MOK_BLOCK8_BLOCKS, mok.MOK_BLOCK8_LINES


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def host(t):
    return t.cpu().numpy()


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda")


def f32(*shape):
    return torch.zeros(*shape, device="cuda")


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")


def orthogonalised(v):
    """The update of a gradient with fewer rows than its matrix has, so of low rank, and the bound of its error's 2-norm.

    A step p(s) = a s + b s^3 + c s^5 carries an error on by its divided differences (p(s) -+ p(t)) / (s -+ t): at most the
    largest |p'|, which is a, or |p'| at the largest s.  Directions outside the gradient's range, s = 0, are carried by a
    itself each time, 485 over five steps, so that 2^-11 of an X of norm 1 comes out as 0.24.  What a step adds is
    block8_reference.orthogonalise's: the roundings of X, G and B to 11 bits."""
    (a, b, c), u = mok.NEWTON_SCHULZ, 2.0 ** -11
    x = v / np.linalg.norm(v)
    x = x.T if x.shape[0] > x.shape[1] else x
    e = u
    for _ in range(5):
        s, r, gram = np.linalg.norm(x, 2), np.linalg.norm(x), x @ x.T
        e = e * max(a, abs(a + 3 * b * s ** 2 + 5 * c * s ** 4))
        e += u * s * s * r * (2 * abs(b) + 3 * abs(c) * s ** 2)
        x = a * x + (b * gram + c * gram @ gram) @ x
        e += u * np.linalg.norm(x)
    return (x if x.shape == v.shape else x.T), e


class Operand:
    """Rows as a token operand, and their slot blocks."""

    def __init__(self, rows, W, kind):
        S = mok.mok_block8_slots(rows, E)
        self.rows, self.W, self.kind = rows, W, kind
        self.codes, self.scales = u8(rows, W), f32(ref.blocks(W), rows)
        self.codes_t = u8(W, S)
        self.scales_t = f32(S // 128, W) if kind == LINES else f32(ref.blocks(W), S // 128)

    def quantise(self, x, offsets, **kw):
        mok.mok_block8_quantise(x, self.rows, self.W, self.codes, self.scales, codes_t=self.codes_t,
                                scales_t=self.scales_t, t_scales=self.kind, offsets=offsets, n_local=E, **kw)


class Weights:
    def __init__(self, N, K):
        self.N, self.K = N, K
        self.codes, self.scales = u8(E, N, K), f32(E, ref.blocks(N), ref.blocks(K))
        self.codes_t, self.scales_t = u8(E, K, N), f32(E, ref.blocks(K), ref.blocks(N))

    def quantise(self, w):
        mok.mok_block8_quantise_weights(w, E, self.N, self.K, self.codes, self.scales, self.codes_t, self.scales_t)


class Step:
    """Forward, backward and update of the experts' matrices for tokens routed to them."""

    def __init__(self, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        R = self.R = T * k
        self.x, self.dout = normal(T, H).bfloat16(), (1e-2 * normal(T, H)).bfloat16()
        self.idx = torch.stack([torch.randperm(E, generator=gen, device="cuda")[:k] for _ in range(T)]).int()
        self.idx[:, 0][self.idx[:, 0] == 3] = 2          # an expert with few tokens
        self.gate = torch.rand(T, k, generator=gen, device="cuda")
        self.w = dict(gu=normal(E, 2 * I, H) * H ** -0.5, d=normal(E, H, I) * I ** -0.5)
        self.m = {n: torch.zeros_like(w) for n, w in self.w.items()}
        self.dw = {n: torch.zeros_like(w) for n, w in self.w.items()}
        self.q = dict(gu=Weights(2 * I, H), d=Weights(H, I))
        self.ws = torch.empty(max(mok.mok_muon_workspace_size(E, 2 * I, H), mok.mok_muon_workspace_size(E, H, I)),
                              dtype=torch.uint8, device="cuda")
        i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.counts, self.offsets, self.soa, self.aos = i32(E), i32(E + 1), i32(R), i32(R)
        self.sched_ws = torch.zeros(mok.mok_schedule_workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
        self.tokens, self.douts = mok.Tokens.from_tensor(self.x), mok.Tokens.from_tensor(self.dout)
        self.ring, self.dy, self.dgate = bf16(R, H), bf16(R, H), f32(T, k)
        self.xq, self.aq = Operand(R, H, BLOCKS), Operand(R, I, BLOCKS)
        self.dyq, self.dhq = Operand(R, H, LINES), Operand(R, 2 * I, LINES)
        self.h, self.y, self.da, self.dx = bf16(R, 2 * I), bf16(R, H), bf16(R, I), bf16(R, H)
        self.out, self.dx_tokens = bf16(T, H), bf16(T, H)
        self.out_t, self.dx_t = mok.Tokens.from_tensor(self.out), mok.Tokens.from_tensor(self.dx_tokens)

    def run(self):
        R, off, q = self.R, self.offsets, self.q
        for n in q:
            q[n].quantise(self.w[n])
        mok.mok_build_schedule(self.idx, T, k, 0, E, self.counts, off, self.soa, self.aos, self.sched_ws)
        mok.mok_dispatch_gather(self.tokens, H, k, self.aos, off, E, 0, R, self.ring, None, R, mok.MOK_ACT_BF16)
        self.xq.quantise(self.ring, off, ring_rows=R)
        mok.mok_block8_gemm(self.xq.codes, self.xq.scales, R, H, q["gu"].codes, q["gu"].scales, 2 * I, self.h, off, E)
        self.aq.quantise(self.h, off, source=mok.MOK_BLOCK8_SWIGLU)
        mok.mok_block8_gemm(self.aq.codes, self.aq.scales, R, I, q["d"].codes, q["d"].scales, H, self.y, off, E)
        mok.mok_combine_slots(self.y, R, self.aos, off, E, R, self.soa, self.gate, k, H, self.out_t)
        # backward
        mok.mok_combine_backward(self.douts, self.y, R, self.aos, off, E, R, self.gate, k, H, self.dy, R, self.dgate)
        self.dyq.quantise(self.dy, off, ring_rows=R)
        mok.mok_block8_gemm(self.dyq.codes, self.dyq.scales, R, H, q["d"].codes_t, q["d"].scales_t, I, self.da, off, E)
        self.dhq.quantise(self.h, off, source=mok.MOK_BLOCK8_SWIGLU_BWD, d=self.da)
        mok.mok_block8_gemm(self.dhq.codes, self.dhq.scales, R, 2 * I, q["gu"].codes_t, q["gu"].scales_t, H, self.dx, off, E)
        mok.mok_dispatch_backward(self.dx, R, self.aos, off, E, R, self.soa, k, H, self.dx_t)
        wgrad = lambda dy, x, dw: mok.mok_block8_wgrad(dy.codes_t, dy.scales_t, dy.W, x.codes_t, x.scales_t, x.W, R, dw,  # noqa: E731
                                                       off, E)
        wgrad(self.dyq, self.aq, self.dw["d"])
        wgrad(self.dhq, self.xq, self.dw["gu"])
        for n, (rows, cols) in dict(gu=(2 * I, H), d=(H, I)).items():
            mok.mok_muon_step(self.w[n], self.dw[n], self.m[n], E, rows, cols, self.ws, lr=1e-2, momentum=0.9,
                              scale=0.2 * max(rows, cols) ** 0.5, weight_decay=0.01)

    def results(self):
        return [self.out, self.dx_tokens, self.dgate, *self.dw.values(), *self.w.values(), *self.m.values()]


def test_training_step():
    s = Step(1)
    before = {n: host(w).astype(np.float64) for n, w in s.w.items()}
    s.run()
    torch.cuda.synchronize()
    counts = host(s.counts).tolist()
    assert sum(counts) == s.R and min(counts) > 0

    def operand(o):
        return host(o.codes), host(o.scales)

    def check(got, operands, counts, w, sw, K):
        a, sa = operands
        want, size = ref.product(a, sa, counts, host(w), host(sw))
        size = size * (K + 2) * 2.0 ** -23 + ref.product(a, sa, counts, host(w), host(sw), drop=True)[1]
        assert np.all(np.abs(host(got.float()) - want) <= size + 2.0 ** -8 * np.abs(want))

    q = s.q
    check(s.h, operand(s.xq), counts, q["gu"].codes, q["gu"].scales, H)
    check(s.y, operand(s.aq), counts, q["d"].codes, q["d"].scales, I)
    check(s.da, operand(s.dyq), counts, q["d"].codes_t, q["d"].scales_t, H)
    check(s.dx, operand(s.dhq), counts, q["gu"].codes_t, q["gu"].scales_t, 2 * I)
    # the operands hold what they were made of: half a step of a code (2^-4 of the value, or of the smallest normal one)
    rows = torch.arange(s.R, device="cuda")
    slot_tokens = s.x[(s.aos // k).long()]
    for o, x in ((s.xq, slot_tokens), (s.dyq, None)):
        a, sa = operand(o)
        v = ref.values(a) * np.repeat(sa.astype(np.float64).T, 128, 1)[:, :o.W]
        if x is None:
            x = (s.dout[(s.aos // k).long()].float() * s.gate.view(-1)[s.aos.long()][:, None]).bfloat16()[rows]
        x = host(x.float()).astype(np.float64)
        each = np.repeat(sa.astype(np.float64).T, 128, 1)[:, :o.W]
        assert np.all(np.abs(v - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * each)
    for n, dy, x in (("d", s.dyq, s.aq), ("gu", s.dhq, s.xq)):
        want, size = ref.wgrad(host(dy.codes_t), host(dy.scales_t), host(x.codes_t), host(x.scales_t), counts)
        assert np.all(np.abs(host(s.dw[n]) - want) <= (max(counts) + 130) * 2.0 ** -23 * size + 2.0 ** -24 * np.abs(want))
        g = host(s.dw[n]).astype(np.float64)
        assert np.array_equal(host(s.m[n]), host(s.dw[n]))   # the first step's momentum is the gradient
        w = host(s.w[n]).astype(np.float64)
        for e in range(E):
            o, e_o = orthogonalised(1.9 * g[e])
            step = 1e-2 * 0.2 * max(o.shape) ** 0.5
            want = before[n][e] * (1 - 1e-2 * 0.01) - step * o
            assert np.linalg.norm(w[e] - want) <= 2.0 ** -22 * np.linalg.norm(want) + step * e_o


def test_gradients_against_differences():
    """The weight gradients of a linear loss along a direction, against the difference of the loss: the operands' rounding
    (2^-4 each way of every value, of random sign) leaves a few percent, far from a wrong or missing term."""
    s = Step(2)
    s.run()
    x, idx, gate = s.x.double(), s.idx.long(), s.gate.double()
    s2 = Step(2)                                          # the weights before the step
    w = {n: t.double() for n, t in s2.w.items()}

    def loss(w):
        total = 0
        for j in range(k):
            for e in range(E):
                rows = (idx[:, j] == e).nonzero().flatten()
                hh = x[rows] @ w["gu"][e].T.contiguous()
                g, u = hh[:, :I], hh[:, I:]
                y = (g * torch.sigmoid(g) * u) @ w["d"][e].T.contiguous()
                total = total + (gate[rows, j, None] * y * s.dout.double()[rows]).sum()
        return total

    for n in w:
        d = s.dw[n].double()
        d = d / d.norm()
        eps = 1e-4
        up, down = ({**w, n: w[n] + e * d} for e in (eps, -eps))
        slope = (loss(up) - loss(down)) / (2 * eps)
        assert abs(slope - s.dw[n].double().norm()) <= 0.1 * s.dw[n].double().norm()


def test_captured_and_replayed():
    """A step in a graph: every replay gives what the eager step gives from the same weights, with other work between."""
    eager, s = Step(3), Step(3)
    warm = Step(3)
    warm.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.run()
    for _ in range(4):
        eager.run()
        torch.cuda.synchronize()
        graph.replay()
        noise = torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        assert torch.isfinite(noise)
        assert all(torch.equal(a, b) for a, b in zip(eager.results(), s.results()))


def test_two_streams_at_once():
    """Steps on two side streams that run at the same time, each with its own buffers."""
    alone, steps = [Step(4), Step(5)], [Step(4), Step(5)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for a in alone:
            a.run()
        torch.cuda.synchronize()
        for stream, s in zip(streams, steps):
            with torch.cuda.stream(stream):
                s.run()
        torch.cuda.synchronize()
    for a, s in zip(alone, steps):
        assert all(torch.equal(x, y) for x, y in zip(a.results(), s.results()))


def test_stream_argument():
    """A call's stream argument: a torch stream or its handle, whatever the current one is."""
    x = torch.randn(300, 256, device="cuda").bfloat16()
    want = u8(300, 256), f32(2, 300)
    mok.mok_block8_quantise(x, 300, 256, *want)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (stream, stream.cuda_stream):
        got = u8(300, 256), f32(2, 300)
        torch.cuda.synchronize()
        mok.mok_block8_quantise(x, 300, 256, *got, stream=given)
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals_on_the_gpu():
    x, codes, scales = torch.zeros(4, 128, device="cuda"), u8(4, 128), f32(1, 4)
    with pytest.raises(ValueError, match="codes_t"):
        mok.mok_block8_quantise(x, 4, 128, codes, scales, codes_t=u8(4, 100), scales_t=f32(1, 128))
    with pytest.raises(ValueError, match="offsets"):
        mok.mok_block8_quantise(x, 4, 128, codes, scales, offsets=torch.zeros(2, dtype=torch.int32, device="cuda"), n_local=2)
    with pytest.raises(mok.MokError):
        mok.mok_block8_quantise(x, 4, 128, codes)         # codes without scales
    with pytest.raises(ValueError, match="d:"):
        mok.mok_block8_quantise(x, 4, 128, codes, scales, source=mok.MOK_BLOCK8_SWIGLU_BWD, d=torch.zeros(4, 64).cuda().half())
    with pytest.raises(mok.MokError):
        mok.mok_block8_gemm(codes, scales, 4, 128, u8(1, 64, 128), f32(1, 1, 1), 64, None)
    with pytest.raises(mok.MokError) as e:
        mok.mok_orthogonalise(x, 1, 4, 128, bf16(4, 128), u8(256))
    assert e.value.status == mok.MOK_ERR_WORKSPACE
    with pytest.raises(mok.MokError):
        mok.mok_block8_wgrad(u8(64, 128), f32(1, 64), 64, u8(64, 128), f32(1, 1), 64, 4, bf16(64, 64), accumulate=1)


def test_no_rows():
    """Nothing routed: the gradients are zero or stay, the rows' buffers are not touched."""
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    y = torch.full((8, 128), -7.0, device="cuda")
    codes, scales = u8(8, 128), f32(1, 8)
    mok.mok_block8_gemm(codes, scales, 8, 128, u8(E, 128, 128), f32(E, 1, 1), 128, y, off, E)
    q = Operand(8, 128, BLOCKS)
    for t in (q.codes, q.codes_t):
        t.fill_(9)
    q.quantise(torch.ones(8, 128, device="cuda"), off)
    assert (y == -7).all() and (q.codes == 9).all() and (q.codes_t == 9).all()
    S = mok.mok_block8_slots(8, E)
    dw = torch.full((E, 128, 64), 3.0, device="cuda")
    args = (u8(128, S), f32(S // 128, 128), 128, u8(64, S), f32(1, S // 128), 64, 8, dw, off, E)
    mok.mok_block8_wgrad(*args, accumulate=1)
    assert (dw == 3).all()
    mok.mok_block8_wgrad(*args)
    assert not dw.any()


def test_overlapping_runs_stay_inside():
    """Offsets that are no partition: every expert all of the rows.  Results are not defined; what lies behind the outputs
    stays, and the next call with a partition is right."""
    R, W = 260, 256
    bad = torch.tensor([0, R] * E, dtype=torch.int32, device="cuda")[:E + 1].contiguous()
    good = torch.tensor([R * e // E for e in range(E + 1)], dtype=torch.int32, device="cuda")
    S = mok.mok_block8_slots(R, E)
    x = torch.randn(R, W, device="cuda").bfloat16()
    sizes = dict(codes=R * W, codes_t=W * S)
    buf = {n: torch.full((v + 4096,), 9, dtype=torch.uint8, device="cuda") for n, v in sizes.items()}
    scales, scales_t = torch.full((2 * R + 1024,), 9.0, device="cuda"), torch.full((S // 128 * W + 1024,), 9.0, device="cuda")
    w, sw = u8(E, 128, W), torch.ones(E, 1, 2, device="cuda")
    y, dw = torch.full((R * 128 + 1024,), 9.0, device="cuda"), torch.full((E * W * W + 1024,), 9.0, device="cuda")
    tail = lambda: [buf["codes"][sizes["codes"]:], buf["codes_t"][sizes["codes_t"]:], scales[2 * R:],  # noqa: E731
                    scales_t[S // 128 * W:], y[R * 128:], dw[E * W * W:]]
    for off in (bad, good):
        mok.mok_block8_quantise(x, R, W, buf["codes"], scales, codes_t=buf["codes_t"], scales_t=scales_t,
                                t_scales=LINES, offsets=off, n_local=E)
        mok.mok_block8_gemm(buf["codes"], scales, R, W, w, sw, 128, y, off, E)
        mok.mok_block8_wgrad(buf["codes_t"], scales_t, W, buf["codes_t"], torch.ones(2, S // 128, device="cuda"), W, R, dw, off, E)
        torch.cuda.synchronize()
        assert all((t == 9).all() for t in tail())
    counts = (good[1:] - good[:-1]).tolist()
    want, size = ref.wgrad(host(buf["codes_t"][:W * S].view(W, S)), host(scales_t[:S // 128 * W].view(-1, W)),
                           host(buf["codes_t"][:W * S].view(W, S)), np.ones((2, S // 128), np.float32), counts)
    got = host(dw[:E * W * W].view(E, W, W))
    assert np.all(np.abs(got - want) <= (max(counts) + 130) * 2.0 ** -23 * size + 2.0 ** -24 * np.abs(want))
