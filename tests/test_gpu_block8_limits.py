"""Block operands at the ends of their ranges: 256 experts, no rows at all, buffers with more than 2^32 values."""
import numpy as np
import pytest
import torch

import block8_reference as ref
import token_dispatch_grouped_top_amd as mok
from test_gpu_block8 import FILL, KIND, dev, host, offsets_of, outputs, rows_like, small_codes

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    yield
    torch.cuda.empty_cache()


def counts_of(rng, n, rows):
    """Rows of n experts: some none, the last one some."""
    c = rng.multinomial(rows, rng.dirichlet(np.full(n, 0.3))).tolist()
    c[-1] += 3
    return c


@pytest.mark.parametrize("rows", [200, 5000])
def test_256_experts(rows):
    rng = np.random.default_rng(rows)
    n, W, N = 256, 192, 128
    counts = counts_of(rng, n, rows)
    rows = sum(counts)
    off = offsets_of(counts)
    x = rows_like(rng, rows, W, torch.bfloat16)
    for kind in ("line", "block"):
        out = outputs(rows, W, n, kind)
        mok.mok_block8_quantise(dev(x, torch.bfloat16), rows, W, out[0], out[1], codes_t=out[2], scales_t=out[3],
                                t_scales=KIND[kind], offsets=off, n_local=n)
        codes, scales = ref.rows_operand(x)
        codes_t, scales_t = ref.slot_operand(x, counts, kind, FILL)
        for got, want in zip(out, (codes, scales, codes_t, scales_t)):
            assert np.array_equal(host(got), want)
    a, w = small_codes(rng, rows, W), small_codes(rng, n, N, W)
    sa = np.exp2(rng.integers(-2, 3, (ref.blocks(W), rows))).astype(np.float32)
    sw = np.exp2(rng.integers(-2, 3, (n, 1, ref.blocks(W)))).astype(np.float32)
    want = torch.from_numpy(ref.product(a, sa, counts, w, sw)[0])
    S = ref.slots(rows, n)
    used = np.zeros(S, np.uint8)
    for c, at in zip(counts, ref.starts(counts)):
        used[at:at + c] = 1
    dy, xt = small_codes(rng, W, S) * used, small_codes(rng, N, S) * used
    sdy = np.exp2(rng.integers(-2, 3, (S // 128, W))).astype(np.float32)
    sx = np.exp2(rng.integers(-2, 3, (1, S // 128))).astype(np.float32)
    want_dw = torch.from_numpy(ref.wgrad(dy, sdy, xt, sx, counts)[0])
    for out in (torch.bfloat16, torch.float32):
        y = torch.full((rows, N), -7.0, dtype=out, device="cuda")
        mok.mok_block8_gemm(dev(a), dev(sa), rows, W, dev(w), dev(sw), N, y, offsets=off, n_local=n)
        assert torch.equal(y.cpu(), want.to(out))
        dw = torch.full((n, W, N), -7.0, dtype=out, device="cuda")
        mok.mok_block8_wgrad(dev(dy), dev(sdy), W, dev(xt), dev(sx), N, rows, dw, offsets=off, n_local=n)
        assert torch.equal(dw.cpu(), want_dw.to(out))


@pytest.mark.parametrize("n", [1, 5])
@pytest.mark.parametrize("M,N", [(64, 128), (512, 768)])
def test_zero_rows(n, M, N):
    """rows = 0: operands may be missing; gradients are zero, or stay."""
    off = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    mok.mok_block8_quantise(torch.zeros(0, 128, device="cuda"), 0, 128, torch.zeros(16, dtype=torch.uint8, device="cuda"),
                            torch.zeros(1, device="cuda"), offsets=off, n_local=n)
    mok.mok_block8_gemm(None, None, 0, 128, None, None, 64, None, offsets=off, n_local=n)
    for out in (torch.bfloat16, torch.float32):
        dw = torch.full((n, M, N), 3.0, dtype=out, device="cuda")
        if out is torch.float32:
            mok.mok_block8_wgrad(None, None, M, None, None, N, 0, dw, offsets=off, n_local=n, accumulate=1)
            assert (dw == 3).all()
        mok.mok_block8_wgrad(None, None, M, None, None, N, 0, dw, offsets=off, n_local=n)
        assert not dw.any()


def test_quantise_many_values():
    """4.3e9 values both ways: the first rows, the last ones and a run in the middle bit for bit."""
    rows, W, n = 600011, 7168, 2
    split = 300101
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, W, dtype=torch.bfloat16, device="cuda")
    for at in range(0, rows, 100000):
        x[at:at + 100000] = torch.randn(min(100000, rows - at), W, generator=gen, device="cuda")
    S = ref.slots(rows, n)
    codes = torch.zeros(rows, W, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(W // 128, rows, device="cuda")
    codes_t = torch.zeros(W, S, dtype=torch.uint8, device="cuda")
    scales_t = torch.zeros(S // 128, W, device="cuda")
    off = torch.tensor([0, split, rows], dtype=torch.int32, device="cuda")
    mok.mok_block8_quantise(x, rows, W, codes, scales, codes_t=codes_t, scales_t=scales_t, offsets=off, n_local=n)
    # whole blocks of the first expert, and the last (part) blocks of both
    first = 128 * ref.blocks(split)
    for row, place, m in ((0, 0, 256), (split - split % 128, first - 128, split % 128),
                          (split + 128 * 1000, first + 128 * 1000, 128),
                          (rows - (rows - split) % 128, first + (rows - split) // 128 * 128, (rows - split) % 128)):
        part = x[row:row + m].float().cpu().numpy()
        c, s = ref.rows_operand(part)
        assert np.array_equal(host(codes[row:row + m]), c) and np.array_equal(host(scales[:, row:row + m]), s)
        ct, st = ref.slot_operand(part, [m], "line")
        k = 128 * ref.blocks(m)
        assert np.array_equal(host(codes_t[:, place:place + k]), ct[:, :k])
        assert np.array_equal(host(scales_t[place // 128:(place + k) // 128]), st[:k // 128])


def test_weights_many_values():
    n, N, K = 40, 16384, 8192
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = torch.empty(n, N, K, dtype=torch.bfloat16, device="cuda")
    for e in range(n):
        w[e] = torch.randn(N, K, generator=gen, device="cuda")
    codes, codes_t = (torch.zeros(n * N * K, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales, scales_t = (torch.zeros(n, N // 128 * (K // 128), device="cuda") for _ in range(2))
    mok.mok_block8_quantise_weights(w, n, N, K, codes, scales, codes_t, scales_t)
    codes, codes_t = codes.view(n, N, K), codes_t.view(n, K, N)
    for e in (0, 33, n - 1):
        largest = w[e].float().abs().view(N // 128, 128, K // 128, 128).amax(3).amax(1)
        assert torch.equal(scales[e].view(N // 128, K // 128), (largest.double() / 448).float())
        assert torch.equal(scales_t[e].view(K // 128, N // 128), (largest.double() / 448).float().T)
        for at in (0, N - 256):
            c, _ = ref.block_operand(w[e, at:at + 256].float().cpu().numpy())
            assert np.array_equal(host(codes[e, at:at + 256]), c)
        for at in range(0, N, 4096):
            assert torch.equal(codes_t[e, :, at:at + 4096], codes[e, at:at + 4096].T)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_wgrad_many_results(out):
    """64 x 8192 x 8448 gradients, of few rows: every one exact."""
    rng = np.random.default_rng(3)
    n, M, N = 64, 8192, 8448
    counts = counts_of(rng, n, 400)
    rows = sum(counts)
    S = ref.slots(rows, n)
    used = np.zeros(S, np.uint8)
    starts = ref.starts(counts)
    for c, at in zip(counts, starts):
        used[at:at + c] = 1
    dy, x = small_codes(rng, M, S) * used, small_codes(rng, N, S) * used
    ones = torch.ones(S // 128, M, device="cuda"), torch.ones(N // 128, S // 128, device="cuda")
    dw = torch.full((n, M, N), -7.0, dtype=out, device="cuda")
    mok.mok_block8_wgrad(dev(dy), ones[0], M, dev(x), ones[1], N, rows, dw, offsets=offsets_of(counts), n_local=n)
    u, v = (torch.from_numpy(ref.values(t).astype(np.float32)).cuda() for t in (dy, x))
    for e, (c, at) in enumerate(zip(counts, starts)):
        assert torch.equal(dw[e], (u[:, at:at + c] @ v[:, at:at + c].T.contiguous()).to(out))


def test_wgrad_long_operands():
    """Operands of 5e9 codes: rows of 700,000 places, zeros but for the first and last blocks of the last expert."""
    n, M, N, rows = 3, 7168, 256, 700000
    counts = [100000, 7, rows - 100007]
    rng = np.random.default_rng(4)
    S, starts = ref.slots(rows, n), ref.starts(counts)
    dy = torch.zeros(M, S, dtype=torch.uint8, device="cuda")
    x = torch.zeros(N, S, dtype=torch.uint8, device="cuda")
    want = torch.zeros(n, M, N, dtype=torch.float64)
    for e, at, c in ((0, 0, 128), (1, int(starts[1]), 7), (2, int(starts[2]), 128), (2, int(starts[2]) + counts[2] // 128 * 128, counts[2] % 128)):
        a, b = small_codes(rng, M, c), small_codes(rng, N, c)
        dy[:, at:at + c], x[:, at:at + c] = dev(a), dev(b)
        want[e] += torch.from_numpy(ref.values(a) @ ref.values(b).T)
    for out in (torch.bfloat16, torch.float32):
        dw = torch.full((n, M, N), -7.0, dtype=out, device="cuda")
        mok.mok_block8_wgrad(dy, torch.ones(S // 128, M, device="cuda"), M, x, torch.ones(2, S // 128, device="cuda"), N,
                             rows, dw, offsets=offsets_of(counts), n_local=n)
        assert torch.equal(dw.cpu(), want.to(out))
