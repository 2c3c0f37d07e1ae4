"""GPU tests of the 8-bit block quantisers and products against tests/block8_reference.py.

Quantised copies are equal bit for bit.  Through SwiGLU the value itself is off by a few roundings of fp32: every code
is the nearest one to a value that near, and so is the scale.  Products: an fp32 sum of n terms whose magnitudes add up
to A is off by at most n roundings of A, each a whole last place (2^-23) at most; the factor of the two scales and its
product with a block's sum add two; the result in bf16 rounds once more (2^-8).  The 8-bit matrix instructions, by which
results in bf16 are formed, drop what lies below 2^-13 of the largest of 64 products (block8_reference.dropped).
"""
import numpy as np
import pytest
import torch

import block8_reference as ref
import token_dispatch_grouped_top_amd as mok

pytestmark = pytest.mark.gpu
FILL = 0xee


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def host(t):
    return t.cpu().numpy()


def offsets_of(counts, rows=None):
    return dev(np.concatenate([[0], np.cumsum(counts)]), torch.int32)


def rows_like(rng, rows, W, dtype):
    """fp32 values that `dtype` holds: rows and columns of unlike size, zeros, a zero block, a large and a tiny one."""
    x = rng.normal(size=(rows, W)) * np.exp(rng.normal(size=(rows, 1)) * 2) * np.exp(rng.normal(size=W))
    x[rng.random((rows, W)) < 0.05] = 0
    x[:, :64] *= rng.random() < 0.5
    if rows > 2:
        x[1] = 0
        x[2] *= 1e30 / max(1e-30, np.abs(x[2]).max())
        x[rows // 2] *= 1e-37
    return torch.from_numpy(x.astype(np.float32)).to(dtype).float().numpy()


def padded(x, dtype, pad, offset=0):
    """x on the GPU in rows `pad` wider, the first `offset` elements behind an allocation."""
    rows, W = x.shape
    flat = torch.full((offset + rows * (W + pad),), float("nan"), dtype=dtype, device="cuda")
    view = flat[offset:].view(rows, W + pad)[:, :W]
    view.copy_(dev(x, dtype))
    return view


def outputs(rows, W, n, kind, f8=False):
    dt = torch.uint8
    S = ref.slots(rows, n)
    codes = torch.full((rows, W), FILL, dtype=dt, device="cuda")
    scales = torch.full((ref.blocks(W), rows), -1.0, device="cuda")
    if not kind:
        return codes, scales, None, None
    codes_t = torch.full((W, S), FILL, dtype=dt, device="cuda")
    scales_t = torch.full((S // 128, W) if kind == "line" else (ref.blocks(W), S // 128), -1.0, device="cuda")
    if f8:
        codes, codes_t = codes.view(torch.float8_e4m3fn), codes_t.view(torch.float8_e4m3fn)
    return codes, scales, codes_t, scales_t


KIND = dict(line=mok.MOK_BLOCK8_LINES, block=mok.MOK_BLOCK8_BLOCKS)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["", "line", "block"])
@pytest.mark.parametrize("counts,W,pad", [([1], 64, 0), ([3, 0, 130], 192, 8), ([128], 128, 0), ([0, 0, 5], 320, 1),
                                          ([129, 256, 1, 127], 256, 3), ([300], 1472, 0)])
def test_quantise_copy(dtype, kind, counts, W, pad):
    rng = np.random.default_rng(len(counts) * W + pad)
    rows, n = sum(counts), len(counts)
    x = rows_like(rng, rows, W, dtype)
    out = outputs(rows, W, n, kind, f8=pad == 8)
    mok.mok_block8_quantise(padded(x, dtype, pad, offset=pad % 2), rows, W, out[0], out[1], codes_t=out[2],
                            scales_t=out[3], t_scales=KIND.get(kind, 0), offsets=offsets_of(counts), n_local=n)
    codes, scales = ref.rows_operand(x)
    assert np.array_equal(host(out[1]), scales)
    assert np.array_equal(host(out[0].view(torch.uint8)), codes)
    if kind:
        codes_t, scales_t = ref.slot_operand(x, counts, kind, FILL)
        assert np.array_equal(host(out[3]), scales_t)
        assert np.array_equal(host(out[2].view(torch.uint8)), codes_t)


@pytest.mark.parametrize("kind", ["", "line", "block"])
def test_quantise_ties_and_special_values(kind):
    """Values in the middle between two codes for each mantissa of the largest; infinities and NaN; blocks of zeros and
    of subnormal values."""
    rng = np.random.default_rng(5)
    rows, W = 256, 128
    q = rng.integers(128, 256, rows)
    p = rng.integers(-255, 256, (rows, W)) * 2.0 ** rng.integers(-9, 1, (rows, W))
    x = np.clip(p, -q[:, None], q[:, None]).astype(np.float32)
    x[:, 0] = q
    x[3], x[4] = 0, -0.0
    x[5] = rng.normal(size=W) * 1e-41
    x[6, 5], x[7, 1], x[8, 9], x[9] = np.inf, -np.inf, np.nan, np.nan
    x[10] = 3e38
    out = outputs(rows, W, 1, kind)
    mok.mok_block8_quantise(dev(x), rows, W, out[0], out[1], codes_t=out[2], scales_t=out[3],
                            t_scales=KIND.get(kind, 0))
    codes, scales = ref.rows_operand(x)
    assert np.array_equal(host(out[1]), scales)
    assert np.array_equal(host(out[0]), codes)
    if kind:
        codes_t, scales_t = ref.slot_operand(x, [rows], kind, FILL)
        assert np.array_equal(host(out[3]), scales_t) and np.array_equal(host(out[2]), codes_t)


def near(codes, scales, x, slack):
    """Whether each code (with its own scale per value) is the nearest to some value within `slack` of x."""
    v, q = ref.values(codes), x / scales
    step = np.where(np.abs(v) < 2.0 ** -6, 2.0 ** -9, np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3))
    return np.all(np.abs(v - q) <= step / 2 + slack / scales)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("source", ["swiglu", "swiglu_bwd"])
@pytest.mark.parametrize("kind", ["", "line", "block"])
@pytest.mark.parametrize("counts,I,pad", [([1], 64, 0), ([3, 0, 130], 192, 8), ([129, 1], 96, 1), ([200], 512, 0)])
def test_quantise_swiglu(dtype, source, kind, counts, I, pad):
    if source == "swiglu" and I % 64:
        I = 128
    rng = np.random.default_rng(I + pad)
    rows, n = sum(counts), len(counts)
    cast = lambda a: torch.from_numpy(a.astype(np.float32)).to(dtype).float().numpy()  # noqa: E731
    h, d = cast(rng.normal(size=(rows, 2 * I)) * 3), cast(rng.normal(size=(rows, I)) * 1e-3)
    h[0, 0], h[0, 1], h[0, 2] = cast(np.array([90.0, -90.0, -100.0]))
    # fp32: exp with its argument's rounding (|g| 2^-24) and one last place, a sum, a division and three products, each
    # a rounding; (1 + g (1 - s)) adds three of its terms' size
    g = np.abs(h[:, :I].astype(np.float64))
    if source == "swiglu":
        W, x = I, ref.swiglu(h)
        slack = np.abs(x) * (g + 8) * 2.0 ** -23 + 1e-37
        kw = dict(source=mok.MOK_BLOCK8_SWIGLU)
    else:
        W = 2 * I
        x, size = ref.swiglu_backward(h, d)
        slack = size * (np.concatenate([g, g], 1) + 12) * 2.0 ** -23 + 1e-37
        kw = dict(source=mok.MOK_BLOCK8_SWIGLU_BWD, d=padded(d, dtype, pad))
    out = outputs(rows, W, n, kind)
    mok.mok_block8_quantise(padded(h, dtype, pad), rows, W, out[0], out[1], codes_t=out[2], scales_t=out[3],
                            t_scales=KIND.get(kind, 0), offsets=offsets_of(counts), n_local=n, **kw)
    scales = host(out[1]).astype(np.float64)
    each = np.repeat(scales.T, 128, 1)[:, :W]
    for b in range(ref.blocks(W)):
        cols = np.s_[:, 128 * b:128 * b + 128]
        want = np.maximum(np.abs(x[cols]).max(1) / 448, 2.0 ** -126)
        assert np.all(np.abs(scales[b] - want) <= slack[cols].max(1) / 448 + want * 2.0 ** -23)
    assert near(host(out[0]), each, x, slack + 2.0 ** -22 * np.abs(x))
    if not kind:
        return
    codes_t, scales_t, first = host(out[2]), host(out[3]).astype(np.float64), 0
    for c, at in zip(counts, ref.starts(counts)):
        for j in range(0, c, 128):
            m, b = min(128, c - j), (at + j) // 128
            part, tol = x[first + j:first + j + m].T, slack[first + j:first + j + m].T
            s = scales_t[b] if kind == "line" else np.repeat(scales_t[:, b], 128)[:W]
            assert near(codes_t[:, at + j:at + j + m], s[:, None], part, tol + 2.0 ** -22 * np.abs(part))
            assert not codes_t[:, at + j + m:at + j + 128].any()
        first += c


def test_quantise_ring_and_short_offsets():
    """Column-blocked rows of a ring, and offsets that end before the rows do: what is behind stays as it was."""
    rng = np.random.default_rng(3)
    W, ring, counts, rows = 192, 150, [70, 0, 60], 140
    R = sum(counts)
    x = rows_like(rng, ring, W, torch.bfloat16)
    # 64-byte column blocks, block-major
    blocked = dev(x, torch.bfloat16).view(ring, W // 32, 32).permute(1, 0, 2).contiguous()
    for kind in ("", "line", "block"):
        out = outputs(rows, W, 3, kind)
        mok.mok_block8_quantise(blocked, rows, W, out[0], out[1], codes_t=out[2], scales_t=out[3],
                                t_scales=KIND.get(kind, 0), offsets=offsets_of(counts), n_local=3, ring_rows=ring)
        codes, scales = ref.rows_operand(x[:R])
        assert np.array_equal(host(out[0])[:R], codes) and np.array_equal(host(out[1])[:, :R], scales)
        assert (host(out[0])[R:] == FILL).all() and (host(out[1])[:, R:] == -1).all()
        if kind:
            codes_t, scales_t = ref.slot_operand(x[:R], counts, kind, FILL)
            end = ref.starts(counts)[-1]
            assert np.array_equal(host(out[2])[:, :end], codes_t[:, :end]) and (host(out[2])[:, end:] == FILL).all()
            got, end = host(out[3]), end // 128
            got, want = (got, scales_t) if kind == "line" else (got.T, scales_t.T)
            assert np.array_equal(got[:end], want[:end]) and (got[end:] == -1).all()
    # rows of a ring begin again at its first row
    out = outputs(rows + 40, W, 1, "line")
    mok.mok_block8_quantise(blocked, rows + 40, W, out[0], out[1], codes_t=out[2], scales_t=out[3], ring_rows=ring)
    assert np.array_equal(host(out[0]), ref.rows_operand(x[np.arange(rows + 40) % ring])[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,N,K", [(1, 64, 64), (3, 192, 320), (2, 128, 128), (1, 448, 1472)])
@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("offset", [0, 1])
def test_quantise_weights(dtype, n, N, K, both, offset):
    rng = np.random.default_rng(N + K)
    w = np.stack([rows_like(rng, N, K, dtype) for _ in range(n)])
    flat = torch.zeros(offset + n * N * K, dtype=dtype, device="cuda")
    flat[offset:] = dev(w, dtype).view(-1)
    codes = torch.full((n, N, K), FILL, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, ref.blocks(N), ref.blocks(K)), -1.0, device="cuda")
    codes_t = torch.full((n, K, N), FILL, dtype=torch.uint8, device="cuda") if both else None
    scales_t = torch.full((n, ref.blocks(K), ref.blocks(N)), -1.0, device="cuda") if both else None
    mok.mok_block8_quantise_weights(flat[offset:], n, N, K, codes, scales, codes_t, scales_t)
    for e in range(n):
        c, s = ref.block_operand(w[e])
        assert np.array_equal(host(scales[e]), s) and np.array_equal(host(codes[e]), c)
        if both:
            assert np.array_equal(host(scales_t[e]), s.T) and np.array_equal(host(codes_t[e]), c.T)


def small_codes(rng, *shape):
    """Codes of the whole numbers -8 to 8: sums of their products are exact in fp32."""
    return ref.encode(rng.integers(-8, 9, shape).astype(np.float32), np.float32(1))


def any_codes(rng, *shape):
    c = rng.integers(0, 256, shape).astype(np.uint8)
    return np.where((c & 0x7f) == 0x7f, 0x70, c).astype(np.uint8)


SHAPES = [([1], 64, 64), ([3, 0, 130], 192, 320), ([0, 0, 5], 128, 64), ([129, 1, 300], 320, 448), ([64, 65], 1472, 192),
          ([700], 576, 512), ([2, 1, 0, 4], 2048, 256), ([0, 0], 128, 128), ([33], 8256, 64)]


@pytest.mark.parametrize("counts,K,N", SHAPES)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gemm(counts, K, N, out):
    rng = np.random.default_rng(K + N)
    rows, n = sum(counts), len(counts)
    extra = 3                                         # rows behind the last expert's
    # whole numbers and powers of two: every result is exact
    a, w = small_codes(rng, rows + extra, K), small_codes(rng, n, N, K)
    sa = np.exp2(rng.integers(-2, 3, (ref.blocks(K), rows + extra))).astype(np.float32)
    sw = np.exp2(rng.integers(-2, 3, (n, ref.blocks(N), ref.blocks(K)))).astype(np.float32)
    y = torch.full((rows + extra, N), -7.0, dtype=out, device="cuda")
    mok.mok_block8_gemm(dev(a), dev(sa), rows + extra, K, dev(w), dev(sw), N, y, offsets=offsets_of(counts), n_local=n)
    want, size = ref.product(a[:rows], sa[:, :rows], counts, w, sw)
    assert size.size == 0 or size.max() * 16 < 2 ** 24
    got = host(y.float())
    assert np.array_equal(got[:rows], host(torch.from_numpy(want).to(out).float())) and (got[rows:] == -7).all()
    # any codes and scales
    a, w = any_codes(rng, rows + extra, K), any_codes(rng, n, N, K)
    sa = np.exp(rng.normal(size=sa.shape) * 2).astype(np.float32)
    sw = np.exp(rng.normal(size=sw.shape)).astype(np.float32)
    mok.mok_block8_gemm(dev(a), dev(sa), rows + extra, K, dev(w).view(torch.float8_e4m3fn), dev(sw), N, y,
                        offsets=offsets_of(counts), n_local=n)
    want, size = ref.product(a[:rows], sa[:, :rows], counts, w, sw)
    if out is torch.bfloat16:
        size = size + ref.product(a[:rows], sa[:, :rows], counts, w, sw, drop=True)[1] * 2.0 ** 23 / (K + 2)
    got = host(y.float())
    tol = (K + 2) * 2.0 ** -23 * size + (2.0 ** -8 if out is torch.bfloat16 else 2.0 ** -24) * np.abs(want)
    assert np.all(np.abs(got[:rows] - want) <= tol) and (got[rows:] == -7).all()


def test_gemm_without_offsets_and_nan():
    """One expert's rows without offsets; a NaN code reaches its own row's and column's results and no others."""
    rng = np.random.default_rng(2)
    rows, K, N = 200, 192, 192
    a, w = small_codes(rng, rows, K), small_codes(rng, 1, N, K)
    a[17, 100], w[0, 65, 3] = 0x7f, 0xff
    sa, sw = np.ones((2, rows), np.float32), np.ones((1, 2, 2), np.float32)
    y = torch.zeros(rows, N, device="cuda")
    mok.mok_block8_gemm(dev(a), dev(sa), rows, K, dev(w), dev(sw), N, y)
    got, want = host(y), ref.product(a, sa, [rows], w, sw)[0]
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(want).sum() == rows + N - 1
    assert np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


def test_gemm_offsets_out_of_range():
    """Offsets that descend, are negative or pass the rows: the rows that exist are computed, nothing else is touched."""
    rng = np.random.default_rng(4)
    rows, K, N = 40, 128, 64
    a, w = small_codes(rng, rows, K), small_codes(rng, 3, N, K)
    sa, sw = np.ones((1, rows), np.float32), np.ones((3, 1, 1), np.float32)
    y = torch.full((rows + 8, N), -7.0, device="cuda")
    mok.mok_block8_gemm(dev(a), dev(sa), rows, K, dev(w), dev(sw), N, y, n_local=3,
                        offsets=dev(np.array([-5, 20, 10, 1 << 30]), torch.int32))
    got = host(y)
    want = ref.product(a[:20], sa[:, :20], [20, 0, 0], w, sw)[0]
    assert np.array_equal(got[:10], want[:10])
    want = ref.product(a[10:], sa[:, 10:], [0, 0, 30], w, sw)[0]
    assert np.array_equal(got[20:40], want[10:]) and (got[rows:] == -7).all()


@pytest.mark.parametrize("counts,M,N", [([1], 64, 64), ([3, 0, 130], 192, 320), ([0, 0, 5], 128, 64),
                                        ([129, 1, 300], 320, 448), ([700], 576, 512), ([0, 0], 64, 128),
                                        ([2, 1, 0, 4], 256, 768)])
@pytest.mark.parametrize("out", ["bf16", "f32", "added"])
def test_wgrad(counts, M, N, out):
    rng = np.random.default_rng(M + N)
    rows, n = sum(counts), len(counts)
    S = ref.slots(rows, n)
    used = np.zeros(S, bool)
    for c, at in zip(counts, ref.starts(counts)):
        used[at:at + c] = True
    end = ref.starts(counts)[-1]
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    for exact in (True, False):
        make = small_codes if exact else any_codes
        dy, x = make(rng, M, S) * used.astype(np.uint8), make(rng, N, S) * used.astype(np.uint8)
        dy[:, end:], x[:, end:] = 0x7f, 0x7f          # behind the last expert's places: not read
        if exact:
            sdy = np.exp2(rng.integers(-2, 3, (S // 128, M))).astype(np.float32)
            sx = np.exp2(rng.integers(-2, 3, (ref.blocks(N), S // 128))).astype(np.float32)
            dw0 = rng.integers(-50, 50, (n, M, N)).astype(np.float32)
        else:
            sdy = np.exp(rng.normal(size=(S // 128, M))).astype(np.float32)
            sx = np.exp(rng.normal(size=(ref.blocks(N), S // 128))).astype(np.float32)
            dw0 = rng.normal(size=(n, M, N)).astype(np.float32) * 100
        dw = dev(dw0).to(dt)
        mok.mok_block8_wgrad(dev(dy), dev(sdy), M, dev(x), dev(sx), N, rows, dw, offsets=offsets_of(counts), n_local=n,
                             accumulate=int(out == "added"))
        want, size = ref.wgrad(dy, sdy, x, sx, counts)
        if out == "added":
            want, size = want + dw0, size + np.abs(dw0)
        got = host(dw.float())
        if exact:
            assert np.array_equal(got, host(torch.from_numpy(want).to(dt).float()))
        else:
            if out == "bf16":
                size = size + ref.wgrad(dy, sdy, x, sx, counts, drop=True)[1] * 2.0 ** 23 / (max(counts) + 131)
            tol = (max(counts) + 131) * 2.0 ** -23 * size + (2.0 ** -8 if out == "bf16" else 2.0 ** -24) * np.abs(want)
            assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("counts,K,N", [([2300], 320, 1280), ([1100, 0, 300, 900], 384, 2368), ([260, 100, 520], 192, 512),
                                        ([257] * 8, 256, 1088)])
def test_gemm_tiles(counts, K, N):
    """Sizes of many tiles, the last of an expert with few rows; every result is exact, and the same when computed again."""
    rng = np.random.default_rng(N)
    rows, n = sum(counts), len(counts)
    a, w = small_codes(rng, rows, K), small_codes(rng, n, N, K)
    sa = np.exp2(rng.integers(-2, 3, (ref.blocks(K), rows))).astype(np.float32)
    sw = np.exp2(rng.integers(-2, 3, (n, ref.blocks(N), ref.blocks(K)))).astype(np.float32)
    want, size = ref.product(a, sa, counts, w, sw)
    assert size.max() * 16 < 2 ** 24
    args = [dev(a), dev(sa), rows, K, dev(w), dev(sw), N]
    for out in (torch.bfloat16, torch.float32):
        for _ in range(3):
            y = torch.full((rows, N), -7.0, dtype=out, device="cuda")
            mok.mok_block8_gemm(*args, y, offsets=offsets_of(counts), n_local=n)
            assert torch.equal(y, torch.from_numpy(want).to(out).cuda())


@pytest.mark.parametrize("counts,K,N", [([2300, 0, 1500, 700], 320, 2816), ([300] * 40, 192, 1088), ([257] * 19, 320, 2048),
                                        ([257] * 22, 256, 1984), ([5000, 1, 0, 130, 900], 128, 2368)])
def test_gemm_large_tiles(counts, K, N):
    """Sizes that take the largest tiles (results in bf16): whole ones, the last round's in one, two and four parts, ones
    of few rows; exact results, and any codes against the bound."""
    test_gemm_tiles(counts, K, N)
    rng = np.random.default_rng(K)
    rows, n = sum(counts), len(counts)
    a, w = any_codes(rng, rows, K), any_codes(rng, n, N, K)
    sa = np.exp(rng.normal(size=(ref.blocks(K), rows))).astype(np.float32)
    sw = np.exp(rng.normal(size=(n, ref.blocks(N), ref.blocks(K)))).astype(np.float32)
    want, size = ref.product(a, sa, counts, w, sw)
    dropped = ref.product(a, sa, counts, w, sw, drop=True)[1]
    for out in (torch.bfloat16, torch.float32):
        y = torch.full((rows, N), -7.0, dtype=out, device="cuda")
        mok.mok_block8_gemm(dev(a), dev(sa), rows, K, dev(w), dev(sw), N, y, offsets=offsets_of(counts), n_local=n)
        tol = (K + 2) * 2.0 ** -23 * size + (2.0 ** -8 * np.abs(want) + dropped if out is torch.bfloat16 else
                                            2.0 ** -24 * np.abs(want))
        assert np.all(np.abs(host(y.float()) - want) <= tol)


@pytest.mark.parametrize("counts,M,N", [([1500], 512, 1344), ([600, 700, 0, 800], 320, 768), ([300] * 20, 512, 576)])
def test_wgrad_tiles(counts, M, N):
    rng = np.random.default_rng(N)
    rows, n = sum(counts), len(counts)
    S = ref.slots(rows, n)
    used = np.zeros(S, np.uint8)
    for c, at in zip(counts, ref.starts(counts)):
        used[at:at + c] = 1
    dy, x = small_codes(rng, M, S) * used, small_codes(rng, N, S) * used
    sdy = np.exp2(rng.integers(-2, 3, (S // 128, M))).astype(np.float32)
    sx = np.exp2(rng.integers(-2, 3, (ref.blocks(N), S // 128))).astype(np.float32)
    want, size = ref.wgrad(dy, sdy, x, sx, counts)
    assert size.max() * 16 < 2 ** 24
    args = [dev(dy), dev(sdy), M, dev(x), dev(sx), N, rows]
    for out in (torch.bfloat16, torch.float32):
        for _ in range(3):
            dw = torch.full((n, M, N), -7.0, dtype=out, device="cuda")
            mok.mok_block8_wgrad(*args, dw, offsets=offsets_of(counts), n_local=n)
            assert torch.equal(dw, torch.from_numpy(want).to(out).cuda())
