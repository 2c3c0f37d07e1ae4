"""Plain forms, in 64 bits, of the 8-bit block operands, their products and the orthogonalised update (numpy).

Codes are held as uint8; `values` says what they stand for.
"""
import numpy as np

_POS = np.array([f * 2.0 ** -9 for f in range(8)] + [(8 + f) * 2.0 ** (e - 10) for e in range(1, 16) for f in range(8)])
_POS[127] = np.nan
VALUES = np.concatenate([_POS, -_POS])


def values(codes):
    return VALUES[codes]


def scale_of(largest):
    return np.maximum((np.asarray(largest, np.float32) / np.float32(448)).astype(np.float32), np.float32(2.0 ** -126))


def encode(x, scale):
    """Codes of fp32 x with the fp32 scale (broadcast): nearest to the fp32 quotient, in the middle the even one."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        q = np.abs((x / np.broadcast_to(scale, x.shape)).astype(np.float32)).astype(np.float64)
    table = _POS[:127]
    low = np.clip(np.searchsorted(table, q, side="right") - 1, 0, 125)
    over = 2 * q - (table[low] + table[low + 1])
    code = low + ((over > 0) | ((over == 0) & (low % 2 == 1)))
    code = np.where(np.signbit(x), code + 128, code)
    return np.where(np.isfinite(x), code, 0xff).astype(np.uint8)


def largest(x, axis):
    return np.max(np.where(np.isfinite(x), np.abs(x), 0), axis=axis)


def blocks(n):
    return -(-n // 128)


def rows_operand(x):
    """codes [R][W] and scales [blocks(W)][R] of fp32 x."""
    R, W = x.shape
    codes, scales = np.zeros((R, W), np.uint8), np.zeros((blocks(W), R), np.float32)
    for b in range(blocks(W)):
        part = x[:, 128 * b:128 * b + 128]
        scales[b] = scale_of(largest(part, 1))
        codes[:, 128 * b:128 * b + 128] = encode(part, scales[b][:, None])
    return codes, scales


def block_operand(w):
    """codes [N][K] and scales [blocks(N)][blocks(K)] of fp32 w."""
    N, K = w.shape
    codes, scales = np.zeros((N, K), np.uint8), np.zeros((blocks(N), blocks(K)), np.float32)
    for i in range(blocks(N)):
        for j in range(blocks(K)):
            at = np.s_[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            scales[i, j] = scale_of(largest(w[at], None))
            codes[at] = encode(w[at], scales[i, j])
    return codes, scales


def slots(rows, n_local):
    return 128 * (blocks(rows) + n_local - 1)


def starts(counts):
    """First place of each expert's slot blocks, and where the last one's end."""
    return np.concatenate([[0], np.cumsum([128 * blocks(c) for c in counts])]).astype(int)


def slot_operand(x, counts, kind, fill=0xee):
    """Transposed codes [W][S] and scales ("line": [S / 128][W], "block": [blocks(W)][S / 128]); what is not written
    holds `fill` and -1."""
    rows, W = x.shape
    S = slots(rows, len(counts))
    codes = np.full((W, S), fill, np.uint8)
    scales = np.full((S // 128, W) if kind == "line" else (blocks(W), S // 128), -1, np.float32)
    first = 0
    for c, at in zip(counts, starts(counts)):
        for j in range(0, c, 128):
            part = np.zeros((128, W), np.float32)
            part[:min(128, c - j)] = x[first + j:first + min(j + 128, c)]
            b = (at + j) // 128
            if kind == "line":
                scales[b] = scale_of(largest(part, 0))
                codes[:, at + j:at + j + 128] = encode(part, scales[b]).T
            else:
                for k in range(blocks(W)):
                    cols = np.s_[128 * k:128 * k + 128]
                    scales[k, b] = scale_of(largest(part[:, cols], None))
                    codes[cols, at + j:at + j + 128] = encode(part[:, cols], scales[k, b]).T
        first += c
    return codes, scales


def swiglu(h):
    g, u = np.split(h.astype(np.float64), 2, 1)
    return g / (1 + np.exp(-g)) * u


def swiglu_backward(h, d):
    """[dg, du], and the magnitudes that are added up in dg."""
    g, u = np.split(h.astype(np.float64), 2, 1)
    s, d = 1 / (1 + np.exp(-g)), d.astype(np.float64)
    dg, du = d * u * s * (1 + g * (1 - s)), d * g * s
    return np.concatenate([dg, du], 1), np.concatenate([np.abs(d * u * s) * (1 + np.abs(g) * (1 - s)), np.abs(du)], 1)


def dropped(u, v):
    """Bound of what the 8-bit matrix instructions drop in u v^T (u [m][K], v [n][K]): of 64 products each but the
    largest is off by less than 2^-13 of that one."""
    out = np.zeros((u.shape[0], v.shape[0]))
    for k in range(0, u.shape[1], 64):
        out += 63 * 2.0 ** -13 * (np.abs(u[:, None, k:k + 64]) * np.abs(v[None, :, k:k + 64])).max(2)
    return out


def product(a, sa, counts, w, sw, drop=False):
    """out [rows][N] of codes a [rows][K], w [n][N][K], and the sums of the terms' magnitudes (drop: dropped())."""
    rows, K = a.shape
    N = w.shape[1]
    out, size = np.zeros((rows, N)), np.zeros((rows, N))
    x = values(a) * np.repeat(sa.astype(np.float64).T, 128, 1)[:, :K]
    first = 0
    for e, c in enumerate(counts):
        y = values(w[e]) * np.repeat(np.repeat(sw[e].astype(np.float64), 128, 0)[:N], 128, 1)[:, :K]
        out[first:first + c] = x[first:first + c] @ y.T
        size[first:first + c] = dropped(x[first:first + c], y) if drop else np.abs(x[first:first + c]) @ np.abs(y).T
        first += c
    return out, size


def wgrad(dy, sdy, x, sx, counts, drop=False):
    """dw [n][M][N] of slot blocks dy [M][S] (lines) and x [N][S] (blocks), and the terms' magnitudes or dropped()."""
    M, N = dy.shape[0], x.shape[0]
    out, size = np.zeros((len(counts), M, N)), np.zeros((len(counts), M, N))
    for e, (c, at) in enumerate(zip(counts, starts(counts))):
        if c == 0:
            continue
        n = 128 * blocks(c)
        b = np.s_[at // 128:(at + n) // 128]
        u = values(dy[:, at:at + n]) * np.repeat(sdy[b].astype(np.float64).T, 128, 1)
        v = values(x[:, at:at + n]) * np.repeat(np.repeat(sx[:, b].astype(np.float64), 128, 0)[:N], 128, 1)
        out[e], size[e] = u @ v.T, dropped(u, v) if drop else np.abs(u) @ np.abs(v).T
    return out, size


def orthogonalise(v, coef, steps):
    """The result, and a bound of the 2-norm of what roundings of X, G and B to 11 bits (u = 2^-11 each) make of it.

    With s = |X|_2 and r = |X|_F, a step X' = a X + (b G + c G^2) X carries an error e of X on by at most a + 3 |b| s^2
    + 5 |c| s^4; G's rounding is u s r at most in the 2-norm of the difference (|G|_F <= s r), which B multiplies by
    |b| + 2 |c| s^2, to which c G^2's and B's own add u |B|_F <= u (|b| + |c| s^2) s r; all of them meet X, so s more;
    X' itself is rounded by u |X'|_F."""
    a, b, c = coef
    x = np.asarray(v, np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    u = 2.0 ** -11
    norm = np.linalg.norm(x)
    x = x / norm if norm else x
    e = u * np.linalg.norm(x)
    for _ in range(steps):
        s, r = np.linalg.norm(x, 2), np.linalg.norm(x)
        gram = x @ x.T
        e = e * (abs(a) + 3 * abs(b) * s ** 2 + 5 * abs(c) * s ** 4)
        e += u * s * s * r * ((abs(b) + 2 * abs(c) * s ** 2) + (abs(b) + abs(c) * s ** 2))
        x = a * x + (b * gram + c * gram @ gram) @ x
        e += u * np.linalg.norm(x)
    return (x.T if tall else x), e
