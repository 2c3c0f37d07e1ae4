"""Plain 64-bit forms of the scored route, its gradient and the AdamW step,
for the tests; numpy only, and the 8-bit states bit for bit from fp32 values."""
import numpy as np

SOFTMAX, SIGMOID = 0, 1


def clean(l):
    """Logits in fp64: NaN and -inf become -inf (not eligible), +inf the largest fp32 value."""
    l = np.asarray(l, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    return np.where(l == np.inf, float(np.finfo(np.float32).max), l)


def scores(l, score):
    """Scores of every expert (rows of cleaned logits); 0 where not eligible."""
    ok = l > -np.inf
    with np.errstate(over="ignore", invalid="ignore"):
        if score == SIGMOID:
            return np.where(ok, 1.0 / (1.0 + np.exp(-l)), 0.0)
        top = np.max(np.where(ok, l, -np.inf), axis=1, keepdims=True)
        e = np.where(ok, np.exp(l - np.where(np.isfinite(top), top, 0.0)), 0.0)
    return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def shares(l, score, picks):
    """u of the picks (their scores over the picks' sum), 0 where a pick is -1."""
    T, k = picks.shape
    lp = np.where(picks >= 0, np.take_along_axis(l, np.maximum(picks, 0), 1), -np.inf)
    ls = -np.logaddexp(0.0, -lp) if score == SIGMOID else lp
    with np.errstate(invalid="ignore"):
        top = ls.max(1, keepdims=True)
        e = np.exp(ls - np.where(np.isfinite(top), top, 0.0))
        return np.where(picks >= 0, e / np.maximum(e.sum(1, keepdims=True), 1e-300), 0.0)


def route(logits, score, k, bias=None, G=1, top_groups=1, top2=False, renorm=False, scale=1.0):
    """(idx int32 [T][k], gate fp64 [T][k], load [E])."""
    return route_and_gaps(logits, score, k, bias, G, top_groups, top2, renorm, scale)[:3]


def _gap(values, same):
    """Smallest distance of neighbours in an order, relative to them; equal ones of the same inputs are no matter."""
    a, b = values[:-1], values[1:]
    with np.errstate(invalid="ignore", divide="ignore"):
        d = np.abs(a - b) / np.maximum(np.maximum(np.abs(a), np.abs(b)), 1e-300)
    return min(d[~same & np.isfinite(b)], default=np.inf)


def route_and_gaps(logits, score, k, bias=None, G=1, top_groups=1, top2=False, renorm=False, scale=1.0):
    """route(), and for each row the smallest relative distance of two values whose order decided it: of the group
    values around the border, of the picks and the first value behind them."""
    l = clean(logits)
    T, E = l.shape
    s = scores(l, score)
    # without a bias the scores' order is the logits'
    c = l.copy() if bias is None else np.where(l > -np.inf, s + np.asarray(bias, np.float64), -np.inf)
    b = np.zeros(E) if bias is None else np.asarray(bias, np.float64)
    gaps = np.full(T, np.inf)
    if top_groups < G:
        for t in range(T):
            rows = c[t].reshape(G, E // G)
            value, inputs = [], []
            for g in range(G):
                order = np.argsort(-rows[g], kind="stable")[:2]
                v = rows[g][order]
                two = top2 and len(v) > 1 and v[1] > -np.inf
                if top2 and bias is None:
                    v = np.where(v > -np.inf, s[t, g * (E // G) + order], -np.inf)
                value.append(v[0] + v[1] if two else v[0])
                ids = g * (E // G) + order[:2 if two else 1]
                inputs.append(tuple((l[t, e], b[e]) for e in ids))
            order = np.argsort(-np.array(value), kind="stable")
            near = order[top_groups - 1:top_groups + 1]
            gaps[t] = _gap(np.array(value)[near], np.array([inputs[near[0]] == inputs[near[1]]]))
            for g in order[top_groups:]:
                rows[g] = -np.inf
    order = np.argsort(-c, axis=1, kind="stable")[:, :k + 1]
    for t in range(T):
        o = order[t]
        same = (l[t, o[1:]] == l[t, o[:-1]]) & (b[o[1:]] == b[o[:-1]])
        gaps[t] = min(gaps[t], _gap(c[t, o], same))
    idx = order[:, :k]
    idx = np.where(np.take_along_axis(c, idx, 1) > -np.inf, idx, -1).astype(np.int32)
    u = shares(l, score, idx) if renorm else np.where(
        idx >= 0, np.take_along_axis(s, np.maximum(idx, 0), 1), 0.0)
    load = np.bincount(idx[idx >= 0].ravel(), minlength=E)
    return idx, scale * u, load, gaps


def gates(logits, score, picks, renorm, scale):
    """Gates of given picks, in fp64 (what the gradient differentiates)."""
    l = clean(logits)
    if renorm:
        return scale * shares(l, score, picks)
    s = np.take_along_axis(scores(l, score), np.maximum(picks, 0), 1)
    return scale * np.where(picks >= 0, s, 0.0)


def usable(logits, picks):
    """Picks with ids out of range or of experts that are not eligible set to -1."""
    l = clean(logits)
    E = l.shape[1]
    ok = (picks >= 0) & (picks < E)
    ok &= np.take_along_axis(l, np.where(ok, picks, 0), 1) > -np.inf
    return np.where(ok, picks, -1)


def route_backward(logits, score, picks, dgate, renorm, scale):
    """(dlogits fp64, size): size bounds the magnitude of the terms each value is summed from."""
    l = clean(logits)
    picks = usable(logits, picks)
    ok = picks >= 0
    w = np.where(ok, scale * np.asarray(dgate, np.float64), 0.0)
    s = scores(l, score)
    at = np.maximum(picks, 0)
    sp = np.where(ok, np.take_along_axis(s, at, 1), 0.0)
    with np.errstate(over="ignore"):
        rest = 1.0 / (1.0 + np.exp(np.take_along_axis(l, at, 1))) if score == SIGMOID else 1.0
    out, size = np.zeros_like(l), np.zeros_like(l)
    rows = np.arange(len(l))
    if renorm:
        u = shares(l, score, picks)
        D, A = (w * u).sum(1, keepdims=True), (np.abs(w) * u).sum(1, keepdims=True)
        d, a = u * rest * (w - D), u * rest * (np.abs(w) + A)
    elif score == SIGMOID:
        d = sp * rest * w
        a = np.abs(d)
    else:
        d, a = sp * w, sp * np.abs(w)
        out -= s * d.sum(1, keepdims=True)
        size += s * a.sum(1, keepdims=True)
    for j in range(picks.shape[1]):
        m = ok[:, j]
        out[rows[m], picks[m, j]] += d[m, j]
        size[rows[m], picks[m, j]] += a[m, j]
    return out, size


# ------------------------------------------------------------------ AdamW
TABLE = np.array([f / 8 * 2.0 ** -6 for f in range(8)] +
                 [(1 + f / 8) * 2.0 ** (e - 7) for e in range(1, 16) for f in range(8)])
TABLE32 = TABLE.astype(np.float32)


def per_value(scale, n):
    return np.repeat(scale, 32)[:n]


def decode(code, scale):
    """fp64 values of codes with their scales (code 0x7f: NaN)."""
    a = TABLE[code & 127] * np.exp2(per_value(scale.astype(np.float64) - 127, len(code)))
    return np.where((code & 127) == 127, np.nan, np.where(code > 127, -a, a))


def hash32(x):
    x = np.asarray(x, np.uint64) & np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0xBB67AE85)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def random_bits(i, tensor, step, seed):
    """(16 bits for m, 16 for r) of elements i of tensor number `tensor`."""
    key = int(hash32(int(hash32(seed + 0x9E3779B1 * step)) + tensor))
    i = np.asarray(i, np.uint64)
    low, high = i & np.uint64(0xFFFFFFFF), i >> np.uint64(32)
    h = hash32(low + ((high * np.uint64(0x6A09E667)) & np.uint64(0xFFFFFFFF)) + np.uint64(key))
    return (h & np.uint64(0xFFFF)).astype(np.int64), (h >> np.uint64(16)).astype(np.int64)


def scale_byte(x):
    """E8M0 byte of each block of 32: the smallest scale with which no finite value passes 448."""
    x = np.where(np.isfinite(x), np.abs(x), 0).astype(np.float32)
    x = np.pad(x, (0, -len(x) % 32)).reshape(-1, 32).max(1).astype(np.float64)
    e = np.full(len(x), -127)
    for cand in range(127, -128, -1):
        e = np.where(x <= 448 * 2.0 ** cand, cand, e)
    return (np.where(x == 0, -127, e) + 127).astype(np.uint8)


def encode_m(m, b16, scale):
    """Codes of fp32 m, by the neighbours in the table and exact fp32 operations."""
    a = (np.abs(m).astype(np.float64) * np.exp2(127 - per_value(scale.astype(np.float64), len(m))))
    bits = a.astype(np.float32).view(np.int32).astype(np.int64)
    normal = ((bits + 16 * b16 + 8) >> 20) - 960
    u = ((b16.astype(np.float32) + np.float32(0.5)) / np.float32(65536)).astype(np.float32)
    tiny = np.floor(a.astype(np.float32) * np.float32(512) + u).astype(np.int64)
    code = np.where(a >= 2.0 ** -6, normal, tiny)
    code = np.where(m < 0, code | 128, code)
    return np.where(np.isfinite(m), code, 0x7F).astype(np.uint8)


def encode_r(r, b16, scale):
    a = (r.astype(np.float64) * np.exp2(127 - per_value(scale.astype(np.float64), len(r)))).astype(np.float32)
    code = np.clip(np.searchsorted(TABLE32, np.where(np.isfinite(a), a, 0), side="right") - 1, 0, 126)
    low, high = TABLE32[code], TABLE32[code + 1]
    u = (b16.astype(np.float32) + np.float32(0.5)) / np.float32(65536)
    code = code + ((a - low) * (a + low) > u * ((high - low) * (high + low)))
    code = np.where((r > 0) & (code == 0), 1, code)
    return np.where(np.isfinite(r), code, 0x7F).astype(np.uint8)


def adamw(p, g, m, v, h, lr_scale=1.0, weight_decay=0.0, dtype=np.float64):
    """(p, m, v, r) after a step; h has lr, beta1, beta2, eps, step, grad_scale.  dtype float32:
    m, v and r by the same fp32 operations as the step's (p in fp64 either way)."""
    f = dtype
    g = np.asarray(g, f) * f(h["grad_scale"])
    m = f(h["beta1"]) * np.asarray(m, f) + f(1 - h["beta1"]) * g
    v = f(h["beta2"]) * np.asarray(v, f) + f(1 - h["beta2"]) * g * g
    r = np.sqrt(v)
    lr = h["lr"] * lr_scale
    hat = (m.astype(np.float64) / (1 - h["beta1"] ** h["step"])) / (
        r.astype(np.float64) / np.sqrt(1 - h["beta2"] ** h["step"]) + h["eps"])
    p = np.asarray(p, np.float64)
    return p * (1 - lr * weight_decay) - lr * hat, m, v, r
