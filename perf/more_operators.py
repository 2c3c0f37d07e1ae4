"""The operators that train experts' matrices in 8 bits, as calls and in plain torch.

Four kinds of work of one GPU's expert share: quantising into E4M3 codes with one fp32 scale for 128 values of a row
(tokens, gradients) or for 128 x 128 values (weights), the experts' products of such operands, their weight
gradients, and the step that orthogonalises a matrix's update by Newton-Schulz products (Muon).

`listed()` and `draw()` give cases, `prepare()` the buffers a program holds before a call, `run()` one pass,
`work()` what a pass has to move and compute, `exact()` the results in 64 bits.
"""
import math
import random

import torch

own = False  # run() makes the library's calls instead of the plain form

_COEF = (3.4445, -4.7750, 2.0315)  # of the Newton-Schulz step
_MUON = dict(lr=3e-4, momentum=0.95, weight_decay=0.1, grad_scale=0.7, steps=5)


# ------------------------------------------------------------------ cases
def _quantise(name, rows, W, source="copy", dtype="bf16", lines="", experts=1, pad=0):
    """source: copy, swiglu or swiglu_bwd; lines: "" (rows only), "line" or "block" (transposed codes too)."""
    return dict(name=name, op="quantise", rows=rows, W=W, source=source, dtype=dtype, lines=lines, experts=experts,
                pad=pad)


def _weights(name, experts, N, K, dtype="bf16", both=True):
    return dict(name=name, op="weights", experts=experts, N=N, K=K, dtype=dtype, both=both)


def _product(name, experts, rows, K, N, skew=0.0, out="bf16"):
    return dict(name=name, op="product", experts=experts, rows=rows, K=K, N=N, skew=skew, out=out)


def _wgrad(name, experts, rows, M, N, skew=0.0, out="bf16", add=False):
    return dict(name=name, op="wgrad", experts=experts, rows=rows, M=M, N=N, skew=skew, out=out, add=add)


def _orth(name, mats, rows, cols, dtype="bf16"):
    return dict(name=name, op="orth", mats=mats, rows=rows, cols=cols, dtype=dtype)


def _muon(name, mats, rows, cols, grads="bf16", nesterov=True, copy=True):
    return dict(name=name, op="muon", mats=mats, rows=rows, cols=cols, grads=grads, nesterov=nesterov, copy=copy)


def listed():
    return [
        # the tokens of a serving step: nothing but latency
        _quantise("quantise_tokens", 4, 7168),
        # the gradient of a training batch's expert rows, for the product with the weights and for the weights' own
        # gradient
        _quantise("quantise_train", 8192, 7168, lines="line", experts=8),
        # SwiGLU of a ragged batch, into the second product's operand and its weight gradient's
        _quantise("quantise_swiglu", 4095, 2048, source="swiglu", lines="block", experts=5),
        # an expert share's gate and up matrices after a step, for the products forward and backward
        _weights("weights_share", 8, 4096, 7168, dtype="f32"),
        # a serving step: a few tokens for each expert, all of the weights
        _product("product_decode", 8, 16, 7168, 4096),
        # a training batch through gate and up
        _product("product_train", 8, 8192, 7168, 4096, skew=0.3),
        # many small experts of odd widths, a few of which get most of the tokens and some none
        _product("product_skewed", 64, 5003, 1472, 2112, skew=1.5, out="f32"),
        # the gradient of the down matrices of the same batch
        _wgrad("wgrad_train", 8, 8192, 7168, 2048, skew=0.3),
        # gradients added up over the parts of a batch, with few tokens for each of many experts
        _wgrad("wgrad_added", 64, 1501, 1472, 704, skew=1.0, out="f32", add=True),
        # the update of a router, for a program that has its own optimizer around it
        _orth("orth_router", 1, 384, 7168, dtype="f32"),
        # many small matrices of odd sizes, taller than wide
        _muon("muon_small", 48, 333, 190, grads="f32", copy=False),
        # the step of an expert share's gate and up matrices
        _muon("muon_experts", 4, 4096, 7168),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi=7168):
    return 64 * _spread(rng, 1, hi // 64)


def draw(rng):
    op = rng.choice(["quantise", "quantise", "weights", "product", "product", "wgrad", "orth", "muon"])
    if op == "quantise":
        W = _width(rng)
        rows = _spread(rng, 1, min(32768, 58720256 // W))
        source = rng.choice(["copy", "copy", "swiglu", "swiglu_bwd"])
        case = _quantise("", rows, W * 2 if source == "swiglu_bwd" else W, source, rng.choice(["bf16", "bf16", "f32"]),
                         rng.choice(["", "line", "block"]), _spread(rng, 1, 32), rng.choice([0, 0, 1, 8]))
    elif op == "weights":
        N, K = _width(rng), _width(rng)
        case = _weights("", _spread(rng, 1, max(1, min(64, 234881024 // (N * K)))), N, K, rng.choice(["bf16", "f32"]),
                        rng.random() < 0.6)
    elif op in ("product", "wgrad"):
        K, N = _width(rng), _width(rng)
        experts = _spread(rng, 1, max(1, min(64, 234881024 // (N * K))))
        rows, skew = _spread(rng, 1, 16384), rng.choice([0.0, 0.3, 1.0, 2.0])
        out = rng.choice(["bf16", "f32"])
        case = _product("", experts, rows, K, N, skew, out) if op == "product" else \
            _wgrad("", experts, rows, K, N, skew, out, out == "f32" and rng.random() < 0.5)
    else:
        rows, cols = _spread(rng, 1, 4096), _spread(rng, 1, 4096)
        mats = _spread(rng, 1, max(1, min(64, 50331648 // (rows * cols))))
        case = _orth("", mats, rows, cols, rng.choice(["bf16", "f32"])) if op == "orth" else \
            _muon("", mats, rows, cols, rng.choice(["bf16", "f32"]), rng.random() < 0.5, rng.random() < 0.5)
    del case["name"]
    return case


# ----------------------------------------------------------------- inputs
def _dtype(case, key="dtype"):
    return torch.bfloat16 if case[key] == "bf16" else torch.float32


def _ceil(a, b):
    return -(-a // b)


def _counts(case, seed):
    """Rows of each expert; the larger skew is, the more of them go to a few."""
    rng = random.Random(seed)
    weight = [math.exp(case.get("skew", 0.5) * rng.gauss(0, 1)) for _ in range(case["experts"])]
    cut, total = [0], sum(weight)
    for w in weight:
        cut.append(cut[-1] + w)
    cut = [round(case["rows"] * c / total) for c in cut]
    return [b - a for a, b in zip(cut, cut[1:])]


def _sums(counts, unit=1):
    out = [0]
    for c in counts:
        out.append(out[-1] + _ceil(c, unit) * unit)
    return out


def _slots(case):
    """Length of the transposed codes' rows: every expert's rows padded to whole blocks."""
    return 128 * (_ceil(case["rows"], 128) + case["experts"] - 1)


def _codes(normal, *shape):
    """Codes of blocks whose largest value is near 448, as a quantiser leaves them."""
    return (normal(*shape) * 110).clamp(-448, 448).to(torch.float8_e4m3fn)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    zeros = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    f8 = torch.float8_e4m3fn
    s, op = dict(case), case["op"]
    if op in ("quantise", "product", "wgrad"):
        s["counts"] = _counts(case, seed)
        s["offsets"] = torch.tensor(_sums(s["counts"]), dtype=torch.int32, device="cuda")
    if op == "quantise":
        rows, W = case["rows"], case["W"]
        width = dict(copy=W, swiglu=2 * W, swiglu_bwd=W)[case["source"]]
        # rows of unlike size, some columns much larger than the rest: what a layer's activations look like
        x = normal(rows, width) * torch.exp(0.5 * normal(rows, 1)) * torch.exp(normal(width))
        s["x"], s["d"] = _padded(x.to(_dtype(case)), case["pad"]), None
        if case["source"] == "swiglu_bwd":
            s["d"] = _padded((1e-3 * normal(rows, W // 2)).to(_dtype(case)), case["pad"])
        s["codes"], s["scales"] = zeros(rows, W, dtype=f8), zeros(_ceil(W, 128), rows)
        s["codes_t"] = s["scales_t"] = None
        if case["lines"]:
            S = _slots(case)
            s["codes_t"] = zeros(W, S, dtype=f8)
            s["scales_t"] = zeros(S // 128, W) if case["lines"] == "line" else zeros(_ceil(W, 128), S // 128)
    elif op == "weights":
        n, N, K = case["experts"], case["N"], case["K"]
        s["w"] = (normal(n, N, K) * K ** -0.5 * torch.exp(0.3 * normal(n, N, 1))).to(_dtype(case))
        s["codes"], s["scales"] = zeros(n, N, K, dtype=f8), zeros(n, _ceil(N, 128), _ceil(K, 128))
        s["codes_t"] = zeros(n, K, N, dtype=f8) if case["both"] else None
        s["scales_t"] = zeros(n, _ceil(K, 128), _ceil(N, 128)) if case["both"] else None
    elif op == "product":
        n, rows, K, N = case["experts"], case["rows"], case["K"], case["N"]
        s["a"], s["sa"] = _codes(normal, rows, K), torch.exp(normal(_ceil(K, 128), rows)) / 448
        s["w"], s["sw"] = _codes(normal, n, N, K), torch.exp(0.3 * normal(n, _ceil(N, 128), _ceil(K, 128))) * 1e-4
        s["y"] = zeros(rows, N, dtype=_dtype(case, "out"))
    elif op == "wgrad":
        n, M, N, S = case["experts"], case["M"], case["N"], _slots(case)
        s["starts"] = _sums(s["counts"], 128)
        place = torch.zeros(S, dtype=torch.bool, device="cuda")
        for c, at in zip(s["counts"], s["starts"]):
            place[at:at + c] = True
        at_rest = zeros((), dtype=f8).view(torch.uint8)
        s["dy"], s["sdy"] = _codes(normal, M, S), torch.exp(normal(S // 128, M)) * 1e-6
        s["x"], s["sx"] = _codes(normal, N, S), torch.exp(0.5 * normal(_ceil(N, 128), S // 128)) / 448
        for name in ("dy", "x"):  # places between the experts hold zeros, as the quantiser leaves them
            s[name] = torch.where(place, s[name].view(torch.uint8), at_rest).view(f8)
        s["dw"] = (1e-3 * normal(n, M, N)).to(_dtype(case, "out"))
    else:
        n, m, c = case["mats"], case["rows"], case["cols"]

        def like_gradients(size):  # a few directions that many tokens agree on, and noise
            few = torch.matmul(normal(n, m, 4) * torch.exp(normal(4)), normal(n, 4, c))
            return size * (normal(n, m, c) + 0.5 * few)
        if op == "orth":
            s["x"] = like_gradients(1e-3).to(_dtype(case))
            s["out"] = torch.empty(n, m, c, dtype=torch.bfloat16, device="cuda")
        else:
            s["p"], s["grad"], s["m"] = 0.03 * normal(n, m, c), like_gradients(1e-3).to(_dtype(case, "grads")), \
                like_gradients(1e-2)
            s["p_bf16"] = s["p"].bfloat16() if case["copy"] else None
        if own:
            import token_dispatch_grouped_top_amd as mok
            s["ws"] = torch.empty(mok.mok_muon_workspace_size(n, m, c), dtype=torch.uint8, device="cuda")
    return s


def _padded(x, pad):
    """x as a view of rows that are `pad` wider."""
    if not pad:
        return x.contiguous()
    wide = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


# ------------------------------------------------------------- plain forms
# The code is that of the quotient in 32 bits.  Scale and quotient are formed in 64 bits and then rounded: of values in
# 16 bits, one in a hundred lies in the middle between two codes.
def _to_codes(x, scale):
    return (x.double() / scale.double()).float().clamp(-448, 448).to(torch.float8_e4m3fn)


def _scale(largest):
    return (largest.double() / 448).float().clamp(min=2.0 ** -126)


def _by_rows(x):
    """Codes of x [..., R, C] with a scale for 128 columns of each row, and the scales [..., R, blocks]."""
    C = x.shape[-1]
    padded = torch.nn.functional.pad(x, (0, -C % 128))
    scale = _scale(padded.abs().unflatten(-1, (-1, 128)).amax(-1))
    return _to_codes(x, scale.repeat_interleave(128, -1)[..., :C]), scale


def _by_blocks(x):
    """Codes of x [..., R, C] with a scale for 128 x 128 values, and the scales."""
    R, C = x.shape[-2:]
    padded = torch.nn.functional.pad(x, (0, -C % 128, 0, -R % 128))
    scale = _scale(padded.abs().unflatten(-1, (-1, 128)).amax(-1).unflatten(-2, (-1, 128)).amax(-2))
    spread = scale.repeat_interleave(128, -1).repeat_interleave(128, -2)[..., :R, :C]
    return _to_codes(x, spread), scale


def _source(s):
    x = s["x"].float()
    if s["source"] == "copy":
        return x
    g, u = x.chunk(2, 1)
    gate = 1 / (1 + torch.exp(-g))
    if s["source"] == "swiglu":
        return g * gate * u
    d = s["d"].float()
    return torch.cat([d * u * gate * (1 + g * (1 - gate)), d * g * gate], 1)


def _plain_quantise(s):
    x = _source(s)
    codes, scale = _by_rows(x)
    s["codes"].copy_(codes)
    s["scales"].copy_(scale.T)
    if s["lines"]:
        starts, ends = _sums(s["counts"], 128), _sums(s["counts"])
        wide = torch.cat([torch.nn.functional.pad(x[b - c:b], (0, 0, 0, -c % 128)) for b, c in zip(ends[1:], s["counts"])])
        codes, scale = (_by_rows if s["lines"] == "line" else _by_blocks)(wide.T)
        s["codes_t"][:, :starts[-1]] = codes
        (s["scales_t"].T if s["lines"] == "line" else s["scales_t"])[:, :starts[-1] // 128] = scale


def _plain_weights(s):
    w = s["w"].float()
    codes, scale = _by_blocks(w)
    s["codes"].copy_(codes)
    s["scales"].copy_(scale)
    if s["both"]:
        s["codes_t"].copy_(codes.view(torch.uint8).mT.contiguous().view(torch.float8_e4m3fn))
        s["scales_t"].copy_(scale.mT)


def _values(codes, scale):
    """What codes [..., C] with a scale for 128 of them stand for."""
    return codes.float() * scale.repeat_interleave(128, -1)[..., :codes.shape[-1]]


def _plain_product(s):
    a, ends = _values(s["a"], s["sa"].T), _sums(s["counts"])
    w = _values(s["w"], s["sw"].repeat_interleave(128, -2)[:, :s["N"]])
    s["y"].copy_(torch.cat([a[b - c:b] @ w[e].T for e, (b, c) in enumerate(zip(ends[1:], s["counts"]))]))


def _plain_wgrad(s):
    dy, x = _values(s["dy"], s["sdy"].T), _values(s["x"], s["sx"].repeat_interleave(128, 0)[:s["N"]])
    dw = torch.stack([dy[:, b:b + c] @ x[:, b:b + c].T for b, c in zip(s["starts"], s["counts"])])
    s["dw"].copy_(s["dw"] + dw if s["add"] else dw)


def _plain_orth(v):
    wide = v.shape[-2] <= v.shape[-1]
    x = v if wide else v.mT
    norm = torch.linalg.vector_norm(x, dim=(-2, -1), keepdim=True, dtype=torch.float64)
    x = (x / norm.clamp(min=1e-300)).float()
    a, b, c = _COEF
    for _ in range(_MUON["steps"]):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x if wide else x.mT


def _plain_muon(s):
    h = _MUON
    g = h["grad_scale"] * s["grad"].float()
    s["m"].mul_(h["momentum"]).add_(g)
    v = g + h["momentum"] * s["m"] if s["nesterov"] else s["m"]
    x = _plain_orth(v)
    s["p"].mul_(1 - h["lr"] * h["weight_decay"]).sub_(h["lr"] * _size(s) * x)
    if s["copy"]:
        s["p_bf16"].copy_(s["p"])


def _size(s):
    """Factor of the orthogonal update with which its values are as large as AdamW's."""
    return 0.2 * math.sqrt(max(s["rows"], s["cols"]))


# -------------------------------------------------------------------- run
def run(state):
    s, op = state, state["op"]
    if own:
        _run_own(s, op)
    elif op == "orth":
        s["out"].copy_(_plain_orth(s["x"].float()))
    else:
        dict(quantise=_plain_quantise, weights=_plain_weights, product=_plain_product, wgrad=_plain_wgrad,
             muon=_plain_muon)[op](s)
    if op in ("quantise", "weights"):
        return {name: s[name] for name in ("codes", "scales", "codes_t", "scales_t")}
    if op == "muon":
        return {name: s[name] for name in ("p", "p_bf16", "m")}
    return s[dict(product="y", wgrad="dw", orth="out")[op]]


def _run_own(s, op):
    import token_dispatch_grouped_top_amd as mok
    if op == "quantise":
        kind = dict(copy=mok.MOK_BLOCK8_COPY, swiglu=mok.MOK_BLOCK8_SWIGLU, swiglu_bwd=mok.MOK_BLOCK8_SWIGLU_BWD)
        mok.mok_block8_quantise(s["x"], s["rows"], s["W"], s["codes"], s["scales"], source=kind[s["source"]], d=s["d"],
                                codes_t=s["codes_t"], scales_t=s["scales_t"],
                                t_scales=mok.MOK_BLOCK8_BLOCKS if s["lines"] == "block" else mok.MOK_BLOCK8_LINES,
                                offsets=s["offsets"], n_local=s["experts"])
    elif op == "weights":
        mok.mok_block8_quantise_weights(s["w"], s["experts"], s["N"], s["K"], s["codes"], s["scales"],
                                        codes_t=s["codes_t"], scales_t=s["scales_t"])
    elif op == "product":
        mok.mok_block8_gemm(s["a"], s["sa"], s["rows"], s["K"], s["w"], s["sw"], s["N"], s["y"], offsets=s["offsets"],
                            n_local=s["experts"])
    elif op == "wgrad":
        mok.mok_block8_wgrad(s["dy"], s["sdy"], s["M"], s["x"], s["sx"], s["N"], s["rows"], s["dw"],
                             offsets=s["offsets"], n_local=s["experts"], accumulate=int(s["add"]))
    elif op == "orth":
        mok.mok_orthogonalise(s["x"], s["mats"], s["rows"], s["cols"], s["out"], s["ws"], steps=_MUON["steps"],
                              coefficients=_COEF)
    else:
        mok.mok_muon_step(s["p"], s["grad"], s["m"], s["mats"], s["rows"], s["cols"], s["ws"], lr=_MUON["lr"],
                          momentum=_MUON["momentum"], weight_decay=_MUON["weight_decay"],
                          grad_scale=_MUON["grad_scale"], scale=_size(s), nesterov=int(s["nesterov"]),
                          steps=_MUON["steps"], coefficients=_COEF, p_bf16=s["p_bf16"])


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "quantise":
        cells, size = case["rows"] * case["W"], 2 if case["dtype"] == "bf16" else 4
        read = dict(copy=1, swiglu=2, swiglu_bwd=1.5)[case["source"]] * size
        return {"bytes": int(cells * (read + (1 + 4 / 128) * (2 if case["lines"] else 1))),
                "flops": cells * dict(copy=3, swiglu=10, swiglu_bwd=12)[case["source"]]}
    if op == "weights":
        cells = case["experts"] * case["N"] * case["K"]
        return {"bytes": cells * ((2 if case["dtype"] == "bf16" else 4) + (2 if case["both"] else 1)), "flops": 3 * cells}
    if op == "product":
        rows, K, N = case["rows"], case["K"], case["N"]
        return {"bytes": rows * K + min(case["experts"], rows) * N * K + rows * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * rows * K * N}
    if op == "wgrad":
        rows, M, N = case["rows"], case["M"], case["N"]
        out = case["experts"] * M * N * (2 if case["out"] == "bf16" else 4) * (2 if case["add"] else 1)
        return {"bytes": rows * (M + N) + out, "flops": 2 * rows * M * N}
    m, n = sorted((case["rows"], case["cols"]))
    cells = case["mats"] * m * n
    size = 2 if case.get("dtype", case.get("grads")) == "bf16" else 4
    # the products of a step are X X^T and A^2, symmetric, and B X
    return {"bytes": cells * (size + 2 if op == "orth" else size + 16 + (2 if case["copy"] else 0)),
            "flops": case["mats"] * _MUON["steps"] * (m * m * n + m ** 3 + 2 * m * m * n)}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return dict(quantise=_exact_quantise, weights=_exact_weights, product=_exact_product, wgrad=_exact_wgrad,
                orth=_exact_orth_out, muon=_exact_muon)[case["op"]](s)


def _table():
    """The values of the codes 0 to 126."""
    return torch.tensor([f * 2.0 ** -9 for f in range(8)] +
                        [(8 + f) * 2.0 ** (e - 10) for e in range(1, 16) for f in range(8)][:119], dtype=torch.float64,
                        device="cuda")


def _exact_code(x, largest):
    """Code of the value nearest to x / scale in 32 bits (in the middle: the even code), and the scale in 32 bits."""
    scale = (largest / 448).float().double().clamp(min=2.0 ** -126)
    table, a = _table(), (x / scale).abs().float().double()
    low = (torch.bucketize(a, table, right=True) - 1).clamp(0, 125)
    over = 2 * a - (table[low] + table[low + 1])
    code = low + ((over > 0) | ((over == 0) & (low % 2 == 1)))
    return (code + 128 * (x < 0)).to(torch.uint8).view(torch.float8_e4m3fn), scale


def _exact_quantise(s):
    x = s["x"].double()
    if s["source"] != "copy":
        half = x.shape[1] // 2
        g, u = x[:, :half], x[:, half:]
        silu, up = torch.sigmoid(g) * g, u
        x = silu * up
        if s["source"] == "swiglu_bwd":
            slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)
            x = torch.cat([s["d"].double() * up * slope, s["d"].double() * silu], 1)
    rows, W = x.shape
    out = {name: None if s[name] is None else s[name].clone() for name in ("codes", "scales", "codes_t", "scales_t")}
    for b, c in enumerate(range(0, W, 128)):
        part = x[:, c:c + 128]
        code, scale = _exact_code(part, part.abs().amax(1, keepdim=True))
        out["codes"].view(torch.uint8)[:, c:c + 128], out["scales"][b] = code.view(torch.uint8), scale[:, 0].float()
    if s["lines"]:
        row = 0
        for count, start in zip(s["counts"], _sums(s["counts"], 128)):
            for j in range(0, count, 128):
                part, at = x[row + j:row + min(j + 128, count)], start + j
                if s["lines"] == "line":
                    code, scale = _exact_code(part, part.abs().amax(0, keepdim=True))
                    out["scales_t"][at // 128] = scale[0].float()
                else:
                    largest = torch.nn.functional.pad(part.abs().amax(0), (0, -W % 128)).view(-1, 128).amax(1)
                    code, scale = _exact_code(part, largest.repeat_interleave(128)[:W])
                    out["scales_t"][:, at // 128] = scale[::128].float()
                out["codes_t"].view(torch.uint8)[:, at:at + part.shape[0]] = code.view(torch.uint8).T
            row += count
    return out


def _exact_weights(s):
    out = {name: None if s[name] is None else s[name].clone() for name in ("codes", "scales", "codes_t", "scales_t")}
    for e in range(s["experts"]):
        w = s["w"][e].double()
        wide = torch.nn.functional.pad(w.abs(), (0, -s["K"] % 128, 0, -s["N"] % 128))
        largest = torch.nn.functional.max_pool2d(wide[None], 128)[0]
        code, _ = _exact_code(w, largest.repeat_interleave(128, 0).repeat_interleave(128, 1)[:s["N"], :s["K"]])
        scale = (largest / 448).float().clamp(min=2.0 ** -126)
        out["codes"].view(torch.uint8)[e], out["scales"][e] = code.view(torch.uint8), scale
        if s["both"]:
            out["codes_t"].view(torch.uint8)[e], out["scales_t"][e] = code.view(torch.uint8).T, scale.T
    return out


def _double(codes):
    """What the codes stand for, in 64 bits."""
    c = codes.view(torch.uint8).long()
    v = torch.cat([_table(), torch.tensor([math.nan], dtype=torch.float64, device="cuda")])
    return torch.cat([v, -v])[c]


def _exact_product(s):
    y, row = torch.zeros(s["rows"], s["N"], dtype=torch.float64, device="cuda"), 0
    for e, count in enumerate(s["counts"]):
        for k in range(0, s["K"], 128) if count else ():
            a = _double(s["a"][row:row + count, k:k + 128]) * s["sa"][k // 128, row:row + count, None].double()
            each = s["sw"][e, :, k // 128].double().repeat_interleave(128)[:s["N"], None]
            y[row:row + count] += torch.mm(a, (_double(s["w"][e][:, k:k + 128]) * each).T.contiguous())
        row += count
    return y


def _exact_wgrad(s):
    dw = s["dw"].double() if s["add"] else torch.zeros(s["dw"].shape, dtype=torch.float64, device="cuda")
    for e, (start, count) in enumerate(zip(s["starts"], s["counts"])):
        for at in range(start, start + count, 128):
            dy = _double(s["dy"][:, at:at + 128]) * s["sdy"][at // 128, :, None].double()
            x = _double(s["x"][:, at:at + 128]) * s["sx"][:, at // 128].double().repeat_interleave(128)[:s["N"], None]
            dw[e] += torch.mm(dy, x.T.contiguous())
    return dw


def _exact_orth(v):
    """The polynomial of each matrix, one after another, on its smaller side."""
    out = torch.empty(v.shape, dtype=torch.float64, device="cuda")
    a, b, c = _COEF
    for i in range(v.shape[0]):
        x = v[i].double()
        tall = x.shape[0] > x.shape[1]
        x = x.T.contiguous() if tall else x
        x = x / x.square().sum().sqrt()
        for _ in range(_MUON["steps"]):
            gram = torch.mm(x, x.T.contiguous())
            x = torch.mm(c * torch.mm(gram, gram) + b * gram + a * torch.eye(len(x), dtype=x.dtype, device="cuda"), x)
        out[i] = x.T if tall else x
    return out


def _exact_orth_out(s):
    return _exact_orth(s["x"])


def _exact_muon(s):
    h = _MUON
    m, g = s["m"].double(), s["grad"].double() * h["grad_scale"]
    m = h["momentum"] * m + g
    x = _exact_orth(g + h["momentum"] * m if s["nesterov"] else m)
    p = s["p"].double() * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * _size(s) * x
    return {"p": p, "p_bf16": p if s["copy"] else None, "m": m}
