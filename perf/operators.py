"""The operators of routed training and serving, as calls and in plain torch.

Four operators of one GPU's share of an MoE layer: the scored route (softmax
or sigmoid scores, a balance bias, groups, top-k, renormalised weights), its
backward, the update of the balance bias from the experts' load, and the AdamW
step over many tensors with states in 32 or 8 bits.

`listed()` and `draw()` give cases, `prepare()` the buffers a program holds
before a call, `run()` one pass, `work()` what a pass has to move and compute,
`exact()` the results in 64 bits.
"""
import math

import torch

own = False  # run() makes the library's calls instead of the plain form

_M32 = 0xFFFFFFFF
_ADAMW = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, step=120, grad_scale=0.7, weight_decay=0.1, seed=20)


# ------------------------------------------------------------------ cases
def _route(name, T, E, k, score, groups=1, top_groups=1, group_rule="max", bias=True, renorm=True, scale=1.0,
           dtype="f32", pad=0, masked=0.0, load=False):
    return dict(name=name, op="route", T=T, E=E, k=k, score=score, groups=groups, top_groups=top_groups,
                group_rule=group_rule, bias=bias, renorm=renorm, scale=scale, dtype=dtype, pad=pad, masked=masked,
                load=load)


def _route_bwd(name, T, E, k, score, renorm=True, scale=1.0, dtype="f32", pad=0, empty=0.0):
    return dict(name=name, op="route_bwd", T=T, E=E, k=k, score=score, renorm=renorm, scale=scale, dtype=dtype,
                pad=pad, empty=empty)


def _adamw(name, sizes, states, grads="bf16", copy=True, scalars="host"):
    return dict(name=name, op="adamw", sizes=sizes, states=states, grads=grads, copy=copy, scalars=scalars)


def listed():
    many = ",".join(str(4096 + 977 * i % 9001 + 3 * i) for i in range(200))
    return [
        # one new token of a serving step: nothing but latency
        _route("route_token", 1, 384, 8, "sigmoid", scale=2.5),
        # one source partition's tokens, 8 of 384 experts, counting the load as a training step does
        _route("route_partition", 1024, 384, 8, "sigmoid", scale=2.5, load=True),
        # a training batch routed within groups, counting the load for the balance bias
        _route("route_groups", 16384, 256, 8, "sigmoid", 8, 4, "top2", scale=2.5, load=True),
        # bf16 logits of a ragged batch in a padded buffer: some experts are switched off, the last rows are padding
        _route("route_masked", 4095, 160, 6, "softmax", 8, 3, "max", bias=False, renorm=False, scale=16.0, dtype="bf16",
               pad=8, masked=0.05),
        # the same training batch's gradient: only picked experts have one
        _route_bwd("bwd_renorm", 16384, 256, 8, "sigmoid", scale=2.5),
        # every expert has a gradient; some picks are empty
        _route_bwd("bwd_dense", 4095, 160, 6, "softmax", renorm=False, scale=16.0, dtype="bf16", pad=8, empty=0.02),
        # the bias of one layer, after its step
        dict(name="bias_layer", op="bias", layers=1, E=384, rate=1e-3, clear=True),
        # the biases of a deep model at once, the loads kept for a report
        dict(name="bias_model", op="bias", layers=60, E=1000, rate=1e-3, clear=False),
        # a router's weights and its bias, gradients in 32 bits
        _adamw("adamw_router", "2752512,384", "f32", grads="f32", copy=False),
        # the expert share of a layer: [8][4096][7168] and [8][7168][2048]
        _adamw("adamw_experts", "234881024,117440512", "f32"),
        # two experts with states in 8 bits, the step's numbers read on the device
        _adamw("adamw_experts_8bit", "58720256,29360128", "8bit", scalars="device"),
        # many small tensors of odd sizes in one step
        _adamw("adamw_many", many, "8bit"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "adamw", "adamw", "bias"])
    if op in ("route", "route_bwd"):
        T = _spread(rng, 1, 32768)
        score, dtype = rng.choice(["sigmoid", "softmax"]), rng.choice(["f32", "bf16"])
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _spread(rng, 4, 512 // groups)
        top_groups = rng.randint(1, groups)
        renorm = rng.random() < 0.6
        k = rng.randint(2 if renorm else 1, min(12, top_groups * (E // groups)))
        scale, pad = rng.choice([1.0, 2.5]), rng.choice([0, 0, 1, 8])
        if op == "route_bwd":
            case = _route_bwd("", T, E, k, score, renorm, scale, dtype, pad, rng.choice([0.0, 0.05]) if T > 64 else 0.0)
        else:
            case = _route("", T, E, k, score, groups, top_groups, rng.choice(["max", "top2"]), rng.random() < 0.7,
                          renorm, scale, dtype, pad, rng.choice([0.0, 0.1]), rng.random() < 0.5)
    elif op == "bias":
        case = dict(name="", op="bias", layers=_spread(rng, 1, 100), E=_spread(rng, 4, 4096), rate=rng.choice([1e-3, 1e-2]),
                    clear=rng.random() < 0.5)
    else:
        count = _spread(rng, 1, 200)
        each = _spread(rng, 64, max(64, (1 << 25) // count))
        sizes = ",".join(str(max(1, int(each * rng.uniform(0.5, 1.5)))) for _ in range(count))
        case = _adamw("", sizes, rng.choice(["f32", "8bit"]), rng.choice(["f32", "bf16"]), rng.random() < 0.5,
                      rng.choice(["host", "device"]))
    del case["name"]
    return case


# ----------------------------------------------------------------- inputs
def _dtype(case, key="dtype"):
    return torch.bfloat16 if case[key] == "bf16" else torch.float32


def _sizes(case):
    return [int(n) for n in case["sizes"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    uniform = lambda *shape: torch.rand(*shape, generator=gen, device="cuda")  # noqa: E731
    state = dict(case)
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        # scores of the router on normalised tokens, plus what makes some experts popular
        logits = normal(T, E) + 0.5 * normal(E)
        if case["masked"]:
            logits[:, uniform(E) < case["masked"]] = -math.inf  # experts that are switched off
            logits[T - int(case["masked"] * T):] = -math.inf    # padding behind the last token
        state["logits"] = _padded(logits.to(_dtype(case)), case["pad"])
        state["bias"] = 0.1 * normal(E) if case["bias"] else None
        state["idx"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        state["gate"] = torch.empty(T, k, device="cuda")
        state["load"] = torch.randint(0, 1000, (E,), generator=gen, device="cuda", dtype=torch.int32) if case["load"] else None
    elif case["op"] == "route_bwd":
        T, E, k = case["T"], case["E"], case["k"]
        logits = (normal(T, E) + 0.5 * normal(E)).to(_dtype(case))
        idx = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k].int()
        idx[uniform(T, k) < case["empty"]] = -1  # picks of tokens with too few eligible experts
        state["logits"], state["idx"], state["dgate"] = _padded(logits, case["pad"]), idx.contiguous(), normal(T, k)
        state["dlogits"] = _padded(torch.zeros(T, E, dtype=_dtype(case), device="cuda"), case["pad"])
    elif case["op"] == "bias":
        shape = (case["layers"], case["E"])
        state["load"] = torch.poisson(200 * torch.exp(0.5 * normal(*shape)), generator=gen).int()
        state["bias"] = 0.1 * normal(*shape)
    else:
        state["flat"], state["tensors"] = _adamw_buffers(case, normal, uniform)
        h = _ADAMW
        state["scalars"] = None
        if case["scalars"] == "device":  # lr, grad_scale, step, skip
            numbers = torch.tensor([h["lr"], h["grad_scale"], 0.0, 0.0], device="cuda")
            numbers.view(torch.int32)[2:] = torch.tensor([h["step"], 0], dtype=torch.int32, device="cuda")
            state["scalars"] = numbers
    if own:
        # what a program keeps beside its buffers: the router's description, the optimizer's list of tensors
        import token_dispatch_grouped_top_amd as mok
        if case["op"] in ("route", "route_bwd"):
            state["router"] = mok.mok_router_desc(
                n_experts=case["E"], top_k=case["k"],
                score=mok.MOK_SCORE_SIGMOID if case["score"] == "sigmoid" else mok.MOK_SCORE_SOFTMAX,
                n_groups=case.get("groups", 1), top_groups=case.get("top_groups", 1),
                group_rule=mok.MOK_GROUP_TOP2 if case.get("group_rule") == "top2" else mok.MOK_GROUP_MAX,
                renorm=int(case["renorm"]), scale=case["scale"])
        elif case["op"] == "adamw":
            state["list"] = mok.AdamwTensors(state["tensors"])
    return state


def _padded(x, pad):
    """x as a view of rows that are `pad` wider."""
    if not pad:
        return x.contiguous()
    wide = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def _adamw_buffers(case, normal, uniform):
    """Parameters, gradients and states, each kind in one buffer in which every tensor begins at a multiple of 256
    values; the buffers, and each tensor's slices of them."""
    sizes = _sizes(case)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + -(-n // 256) * 256)
    total = starts[-1]
    p = 0.02 * normal(total)
    grad = (1e-2 * normal(total)).to(_dtype(case, "grads"))
    m = grad.float() + 5e-3 * normal(total)
    v = 1e-4 * (uniform(total) + 0.05)
    flat = dict(p=p, m=m, v=v)
    if case["states"] == "8bit":
        middle = torch.full((total,), 1 << 15, dtype=torch.int32, device=p.device)
        flat["m"], flat["m_scale"] = _encode_m(m, middle)
        flat["v"], flat["v_scale"] = _encode_r(v.sqrt(), middle)
    if case["copy"]:
        flat["p_bf16"] = p.bfloat16()
    cut = lambda name, x, at, n: x[at // 32:at // 32 + -(-n // 32)] if name.endswith("scale") else x[at:at + n]  # noqa: E731
    tensors = [{name: cut(name, x, at, n) for name, x in [*flat.items(), ("grad", grad)]} for at, n in zip(starts, sizes)]
    for i, t in enumerate(tensors):
        t["weight_decay"] = 0.0 if i % 2 else _ADAMW["weight_decay"]  # none on biases and norms
    return flat, tensors


# -------------------------------------------------- 8-bit states (blocks of 32)
# E4M3 values with one scale 2^(byte - 127) for 32 of them, the smallest with
# which the largest does not pass 448.  m is rounded up or down at random, so
# that its mean is kept; so is v, held as r = sqrt(v).  With nearest rounding a
# state would stand still: a step often moves it by less than half a quantum.
def _blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % 32)).view(-1, 32)


def _two(e):
    """2^e for whole e from -126 to 127."""
    return ((e + 127) << 23).view(torch.float32)


def _scale_exp(x):
    bits = _blocks(x.abs()).amax(1).view(torch.int32)
    return ((bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(-127, 127)


def _per_value(x, n):
    return x.repeat_interleave(32)[:n]


def _decode(code, scale):
    c = code.int()
    e, f = (c >> 3) & 15, c & 7
    a = torch.where(e > 0, 8 + f, f).float() * _two(e.clamp(min=1) - 10)
    return torch.where(c > 127, -a, a) * _per_value(_two((scale.int() - 127).clamp(min=-126)), code.numel())


def _code_below(a):
    """The code of the largest E4M3 value that is not above a (at most 448)."""
    return torch.where(a >= 2.0 ** -6, (a.view(torch.int32) >> 20) - 960, (a * 512).int())


def _encode_m(m, noise):
    exp = _scale_exp(m)
    a = m.abs() * _per_value(_two(-exp), m.numel())
    code = torch.where(a >= 2.0 ** -6, ((a.view(torch.int32) + 16 * noise + 8) >> 20) - 960,
                       (a * 512 + (noise + 0.5) / 65536).int())
    return torch.where(m < 0, code | 128, code).to(torch.uint8), (exp + 127).to(torch.uint8)


def _encode_r(r, noise):
    exp = _scale_exp(r)
    a = r * _per_value(_two(-exp), r.numel())
    code = _code_below(a)
    unit = torch.full_like(exp, 127)
    low, high = _decode(code, unit), _decode(code + 1, unit)
    up = (a - low) * (a + low) > (noise + 0.5) / 65536 * ((high - low) * (high + low))  # the mean of r^2 is kept
    code = torch.where(r > 0, (code + up).clamp(min=1), 0)
    return code.to(torch.uint8), (exp + 127).to(torch.uint8)


def _hash(x):
    x = x & _M32
    x = ((x ^ (x >> 16)) * 0x9E3779B1) & _M32
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & _M32
    return x ^ (x >> 16)


def _noise(n, tensor, device):
    """32 bits for each element of the step's tensor number `tensor`: 16 for m, 16 for v."""
    key = _hash(_hash(_ADAMW["seed"] + 0x9E3779B1 * _ADAMW["step"]) + tensor)
    h = _hash(torch.arange(n, device=device) + key)
    return (h & 0xFFFF).int(), (h >> 16).int()


# ------------------------------------------------------------- plain forms
def _scores(logits, score):
    """Scores of the eligible experts, 0 for the others (a logit of -inf or NaN)."""
    eligible = logits > -math.inf
    if score == "sigmoid":
        return torch.where(eligible, 1 / (1 + torch.exp(-logits)), 0), eligible
    top = torch.where(eligible, logits, torch.finfo(logits.dtype).min).amax(1, keepdim=True)
    e = torch.where(eligible, torch.exp(logits - top), 0)
    return e / e.sum(1, keepdim=True).clamp(min=1e-30), eligible


def _largest(x, k):
    """Values and places of the k largest of each row; equal ones in the order of their places."""
    values, places = torch.sort(x, dim=1, descending=True, stable=True)
    return values[:, :k], places[:, :k]


def _plain_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    # 64 bits for the order: two experts' scores can be nearer to each other than 32 bits tell
    choice, eligible = _scores(s["logits"].double(), s["score"])
    if s["bias"] is not None:
        choice = choice + s["bias"].double()
    choice = torch.where(eligible, choice, -math.inf)
    if G > 1:
        best = _largest(choice.reshape(T * G, E // G), 2)[0]
        group = best[:, 0]
        if s["group_rule"] == "top2":
            group = group + torch.where(best[:, -1] > -math.inf, best[:, -1], 0)
        chosen = torch.zeros(T, G, dtype=torch.bool, device=choice.device)
        chosen.scatter_(1, _largest(group.view(T, G), s["top_groups"])[1], True)
        choice = torch.where(chosen.repeat_interleave(E // G, 1), choice, -math.inf)
    values, places = _largest(choice, k)
    picked = values > -math.inf
    scores = torch.where(picked, _scores(s["logits"].float(), s["score"])[0].gather(1, places), 0)
    if s["renorm"]:
        scores = scores / scores.sum(1, keepdim=True).clamp(min=1e-30)
    s["idx"].copy_(torch.where(picked, places, -1))
    s["gate"].copy_(s["scale"] * scores)
    if s["load"] is not None:
        s["load"].scatter_add_(0, places.reshape(-1), picked.reshape(-1).int())


def _plain_route_bwd(s):
    picked = s["idx"] >= 0
    at = s["idx"].clamp(min=0).long()
    scores = _scores(s["logits"].float(), s["score"])[0]
    at_picks = torch.where(picked, scores.gather(1, at), 0)
    dgate = torch.where(picked, s["scale"] * s["dgate"], 0)
    if s["renorm"]:  # gate = scale * u, u = scores / their sum
        u = at_picks / at_picks.sum(1, keepdim=True).clamp(min=1e-30)
        d = u * (dgate - (u * dgate).sum(1, keepdim=True))
        d = d * (1 - at_picks) if s["score"] == "sigmoid" else d
        rest = 0
    elif s["score"] == "sigmoid":
        d, rest = dgate * at_picks * (1 - at_picks), 0
    else:
        d, rest = dgate * at_picks, -scores * (dgate * at_picks).sum(1, keepdim=True)
    grad = torch.zeros_like(scores).scatter_add_(1, at, torch.where(picked, d, 0)) + rest
    s["dlogits"].copy_(grad)


def _plain_bias(s):
    load = s["load"].long()
    s["bias"] += s["rate"] * torch.sign(load.sum(1, keepdim=True) - s["E"] * load).float()
    if s["clear"]:
        s["load"].zero_()


def _plain_adamw(s, t, tensor):
    h = _ADAMW
    quantised = s["states"] == "8bit"
    g = t["grad"].float() * h["grad_scale"]
    m = _decode(t["m"], t["m_scale"]) if quantised else t["m"]
    v = _decode(t["v"], t["v_scale"]).square() if quantised else t["v"]
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g * g
    r = v.sqrt()
    change = m / (r / math.sqrt(1 - h["beta2"] ** h["step"]) + h["eps"])
    t["p"].mul_(1 - h["lr"] * t["weight_decay"]).sub_(h["lr"] / (1 - h["beta1"] ** h["step"]) * change)
    new = dict(m=m, v=v)
    if quantised:
        noise = _noise(g.numel(), tensor, g.device)
        new["m"], new["m_scale"] = _encode_m(m, noise[0])
        new["v"], new["v_scale"] = _encode_r(r, noise[1])
    if s["copy"]:
        new["p_bf16"] = t["p"]
    [t[name].copy_(x) for name, x in new.items()]


# -------------------------------------------------------------------- run
def run(state):
    s, op = state, state["op"]
    if own:
        import token_dispatch_grouped_top_amd as mok
        if op == "route":
            mok.mok_route_scored(s["router"], s["logits"], s["T"], s["idx"], s["gate"], bias=s["bias"], load=s["load"])
        elif op == "route_bwd":
            mok.mok_route_scored_backward(s["router"], s["logits"], s["T"], s["idx"], s["dgate"], s["dlogits"])
        elif op == "bias":
            mok.mok_route_bias_update(s["load"], s["layers"], s["E"], s["rate"], s["bias"], clear_load=int(s["clear"]))
        else:
            mok.mok_adamw_step(s["list"], lr=_ADAMW["lr"], beta1=_ADAMW["beta1"], beta2=_ADAMW["beta2"],
                               eps=_ADAMW["eps"], step=_ADAMW["step"], grad_scale=_ADAMW["grad_scale"],
                               seed=_ADAMW["seed"], scalars=s["scalars"])
    elif op == "adamw":
        [_plain_adamw(s, t, i) for i, t in enumerate(s["tensors"])]
    else:
        dict(route=_plain_route, route_bwd=_plain_route_bwd, bias=_plain_bias)[op](s)
    if op == "route":
        return {"idx": s["idx"], "gate": s["gate"], "load": s["load"]}
    if op == "route_bwd":
        return s["dlogits"]
    if op == "bias":
        return {"bias": s["bias"], "load": s["load"]}
    return {name: _values(name, x) for name, x in s["flat"].items()}


def _values(name, x):
    """A buffer of codes as the values that they stand for (a view)."""
    if x.dtype != torch.uint8:
        return x
    return x.view(torch.float8_e8m0fnu if name.endswith("scale") else torch.float8_e4m3fn)


# ------------------------------------------------------------------- work
def work(case):
    if case["op"] == "bias":
        cells = case["layers"] * case["E"]
        return {"bytes": cells * (4 + 8 + (4 if case["clear"] else 0)), "flops": 3 * cells}
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        state = 4 * (1 + 1 / 32) if case["states"] == "8bit" else 16
        return {"bytes": int(n * (8 + state + (2 if case["grads"] == "bf16" else 4) + (2 if case["copy"] else 0))),
                "flops": 16 * n}
    T, E, k, size = case["T"], case["E"], case["k"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "route":
        return {"bytes": T * E * size + 8 * T * k + (4 * E if case["bias"] else 0) + (8 * E if case["load"] else 0),
                "flops": T * E * 4 + T * k * 4}
    dense = case["score"] == "softmax" and not case["renorm"]
    return {"bytes": T * E * size + T * k * 8 + (T * E if dense else T * k) * size,  # every gradient is written
            "flops": (6 * T * E if dense else 0) + 10 * T * k}


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return dict(route=_exact_route, route_bwd=_exact_route_bwd, bias=_exact_bias, adamw=_exact_adamw)[case["op"]](s)


def _log_scores(logits, score):
    """Logarithms of the scores, -inf for an expert that is not eligible."""
    if score == "sigmoid":
        return -torch.logaddexp(torch.zeros_like(logits), -logits)
    return logits - torch.logsumexp(logits, 1, keepdim=True).nan_to_num(neginf=0.0)


def _exact_gates(s, logits, picks):
    """Gates of given picks (a list of columns of expert ids, -1 for none)."""
    log = _log_scores(logits, s["score"])
    log = torch.stack([torch.where(p >= 0, log.gather(1, p.clamp(min=0)[:, None])[:, 0], -math.inf) for p in picks], 1)
    if s["renorm"]:
        log = log - torch.logsumexp(log, 1, keepdim=True).nan_to_num(neginf=0.0)
    return s["scale"] * log.exp()


def _exact_route(s):
    logits = s["logits"].double()
    choice = _log_scores(logits, s["score"]).exp() + (0 if s["bias"] is None else s["bias"].double())
    choice[logits == -math.inf] = -math.inf
    expert = torch.arange(s["E"], device="cuda").expand_as(choice)

    def first(x, best):  # the lowest place of the row's largest value
        return torch.where(x == best[:, None], torch.arange(x.shape[1], device="cuda"), x.shape[1]).amin(1)

    parts = list(choice.split(s["E"] // s["groups"], 1))
    of_group = []
    for part in parts:
        best = part.amax(1)
        if s["group_rule"] == "top2" and part.shape[1] > 1:
            rest = part.scatter(1, first(part, best)[:, None], -math.inf).amax(1)
            best = torch.where(rest > -math.inf, best + rest, best)
        of_group.append(best)
    of_group = torch.stack(of_group, 1)
    open_ = torch.zeros_like(of_group, dtype=torch.bool)
    for _ in range(s["top_groups"]):
        at = first(of_group, of_group.amax(1))[:, None]
        open_.scatter_(1, at, True)
        of_group = of_group.masked_fill(open_, -math.inf)
    choice = choice.masked_fill(~open_.gather(1, expert // (s["E"] // s["groups"])), -math.inf)
    picks = []
    for _ in range(s["k"]):
        best = choice.amax(1)
        at = first(choice, best)
        picks.append(torch.where(best > -math.inf, at, -1))
        choice = choice.scatter(1, at[:, None], -math.inf)
    idx = torch.stack(picks, 1)
    load = s["load"]
    if load is not None:
        load = load + (idx.reshape(-1, 1) == torch.arange(s["E"], device="cuda")).sum(0).int()
    return {"idx": idx.int(), "gate": _exact_gates(s, logits, picks), "load": load}


def _exact_route_bwd(s):
    logits = s["logits"].double().requires_grad_()
    gates = _exact_gates(s, logits, list(s["idx"].long().unbind(1)))
    # the gates' derivative by differentiating their definition; rows without a pick have none
    grad, = torch.autograd.grad((gates * s["dgate"].double()).sum(), logits)
    return torch.where((s["idx"] >= 0).any(1, keepdim=True), grad, 0)


def _exact_bias(s):
    load = s["load"].double()
    step = s["rate"] * ((load < load.mean(1, keepdim=True)).double() - (load > load.mean(1, keepdim=True)).double())
    return {"bias": s["bias"].double() + step, "load": torch.zeros_like(s["load"]) if s["clear"] else s["load"]}


def _exact_adamw(s):
    h = _ADAMW
    out = {name: x.double() if x.dtype != torch.uint8 else x for name, x in s["flat"].items()}
    table = torch.tensor([f / 8 * 2.0 ** -6 for f in range(8)] +
                         [(1 + f / 8) * 2.0 ** (e - 7) for e in range(1, 16) for f in range(8)], dtype=torch.float64,
                         device="cuda")
    at = {}
    for i, t in enumerate(s["tensors"]):
        n = t["p"].numel()
        where = slice(at.get("end", 0), at.get("end", 0) + n)
        blocks = slice(where.start // 32, where.start // 32 + -(-n // 32))
        at["end"] = where.start + -(-n // 256) * 256
        g = t["grad"].double() * h["grad_scale"]
        m, r = t["m"], t["v"]
        if s["states"] == "8bit":
            m, r = ((table[(c & 127).long()] * (1 - (c >> 7).double() * 2)) *
                    torch.exp2(t[scale].double() - 127).repeat_interleave(32)[:n]
                    for c, scale in ((m, "m_scale"), (r, "v_scale")))
            v = r * r
        else:
            m, v = m.double(), r.double()
        m = m + (1 - h["beta1"]) * (g - m)
        v = v + (1 - h["beta2"]) * (g * g - v)
        hat = (m / (1 - h["beta1"] ** h["step"])) / ((v / (1 - h["beta2"] ** h["step"])).sqrt() + h["eps"])
        p = t["p"].double()
        p = p - h["lr"] * (hat + t["weight_decay"] * p)
        out["p"][where] = p
        if s["copy"]:
            out["p_bf16"][where] = p
        if s["states"] != "8bit":
            out["m"][where], out["v"][where] = m, v
            continue
        for name, x, u in (("m", m, 0), ("v", v.sqrt(), 1)):
            largest = _blocks(x.abs()).amax(1)
            exp = torch.ceil(torch.log2(largest / 448)).clamp(-127, 127)
            a = x.abs() / torch.exp2(exp).repeat_interleave(32)[:n]
            code = (torch.bucketize(a, table, right=True) - 1).clamp(0, 126)
            low, high = table[code], table[code + 1]
            u = (_noise(n, i, "cuda")[u].double() + 0.5) / 65536
            if name == "m":
                code = code + (a - low >= (1 - u) * (high - low))
            else:
                code = code + (a * a - low * low > u * (high * high - low * low))
            if name == "v":
                code = torch.where(x > 0, code.clamp(min=1), 0)
            out[name][where] = (code + 128 * (x < 0)).to(torch.uint8)
            out[name + "_scale"][blocks] = (exp + 127).to(torch.uint8)
    return {name: _values(name, x) for name, x in out.items()}
