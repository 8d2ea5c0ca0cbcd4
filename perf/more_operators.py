"""Cases for the routing of tokens to experts and the products in 8-bit integers.

Five operators of a mixture of experts, or of a dense layer, held in 8 bits:

route    router logits -> each token's experts and weights, and the order of
         rows that the experts' products take
combine  the experts' rows, weighted and added up for each token
encode   x (or silu(gate) * up) -> 8-bit integers with a scale a row, and back
         to values
product  y = X W^T of two such tensors: scales for each token and channel
experts  products grouped by expert: every run of sorted rows meets its own
         expert's weight, rows gathered from the tokens

``run`` computes them in elementary torch operations, or, where ``own`` is true,
by the calls of nvfp4_razer_w4a16_amd.  Shapes are those of the package's
workloads (Llama-3-8B-shaped layers, the [28672, 8192] weight, 8 experts of
[14336, 4096]) or generic.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
UNIT = 16  # columns of an 8-bit tensor come in this many


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one decoded token, 8 of 256 experts out of 4 of 8 groups, a bias for balance: launch latency
        {"name": "route_token", "op": "route", "tokens": 1, "experts": 256, "top": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "kept": 4, "best": 2, "renorm": True, "scale": 2.5, "padded": 0, "dtype": "f32"},
        # a batch of sequences (an odd count, some of it padding) through a plain softmax router in 16 bits, where
        # equal logits are common
        {"name": "route_batch", "op": "route", "tokens": 333, "experts": 64, "top": 6, "score": "softmax",
         "bias": False, "groups": 1, "kept": 1, "best": 1, "renorm": False, "scale": 1.0, "padded": 13,
         "dtype": "bf16"},
        # long prompts
        {"name": "route_prompt", "op": "route", "tokens": 8192, "experts": 256, "top": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "kept": 4, "best": 2, "renorm": True, "scale": 2.5, "padded": 0, "dtype": "f32"},
        # one decoded token's 8 expert rows
        {"name": "combine_token", "op": "combine", "tokens": 1, "top": 8, "cols": 4096, "add": True, "padded": 0,
         "dtype": "bf16"},
        # prompts' rows, with the residual
        {"name": "combine_prompt", "op": "combine", "tokens": 8192, "top": 8, "cols": 4096, "add": True, "padded": 0,
         "dtype": "bf16"},
        # one token's hidden state ahead of a projection: launch latency
        {"name": "encode_token", "op": "encode", "rows": 1, "cols": 4096, "gated": False, "dtype": "f16"},
        # a prompt's inner state (an odd length) ahead of the down projection
        {"name": "gated_prompt", "op": "encode", "rows": 2041, "cols": 14336, "gated": True, "dtype": "bf16"},
        # one decoded token through an up projection
        {"name": "product_token", "op": "product", "m": 1, "n": 14336, "k": 4096, "dtype": "f16"},
        # a running batch of sequences (an odd count) through a large MLP weight
        {"name": "product_batch", "op": "product", "m": 27, "n": 28672, "k": 8192, "dtype": "bf16"},
        # a long prompt through the same weight
        {"name": "product_prefill", "op": "product", "m": 2048, "n": 28672, "k": 8192, "dtype": "bf16"},
        # 8 decoded tokens, 2 of 8 experts each
        {"name": "experts_token", "op": "experts", "tokens": 8, "top": 2, "experts": 8, "n": 14336, "k": 4096,
         "routing": 1, "dtype": "bf16"},
        # a prompt through the same experts
        {"name": "experts_prefill", "op": "experts", "tokens": 4096, "top": 2, "experts": 8, "n": 14336, "k": 4096,
         "routing": 2, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "combine", "encode", "product", "experts"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    half = rng.choice(["f16", "bf16"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        each = _log(rng, 4, 256 // groups)
        kept = rng.randint(1, groups)
        tokens = _log(rng, 1, 8192)
        return {"op": op, "tokens": tokens, "experts": groups * each, "top": rng.randint(1, min(8, kept * each)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "kept": kept, "best": rng.randint(1, 2), "renorm": rng.random() < 0.5,
                "scale": rng.choice([1.0, 2.5]), "padded": rng.choice([0, tokens // 7]), "dtype": dtype}
    if op == "combine":
        top, cols = rng.randint(1, 8), _log(rng, 64, 8192)
        tokens = _log(rng, 1, min(8192, 8192 * 8 * 4096 * 2 // (SIZES[dtype] * top * cols)))
        return {"op": op, "tokens": tokens, "top": top, "cols": cols, "add": rng.random() < 0.5,
                "padded": rng.choice([0, tokens // 7]), "dtype": dtype}
    if op == "encode":
        gated = rng.random() < 0.5
        return {"op": op, "rows": _log(rng, 1, 2041), "cols": UNIT * _log(rng, 4, 14336 // UNIT), "gated": gated,
                "dtype": half if gated else dtype}
    if op == "product":
        return {"op": op, "m": _log(rng, 1, 2048), "n": _log(rng, 64, 28672), "k": UNIT * _log(rng, 8, 512),
                "dtype": dtype}
    experts = _log(rng, 2, 64)
    n, top = _log(rng, 64, min(14336, 14336 * 8 // experts)), rng.randint(1, min(4, experts))
    return {"op": op, "tokens": _log(rng, 1, 8192 // max(top, 2)), "top": top, "experts": experts, "n": n,
            "k": UNIT * _log(rng, 8, 256), "routing": rng.randrange(1000), "dtype": dtype}


def _chosen(case):
    """Experts of each token: `top` different ones, some being likelier than others."""
    r = random.Random(1000 * case["routing"] + case["experts"])
    e = case["experts"]
    liking = [math.exp(r.gauss(0.0, 0.7)) for _ in range(e)]
    chosen = []
    for _ in range(case["tokens"]):
        score = [(-math.log(1.0 - r.random()) / liking[i], i) for i in range(e)]
        chosen.append([i for _, i in sorted(score)[:case["top"]]])
    return chosen


def _group_sizes(case):
    sizes = [0] * case["experts"]
    for token in _chosen(case):
        for e in token:
            sizes[e] += 1
    return sizes


# ---- inputs ------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, rows, cols):
    """N(0, 1) with a few outlier channels, as hidden states of a transformer have."""
    x = _normal(gen, rows, cols)
    at = torch.randint(0, cols, (8,), generator=gen, device="cuda")
    x[:, at] *= 20.0
    return x


def _weight(gen, rows, cols):
    """Weights of scale 0.02, some channels larger than others."""
    return _normal(gen, rows, cols).mul_(0.02).mul_(torch.exp(0.5 * _normal(gen, rows, 1)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": dict(case), "dtype": dt}
    if op == "route":
        t, e = case["tokens"], case["experts"]
        # some experts are likelier than others, for every token
        logits = 1.5 * _normal(gen, t, e) + 0.7 * _normal(gen, 1, e)
        if case["padded"]:
            logits[t - case["padded"]:] = -math.inf
        s["logits"] = logits.to(dt)
        s["bias"] = 0.1 * _normal(gen, e) if case["bias"] else None
    elif op == "combine":
        t, top, cols = case["tokens"], case["top"], case["cols"]
        # each token's experts of 64: where the rows of a token lie among the sorted ones
        experts = torch.argsort(_normal(gen, t, 64), 1)[:, :top]
        weights = torch.exp(_normal(gen, t, top))
        s["weights"] = weights / weights.sum(1, keepdim=True)
        if case["padded"]:
            experts[t - case["padded"]:] = -1
            s["weights"][t - case["padded"]:] = 0.0
        s["slots"] = _order(experts, 64)[2]
        s["y"] = _activations(gen, t * top, cols).to(dt)
        s["add"] = (3.0 * _activations(gen, t, cols)).to(dt) if case["add"] else None
    elif op == "encode":
        if case["gated"]:
            s["x"] = _normal(gen, case["rows"], 2 * case["cols"]).mul_(1.5).to(dt)
        else:
            s["x"] = _activations(gen, case["rows"], case["cols"]).to(dt)
    elif op == "product":
        s["x"] = _codes(_activations(gen, case["m"], case["k"]))
        s["w"] = _codes(_weight(gen, case["n"], case["k"]))
    else:
        chosen = torch.tensor(_chosen(case)).cuda()
        s["x"] = _codes(_activations(gen, case["tokens"], case["k"]))
        s["w"] = _codes(_weight(gen, case["experts"] * case["n"], case["k"]))
        s["offsets"], s["x_rows"], _ = _order(chosen, case["experts"])
        s["capacity"] = max(_group_sizes(case))  # the dispatcher's bound on the rows of one expert
    return s


# ---- elementary operations ---------------------------------------------------

def _order(experts, count):
    """(offsets, rows, slots) of the experts [T, k] of each token, -1 for none: the pairs (token, choice) sorted by
    expert, then token."""
    t, top = experts.shape
    flat = torch.where(experts >= 0, experts, count).reshape(-1)
    order = torch.argsort(flat, stable=True)
    offsets = torch.searchsorted(flat[order].contiguous(), torch.arange(count + 1, device=flat.device))
    at = torch.arange(t * top, device=flat.device)
    rows = torch.where(at < offsets[count], order // top, -1)
    slots = torch.empty_like(at)
    slots[order] = at
    slots = torch.where(experts >= 0, slots.view(t, top), -1)
    return offsets.to(torch.int32), rows.to(torch.int32), slots.to(torch.int32)


def _codes(x):
    """{codes, scales} of fp32 x [rows, cols]: codes are whole numbers from -127 to 127."""
    amax = x.abs().amax(-1, keepdim=True)
    full = torch.full_like(amax, 127.0)
    inverse = torch.where(amax > 0, full / amax, 0.0)
    return {"codes": torch.round(x * inverse).to(torch.int8), "scales": (amax / full).reshape(-1)}


def _values(t):
    return t["codes"].float() * t["scales"].unsqueeze(1)


def _best(key, count):
    """The `count` largest entries of each row and where they are, the lowest index first among equals."""
    value, at = torch.sort(key, dim=-1, descending=True, stable=True)
    return value[..., :count], at[..., :count]


def _route(s):
    c = s["case"]
    t, e = s["logits"].shape
    # in 64 bits: scores that are all but equal decide which expert is chosen
    logits = s["logits"].double()
    live = logits > -math.inf
    if c["score"] == "softmax":
        top = logits.amax(-1, keepdim=True)
        p = torch.where(live, torch.exp(logits - torch.where(top > -math.inf, top, 0.0)), 0.0)
        p = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
    else:
        p = 1.0 / (1.0 + torch.exp(-logits))
    key = p if s["bias"] is None else p + s["bias"].double()
    key = torch.where(live, key, -math.inf)
    if c["groups"] > 1:
        value, _ = _best(key.view(t, c["groups"], -1), c["best"])
        group = torch.where(value > -math.inf, value, 0.0).sum(-1)
        group = torch.where(value[..., 0] > -math.inf, group, -math.inf)
        _, at = _best(group, c["kept"])
        kept = torch.zeros_like(group, dtype=torch.bool).scatter_(1, at, True)
        key = torch.where(kept.repeat_interleave(e // c["groups"], 1), key, -math.inf)
    value, at = _best(key, c["top"])
    ok = value > -math.inf
    w = torch.where(ok, p.gather(1, at), 0.0)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
    experts = torch.where(ok, at, -1)
    offsets, rows, slots = _order(experts, e)
    return {"experts": experts.to(torch.int32), "weights": (w * c["scale"]).float(), "offsets": offsets, "rows": rows,
            "slots": slots}


def _plain(s):
    op, dt = s["case"]["op"], s["dtype"]
    if op == "route":
        return _route(s)
    if op == "combine":
        slots = s["slots"].long()
        w = torch.where(slots >= 0, s["weights"], 0.0)
        out = (s["y"][slots.clamp_min(0)].float() * w.unsqueeze(-1)).sum(1)
        return (out if s["add"] is None else out + s["add"].float()).to(dt)
    if op == "encode":
        x = s["x"].float()
        if s["case"]["gated"]:
            g, u = x[:, :s["case"]["cols"]], x[:, s["case"]["cols"]:]
            x = g / (1.0 + torch.exp(-g)) * u
        return _values(_codes(x)).to(dt)
    if op == "product":
        y = s["x"]["codes"].float() @ s["w"]["codes"].float().t()
        return (y * s["x"]["scales"].unsqueeze(1) * s["w"]["scales"]).to(dt)
    # every expert's rows padded to the capacity, one product per expert
    e, off, cap = s["case"]["experts"], s["offsets"].long(), s["capacity"]
    x = _values(s["x"])[s["x_rows"].long()]
    slot = torch.arange(cap, device=x.device)
    live = slot < (off[1:] - off[:-1]).unsqueeze(1)
    at = (off[:-1].unsqueeze(1) + slot).clamp_max(x.shape[0] - 1)
    w = _values(s["w"]).view(e, s["case"]["n"], -1)
    return torch.bmm(x[at], w.transpose(1, 2).contiguous())[live].to(dt)


# ---- one pass ----------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return _plain(s)
    import nvfp4_razer_w4a16_amd as rz

    c, op, dt = s["case"], s["case"]["op"], s["dtype"]
    if op == "route":
        r = rz.razer_moe_route(s["logits"], c["top"], score=c["score"], bias=s["bias"], groups=c["groups"],
                               groups_kept=c["kept"], group_best=c["best"], renormalise=c["renorm"], scale=c["scale"])
        return {"experts": r.experts, "weights": r.weights, "offsets": r.offsets, "rows": r.rows, "slots": r.slots}
    if op == "combine":
        return rz.razer_moe_combine(s["y"], s["slots"], s["weights"], add=s["add"])
    if op == "encode":
        t = rz.razer_i8_quantize_gated(s["x"]) if c["gated"] else rz.razer_i8_quantize(s["x"])
        return rz.razer_i8_dequant(t, dt)
    x, w = rz.I8Tensor.of(**s["x"]), rz.I8Tensor.of(**s["w"])
    if op == "product":
        return rz.razer_i8_gemm(x, w, dt)
    return rz.razer_i8_gemm_grouped(x, w, s["offsets"], s["x_rows"], dt)


def work(case):
    op, size = case["op"], SIZES[case["dtype"]]
    if op == "route":
        # logits in; experts, weights, rows and slots out, and the offsets; a score and a comparison a choice
        t, e, top = case["tokens"], case["experts"], case["top"]
        return {"bytes": t * e * size + 16 * t * top + 4 * (e + 1) + (4 * e if case["bias"] else 0),
                "flops": t * e * (8 + top)}
    if op == "combine":
        t, top, cols = case["tokens"], case["top"], case["cols"]
        rows = (t - case["padded"]) * top
        return {"bytes": (rows + t * (2 if case["add"] else 1)) * cols * size + 8 * t * top, "flops": 2 * rows * cols}
    if op == "encode":
        # values in, the 8-bit tensor, values out
        n = case["rows"] * case["cols"]
        return {"bytes": n * size * (3 if case["gated"] else 2) + n + 4 * case["rows"],
                "flops": n * (14 if case["gated"] else 4)}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * (k + 4) + m * n * size, "flops": 2 * m * n * k}
    sizes, n, k = _group_sizes(case), case["n"], case["k"]
    total, used = sum(sizes), sum(c > 0 for c in sizes)
    return {"bytes": ((case["tokens"] + used * n) * (k + 4) + total * n * size + 4 * (total + len(sizes) + 1)),
            "flops": 2 * total * n * k}


# ---- the definition in 64 bits -----------------------------------------------

def _exact_weights(s):
    """Weights of the chosen experts, the best first: an expert's rank is the number of those that go before it."""
    c, logits = s["case"], s["logits"].double()
    t, e = logits.shape
    padded = torch.isinf(logits[:, 0])
    logits = torch.where(padded.unsqueeze(1), 0.0, logits)
    p = torch.softmax(logits, -1) if c["score"] == "softmax" else torch.sigmoid(logits)
    key = p if s["bias"] is None else p + s["bias"].double()

    def rank(k):
        low = torch.arange(k.shape[1], device=k.device)
        before = (k.unsqueeze(1) > k.unsqueeze(2)) | ((k.unsqueeze(1) == k.unsqueeze(2)) & (low < low.unsqueeze(1)))
        return before.sum(-1)

    out = []
    for a in range(0, t, 512):
        k, q = key[a:a + 512], p[a:a + 512]
        if c["groups"] > 1:
            parts = k.reshape(k.shape[0], c["groups"], -1)
            place = torch.stack([rank(parts[:, i]) for i in range(c["groups"])], 1)
            group = torch.where(place < c["best"], parts, 0.0).sum(-1)
            k = torch.where((rank(group) < c["kept"]).unsqueeze(-1), parts, -math.inf).reshape(k.shape)
        place = rank(k)
        w = torch.zeros(k.shape[0], e, dtype=torch.float64, device=k.device).scatter_(1, place, q)[:, :c["top"]]
        out.append(w / w.sum(-1, keepdim=True) if c["renorm"] else w)
    w = torch.cat(out) * c["scale"]
    return torch.where(padded.unsqueeze(1), 0.0, w)


def _exact_values(t):
    return t["codes"].double() * t["scales"].double().reshape(-1, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return {"experts": None, "weights": _exact_weights(s), "offsets": None, "rows": None, "slots": None}
    if op == "combine":
        total = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        live = case["tokens"] - case["padded"]
        for j in range(case["top"]):
            total[:live] += s["weights"][:live, j:j + 1].double() * s["y"][s["slots"][:live, j].long()].double()
        return total if s["add"] is None else total + s["add"].double()
    if op == "encode":
        x = s["x"].double()
        if case["gated"]:
            x = x[:, :case["cols"]] * torch.sigmoid(x[:, :case["cols"]]) * x[:, case["cols"]:]
        step = x.abs().amax(-1, keepdim=True) / 127
        return torch.round(x / step) * step
    if op == "product":
        y = torch.mm(s["x"]["codes"].double(), s["w"]["codes"].double().t())
        return y * s["x"]["scales"].double().reshape(-1, 1) * s["w"]["scales"].double()
    x, w = _exact_values(s["x"]), _exact_values(s["w"])
    off, n, rows = s["offsets"].tolist(), case["n"], s["x_rows"].long()
    return torch.cat([torch.mm(x[rows[a:b]], w[i * n:(i + 1) * n].t())
                      for i, (a, b) in enumerate(zip(off[:-1], off[1:]))])
