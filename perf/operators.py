"""Cases for the microscaled 4-bit (MXFP4) operators and the block norm.

Five operators of a transformer block whose linear layers are held in 4 bits:

encode   x -> MXFP4 (32-element blocks, power-of-two block scales) and back to
         values: what a checkpoint converter or a calibration run does
product  y = X W^T of two MXFP4 tensors
gated    silu(gate) * up packed to MXFP4, then the down projection
experts  products grouped by expert: every run of sorted rows meets its own
         expert's weight, rows gathered from the packed tokens
norm     h' = h + s * gate * rmsnorm(y; post), x = rmsnorm(h'; pre); x comes
         out as values, or packed and multiplied by a projection weight

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, by the calls of nvfp4_razer_w4a16_amd.  Shapes are those of
the package's workloads (Llama-3-8B-shaped layers, [28672, 8192] and
[4096, 4096] weights) or generic.
"""
import math
import random

import torch

own = False

BLOCK = 32
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one token's hidden state, packed ahead of a projection: launch latency
        {"name": "encode_token", "op": "encode", "rows": 1, "cols": 4096, "dtype": "f16"},
        # converting an up projection of a checkpoint
        {"name": "encode_weight", "op": "encode", "rows": 14336, "cols": 4096, "dtype": "f32"},
        # one decoded token through an up projection
        {"name": "product_token", "op": "product", "m": 1, "n": 14336, "k": 4096, "dtype": "f16"},
        # a running batch of sequences (an odd count) through a large MLP weight
        {"name": "product_batch", "op": "product", "m": 27, "n": 28672, "k": 8192, "dtype": "bf16"},
        # a long prompt through the same weight
        {"name": "product_prefill", "op": "product", "m": 2048, "n": 28672, "k": 8192, "dtype": "bf16"},
        # the second half of an MLP for one token
        {"name": "gated_token", "op": "gated", "m": 1, "n": 4096, "k": 14336, "dtype": "f16"},
        # and for a prompt of an odd length
        {"name": "gated_prefill", "op": "gated", "m": 2041, "n": 4096, "k": 14336, "dtype": "bf16"},
        # 8 decoded tokens, 2 of 8 experts each (three experts get none)
        {"name": "experts_token", "op": "experts", "tokens": 8, "top": 2, "experts": 8, "n": 14336, "k": 4096,
         "routing": 1, "dtype": "bf16"},
        # a prompt through the same experts
        {"name": "experts_prefill", "op": "experts", "tokens": 4096, "top": 2, "experts": 8, "n": 14336, "k": 4096,
         "routing": 2, "dtype": "bf16"},
        # many small experts with ragged runs of rows; an odd output width
        {"name": "experts_ragged", "op": "experts", "tokens": 333, "top": 3, "experts": 64, "n": 1503, "k": 2080,
         "routing": 3, "dtype": "f32"},
        # between two layers of one decoded token: the norms, then the packed state through a qkv projection
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "gates": 0, "n": 6144, "dtype": "f16"},
        # between two layers of a prompt, one gate row per sequence
        {"name": "norm_prefill", "op": "norm", "rows": 4096, "cols": 8192, "gates": 4, "n": 0, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["encode", "product", "gated", "experts", "norm"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "encode":
        return {"op": op, "rows": _log(rng, 1, 14336), "cols": BLOCK * _log(rng, 1, 256), "dtype": dtype}
    if op == "product":
        return {"op": op, "m": _log(rng, 1, 2048), "n": _log(rng, 64, 28672), "k": BLOCK * _log(rng, 4, 256),
                "dtype": dtype}
    half = rng.choice(["f16", "bf16"])  # a product of states that were packed on the way comes out in 16 bits
    if op == "gated":
        return {"op": op, "m": _log(rng, 1, 2048), "n": _log(rng, 64, 8192), "k": BLOCK * _log(rng, 4, 448),
                "dtype": half}
    if op == "experts":
        experts = _log(rng, 2, 64)
        n, top = _log(rng, 64, min(14336, 14336 * 8 // experts)), rng.randint(1, min(4, experts))
        return {"op": op, "tokens": _log(rng, 1, 8192 // max(top, 2)), "top": top, "experts": experts,
                "n": n, "k": BLOCK * _log(rng, 4, 128), "routing": rng.randrange(1000), "dtype": dtype}
    rows, packed = _log(rng, 1, 4096), rng.random() < 0.5
    gates = rng.choice([0, 1, rows] + [d for d in (2, 4, 8) if rows % d == 0])
    return {"op": op, "rows": rows, "cols": BLOCK * _log(rng, 4, 256), "gates": gates,
            "n": _log(rng, 64, 8192) if packed else 0, "dtype": half if packed else dtype}


def _group_sizes(case):
    """Rows of each expert: each token takes `top` different experts, some experts being likelier than others."""
    r = random.Random(1000 * case["routing"] + case["experts"])
    e = case["experts"]
    liking = [math.exp(r.gauss(0.0, 0.7)) for _ in range(e)]
    sizes = [0] * e
    for _ in range(case["tokens"]):
        score = [(-math.log(1.0 - r.random()) / liking[i], i) for i in range(e)]
        for _, i in sorted(score)[:case["top"]]:
            sizes[i] += 1
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
    """Student-t-like weights of scale 0.02: a normal over the root of a mean of squares, one root per block."""
    w = _normal(gen, rows, cols).mul_(0.02)
    s = _normal(gen, rows, cols // BLOCK, 5).square_().mean(-1).sqrt_().clamp_min_(0.2)
    return (w.view(rows, cols // BLOCK, BLOCK) / s.unsqueeze(-1)).view(rows, cols)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": dict(case), "dtype": dt}
    if op == "encode":
        s["x"] = _activations(gen, case["rows"], case["cols"]).to(dt)
    elif op == "product":
        s["x"] = _pack(_activations(gen, case["m"], case["k"]))
        s["w"] = _pack(_weight(gen, case["n"], case["k"]))
    elif op == "gated":
        s["gu"] = _normal(gen, case["m"], 2 * case["k"]).mul_(1.5).to(dt)
        s["w"] = _pack(_weight(gen, case["n"], case["k"]))
    elif op == "experts":
        sizes, e = _group_sizes(case), case["experts"]
        total = sum(sizes)
        s["x"] = _pack(_activations(gen, case["tokens"], case["k"]))
        s["w"] = _pack(_weight(gen, e * case["n"], case["k"]))
        offsets = [0]
        for c in sizes:
            offsets.append(offsets[-1] + c)
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32).cuda()
        s["capacity"] = max(sizes)  # the dispatcher's bound on the rows of one expert
        # the token of every sorted row, as a router's sort leaves them
        s["x_rows"] = torch.randint(0, case["tokens"], (total,), generator=gen, device="cuda").to(torch.int32)
    else:
        rows, cols, gates = case["rows"], case["cols"], case["gates"]
        s["y"] = _activations(gen, rows, cols).to(dt)
        s["h"] = (_activations(gen, rows, cols) * 3.0).to(dt)
        s["post"] = (1.0 + 0.1 * _normal(gen, cols)).to(dt)
        s["pre"] = (1.0 + 0.1 * _normal(gen, cols)).to(dt)
        s["gate"] = (0.5 * _normal(gen, gates, cols)).to(dt) if gates else None
        if case["n"]:
            s["w"] = _pack(_weight(gen, case["n"], cols))
    return s


# ---- the format in elementary operations -------------------------------------

def _pow2(e):
    """2^(e - 127) of scale bytes, exactly."""
    e = e.to(torch.int32)
    return torch.where(e > 0, e << 23, 0x00400000).view(torch.float32)


def _codes(x):
    """(codes, scale bytes) of fp32 x [rows, cols], one code a byte."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // BLOCK, BLOCK)
    top = b.abs().amax(-1).contiguous().view(torch.int32) >> 23  # floor(log2) + 127
    scale = (top - 2).clamp_min(0)
    v = b / _pow2(scale).unsqueeze(-1)
    a = v.abs()
    # halfway cases go to the even code
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    c = c + torch.where(v < 0, 8, 0)
    return c.to(torch.uint8).reshape(rows, cols), scale.to(torch.uint8)


def _pack(x):
    """{codes, scales} as the library holds them: two codes a byte, the even column in the low half."""
    c, scales = _codes(x)
    return {"codes": c[:, 0::2] | (c[:, 1::2] << 4), "scales": scales}


def _values(codes, scales):
    rows, cols = codes.shape
    mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    v = torch.cat([mag, -mag])[codes.to(torch.int32)]
    return (v.view(rows, cols // BLOCK, BLOCK) * _pow2(scales).unsqueeze(-1)).view(rows, cols)


def _unpack(t):
    c = t["codes"]
    return _values(torch.stack([c & 15, c >> 4], -1).view(c.shape[0], -1), t["scales"])


def _rmsnorm(v, w):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS) * w.float()


def _plain(s):
    op, dt = s["case"]["op"], s["dtype"]
    if op == "encode":
        return _values(*_codes(s["x"].float())).to(dt)
    if op == "product":
        return (_unpack(s["x"]) @ _unpack(s["w"]).t()).to(dt)
    if op == "gated":
        k = s["case"]["k"]
        g, u = s["gu"][:, :k].float(), s["gu"][:, k:].float()
        p = g / (1.0 + torch.exp(-g)) * u
        return (_values(*_codes(p)) @ _unpack(s["w"]).t()).to(dt)
    if op == "experts":
        # every expert's rows padded to the capacity, one product per expert
        e, off, cap = s["case"]["experts"], s["offsets"].long(), s["capacity"]
        x = _unpack(s["x"])[s["x_rows"].long()]
        slot = torch.arange(cap, device=x.device)
        live = slot < (off[1:] - off[:-1]).unsqueeze(1)
        at = (off[:-1].unsqueeze(1) + slot).clamp_max(x.shape[0] - 1)
        w = _unpack(s["w"]).view(e, s["case"]["n"], -1)
        return torch.bmm(x[at], w.transpose(1, 2).contiguous())[live].to(dt)
    post = _rmsnorm(s["y"].float(), s["post"])
    if s["gate"] is not None:
        post = post * s["gate"].float().repeat_interleave(post.shape[0] // s["gate"].shape[0], 0)
    h = s["h"].float() + 0.5 * post
    x = _rmsnorm(h, s["pre"])
    if s["case"]["n"]:
        x = _values(*_codes(x)) @ _unpack(s["w"]).t()
    return h.to(dt), x.to(dt)


# ---- one pass ----------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return _plain(s)
    import nvfp4_razer_w4a16_amd as rz

    op, dt = s["case"]["op"], s["dtype"]
    if op == "encode":
        return rz.razer_mx_dequant(rz.razer_mx_quantize(s["x"]), dt)
    w = rz.MxTensor.of(**s["w"]) if "w" in s else None
    if op == "product":
        return rz.razer_mx_gemm(rz.MxTensor.of(**s["x"]), w, dt)
    if op == "gated":
        return rz.razer_mx_gemm(rz.razer_mx_quantize_gated(s["gu"]), w, dt)
    if op == "experts":
        return rz.razer_mx_gemm_grouped(rz.MxTensor.of(**s["x"]), w, s["offsets"], s["x_rows"], dt)
    h, x = rz.razer_block_norm(s["y"], s["h"], post_weight=s["post"], gate=s["gate"], residual_scale=0.5,
                               pre_weight=s["pre"], eps=EPS, packed=w is not None)
    return h, (x if w is None else rz.razer_mx_gemm(x, w, dt))


def _packed_bytes(rows, cols):
    return rows * cols // 2 + rows * cols // BLOCK


def work(case):
    op, size = case["op"], SIZES[case["dtype"]]
    if op == "encode":
        # values in, the packed tensor, values out; a compare, a scale and a rounding each way
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * size + _packed_bytes(case["rows"], case["cols"]), "flops": 4 * n}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _packed_bytes(m, k) + _packed_bytes(n, k) + m * n * size, "flops": 2 * m * n * k}
    if op == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * k * size + _packed_bytes(n, k) + m * n * size, "flops": 2 * m * n * k + 8 * m * k}
    if op == "experts":
        sizes, n, k = _group_sizes(case), case["n"], case["k"]
        total, used = sum(sizes), sum(c > 0 for c in sizes)
        return {"bytes": (_packed_bytes(min(total, case["tokens"]), k) + _packed_bytes(used * n, k)
                          + total * n * size + 4 * (total + len(sizes) + 1)),
                "flops": 2 * total * n * k}
    rows, cols, n = case["rows"], case["cols"], case["n"]
    b = 3 * rows * cols * size + (2 + case["gates"]) * cols * size
    b += _packed_bytes(n, cols) + rows * n * size if n else rows * cols * size
    return {"bytes": b, "flops": 12 * rows * cols + 2 * rows * n * cols}


# ---- the definition in 64 bits -----------------------------------------------

def _exact_round(x):
    """MXFP4 values of x in float64: the block's largest magnitude sets the power of two, each quotient is rounded
    to the grid of its binade, halves to even."""
    x = x.double()
    b = x.reshape(x.shape[0], -1, BLOCK)
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))  # amax = f * 2^e, f in [0.5, 1)
    unit = torch.exp2((e - 3).clamp_min(-127).double())
    v = b / unit
    step = torch.where(v.abs() >= 4, 2.0, torch.where(v.abs() >= 2, 1.0, 0.5)).double()
    return (torch.clamp(torch.round(v / step) * step, -6, 6) * unit).reshape(x.shape)


def _exact_values(t):
    codes, scales = t["codes"].to(torch.int64), t["scales"].double()
    c = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes % 16, codes // 16
    # two bits of exponent, one of fraction, bias 1
    exp, frac = (c % 8) // 2, (c % 2).double()
    mag = torch.where(exp > 0, (2 + frac) * torch.exp2((exp - 2).double()), frac / 2)
    v = torch.where(c >= 8, -mag, mag)
    return (v.reshape(v.shape[0], -1, BLOCK) * torch.exp2(scales - 127).unsqueeze(-1)).reshape(v.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "encode":
        return _exact_round(s["x"])
    w = _exact_values(s["w"]) if "w" in s else None
    if op == "product":
        return torch.mm(_exact_values(s["x"]), w.t())
    if op == "gated":
        gu = s["gu"].double()
        g, u = gu[:, :case["k"]], gu[:, case["k"]:]
        return torch.mm(_exact_round(g * torch.sigmoid(g) * u), w.t())
    if op == "experts":
        x = _exact_values(s["x"])
        off, n = s["offsets"].tolist(), case["n"]
        rows = s["x_rows"].long()
        return torch.cat([torch.mm(x[rows[a:b]], w[i * n:(i + 1) * n].t())
                          for i, (a, b) in enumerate(zip(off[:-1], off[1:]))])
    y, h = s["y"].double(), s["h"].double()
    y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * s["post"].double()
    if s["gate"] is not None:
        per = y.shape[0] // s["gate"].shape[0]
        y = (y.reshape(-1, per, y.shape[1]) * s["gate"].double().unsqueeze(1)).reshape(y.shape)
    h = h + y / 2
    x = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["pre"].double()
    return h, (x if w is None else torch.mm(_exact_round(x), w.t()))
