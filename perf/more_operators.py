"""More operators of a transformer block, as cases that can be measured.

Three operators between and inside a block's linears:

* ``quant``: a tensor quantized to microscaled 4-bit floating point and read back (``ck_mx4_act_quant`` or
  ``ck_mx4_weight_prep``, then ``ck_mx4_dequant``): E2M1 values with one power-of-two scale for 32 of them;
* ``linear``: the linear on such weights (``ck_mx4_linear``): optional SwiGLU, Hadamard rotation and quantization of
  the activation, the 4-bit product, bias and residual;
* ``norm``: what joins two sub-blocks (``ck_block_norm``): the branch's own norm, its gate and scale, the residual
  sum, and the next sub-block's norm with its modulation.

``run`` computes each in its plain form (elementary torch operations in 32 bits) or, with ``own`` set, through the
library.
"""
import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # E2M1 magnitudes, by code


def _quant(name, m, k, dtype):
    return {"name": name, "op": "quant", "m": m, "k": k, "dtype": dtype}


def _linear(name, m, k, n, act, group, bias, residual):
    return {"name": name, "op": "linear", "m": m, "k": k, "n": n, "act": act, "group": group, "bias": bias,
            "residual": residual}


def _norm(name, b, t, w, dtype, kind, branch, gate, mod, residual_scale, branch_scale):
    """branch: the branch's norm ("none" for no norm); gate, mod: what the gate and the modulation are given for
    ("no", "channel", "sequence" or "token")."""
    return {"name": name, "op": "norm", "b": b, "t": t, "w": w, "dtype": dtype, "kind": kind, "branch": branch,
            "gate": gate, "mod": mod, "residual_scale": residual_scale, "branch_scale": branch_scale}


def listed():
    return [
        # the activations of 16 tokens being decoded: latency alone
        _quant("quant tokens", 16, 4096, "bf16"),
        # a checkpoint's FP32 weight, quantized at load
        _quant("quant weight", 12288, 4096, "fp32"),
        # one new token through an up projection: the weight stream
        _linear("linear one token", 1, 4096, 12288, "none", 128, False, False),
        # 16 tokens through the down projection of a SwiGLU MLP (c3's K and N), with the block's residual
        _linear("linear 16 tokens", 16, 12288, 4096, "swiglu", 128, False, True),
        # odd row and column counts, a K that is no multiple of 256, bias and residual
        _linear("linear odd", 333, 2112, 1040, "none", 64, True, True),
        # a prompt of 1024 tokens through an attention projection (c4's K and N)
        _linear("linear prompt", 1024, 4096, 4096, "none", 128, True, False),
        # the packed gate and up projection over an image latent
        _linear("linear gate and up", 4096, 4096, 24576, "none", 128, False, False),
        # the SwiGLU down projection over four long sequences (c3's K and N)
        _linear("linear down, long", 16384, 12288, 4096, "swiglu", 128, False, True),
        # one new token of 16 sequences in a decoder layer: residual sum and the next norm
        _norm("norm one token", 16, 1, 4096, "bf16", "rms", "none", "no", "no", 1.0, 1.0),
        # an image block with per-sequence gate, scale and shift around plain layer norms
        _norm("norm image block", 2, 4096, 4096, "bf16", "layer", "none", "sequence", "sequence", 1.0, 1.0),
        # odd token and channel counts, a norm on both sides, scaled branch
        _norm("norm odd", 3, 777, 1160, "fp16", "layer", "rms", "channel", "token", 1.5, 0.22),
        # the prefill of four long sequences, RMS norms before and after each sub-block
        _norm("norm long", 4, 16384, 4096, "bf16", "rms", "rms", "no", "no", 1.0, 1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Another case of the same ranges, no dearer than the largest listed one of its operator."""
    most = {op: [work(c) for c in listed() if c["op"] == op] for op in ("quant", "linear", "norm")}
    while True:
        op = rng.choice(["quant", "linear", "linear", "linear", "norm", "norm"])
        if op == "quant":
            case = _quant("", _log(rng, 1, 16384), 64 * _log(rng, 1, 192), rng.choice(["bf16", "bf16", "fp32"]))
        elif op == "linear":
            k = 64 * _log(rng, 2, 192)
            group = rng.choice([g for g in (1, 32, 64, 64, 128, 128, 128, 256) if k % g == 0])
            case = _linear("", 1 if rng.random() < 0.2 else _log(rng, 2, 16384), k, 16 * _log(rng, 4, 1536),
                           rng.choice(["none", "none", "swiglu"]), group, rng.random() < 0.3, rng.random() < 0.4)
        else:
            case = _norm("", rng.randint(1, 8), 1 if rng.random() < 0.2 else _log(rng, 2, 16384),
                         8 * _log(rng, 8, 1024), rng.choice(["bf16", "bf16", "fp16"]), rng.choice(["rms", "layer"]),
                         rng.choice(["none", "none", "rms", "layer"]),
                         rng.choice(["no", "channel", "sequence", "token"]),
                         rng.choice(["no", "sequence", "token"]), rng.choice([1.0, 1.0, 2.5]),
                         rng.choice([1.0, 1.0, 0.22]))
        w = work(case)
        if all(w[x] <= max(o[x] for o in most[op]) for x in ("bytes", "flops")):
            del case["name"]
            return case


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _activations(g, rows, width):
    """Near-normal values with one channel in a hundred twenty times larger."""
    x = torch.randn(rows, width, generator=g, device=DEV)
    return x.mul_(torch.where(torch.rand(width, generator=g, device=DEV) < 0.01, 20.0, 1.0))


def _power_of_two(e):
    """2^e for whole e in [-126, 127], in 32 bits."""
    return ((e + 127) << 23).view(torch.float32)


def _microscale(v):
    """E2M1 values [rows, k / 32, 32] (to the nearest, ties to the even code) and exponents [rows, k / 32, 1] of v."""
    u = v.view(v.shape[0], -1, 32)
    e = torch.frexp(u.abs().amax(-1, keepdim=True))[1].int() - 3      # floor(log2(largest)) - 2
    e = e.clamp_(-126, 126)
    u = u * _power_of_two(-e)
    a = u.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(u / step).mul_(step).clamp_(-6, 6), e


def _codes(q, e):
    """Row-major codes, two in a byte (the even k low), and biased exponents."""
    a = q.abs().view(q.shape[0], -1)
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, 2 + a, 4 + a / 2)).to(torch.uint8)
    code |= (q.view(q.shape[0], -1) < 0).to(torch.uint8) << 3
    return code[:, 0::2] | (code[:, 1::2] << 4), (e[..., 0] + 127).to(torch.uint8)


def _values(codes, scales):
    """The values that codes and exponents stand for, in 32 bits."""
    levels = torch.tensor(LEVELS, device=DEV)
    levels = torch.cat([levels, -levels])
    code = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1)
    v = levels[code.int()].view(codes.shape[0], -1, 32)
    return (v * _power_of_two(scales.int() - 127).unsqueeze(-1)).view(codes.shape[0], -1)


def prepare(case, seed):
    g, s = _gen(seed), {"case": case}
    if case["op"] == "quant":
        if case["dtype"] == "fp32":
            s["x"] = torch.randn(case["m"], case["k"], generator=g, device=DEV).mul_(0.02)
        else:
            s["x"] = _activations(g, case["m"], case["k"]).to(TYPES[case["dtype"]])
        return s
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        s["x"] = _activations(g, m, 2 * k if case["act"] == "swiglu" else k).to(torch.bfloat16)
        # weights as a checkpoint holds them: row-major codes and scales
        s["codes"], s["scales"] = _codes(*_microscale(torch.randn(n, k, generator=g, device=DEV).mul_(0.02)))
        s["bias"] = 0.1 * torch.randn(n, generator=g, device=DEV) if case["bias"] else None
        s["residual"] = torch.randn(m, n, generator=g, device=DEV).to(torch.bfloat16) if case["residual"] else None
        if own:   # laid out once, at load
            import swiglu_mlp_amd as ck
            s["weight"] = ck.ck_mx4_weight_pack(s["codes"], s["scales"])
        return s
    b, t, w, dt = case["b"], case["t"], case["w"], TYPES[case["dtype"]]

    def modulation(given, size):
        shape = {"no": None, "channel": (w,), "sequence": (b, w), "token": (b, t, w)}[given]
        return None if shape is None else (size * torch.randn(shape, generator=g, device=DEV)).to(dt)

    # a residual stream with a mean and a few large channels, and a branch's output
    s["x"] = (_activations(g, b * t, w) + 0.3).view(b, t, w).to(dt)
    s["branch"] = torch.randn(b, t, w, generator=g, device=DEV).to(dt)
    s["gate"], s["scale"], s["shift"] = (modulation(case[c], 0.5) for c in ("gate", "mod", "mod"))

    def gain():
        return 1 + 0.2 * torch.randn(w, generator=g, device=DEV)

    plain = case["mod"] != "no"    # with a modulation the norm has no gain of its own
    s["weight"] = None if plain else gain()
    s["bias"] = None if plain or case["kind"] == "rms" else 0.1 * gain()
    s["branch_weight"] = None if case["branch"] == "none" else gain()
    s["branch_bias"] = 0.1 * gain() if case["branch"] == "layer" else None
    return s


def _rotate(v, group):
    """v times the normalised Hadamard matrix of each group of channels."""
    if group == 1:
        return v
    h = torch.ones(1, 1, device=v.device)
    while h.shape[0] < group:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return torch.matmul(v.view(-1, group), h * group ** -0.5).view(v.shape)


def _plain_linear(s):
    case = s["case"]
    v = s["x"].float()
    if case["act"] == "swiglu":
        gate, up = v[:, :case["k"]], v[:, case["k"]:]
        v = gate / (1 + torch.exp(-gate)) * up
    q, e = _microscale(_rotate(v, case["group"]))
    v = (q * _power_of_two(e)).view(case["m"], case["k"])
    y = torch.matmul(v, _values(s["codes"], s["scales"]).T)
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


def _plain_normed(v, kind, weight, bias):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    v = v if weight is None else v * weight
    return v if bias is None else v + bias


def _along(m):
    """A modulation as something that [batch, tokens, width] broadcasts with."""
    return m.float().unsqueeze(1) if m.dim() == 2 else m.float()


def _plain_norm(s):
    case = s["case"]
    y = _plain_normed(s["branch"].float(), case["branch"], s["branch_weight"], s["branch_bias"])
    if s["gate"] is not None:
        y = y * _along(s["gate"])
    r = case["residual_scale"] * s["x"].float() + case["branch_scale"] * y
    h = _plain_normed(r, case["kind"], s["weight"], s["bias"])
    if s["scale"] is not None:
        h = h * (1 + _along(s["scale"])) + _along(s["shift"])
    return r.to(s["x"].dtype), h.to(s["x"].dtype)


def run(s):
    case = s["case"]
    if case["op"] == "quant":
        if own:
            import swiglu_mlp_amd as ck
            quantize = ck.ck_mx4_weight_prep if case["dtype"] == "fp32" else ck.ck_mx4_act_quant
            return ck.ck_mx4_dequant(*quantize(s["x"], group=1), rows=case["m"], k=case["k"])
        q, e = _microscale(s["x"].float())
        return (q * _power_of_two(e)).view(s["x"].shape).to(torch.bfloat16)
    if case["op"] == "linear":
        if own:
            import swiglu_mlp_amd as ck
            return ck.ck_mx4_linear(s["x"], *s["weight"], n=case["n"], group=case["group"], input_act=case["act"],
                                    bias=s["bias"], residual=s["residual"])
        return _plain_linear(s)
    if own:
        import swiglu_mlp_amd as ck
        return ck.ck_block_norm(s["x"], s["branch"], gate=s["gate"], residual_scale=case["residual_scale"],
                                branch_scale=case["branch_scale"], branch_norm=case["branch"],
                                branch_weight=s["branch_weight"], branch_bias=s["branch_bias"], norm=case["kind"],
                                weight=s["weight"], bias=s["bias"], scale=s["scale"], shift=s["shift"], eps=EPS)
    return _plain_norm(s)


def work(case):
    """Each input read once and each output written once (4-bit values with their scales: 17 / 32 byte); products and
    sums of the formula."""
    if case["op"] == "quant":
        n = case["m"] * case["k"]
        return {"bytes": n * ((4 if case["dtype"] == "fp32" else 2) + 2) + n * 17 // 32, "flops": 4 * n}
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        x = m * k * (4 if case["act"] == "swiglu" else 2)
        extra = (4 * n if case["bias"] else 0) + (2 * m * n if case["residual"] else 0)
        return {"bytes": x + n * k * 17 // 32 + 2 * m * n + extra, "flops": 2 * m * n * k}
    n, size = case["b"] * case["t"] * case["w"], {"no": 0, "channel": 1, "sequence": case["b"],
                                                  "token": case["b"] * case["t"]}
    return {"bytes": 8 * n + 2 * case["w"] * (size[case["gate"]] + 2 * size[case["mod"]]) + 8 * case["w"],
            "flops": (12 if case["branch"] == "none" else 17) * n}


# ---- the definitions in 64 bits ----


def _exact_microscaled(v):
    """Each 32 values as the nearest of +-LEVELS times 2^(floor(log2 of the largest) - 2), ties to the even code."""
    rows, k = v.shape
    v = v.double().view(rows, k // 32, 32)
    unit = torch.exp2(torch.floor(torch.log2(v.abs().amax(-1, keepdim=True).clamp_min(1e-30))) - 2)
    a = v.abs() / unit
    out = torch.zeros_like(a)
    for code in range(1, 8):    # a value passes the middle below an odd code only when it is above it
        middle = (LEVELS[code - 1] + LEVELS[code]) / 2
        out = torch.where(a > middle if code % 2 else a >= middle, LEVELS[code], out)
    return (torch.copysign(out, v) * unit).view(rows, k)


def _exact_rotated(v, group):
    """The butterflies of the Hadamard transform, one stride after the other."""
    v, h = v.reshape(-1, group), 1
    while h < group:
        p = v.view(-1, group // (2 * h), 2, h)
        v = torch.stack([p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]], 2).view(-1, group)
        h *= 2
    return v / math.sqrt(group)


def _exact_weight(codes, scales):
    lo, hi = (codes & 15).long(), (codes >> 4).long()
    code = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.long, device=DEV)
    code[:, 0::2], code[:, 1::2] = lo, hi
    size = torch.tensor(LEVELS, dtype=torch.float64, device=DEV)[code & 7]
    size = torch.where(code >= 8, -size, size)
    return size * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def _exact_normed(v, kind, weight, bias):
    if kind == "none":
        return v
    mean = v.mean(-1, keepdim=True) if kind == "layer" else 0.0
    spread = torch.sqrt(((v - mean) ** 2).mean(-1, keepdim=True) + EPS)
    v = (v - mean) / spread * (1.0 if weight is None else weight.double())
    return v + (0.0 if bias is None else bias.double())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_microscaled(s["x"])
    if case["op"] == "linear":
        w, k = _exact_weight(s["codes"], s["scales"]), case["k"]
        y = torch.empty(case["m"], case["n"], dtype=torch.float64, device=DEV)
        for at in range(0, case["m"], 2048):
            v = s["x"][at:at + 2048].double()
            if case["act"] == "swiglu":
                v = v[:, :k] * torch.sigmoid(v[:, :k]) * v[:, k:]
            rows = v.shape[0]
            v = _exact_microscaled(_exact_rotated(v, case["group"]).reshape(rows, k))
            y[at:at + 2048] = v @ w.T
        if s["bias"] is not None:
            y += s["bias"].double()
        if s["residual"] is not None:
            y += s["residual"].double()
        return y
    b, w = case["b"], case["w"]
    r_all, h_all = [], []
    for i in range(b):
        y = _exact_normed(s["branch"][i].double(), case["branch"], s["branch_weight"], s["branch_bias"])
        gate, scale, shift = (None if s[c] is None else (s[c] if s[c].dim() == 1 else s[c][i]).double()
                              for c in ("gate", "scale", "shift"))
        y = y if gate is None else y * gate.view(-1, w)
        r = s["x"][i].double() * case["residual_scale"] + y * case["branch_scale"]
        h = _exact_normed(r, case["kind"], s["weight"], s["bias"])
        h = h if scale is None else h * (scale.view(-1, w) + 1) + shift.view(-1, w)
        r_all.append(r)
        h_all.append(h)
    return torch.stack(r_all), torch.stack(h_all)
