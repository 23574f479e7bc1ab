"""The attention-side operators, as cases that can be measured.

Two operators surround the INT8 projections of a transformer block whose queries look at an encoder's states:

* ``norm``: the RMS norm of every query and key head with the position rotation in the same pass
  (``ck_qk_norm_rope``);
* ``attn``: attention of the queries over encoder keys and values of another length (``ck_cross_attn``), from the
  many rows of an image or video latent down to one token per sequence.

``run`` computes either in its plain form (elementary torch operations in 32 bits) or, with ``own`` set, through the
library.  Tensors are ``[batch, tokens, heads, head_dim]`` views of projection outputs, as a block has them.
"""
import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def _norm(name, b, tq, tk, hq, hkv, d, rot, pairing, dtype, packed, k_rope, pos):
    return {"name": name, "op": "norm", "b": b, "tq": tq, "tk": tk, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "pairing": pairing, "dtype": dtype, "packed": packed, "k_rope": k_rope, "pos": pos}


def _attn(name, bk, share, tq, tk, hq, hkv, d, dtype, lens, mask):
    return {"name": name, "op": "attn", "bk": bk, "share": share, "tq": tq, "tk": tk, "hq": hq, "hkv": hkv, "d": d,
            "dtype": dtype, "lens": lens, "mask": mask}


def listed():
    return [
        # one new token of 16 sequences in a decoder layer, each at its own position: latency alone
        _norm("norm one token", 16, 1, 1, 32, 8, 128, 128, "half", "bf16", True, True, True),
        # an image latent's queries (rotated) and a prompt's keys (no positions), 24 heads of 128 channels
        _norm("norm image and prompt", 2, 4096, 512, 24, 24, 128, 128, "interleaved", "bf16", False, False, False),
        # odd token and head counts, half of the channels rotated, packed [q | k | v] rows
        _norm("norm odd", 3, 777, 777, 14, 2, 64, 32, "half", "fp16", True, True, False),
        # the prefill of four long sequences, packed [q | k | v] rows
        _norm("norm long", 4, 16384, 16384, 32, 8, 128, 128, "half", "bf16", True, True, False),
        # one token of 5 beams for each of 2 utterances, the beams sharing the encoder's states
        _attn("attn beams", 2, 5, 1, 1500, 16, 16, 64, "fp16", "full", 0),
        # one token of 32 sequences, 4 query heads to a key head, encoder states padded to 4096 (one of them empty)
        _attn("attn one token", 32, 1, 1, 4096, 32, 8, 128, "bf16", "ragged", 0),
        # one token over a single very long encoded document
        _attn("attn one token, long", 1, 1, 1, 131072, 32, 8, 128, "bf16", "full", 0),
        # 64 learned queries over the patches of four pictures: few rows, many keys
        _attn("attn learned queries", 4, 1, 64, 4096, 16, 16, 64, "bf16", "full", 0),
        # a small image latent over a 77-token prompt, 72 channels a head
        _attn("attn short prompt", 2, 1, 1024, 77, 16, 16, 72, "fp16", "full", 0),
        # padded encoder batch: odd query and key counts, grouped heads, one sequence without any state
        _attn("attn padded batch", 7, 1, 333, 1023, 20, 4, 80, "fp16", "ragged", 0),
        # the image block of c5's width (24 heads of 128) over a 512-token prompt with dropped tokens
        _attn("attn image, masked prompt", 2, 1, 4096, 512, 24, 24, 128, "bf16", "full", 70),
        # a long video latent over the states of a long context
        _attn("attn video", 1, 1, 16384, 4096, 24, 24, 128, "bf16", "full", 0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Another case of the same ranges, no dearer than the largest listed one of its operator."""
    while True:
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        g = rng.choice([1, 1, 2, 4, 8])
        hkv = rng.randint(1, 24) if g == 1 else rng.randint(1, 8)
        if rng.random() < 0.35:
            d = rng.choice([64, 72, 80, 96, 128, 128])
            pairing = rng.choice(["half", "interleaved"])
            rot = rng.choice([d // 16 * 16, max(16, d // 2 // 16 * 16)])
            tq = _log(rng, 1, 16384)
            packed = rng.random() < 0.5
            tk = tq if packed else _log(rng, 1, 4096)
            case = _norm("", rng.randint(1, 8), tq, tk, g * hkv, hkv, d, rot, pairing, dtype, packed,
                         rng.random() < 0.7, rng.random() < 0.4)
            most = work(listed()[3])["bytes"]
            fits = work(case)["bytes"] <= most
        else:
            d = rng.choice([64, 64, 72, 80, 96, 128, 128, 128])
            tq = 1 if rng.random() < 0.3 else _log(rng, 2, 16384)
            case = _attn("", rng.randint(1, 16), rng.choice([1, 1, 1, 4]), tq, _log(rng, 1, 131072 if tq == 1 else 8192),
                         g * hkv, hkv, d, dtype, rng.choice(["full", "full", "ragged"]), rng.choice([0, 0, 0, 70]))
            w, small, large = work(case), work(listed()[6])["bytes"], work(listed()[11])
            scores = case["bk"] * case["share"] * case["hq"] * case["tq"] * case["tk"]
            fits = (w["bytes"] <= (small if tq == 1 else large["bytes"]) and w["flops"] <= large["flops"]
                    and scores <= 24 * 16384 * 4096)
        if fits:
            del case["name"]
            return case


def _lens(case):
    """Valid keys of each encoder sequence: all, or spread evenly from none to all."""
    bk, tk = case["bk"], case["tk"]
    if case["lens"] == "full" or bk == 1:
        return [tk] * bk
    return [tk * i // (bk - 1) for i in range(bk)]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _projection(g, tokens, width, dtype):
    """A projection's output: near-normal values with one channel in a hundred twenty times larger."""
    x = torch.randn(tokens, width, generator=g, device=DEV)
    x *= torch.where(torch.rand(width, generator=g, device=DEV) < 0.01, 20.0, 1.0)
    return x.to(dtype)


def _tables(positions, rot):
    """Rotation tables [positions, rot / 2] in 32 bits, angles position * 10000^(-2 i / rot)."""
    f = torch.pow(10000.0, -torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    g, dt, d, hq, hkv = _gen(seed), TYPES[case["dtype"]], case["d"], case["hq"], case["hkv"]
    s = {"case": case}
    if case["op"] == "norm":
        b, tq, tk = case["b"], case["tq"], case["tk"]
        if case["packed"]:
            qkv = _projection(g, b * tq, (hq + 2 * hkv) * d, dt).view(b, tq, hq + 2 * hkv, d)
            s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv]
        else:
            s["q"] = _projection(g, b * tq, hq * d, dt).view(b, tq, hq, d)
            s["k"] = _projection(g, b * tk, 2 * hkv * d, dt).view(b, tk, 2 * hkv, d)[:, :, :hkv]
        s["qw"], s["kw"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV) for _ in range(2))
        s["rope"] = _tables(max(tq, tk) + 1000, case["rot"])
        s["k_rope"] = s["rope"] if case["k_rope"] else None
        s["qp"] = s["kp"] = None
        if case["pos"]:   # every sequence at an offset of its own
            first = torch.randint(0, 1000, (b, 1), generator=g, device=DEV, dtype=torch.int32)
            s["qp"] = first + torch.arange(tq, device=DEV, dtype=torch.int32)
            s["kp"] = first + torch.arange(tk, device=DEV, dtype=torch.int32) if case["k_rope"] else None
        return s
    bk, n, tq, tk = case["bk"], case["share"], case["tq"], case["tk"]
    # queries and keys after their norms: unit channels times a gain
    s["q"] = (1.5 * torch.randn(bk * n, tq, hq, d, generator=g, device=DEV)).to(dt)
    kv = torch.randn(bk, tk, 2 * hkv, d, generator=g, device=DEV)
    kv[:, :, hkv:] += 0.5 * torch.randn(hkv, d, generator=g, device=DEV)   # values with a mean in each channel
    kv = kv.to(dt)
    s["k"], s["v"] = kv[:, :, :hkv], kv[:, :, hkv:]
    s["len"] = None if case["lens"] == "full" else torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
    s["mask"] = torch.rand(bk, tk, generator=g, device=DEV) * 100 < case["mask"] if case["mask"] else None
    return s


def _plain_norm(x, weight, rope, pos, pairing):
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight
    if rope is None:
        return y.to(x.dtype)
    cos, sin = rope
    half = cos.shape[1]
    at = torch.arange(x.shape[1], device=x.device)[None] if pos is None else pos.long()
    cos, sin = cos[at][:, :, None], sin[at][:, :, None]       # [batch or 1, tokens, 1, half]
    r, rest = y[..., :2 * half], y[..., 2 * half:]
    if pairing == "half":
        a, b = r[..., :half], r[..., half:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, rest], -1).to(x.dtype)


def _plain_attn(q, k, v, kv_len, key_mask):
    (b, tq, hq, d), (bk, tk, hkv, _) = q.shape, k.shape
    n, g = b // bk, hq // hkv
    # the rows of one encoder sequence and key head: its sharing sequences, their tokens and the grouped heads
    rows = q.float().view(bk, n, tq, hkv, g, d).permute(0, 3, 1, 2, 4, 5).reshape(bk, hkv, n * tq * g, d)
    kt = k.float().permute(0, 2, 3, 1).contiguous()
    s = torch.matmul(rows, kt).mul_(d ** -0.5)
    allowed = torch.ones(bk, tk, dtype=torch.bool, device=q.device)
    if kv_len is not None:
        allowed = allowed & (torch.arange(tk, device=q.device) < kv_len[:, None])
    if key_mask is not None:
        allowed = allowed & key_mask
    s.masked_fill_(~allowed[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.float().permute(0, 2, 1, 3).contiguous()) / torch.where(total == 0, 1.0, total)
    return o.view(bk, hkv, n, tq, g, d).permute(0, 2, 3, 1, 4, 5).reshape(b, tq, hq, d).to(q.dtype)


def run(s):
    case = s["case"]
    if case["op"] == "norm":
        if own:
            import swiglu_mlp_amd as ck
            return ck.ck_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], q_rope=s["rope"], k_rope=s["k_rope"],
                                      q_pos=s["qp"], k_pos=s["kp"], pairing=case["pairing"], eps=EPS)
        return (_plain_norm(s["q"], s["qw"], s["rope"], s["qp"], case["pairing"]),
                _plain_norm(s["k"], s["kw"], s["k_rope"], s["kp"], case["pairing"]))
    if own:
        import swiglu_mlp_amd as ck
        return ck.ck_cross_attn(s["q"], s["k"], s["v"], kv_len=s["len"], key_mask=s["mask"])
    return _plain_attn(s["q"], s["k"], s["v"], s["len"], s["mask"])


def work(case):
    """Each input read once and each output written once; products and sums of the formula."""
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    if case["op"] == "norm":
        nq, nk = case["b"] * case["tq"] * hq * d, case["b"] * case["tk"] * hkv * d
        table = 8 * (case["rot"] // 2) * max(case["tq"], case["tk"] if case["k_rope"] else 0)
        pos = 4 * case["b"] * (case["tq"] + (case["tk"] if case["k_rope"] else 0)) if case["pos"] else 0
        return {"bytes": 4 * (nq + nk) + table + pos + 8 * d, "flops": 7 * (nq + nk)}
    keys = sum(_lens(case)) * (case["mask"] / 100 if case["mask"] else 1)   # (encoder sequence, key) pairs read
    rows = case["share"] * case["tq"] * hq                                  # of one encoder sequence
    return {"bytes": int(4 * case["bk"] * rows * d + 4 * keys * hkv * d + (case["bk"] * case["tk"] if case["mask"] else 0)),
            "flops": int(4 * rows * keys * d)}


def _exact_norm(x, w, rope, pos, pairing):
    """Each head divided by the root of its mean square, then pair i turned by its token's angle, as a complex number."""
    x = x.double()
    z = x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + EPS) * w.double()
    if rope is None:
        return z
    turn = torch.complex(rope[0].double(), rope[1].double())
    rot = 2 * turn.shape[1]
    turn = turn[:x.shape[1]].unsqueeze(0) if pos is None else turn[pos.long()]
    first, second = (z[..., :rot // 2], z[..., rot // 2:rot]) if pairing == "half" else (z[..., 0:rot:2], z[..., 1:rot:2])
    c = torch.complex(first.contiguous(), second.contiguous()) * turn.unsqueeze(2)
    out = z.clone()
    if pairing == "half":
        out[..., :rot // 2], out[..., rot // 2:rot] = c.real, c.imag
    else:
        out[..., 0:rot:2], out[..., 1:rot:2] = c.real, c.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return (_exact_norm(s["q"], s["qw"], s["rope"], s["qp"], case["pairing"]),
                _exact_norm(s["k"], s["kw"], s["k_rope"], s["kp"], case["pairing"]))
    q, k, v = s["q"], s["k"], s["v"]
    n, g = case["share"], case["hq"] // case["hkv"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    for i, valid in enumerate(_lens(case)):
        keep = torch.arange(valid, device=DEV)
        if s["mask"] is not None:
            keep = keep[s["mask"][i, :valid]]
        if not len(keep):
            continue   # a row without any key is zero
        for h in range(case["hq"]):
            kk, vv = k[i, keep, h // g].double(), v[i, keep, h // g].double()
            for b in range(i * n, i * n + n):
                out[b, :, h] = torch.softmax(q[b, :, h].double() @ kk.T.contiguous() / math.sqrt(case["d"]), -1) @ vv
    return out
