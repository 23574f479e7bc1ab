"""ck_block_norm against its formula in 64 bits.

Bounds, u the largest relative error of a rounding to the 16-bit type (2^-8 for
BF16, 2^-11 for FP16; FP16 values below 2^-14 round to multiples of 2^-24), f =
2^-24, W the width:
  a norm   a sum over the row is at most W roundings off, W f of its terms' sizes: the
           mean W f mean |v|, the mean square W f of itself (half of that in its root);
           then a reciprocal root within 2 f and four more roundings.  With N(v) =
           (v - mean) R w + b: (W + 8) f (|v| + mean |v|) R |w|, and f |b|.
  r        the branch's norm times gate and branch_scale, two products and one sum,
           each f of its size: below, e_r.
  h        the norm of an r that is e_r off: e_r and its mean over the row through R |w|,
           and through R itself (|N| times the root mean square of e_r R); products and
           sums of the modulation f of their sizes.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import swiglu_mlp_amd as ck  # noqa: E402

DEV = "cuda:0"
BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, FP16: 2.0 ** -11}
TINY = {BF16: 0.0, FP16: 2.0 ** -25}
F = 2.0 ** -24
EPS = 1e-6


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def say(msg):
    print(f"[block norm] {msg}", flush=True)


def normed(v, err, kind, w, b, eps):
    """(N(v), bound of its error) for a v that is `err` off."""
    if kind in (None, "none"):
        return v, err
    width = v.shape[-1]
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
    root = 1 / torch.sqrt(((v - mean) ** 2).mean(-1, keepdim=True) + eps)
    w = torch.ones(width, device=DEV, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(width, device=DEV, dtype=torch.float64) if b is None else b.double()
    z = (v - mean) * root
    avg = v.abs().mean(-1, keepdim=True) if kind == "layer" else 0.0
    e = err + (err.mean(-1, keepdim=True) if kind == "layer" else 0.0) + (width + 8) * F * (v.abs() + avg)
    spread = (e ** 2).mean(-1, keepdim=True).sqrt() * root + (width + 8) * F
    return z * w + b, (e * root + z.abs() * spread) * w.abs() + 2 * F * (z * w).abs() + F * b.abs()


def reference(x, branch=None, gate=None, residual_scale=1.0, branch_scale=1.0, branch_norm=None, branch_weight=None,
              branch_bias=None, norm="rms", weight=None, bias=None, scale=None, shift=None, eps=EPS):
    """(r, its bound, h, its bound)."""
    def along(m):
        return None if m is None else (m.double().unsqueeze(1) if m.dim() == 2 and x.dim() == 3 else m.double())

    x64 = x.double()
    r, err = x64 * residual_scale, F * (x64 * residual_scale).abs()
    if branch is not None:
        y, e = normed(branch.double(), torch.zeros_like(x64), branch_norm, branch_weight, branch_bias, eps)
        g = along(gate)
        if g is not None:
            y, e = y * g, e * g.abs() + F * (y * g).abs()
        r = r + branch_scale * y
        err = err + abs(branch_scale) * e + 2 * F * (abs(branch_scale) * y.abs() + r.abs())
    h, eh = normed(r, err, norm, weight, bias, eps)
    s, t = along(scale), along(shift)
    if s is not None:
        eh = eh * (1 + s).abs() + F * ((h * s).abs() + (h * (1 + s)).abs())
        h = h * (1 + s)
    if t is not None:
        h = h + t
        eh = eh + F * h.abs()
    return r, err, h, eh


def close(got, want, err, dtype, what):
    assert got.dtype == dtype
    bound = err + U[dtype] * (want.abs() + err) + TINY[dtype]
    off = (got.double() - want).abs()
    assert (off <= bound).all(), (what, (off / bound).max().item())


def check(x, branch, kw, what):
    r, er, h, eh = reference(x, branch, **kw)
    got = ck.ck_block_norm(x, branch, eps=EPS, **kw)
    if branch is None:
        close(got, h, eh, x.dtype, what)
    elif kw.get("norm", "rms") in (None, "none"):
        close(got, r, er, x.dtype, what)
    else:
        close(got[0], r, er, x.dtype, (what, "r"))
        close(got[1], h, eh, x.dtype, (what, "h"))
    return got


def stream(g, *shape, dtype=BF16):
    x = torch.randn(*shape, generator=g, device=DEV)
    x *= torch.where(torch.rand(shape[-1], generator=g, device=DEV) < 0.02, 20.0, 1.0)
    return (x + 0.3).to(dtype)


WIDTHS = [8, 16, 64, 72, 200, 504, 512, 520, 1024, 1032, 1160, 2048, 2056, 4088, 4096, 4104, 6200, 8192, 8200, 12288, 16384]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("w", WIDTHS)
def test_widths(w, dtype):
    say(f"width {w} {dtype}")
    g = gen(w)
    for b, t in ((1, 1), (3, 7), (2, 100 if w > 4096 else 400)):
        x, y = stream(g, b, t, w, dtype=dtype), torch.randn(b, t, w, generator=g, device=DEV).to(dtype)
        weight, bias = 1 + 0.2 * torch.randn(w, generator=g, device=DEV), torch.randn(w, generator=g, device=DEV)
        check(x, y, dict(weight=weight), (w, b, t, "rms"))
        check(x, y, dict(norm="layer", branch_norm="rms", branch_weight=weight, weight=weight, bias=bias), (w, b, t, "both"))
        check(x, None, dict(norm="layer"), (w, b, t, "first"))


@pytest.mark.parametrize("rows", [1, 2, 5, 63, 600, 3000, 9000])
@pytest.mark.parametrize("w", [64, 1160, 4096])
def test_rows(rows, w):
    g = gen(rows + w)
    x, y = stream(g, rows, w), torch.randn(rows, w, generator=g, device=DEV).to(BF16)
    check(x, y, dict(branch_norm="layer", residual_scale=1.5, branch_scale=-0.22), (rows, w))


@pytest.mark.parametrize("mod", [BF16, F32])
@pytest.mark.parametrize("branch_norm", [None, "rms", "layer"])
@pytest.mark.parametrize("norm", [None, "rms", "layer"])
def test_modulations(norm, branch_norm, mod):
    g, b, t, w = gen(1), 3, 21, 136
    x, y = stream(g, b, t, w), torch.randn(b, t, w, generator=g, device=DEV).to(BF16)
    bw = 1 + 0.2 * torch.randn(w, generator=g, device=DEV)
    for shape in ((w,), (b, w), (b, t, w)):
        gate, scale, shift = (torch.randn(shape, generator=g, device=DEV).to(mod) for _ in range(3))
        kw = dict(gate=gate, branch_norm=branch_norm, norm=norm, branch_scale=0.5)
        if branch_norm:
            kw.update(branch_weight=bw, branch_bias=bw - 1)
        if norm:
            kw.update(scale=scale, shift=shift, weight=bw)
        check(x, y, kw, (shape, norm, branch_norm))
        if norm:
            check(x, None, dict(norm=norm, scale=scale), (shape, "scale"))
            check(x, None, dict(norm=norm, shift=shift, bias=bw), (shape, "shift"))


def test_columns_of_a_packed_modulation_and_strided_rows():
    g, b, t, w = gen(2), 2, 33, 264
    packed = torch.randn(b, 6 * w, generator=g, device=DEV).to(BF16)
    gate, scale, shift = (packed[:, i * w:(i + 1) * w] for i in (2, 4, 3))
    wide = stream(g, b, t, 3 * w)
    x, y = wide[..., :w], wide[..., 2 * w:]
    want = check(x, y, dict(gate=gate, scale=scale, shift=shift, norm="layer"), "strided")
    # a transposed batch, and a modulation that all tokens of a batch of views share
    xt, yt = x.transpose(0, 1).contiguous().transpose(0, 1), y.transpose(0, 1)
    with pytest.raises(ValueError):
        ck.ck_block_norm(xt, yt.contiguous().permute(2, 1, 0))
    got = ck.ck_block_norm(xt, y, gate=gate[:, None].expand(b, t, w), scale=scale, shift=shift, norm="layer", eps=EPS)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_in_place_and_given_outputs():
    g, b, t, w = gen(3), 2, 40, 1160
    x, y = stream(g, b, t, w), torch.randn(b, t, w, generator=g, device=DEV).to(BF16)
    kw = dict(norm="layer", branch_norm="rms", eps=EPS)
    r, h = ck.ck_block_norm(x, y, **kw)
    buf = torch.zeros(b, t, 3 * w, dtype=BF16, device=DEV)
    for xo, ho in ((x.clone(), None), (buf[..., :w], buf[..., 2 * w:])):
        xi, yi = (x, y) if ho is not None else (xo, y.clone())
        got = ck.ck_block_norm(xi, yi, x_out=xo, out=yi if ho is None else ho, **kw)
        assert torch.equal(got[0], r) and torch.equal(got[1], h) and got[0].data_ptr() == xo.data_ptr()
    assert not buf[..., w:2 * w].any()
    z = x.clone()
    assert torch.equal(ck.ck_block_norm(z, out=z, eps=EPS), ck.ck_block_norm(x, eps=EPS)) and not torch.equal(z, x)


def test_zero_rows_large_means_and_not_finite_values():
    g, w = gen(4), 512
    x = stream(g, 6, w)
    x[0] = 0
    x[1] = 1000 + torch.randn(w, generator=g, device=DEV).to(BF16)      # a mean far above the spread
    x[2] = 7.0                                                         # no spread at all
    x[3] = (x[3].float() * 1e16).to(BF16)                              # large squares
    for norm in ("rms", "layer"):
        check(x, None, dict(norm=norm), norm)
    bad = x.clone()
    bad[4, 9], bad[5, 3] = math.nan, math.inf
    for norm in ("rms", "layer"):
        got, want = ck.ck_block_norm(bad, norm=norm, eps=EPS), ck.ck_block_norm(x, norm=norm, eps=EPS)
        assert torch.equal(got[:4], want[:4]) and torch.isnan(got[4]).all() and torch.isnan(got[5, 3])
        y = torch.randn(6, w, generator=g, device=DEV).to(BF16)
        r, h = ck.ck_block_norm(bad, y, norm=norm, eps=EPS)
        assert torch.isnan(r[4, 9]) and torch.isinf(r[5, 3]) and torch.isfinite(r).sum() == 6 * w - 2


def test_h_is_of_the_unrounded_sum():
    """A branch far below the residual's rounding still reaches h: with x = c constant, h is the branch's norm."""
    w = 1024
    y = torch.randn(8, w, generator=gen(5), device=DEV).to(BF16)
    x = torch.full((8, w), 64.0, dtype=BF16, device=DEV)
    r, h = ck.ck_block_norm(x, y, branch_scale=2.0 ** -7, norm="layer", eps=EPS)
    want = torch.nn.functional.layer_norm(y.double() * 2.0 ** -7, (w,), eps=EPS)
    assert ((h.double() - want).norm() / want.norm()).item() < 2.0 ** -7
    check(x, y, dict(branch_scale=2.0 ** -7, norm="layer"), "small branch")


def test_offsets_past_32_bits():
    """Rows more than 2^32 bytes apart, and more than 2^32 elements in all."""
    w = 4096
    rows = 540_000                                   # 2.2e9 values, 4.4 GB
    x = torch.zeros(rows, w, dtype=BF16, device=DEV)
    at = [0, 1, 262144, 524288, 530000, rows - 1]
    x[at] = stream(gen(6), len(at), w)
    want = ck.ck_block_norm(x[at].contiguous(), eps=EPS)
    got = ck.ck_block_norm(x, eps=EPS)
    assert torch.equal(got[at], want)
    got[at] = 0
    assert not got.any()
    far = x.view(-1).as_strided((2, 2, w), (2 ** 31, w, 1))
    want = ck.ck_block_norm(far.contiguous(), eps=EPS)
    assert torch.equal(ck.ck_block_norm(far, eps=EPS), want)
    ck.ck_block_norm(far, eps=EPS, out=far)
    assert torch.equal(far, want)


def test_empty():
    for shape in ((0, 64), (2, 0, 64), (0, 3, 64)):
        x = torch.empty(shape, dtype=BF16, device=DEV)
        r, h = ck.ck_block_norm(x, x)
        assert r.shape == h.shape == x.shape


def test_same_bits_every_time_on_a_stream_and_in_a_graph():
    cases = []
    for b, t, w in ((16, 1, 4096), (2, 300, 1160), (1, 5000, 64), (1, 40, 16384)):
        g = gen(w)
        x, y = stream(g, b, t, w), torch.randn(b, t, w, generator=g, device=DEV).to(BF16)
        m = torch.randn(b, w, generator=g, device=DEV).to(BF16)
        cases.append((x, y, m, torch.empty_like(x), torch.empty_like(x)))

    def step():
        for x, y, m, r, h in cases:
            ck.ck_block_norm(x, y, gate=m, scale=m, shift=m, norm="layer", branch_norm="rms", x_out=r, out=h)

    step()
    want = [(c[3].clone(), c[4].clone()) for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for c in cases:
            c[3].fill_(i), c[4].fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        for c, (r, h) in zip(cases, want):
            assert torch.equal(c[3], r) and torch.equal(c[4], h)
        assert torch.equal(ck.ck_block_norm(cases[0][0]), ck.ck_block_norm(cases[0][0].clone()))


def test_refusals():
    x, w = torch.randn(2, 4, 64, device=DEV).to(BF16), torch.ones(64, device=DEV)
    n = ck.ck_block_norm

    def no(*a, **kw):
        with pytest.raises(ValueError):
            n(*a, **kw)

    no(x.float()), no(x.cpu()), no(x[0, 0]), no(x[..., :60]), no(x[..., 4:]), no(None), no(x, norm=None), no(x, norm="batch")
    no(x, x.to(FP16)), no(x, x[:, :3]), no(x, x.cpu()), no(x, branch_norm="mean"), no(x, branch_norm="rms")
    no(x, gate=w), no(x, x_out=x), no(x, x, norm=None, out=x), no(x, x, norm=None, scale=w), no(x, x, branch_weight=w)
    no(x, weight=w[:32]), no(x, weight=w.to(BF16)), no(x, weight=w.cpu()), no(x, bias=torch.ones(128, device=DEV)[::2])
    no(x, x, gate=w.double()), no(x, x, gate=w.to(FP16)), no(x, x, gate=w, scale=w.to(BF16)), no(x, scale=w[:8])
    no(x, scale=torch.ones(3, 64, device=DEV)), no(x, scale=torch.ones(4, 64, device=DEV)), no(x[0], scale=torch.ones(2, 64, device=DEV))
    no(torch.ones(1, 16392, dtype=BF16, device=DEV)), no(x.transpose(1, 2)), no(x, out=x.transpose(1, 2))
    no(x, out=x[:, :, :32]), no(x, out=torch.empty(2, 4, 64, device=DEV)), no(x, out=x[:1].expand(2, 4, 64))
    for eps in (0.0, math.nan, math.inf, -1.0):
        with pytest.raises(ck.CKError):
            n(x, eps=eps)
    for bad in (math.nan, math.inf):
        with pytest.raises(ck.CKError):
            n(x, x, branch_scale=bad)
        with pytest.raises(ck.CKError):
            n(x, x, residual_scale=bad)


def test_refusals_of_shared_memory():
    buf = torch.randn(1 << 16, device=DEV).to(BF16)
    x, y, o = (buf[i << 12:(i << 12) + 2 * 3 * 64].view(2, 3, 64) for i in range(3))
    shifted = buf[8:8 + 384].view(2, 3, 64)
    m, f = buf[1 << 15:(1 << 15) + 64], buf[1 << 14:(1 << 14) + 128].view(F32)
    ck.ck_block_norm(x, y, gate=m, weight=f, x_out=o)
    for kw in (dict(x_out=shifted), dict(out=shifted), dict(out=buf[(1 << 12) - 8:(1 << 12) + 376].view(2, 3, 64)),
               dict(x_out=o, out=o), dict(x_out=x, out=x), dict(gate=o[0, 0], x_out=o), dict(scale=o[1, 2], out=o),
               dict(shift=o[:, 0], out=o), dict(weight=o.view(-1)[:128].view(F32), out=o),
               dict(bias=o.view(-1)[256:384].view(F32), x_out=o),
               dict(branch_norm="rms", branch_weight=o.view(-1)[:128].view(F32), x_out=o),
               dict(out=buf.as_strided((2, 3, 64), (192, 32, 1), 1 << 13))):
        with pytest.raises(ValueError):
            ck.ck_block_norm(x, y, **kw)


# ---------------------------------------------------------------- a block of norms, 4-bit linears and attention
def test_block_of_norms_linears_and_attention():
    """The example block against FP32 with unquantized weights.  Either operand of a 4-bit linear is a value's last step
    off at most: a relative (1/4) / sqrt(3) = 0.144 as a root mean square, sqrt(2) times that with both.  A branch has two
    linears in a row with a softmax' average or a product of halves between them: 2 x 0.204 of its size.  The sum of the
    branches' errors, each of its gated size, bounds the block's; and a block without its branches is further off."""
    import os
    import sys
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    from examples import gated_block as gb
    weights, x, modulation, rope = gb.synthetic(b=3, t=70, heads=4, d=64, inner=512)
    kept = x.clone()
    block = gb.GatedBlock(weights, 4)
    y = block(x, modulation, rope)
    assert torch.equal(x, kept)
    want, first, second = gb.reference(weights, 4, x, modulation, rope)
    off = (y.float() - want).norm()
    bound = 2 * math.sqrt(2) * 0.25 / math.sqrt(3) * (first.norm() + second.norm()) + U[BF16] * 3 * want.norm()
    say(f"block: off {off.item():.3f}, bound {bound.item():.3f}, branches {(first + second).norm().item():.3f}")
    assert off < bound and off < (first + second).norm()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = block(x, modulation, rope)
    for _ in range(3):
        z.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, y) and torch.equal(block(x, modulation, rope), y)


def test_modulations_of_one_token_or_one_sequence():
    """[batch, 1, width], as the chunks of a modulation come, and [1, tokens, width]: the same as written out."""
    g, b, t, w = gen(7), 3, 21, 136
    x, y = stream(g, b, t, w), torch.randn(b, t, w, generator=g, device=DEV).to(BF16)
    for mod in (BF16, F32):
        for shape in ((b, 1, w), (1, t, w), (1, 1, w)):
            wide = torch.randn(shape[0], shape[1], 6 * w, generator=g, device=DEV).to(mod)
            gate, scale, shift = (wide[..., i * w:(i + 1) * w] for i in (0, 3, 5))
            got = check_expanded(x, y, gate, scale, shift)
            assert all(torch.equal(p, q) for p, q in zip(got, ck.ck_block_norm(
                x, y, norm="layer", eps=EPS, **{n: m.expand(b, t, w).contiguous() for n, m in
                                                (("gate", gate), ("scale", scale), ("shift", shift))})))
    x2, m = x[0], torch.randn(1, w, generator=g, device=DEV)
    assert torch.equal(ck.ck_block_norm(x2, scale=m, eps=EPS), ck.ck_block_norm(x2, scale=m[0], eps=EPS))
    for bad in ((b, 2, w), (2, 1, w), (b, 1, w - 8), (1, b, 1, w), (b, t, 1)):
        with pytest.raises(ValueError):
            ck.ck_block_norm(x, scale=torch.ones(bad, device=DEV))
    with pytest.raises(ValueError):     # the channels of every second place
        ck.ck_block_norm(x, scale=torch.ones(b, 1, 2 * w, device=DEV)[..., ::2])
    with pytest.raises(ValueError):     # an output that overlaps such a modulation
        ck.ck_block_norm(x, scale=x[:, :1], out=x)


def check_expanded(x, y, gate, scale, shift):
    """Against the formula, which broadcasts."""
    r, er, h, eh = reference(x, y, gate.expand(x.shape), norm="layer", scale=scale.expand(x.shape),
                             shift=shift.expand(x.shape))
    got = ck.ck_block_norm(x, y, gate=gate, norm="layer", scale=scale, shift=shift, eps=EPS)
    close(got[0], r, er, x.dtype, (gate.shape, "r"))
    close(got[1], h, eh, x.dtype, (gate.shape, "h"))
    return got
