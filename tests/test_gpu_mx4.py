"""The MX FP4 linears (ck_mx4_*) against their definition in 64 bits.

What is exact: without a rotation and an activation the quantizer's steps are
(a power of two and one rounding to a grid), so codes and scales equal the
definition's; codes to values is exact.

Bounds elsewhere, u = 2^-8 the largest relative error of a rounding to BF16:
  rotated values  group sums of FP32 numbers: log2(group) roundings of partial sums
                  that |a|'s sum bounds and one product, so within
                  t = (log2(group) + 2) 2^-24 sum |a| / sqrt(group); with SwiGLU
                  each a is 4 2^-24 |a| off before that, and for a negative gate g
                  another |g| 2^-24 |a|: under 2^-21 |a| in all down to g = -4, and below
                  that |a| < |u| / 13 falls faster than |g| grows.  A code is then the
                  nearest of values within t, and a scale that of such a maximum.
  product         every one of the k products is exact in FP32 and passes at most 128
                  roundings in its instruction and one in each of the at most
                  k / 64 sums that follow, of partial sums within A = sum |x w|:
                  (128 + k / 64) 2^-23 A (2^-23: the matrix cores may truncate),
                  the bias' and the residual's sums 2^-24 of their terms, and u |y|.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import swiglu_mlp_amd as ck  # noqa: E402

DEV = "cuda:0"
BF16 = torch.bfloat16
U = 2.0 ** -8
LEVELS = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def say(msg):
    print(f"[mx4] {msg}", flush=True)


def values(codes, scales):
    """Row-major codes and scales as 64-bit values (NaN scales: NaN)."""
    c = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1).long()
    v = LEVELS[c & 7] * torch.where(c >= 8, -1.0, 1.0)
    s = torch.exp2(scales.double() - 127)
    s[scales == 255] = math.nan
    return v * s.repeat_interleave(32, 1)


def blocked(codes, scales):
    """Row-major codes and scales in the blocked layout, by its definition."""
    n, k = codes.shape[0], 2 * codes.shape[1]
    rp, kp = (n + 31) // 32 * 32, (k + 255) // 256 * 256
    c = torch.zeros(rp, kp // 2, dtype=torch.uint8, device=DEV)
    s = torch.zeros(rp, kp // 32, dtype=torch.uint8, device=DEV)
    c[:n, :k // 2], s[:n, :k // 32] = codes, scales
    # [block row, r, k / 64, half, 16] -> [block row, k / 64, half, r, 16];  [.., r, k / 256, j, half] -> [.., half, r, j]
    c = c.view(rp // 32, 32, kp // 64, 2, 16).permute(0, 2, 3, 1, 4).reshape(rp // 32, kp // 64, 1024)
    s = s.view(rp // 32, 32, kp // 256, 4, 2).permute(0, 2, 4, 1, 3).reshape(rp // 32, kp // 256, 256)
    return c.contiguous(), s.contiguous()


def rounded(v, scale):
    """(v 2^-e) to the nearest E2M1 value, ties to the even code, in 64 bits, times 2^e."""
    a = v.abs() / scale
    code = torch.zeros_like(a, dtype=torch.long)
    for c in range(1, 8):
        middle = (LEVELS[c - 1] + LEVELS[c]) / 2
        code = torch.where(a > middle if c % 2 else a >= middle, c, code)
    return LEVELS[code] * scale * torch.where(v < 0, -1.0, 1.0)


def scale_of(v):
    """The scale bytes of v [rows, blocks, 32] (64 bits)."""
    top = v.abs().amax(-1)
    e = torch.frexp(top)[1].long() - 1 - 2 + 127
    e = torch.where(top == 0, 0, e.clamp(min=0))
    return torch.where(torch.isfinite(v).all(-1), e, 255)


def hadamard(group):
    h = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    while h.shape[0] < group:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def activation(m, k, seed, act=None, outliers=True):
    x = torch.randn(m, 2 * k if act else k, generator=gen(seed), device=DEV)
    if outliers:
        x *= torch.where(torch.rand(x.shape[1], generator=gen(seed + 1), device=DEV) < 0.02, 20.0, 1.0)
    return x.to(BF16)


# ---------------------------------------------------------------- quantization
def check_exact(v, codes, scales, what):
    """Codes and scales (row-major) of v, quantized without a rotation."""
    rows, k = v.shape
    b = v.double().view(rows, k // 32, 32)
    want = scale_of(b)
    assert torch.equal(scales.long(), want), what
    s = torch.exp2(want.double() - 127).unsqueeze(-1)
    got, ref = values(codes, scales).view_as(b), rounded(b, s)
    ok = (want != 255).unsqueeze(-1)
    assert torch.equal(torch.where(ok, got, 0.0), torch.where(ok, ref, 0.0)), what


@pytest.mark.parametrize("m,k", [(1, 64), (1, 4096), (2, 192), (7, 320), (31, 256), (32, 512), (33, 2112), (77, 64),
                                 (300, 1088), (5, 32768)])
def test_quantize_exact(m, k):
    say(f"quantize {m} x {k}")
    x = activation(m, k, m + k)
    codes, scales = ck.ck_mx4_act_quant(x, group=1, layout="rows")
    check_exact(x, codes, scales, "activation")
    w = 0.02 * torch.randn(m, k, generator=gen(k), device=DEV)
    wc, ws = ck.ck_mx4_weight_prep(w, group=1, layout="rows")
    check_exact(w, wc, ws, "weight")
    # the blocked layout holds the same bytes (an activation's padding rows are not written)
    for a, rows, f, v in ((x, (codes, scales), ck.ck_mx4_act_quant, m), (w, (wc, ws), ck.ck_mx4_weight_prep, m)):
        bc, bs = f(a, group=1)
        rc, rs = blocked(*rows)
        r = torch.arange(32, device=DEV) < m - 32 * torch.arange(bc.shape[0], device=DEV)[:, None]
        live = r[:, None, None, :, None].expand(-1, bc.shape[1], 2, 32, 16).reshape(bc.shape)
        live_s = r[:, None, None, :, None].expand(-1, bs.shape[1], 2, 32, 4).reshape(bs.shape)
        assert torch.equal(values(torch.where(live, bc, 0).view(-1, 1024), torch.full((1,), 127, device=DEV, dtype=torch.uint8)
                                  .expand(bc.numel() // 1024, 64)),
                           values(torch.where(live, rc, 0).view(-1, 1024), torch.full((1,), 127, device=DEV, dtype=torch.uint8)
                                  .expand(bc.numel() // 1024, 64)))
        assert torch.equal(torch.where(live_s, bs, 0), torch.where(live_s, rs, 0))
        assert torch.equal(ck.ck_mx4_dequant(bc, bs, rows=m, k=k).double(), values(*rows))
        assert torch.equal(ck.ck_mx4_dequant(*rows).double(), values(*rows))
        if f is ck.ck_mx4_weight_prep:
            pc, ps = ck.ck_mx4_weight_pack(*rows)
            assert torch.equal(pc, rc) and torch.equal(ps, rs)


def test_quantize_borders():
    """Every tie, every exponent, subnormals, zeros, and values that are not finite."""
    mids = [0.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9, 0.5, 1.0, 1.5, 3.0, 4.0]
    rows = []
    for e in list(range(-133, -110)) + list(range(-20, 20)) + list(range(100, 125)):
        v = [m * 2.0 ** e for m in mids] + [-m * 2.0 ** e for m in mids]
        rows.append(v + [0.0] * 32)
    x = torch.tensor(rows, dtype=torch.float64, device=DEV).to(BF16)
    check_exact(x, *ck.ck_mx4_act_quant(x, group=1, layout="rows"), "borders")
    w = torch.tensor(rows, dtype=torch.float64, device=DEV)
    w = (w * (1 + 2.0 ** -23 * torch.randint(-1, 2, w.shape, generator=gen(5), device=DEV))).float()
    check_exact(w, *ck.ck_mx4_weight_prep(w, group=1, layout="rows"), "next to borders")
    x = activation(6, 128, 3)
    x[0, 5], x[1, 40], x[2, 100], x[3, 0] = math.nan, math.inf, -math.inf, 3.38e38
    for layout in ("rows", "blocked"):
        codes, scales = ck.ck_mx4_act_quant(x, group=1, layout=layout)
        v = ck.ck_mx4_dequant(codes, scales, rows=6, k=128)
        bad = torch.isnan(v).view(6, 4, 32)
        want = torch.zeros(6, 4, dtype=torch.bool, device=DEV)
        want[0, 0] = want[1, 1] = want[2, 3] = True
        assert torch.equal(bad.all(-1), want) and torch.equal(bad.any(-1), want)
        # through the product: the row, and no other
        if layout == "blocked":
            y = ck.ck_mx4_gemm_bf16(codes, scales, *ck.ck_mx4_weight_prep(torch.randn(48, 128, device=DEV), 1), m=6, n=48)
            # (row 3 holds 2.55e38: times a weight of 1.5 it is past BF16's range, infinite but no NaN)
            assert torch.isnan(y[:3]).all() and not torch.isnan(y[3]).any() and torch.isfinite(y[4:]).all()


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("group", [2, 4, 8, 16, 32, 64, 128, 256])
def test_quantize_rotated(group, act):
    m, k = 37, 1280
    say(f"quantize group {group} {act}")
    x = activation(m, k, group, act)
    a = x.double()
    if act:
        a = a[:, :k] * torch.sigmoid(a[:, :k]) * a[:, k:]
    v = (a.view(m, k // group, group) @ hadamard(group) / math.sqrt(group)).view(m, k // 32, 32)
    size = (a.abs().view(m, k // group, group).sum(-1, keepdim=True) / math.sqrt(group)).expand(m, k // group, group)
    t = ((math.log2(group) + 2) * 2.0 ** -24 + (2.0 ** -21 if act else 0)) * size.reshape(m, k // 32, 32)
    codes, scales = ck.ck_mx4_act_quant(x, act, group, layout="rows")
    top, slack = v.abs().amax(-1), t.amax(-1)
    lo, hi = (scale_of((top + d * slack).unsqueeze(-1)) for d in (-1, 1))
    s = scales.long()
    assert ((s == lo) | (s == hi)).all()
    unit = torch.exp2(s.double() - 127).unsqueeze(-1)
    got = values(codes, scales).view_as(v)
    near = torch.minimum((got - rounded(v - t, unit)).abs(), (got - rounded(v + t, unit)).abs())
    assert near.max().item() == 0
    # a weight, through the same rotation
    if act is None:
        w = x.float()
        wc, ws = ck.ck_mx4_weight_prep(w, group, layout="rows")
        assert torch.equal(values(wc, ws), values(codes, scales))


def test_quantize_strided_rows_and_k():
    x = activation(40, 512, 9)
    want = ck.ck_mx4_act_quant(x[:, 128:384].contiguous(), group=64, layout="rows")
    for got in (ck.ck_mx4_act_quant(x[:, 128:384], group=64, layout="rows"),
                ck.ck_mx4_act_quant(x[:, 128:], group=64, k=256, layout="rows")):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_dequantize_every_code():
    scales = torch.arange(256, device=DEV).to(torch.uint8).repeat_interleave(2).view(256, 2)
    codes = torch.arange(256, device=DEV).to(torch.uint8).roll(3)[:32].expand(256, 32).contiguous()
    codes = codes + torch.arange(256, device=DEV).to(torch.uint8)[:, None]
    want = values(codes, scales)
    top = torch.finfo(BF16).max
    for got in (ck.ck_mx4_dequant(codes, scales), ck.ck_mx4_dequant(*ck.ck_mx4_weight_pack(codes, scales), k=64)):
        got = got.double()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        ok = ~torch.isnan(want) & (want.abs() <= top)
        assert torch.equal(got[ok], want[ok])
        assert torch.isinf(got[~ok & ~torch.isnan(want)]).all()


# ---------------------------------------------------------------- product
def random_operand(rows, k, seed, spread=8):
    codes = torch.randint(0, 256, (rows, k // 2), generator=gen(seed), device=DEV).to(torch.uint8)
    scales = torch.randint(127 - spread, 128 + spread, (rows, k // 32), generator=gen(seed + 1), device=DEV).to(torch.uint8)
    return codes, scales


def check_product(y, xv, wv, bias=None, residual=None, what=""):
    k = xv.shape[1]
    y64, size = xv @ wv.T, xv.abs() @ wv.abs().T
    bound = (128 + k / 64) * 2.0 ** -23 * size
    for extra in (bias, residual):
        if extra is not None:
            bound = bound + 2.0 ** -24 * (y64.abs() + extra.double().abs())
            y64 = y64 + extra.double()
    bound = bound + U * y64.abs()
    off = (y.double() - y64).abs()
    assert torch.isfinite(y).all(), what
    assert (off <= bound * (1 + 2.0 ** -8) + 1e-38).all(), (what, (off / (bound + 1e-38)).max().item())


# every kernel and tile, one or more tiles a workgroup, even and odd shares of k
SIZES = [(1, 16, 64), (1, 12288, 4096), (2, 48, 128), (3, 4096, 12288), (8, 1040, 2112), (15, 80, 320), (16, 4096, 4096),
         (17, 512, 1024), (31, 272, 192), (32, 2048, 12288), (33, 96, 512), (48, 4096, 8192), (63, 1040, 256),
         (64, 64, 32768), (65, 144, 448), (96, 12288, 1024), (128, 128, 12288), (129, 528, 2112), (200, 1024, 8192),
         (256, 256, 256), (257, 272, 64), (333, 1040, 2112), (512, 4096, 512), (1000, 240, 12288), (1024, 1024, 1024),
         (1025, 2064, 576), (2048, 4096, 320), (4096, 4096, 256), (5000, 2992, 448),
         (20, 8208, 512), (6000, 6000, 2112), (6200, 10000, 2304), (9000, 8000, 320), (2500, 2000, 4160),
         (450, 4080, 2816), (500, 4096, 4416), (1000, 4080, 2368), (980, 4096, 1600), (97, 176, 1088), (250, 4000, 4160)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_product(m, n, k):
    say(f"product {m} x {n} x {k}")
    x, w = random_operand(m, k, m + n), random_operand(n, k, n + k + 1)
    xv, wv = values(*x), values(*w)
    xb, wb = blocked(*x), ck.ck_mx4_weight_pack(*w)
    bias = torch.randn(n, generator=gen(1), device=DEV) * 10
    residual = (torch.randn(m, n, generator=gen(2), device=DEV) * 30).to(BF16)
    for b, r in ((None, None), (bias, residual), (bias, None), (None, residual)):
        y = ck.ck_mx4_gemm_bf16(*xb, *wb, m=m, n=n, bias=b, residual=r)
        check_product(y, xv, wv, b, r, (m, n, k, b is not None, r is not None))
        if b is None and r is not None:   # in place, and again: the same bits
            out = residual.clone()
            ck.ck_mx4_gemm_bf16(*xb, *wb, m=m, n=n, residual=out, out=out)
            assert torch.equal(out, y)


def test_product_leaves_padding_and_neighbours_alone():
    """Rows behind the last one, NaN scales in padding rows, and the memory around y."""
    m, n, k = 45, 80, 320
    x, w = random_operand(m, k, 1), random_operand(n, k, 2)
    (xc, xs), wb = blocked(*x), ck.ck_mx4_weight_pack(*w)
    pad = torch.arange(32, device=DEV) >= m - 32
    xs.view(2, -1, 2, 32, 4)[1][:, :, pad] = 255
    buf = torch.full((m * n + 64,), 7.0, dtype=BF16, device=DEV)
    y = buf[32:32 + m * n].view(m, n)
    ck.ck_mx4_gemm_bf16(xc, xs, *wb, m=m, n=n, out=y)
    check_product(y, values(*x), values(*w))
    assert (buf[:32] == 7).all() and (buf[32 + m * n:] == 7).all()


@pytest.mark.parametrize("m", [1, 5, 40, 300])
def test_product_extreme_scales(m):
    """Products of the largest and the smallest scales, and rows that are zero."""
    n, k = 64, 256
    x, w = random_operand(m, k, 11), random_operand(n, k, 12)
    x[1].fill_(254), w[1].fill_(0)
    x[0][0] = 0
    y = ck.ck_mx4_gemm_bf16(*blocked(*x), *ck.ck_mx4_weight_pack(*w), m=m, n=n)
    check_product(y, values(*x), values(*w))
    assert (y[0] == 0).all()


# ---------------------------------------------------------------- linear
@pytest.mark.parametrize("m,n,k,act,group", [
    (1, 12288, 4096, None, 128), (1, 4096, 12288, "swiglu", 128), (1, 48, 64, None, 64), (1, 4096, 320, None, 32),
    (2, 1040, 2112, "swiglu", 64), (2, 512, 8192, None, 256), (2, 512, 32768, None, 1), (3, 528, 1024, None, 1),
    (7, 256, 4096, "swiglu", 16), (16, 4096, 12288, "swiglu", 128), (33, 144, 576, None, 2), (64, 2048, 4096, None, 128),
    (100, 1040, 2112, "swiglu", 64), (333, 1040, 2112, None, 64), (1024, 512, 1280, "swiglu", 256), (2100, 272, 448, None, 32)])
def test_linear(m, n, k, act, group):
    """The linear is the quantizer and then the product."""
    say(f"linear {m} x {n} x {k} {act} {group}")
    x = activation(m, k, m + k, act)
    w = 0.02 * torch.randn(n, k, generator=gen(n), device=DEV)
    wb = ck.ck_mx4_weight_prep(w, group)
    wv = values(*ck.ck_mx4_weight_prep(w, group, layout="rows"))
    xv = values(*ck.ck_mx4_act_quant(x, act, group, layout="rows"))
    bias = torch.randn(n, generator=gen(1), device=DEV)
    residual = torch.randn(m, n, generator=gen(2), device=DEV).to(BF16)
    for b, r in ((None, None), (bias, residual)):
        y = ck.ck_mx4_linear(x, *wb, n=n, group=group, input_act=act, bias=b, residual=r)
        check_product(y, xv, wv, b, r, (b is not None))
        wide = torch.zeros(m, x.shape[1] + 72, dtype=BF16, device=DEV)
        wide[:, 8:8 + x.shape[1]] = x
        assert torch.equal(y, ck.ck_mx4_linear(wide[:, 8:8 + x.shape[1]], *wb, n=n, group=group, input_act=act, bias=b,
                                               residual=r))
        need = ck.lib().ck_mx4_linear_workspace_size(m, k, n)
        ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        out = torch.empty_like(y) if r is None else r.clone()
        ck.ck_mx4_linear(x, *wb, n=n, group=group, input_act=act, bias=b, residual=None if r is None else out, out=out,
                         workspace=ws)
        assert torch.equal(out, y)


@pytest.mark.parametrize("m,act", [(1, None), (2, "swiglu"), (70, None)])
def test_linear_zero_and_not_finite_rows(m, act):
    k, n = 512, 96
    x = activation(m, k, 4, act)
    x[0] = 0
    wb = ck.ck_mx4_weight_prep(torch.randn(n, k, generator=gen(3), device=DEV), 128)
    y = ck.ck_mx4_linear(x, *wb, input_act=act)
    assert (y[0] == 0).all() and (m == 1 or (y[1:] != 0).any(1).all())
    x[0, 3] = math.nan
    y = ck.ck_mx4_linear(x, *wb, input_act=act)
    assert torch.isnan(y[0]).all() and torch.isfinite(y[1:]).all()


def test_linear_against_the_unquantized_weight():
    """4-bit values with 3 significant bits, a scale for 32: about 11% off a product with unquantized operands, for near-
    normal operands; the rotation keeps outlier channels within the same class."""
    m, k, n = 256, 4096, 512
    x, w = activation(m, k, 8), torch.randn(n, k, generator=gen(9), device=DEV)
    want = x.double() @ w.double().T
    y = ck.ck_mx4_linear(x, *ck.ck_mx4_weight_prep(w, 128))
    rel = ((y.double() - want).norm() / want.norm()).item()
    say(f"relative L2 {rel:.4f}")
    # one operand: a relative step of 2^-1 to 2^-2 of the value, uniform error: at most (1/4) / sqrt(3) = 0.144 each
    assert rel < math.sqrt(2) * 0.25 / math.sqrt(3)


def test_linear_empty():
    wb = ck.ck_mx4_weight_prep(torch.randn(64, 128, device=DEV), 64)
    assert ck.ck_mx4_linear(torch.empty(0, 128, dtype=BF16, device=DEV), *wb, group=64).shape == (0, 64)
    codes, scales = ck.ck_mx4_act_quant(torch.empty(0, 128, dtype=BF16, device=DEV), group=64)
    assert codes.shape == (0, 4, 1024) and ck.ck_mx4_dequant(codes, scales, rows=0, k=128).shape == (0, 128)
    w0 = ck.ck_mx4_weight_prep(torch.empty(0, 128, device=DEV), 64)
    assert ck.ck_mx4_linear(torch.ones(3, 128, dtype=BF16, device=DEV), *w0, group=64).shape == (3, 0)


def test_codes_past_32_bit_offsets():
    """Operands and outputs whose offsets pass 2^31 and 2^32 bytes."""
    m, k = 139_000, 16384          # x: 4.6 GB, codes: 1.1 GB; y: 139000 x 8192 BF16, 2.3 GB
    x = torch.zeros(m, k, dtype=BF16, device=DEV)
    rows = [0, 65535, 65536, 131071, 131072, m - 1]
    x[rows] = activation(len(rows), k, 21)
    wb = ck.ck_mx4_weight_prep(0.02 * torch.randn(8192, k, generator=gen(22), device=DEV), 128)
    want = ck.ck_mx4_linear(x[rows].contiguous(), *wb)
    y = ck.ck_mx4_linear(x, *wb)
    # few rows and many may sum in another order: FP32 sums, then one rounding
    assert ((y[rows].double() - want.double()).abs() <= 2 * U * want.double().abs() + 2.0 ** -12).all()
    y[rows] = 0
    assert not y.any()
    del y
    codes, scales = ck.ck_mx4_act_quant(x)
    v = ck.ck_mx4_dequant(codes, scales, rows=m, k=k)
    small = ck.ck_mx4_act_quant(x[rows].contiguous(), layout="rows")
    assert torch.equal(v[rows].double(), values(*small))


# ---------------------------------------------------------------- streams, graphs, refusals
def test_same_bits_every_time_on_a_stream_and_in_a_graph():
    cases = []
    for m, n, k, act in ((1, 512, 1024, None), (2, 512, 1024, "swiglu"), (16, 512, 8192, None), (96, 256, 8192, None),
                         (300, 512, 1024, "swiglu"), (2048, 2048, 512, None)):
        x = activation(m, k, m, act)
        wb = ck.ck_mx4_weight_prep(torch.randn(n, k, generator=gen(n + k), device=DEV), 128)
        cases.append((x, wb, act, torch.empty(m, n, dtype=BF16, device=DEV)))

    def step():
        for x, wb, act, y in cases:
            ck.ck_mx4_linear(x, *wb, input_act=act, out=y)

    step()
    want = [c[3].clone() for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c[3], w)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            step()
    for i in range(4):
        for c in cases:
            c[3].fill_(i)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert torch.equal(c[3], w)
        eager = ck.ck_mx4_linear(cases[4][0], *cases[4][1], input_act=cases[4][2])
        assert torch.equal(eager, want[4])


def test_refusals():
    x = activation(4, 256, 1)
    wb = ck.ck_mx4_weight_prep(torch.randn(48, 256, device=DEV), 64)
    codes, scales = ck.ck_mx4_act_quant(x, group=64)
    rc, rs = ck.ck_mx4_act_quant(x, group=64, layout="rows")

    def no(f, *a, **kw):
        with pytest.raises(ValueError):
            f(*a, **kw)

    q, wp = ck.ck_mx4_act_quant, ck.ck_mx4_weight_prep
    no(q, x.float()), no(q, x.cpu()), no(q, x[0]), no(q, x, group=3), no(q, x, group=512), no(q, x[:, :200])
    no(q, x, k=512), no(q, x, "gelu"), no(q, x.t()), no(q, x[:, 4:]), no(q, x, layout="decode"), no(q, x[:, :64], group=128)
    no(q, x, "swiglu", k=256)
    no(wp, x), no(wp, torch.randn(4, 256, device=DEV)[:, :128]), no(wp, torch.randn(4, 100, device=DEV), 1)
    pk = ck.ck_mx4_weight_pack
    no(pk, rc, rs[:, :4]), no(pk, rc.int(), rs), no(pk, rc[:, :16], rs[:, :1]), no(pk, codes, scales), no(pk, rc.cpu(), rs)
    d = ck.ck_mx4_dequant
    no(d, rc, scales), no(d, codes, rs), no(d, codes, scales, rows=40), no(d, codes, scales, k=512), no(d, rc, rs, rows=3)
    no(d, codes, scales, k=0), no(d, codes, scales, rows=-1)
    g = ck.ck_mx4_gemm_bf16
    no(g, codes, scales, *wb, m=33), no(g, codes, scales, *wb, m=-1), no(g, codes, scales, *wb, m=4, n=40)
    no(g, codes, scales, *wb, m=4, n=96), no(g, rc, rs, *wb, m=4), no(g, codes, wb[1], *wb, m=4)
    no(g, codes, scales, *wp(torch.randn(48, 512, device=DEV), 64), m=4)
    lin = ck.ck_mx4_linear
    no(lin, x.float(), *wb), no(lin, x, *wb, group=0), no(lin, x, *wb, n=40), no(lin, x, wb[0], wb[0])
    no(lin, x[:, :128], *wp(torch.randn(48, 512, device=DEV), 64), group=64), no(lin, x, *wb, bias=torch.zeros(48, device=DEV))
    no(lin, x, *wb, bias=torch.zeros(64, device=DEV).to(BF16)), no(lin, x, *wb, residual=torch.zeros(4, 48, dtype=BF16, device=DEV))
    no(lin, x, *wb, out=torch.zeros(4, 64, device=DEV)), 
    wide = activation(40, 4096, 1)
    w4 = ck.ck_mx4_weight_prep(torch.randn(48, 4096, device=DEV), 64)
    no(lin, wide, *w4, group=64, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    no(lin, x.cpu(), *wb), no(lin, x, wb[0].cpu(), wb[1]), no(lin, x, *wb, input_act="relu")


def test_refusals_of_shared_memory():
    k, n, m = 256, 64, 72           # (too many rows for one kernel without a workspace)
    need = ck.lib().ck_mx4_linear_workspace_size(m, k, n)
    buf = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)

    def part(at, dtype, *shape):
        size = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
        return buf[at:at + size].view(dtype).view(*shape)

    x, y = part(1 << 19, BF16, m, k), part(1 << 14, BF16, m, n)
    wc, ws = part(1 << 15, torch.uint8, 2, 4, 1024), part(1 << 16, torch.uint8, 2, 1, 256)
    room, bias = buf[1 << 18:(1 << 18) + need], part(1 << 17, torch.float32, n)
    kw = dict(group=64, bias=bias)
    ck.ck_mx4_linear(x, wc, ws, out=y, workspace=room, **kw)
    for bad in ({"out": part((1 << 19) + m * k * 2 - 16, BF16, m, n)}, {"out": part((1 << 15) - 16, BF16, m, n)},
                {"out": part((1 << 16) + 256, BF16, m, n)}, {"out": part(1 << 17, BF16, m, n)},
                {"residual": part((1 << 14) + 16, BF16, m, n), "out": y}, {"workspace": buf[(1 << 19) - 256:(1 << 19) - 256 + need]},
                {"workspace": buf[1 << 14:(1 << 14) + need], "out": y}, {"workspace": buf[(1 << 18) + 16:(1 << 18) + 16 + need]},
                {"workspace": buf[1 << 17:(1 << 17) + need]}):
        with pytest.raises(ValueError):
            ck.ck_mx4_linear(x, wc, ws, **{**kw, **bad})


# ---------------------------------------------------------------- padding
def fill_free_memory(byte):
    """What the allocator hands out next holds `byte`."""
    del [torch.full((1 << i,), byte, dtype=torch.uint8, device=DEV) for i in range(9, 25) for _ in range(4)][:]


@pytest.mark.parametrize("n,k,group", [(16, 64, 1), (48, 320, 64), (48, 256, 256), (80, 4096, 128), (272, 576, 2)])
def test_weight_padding_is_zero(n, k, group):
    """Quantized here or packed, a weight is the same bytes, and the features that it pads to are zero."""
    w = torch.randn(n, k, generator=gen(n), device=DEV)
    rows = ck.ck_mx4_weight_prep(w, group, layout="rows")
    x = activation(40, k, 5)
    want = ck.ck_mx4_linear(x, *ck.ck_mx4_weight_pack(*rows), n=n, group=group)
    for byte in (255, 0x7f):
        fill_free_memory(byte)
        wb = ck.ck_mx4_weight_prep(w, group)
        assert all(torch.equal(a, b) for a, b in zip(wb, blocked(*rows)))
        for m in (1, 40):
            y = ck.ck_mx4_linear(x[:m], *wb, group=group)
            assert y.shape == (m, (n + 31) // 32 * 32) and torch.equal(y[:, :n], want[:m]) and not y[:, n:].any()
        xb = ck.ck_mx4_act_quant(x, group=group)
        y = ck.ck_mx4_gemm_bf16(*xb, *wb, m=40)
        assert torch.equal(y[:, :n], want) and not y[:, n:].any()
        v = ck.ck_mx4_dequant(*wb)
        assert torch.equal(v[:n, :k].double(), values(*rows)) and not v[n:].any() and not v[:, k:].any()


@pytest.mark.parametrize("m", [0, 1, 16, 17, 32, 45])
@pytest.mark.parametrize("k,group,act", [(64, 1, None), (320, 64, None), (832, 64, "swiglu"), (4096, 128, "swiglu")])
def test_activation_padding_is_zero(m, k, group, act):
    x = activation(m, k, 6, act)
    rows = ck.ck_mx4_act_quant(x, act, group, layout="rows")
    fill_free_memory(255)
    xb = ck.ck_mx4_act_quant(x, act, group)
    if m:   # (the definition above reshapes no empty tensor)
        assert all(torch.equal(a, b) for a, b in zip(xb, blocked(*rows)))
    v = ck.ck_mx4_dequant(*xb)
    want = values(*rows) if m else v[:0, :k].double()
    assert torch.equal(v[:m, :k].double(), want) and not v[m:].any() and not v[:, k:].any()


def test_in_features_that_pad_to_the_same_width():
    """A blocked weight is padded to 256 values of k, and its codes say how many they hold."""
    import copy
    import io
    for k, others in ((192, (64, 128, 256)), (256, (64, 192)), (320, (384, 448, 512)), (4096, (4032, 3904))):
        rows = ck.ck_mx4_weight_prep(torch.randn(48, k, generator=gen(k), device=DEV), 64, layout="rows")
        prepared = ck.ck_mx4_weight_prep(torch.randn(48, k, generator=gen(k), device=DEV), 64)
        for wb in (prepared, ck.ck_mx4_weight_pack(*rows)):
            for act in (None, "swiglu"):
                for m in (1, 40):
                    y = ck.ck_mx4_linear(activation(m, k, 3, act), *wb, n=48, group=64, input_act=act)
                    assert torch.equal(y, ck.ck_mx4_linear(activation(m, k, 3, act), *wb, n=48, group=64, input_act=act, k=k))
                    for other in others:
                        x = activation(m, other, 3, act)
                        with pytest.raises(ValueError):
                            ck.ck_mx4_linear(x, *wb, n=48, group=64, input_act=act)
                        with pytest.raises(ValueError):
                            ck.ck_mx4_linear(x, *wb, n=48, group=64, input_act=act, k=other)
            for other in others:
                xb = ck.ck_mx4_act_quant(activation(40, other, 3), group=64)
                with pytest.raises(ValueError):
                    ck.ck_mx4_gemm_bf16(*xb, *wb, m=40, n=48)
            # copies that know it still, and ones that have to be told
            buf = io.BytesIO()
            torch.save(wb, buf)
            buf.seek(0)
            for again in (copy.deepcopy(wb), torch.load(buf, weights_only=True)):
                with pytest.raises(ValueError):
                    ck.ck_mx4_linear(activation(2, others[0], 3), *again, n=48, group=64)
            bare = [t.clone() for t in wb]
            x = activation(40, k, 3)
            assert torch.equal(ck.ck_mx4_linear(x, *bare, n=48, group=64, k=k), ck.ck_mx4_linear(x, *wb, n=48, group=64))
            for other in others:
                with pytest.raises(ValueError):
                    ck.ck_mx4_linear(activation(40, other, 3), *bare, n=48, group=64, k=k)
    with pytest.raises(ValueError):
        ck.ck_mx4_linear(x, *bare, n=48, group=64, k=4096.0)


# the quantizer in the product's launch: every row count that a workgroup's 512 blocks of 32 allow, rows whose blocks are
# no multiple of 8, both tile widths with and without SwiGLU, and the first sizes past the limit
@pytest.mark.parametrize("m,n,k,act,group", [
    (1, 8208, 2112, "swiglu", 64), (1, 8192, 16384, None, 128), (4, 8192, 4096, "swiglu", 256), (16, 528, 1024, None, 256),
    (16, 144, 1024, "swiglu", 128), (16, 8240, 64, None, 64), (9, 80, 320, None, 64), (5, 48, 2112, "swiglu", 32),
    (13, 96, 1088, None, 1), (12, 64, 1280, "swiglu", 256), (17, 80, 64, None, 64), (16, 96, 1088, "swiglu", 64),
    (2, 48, 8256, None, 64), (1, 8224, 16448, None, 64)])
def test_linear_in_one_launch(m, n, k, act, group):
    one = m <= 16 and m * ((k + 255) // 256 * 256) <= 16384
    assert (ck.lib().ck_mx4_linear_workspace_size(m, k, n) == 0) == one
    test_linear(m, n, k, act, group)


def test_swiglu_gates():
    """silu(gate) up without a rotation, gates from -87 to 40 in order, so that a block's are of one size.  In units of
    2^-24 of the value: the exponential 2, the sum 1, the reciprocal 2, the two products 1 each, and in the exponent log2(e)
    as a float 0.23 and the product with it 1, each times |gate|, which reach the value by the share e^-g / (1 + e^-g), at
    most 1 for a negative gate and 0.28 / |gate| for a positive one: (8 + 1.25 max(-gate, 0)) 2^-24."""
    m, k = 48, 4096
    g = torch.linspace(-87, 40, m * k, device=DEV).view(m, k).to(BF16)
    u = torch.randn(m, k, generator=gen(31), device=DEV).to(BF16)
    u = torch.where(u == 0, 1.0, u)
    v = (g.double() * torch.sigmoid(g.double()) * u.double()).view(m, k // 32, 32)
    t = (8 + 1.25 * (-g.double()).clamp(min=0)).view_as(v) * 2.0 ** -24 * v.abs()
    codes, scales = ck.ck_mx4_act_quant(torch.cat([g, u], 1), "swiglu", 1, layout="rows")
    s = scales.long()
    lo, hi = (scale_of((v.abs() + d * t).amax(-1, keepdim=True)) for d in (-1, 1))
    assert ((s == lo) | (s == hi)).all()
    unit = torch.exp2(s.double() - 127).unsqueeze(-1)
    got = values(codes, scales).view_as(v)
    assert torch.minimum((got - rounded(v - t, unit)).abs(), (got - rounded(v + t, unit)).abs()).max().item() == 0


@pytest.mark.parametrize("m,n,k,act", [(1024, 1024, 1024, None), (4100, 4112, 512, "swiglu"), (530, 4096, 1088, None)])
def test_linear_whatever_the_memory_held(m, n, k, act):
    """The same bits from workspaces and outputs that held anything, several tiles a workgroup among them."""
    x = activation(m, k, 8, act)
    wb = ck.ck_mx4_weight_prep(torch.randn(n, k, generator=gen(9), device=DEV), 64)
    room = torch.empty(ck.lib().ck_mx4_linear_workspace_size(m, k, n), dtype=torch.uint8, device=DEV)
    out = torch.empty(m, n, dtype=BF16, device=DEV)
    want = None
    for byte in (0, 255, 0x7f, 0x80, 1):
        room.fill_(byte)
        out.view(torch.uint8).fill_(byte)
        ck.ck_mx4_linear(x, *wb, n=n, group=64, input_act=act, out=out, workspace=room)
        want = out.clone() if want is None else want
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
