"""The attention-side operators (ck_qk_norm_rope, ck_cross_attn) against their
formulas in 64 bits.

Bounds, u being the largest relative error of a rounding to the 16-bit type
(2^-8 for BF16's 8 significant bits, 2^-11 for FP16's 11):
  norm   one rounding of the output, u |y|; the FP32 steps before it (a sum of
         d squares, a reciprocal root and at most 5 products and sums) add less
         than (d + 16) 2^-24 of the pair's size |z_a| + |z_b|; FP16 outputs
         below 2^-14 round to multiples of 2^-24.
  attn   with A = sum p |v| / sum p: p's rounding u A, o's rounding u |o|, an
         FP32 score error of (d + 4) 2^-24 scale sum |q| |k| in the exponent
         (twice: in p and in the sum of p), and 2^-18 A for the exponentials
         and the FP32 sums of up to thousands of terms; FP16 p below 2^-14
         round to multiples of 2^-24 (they are scaled by 2^6): n 2^-31 max |v|.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import swiglu_mlp_amd as ck  # noqa: E402

DEV = "cuda:0"
BF16, FP16 = torch.bfloat16, torch.float16
U = {BF16: 2.0 ** -8, FP16: 2.0 ** -11}
TINY = {BF16: 0.0, FP16: 2.0 ** -25}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def say(msg):
    print(f"[attention] {msg}", flush=True)


# ---------------------------------------------------------------- norm
def norm_ref(x, w, rope, pos, pairing, eps):
    """(y, size) in 64 bits: the values and |z_a| + |z_b| of each one's pair."""
    z = x.double()
    z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + eps)
    if w is not None:
        z = z * w.double()
    if rope is None:
        return z, z.abs()
    cos, sin = (r.double() for r in rope)
    half = cos.shape[1]
    at = torch.arange(x.shape[1], device=DEV).expand(x.shape[:2]) if pos is None else pos.long()
    ok = (at >= 0) & (at < cos.shape[0])
    at = torch.where(ok, at, 0)
    c, s = cos[at].unsqueeze(2), sin[at].unsqueeze(2)
    ia = torch.arange(half, device=DEV) if pairing == "half" else 2 * torch.arange(half, device=DEV)
    ib = ia + half if pairing == "half" else ia + 1
    y, size = z.clone(), z.abs()
    y[..., ia] = z[..., ia] * c - z[..., ib] * s
    y[..., ib] = z[..., ib] * c + z[..., ia] * s
    size[..., ia] = size[..., ib] = z[..., ia].abs() + z[..., ib].abs()
    y[~ok] = math.nan
    return y, size


def check_norm(y, x, w, rope, pos, pairing, eps):
    ref, size = norm_ref(x, w, rope, pos, pairing, eps)
    bound = U[x.dtype] * ref.abs() + (x.shape[-1] + 16) * 2.0 ** -24 * size + TINY[x.dtype]
    nan = ref.isnan()
    assert torch.equal(y.isnan(), nan)
    off = ((y.double() - ref).abs() - bound)[~nan]
    assert off.numel() == 0 or off.max().item() <= 0, f"over the bound by {off.max().item()}"


def tables(rows, rot, g):
    a = torch.rand(rows, rot // 2, generator=g, device=DEV) * 2 * math.pi
    return a.cos(), a.sin()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("b,tq,tk,hq,hkv,d,rot,pairing", [
    (1, 1, 1, 1, 1, 8, 8, "interleaved"),
    (1, 1, 1, 1, 1, 16, 16, "half"),
    (16, 1, 1, 32, 8, 128, 128, "half"),
    (2, 3, 5, 7, 2, 64, 64, "half"),
    (2, 33, 7, 5, 5, 64, 32, "half"),
    (3, 17, 18, 3, 1, 72, 64, "half"),
    (3, 17, 18, 3, 1, 72, 72, "interleaved"),
    (1, 129, 65, 14, 2, 80, 80, "half"),
    (2, 31, 1, 9, 9, 96, 48, "half"),
    (2, 31, 1, 9, 9, 104, 40, "interleaved"),
    (1, 500, 300, 24, 24, 128, 128, "interleaved"),
    (4, 700, 700, 32, 8, 128, 64, "half"),
    (1, 9, 4, 3, 2, 136, 128, "half"),
    (2, 65, 64, 5, 1, 256, 256, "half"),
    (2, 65, 64, 5, 1, 256, 128, "interleaved"),
    (1, 40, 40, 2, 2, 128, 0, "half"),
])
def test_norm_values(b, tq, tk, hq, hkv, d, rot, pairing, dtype):
    say(f"norm b={b} tq={tq} tk={tk} hq={hq} hkv={hkv} d={d} rot={rot} {pairing} {dtype}")
    g = gen(1)
    q = (3 * torch.randn(b, tq, hq, d, generator=g, device=DEV)).to(dtype)
    kv = torch.randn(b, tk, 2 * hkv, d, generator=g, device=DEV).to(dtype)
    k = kv[:, :, :hkv]
    qw, kw = (1 + 0.3 * torch.randn(d, generator=g, device=DEV) for _ in range(2))
    rope = tables(max(tq, tk), rot, g) if rot else None
    for qweight, kweight, qr, kr in ((qw, kw, rope, rope), (None, kw, None, rope), (qw, None, rope, None)):
        y, z = ck.ck_qk_norm_rope(q, k, qweight, kweight, q_rope=qr, k_rope=kr, pairing=pairing, eps=1e-5)
        check_norm(y, q, qweight, qr, None, pairing, 1e-5)
        check_norm(z, k, kweight, kr, None, pairing, 1e-5)
    y = ck.ck_qk_norm_rope(q, q_weight=qw, q_rope=rope, pairing=pairing)
    check_norm(y, q, qw, rope, None, pairing, 1e-6)


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_norm_positions_and_positions_outside(pairing):
    g = gen(2)
    b, t, h, d = 3, 50, 6, 64
    q = torch.randn(b, t, h, d, generator=g, device=DEV).to(BF16)
    rope = tables(77, d, g)
    pos = torch.randint(0, 77, (b, t + 3), generator=g, device=DEV, dtype=torch.int32)[:, :t]
    pos[0, 0], pos[1, 7], pos[2, 49], pos[2, 48] = -1, 77, 2 ** 31 - 1, -2 ** 31
    y = ck.ck_qk_norm_rope(q, q_rope=rope, q_pos=pos, pairing=pairing)
    check_norm(y, q, None, rope, pos, pairing, 1e-6)
    assert y[1, 7].isnan().all() and y[1, 6].isfinite().all()


def test_norm_in_place_on_packed_rows_and_into_columns():
    g = gen(3)
    b, t, hq, hkv, d = 2, 45, 6, 2, 128
    qkv = torch.randn(b, t, hq + 2 * hkv, d, generator=g, device=DEV).to(BF16)
    was = qkv.clone()
    rope = tables(t, d, g)
    q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv]
    y, z = ck.ck_qk_norm_rope(q, k, q_rope=rope, k_rope=rope, q_out=q, k_out=k)
    assert y is q and z is k
    check_norm(y, was[:, :, :hq], None, rope, None, "half", 1e-6)
    check_norm(z, was[:, :, hq:hq + hkv], None, rope, None, "half", 1e-6)
    assert torch.equal(qkv[:, :, hq + hkv:], was[:, :, hq + hkv:])
    # k into the columns that held v, q elsewhere
    y, z = ck.ck_qk_norm_rope(was[:, :, :hq], was[:, :, hq:hq + hkv], q_rope=rope, k_rope=rope,
                              k_out=was[:, :, hq + hkv:])
    assert torch.equal(z, qkv[:, :, hq:hq + hkv]) and torch.equal(y, qkv[:, :, :hq])


def apart_views(layout, g):
    """(buffer, q, k, v) in one buffer, sharing no element, in the layouts that projections and caches leave them in."""
    hq, hkv, d = 6, 2, 128
    if layout == "one token":              # decode: packed [q | k | v] rows of one token a sequence
        x = torch.randn(16, 1, hq + 2 * hkv, d, generator=g, device=DEV).to(BF16)
        return x, x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
    if layout == "one sequence, one token":
        x = torch.randn(1, 1, hq + 2 * hkv, d, generator=g, device=DEV).to(BF16)
        return x, x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
    if layout == "one token of many":      # the last token's queries over packed rows of all tokens
        x = torch.randn(3, 9, hq + 2 * hkv, d, generator=g, device=DEV).to(BF16)
        return x, x[:, 8:, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
    if layout == "heads first":            # [batch, q | k | v heads, tokens, d]
        x = torch.randn(3, hq + 2 * hkv, 7, d, generator=g, device=DEV).to(BF16)
        y = x.transpose(1, 2)
        return x, y[:, :, :hq], y[:, :, hq:hq + hkv], y[:, :, hq + hkv:]
    x = torch.randn(3, 5, hkv, 4 + 2, d, generator=g, device=DEV).to(BF16)   # grouped: a key head's q, k and v
    return x, x[:, :, 0, :-2], x[:, :, :, -2], x[:, :, :, -1]


@pytest.mark.parametrize("layout", ["one token", "one sequence, one token", "one token of many", "heads first",
                                    "grouped"])
def test_in_place_and_into_columns_of_one_buffer(layout):
    x, q, k, v = apart_views(layout, gen(14))
    was, was_q, was_k, was_v = apart_views(layout, gen(14))
    rope = tables(9, 128, gen(15))
    y, z = ck.ck_qk_norm_rope(q, k, q_rope=rope, k_rope=rope, q_out=q, k_out=k)
    assert y is q and z is k
    check_norm(y, was_q, None, rope, None, "half", 1e-6)
    check_norm(z, was_k, None, rope, None, "half", 1e-6)
    assert torch.equal(v, was_v)
    # k into v's place, then attention into the queries' own place: the same buffer, nothing of it read and written
    ck.ck_qk_norm_rope(was_q, was_k, q_rope=rope, k_rope=rope, k_out=was_v)
    assert torch.equal(was_v, k)
    queries = q.clone()
    o = ck.ck_cross_attn(queries, k, v, out=q)
    assert o is q
    check_attn(o, queries, k, v)
    # elements in common are refused as before
    for f in (lambda: ck.ck_qk_norm_rope(q, k, k_out=q[:, :k.shape[1], :2]),
              lambda: ck.ck_cross_attn(q, k, v, out=q),
              lambda: ck.ck_cross_attn(v, k, v, out=v)):
        with pytest.raises(ValueError):
            f()


def test_norm_strides_zeros_and_extremes():
    g = gen(4)
    # heads before tokens in memory, a batch-expanded tensor, a zero head and FP16 extremes
    x = torch.randn(1, 5, 33, 64, generator=g, device=DEV).to(FP16)
    x[0, 0, 0] = 0
    x[0, 1, 1] = 65504
    x[0, 2, 2] = 2.0 ** -24
    q = x.transpose(1, 2).expand(3, 33, 5, 64)
    y = ck.ck_qk_norm_rope(q)
    check_norm(y, q, None, None, None, "half", 1e-6)
    assert (y[:, 0, 0] == 0).all()
    b = torch.full((1, 1, 2, 64), 1e-20, device=DEV).to(BF16)   # squares far below eps
    check_norm(ck.ck_qk_norm_rope(b), b, None, None, None, "half", 1e-6)


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [32, 64])
def test_norm_infinities_stay_in_their_pairs(pairing, rot):
    # a head with an infinity has an infinite mean square: its finite channels are 0, the infinite one is NaN, and so is
    # the other channel of its pair if it is turned
    g = gen(24)
    q = torch.randn(1, 70, 3, 64, generator=g, device=DEV).to(BF16)
    for c in range(64):
        q[0, c, 1, c] = math.inf if c % 2 else -math.inf
    q[0, 65, 2, 40] = math.nan
    rope = tables(70, rot, g)
    w = 1 + 0.3 * torch.randn(64, generator=g, device=DEV)
    w[50] = math.inf                               # a weight's infinity stays in its channel
    for weight in (None, w):
        y = ck.ck_qk_norm_rope(q, q_weight=weight, q_rope=rope, pairing=pairing)
        ref, _ = norm_ref(q, weight, rope, None, pairing, 1e-6)
        assert torch.equal(y.isnan(), ref.isnan())
        assert torch.equal(y.isinf(), ref.isinf())
        rest = ref.isfinite()
        assert torch.equal(y[rest] == 0, ref[rest] == 0)


@pytest.mark.parametrize("pairing,dtype", [("half", BF16), ("interleaved", FP16)])
def test_norm_past_the_caches(pairing, dtype):
    # over 256 MiB read and written: the nontemporal form
    g = gen(12)
    qkv = torch.randn(1, 13_500, 40, 128, generator=g, device=DEV).to(dtype)
    rope = tables(13_500, 128, g)
    y, z = ck.ck_qk_norm_rope(qkv[:, :, :35], qkv[:, :, 35:], q_rope=rope, k_rope=rope, pairing=pairing)
    check_norm(y, qkv[:, :, :35], None, rope, None, pairing, 1e-6)
    check_norm(z, qkv[:, :, 35:], None, rope, None, pairing, 1e-6)


def test_norm_empty():
    q = torch.empty(2, 0, 4, 64, dtype=BF16, device=DEV)
    k = torch.randn(2, 3, 4, 64, device=DEV).to(BF16)
    y, z = ck.ck_qk_norm_rope(q, k)
    assert y.shape == q.shape
    check_norm(z, k, None, None, None, "half", 1e-6)


# ---------------------------------------------------------------- attention
def attn_ref(q, k, v, scale, allowed):
    """(o, bound): 64-bit attention with allowed [kv_batch, tk], and how far the
    kernel may be."""
    b, tq, h, d = q.shape
    kb, tk, kh, _ = k.shape
    n, g = b // kb, h // kh
    o = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(o)
    for i in range(b):
        keep = allowed[i // n].nonzero()[:, 0]
        if not len(keep):
            continue
        for j in range(h):
            qq, kk, vv = q[i, :, j].double(), k[i // n, keep, j // g].double(), v[i // n, keep, j // g].double()
            s = scale * (qq @ kk.T.contiguous())
            p = torch.softmax(s, -1)
            o[i, :, j] = p @ vv
            a = p @ vv.abs()
            ds = (d + 4) * 2.0 ** -24 * scale * (qq.abs() @ kk.abs().T.contiguous()).amax(-1, keepdim=True)
            u = U[q.dtype]
            bound[i, :, j] = (1.01 * u + 2 * ds + 2.0 ** -18) * a + 1.01 * u * o[i, :, j].abs() + TINY[q.dtype]
            if q.dtype == FP16:
                bound[i, :, j] += len(keep) * 2.0 ** -31 * vv.abs().max()
    return o, bound


def check_attn(y, q, k, v, scale=None, kv_len=None, key_mask=None):
    kb, tk = k.shape[:2]
    allowed = torch.ones(kb, tk, dtype=torch.bool, device=DEV)
    if kv_len is not None:
        allowed &= torch.arange(tk, device=DEV) < kv_len[:, None]
    if key_mask is not None:
        allowed &= key_mask.bool()
    ref, bound = attn_ref(q, k, v, q.shape[-1] ** -0.5 if scale is None else scale, allowed)
    assert y.isfinite().all()
    off = (y.double() - ref).abs() - bound
    assert off.numel() == 0 or off.max().item() <= 0, f"over the bound by {off.max().item()}"


def make(kb, share, tq, tk, h, kh, d, dtype, seed=5, gain=1.5):
    g = gen(seed)
    q = (gain * torch.randn(kb * share, tq, h, d, generator=g, device=DEV)).to(dtype)
    kv = torch.randn(kb, tk, 2 * kh, d, generator=g, device=DEV)
    kv[:, :, kh:] += 0.5
    kv = kv.to(dtype)
    return q, kv[:, :, :kh], kv[:, :, kh:]


SHAPES = [
    # kv_batch, share, tq, tk, heads, kv_heads, d
    (1, 1, 1, 1, 1, 1, 64),
    (1, 1, 1, 64, 1, 1, 128),
    (2, 1, 1, 65, 4, 2, 128),
    (3, 5, 1, 150, 4, 4, 64),
    (2, 1, 1, 2048, 32, 8, 128),
    (1, 4, 1, 3000, 16, 2, 80),
    (1, 1, 1, 9000, 4, 1, 128),
    (2, 1, 7, 1, 3, 1, 128),
    (1, 1, 31, 63, 2, 2, 8),
    (1, 1, 32, 127, 2, 2, 96),
    (1, 2, 33, 129, 6, 3, 72),
    (2, 1, 64, 2000, 4, 4, 64),
    (2, 1, 127, 64, 2, 1, 104),
    (2, 1, 129, 77, 3, 3, 128),
    (1, 1, 257, 333, 5, 5, 112),
    (1, 3, 100, 640, 8, 2, 88),
    (2, 1, 1000, 512, 6, 6, 128),
    (1, 1, 2049, 191, 24, 24, 128),
    (1, 1, 4100, 1100, 8, 8, 64),
    (600, 1, 1, 5, 4, 2, 64),
    (90, 1, 130, 3, 4, 4, 128),
]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("kb,share,tq,tk,h,kh,d", SHAPES)
def test_attn_values(kb, share, tq, tk, h, kh, d, dtype):
    say(f"attn kb={kb} share={share} tq={tq} tk={tk} h={h} kh={kh} d={d} {dtype}")
    q, k, v = make(kb, share, tq, tk, h, kh, d, dtype)
    check_attn(ck.ck_cross_attn(q, k, v), q, k, v)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("kb,share,tq,tk,h,kh,d", [
    (5, 1, 1, 300, 8, 2, 128),
    (5, 2, 1, 1500, 4, 4, 64),
    (4, 1, 40, 200, 3, 3, 96),
    (5, 1, 200, 517, 6, 2, 80),
    (3, 1, 600, 320, 4, 4, 128),
])
def test_attn_lengths_and_masks(kb, share, tq, tk, h, kh, d, dtype):
    say(f"attn masks kb={kb} share={share} tq={tq} tk={tk} h={h} kh={kh} d={d} {dtype}")
    q, k, v = make(kb, share, tq, tk, h, kh, d, dtype)
    g = gen(6)
    lens = torch.tensor([0, 1, 64, tk, tk + 9][:kb], dtype=torch.int32, device=DEV)
    lens[0] = 0 if kb > 3 else -5                                  # taken as none
    mask = torch.rand(kb, tk + 5, generator=g, device=DEV)[:, :tk] < 0.6
    mask[-1] = False
    mask[-1, tk - 1] = True                                        # one key only, the last
    y = ck.ck_cross_attn(q, k, v, kv_len=lens)
    check_attn(y, q, k, v, kv_len=lens)
    assert (y[:share] == 0).all()
    check_attn(ck.ck_cross_attn(q, k, v, key_mask=mask), q, k, v, key_mask=mask)
    check_attn(ck.ck_cross_attn(q, k, v, key_mask=mask.to(torch.uint8) * 7), q, k, v, key_mask=mask)
    check_attn(ck.ck_cross_attn(q, k, v, kv_len=lens, key_mask=mask), q, k, v, kv_len=lens, key_mask=mask)
    none = torch.zeros(kb, tk, dtype=torch.bool, device=DEV)
    assert (ck.ck_cross_attn(q, k, v, key_mask=none) == 0).all()
    none[:, 130:135] = True                                        # whole tiles without a key first
    check_attn(ck.ck_cross_attn(q, k, v, key_mask=none), q, k, v, key_mask=none)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("kb,share,tq,tk,h,kh,d", [
    (1, 1, 1000, 2048, 8, 8, 128),
    (2, 1, 300, 1300, 4, 2, 72),
    (1, 2, 300, 3000, 3, 3, 64),
    (1, 1, 200, 5000, 16, 2, 128),
    (1, 1, 515, 20000, 1, 1, 96),
    (5, 1, 180, 1700, 8, 2, 80),
])
def test_attn_many_rows_with_split_keys(kb, share, tq, tk, h, kh, d, dtype):
    # tiles of 128 rows whose keys go to several workgroups: whole, with lengths that end before, in and after a split,
    # and with a mask that leaves the last sequence one key and the splits before it none
    say(f"attn split tiles kb={kb} share={share} tq={tq} tk={tk} h={h} kh={kh} d={d} {dtype}")
    assert share * tq * (h // kh) > 512 and ck.lib().ck_cross_attn_workspace_size(kb * share, kb, tq, tk, h, kh, d) > 0
    q, k, v = make(kb, share, tq, tk, h, kh, d, dtype)
    check_attn(ck.ck_cross_attn(q, k, v), q, k, v)
    lens = torch.tensor([tk // 2 + 1, 0, tk + 3, 100, tk - 1][:kb], dtype=torch.int32, device=DEV)
    mask = torch.rand(kb, tk, generator=gen(21), device=DEV) < 0.6
    mask[-1] = False
    mask[-1, tk - 1 if kb == 1 else 70] = True
    check_attn(ck.ck_cross_attn(q, k, v, kv_len=lens), q, k, v, kv_len=lens)
    check_attn(ck.ck_cross_attn(q, k, v, key_mask=mask), q, k, v, key_mask=mask)
    check_attn(ck.ck_cross_attn(q, k, v, kv_len=lens, key_mask=mask), q, k, v, kv_len=lens, key_mask=mask)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("kb,tq,kh,d", [
    (16, 1, 16, 64),      # slices, two splits of which the first has two lists
    (16, 1, 16, 128),     # slices, one token
    (2, 40, 80, 96),      # slices, two row tiles
    (2, 2100, 8, 64),     # tiles, one key group
    (2, 1600, 8, 128),    # tiles, two key groups
])
def test_attn_masks_over_several_lists(kb, tq, kh, d, dtype):
    # 9001 keys are listed 4096 at a time: every list with keys (odd and even numbers of 32- and 64-key tiles, full
    # and partly filled last ones), lists of few keys, of one, of none, and of all
    tk, g = 9001, gen(22)
    q, k, v = make(kb, 1, tq, tk, kh, kh, d, dtype)
    kept = [(2458, 2459, 500), (64 * 39 - 5, 64 * 20, 3), (33, 4096, 809), (4096, 0, 32), (0, 65, 0), (1, 1, 1), (0, 0, 64)]
    for first in range(0, len(kept), kb):
        mask = torch.zeros(kb, tk, dtype=torch.bool, device=DEV)
        for i in range(kb):
            for j, n in enumerate(kept[(first + i) % len(kept)]):
                size = min(4096, tk - 4096 * j)
                mask[i, 4096 * j + torch.randperm(size, generator=g, device=DEV)[:n]] = True
        check_attn(ck.ck_cross_attn(q, k, v, key_mask=mask), q, k, v, key_mask=mask)
    lens = torch.randint(4000, tk + 1, (kb,), generator=g, device=DEV, dtype=torch.int32)
    check_attn(ck.ck_cross_attn(q, k, v, kv_len=lens, key_mask=mask), q, k, v, kv_len=lens, key_mask=mask)


@pytest.mark.parametrize("tq", [1, 40, 700, 1700])   # slices, tiles of two key groups and of one
def test_keys_far_apart(tq):
    # keys almost 2^23 elements apart: lists of 126 keys at a time, so that a listed key's offset stays in 32 bits
    tk, kh, d, pitch = 600, 20, 64, (1 << 23) - 8
    say(f"keys far apart tq={tq}")
    g = gen(23)
    room = torch.empty(tk * pitch, dtype=BF16, device=DEV)
    k = room.as_strided((1, tk, kh, d), (tk * pitch, pitch, d, 1))
    v = room.as_strided((1, tk, kh, d), (tk * pitch, pitch, d, 1), kh * d)
    was = torch.randn(1, tk, kh, d, generator=g, device=DEV).to(BF16)
    k.copy_(was)
    v.copy_(torch.randn(1, tk, kh, d, generator=g, device=DEV) + 0.5)
    q = torch.randn(1, tq, kh, d, generator=g, device=DEV).to(BF16)
    _, k = ck.ck_qk_norm_rope(q, k, k_out=k)
    check_norm(k, was, None, None, None, "half", 1e-6)
    check_attn(ck.ck_cross_attn(q, k, v), q, k, v)
    mask = torch.rand(1, tk, generator=g, device=DEV) < 0.6
    check_attn(ck.ck_cross_attn(q, k, v, key_mask=mask), q, k, v, key_mask=mask)
    mask[:, 126:300] = False
    check_attn(ck.ck_cross_attn(q, k, v, key_mask=mask), q, k, v, key_mask=mask)


@pytest.mark.parametrize("kb", [2, 15, 16, 17, 70])
@pytest.mark.parametrize("tq", [1, 130])
def test_attn_lengths_in_any_order(kb, tq):
    # the longest sequences are taken first, up to 16 of them; equal lengths, none and all among them
    q, k, v = make(kb, 1, tq, 100, 2, 2, 64, BF16)
    lens = torch.randint(-3, 104, (kb,), generator=gen(13), device=DEV, dtype=torch.int32)
    lens[: kb // 3] = 50
    check_attn(ck.ck_cross_attn(q, k, v, kv_len=lens), q, k, v, kv_len=lens)


@pytest.mark.parametrize("tq,share", [(1, 1), (1, 3), (50, 1), (300, 1)])
def test_attn_nan_and_inf_in_masked_places(tq, share):
    q, k, v = make(2, share, tq, 400, 4, 2, 128, BF16)
    mask = torch.rand(2, 400, generator=gen(7), device=DEV) < 0.5
    lens = torch.tensor([300, 129], dtype=torch.int32, device=DEV)
    want = ck.ck_cross_attn(q, k, v, kv_len=lens, key_mask=mask)
    check_attn(want, q, k, v, kv_len=lens, key_mask=mask)
    out = ~mask | (torch.arange(400, device=DEV) >= lens[:, None])
    for bad in (math.nan, math.inf, -math.inf):
        k2, v2 = k.clone(), v.clone()
        k2[out] = bad
        v2[out] = bad
        assert torch.equal(ck.ck_cross_attn(q, k2, v2, kv_len=lens, key_mask=mask), want)


@pytest.mark.parametrize("tq", [1, 200])
def test_attn_allowed_nan_and_inf_spread_as_the_formula_says(tq):
    q, k, v = make(2, 1, tq, 200, 2, 1, 64, BF16)
    k, v = k.clone(), v.clone()
    k[0, 77, 0, 3] = math.nan
    v[1, 150, 0, 5] = math.inf
    y = ck.ck_cross_attn(q, k, v)
    assert y[0].isnan().all()
    assert (y[1, :, :, 5] == math.inf).all() and y[1, :, :, 6].isfinite().all()
    # every score -inf: the softmax of the formula is 0 / 0
    k[1] = -math.inf
    q2 = q.abs() + 1
    assert ck.ck_cross_attn(q2, k, v)[1].isnan().all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("tq", [1, 40, 300])
def test_attn_growing_scores(tq, dtype):
    # scores that grow along the keys, so the running maximum moves in every
    # tile, with a spread of far over 2^16 in the probabilities
    q, k, v = make(1, 1, tq, 700, 2, 2, 64, dtype)
    q = q.abs()
    k = (torch.arange(700, device=DEV)[None, :, None, None] / 60.0 * torch.ones_like(k) + 0.1 * k.float()).to(dtype)
    check_attn(ck.ck_cross_attn(q, k, v), q, k, v)
    check_attn(ck.ck_cross_attn(q, k.flip(1).contiguous(), v), q, k.flip(1), v)


@pytest.mark.parametrize("dtype,d,tk", [(BF16, 128, 70_000), (FP16, 64, 131_072), (BF16, 80, 120_001)])
def test_attn_past_the_caches(dtype, d, tk):
    # over 256 MiB of keys and values for one row tile: the streamed form
    q, k, v = make(1, 3, 1, tk, 16, 8, d, dtype)
    check_attn(ck.ck_cross_attn(q, k, v), q, k, v)
    q, k, v = make(2, 1, 1, tk, 16, 8, d, dtype)
    lens = torch.tensor([tk - 77, 333], dtype=torch.int32, device=DEV)
    check_attn(ck.ck_cross_attn(q, k, v, kv_len=lens), q, k, v, kv_len=lens)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 2.0])
def test_attn_scale(scale):
    q, k, v = make(1, 1, 70, 130, 2, 2, 64, BF16, gain=0.5)
    check_attn(ck.ck_cross_attn(q, k, v, scale=scale), q, k, v, scale=scale)


@pytest.mark.parametrize("tq", [1, 3, 150])
def test_attn_views_and_out(tq):
    g = gen(8)
    # heads before tokens for q, keys and values as columns of different packed
    # rows, an expanded key batch, and the output into columns of a wider buffer
    q = torch.randn(4, 6, tq, 64, generator=g, device=DEV).to(BF16).transpose(1, 2)
    k = torch.randn(1, 210, 5, 64, generator=g, device=DEV).to(BF16)[:, :, 1:4].expand(2, 210, 3, 64)
    v = torch.randn(2, 3, 210, 72, generator=g, device=DEV).to(BF16)[..., 8:].transpose(1, 2)
    wide = torch.full((4, tq, 9, 64), 7.0, dtype=BF16, device=DEV)
    y = ck.ck_cross_attn(q, k, v, out=wide[:, :, 2:8])
    check_attn(y, q, k, v)
    assert (wide[:, :, :2] == 7).all() and (wide[:, :, 8:] == 7).all()
    assert torch.equal(ck.ck_cross_attn(q, k, v), y)


@pytest.mark.parametrize("tq", [1, 40, 300])
def test_heads_far_apart(tq):
    # [batch, heads, tokens, 128] of 70000 tokens: heads 8.96 million elements apart; the norm in place, then attention
    tk, g = 70_000, gen(20)
    kv = torch.randn(1, 4, tk, 128, generator=g, device=DEV).to(BF16)
    k, v = kv[:, :2].transpose(1, 2), kv[:, 2:].transpose(1, 2)
    was = k.clone()
    q = torch.randn(1, 4, tk, 128, generator=g, device=DEV).to(BF16).transpose(1, 2)[:, :tq]
    _, k = ck.ck_qk_norm_rope(q, k, k_out=k)
    check_norm(k, was, None, None, None, "half", 1e-6)
    o = torch.empty(1, 4, tk, 128, dtype=BF16, device=DEV).transpose(1, 2)[:, :tq]
    check_attn(ck.ck_cross_attn(q, k, v, out=o), q, k, v)


def test_attn_no_keys_no_rows():
    q = torch.randn(2, 3, 4, 64, device=DEV).to(BF16)
    k = torch.empty(2, 0, 2, 64, dtype=BF16, device=DEV)
    assert (ck.ck_cross_attn(q, k, k) == 0).all()
    k = torch.randn(2, 9, 2, 64, device=DEV).to(BF16)
    assert ck.ck_cross_attn(q[:, :0], k, k).shape == (2, 0, 4, 64)
    assert ck.ck_cross_attn(q[:0], k[:0], k[:0]).shape == (0, 3, 4, 64)


@pytest.mark.parametrize("tq", [1, 40, 300])
def test_attn_offsets_past_32_bits(tq):
    # 5 GB keys and 5 GB values; only the last keys are allowed and written
    tk, kh, d = 300_000, 64, 128
    k = torch.empty(1, tk, kh, d, dtype=BF16, device=DEV)
    v = torch.empty(1, tk, kh, d, dtype=BF16, device=DEV)
    g = gen(9)
    k[:, -100:] = torch.randn(1, 100, kh, d, generator=g, device=DEV).to(BF16)
    v[:, -100:] = torch.randn(1, 100, kh, d, generator=g, device=DEV).to(BF16)
    mask = torch.zeros(1, tk, dtype=torch.bool, device=DEV)
    mask[:, -100:] = True
    q = torch.randn(1, tq, kh, d, generator=g, device=DEV).to(BF16)
    y = ck.ck_cross_attn(q, k, v, key_mask=mask)
    check_attn(y, q, k[:, -100:], v[:, -100:])


def test_same_bits_every_time_on_a_stream_and_in_a_graph():
    cases = []
    for shape in ((2, 1, 1, 3000, 8, 2, 128), (1, 1, 300, 400, 4, 4, 64), (2, 2, 20, 2000, 2, 2, 128)):
        q, k, v = make(*shape, BF16)
        rope = tables(shape[2], shape[6], gen(10))
        cases.append((q, k, v, rope, torch.empty_like(q), torch.empty_like(q)))

    def step():
        for q, k, v, rope, n, o in cases:
            ck.ck_qk_norm_rope(q, q_rope=rope, q_out=n)
            ck.ck_cross_attn(n, k, v, out=o)

    step()
    want = [(c[4].clone(), c[5].clone()) for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for c, (n, o) in zip(cases, want):
        assert torch.equal(c[4], n) and torch.equal(c[5], o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for c in cases:
            c[4].fill_(i), c[5].fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        for c, (n, o) in zip(cases, want):
            assert torch.equal(c[4], n) and torch.equal(c[5], o)
        eager = ck.ck_cross_attn(want[0][0], cases[0][1], cases[0][2])
        assert torch.equal(eager, want[0][1])


# ---------------------------------------------------------------- refusals
def test_refusals():
    q = torch.randn(2, 4, 4, 64, device=DEV).to(BF16)
    k = torch.randn(2, 6, 2, 64, device=DEV).to(BF16)
    rope = tables(8, 64, gen(11))
    w = torch.ones(64, device=DEV)

    def no(f, *a, **kw):
        with pytest.raises(ValueError):
            f(*a, **kw)

    n = ck.ck_qk_norm_rope
    no(n, q.float()), no(n, q.cpu()), no(n, q[0]), no(n, q[..., :60]), no(n, q.transpose(2, 3))
    no(n, q, k.to(FP16)), no(n, q, k[..., :32]), no(n, q, q_weight=w[:32]), no(n, q, q_weight=w.to(BF16))
    no(n, q, q_rope=(rope[0][:3], rope[1][:3])), no(n, q, q_rope=rope[0]), no(n, q, pairing="quarter")
    no(n, q, q_rope=(rope[0], rope[1][:, :16])), no(n, q, k_rope=rope)
    no(n, q, q_rope=tables(8, 24, gen(1))), no(n, q, q_rope=tables(8, 80, gen(1)))
    no(n, q, k, q_rope=rope, k_rope=tables(8, 32, gen(1)))
    no(n, q, q_pos=torch.zeros(2, 4, dtype=torch.int32, device=DEV))
    no(n, q, q_rope=rope, q_pos=torch.zeros(2, 4, dtype=torch.int64, device=DEV))
    no(n, q, q_rope=rope, q_pos=torch.zeros(2, 5, dtype=torch.int32, device=DEV))
    no(n, q, q_out=q[:, :, :2]), no(n, q[:, :3], q_out=q[:, 1:]), no(n, q, q_out=torch.empty_like(q).to(FP16))
    no(n, q[:, :, 1:], k, q_out=q[:, :, :3])
    no(n, torch.randn(1, 1, 1, 264, device=DEV).to(BF16))
    no(n, torch.randn(1, 4, 2, 68, device=DEV).to(BF16)[..., 4:])        # not 16-byte aligned
    with pytest.raises(ck.CKError):
        n(q, eps=0.0)
    with pytest.raises(ck.CKError):
        n(q, eps=math.nan)
    c = ck.ck_cross_attn
    no(c, q, k, k[:, :5]), no(c, q, k.to(FP16), k), no(c, q.cpu(), k, k), no(c, q, k[..., :32], k[..., :32])
    no(c, q[:1], k, k), no(c, q[:, :, :3], k, k), no(c, q, k, k, scale=0.0), no(c, q, k, k, scale=math.inf)
    no(c, q, k, k, scale=-1.0), no(c, q, k, k, scale=math.nan)
    no(c, q, k, k, kv_len=torch.zeros(2, device=DEV)), no(c, q, k, k, kv_len=torch.zeros(3, dtype=torch.int32, device=DEV))
    no(c, q, k, k, key_mask=torch.ones(2, 5, dtype=torch.bool, device=DEV))
    no(c, q, k, k, key_mask=torch.ones(2, 6, device=DEV)), no(c, q, k, k, key_mask=torch.ones(2, 6, dtype=torch.bool))
    no(c, q, k, k, out=q), no(c, q, k, k, out=q[:, :, :2])
    big = torch.randn(1, 1, 1, 136, device=DEV).to(BF16)
    no(c, big, big, big)
    need = ck.lib().ck_cross_attn_workspace_size(1, 1, 1, 100_000, 1, 1, 64)
    if need:
        z = torch.zeros(1, 100_000, 1, 64, dtype=BF16, device=DEV)
        no(c, z[:, :1], z, z, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))


def test_refusals_of_shared_memory():
    """Outputs and the workspace share no memory with anything the call reads, the small tensors included."""
    def part(buf, at, dtype, *shape):
        n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
        return buf[at:at + n].view(dtype).view(*shape)

    buf = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    q, out = (part(buf, i << 14, BF16, 2, 4, 4, 64) for i in range(2))
    rope = tuple(part(buf, 1 << 18 | i << 12, torch.float32, 8, 32) for i in range(2))
    w = part(buf, 3 << 18, torch.float32, 64)
    pos = part(buf, 3 << 18 | 1024, torch.int32, 2, 4)
    q.copy_(torch.randn(2, 4, 4, 64, generator=gen(16), device=DEV))
    want = ck.ck_qk_norm_rope(q, q, w, w, q_rope=rope, k_rope=rope, q_pos=pos, k_pos=pos)[0]
    kw = dict(q_weight=w, q_rope=rope, q_pos=pos)
    assert torch.equal(ck.ck_qk_norm_rope(q, q_out=out, **kw), want)   # one buffer, nothing in common
    at = out.data_ptr() - buf.data_ptr()
    clash = [{"q_weight": part(buf, at, torch.float32, 64)}, {"q_weight": part(buf, at + 4096 - 256, torch.float32, 64)},
             {"q_rope": (rope[0], part(buf, at + 16, torch.float32, 8, 32))},
             {"q_rope": (part(buf, at - 16, torch.float32, 8, 32), rope[1])}, {"q_pos": part(buf, at, torch.int32, 2, 4)}]
    for c in clash:
        with pytest.raises(ValueError):
            ck.ck_qk_norm_rope(q, q_out=out, **{**kw, **c})
        for n, t in (("q", out), ("k", out)):   # of either side with either output
            with pytest.raises(ValueError):
                ck.ck_qk_norm_rope(q, q.clone(), **{n + "_out": t}, **{**kw, **{k.replace("q_", "k_"): v for k, v in kw.items()},
                                                                      **{k.replace("q_", "k_"): v for k, v in c.items()}})

    tk = 100_000
    k = torch.randn(1, tk, 1, 64, generator=gen(17), device=DEV).to(BF16)
    need = ck.lib().ck_cross_attn_workspace_size(1, 1, 1, tk, 1, 1, 64)
    assert need > 0
    q = torch.randn(1, 1, 1, 64, generator=gen(18), device=DEV).to(BF16)
    mask = torch.ones(1, tk, dtype=torch.bool, device=DEV)
    lens = torch.full((1,), tk, dtype=torch.int32, device=DEV)
    room = torch.zeros(need + (1 << 18), dtype=torch.uint8, device=DEV)
    ws, rest = room[:need], room[need:]
    out = part(rest, 0, BF16, 1, 1, 1, 64)
    want = ck.ck_cross_attn(q, k, k, kv_len=lens, key_mask=mask)
    assert torch.equal(ck.ck_cross_attn(q, k, k, kv_len=lens, key_mask=mask, out=out, workspace=ws), want)
    for kw in ({"out": part(room, need - 16, BF16, 1, 1, 1, 64), "workspace": ws},
               {"kv_len": part(room, need - 4, torch.int32, 1), "workspace": ws},
               {"key_mask": part(room, need - 1, torch.bool, 1, tk), "workspace": ws},
               {"kv_len": part(rest, 64, torch.int32, 1), "out": out},
               {"key_mask": part(rest, 127, torch.bool, 1, tk), "out": out},
               {"workspace": k.view(torch.uint8).view(-1)[:need]}):
        with pytest.raises(ValueError):
            ck.ck_cross_attn(q, k, k, **kw)
    with pytest.raises(ValueError):
        ck.ck_cross_attn(part(room, 0, BF16, 1, 1, 1, 64), k, k, workspace=ws)
    with pytest.raises(ValueError):      # a key that is no [batch, tokens, heads, d]
        ck.ck_qk_norm_rope(q, k[None], q_out=torch.empty_like(q))


def test_refusals_of_outputs_that_hold_an_element_twice():
    q = torch.randn(2, 4, 4, 64, generator=gen(19), device=DEV).to(BF16)
    buf = torch.empty(1 << 16, dtype=BF16, device=DEV)
    for strides in ((1024, 128, 64, 1), (1024, 256, 32, 1), (64, 256, 64, 1), (256, 256, 64, 1), (0, 256, 64, 1)):
        out = buf.as_strided(q.shape, strides)
        for f in (lambda: ck.ck_qk_norm_rope(q, q_out=out), lambda: ck.ck_qk_norm_rope(q, q, k_out=out),
                  lambda: ck.ck_cross_attn(q, q, q, out=out)):
            with pytest.raises(ValueError):
                f()
    want = ck.ck_cross_attn(q, q, q)
    for strides in ((1024, 256, 64, 1), (256, 512, 64, 1), (2048, 64, 256, 1)):
        assert torch.equal(ck.ck_cross_attn(q, q, q, out=buf.as_strided(q.shape, strides)), want)


# ---------------------------------------------------------------- the block of both
def test_block_of_linears_norms_and_attention():
    """The example block against FP32 with unquantized weights.  Its INT8 linears are of the 1 to 2% class (relative
    L2); four in a row, with residuals that are not quantized, stay under 5%."""
    import os
    import sys
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    from examples import cross_block as cb
    weights, x, context, rope, lens = cb.synthetic(b=3, t=50, s=33, heads=4, d=64, context=256, inner=512)
    lens[0] = 0                                    # a prompt without states: attention adds nothing
    y = cb.CrossBlock(weights, 4)(x, context, rope, lens).float()
    one = lens.clone().clamp(min=1)                # (the reference has no empty softmax)
    want = cb.reference(weights, 4, x, context, rope, one)
    want[0] = cb.reference({**weights, "w_o": 0 * weights["w_o"]}, 4, x[:1], context[:1], rope, one[:1])[0]
    for i in range(3):
        assert ((y[i] - want[i]).norm() / want[i].norm()).item() < 0.05
