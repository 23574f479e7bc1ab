"""C ABI checks of the attention-side calls that need no GPU: bad arguments are
refused on the host with the documented status, nothing is enqueued."""
import ctypes
import math

import pytest

import swiglu_mlp_amd as ck

OK, EINVAL, ESHAPE, EUNSUP, EWS = 0, 1, 2, 3, 4
FAKE = 1 << 20          # an aligned non-null address that is never dereferenced


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("sb", ctypes.c_int64), ("st", ctypes.c_int64), ("sh", ctypes.c_int64)]


class Side(ctypes.Structure):
    _fields_ = [("x", Heads), ("y", Heads), ("batch", ctypes.c_int64), ("tokens", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("weight", ctypes.c_void_p), ("cos", ctypes.c_void_p),
                ("sin", ctypes.c_void_p), ("table", ctypes.c_int64), ("pos", ctypes.c_void_p), ("pos_st", ctypes.c_int64)]


@pytest.fixture(scope="module")
def L():
    return ck.lib()


def heads(data=FAKE, sb=4096, st=512, sh=64):
    return Heads(data, sb, st, sh)


def side(batch=0, tokens=4, n=2, **kw):
    """An empty side by default: every check before the launch, no launch."""
    s = Side(heads(), heads(), batch, tokens, n, FAKE, FAKE, FAKE, 16, None, 0)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def norm(L, q, k=None, d=64, rot=64, pairing=0, dtype=0, eps=1e-6):
    return L.ck_qk_norm_rope(ctypes.byref(q) if q is not None else None, ctypes.byref(k) if k is not None else None,
                             d, rot, pairing, dtype, eps, None)


def test_norm_checks(L):
    assert norm(L, side()) == OK and norm(L, side(), side()) == OK
    assert norm(L, None) == EINVAL
    for kw, want in (({"pairing": 2}, EINVAL), ({"dtype": 2}, EINVAL), ({"dtype": -1}, EINVAL), ({"eps": 0.0}, EINVAL),
                     ({"eps": math.nan}, EINVAL), ({"eps": math.inf}, EINVAL), ({"eps": -1.0}, EINVAL),
                     ({"d": 0}, ESHAPE), ({"d": 12}, ESHAPE), ({"d": 264, "rot": 0}, EUNSUP), ({"rot": -16}, ESHAPE),
                     ({"rot": 80}, ESHAPE), ({"rot": 24}, ESHAPE), ({"rot": 20, "pairing": 1}, ESHAPE),
                     ({"rot": 24, "pairing": 1}, OK)):
        assert norm(L, side(), **kw) == want, kw
    # an empty side is skipped, its pointers unread
    assert norm(L, side(x=heads(None), y=heads(None), weight=None, cos=None)) == OK
    # from here on a bad key side next to an empty query side
    for kw, want in (({"batch": -1}, ESHAPE), ({"tokens": -1}, ESHAPE), ({"heads": -1}, ESHAPE),
                     ({"tokens": 1 << 24, "table": 1 << 24}, EUNSUP), ({"batch": 1 << 33, "tokens": 1 << 33}, EUNSUP),
                     ({"x": heads(None)}, EINVAL), ({"x": heads(FAKE + 8)}, EINVAL), ({"y": heads(None)}, EINVAL),
                     ({"x": heads(st=516)}, ESHAPE), ({"x": heads(sh=-64)}, ESHAPE), ({"x": heads(st=1 << 23)}, ESHAPE),
                     ({"y": heads(sb=1 << 40)}, ESHAPE), ({"weight": FAKE + 4}, EINVAL), ({"cos": None}, EINVAL),
                     ({"sin": FAKE + 4}, EINVAL), ({"table": 0}, ESHAPE), ({"table": 3}, ESHAPE),
                     ({"pos": FAKE + 2}, EINVAL), ({"pos": FAKE, "pos_st": -1}, ESHAPE)):
        assert norm(L, side(), side(**{"batch": 1, **kw})) == want, kw


def test_extension_loads_and_refuses_cpu_tensors():
    import torch
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    for bad in (q, None, 3, [q]):
        with pytest.raises(ValueError):
            ck.ck_qk_norm_rope(bad)
        with pytest.raises(ValueError):
            ck.ck_cross_attn(bad, q, q)
    with pytest.raises(ValueError):
        ck.ck_qk_norm_rope(q, pairing="pairs")
    with pytest.raises(ValueError):
        ck.ck_qk_norm_rope(q, q_rope=q)


def attn(L, q=None, k=None, v=None, o=None, batch=2, kv_batch=2, tq=0, tk=8, h=4, kh=2, d=64, dtype=0, scale=0.125,
         kv_len=None, mask=None, mask_st=0, ws=None, ws_n=0):
    r = [ctypes.byref(x or heads()) for x in (q, k, v, o)]
    return L.ck_cross_attn(*r, batch, kv_batch, tq, tk, h, kh, d, dtype, scale, kv_len, mask, mask_st, ws, ws_n, None)


def test_attention_checks(L):
    assert attn(L) == OK                      # no query: nothing is launched
    for kw, want in (({"dtype": 3}, EINVAL), ({"scale": 0.0}, EINVAL), ({"scale": -1.0}, EINVAL),
                     ({"scale": math.nan}, EINVAL), ({"scale": math.inf}, EINVAL), ({"d": 4}, ESHAPE), ({"d": 68}, ESHAPE),
                     ({"d": 136}, EUNSUP), ({"tq": -1}, ESHAPE), ({"tk": -1}, ESHAPE), ({"batch": -2}, ESHAPE)):
        assert attn(L, **kw) == want, kw
    one = {"tq": 1}
    for kw, want in (({"kv_batch": 0}, ESHAPE), ({"batch": 3}, ESHAPE), ({"h": 3}, ESHAPE), ({"kh": 0}, ESHAPE),
                     ({"tk": 1 << 31}, EUNSUP), ({"tq": 1 << 27}, EUNSUP), ({"batch": 1 << 21, "kv_batch": 1 << 21}, EUNSUP), ({"q": heads(None)}, EINVAL),
                     ({"k": heads(FAKE + 2)}, EINVAL), ({"v": heads(st=12)}, ESHAPE), ({"o": heads(sh=4)}, ESHAPE),
                     ({"kv_len": FAKE + 1}, EINVAL), ({"mask": FAKE, "mask_st": -1}, ESHAPE)):
        assert attn(L, **{**one, **kw}) == want, kw


def test_attention_workspace(L):
    size = L.ck_cross_attn_workspace_size
    assert size(2, 2, 0, 8, 4, 2, 64) == 0 and size(2, 2, 1, 0, 4, 2, 64) == 0 and size(2, 3, 1, 8, 4, 2, 64) == 0
    # a long row of one key head is split, each split holding d + 2 floats a row
    n = size(1, 1, 1, 100_000, 1, 1, 64)
    assert n > 0 and n % 256 == 0 and n >= 2 * 66 * 4
    assert size(2, 2, 4096, 512, 24, 24, 128) == 0          # enough row tiles: no split
    for ws, ws_n in ((None, n), (FAKE, n - 1), (FAKE + 16, n)):
        assert attn(L, batch=1, kv_batch=1, tq=1, tk=100_000, h=1, kh=1, ws=ws, ws_n=ws_n) == EWS


def test_head_strides_of_long_caches(L):
    # [batch, heads, tokens, d] from 65536 tokens of 128 channels on: a head stride past 2^23.  Accepted ones get as far
    # as the next argument's refusal; nothing is launched
    for sh, want in ((1 << 23, EINVAL), (1 << 30, EINVAL), ((1 << 40) - 8, EINVAL), (1 << 40, ESHAPE), ((1 << 23) + 4, ESHAPE)):
        h = heads(sh=sh)
        for bad in ({"x": h}, {"y": h}):
            assert norm(L, side(), side(batch=1, weight=FAKE + 4, **bad)) == want, sh
        for name in "qkvo":
            assert attn(L, tq=1, kv_len=FAKE + 1, **{name: h}) == want, (name, sh)
