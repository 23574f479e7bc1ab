"""C ABI checks of the MX FP4 and block norm calls that need no GPU: bad arguments
are refused on the host with the documented status, nothing is enqueued."""
import ctypes
import math

import pytest

import swiglu_mlp_amd as ck

OK, EINVAL, ESHAPE, EUNSUP, EWS = 0, 1, 2, 3, 4
FAKE = 1 << 20          # an aligned non-null address that is never dereferenced
ROWS, BLOCKED, DECODE = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    return ck.lib()


def test_mx4_sizes(L):
    for r, want in ((-1, 0), (0, 0), (1, 32), (32, 32), (33, 64), ((1 << 30) + 1, (1 << 30) + 32)):
        assert L.ck_mx4_rows(r) == want
    for k, want in ((0, 0), (64, 256), (256, 256), (320, 512)):
        assert L.ck_mx4_cols(k) == want
    size = L.ck_mx4_linear_workspace_size
    for m, k, n in ((0, 256, 64), (4, 256, 0), (-4, 256, 64), (4, 100, 64), (4, 256, 24), (4, 32832, 64), (1 << 40, 256, 64)):
        assert size(m, k, n) == 0
    # codes and scales of 33 rows x 320, padded to 64 x 512
    assert size(33, 320, 64) == 64 * 512 // 2 + 64 * 512 // 32


def quant_cases():
    return (({"k": 100}, ESHAPE), ({"k": 0}, ESHAPE), ({"k": 192, "group": 128}, ESHAPE), ({"group": 3}, EUNSUP),
            ({"group": 512}, EUNSUP), ({"group": 0}, EUNSUP), ({"k": 32832, "group": 1}, EUNSUP), ({"rows": -1}, ESHAPE),
            ({"rows": 1 << 31}, EUNSUP), ({"rows": 1 << 26}, EUNSUP), ({"layout": DECODE}, EINVAL), ({"layout": -1}, EINVAL),
            ({"rows": 0}, OK), ({"src": None}, EINVAL), ({"src": FAKE + 8}, EINVAL), ({"codes": None}, EINVAL),
            ({"codes": FAKE + 8}, EINVAL), ({"scales": None}, EINVAL), ({"scales": FAKE + 4}, EINVAL))


def test_mx4_quantizers(L):
    def prep(src=FAKE, rows=8, k=256, group=64, layout=BLOCKED, codes=FAKE, scales=FAKE):
        return L.ck_mx4_weight_prep(src, rows, k, group, layout, codes, scales, None)

    def act(src=FAKE, rows=8, k=256, group=64, layout=BLOCKED, codes=FAKE, scales=FAKE, ld=None, kind=0):
        return L.ck_mx4_act_quant(src, k if ld is None else ld, rows, k, kind, group, layout, codes, scales, None)

    for kw, want in quant_cases():
        assert prep(**kw) == want, kw
        assert act(**kw) == want, kw
    for kw, want in (({"ld": 192}, ESHAPE), ({"ld": 260}, ESHAPE), ({"kind": 2}, EINVAL), ({"kind": 1}, ESHAPE),
                     ({"kind": 1, "ld": 512, "rows": 0}, OK)):
        assert act(**kw) == want, kw


def test_mx4_pack_and_dequantize(L):
    def pack(c=FAKE, s=FAKE, n=8, k=256, oc=FAKE, os=FAKE):
        return L.ck_mx4_weight_pack(c, s, n, k, oc, os, None)

    def deq(c=FAKE, s=FAKE, n=8, k=256, layout=ROWS, y=FAKE):
        return L.ck_mx4_dequant(c, s, n, k, layout, y, None)

    for f in (pack, deq):
        for kw, want in (({"n": -1}, ESHAPE), ({"n": 0}, OK), ({"k": 32}, ESHAPE), ({"k": 33024}, EUNSUP), ({"n": 1 << 30}, EUNSUP),
                         ({"c": None}, EINVAL), ({"c": FAKE + 4}, EINVAL), ({"s": None}, EINVAL)):
            assert f(**kw) == want, (f.__name__, kw)
    for kw in ({"oc": None}, {"os": None}, {"oc": FAKE + 8}, {"os": FAKE + 8}):
        assert pack(**kw) == EINVAL
    for kw in ({"layout": DECODE}, {"y": None}, {"y": FAKE + 2}):
        assert deq(**kw) == EINVAL


def test_mx4_products(L):
    def gemm(xc=FAKE, xs=FAKE, wc=FAKE, ws=FAKE, bias=None, res=None, m=8, n=64, k=256, y=FAKE):
        return L.ck_mx4_gemm_bf16(xc, xs, wc, ws, bias, res, m, n, k, y, None)

    def lin(x=FAKE, ld=None, act=0, wc=FAKE, ws=FAKE, bias=None, res=None, m=8, n=64, k=256, group=64, y=FAKE, room=FAKE,
            size=1 << 40):
        return L.ck_mx4_linear(x, (k * (1 + act)) if ld is None else ld, act, wc, ws, bias, res, m, n, k, group, y, room, size,
                               None)

    for f in (gemm, lin):
        for kw, want in (({"m": 0}, OK), ({"n": 0}, OK), ({"m": -1}, ESHAPE), ({"n": -16}, ESHAPE), ({"n": 40}, ESHAPE),
                         ({"k": 96}, ESHAPE), ({"k": 33024}, EUNSUP), ({"m": 1 << 31}, EUNSUP), ({"n": 1 << 26}, EUNSUP),
                         ({"m": 1 << 20, "n": 1 << 20}, EUNSUP), ({"wc": None}, EINVAL), ({"wc": FAKE + 8}, EINVAL),
                         ({"ws": None}, EINVAL), ({"ws": FAKE + 8}, EINVAL), ({"bias": FAKE + 4}, EINVAL),
                         ({"res": FAKE + 8}, EINVAL), ({"y": None}, EINVAL), ({"y": FAKE + 8}, EINVAL)):
            assert f(**kw) == want, (f.__name__, kw)
    for kw in ({"xc": None}, {"xs": None}, {"xc": FAKE + 8}, {"xs": FAKE + 8}):
        assert gemm(**kw) == EINVAL
    for kw, want in (({"x": None}, EINVAL), ({"x": FAKE + 8}, EINVAL), ({"ld": 248}, ESHAPE), ({"ld": 260}, ESHAPE),
                     ({"act": 1, "ld": 256}, ESHAPE), ({"act": 3}, EINVAL), ({"group": 5}, EUNSUP),
                     ({"k": 320, "group": 128}, ESHAPE)):
        assert lin(**kw) == want, kw
    assert L.ck_mx4_linear_workspace_size(8, 256, 64) == 0      # few rows: one kernel, no workspace
    need = L.ck_mx4_linear_workspace_size(40, 4096, 64)
    assert need > 0
    for kw in ({"room": None}, {"size": need - 1}, {"room": FAKE + 16}):
        assert lin(m=40, k=4096, **kw) == EWS


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("sb", ctypes.c_int64), ("st", ctypes.c_int64)]


class Norm(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class Args(ctypes.Structure):
    _fields_ = ([(n, Rows) for n in ("x", "branch", "x_out", "out")] +
                [(n, ctypes.c_int64) for n in ("batch", "tokens", "width")] + [("branch_norm", Norm), ("norm", Norm)] +
                [(n, Rows) for n in ("gate", "scale", "shift")] + [("dtype", ctypes.c_int32), ("mod_dtype", ctypes.c_int32)] +
                [(n, ctypes.c_float) for n in ("residual_scale", "branch_scale", "eps")])


def rows(data=FAKE, sb=4096, st=64):
    return Rows(data, sb, st)


def args(**kw):
    """An empty batch by default: every check of shapes and types, no launch."""
    a = Args(rows(), rows(), rows(), rows(), 0, 4, 64, Norm(1, FAKE, FAKE), Norm(2, FAKE, FAKE), rows(), rows(), rows(), 0, 0,
             1.0, 1.0, 1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_block_norm_checks(L):
    f = L.ck_block_norm
    assert f(None, None) == EINVAL and f(ctypes.byref(args()), None) == OK
    none = Rows(None, 0, 0)
    for kw, want in (({"dtype": 2}, EINVAL), ({"dtype": -1}, EINVAL), ({"mod_dtype": 1}, EINVAL), ({"mod_dtype": 2}, OK),
                     ({"dtype": 1, "mod_dtype": 1}, OK), ({"eps": 0.0}, EINVAL), ({"eps": math.nan}, EINVAL),
                     ({"eps": math.inf}, EINVAL), ({"residual_scale": math.nan}, EINVAL), ({"branch_scale": math.inf}, EINVAL),
                     ({"batch": -1}, ESHAPE), ({"tokens": -1}, ESHAPE), ({"width": 0}, ESHAPE), ({"width": 12}, ESHAPE),
                     ({"width": 16392}, EUNSUP), ({"batch": 1 << 12, "tokens": 1 << 12}, EUNSUP),
                     ({"batch": 1 << 62, "tokens": 4}, EUNSUP), ({"norm": Norm(3, None, None)}, EINVAL),
                     ({"branch_norm": Norm(-1, None, None)}, EINVAL), ({"norm": Norm(1, FAKE + 4, None)}, EINVAL),
                     ({"norm": Norm(1, None, FAKE + 8)}, EINVAL), ({"branch_norm": Norm(0, FAKE, None)}, EINVAL),
                     ({"branch": none}, EINVAL), ({"norm": Norm(0, None, None)}, EINVAL), ({"x": rows(FAKE + 8)}, EINVAL),
                     ({"out": rows(FAKE + 2)}, EINVAL), ({"x_out": rows(st=12)}, ESHAPE), ({"branch": rows(sb=-8)}, ESHAPE),
                     ({"x": rows(sb=1 << 40)}, ESHAPE), ({"gate": rows(FAKE + 8)}, EINVAL), ({"scale": rows(st=4)}, ESHAPE),
                     ({"scale": rows(st=4), "mod_dtype": 2}, OK), ({"shift": rows(st=2), "mod_dtype": 2}, ESHAPE),
                     ({"gate": rows(st=0, sb=0)}, OK), ({"x": none}, OK)):
        assert f(ctypes.byref(args(**kw)), None) == want, kw
    plain = {"branch": none, "x_out": none, "branch_norm": Norm(0, None, None), "gate": none}
    assert f(ctypes.byref(args(**plain)), None) == OK
    for kw in ({"x_out": rows()}, {"gate": rows()}, {"branch_norm": Norm(1, None, None)}):
        assert f(ctypes.byref(args(**{**plain, **kw})), None) == EINVAL, kw
    for kw in ({"x": none}, {"x_out": none, "out": none}):      # rows to work on, and nothing to read or write
        assert f(ctypes.byref(args(batch=1, **kw)), None) == EINVAL, kw


def test_binding_refuses_cpu_tensors():
    import torch
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w, u8 = torch.zeros(32, 256), torch.zeros(1, 4, 1024, dtype=torch.uint8)
    for f, a in ((ck.ck_mx4_weight_prep, (w,)), (ck.ck_mx4_act_quant, (x,)), (ck.ck_mx4_dequant, (u8, u8)),
                 (ck.ck_mx4_weight_pack, (u8[0], u8[0])), (ck.ck_mx4_linear, (x, u8, u8)), (ck.ck_block_norm, (x,)),
                 (ck.ck_mx4_act_quant, (None,)), (ck.ck_block_norm, (x.numpy() if x.dtype == torch.float32 else 3,))):
        with pytest.raises(ValueError):
            f(*a)
    with pytest.raises(ValueError):
        ck.ck_mx4_gemm_bf16(u8, u8, u8, u8, m=4)
