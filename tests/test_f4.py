"""4-bit floats on the CPU: the plain forms the GPU tests compare with, the
package size, and every refusal of tq_quantize_f4, tq_linear_f4,
tq_linear_experts_f4 and of tq_unpack / tq_linear with a 4-bit descriptor
(fake, never dereferenced addresses: rejected before any launch)."""
import ctypes as C

import pytest
import torch

from tests import f4_util as F


@pytest.fixture(scope="module")
def tq():
    from packed_weight_matmul_b200 import build
    if build.needs_build():
        build.build()
    from packed_weight_matmul_b200 import tq as _tq
    return _tq


# ---- the plain forms -----------------------------------------------------------

def test_e2m1_ties_and_saturation():
    q = torch.tensor([0, .25, .26, .75, .74, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5,
                      3.49, 5, 5.01, 6, 7, 1e9], dtype=torch.float64)
    want = [0, 0, 1, 2, 1, 2, 3, 4, 4, 5, 6, 5, 6, 7, 7, 7, 7]
    assert F.e2m1(q).tolist() == want


def test_e4m3_against_torch():
    r = torch.rand(20000, dtype=torch.float64) * torch.exp2(
        torch.rand(20000, dtype=torch.float64) * 22 - 13)
    r = torch.cat([r, F.e4m3_value(torch.arange(127)),
                   (F.e4m3_value(torch.arange(126)) +
                    F.e4m3_value(torch.arange(1, 127))) / 2])
    r = r.clamp_max(448).float().double()
    want = r.float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(F.e4m3(r).to(torch.uint8), want)
    b = torch.arange(128, dtype=torch.uint8)
    assert torch.equal(F.e4m3_value(b).nan_to_num(-1),
                       b.view(torch.float8_e4m3fn).double().nan_to_num(-1))


def test_e8m0_against_torch():
    b = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    assert torch.equal(F.e8m0_value(b).nan_to_num(-1),
                       b.view(torch.float8_e8m0fnu).double().nan_to_num(-1))


def test_quantize_example():
    # the block maximum 5.5 has floor(log2) = 2, so the MX4 scale is 1
    W = torch.zeros(1, 32)
    W[0, :6] = torch.tensor([5.5, -0.2, 0.3, -2.5, 7.0 / 4, -0.0])
    codes, scales, bad = F.quantize(W.bfloat16(), F.MX4)
    assert scales.item() == 127 and not bad
    assert codes[0, :6].tolist() == [7, 8, 1, 12, 4, 8]
    # NV4 with g = 1/6 * 5.5 / 448: the largest scale is 448
    g = F.tensor_scale(W)
    _, s, _ = F.quantize(W.bfloat16(), F.NV4, g)
    assert s[0].tolist() == [126, 0]


# ---- host checks ------------------------------------------------------------------

def test_packed_bytes(tq):
    assert tq.tq_packed_bytes(tq.TQ_FMT_MX4, 3, 64) == 3 * (32 + 2)
    assert tq.tq_packed_bytes(tq.TQ_FMT_NV4, 3, 64) == 3 * (32 + 4) + 4
    assert tq.tq_packed_bytes(tq.TQ_FMT_MX4, 3, 48) == 0


def desc(tq, fmt=None, **kw):
    d = dict(format=tq.TQ_FMT_NV4 if fmt is None else fmt, group=0, planes=1,
             rows_per_scale=0, n_rows=4, k_cols=128, codes=0x10000,
             scales=0x20000, lut=None, codes_plane_stride=0,
             scales_plane_stride=0, lut_rows=0)
    d.update(kw)
    return tq.tq_weights(**d)


BAD_DESC = [
    (dict(codes=None), "INVALID_ARG"), (dict(scales=None), "INVALID_ARG"),
    (dict(planes=2), "INVALID_ARG"), (dict(planes=0), "INVALID_ARG"),
    (dict(lut_rows=32), "INVALID_ARG"),
    (dict(rows_per_scale=1), "INVALID_ARG"),
    (dict(codes_plane_stride=64), "INVALID_ARG"),
    (dict(scales_plane_stride=64), "INVALID_ARG"),
    (dict(n_rows=-1), "INVALID_ARG"), (dict(k_cols=-32), "INVALID_ARG"),
    (dict(format=9), "INVALID_ARG"), (dict(group=32), "UNSUPPORTED"),
    (dict(format=4, group=16), "UNSUPPORTED"),
    (dict(format=4, lut=0x30000), "INVALID_ARG"),
    (dict(k_cols=1 << 28), "UNSUPPORTED"), (dict(k_cols=48), "SHAPE"), (dict(codes=0x10008), "ALIGNMENT"),
    (dict(scales=0x20004), "ALIGNMENT"), (dict(lut=0x30002), "ALIGNMENT"),
]


@pytest.mark.parametrize("kw,err", BAD_DESC)
def test_descriptor_refusals(tq, kw, err):
    L, want = tq.lib(), getattr(tq, "TQ_ERR_" + err)
    w, good = desc(tq, **kw), desc(tq)
    assert L.tq_linear(C.byref(w), 0x40000, 1, 128, 0x50000, 4, None) == want
    assert L.tq_unpack(C.byref(w), 0x40000, None, None) == want
    assert L.tq_linear_f4(C.byref(w), C.byref(good), 0x50000, 4, 0,
                          None) == want
    assert L.tq_linear_f4(C.byref(good), C.byref(w), 0x50000, 4, 0,
                          None) == want
    assert L.tq_linear_experts_f4(C.byref(w), 2, 0x60000, 1, 0x40000, 128,
                                  0x50000, 4, None, None) == want


def test_quantize_refusals(tq):
    def call(W=0x10000, n=4, k=64, ldw=64, fmt=4, codes=0x20000,
             scales=0x30000, ts=None, given=0, st=None):
        return tq.lib().tq_quantize_f4(W, n, k, ldw, fmt, codes, scales, ts,
                                       given, st, None)
    bad, shape, align = (tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_SHAPE,
                         tq.TQ_ERR_ALIGNMENT)
    assert call(W=None) == bad and call(codes=None) == bad
    assert call(scales=None) == bad
    assert call(fmt=1) == bad and call(fmt=6) == bad
    assert call(n=-1) == bad and call(k=-32) == bad
    assert call(ts=0x40000) == bad  # MX4 has no tensor scale
    assert call(given=1) == bad
    assert call(fmt=5) == bad  # NV4 needs one
    assert call(k=48) == shape and call(ldw=56) == shape
    assert call(W=0x10008) == align and call(ldw=68) == align
    assert call(codes=0x20004) == align and call(scales=0x30008) == align
    assert call(fmt=5, ts=0x40002) == align and call(st=0x50001) == align
    assert call(n=0, W=None, codes=None, scales=None) == tq.TQ_OK
    assert call(k=0, ldw=0) == tq.TQ_OK


def test_linear_refusals(tq):
    w = desc(tq)

    def call(x=0x40000, b=1, ldx=128, y=0x50000, ldy=4, w=w):
        return tq.lib().tq_linear(C.byref(w), x, b, ldx, y, ldy, None)
    assert call(x=None) == tq.TQ_ERR_INVALID_ARG
    assert call(y=None) == tq.TQ_ERR_INVALID_ARG
    assert call(b=0) == tq.TQ_ERR_INVALID_ARG
    assert call(ldx=120) == tq.TQ_ERR_SHAPE and call(ldy=3) == tq.TQ_ERR_SHAPE
    assert call(x=0x40008) == tq.TQ_ERR_ALIGNMENT
    assert call(ldx=132) == tq.TQ_ERR_ALIGNMENT
    assert call(y=0x50002) == tq.TQ_ERR_ALIGNMENT
    assert call(w=desc(tq, n_rows=0), ldy=0) == tq.TQ_OK


def test_linear_workspace_refusals(tq):
    big = desc(tq, n_rows=8192, k_cols=8192)

    def need(w, b):
        return tq.lib().tq_linear_workspace(C.byref(w), b)
    # digit rows of x: 8 rows of codes and scales each, and two words per row
    for b in (3, 64, 512):
        assert need(big, b) >= b * (8 * 8192 * 9 // 16 + 8)
    assert need(big, 5000) == need(big, 512)  # 512 rows at a time
    assert need(big, 1) == 0 and need(big, 0) == 0 and need(big, -1) == 0
    assert need(desc(tq), 64) == 0  # little: the plain kernel
    assert need(desc(tq, n_rows=8192, k_cols=8192, codes=None), 64) == 0
    assert need(desc(tq, n_rows=0, k_cols=8192), 64) == 0
    a = tq.tq_weights(format=tq.TQ_FMT_A, group=64, planes=1, rows_per_scale=0,
                      n_rows=8192, k_cols=8192, codes=0x10000, scales=0x20000)
    assert need(a, 64) == 0
    assert tq.lib().tq_linear_workspace(None, 64) == 0

    def call(x=0x40000, b=64, ldx=8192, y=0x50000, ldy=8192, ws=0x60000,
             size=0, w=big):
        return tq.lib().tq_linear_ws(C.byref(w), x, b, ldx, y, ldy, ws, size,
                                     None)
    size = need(big, 64)
    assert call(ws=0x60080, size=size) == tq.TQ_ERR_ALIGNMENT
    assert call(x=None) == tq.TQ_ERR_INVALID_ARG
    assert call(y=None) == tq.TQ_ERR_INVALID_ARG
    assert call(b=0) == tq.TQ_ERR_INVALID_ARG
    assert call(ldx=8184) == tq.TQ_ERR_SHAPE
    assert call(ldy=8191) == tq.TQ_ERR_SHAPE
    assert call(x=0x40008) == tq.TQ_ERR_ALIGNMENT
    assert call(ldx=8196) == tq.TQ_ERR_ALIGNMENT
    assert call(y=0x50002) == tq.TQ_ERR_ALIGNMENT
    assert call(w=desc(tq, n_rows=0), b=1, ldx=128) == tq.TQ_OK


def test_product_refusals(tq):
    w, x = desc(tq), desc(tq, n_rows=3)

    def call(w=w, x=x, y=0x50000, ldy=4, yt=0):
        return tq.lib().tq_linear_f4(C.byref(w), C.byref(x), y, ldy, yt, None)
    assert call(x=desc(tq, fmt=4)) == tq.TQ_ERR_INVALID_ARG
    assert call(y=None) == tq.TQ_ERR_INVALID_ARG
    assert call(yt=2) == tq.TQ_ERR_INVALID_ARG
    assert call(x=desc(tq, k_cols=64)) == tq.TQ_ERR_SHAPE
    assert call(ldy=3) == tq.TQ_ERR_SHAPE
    assert call(y=0x50002) == tq.TQ_ERR_ALIGNMENT
    assert call(y=0x50001, yt=1) == tq.TQ_ERR_ALIGNMENT
    big = desc(tq, n_rows=1 << 30)
    assert call(w=big, ldy=1 << 30) == tq.TQ_ERR_UNSUPPORTED
    assert call(x=big) == tq.TQ_ERR_UNSUPPORTED
    a = tq.tq_weights(format=tq.TQ_FMT_A, group=64, planes=1, rows_per_scale=0,
                      n_rows=4, k_cols=128, codes=0x10000, scales=0x20000)
    assert call(w=a) == tq.TQ_ERR_INVALID_ARG
    assert call(w=a, x=a) == tq.TQ_ERR_INVALID_ARG
    assert call(x=desc(tq, n_rows=0)) == tq.TQ_OK
    assert call(w=desc(tq, n_rows=0), ldy=0) == tq.TQ_OK
    assert tq.lib().tq_linear_f4(None, C.byref(x), 0x50000, 4, 0,
                                 None) == tq.TQ_ERR_INVALID_ARG
    assert tq.lib().tq_linear_f4(C.byref(w), None, 0x50000, 4, 0,
                                 None) == tq.TQ_ERR_INVALID_ARG


def test_experts_refusals(tq):
    def call(w=None, e=3, ids=0x60000, t=2, x=0x40000, ldx=128, y=0x50000,
             ldy=4, st=None):
        return tq.lib().tq_linear_experts_f4(
            C.byref(desc(tq) if w is None else w), e, ids, t, x, ldx, y, ldy,
            st, None)
    bad = tq.TQ_ERR_INVALID_ARG
    assert call(e=0) == bad and call(t=-1) == bad and call(ids=None) == bad
    assert call(x=None) == bad and call(y=None) == bad
    assert call(t=65536) == tq.TQ_ERR_UNSUPPORTED
    assert call(e=65536) == tq.TQ_ERR_UNSUPPORTED
    assert call(w=desc(tq, n_rows=0)) == tq.TQ_ERR_SHAPE
    assert call(w=desc(tq, k_cols=0)) == tq.TQ_ERR_SHAPE
    assert call(ldx=64) == tq.TQ_ERR_SHAPE and call(ldy=3) == tq.TQ_ERR_SHAPE
    for kw in (dict(ids=0x60002), dict(x=0x40008), dict(ldx=132),
               dict(y=0x50002), dict(st=0x70001)):
        assert call(**kw) == tq.TQ_ERR_ALIGNMENT
    assert call(t=0, ids=None, x=None, y=None) == tq.TQ_OK


def test_binding_refuses_short_packages(tq):
    c, s = torch.zeros(6, 16, dtype=torch.uint8), torch.zeros(
        6, 2, dtype=torch.uint8)
    g = torch.ones(3)
    assert tq.weights_nv4(c, s, g, 2, 32).n == 2  # three experts
    for args in ((c, s, g, 7, 32), (c, s[:5], None), (c[:, :8], s, g, 6, 32),
                 (c, s, torch.ones(0))):
        with pytest.raises(tq.TqError) as e:
            tq.weights_nv4(*args)
        assert e.value.status == tq.TQ_ERR_SHAPE
    with pytest.raises(tq.TqError):
        tq.weights_mx4(c, s[:, :0])


def test_binding_refuses_host_tensors(tq):
    W = torch.zeros(2, 32, dtype=torch.bfloat16)
    c, s = torch.zeros(2, 16, dtype=torch.uint8), torch.zeros(
        2, 1, dtype=torch.uint8)
    with pytest.raises(tq.TqError):
        tq.tq_quantize_f4(W, tq.TQ_FMT_MX4, c, s)
    w = tq.weights_mx4(c, s)
    assert (w.n, w.k) == (2, 32)
    with pytest.raises(tq.TqError):
        tq.tq_linear_f4(w, w, torch.zeros(2, 2))
    with pytest.raises(tq.TqError):
        tq.tq_linear_experts_f4(w, 1, torch.zeros(1, dtype=torch.int32), W,
                                torch.zeros(1, 2))
