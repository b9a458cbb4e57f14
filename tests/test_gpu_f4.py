"""GPU parity of the 4-bit float operators with their plain 64-bit forms
(f4_util): quantizer and decoder bit for bit, the products exactly on inputs
whose sums are exact in fp32 and within a derived bound otherwise, at ragged
sizes, odd batches, padded strides, special scales and values; then the
operators in a row, captured and replayed, and on another stream."""
import numpy as np
import pytest
import torch

from tests import f4_util as F
from tests import gpu_util as U

pytestmark = pytest.mark.gpu

MX4, NV4 = F.MX4, F.NV4
FMTS = [pytest.param(MX4, id="mx4"), pytest.param(NV4, id="nv4")]


def gen(seed):
    return torch.Generator(device=U.DEV).manual_seed(seed)


def quantize(W, fmt, g=None):
    """Library call on a bf16 matrix (any row stride); outputs pre-filled."""
    tq, (n, k) = U.tq(), W.shape
    codes = torch.full((n, k // 2), 0xAB, dtype=torch.uint8, device=U.DEV)
    scales = torch.full((n, k // F.BLOCK[fmt]), 0xCD, dtype=torch.uint8,
                        device=U.DEV)
    st = U.status_tensor()
    ts = None
    if fmt == NV4:
        ts = torch.full((1,), float("nan"), device=U.DEV) if g is None else \
            g.reshape(1).clone()
    tq.tq_quantize_f4(W, fmt, codes, scales, ts, g is not None, st)
    torch.cuda.synchronize()
    return codes, scales, ts, int(st.item())


def weights(fmt, codes, scales, g=None, n=None, k=None):
    return U.tq().weights_mx4(codes, scales, n, k) if fmt == MX4 else \
        U.tq().weights_nv4(codes, scales, g, n, k)


def check_quantize(W, fmt, g=None):
    codes, scales, ts, st = quantize(W, fmt, g)
    if fmt == NV4 and g is None:
        g = F.tensor_scale(W)
        assert ts.item() == g.item()
    rc, rs, bad = F.quantize(W, fmt, g)
    assert st == (U.tq().TQ_ERR_NONFINITE if bad else 0)
    assert torch.equal(scales, rs)
    assert torch.equal(F.unpack_codes(codes), rc)
    return codes, scales, g


def sample(n, k, seed, scale=0.02):
    return (scale * torch.randn(n, k, generator=gen(seed), device=U.DEV) *
            torch.exp2(6 * torch.rand(n, 1, generator=gen(seed + 1),
                                      device=U.DEV) - 3)).bfloat16()


# ---- quantizer and decoder ----------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k", [(1, 32), (1, 64), (3, 96), (37, 544),
                                 (129, 1056), (512, 4096), (5, 21504)])
def test_quantize(fmt, n, k):
    check_quantize(sample(n, k, n + k), fmt)
    if fmt == NV4:
        for f in (1.0, 1.37, 0.2, 9.0):
            W = sample(n, k, n + k + 2)
            check_quantize(W, fmt, F.tensor_scale(W) * f)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_row_stride(fmt):
    wide = sample(40, 512, 3)
    check_quantize(wide[:, 64:320], fmt)
    check_quantize(wide[::3, 96:128], fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_every_bf16_magnitude(fmt):
    """Every finite bf16 value next to block maxima of many sizes: ties and
    values next to a border among them."""
    bits = torch.arange(65536, device=U.DEV, dtype=torch.int32)
    v = bits.to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    W = v[torch.randint(0, v.numel(), (2048, 256), generator=gen(1),
                        device=U.DEV)]
    e = torch.randint(-120, 120, (2048, 16), generator=gen(2), device=U.DEV)
    near = torch.randn(2048, 16, 16, generator=gen(3), device=U.DEV) * \
        torch.exp2(e.float())[..., None]
    check_quantize(W.contiguous(), fmt)
    check_quantize(near.view(2048, 256).bfloat16(), fmt)
    if fmt == NV4:
        for g in (2.0 ** -126, 1e-42, 1e-20, 1.0, 3e38, 0.7):
            check_quantize(near.view(2048, 256).bfloat16(), fmt,
                           torch.tensor(g, device=U.DEV))


def test_quantize_on_borders():
    """Quotients exactly on every border of E2M1 and E4M3, and one bf16 step
    beside it."""
    borders = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0],
                           device=U.DEV)
    rows = []
    for s in (1.0, 1.125, 1.75, 0.5, 3.25):
        b = borders * s
        up = (b.bfloat16().view(torch.int16) + 1).view(torch.bfloat16).float()
        dn = (b.bfloat16().view(torch.int16) - 1).view(torch.bfloat16).float()
        for t in (b, up, dn, -b):
            r = torch.zeros(32, device=U.DEV)
            r[:8], r[8:16] = t, t.flip(0)
            r[16:24], r[0] = t, 6 * s
            r[16] = 6 * s
            rows.append(r)
    W = torch.stack(rows).bfloat16()
    check_quantize(W, MX4)
    for g in (1.0, 0.5, 1.5, 1 / 3, 0.1):
        check_quantize(W, NV4, torch.tensor(g, device=U.DEV))
    # block maxima at 6 g times every E4M3 value and every midpoint
    v = F.e4m3_value(torch.arange(127, device=U.DEV))
    t = torch.cat([v, (v[1:] + v[:-1]) / 2]) * 6
    W = torch.zeros(t.numel(), 32, device=U.DEV)
    W[:, 0], W[:, 16] = t, -t
    for g in (1.0, 0.25):
        check_quantize(W.mul(g).bfloat16(), NV4,
                       torch.tensor(g, device=U.DEV))


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_zero_and_nonfinite(fmt):
    W = torch.zeros(6, 96, dtype=torch.bfloat16, device=U.DEV)
    W[1] = -0.0
    W[2, 5] = 1e-39  # subnormal
    check_quantize(W, fmt)
    check_quantize(torch.zeros_like(W), fmt)
    W[3, 7], W[4, 40], W[5, 95] = float("nan"), float("inf"), -float("inf")
    W[3, 8:16] = 3.0
    check_quantize(W, fmt)


def test_quantize_refuses_bad_tensor_scale():
    tq = U.tq()
    W = sample(4, 64, 1)
    for g in (0.0, -1.0, float("nan"), float("inf")):
        codes, scales, ts, st = quantize(W, NV4,
                                         torch.tensor(g, device=U.DEV))
        assert st == tq.TQ_ERR_INVALID_ARG
        assert (scales == 0x7F).all() and (codes == 0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_unpack_every_code_and_scale(fmt):
    """All 16 codes under all scale bytes, bit for bit."""
    tq = U.tq()
    top = 256 if fmt == MX4 else 128
    n = top
    codes = torch.arange(32, device=U.DEV, dtype=torch.int32).to(
        torch.uint8).remainder(16).repeat(n, 1)
    per = 32 // F.BLOCK[fmt]
    scales = torch.arange(n, device=U.DEV, dtype=torch.int32).to(
        torch.uint8)[:, None].repeat(1, per).contiguous()
    out = torch.empty(n, 32, dtype=torch.bfloat16, device=U.DEV)
    for g in ([None] if fmt == MX4 else [None, 1.0, 0.0371, 3e-5]):
        gt = None if g is None else torch.full((1,), g, device=U.DEV)
        st = U.status_tensor()
        tq.tq_unpack(weights(fmt, F.pack(codes), scales, gt), out, st)
        torch.cuda.synchronize()
        ref = F.values(codes, scales, fmt).float()
        ref = (ref if gt is None else ref * gt).bfloat16()
        nan = torch.isnan(ref)
        assert torch.equal(nan, torch.isnan(out)) and int(st.item()) == 0
        assert torch.equal(out[~nan].view(torch.int16),
                           ref[~nan].view(torch.int16))


def test_unpack_reports_signed_scale():
    tq = U.tq()
    st = U.status_tensor()
    codes = torch.full((2, 16), 0x22, dtype=torch.uint8, device=U.DEV)
    scales = torch.full((2, 2), 0x38, dtype=torch.uint8, device=U.DEV)
    scales[1, 1] = 0xB8
    out = torch.empty(2, 32, dtype=torch.bfloat16, device=U.DEV)
    tq.tq_unpack(tq.weights_nv4(codes, scales), out, st)
    torch.cuda.synchronize()
    assert int(st.item()) == tq.TQ_ERR_BAD_CODE and (out == 1).all()


# ---- products -----------------------------------------------------------------------

def exact_package(fmt, n, k, seed):
    """Codes and scales whose products with small integers sum exactly in
    fp32: weights are multiples of 1/4 up to 24."""
    codes = torch.randint(0, 16, (n, k), generator=gen(seed), device=U.DEV,
                          dtype=torch.uint8)
    pick = torch.tensor([126, 127, 128, 129] if fmt == MX4 else
                        [0x30, 0x38, 0x40, 0x44], dtype=torch.uint8,
                        device=U.DEV)  # 0.5, 1, 2, then 4 or 3
    scales = pick[torch.randint(0, 4, (n, k // F.BLOCK[fmt]),
                                generator=gen(seed + 1), device=U.DEV)]
    return codes, scales


def integers(b, k, seed, top=3):
    return torch.randint(-top, top + 1, (b, k), generator=gen(seed),
                         device=U.DEV).bfloat16()


def run_linear(w, x, pad=0, fill=float("nan")):
    b, n = x.shape[0], w.n
    y = torch.full((b, n + pad), fill, device=U.DEV)
    U.tq().tq_linear(w, x, y, batch=b, ldx=x.stride(0) if b > 1 else
                     max(x.shape[1], 8), ldy=n + pad)
    torch.cuda.synchronize()
    return y


BATCHES = [1, 2, 5, 8, 9, 16, 17, 31, 33, 64, 65, 130]
SHAPES = [(1, 32), (5, 64), (16, 96), (127, 160), (128, 256), (130, 288),
          (257, 544), (64, 2080), (1003, 4128)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k", SHAPES)
def test_linear_exact(fmt, n, k):
    codes, scales = exact_package(fmt, n, k, n + k)
    w64 = F.values(codes, scales, fmt)
    w = weights(fmt, F.pack(codes), scales, None)
    for b in BATCHES:
        x = integers(b, k, b)
        y = run_linear(w, x)
        assert torch.equal(y.double(), x.double() @ w64.t()), f"batch {b}"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k,b", [(130, 288, 33), (257, 544, 64),
                                   (64, 2080, 65), (1003, 4128, 130)])
def test_linear_without_workspace(fmt, n, k, b):
    """Batches for which a workspace would help."""
    codes, scales = exact_package(fmt, n, k, n + k)
    w, x = weights(fmt, F.pack(codes), scales, None), integers(b, k, b)
    y = torch.full((b, n), float("nan"), device=U.DEV)
    assert U.tq().lib().tq_linear(w.desc, x.data_ptr(), b, k, y.data_ptr(), n,
                                  None) == U.tq().TQ_OK
    torch.cuda.synchronize()
    assert torch.equal(y.double(),
                       x.double() @ F.values(codes, scales, fmt).t())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k,b", [(300, 1024, 1), (300, 1056, 7),
                                   (1000, 5376, 16), (520, 8192, 40),
                                   (200, 21504, 64), (96, 21504, 3)])
def test_linear_quantized(fmt, n, k, b):
    W = sample(n, k, n + b)
    x = torch.randn(b, k, generator=gen(b), device=U.DEV).bfloat16()
    x *= torch.exp2(torch.randint(-20, 20, (b, 1), generator=gen(4),
                                  device=U.DEV).float()).bfloat16()
    codes, scales, g = check_quantize(W, fmt)
    y = run_linear(weights(fmt, codes, scales, g), x)
    w64 = F.values(F.unpack_codes(codes), scales, fmt)
    if g is not None:
        w64 = w64 * g.double()
    F.check(y, x.double() @ w64.t(), F.sum_bound(w64, x.double(), k))


@pytest.mark.parametrize("fmt", FMTS)
def test_linear_padded_strides(fmt):
    n, k, b = 77, 544, 11
    codes, scales = exact_package(fmt, n, k, 5)
    w = weights(fmt, F.pack(codes), scales, None)
    wide = torch.full((b, k + 24), float("nan"), dtype=torch.bfloat16,
                      device=U.DEV)
    wide[:, :k] = integers(b, k, 6)
    y = run_linear(w, wide[:, :k], pad=5, fill=7.0)
    assert (y[:, n:] == 7.0).all()
    assert torch.equal(y[:, :n].double(),
                       wide[:, :k].double() @ F.values(codes, scales, fmt).t())


@pytest.mark.parametrize("b", [1, 6, 20])
def test_linear_scale_range(b):
    """MX4 scales over the whole range of a bf16 matrix inside one row, and x
    over many powers of two: within the bound, relative to the row's
    largest."""
    n, k = 70, 1056
    codes = torch.randint(0, 16, (n, k), generator=gen(1), device=U.DEV,
                          dtype=torch.uint8)
    scales = torch.randint(20, 200, (n, k // 32), generator=gen(2),
                           device=U.DEV).to(torch.uint8)
    scales[:8] = torch.arange(120, 120 + k // 32, device=U.DEV).to(torch.uint8)
    scales[8:16] = scales[:8].flip(1)
    x = (torch.randn(b, k, generator=gen(3), device=U.DEV) * torch.exp2(
        torch.randint(-30, 5, (b, k), generator=gen(4),
                      device=U.DEV).float())).bfloat16()
    y = run_linear(weights(MX4, F.pack(codes), scales), x)
    w64 = F.values(codes, scales, MX4)
    F.check(y, x.double() @ w64.t(), F.sum_bound(w64, x.double(), k))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("b", [1, 4, 20, 64])
def test_linear_special_values(fmt, b):
    """NaN scales poison their row, NaN and Inf in x their batch row, all-zero
    rows and x give exactly 0; nothing else changes."""
    n, k = 130, 1056
    codes, scales = exact_package(fmt, n, k, 9)
    codes[3] = 0
    codes[:, 100] = 2  # no 0 * Inf in the checked column
    x = integers(b, k, 10)
    x[b // 2] = 0
    scales[77, 1] = 255 if fmt == MX4 else 127
    if b > 2:
        x[1, 100] = float("inf")
        x[2, 31] = float("nan")
    y = run_linear(weights(fmt, F.pack(codes), scales, None), x)
    ref = x.double() @ F.values(codes, scales, fmt).t()
    nan = torch.isnan(ref)
    assert torch.equal(nan, torch.isnan(y))
    assert torch.equal(y[~nan].double(), ref[~nan])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("b", [2, 16, 48])
def test_linear_huge_and_tiny_x(fmt, b):
    """bf16 values at both ends of the range, subnormals among them."""
    n, k = 33, 288
    codes, scales = exact_package(fmt, n, k, 11)
    x = integers(b, k, 12).double()
    x[0] *= 2.0 ** -133
    x[1] *= 2.0 ** 110
    y = run_linear(weights(fmt, F.pack(codes), scales, None), x.bfloat16())
    ref = x @ F.values(codes, scales, fmt).t()
    assert torch.equal(y.double(), ref)


def run_product(w, x, dtype, pad=0):
    y = torch.full((x.n, w.n + pad), 7.0, device=U.DEV, dtype=dtype)
    U.tq().tq_linear_f4(w, x, y)
    torch.cuda.synchronize()
    assert (y[:, w.n:] == 7.0).all()
    return y[:, :w.n]


PRODUCTS = [(1, 32, 1), (5, 64, 3), (128, 256, 16), (130, 288, 17),
            (127, 96, 130), (257, 544, 65), (64, 2080, 40), (384, 1024, 256),
            (300, 1056, 300), (1003, 4128, 13), (640, 512, 513)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k,b", PRODUCTS)
def test_product_exact(fmt, n, k, b):
    cw, sw = exact_package(fmt, n, k, n + b)
    cx, sx = exact_package(fmt, b, k, k + b + 1)
    # products are multiples of 1/16 up to 576: exact in fp32 up to K = 1820,
    # so longer rows keep their codes small (multiples of 1/16 up to 1)
    if k > 1820:
        cw, cx = cw & 9, cx & 9
    ref = F.values(cx, sx, fmt) @ F.values(cw, sw, fmt).t()
    w = weights(fmt, F.pack(cw), sw, None)
    x = weights(fmt, F.pack(cx), sx, None)
    y = run_product(w, x, torch.float32)
    assert torch.equal(y.double(), ref)
    y = run_product(w, x, torch.bfloat16, pad=3)
    assert torch.equal(y, ref.float().bfloat16())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k,b", [(300, 5376, 48), (1000, 2048, 129),
                                   (130, 21504, 7), (520, 8192, 260)])
def test_product_quantized(fmt, n, k, b):
    W, X = sample(n, k, n + b), sample(b, k, k + b, scale=1.0)
    cw, sw, gw = check_quantize(W, fmt)
    cx, sx, gx = check_quantize(X, fmt)
    w64 = F.values(F.unpack_codes(cw), sw, fmt)
    x64 = F.values(F.unpack_codes(cx), sx, fmt)
    if fmt == NV4:
        w64, x64 = w64 * gw.double(), x64 * gx.double()
    ref, tol = x64 @ w64.t(), F.sum_bound(w64, x64, k)
    w, x = weights(fmt, cw, sw, gw), weights(fmt, cx, sx, gx)
    F.check(run_product(w, x, torch.float32), ref, tol)
    F.check(run_product(w, x, torch.bfloat16), ref,
            tol + ref.abs() * (torch.finfo(torch.bfloat16).eps / 2))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("b", [5, 70, 200])
def test_product_nan_scales(fmt, b):
    n, k = 200, 544
    cw, sw = exact_package(fmt, n, k, 1)
    cx, sx = exact_package(fmt, b, k, 2)
    nan = 255 if fmt == MX4 else 127
    sw[190, 3], sx[b - 1, 0] = nan, nan
    cw[17], cx[2] = 0, 8  # all zero, all -0
    y = run_product(weights(fmt, F.pack(cw), sw, None),
                    weights(fmt, F.pack(cx), sx, None), torch.float32)
    ref = F.values(cx, sx, fmt) @ F.values(cw, sw, fmt).t()
    keep = ~torch.isnan(ref)
    assert torch.equal(torch.isnan(y), ~keep)
    assert torch.equal(y[keep].double(), ref[keep])


# ---- bf16 rows written as digit rows ------------------------------------------------

def linear_ws(w, x, used=True):
    """tq_linear_ws with a workspace that was filled with 0xFF before."""
    tq, b = U.tq(), x.shape[0]
    need = tq.lib().tq_linear_workspace(w.desc, b)
    assert (need > 0) == used
    ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=U.DEV)
    y = torch.full((b, w.n), float("nan"), device=U.DEV)
    st = tq.lib().tq_linear_ws(
        w.desc, x.data_ptr(), b, x.stride(0), y.data_ptr(), w.n,
        ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == tq.TQ_OK and (ws[need:] == 0xFF).all()
    return y


# n, k, batches: many weights from 3 rows on (NV4: n >= k), fewer weights past
# 16 or 32 rows; ragged tiles, a last stage of 32 to 160 codes, several chunks of
# 512 rows
DIGITS = [(MX4, 4096, 8192, (3, 5, 8, 9, 20)), (MX4, 1003, 33472, (4, 7)),
          (NV4, 16400, 4128, (3, 8, 13, 33)), (NV4, 5800, 5792, (17, 30)),
          (MX4, 4100, 4128, (17,)),
          (MX4, 2080, 4128, (33, 65, 130)), (NV4, 2080, 4128, (40, 64, 97)),
          (MX4, 70, 32, (9500,)),
          (MX4, 1100, 1952, (600, 1030)), (NV4, 1100, 1952, (513,))]


@pytest.mark.parametrize("fmt,n,k,batches", DIGITS)
def test_digit_rows_exact(fmt, n, k, batches):
    """Integers times exact packages, with rows of zeros, NaN and Inf."""
    codes, scales = exact_package(fmt, n, k, n + k)
    if k > 20000:  # partial sums below 2^22 in steps of 1/4
        codes &= 11
    col = min(100, k - 1)
    codes[:, col] = 2  # no 0 * Inf in the checked column
    codes[n // 2] = 0
    codes[n // 2, col] = 1
    scales[n - 2, -1] = 255 if fmt == MX4 else 127
    w64 = F.values(codes, scales, fmt)
    w = weights(fmt, F.pack(codes), scales, None)
    for b in batches:
        x = integers(b, k, b)
        x[b // 2] = 0
        x[1, col] = float("inf")
        if b > 3:
            x[2, 31] = float("nan")
            x[3, col] = -float("inf")
        ref = x.double() @ w64.t()
        y = linear_ws(w, x)
        nan = torch.isnan(ref)
        assert torch.equal(nan, torch.isnan(y)), f"batch {b}"
        assert torch.equal(y[~nan].double(), ref[~nan]), f"batch {b}"
        again = run_linear(w, x)  # the binding brings its own workspace
        assert torch.equal(again[~nan], y[~nan])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k,b", [(16384, 4128, 6), (2080, 4128, 40),
                                   (1100, 1952, 515)])
def test_digit_rows_range(fmt, n, k, b):
    """x over many powers of two inside a row, rows at both ends of the
    range, from rows with a padded stride."""
    W = sample(n, k, 31)
    codes, scales, g, _ = quantize(W, fmt)
    wide = torch.full((b, k + 40), float("nan"), dtype=torch.bfloat16,
                      device=U.DEV)
    x = wide[:, :k]
    x.copy_(torch.randn(b, k, generator=gen(3), device=U.DEV) * torch.exp2(
        torch.randint(-30, 5, (b, k), generator=gen(4), device=U.DEV).float()))
    x[0] = (x[0].double() * 2.0 ** 100).bfloat16()
    x[1] = (x[1].double() * 2.0 ** -110).bfloat16()
    w = weights(fmt, codes, scales, g)
    w64 = F.values(F.unpack_codes(codes), scales, fmt)
    if g is not None:
        w64 = w64 * g.double()
    y = linear_ws(w, x)
    F.check(y, x.double() @ w64.t(), F.sum_bound(w64, x.double(), k))
    assert torch.equal(y, linear_ws(w, x))  # the same bits every time


def test_digit_rows_small_workspace():
    """One byte too few: the plain kernels, the workspace untouched."""
    tq = U.tq()
    codes, scales = exact_package(MX4, 2080, 4128, 1)
    w = weights(MX4, F.pack(codes), scales)
    x = integers(40, 4128, 2)
    need = tq.lib().tq_linear_workspace(w.desc, 40)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=U.DEV)
    y = torch.full((40, 2080), float("nan"), device=U.DEV)
    for ptr, size in ((ws.data_ptr(), need - 1), (None, 0), (None, need)):
        y.fill_(float("nan"))
        assert tq.lib().tq_linear_ws(w.desc, x.data_ptr(), 40, 4128,
                                     y.data_ptr(), 2080, ptr, size,
                                     None) == tq.TQ_OK
        torch.cuda.synchronize()
        assert torch.equal(y.double(),
                           x.double() @ F.values(codes, scales, MX4).t())
    assert (ws == 0xFF).all()


def test_digit_rows_streams_and_graphs():
    """Two streams at once, and two captured graphs replayed in turn, each
    with scratch of its own."""
    tq = U.tq()
    codes, scales = exact_package(NV4, 2080, 4128, 5)
    w64 = F.values(codes, scales, NV4)
    w = weights(NV4, F.pack(codes), scales)
    xs = [integers(b, 4128, b) for b in (40, 70)]
    ys = [torch.zeros(x.shape[0], 2080, device=U.DEV) for x in xs]
    refs = [x.double() @ w64.t() for x in xs]
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in (0, 1):
            tq.tq_linear(w, xs[i], ys[i], stream=sides[i])
    torch.cuda.synchronize()
    assert all(torch.equal(y.double(), r) for y, r in zip(ys, refs))
    graphs = []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tq.tq_linear(w, xs[i], ys[i])
        graphs.append(g)
    for i in (0, 1, 1, 0):
        ys[i].zero_()
        xs[i].copy_(-xs[i])
        refs[i] = -refs[i]
        graphs[i].replay()
        tq.tq_linear(w, xs[1 - i], ys[1 - i])
        torch.cuda.synchronize()
        assert all(torch.equal(y.double(), r) for y, r in zip(ys, refs))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [40, 200, 600])
def test_product_with_itself(fmt, n):
    """x and w may be the same matrix."""
    c, s = exact_package(fmt, n, 544, 3)
    w = weights(fmt, F.pack(c), s, None)
    w64 = F.values(c, s, fmt)
    assert torch.equal(run_product(w, w, torch.float32).double(),
                       w64 @ w64.t())


def test_scalar_tensor_scale():
    """The tensor scale may be a tensor without dimensions."""
    tq, W = U.tq(), sample(4, 64, 1)
    c = torch.empty(4, 32, dtype=torch.uint8, device=U.DEV)
    s = torch.empty(4, 4, dtype=torch.uint8, device=U.DEV)
    g = torch.empty((), device=U.DEV)
    tq.tq_quantize_f4(W, NV4, c, s, g)
    torch.cuda.synchronize()
    assert g.item() == F.tensor_scale(W).item()


# ---- experts ------------------------------------------------------------------------

def run_experts(fmt, E, n, k, ids, seed, pad=0):
    tq, t = U.tq(), len(ids)
    codes, scales = exact_package(fmt, E * n, k, seed)
    g = None
    if fmt == NV4:
        g = torch.exp2(torch.arange(E, device=U.DEV).float() % 5 - 2)
    x = torch.full((t, k + pad), float("nan"), dtype=torch.bfloat16,
                   device=U.DEV)
    x[:, :k] = integers(t, k, seed + 3)
    y = torch.full((t, n + pad), 7.0, device=U.DEV)
    idd = torch.tensor(ids, dtype=torch.int32, device=U.DEV)
    st = U.status_tensor()
    w = weights(fmt, F.pack(codes), scales, g, n, k)
    tq.tq_linear_experts_f4(w, E, idd, x, y, status=st)
    torch.cuda.synchronize()
    assert (y[:, n:] == 7.0).all()
    w64 = F.values(codes, scales, fmt).view(E, n, k)
    if g is not None:
        w64 = w64 * g.double()[:, None, None]
    ref = torch.full((t, n), float("nan"), dtype=torch.float64, device=U.DEV)
    for i, e in enumerate(ids):
        if 0 <= e < E:
            ref[i] = w64[e] @ x[i, :k].double()
    y = y[:, :n].double()
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(y), nan)
    assert torch.equal(y[~nan], ref[~nan])
    return int(st.item())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("E,n,k,t", [(1, 1, 32, 1), (3, 37, 96, 5),
                                     (5, 130, 288, 40), (16, 256, 544, 64),
                                     (2, 129, 1056, 300), (64, 80, 512, 33)])
def test_experts(fmt, E, n, k, t):
    rng = np.random.default_rng(E + t)
    ids = [int(v) for v in rng.integers(0, E, t)]
    assert run_experts(fmt, E, n, k, ids, 7) == 0
    assert run_experts(fmt, E, n, k, ids, 8, pad=8) == 0
    assert run_experts(fmt, E, n, k, [E - 1] * t, 9) == 0  # all to one


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("E,n,k,t", [(3, 40, 96, 2500), (40, 20, 64, 4100),
                                     (2000, 3, 32, 1500), (5000, 2, 32, 5200),
                                     (5000, 2, 32, 3000), (128, 70, 288, 500)])
def test_experts_many_rows(fmt, E, n, k, t):
    """More ids than are looked through at once; more experts than the map of
    the slots holds; an expert that takes nearly all rows."""
    rng = np.random.default_rng(E + t)
    ids = rng.integers(0, E, t)
    assert run_experts(fmt, E, n, k, ids.tolist(), 7) == 0
    ids[rng.random(t) < 0.9] = E // 2
    ids[[5, t - 1]] = E, -1
    assert run_experts(fmt, E, n, k, ids.tolist(), 8) == \
        U.tq().TQ_ERR_INVALID_ARG


@pytest.mark.parametrize("fmt", FMTS)
def test_experts_invalid_ids(fmt):
    ids = [0, 7, 1, -1, 2, 2 ** 31 - 1, -2 ** 31] + [1] * 70 + [3]
    assert run_experts(fmt, 3, 150, 288, ids, 3) == \
        U.tq().TQ_ERR_INVALID_ARG
    assert run_experts(fmt, 2, 20, 64, [5, 9], 3) == U.tq().TQ_ERR_INVALID_ARG


def test_experts_binding_refusals():
    tq = U.tq()
    codes, scales = exact_package(NV4, 3 * 8, 64, 1)
    g = torch.ones(3, device=U.DEV)
    w = weights(NV4, F.pack(codes), scales, g, 8, 64)
    ids = torch.zeros(4, dtype=torch.int32, device=U.DEV)
    x, y = integers(4, 64, 2), torch.zeros(4, 8, device=U.DEV)
    tq.tq_linear_experts_f4(w, 3, ids, x, y)
    short = weights(NV4, F.pack(codes), scales, g[:2], 8, 64)
    for args in ((w, 4, ids, x, y), (short, 3, ids, x, y),
                 (w, 3, ids.view(2, 2), x, y), (w, 3, ids.long(), x, y),
                 (w, 3, ids, x[:3], y), (w, 3, ids, x, y[:, :7]),
                 (w, 3, ids, x[:, ::2], y), (w, 3, ids, x.float(), y)):
        with pytest.raises(tq.TqError):
            tq.tq_linear_experts_f4(*args)
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k,b", [(130, 288, 1), (130, 288, 7), (257, 544, 30),
                                   (300, 288, 70), (2080, 4128, 40),
                                   (640, 512, 300)])
def test_rows_behind_the_batch(fmt, n, k, b):
    """y may have more rows than the batch; they stay as they were."""
    tq = U.tq()
    codes, scales = exact_package(fmt, n, k, 4)
    w = weights(fmt, F.pack(codes), scales, None)
    cx, sx = exact_package(fmt, b, k, 5)
    xw = weights(fmt, F.pack(cx), sx, None)
    x = integers(b, k, 6)
    ids = torch.zeros(b, dtype=torch.int32, device=U.DEV)
    for run in (lambda y: tq.tq_linear(w, x, y),
                lambda y: tq.tq_linear_f4(w, xw, y),
                lambda y: tq.tq_linear_experts_f4(w, 1, ids, x, y)):
        y = torch.full((b + 40, n), 7.0, device=U.DEV)
        run(y)
        torch.cuda.synchronize()
        assert (y[b:] == 7.0).all()


# ---- in a row -----------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
def test_layer_in_a_row(fmt):
    """A layer as it is used: quantize the weights once, then per step either
    the bf16 rows against them or the quantized rows; eager, on another
    stream, and captured into a graph that is replayed on new rows."""
    tq = U.tq()
    n, k, b = 384, 1024, 24
    W = sample(n, k, 1)
    codes, scales, g, _ = quantize(W, fmt)
    w = weights(fmt, codes, scales, g)
    xc = torch.empty(b, k // 2, dtype=torch.uint8, device=U.DEV)
    xs = torch.empty(b, k // F.BLOCK[fmt], dtype=torch.uint8, device=U.DEV)
    xg = torch.empty(1, device=U.DEV) if fmt == NV4 else None
    xw = weights(fmt, xc, xs, xg)
    x = torch.empty(b, k, dtype=torch.bfloat16, device=U.DEV)
    y1 = torch.empty(b, n, device=U.DEV)
    y2 = torch.empty(b, n, device=U.DEV)

    def step():
        tq.tq_linear(w, x, y1)
        tq.tq_quantize_f4(x, fmt, xc, xs, xg)
        tq.tq_linear_f4(w, xw, y2)

    def check(seed, run):
        x.copy_(torch.randn(b, k, generator=gen(seed), device=U.DEV))
        y1.fill_(float("nan"))
        y2.fill_(float("nan"))
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        w64 = F.values(F.unpack_codes(codes), scales, fmt)
        if g is not None:
            w64 = w64 * g.double()
        F.check(y1, x.double() @ w64.t(), F.sum_bound(w64, x.double(), k))
        gx = F.tensor_scale(x) if fmt == NV4 else None
        rc, rs, _ = F.quantize(x, fmt, gx)
        assert torch.equal(F.unpack_codes(xc), rc) and torch.equal(xs, rs)
        x64 = F.values(rc, rs, fmt) * (1 if gx is None else gx.double())
        F.check(y2, x64 @ w64.t(), F.sum_bound(w64, x64, k))
        return y1.clone(), y2.clone()

    a = check(1, step)
    again = check(1, step)
    assert torch.equal(a[0], again[0]) and torch.equal(a[1], again[1])
    side = torch.cuda.Stream()

    def on_side():
        with torch.cuda.stream(side):
            step()
    other = check(1, on_side)
    assert torch.equal(a[0], other[0]) and torch.equal(a[1], other[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 5, 6):
        out = check(seed, graph.replay)
        if seed == 1:
            assert torch.equal(a[0], out[0]) and torch.equal(a[1], out[1])
