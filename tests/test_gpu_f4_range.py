"""GPU tests of the 4-bit products where the values, not the sizes, are the
hard part: block scales far apart, all-zero blocks under large scales, Inf
against small blocks, intermediate results outside fp32's range, every digit of
the digit rows, long sums of one sign. References in 64 bits (f4_util)."""
import pytest
import torch

from tests import f4_util as F
from tests import gpu_util as U
from tests.test_gpu_f4 import (FMTS, MX4, NV4, exact_package, gen, integers,
                               linear_ws, run_linear, weights)

pytestmark = pytest.mark.gpu

# one of each kernel and row count per pass: digits made on the spot, the row
# kernel with 8, 16, 32 and 64 rows
BATCHES = [1, 3, 5, 12, 20, 64]


def plain_linear(w, x):
    """tq_linear of the C ABI: never a workspace."""
    tq, b = U.tq(), x.shape[0]
    y = torch.full((b, w.n), float("nan"), device=U.DEV)
    assert tq.lib().tq_linear(w.desc, x.data_ptr(), b, x.stride(0),
                              y.data_ptr(), w.n, None) == tq.TQ_OK
    torch.cuda.synchronize()
    return y


def run_experts(w, E, ids, x):
    y = torch.full((x.shape[0], w.n), float("nan"), device=U.DEV)
    U.tq().tq_linear_experts_f4(w, E, ids, x, y)
    torch.cuda.synchronize()
    return y


def expert_ids(t, E, seed=5):
    return torch.randint(0, E, (t,), generator=gen(seed), device=U.DEV,
                         dtype=torch.int32)


def expert_ref(w64, ids, x, n):
    w64 = w64.view(-1, n, w64.shape[1])
    return torch.stack([w64[e] @ r for e, r in zip(ids.tolist(), x.double())])


def same(y, ref, what):
    """Equal, NaN and Inf in the same places."""
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(y), nan), f"{what}: NaN"
    assert torch.equal(y.double()[~nan], ref[~nan]), what


def every_path(fmt, codes, scales, g, x_of, n, what):
    """x_of(rows): bf16 rows whose products with the package are exact in fp32.
    Compares every kernel for bf16 rows; g: tensor scale (float) or None."""
    w64 = F.values(codes, scales, fmt) * (1.0 if g is None else g)
    gt = None if g is None else torch.full((1,), g, device=U.DEV)
    w = weights(fmt, F.pack(codes), scales, gt)
    for b in BATCHES:
        x = x_of(b)
        ref = x.double() @ w64.t()
        same(run_linear(w, x), ref, f"{what}, {b} rows")
        same(plain_linear(w, x), ref, f"{what}, {b} rows, no workspace")
    E = codes.shape[0] // n
    ge = None if g is None else gt.repeat(E)
    we = weights(fmt, F.pack(codes), scales, ge, n, codes.shape[1])
    for t in (E, 5 * E + 1, 40 * E):
        x, ids = x_of(t), expert_ids(t, E)
        same(run_experts(we, E, ids, x), expert_ref(w64, ids, x, n),
             f"{what}, {t} rows over {E} experts")


KS = [1056, 1024]  # a ragged last stage; rows of whole stages


# ---- MX4 block scales ------------------------------------------------------------

@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("low,zero", [(126, 200), (126, 254), (20, 254),
                                      (1, 160)])
def test_zero_block_under_large_scale(k, low, zero):
    """A block of zero codes may carry any scale: it weighs nothing, and the
    other blocks keep their values."""
    n, E = 70, 4
    codes, scales = exact_package(MX4, n * E, k, 1)
    scales = (scales.int() + low - 126).to(torch.uint8)
    for j in (0, 3, k // 32 - 1):
        codes[:, 32 * j:32 * j + 32] &= 8
        scales[:, j] = zero
    scales[5] = zero  # a row of zeros under large scales
    codes[5] = 0
    s = 2.0 ** (100 if low < 126 else 0)
    every_path(MX4, codes, scales, None,
               lambda b: (integers(b, k, b) * s).bfloat16(), n, "zero blocks")


@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("down", [28, 60, 110])
def test_small_blocks_count(k, down):
    """Blocks far below the row's largest keep their values: x is 0 where the
    large blocks are."""
    n, E = 70, 4
    codes, scales = exact_package(MX4, n * E, k, 3)
    small = torch.arange(k // 32, device=U.DEV) % 3 == 1
    scales[:, small] -= down
    mask = small.repeat_interleave(32)

    def x_of(b):
        return torch.where(mask, integers(b, k, b), 0).bfloat16()
    every_path(MX4, codes, scales, None, x_of, n, "small blocks")


@pytest.mark.parametrize("k", KS)
def test_inf_against_small_blocks(k):
    """Inf times a small weight is Inf, not NaN."""
    n, E = 70, 4
    codes, scales = exact_package(MX4, n * E, k, 4)
    scales[:, 2] = 90
    scales[:, 5] = 4
    codes[:, 64:96] |= 1  # no 0 * Inf
    codes[:, 160:192] |= 1

    def x_of(b):
        x = integers(b, k, b)
        x[:, 64:96], x[:, 160:192] = 0, 0
        x[0, 70] = float("inf")
        x[b // 2, 165] = -float("inf")
        return x
    every_path(MX4, codes, scales, None, x_of, n, "Inf")


@pytest.mark.parametrize("k", KS)
def test_nan_scale_beside_the_largest(k):
    """A NaN scale next to scales of 250 to 254, from the first block on or
    later; zero codes under it."""
    n, E = 70, 4
    codes, scales = exact_package(MX4, n * E, k, 5)
    scales = (scales.int() + 124).to(torch.uint8).clamp_max(254)
    for r, j in ((3, 0), (9, 7), (69, k // 32 - 1), (140, 1)):
        scales[r, j] = 255
    codes[9, 7 * 32:8 * 32] = 0
    every_path(MX4, codes, scales, None,
               lambda b: (integers(b, k, b) * 2.0 ** -60).bfloat16(), n, "NaN")


# ---- range -----------------------------------------------------------------------

@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("shift,e", [(122, -80), (-118, 100), (90, 20),
                                     (0, -120), (60, -120)])
def test_scales_and_x_at_opposite_ends(k, shift, e):
    """Large weights times small x, and the other way round."""
    n, E = 70, 4
    codes, scales = exact_package(MX4, n * E, k, 6)
    scales = (scales.int() + shift).to(torch.uint8)
    every_path(MX4, codes, scales, None,
               lambda b: (integers(b, k, b).double() * 2.0 ** e).bfloat16(), n,
               "opposite ends")


@pytest.mark.parametrize("k", KS)
@pytest.mark.parametrize("e,g", [(124, -100), (124, -20), (-125, 100),
                                 (-60, 126), (0, -140)])
def test_tensor_scale_range(k, e, g):
    """Sums that leave fp32's range before the tensor scale brings them back."""
    n, E = 70, 4
    codes, scales = exact_package(NV4, n * E, k, 7)
    every_path(NV4, codes, scales, 2.0 ** g,
               lambda b: (integers(b, k, b).double() * 2.0 ** e).bfloat16(), n,
               "tensor scale")


@pytest.mark.parametrize("fmt,n,k,b", [(MX4, 4096, 8192, 5),
                                       (MX4, 2080, 4128, 40),
                                       (NV4, 16400, 4128, 5),
                                       (NV4, 2080, 4128, 40)])
def test_digit_rows_at_opposite_ends(fmt, n, k, b):
    codes, scales = exact_package(fmt, n, k, 8)
    codes &= 11  # partial sums below 2^22 in steps of 1/4
    for shift, e in ((122, -80), (-118, 100)) if fmt == MX4 else (
            (-100, 124), (100, -125)):
        x = (integers(b, k, b).double() * 2.0 ** e).bfloat16()
        if fmt == MX4:
            s, g, f = (scales.int() + shift).to(torch.uint8), None, 1.0
        else:
            s, f = scales, 2.0 ** shift
            g = torch.full((1,), f, device=U.DEV)
        w = weights(fmt, F.pack(codes), s, g)
        same(linear_ws(w, x), x.double() @ (F.values(codes, s, fmt) * f).t(),
             f"2^{shift}")


@pytest.mark.parametrize("n,k,b", [(130, 288, 20), (257, 544, 130),
                                   (640, 512, 513)])
@pytest.mark.parametrize("gw,gx,s", [(-75, -75, 0x78), (65, 65, 0x01),
                                     (100, -120, 0x38), (-140, 126, 0x38)])
def test_product_tensor_scales(n, k, b, gw, gx, s):
    """The product of the tensor scales may lie outside fp32's range."""
    cw, _ = exact_package(NV4, n, k, 9)
    cx, _ = exact_package(NV4, b, k, 10)
    cw, cx = cw & 11, cx & 11  # 0, 0.5, 1, 1.5: sums of multiples of 1/4
    cw[3], cx[b - 1] = 0, 0
    sw = torch.full((n, k // 16), s, dtype=torch.uint8, device=U.DEV)
    sx = torch.full((b, k // 16), s, dtype=torch.uint8, device=U.DEV)
    ts = [torch.full((1,), 2.0 ** e, device=U.DEV) for e in (gw, gx)]
    ref = F.values(cx, sx, NV4) @ F.values(cw, sw, NV4).t() * \
        2.0 ** gw * 2.0 ** gx
    w, x = weights(NV4, F.pack(cw), sw, ts[0]), weights(NV4, F.pack(cx), sx,
                                                        ts[1])
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.full((b, n), float("nan"), device=U.DEV, dtype=dtype)
        U.tq().tq_linear_f4(w, x, y)
        torch.cuda.synchronize()
        assert torch.equal(y, ref.to(dtype))


# ---- long sums -----------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("b", [5, 16, 32, 64])
def test_long_sums_of_one_sign(fmt, b):
    """K = 21504 in one CTA (the GPU is full without a split of K), all terms
    positive, so that sums which are cut instead of rounded show up.

    A tensor core chains at most 16 products of 16 k, cut at 2^-23 of their
    sum each; then K / 128 or fewer additions in fp32 follow, off by 2^-24 of
    the sum each, and a few roundings at the end. x is held to 2^-31 of its
    row's largest, which is less than all of these."""
    n, k = 21504, 21504
    packed = torch.randint(0, 256, (n, k // 2), generator=gen(1),
                           device=U.DEV, dtype=torch.uint8) & 0x77
    scales = torch.full((n, k // F.BLOCK[fmt]), 127 if fmt == MX4 else 0x38,
                        dtype=torch.uint8, device=U.DEV)
    w = weights(fmt, packed, scales)
    x = torch.randn(b, k, generator=gen(2), device=U.DEV).abs().bfloat16()
    y = plain_linear(w, x)
    rows = torch.arange(0, n, 83, device=U.DEV)
    w64 = F.values(F.unpack_codes(packed[rows]), scales[rows], fmt)
    ref = x.double() @ w64.t()
    err = ((y[:, rows].double() - ref) / ref).abs().max().item()
    assert err <= (2 * 16 + k // 128 + 4) * 2.0 ** -24, err
