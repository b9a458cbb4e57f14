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
@pytest.mark.parametrize("low,zero", [(126, 254), (20, 254), (1, 200)])
def test_zero_blocks_before_the_first_weight(k, low, zero):
    """Nothing but zero codes under a large scale for hundreds of columns."""
    n, E = 70, 4
    codes, scales = exact_package(MX4, n * E, k, 2)
    scales = (scales.int() + low - 126).to(torch.uint8)
    for j in list(range(8)) + list(range(16, 24)):
        codes[:, 32 * j:32 * j + 32] &= 8
        scales[:, j] = zero
    s = 2.0 ** (100 if low < 126 else 0)

    def x_of(b):
        x = (integers(b, k, b) * s).bfloat16()
        x[b // 2, 5] = float("nan")  # only this row
        return x
    every_path(MX4, codes, scales, None, x_of, n, "zero blocks")


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


# ---- digits ------------------------------------------------------------------------

def digit_x(fmt, b, k, seed):
    """In every block one 1 where the weight is 0, and values that are integers
    in 2^-22 down to 2^-20 of it: all 8 digits of base 8 occur."""
    size = F.BLOCK[fmt]
    e = torch.randint(5, 21, (b, k), generator=gen(seed), device=U.DEV)
    m = torch.randint(-7, 8, (b, k), generator=gen(seed + 1), device=U.DEV)
    here = torch.rand(b, k, generator=gen(seed + 2), device=U.DEV) < 60.0 / k
    few = torch.rand(b, k, generator=gen(seed + 3), device=U.DEV) < 0.1
    x = torch.where(few | (e > 14), m, 0) * torch.exp2(-e.float())
    x = torch.where(here | (e > 16), x, torch.zeros_like(x))
    x[:, 7::size] = 1.0
    return x.bfloat16()


def digit_package(fmt, n, k, seed):
    """Weights 0, 1, -1 with unit scales, 0 in column 7 of every block."""
    size = F.BLOCK[fmt]
    pick = torch.tensor([0, 2, 10], dtype=torch.uint8, device=U.DEV)
    codes = pick[torch.randint(0, 3, (n, k), generator=gen(seed),
                               device=U.DEV)]
    codes[:, 7::size] = 0
    scales = torch.full((n, k // size), 127 if fmt == MX4 else 0x38,
                        dtype=torch.uint8, device=U.DEV)
    return codes, scales


def check_exactness(fmt, codes, scales, x):
    """The sums of magnitudes stay below 2^24 units of 2^-22."""
    w64 = F.values(codes, scales, fmt)
    assert (x.double().abs() @ w64.abs().t()).max() < 4.0


@pytest.mark.parametrize("fmt", FMTS)
def test_every_digit(fmt):
    """Digits made on the spot: up to 4 rows, and experts."""
    n, k, E = 130, 1056, 16
    codes, scales = digit_package(fmt, n * E, k, 1)
    w64 = F.values(codes, scales, fmt)
    w = weights(fmt, F.pack(codes), scales, None)
    for b in (1, 2, 3, 4, 7, 20, 64):
        x = digit_x(fmt, b, k, b)
        check_exactness(fmt, codes, scales, x)
        same(run_linear(w, x), x.double() @ w64.t(), f"{b} rows")
    we = weights(fmt, F.pack(codes), scales, None, n, k)
    for t in (1, 9, E, 3 * E):
        x, ids = digit_x(fmt, t, k, t), expert_ids(t, E)
        same(run_experts(we, E, ids, x), expert_ref(w64, ids, x, n),
             f"{t} expert rows")


@pytest.mark.parametrize("fmt,n,k,batches", [
    (MX4, 4096, 8192, (3, 5, 8, 9, 20)), (NV4, 16400, 4128, (3, 8, 13)),
    (MX4, 2080, 4128, (33, 130)), (NV4, 2080, 4128, (40,)),
    (MX4, 1100, 1952, (600,)), (NV4, 1100, 1952, (513,))])
def test_every_digit_row(fmt, n, k, batches):
    """Digits written to a workspace, on both sides of 64 digit rows."""
    codes, scales = digit_package(fmt, n, k, 2)
    w64 = F.values(codes, scales, fmt)
    w = weights(fmt, F.pack(codes), scales, None)
    for b in batches:
        x = digit_x(fmt, b, k, b)
        check_exactness(fmt, codes, scales, x)
        same(linear_ws(w, x), x.double() @ w64.t(), f"{b} rows")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k,b", [(4096, 8192, 4), (2080, 4128, 40),
                                   (16400, 4128, 7), (300, 1056, 2)])
def test_integers_of_8_bits(fmt, n, k, b):
    """x of 8 significant bits times 0, 1, -1."""
    codes, scales = digit_package(fmt, n, k, 3)
    x = integers(b, k, 4, top=255)
    y = run_linear(weights(fmt, F.pack(codes), scales, None), x)
    same(y, x.double() @ F.values(codes, scales, fmt).t(), "8 bits")


def value_bound(fmt, w, x, k):
    """Bound on |y - y_exact| as include/tq.h states it: k additions, each off
    by at most 2^-23 of the sum of magnitudes, and x off by at most 2^-23 of
    the largest value of its block or 2^-39 of its row's."""
    size, ax, aw = F.BLOCK[fmt], x.abs(), w.abs()
    top = ax.view(x.shape[0], -1, size).amax(2)
    sums = aw.view(w.shape[0], -1, size).sum(2)
    return (k + 8) * 2.0 ** -23 * (ax @ aw.t()) + \
        2.0 ** -23 * (top @ sums.t()) + \
        2.0 ** -39 * ax.amax(1)[:, None] * aw.sum(1)[None, :] + 1e-37


def far_below(fmt, b, k, seed, low):
    """In column 7 of every block a large value (weight 0), the others 2^-16 to
    2^-low of it: what they lose shows."""
    e = torch.randint(16, low + 1, (b, k), generator=gen(seed), device=U.DEV)
    m = 1 + torch.rand(b, k, generator=gen(seed + 1), device=U.DEV)
    x = m * torch.exp2(-e.float())
    x[:, 7::F.BLOCK[fmt]] = 1.0
    x[:, 1::3] *= -1
    return x.bfloat16()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("low", [20, 30, 45])
def test_values_far_below_their_block(fmt, low):
    n, k, E = 130, 1056, 16
    codes, scales = digit_package(fmt, n * E, k, 4)
    w64 = F.values(codes, scales, fmt)
    w = weights(fmt, F.pack(codes), scales, None)
    for b in BATCHES:
        x = far_below(fmt, b, k, b, low)
        F.check(run_linear(w, x), x.double() @ w64.t(),
                value_bound(fmt, w64, x.double(), k), f"{b} rows")
    we = weights(fmt, F.pack(codes), scales, None, n, k)
    x, ids = far_below(fmt, E, k, 3, low), expert_ids(E, E)
    tol = value_bound(fmt, w64, x.double(), k).view(E, E, n)
    F.check(run_experts(we, E, ids, x), expert_ref(w64, ids, x, n),
            tol[torch.arange(E, device=U.DEV), ids.long()], "experts")


@pytest.mark.parametrize("fmt,n,k,b", [(MX4, 4096, 8192, 5),
                                       (MX4, 2080, 4128, 40),
                                       (NV4, 16400, 4128, 5),
                                       (NV4, 2080, 4128, 40)])
def test_digit_rows_far_below_their_block(fmt, n, k, b):
    codes, scales = digit_package(fmt, n, k, 5)
    w64 = F.values(codes, scales, fmt)
    w = weights(fmt, F.pack(codes), scales, None)
    for low in (20, 45):
        x = far_below(fmt, b, k, b, low)
        F.check(linear_ws(w, x), x.double() @ w64.t(),
                value_bound(fmt, w64, x.double(), k), f"2^-{low}")


def test_ones_beside_the_smallest():
    """x = (1, then values just below 2^-23), the 1 at weight 0: half of the
    sum may be lost to the digits, and no more."""
    k = 32
    codes = torch.full((4, k), 7, dtype=torch.uint8, device=U.DEV)  # 6
    codes[:, 0] = 0
    scales = torch.full((4, 1), 127, dtype=torch.uint8, device=U.DEV)
    w64 = F.values(codes, scales, MX4)
    for b in (1, 5):
        x = torch.full((b, k), 1.9921875 * 2.0 ** -24, device=U.DEV)
        x[:, 0] = 1.0
        x = x.bfloat16()
        F.check(run_linear(weights(MX4, F.pack(codes), scales), x),
                x.double() @ w64.t(), value_bound(MX4, w64, x.double(), k))


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
