"""Plain 64-bit forms of the 4-bit float formats (TQ_FMT_MX4, TQ_FMT_NV4) for
the tests: torch fp64, elementary operations, no code of the library."""
import torch

MX4, NV4 = 4, 5
BLOCK = {MX4: 32, NV4: 16}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
INF, NAN = float("inf"), float("nan")


def e2m1(q):
    """Codes 0..7 of non-negative fp64 values: nearest, ties to the even
    code, at most 6."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=q.device)
    d = (q.clamp_max(6.0)[..., None] - grid).abs()
    best = d.min(-1, keepdim=True).values
    even_first = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=q.device)
    # weights 8..1 make the first of two equally near codes the only maximum
    first = torch.arange(8, 0, -1, device=q.device)
    return even_first[((d == best)[..., even_first] * first).argmax(-1)]


def e4m3(r):
    """Bytes of non-negative fp64 values: nearest, ties to the even byte, at
    most 448."""
    b = torch.arange(127, device=r.device)
    grid = e4m3_value(b)
    i = torch.searchsorted(grid, r).clamp(1, 126)
    lo, hi = grid[i - 1], grid[i]
    up = (r - lo > hi - r) | ((r - lo == hi - r) & (i % 2 == 0))
    return torch.where(up, i, i - 1)


def e4m3_value(b):
    b = b.long()
    m, e = (b % 8).double(), (b // 8) % 16
    v = torch.where(e > 0, torch.ldexp(8 + m, e - 10), m / 512)
    return torch.where(b % 128 == 127, torch.full_like(v, NAN), v)


def e8m0_value(b):
    b = b.long()
    one = torch.ones_like(b, dtype=torch.float64)
    return torch.where(b == 255, one * NAN, torch.ldexp(one, b - 127))


def scale_value(b, fmt):
    return e8m0_value(b) if fmt == MX4 else e4m3_value(b)


def tensor_scale(W):
    a = W.double().abs()
    a = a[torch.isfinite(a)]
    top = a.max() if a.numel() else torch.zeros((), dtype=torch.float64,
                                                device=W.device)
    return torch.ones_like(top).float() if top == 0 else (top / 2688).float()


def quantize(W, fmt, g=None):
    """(codes uint8 [n][k], scale bytes uint8 [n][k / block], bad) of a bf16
    matrix; bad: some value is not finite."""
    n, k = W.shape
    v = W.double().view(n, -1, BLOCK[fmt])
    a = v.abs()
    broken = ~torch.isfinite(a).all(2)
    top = torch.where(broken, torch.zeros_like(a[..., 0]), a.amax(2))
    if fmt == MX4:
        e = (torch.frexp(top)[1] - 1).clamp(-125, 127) - 2
        e = torch.where(top == 0, torch.full_like(e, -127), e)
        byte = (e + 127).long()
        unit = torch.ldexp(torch.ones_like(top), e)
        nan = 255
    else:
        byte = e4m3(top / (6.0 * g.double()))
        unit = e4m3_value(byte) * g.double()
        nan = 127
    q = a / unit[..., None]
    q = torch.where((unit[..., None] == 0) | broken[..., None],
                    torch.zeros_like(q), q)
    sign = torch.signbit(v) & ~broken[..., None]
    code = e2m1(q) + 8 * sign.long()
    byte = torch.where(broken, torch.full_like(byte, nan), byte)
    return code.view(n, k).to(torch.uint8), byte.to(torch.uint8), \
        bool(broken.any())


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous()


def unpack_codes(packed):
    return torch.stack((packed & 15, packed >> 4), 2).view(packed.shape[0], -1)


def values(codes, scales, fmt):
    """fp64 weights (without the tensor scale) of codes [n][k]."""
    grid = torch.tensor(GRID + tuple(-x for x in GRID), dtype=torch.float64,
                        device=codes.device)
    w = grid[codes.long()].view(codes.shape[0], -1, BLOCK[fmt])
    return (w * scale_value(scales, fmt)[..., None]).view(codes.shape)


def sum_bound(w, x, k):
    """Bound on |y - y_exact| of y = x w^T summed in 32 bits: k additions, each
    off by at most one unit of 2^-23 of the sum of magnitudes (a tensor core
    may cut instead of rounding); operands held relative to the largest of
    their row lose at most 2^-26 of it."""
    aw, ax = w.abs(), x.abs()
    return (k + 8) * 2.0 ** -23 * (ax @ aw.t()) + 2.0 ** -26 * (
        ax.sum(1)[:, None] * aw.amax(1)[None, :] +
        ax.amax(1)[:, None] * aw.sum(1)[None, :]) + 1e-37


def check(y, ref, tol, what=""):
    y = y.double()
    nan = torch.isnan(ref)
    assert torch.equal(nan, torch.isnan(y)), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(y[inf], ref[inf]), f"{what}: Inf in other places"
    fine = ~(nan | inf)
    err = (y - ref).abs()[fine]
    bad = ~(err <= tol.expand_as(ref)[fine])
    assert not bad.any(), (f"{what}: {int(bad.sum())} outputs out of "
                           f"tolerance, largest error {err.max().item():.3g}")
