"""What the binding refuses of tensors given to the 4-bit entry points: it
takes pointers, so layouts, types, sizes and devices that the C ABI cannot see
are checked first. Sizes and types come before the device, so host tensors
show each check without a GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def tq():
    from packed_weight_matmul_b200 import build
    if build.needs_build():
        build.build()
    from packed_weight_matmul_b200 import tq as _tq
    return _tq


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def refused(tq, status, call, *args, **kw):
    with pytest.raises(tq.TqError) as e:
        call(*args, **kw)
    assert e.value.status == status


# ---- descriptors --------------------------------------------------------------

def test_descriptors_take_dense_tensors(tq):
    n, k = 4, 64
    assert tq.weights_mx4(u8(n, 32), u8(n, 2)).k == k
    assert tq.weights_nv4(u8(n, 32), u8(n, 4), torch.ones(1)).k == k
    # stacked experts, other byte types, more than is needed
    assert tq.weights_mx4(u8(3, n, 32), u8(3, n, 2), n, k).n == n
    assert tq.weights_mx4(u8(n + 2, 32), u8(n + 1, 2), n, k).n == n
    assert tq.weights_nv4(u8(n, 32).view(torch.int8),
                          u8(n, 4).view(torch.float8_e4m3fn),
                          torch.ones(())).n == n


def test_descriptors_refuse_views_that_are_not_dense(tq):
    n, bad = 4, tq.TQ_ERR_INVALID_ARG
    wide, scales = u8(n, 64), u8(n, 2)
    refused(tq, bad, tq.weights_mx4, wide[:, :32], scales)  # columns
    refused(tq, bad, tq.weights_mx4, u8(32, n).t(), scales)  # transposed
    refused(tq, bad, tq.weights_mx4, u8(2 * n, 32)[::2], scales)  # rows
    refused(tq, bad, tq.weights_mx4, u8(n, 32), u8(n, 4)[:, :2])
    refused(tq, bad, tq.weights_mx4, u8(n, 32), u8(2, n).t())
    refused(tq, bad, tq.weights_nv4, u8(n, 32), u8(n, 4), torch.ones(6)[::2])
    refused(tq, bad, tq.weights_mx4, u8(1, 32).expand(n, 32), scales)


def test_descriptors_refuse_other_types(tq):
    n, bad = 4, tq.TQ_ERR_INVALID_ARG
    codes, scales = u8(n, 32), u8(n, 4)
    refused(tq, bad, tq.weights_nv4, codes.int(), scales)
    refused(tq, bad, tq.weights_nv4, codes, scales.float())
    for t in (torch.float64, torch.bfloat16, torch.int32):
        refused(tq, bad, tq.weights_nv4, codes, scales,
                torch.ones(1, dtype=t))


def test_descriptors_refuse_two_devices(tq):
    there = torch.zeros(4, 4, dtype=torch.uint8, device="meta")
    refused(tq, tq.TQ_ERR_INVALID_ARG, tq.weights_nv4, u8(4, 32), there)
    refused(tq, tq.TQ_ERR_INVALID_ARG, tq.weights_nv4, u8(4, 32), u8(4, 4),
            torch.ones(1, device="meta"))


# ---- calls --------------------------------------------------------------------

def linear_args(tq, n=6, k=64, b=3):
    return (tq.weights_mx4(u8(n, k // 2), u8(n, k // 32)),
            torch.zeros(b, k, dtype=torch.bfloat16), torch.zeros(b, n))


def test_linear_refuses_short_tensors(tq):
    """Nothing is read or written past the end of x or y."""
    short = tq.TQ_ERR_SHAPE
    w, x, y = linear_args(tq)
    refused(tq, short, tq.tq_linear, w, x, y[:2])  # rows of y
    refused(tq, short, tq.tq_linear, w, x, y[:, :5])  # columns
    refused(tq, short, tq.tq_linear, w, x[:, :32], y)
    refused(tq, short, tq.tq_linear, w, x, y, batch=4)
    refused(tq, short, tq.tq_linear, w, x, y, ldx=72)
    refused(tq, short, tq.tq_linear, w, x, y, ldy=7)
    refused(tq, short, tq.tq_linear, w, x[0], y)  # one row of 64, not 64 rows


def test_linear_refuses_other_tensors(tq):
    bad = tq.TQ_ERR_INVALID_ARG
    w, x, y = linear_args(tq)
    wide = torch.zeros(3, 128, dtype=torch.bfloat16)
    refused(tq, bad, tq.tq_linear, w, x.float(), y)
    refused(tq, bad, tq.tq_linear, w, x.half(), y)
    refused(tq, bad, tq.tq_linear, w, wide[:, ::2], y)
    refused(tq, bad, tq.tq_linear, w, x, y.bfloat16())
    refused(tq, bad, tq.tq_linear, w, x, y.double())
    refused(tq, bad, tq.tq_linear, w, x, torch.zeros(6, 3).t())
    refused(tq, bad, tq.tq_linear, w, x, y)  # all on the host


def test_unpack_refuses(tq):
    w, _, _ = linear_args(tq)
    out = torch.zeros(6, 64, dtype=torch.bfloat16)
    refused(tq, tq.TQ_ERR_SHAPE, tq.tq_unpack, w, out[:5])
    bad = tq.TQ_ERR_INVALID_ARG
    refused(tq, bad, tq.tq_unpack, w, out.float())
    refused(tq, bad, tq.tq_unpack, w,
            torch.zeros(6, 128, dtype=torch.bfloat16)[:, ::2])
    refused(tq, bad, tq.tq_unpack, w, out)


@pytest.mark.gpu
def test_calls_refuse_host_tensors_beside_device_ones(tq):
    """The package, the status word, one of x and y on the host."""
    bad, d = tq.TQ_ERR_INVALID_ARG, "cuda:0"
    n, k, b = 6, 64, 3
    host, x, y = linear_args(tq, n, k, b)
    w = tq.weights_mx4(u8(n, k // 2).to(d), u8(n, k // 32).to(d))
    xd, yd = x.to(d), y.to(d)
    ids = torch.zeros(b, dtype=torch.int32, device=d)
    xw = tq.weights_mx4(u8(b, k // 2).to(d), u8(b, k // 32).to(d))
    xhost = tq.weights_mx4(u8(b, k // 2), u8(b, k // 32))
    out = torch.zeros(n, k, dtype=torch.bfloat16, device=d)
    status = torch.zeros(1, dtype=torch.int32)
    refused(tq, bad, tq.tq_linear, host, xd, yd)
    refused(tq, bad, tq.tq_linear, w, x, yd)
    refused(tq, bad, tq.tq_linear, w, xd, y)
    refused(tq, bad, tq.tq_unpack, host, out)
    refused(tq, bad, tq.tq_unpack, w, out, status)
    refused(tq, bad, tq.tq_linear_f4, host, xw, yd)
    refused(tq, bad, tq.tq_linear_f4, w, xhost, yd)
    refused(tq, bad, tq.tq_linear_experts_f4, host, 1, ids, xd, yd)
    refused(tq, bad, tq.tq_linear_experts_f4, w, 1, ids, xd, yd, status)
    refused(tq, bad, tq.tq_linear_experts_f4, w, 1, ids, xd, yd, ids.long())
    refused(tq, bad, tq.tq_quantize_f4, xd, tq.TQ_FMT_MX4,
            torch.empty_like(xw._keep[0]), torch.empty_like(xw._keep[1]),
            dev_status=status)
    for call in (lambda: tq.tq_linear(w, xd, yd),
                 lambda: tq.tq_linear(w, xd.view(-1), yd.view(-1), batch=b),
                 lambda: tq.tq_linear(w, xd.data_ptr(), yd.data_ptr(), batch=b,
                                      ldx=k, ldy=n),
                 lambda: tq.tq_linear_f4(w, xw, yd),
                 lambda: tq.tq_linear_experts_f4(w, 1, ids, xd, yd)):
        yd.fill_(7.0)
        call()
        assert (yd == 0).all()
    out.fill_(7.0)
    tq.tq_unpack(w, out)
    assert (out == 0).all()


@pytest.mark.gpu
def test_stream_is_torchs_current_one(tq):
    torch.zeros(1, device="cuda:0")
    side = torch.cuda.Stream()
    for device in (None, torch.cuda.current_device()):
        assert tq._stream(None, device) == \
            torch.cuda.current_stream().cuda_stream
        with torch.cuda.stream(side):
            assert tq._stream(None, device) == side.cuda_stream
    assert tq._stream(side) == side.cuda_stream and tq._stream(7) == 7
