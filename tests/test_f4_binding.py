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
