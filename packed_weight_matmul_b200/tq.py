"""Thin ctypes binding of libtq.so (include/tq.h), for torch tensors.

Argument marshalling only: every step of the computation runs in the CUDA
library. The names follow the C entry points. Importing this module loads
libtq.so and raises TqError if it has not been built: there is no fallback.

Device tensors are passed by pointer; the CUDA stream defaults to torch's
current stream. A non-TQ_OK status raises TqError (status in `.status`).
"""
import contextlib
import ctypes as C
import os

import numpy as np
import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                        "libtq.so")

TQ_OK, TQ_ERR_INVALID_ARG, TQ_ERR_SHAPE, TQ_ERR_ALIGNMENT = 0, 1, 2, 3
TQ_ERR_UNSUPPORTED, TQ_ERR_BAD_CODE, TQ_ERR_NONFINITE = 4, 5, 6
TQ_ERR_RANGE, TQ_ERR_TIMEOUT, TQ_ERR_CUDA = 7, 8, 9
TQ_FMT_A, TQ_FMT_B, TQ_FMT_B7, TQ_FMT_MX4, TQ_FMT_NV4 = 1, 2, 3, 4, 5
TQ_Y_F32, TQ_Y_BF16 = 0, 1
F4_BLOCK = {TQ_FMT_MX4: 32, TQ_FMT_NV4: 16}

# Every entry point declared in include/tq.h.
ENTRY_POINTS = ("tq_packed_bytes", "tq_build_lut", "tq_quantize_pack",
                "tq_unpack", "tq_linear", "tq_status_string",
                "tq_encode_b", "tq_testing_linear_wait_fault",
                "tq_testing_force_linear_path", "tq_testing_tc_self_check",
                "tq_testing_tc_trace", "tq_linear_experts", "tq_pack7",
                "tq_build_lut7", "tq_testing_tc_split", "tq_quantize_f4",
                "tq_linear_f4", "tq_linear_experts_f4",
                "tq_linear_workspace", "tq_linear_ws")


class TqError(RuntimeError):
    def __init__(self, status, what=""):
        msg = _lib.tq_status_string(status).decode() if _lib else str(status)
        super().__init__(f"{what}: {msg}" if what else msg)
        self.status = status


class tq_weights(C.Structure):
    _fields_ = [("format", C.c_int32), ("group", C.c_int32),
                ("planes", C.c_int32), ("rows_per_scale", C.c_int32),
                ("n_rows", C.c_int64), ("k_cols", C.c_int64),
                ("codes", C.c_void_p), ("scales", C.c_void_p),
                ("lut", C.c_void_p), ("codes_plane_stride", C.c_int64),
                ("scales_plane_stride", C.c_int64),
                ("lut_rows", C.c_int64)]


class tq_experts(C.Structure):
    _fields_ = [("n_experts", C.c_int32), ("n_hot", C.c_int32),
                ("group", C.c_int32), ("reserved", C.c_int32),
                ("n_rows", C.c_int64), ("k_cols", C.c_int64),
                ("codes", C.c_void_p), ("scales", C.c_void_p),
                ("codes2", C.c_void_p), ("scales2", C.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m packed_weight_matmul_b200.build`")
    L = C.CDLL(LIB_PATH)
    i32, i64, P = C.c_int32, C.c_int64, C.c_void_p
    L.tq_packed_bytes.restype = C.c_size_t
    L.tq_packed_bytes.argtypes = [i32, i64, i64, i32, i32]
    L.tq_build_lut.restype = C.c_int
    L.tq_build_lut.argtypes = [C.c_float, P, P]
    L.tq_quantize_pack.restype = C.c_int
    L.tq_quantize_pack.argtypes = [P, i64, i64, i32, i32, P, P, P, P]
    L.tq_unpack.restype = C.c_int
    L.tq_unpack.argtypes = [C.POINTER(tq_weights), P, P, P]
    L.tq_linear.restype = C.c_int
    L.tq_linear.argtypes = [C.POINTER(tq_weights), P, i64, i64, P, i64, P]
    L.tq_encode_b.restype = C.c_int
    L.tq_encode_b.argtypes = [P, i64, i64, P, C.c_float, i32, P, P, P, P, P]
    L.tq_status_string.restype = C.c_char_p
    L.tq_status_string.argtypes = [C.c_int]
    L.tq_testing_linear_wait_fault.restype = C.c_int
    L.tq_testing_linear_wait_fault.argtypes = [i32, C.c_uint64]
    L.tq_testing_force_linear_path.restype = C.c_int
    L.tq_testing_force_linear_path.argtypes = [i32]
    L.tq_testing_tc_split.restype = C.c_int
    L.tq_testing_tc_split.argtypes = [i32, i32]
    L.tq_testing_tc_self_check.restype = C.c_int
    L.tq_testing_tc_self_check.argtypes = [i32, P, i32]
    L.tq_testing_tc_trace.restype = C.c_int
    L.tq_testing_tc_trace.argtypes = [P]
    L.tq_pack7.restype = C.c_int
    L.tq_pack7.argtypes = [P, i64, i64, P, P, P, P, P]
    L.tq_build_lut7.restype = C.c_int
    L.tq_build_lut7.argtypes = [P, P, P]
    L.tq_linear_experts.restype = C.c_int
    L.tq_linear_experts.argtypes = [C.POINTER(tq_experts), P, i64, P, i64, P,
                                    i64, P, P]
    L.tq_quantize_f4.restype = C.c_int
    L.tq_quantize_f4.argtypes = [P, i64, i64, i64, i32, P, P, P, i32, P, P]
    L.tq_linear_workspace.restype = C.c_size_t
    L.tq_linear_workspace.argtypes = [C.POINTER(tq_weights), i64]
    L.tq_linear_ws.restype = C.c_int
    L.tq_linear_ws.argtypes = [C.POINTER(tq_weights), P, i64, i64, P, i64, P,
                               C.c_size_t, P]
    L.tq_linear_f4.restype = C.c_int
    L.tq_linear_f4.argtypes = [C.POINTER(tq_weights), C.POINTER(tq_weights),
                               P, i64, i32, P]
    L.tq_linear_experts_f4.restype = C.c_int
    L.tq_linear_experts_f4.argtypes = [C.POINTER(tq_weights), i32, P, i64, P,
                                       i64, P, i64, P, P]
    return L


_lib = None
_lib = _load()


def lib():
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# torch's own functions behind current_stream and current_device, which take 2
# us less per call; the public ones where torch has them no longer.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or \
    torch.cuda.current_device


def _stream(stream, device=None):
    """`device`: the current one, where the caller knows it."""
    if stream is None:
        return _raw_stream(_current_device() if device is None else device)
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return stream


def _torch_stream(stream):
    """Context in which `stream` (as the calls take it) is torch's current
    stream."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream) if stream else \
            torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _check(status, what):
    if status != TQ_OK:
        raise TqError(status, what)


# ---- host entry points --------------------------------------------------------

def tq_packed_bytes(fmt: int, n: int, k: int, group: int = 64,
                    planes: int = 1) -> int:
    return _lib.tq_packed_bytes(fmt, n, k, group, planes)


def tq_build_lut(alpha: float, ladder) -> np.ndarray:
    lad = np.ascontiguousarray(np.asarray(ladder, np.float32))
    assert lad.shape == (5,)
    out = np.zeros(256, np.float32)
    _check(_lib.tq_build_lut(C.c_float(alpha),
                             lad.ctypes.data_as(C.c_void_p),
                             out.ctypes.data_as(C.c_void_p)), "tq_build_lut")
    return out


def tq_build_lut7(lut, used) -> np.ndarray:
    """Host: LUT7[i] = lut[used[i]] for a 7-bit layer (128 entries)."""
    lut = np.ascontiguousarray(np.asarray(lut, np.float32))
    used = np.ascontiguousarray(np.asarray(used, np.uint8))
    assert lut.shape == (256,) and used.shape == (128,)
    out = np.zeros(128, np.float32)
    _check(_lib.tq_build_lut7(lut.ctypes.data_as(C.c_void_p),
                              used.ctypes.data_as(C.c_void_p),
                              out.ctypes.data_as(C.c_void_p)), "tq_build_lut7")
    return out


def tq_pack7(codes, used_out, n_used_out, packed_out, dev_status=None,
             stream=None, check=True):
    n, k = codes.shape
    st = _lib.tq_pack7(_ptr(codes), n, k, _ptr(used_out), _ptr(n_used_out),
                       _ptr(packed_out), _ptr(dev_status), _stream(stream))
    if check:
        _check(st, "tq_pack7")
    return st


def tq_linear_experts(w: "Experts", ids, x, y, n_tokens=None, ldx=None,
                      ldy=None, status=None, stream=None, check=True):
    if n_tokens is None:
        n_tokens = ids.shape[0]
    if ldx is None:
        ldx = x.stride(0)
    if ldy is None:
        ldy = y.stride(0)
    st = _lib.tq_linear_experts(C.byref(w.desc), _ptr(ids), n_tokens, _ptr(x),
                                ldx, _ptr(y), ldy, _ptr(status),
                                _stream(stream))
    if check:
        _check(st, "tq_linear_experts")
    return st


def tq_testing_linear_wait_fault(withhold_first_arrive: bool,
                                 wait_limit_ns: int = 0) -> None:
    """Test hook (include/tq_testing.h): make the tensor-core tq_linear
    kernels time out on purpose, with a short wait limit."""
    _check(_lib.tq_testing_linear_wait_fault(int(bool(withhold_first_arrive)),
                                             int(wait_limit_ns)),
           "tq_testing_linear_wait_fault")


def tq_testing_force_linear_path(path: int) -> None:
    """Test hook (include/tq_testing.h): 0 automatic dispatch, 1 CUDA-core
    kernels, 2 tensor-core kernel, 3 tensor-core kernel with the Format B
    code book always split into bf16 hi + lo operands."""
    _check(_lib.tq_testing_force_linear_path(int(path)),
           "tq_testing_force_linear_path")


def tq_testing_tc_split(ks: int, max_clusters: int = 0) -> None:
    """Test hook (include/tq_testing.h): split of K over clusters of ks
    CTAs (0 = planner's choice) and a cap on the number of clusters."""
    _check(_lib.tq_testing_tc_split(int(ks), int(max_clusters)),
           "tq_testing_tc_split")


def tq_testing_tc_self_check(enable: bool, read: bool = False,
                             reset: bool = False):
    """Test hook (include/tq_testing.h): select the self-checking
    tensor-core kernel; with read=True return its record (4 integers)."""
    rec = np.zeros(4, np.uint64)
    _check(_lib.tq_testing_tc_self_check(
        int(bool(enable)), rec.ctypes.data_as(C.c_void_p) if read else None,
        int(bool(reset))), "tq_testing_tc_self_check")
    return [int(v) for v in rec] if read else None


def tq_testing_tc_trace(buffer) -> None:
    """Test hook (include/tq_testing.h): progress trace of the self-checking
    tensor-core kernel into a pinned host tensor (int64), or None."""
    _check(_lib.tq_testing_tc_trace(None if buffer is None else
                                    buffer.data_ptr()),
           "tq_testing_tc_trace")


def tq_status_string(status: int) -> str:
    return _lib.tq_status_string(status).decode()


# ---- weight descriptors --------------------------------------------------------

class Weights:
    """A tq_weights descriptor that keeps its tensors alive."""

    def __init__(self, desc: tq_weights, keep, device=None):
        self.desc = desc
        self.ref = C.byref(desc)
        self._keep = keep
        # 4-bit formats: device number (-1 on the host), sizes as plain numbers
        # and bytes of workspace by batch (attributes of a ctypes structure and
        # calls through ctypes take several times as long)
        self.device = device
        self.shape = (desc.n_rows, desc.k_cols)
        self.count = desc.n_rows * desc.k_cols
        self._workspaces = {}

    def workspace(self, batch):
        """tq_linear_workspace."""
        need = self._workspaces.get(batch)
        if need is None:
            need = _lib.tq_linear_workspace(self.ref, batch)
            self._workspaces[batch] = need
        return need

    @property
    def n(self):
        return self.desc.n_rows

    @property
    def k(self):
        return self.desc.k_cols


def weights_a(codes, scales, n, k, group=64, planes=1, codes_plane_stride=0,
              scales_plane_stride=0) -> Weights:
    d = tq_weights(format=TQ_FMT_A, group=group, planes=planes,
                   rows_per_scale=0, n_rows=n, k_cols=k, codes=_ptr(codes),
                   scales=_ptr(scales), lut=None,
                   codes_plane_stride=codes_plane_stride,
                   scales_plane_stride=scales_plane_stride)
    return Weights(d, (codes, scales))


class Experts:
    """A tq_experts descriptor that keeps its tensors alive."""

    def __init__(self, desc: tq_experts, keep):
        self.desc = desc
        self._keep = keep

    @property
    def n(self):
        return self.desc.n_rows

    @property
    def k(self):
        return self.desc.k_cols


def experts_a(codes, scales, n_experts, n, k, n_hot=0, codes2=None,
              scales2=None, group=64) -> Experts:
    """Plane 1 of every expert in codes / scales ([E][N][K/G][13] bytes,
    [E][N][K/G] fp16); plane 2 of experts 0 .. n_hot - 1 in codes2 /
    scales2 (same layout)."""
    d = tq_experts(n_experts=n_experts, n_hot=n_hot, group=group, reserved=0,
                   n_rows=n, k_cols=k, codes=_ptr(codes), scales=_ptr(scales),
                   codes2=_ptr(codes2), scales2=_ptr(scales2))
    return Experts(d, (codes, scales, codes2, scales2))


def weights_b7(packed, lut7, n, k, rho=None, rows_per_scale=0) -> Weights:
    """7-bit layer: packed indices [n][14 k / 16] and LUT7 [128]."""
    d = tq_weights(format=TQ_FMT_B7, group=0, planes=1,
                   rows_per_scale=rows_per_scale if rho is not None else 0,
                   n_rows=n, k_cols=k, codes=_ptr(packed), scales=_ptr(rho),
                   lut=_ptr(lut7), codes_plane_stride=0, scales_plane_stride=0,
                   lut_rows=0)
    return Weights(d, (packed, lut7, rho))


def weights_b(codes, lut, rho=None, rows_per_scale=0, n=None, k=None,
              lut_rows=0) -> Weights:
    """lut: one code book (256 fp32), or with lut_rows > 0 one per block of
    lut_rows rows ([ceil(n / lut_rows)][256], the adaptive alphabet)."""
    if n is None:
        n, k = codes.shape
    d = tq_weights(format=TQ_FMT_B, group=0, planes=1,
                   rows_per_scale=rows_per_scale if rho is not None else 0,
                   n_rows=n, k_cols=k, codes=_ptr(codes), scales=_ptr(rho),
                   lut=_ptr(lut), codes_plane_stride=0, scales_plane_stride=0,
                   lut_rows=lut_rows)
    return Weights(d, (codes, lut, rho))


def _f4_stacked(fmt, codes, scales, lut, count, n, k, what):
    """Whether the tensors hold `count` matrices of n x k."""
    if codes.numel() * 2 < count * n * k or \
            scales.numel() * F4_BLOCK[fmt] < count * n * k or \
            (lut is not None and lut.numel() < count):
        raise TqError(TQ_ERR_SHAPE, f"{what}: fewer than {count} x {n} x {k}")


def _weights_f4(fmt, codes, scales, lut, n, k) -> Weights:
    if n is None:
        n, k = codes.shape[0], codes.shape[1] * 2
    _f4_stacked(fmt, codes, scales, lut, 1, n, k, "weights")
    for t, types, what in ((codes, _U8, "codes"), (scales, _U8, "scales"),
                           (lut, _F32, "tensor scale")):
        if t is not None and (t.dtype not in types or
                              not t.is_contiguous() or
                              t.device != codes.device):
            raise TqError(TQ_ERR_INVALID_ARG, f"weights: {what} {t.dtype}, "
                          f"strides {t.stride()}, on {t.device}")
    d = tq_weights(format=fmt, group=F4_BLOCK[fmt], planes=1,
                   rows_per_scale=0, n_rows=n, k_cols=k, codes=_ptr(codes),
                   scales=_ptr(scales), lut=_ptr(lut), codes_plane_stride=0,
                   scales_plane_stride=0, lut_rows=0)
    return Weights(d, (codes, scales, lut), codes.get_device())


def weights_mx4(codes, scales, n=None, k=None) -> Weights:
    """4-bit floats, blocks of 32: codes [n][k/2] (low four bits = lower k),
    E8M0 scale bytes [n][k/32], both dense. For tq_linear_experts_f4: the
    stacked experts, n the rows of one."""
    return _weights_f4(TQ_FMT_MX4, codes, scales, None, n, k)


def weights_nv4(codes, scales, tensor_scale=None, n=None, k=None) -> Weights:
    """4-bit floats, blocks of 16: codes [n][k/2], E4M3 scale bytes [n][k/16]
    and the fp32 tensor scale (device, 1 value; one per expert for
    tq_linear_experts_f4; None: 1)."""
    return _weights_f4(TQ_FMT_NV4, codes, scales, tensor_scale, n, k)


# ---- GPU entry points -----------------------------------------------------------

def tq_quantize_pack(W, group, planes, codes_out, scales_out, dev_status=None,
                     stream=None, n=None, k=None, check=True):
    if n is None:
        n, k = W.shape
    st = _lib.tq_quantize_pack(_ptr(W), n, k, group, planes, _ptr(codes_out),
                               _ptr(scales_out), _ptr(dev_status),
                               _stream(stream))
    if check:
        _check(st, "tq_quantize_pack")
    return st


def tq_encode_b(W, ladder, zeta, rows_per_scale, codes_out, rho_out,
                alpha_out, dev_status=None, stream=None, n=None, k=None,
                check=True):
    """Format B encoder: W bf16 [n][k] (device) -> codes_out uint8 [n][k],
    rho_out fp16 [ceil(n / rows_per_scale)] (None when rows_per_scale = 0),
    alpha_out fp32 [1] (all device). `ladder` is 5 host floats."""
    if n is None:
        n, k = W.shape
    lad = np.ascontiguousarray(np.asarray(ladder, np.float32))
    assert lad.shape == (5,)
    st = _lib.tq_encode_b(_ptr(W), n, k, lad.ctypes.data_as(C.c_void_p),
                          C.c_float(zeta), rows_per_scale, _ptr(codes_out),
                          _ptr(rho_out), _ptr(alpha_out), _ptr(dev_status),
                          _stream(stream))
    if check:
        _check(st, "tq_encode_b")
    return st


def tq_unpack(w: Weights, out, dev_status=None, stream=None, check=True):
    dev = w.device
    if dev is not None:
        if not (dev >= 0 and dev == _current_device() and
                _f4_plain(out, torch.bfloat16, dev, w.count)):
            _f4_operands(w, ((out, _BF16, 1, 0, w.count),), "tq_unpack")
            if not (isinstance(out, int) or out.is_contiguous()):
                raise TqError(TQ_ERR_INVALID_ARG, "tq_unpack: not dense")
        if dev_status is not None:
            _f4_status(dev_status, dev, "tq_unpack: dev_status")
    st = _lib.tq_unpack(w.ref, _ptr(out), _ptr(dev_status),
                        _raw_stream(dev) if stream is None and dev is not None
                        else _stream(stream))
    if check:
        _check(st, "tq_unpack")
    return st


def tq_linear(w: Weights, x, y, batch=None, ldx=None, ldy=None, stream=None,
              check=True):
    if batch is None:
        batch = x.shape[0]
    if ldx is None:
        ldx = x.stride(0) if x.dim() == 2 else w.k
    if ldy is None:
        ldy = y.stride(0) if y.dim() == 2 else w.n
    need = 0
    if w.device is not None:
        n, k = w.shape
        dev = w.device
        if not (dev >= 0 and dev == _current_device() and
                _f4_plain(x, torch.bfloat16, dev, (batch - 1) * ldx + k) and
                _f4_plain(y, torch.float32, dev, (batch - 1) * ldy + n)):
            _f4_operands(w, ((x, _BF16, batch, ldx, k),
                             (y, _F32, batch, ldy, n)), "tq_linear")
        need = w.workspace(batch)
    if need:
        # scratch from torch's allocator, on the stream that uses it
        with _torch_stream(stream):
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            st = _lib.tq_linear_ws(w.ref, _ptr(x), batch, ldx,
                                   _ptr(y), ldy, ws.data_ptr(), need,
                                   _stream(None))
    else:
        st = _lib.tq_linear(w.ref, _ptr(x), batch, ldx, _ptr(y), ldy,
                            _stream(stream, w.device))
    if check:
        _check(st, "tq_linear")
    return st


def _f4_device(t, what):
    """The current device, on which t has to lie."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        raise TqError(TQ_ERR_INVALID_ARG, f"{what}: not on the current device")
    return dev


def _f4_types(t, dtypes, what):
    """The 4-bit entry points check what the C ABI cannot see of a tensor:
    that it has the element type it is read as and dense rows, and (see the
    callers) that it is large enough and lies on the current device."""
    if t.dtype not in dtypes:
        raise TqError(TQ_ERR_INVALID_ARG, f"{what}: {t.dtype}")
    if not t.is_contiguous() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise TqError(TQ_ERR_INVALID_ARG, f"{what}: rows are not dense")


def _f4_tensor(t, dtypes, dev, what):
    _f4_types(t, dtypes, what)
    if t.get_device() != dev:
        raise TqError(TQ_ERR_INVALID_ARG, f"{what}: not on the current device")


def _f4_plain(t, dtype, dev, count):
    """The common case in few steps: dense, `count` elements at least."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and
            t.is_contiguous() and t.numel() >= count and
            t.get_device() == dev)


def _f4_operands(w, operands, what):
    """(tensor, element types, rows, distance of the rows, columns) each: the
    rows have to lie within the tensor. Plain pointers are taken as they
    are."""
    tensors = [o for o in operands if not isinstance(o[0], int)]
    for t, _, rows, ld, cols in tensors:
        have = t.numel()
        if have and not t.is_contiguous():
            have = 1 + sum((s - 1) * d for s, d in zip(t.shape, t.stride()))
        if cols and rows > 0 and have < (rows - 1) * ld + cols:
            raise TqError(TQ_ERR_SHAPE, f"{what}: {tuple(t.shape)}")
    for t, dtypes, _, _, _ in tensors:
        _f4_types(t, dtypes, what)
    for t, _, _, _, _ in tensors:
        _f4_device(t, what)
    if w.device < 0 or w.device != _current_device():
        raise TqError(TQ_ERR_INVALID_ARG,
                      f"{what}: weights not on the current device")


def _f4_package(w, dev, what):
    """Whether the package lies on the device (other formats: not known)."""
    if w.device is not None and w.device != dev:
        raise TqError(TQ_ERR_INVALID_ARG, f"{what}: not on the current device")


def _f4_status(t, dev, what):
    if isinstance(t, torch.Tensor):
        _f4_tensor(t, (torch.int32,), dev, what)


def _rows(t):
    """Distance of a matrix's rows (any value is right for a single row)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


_BF16, _F32 = (torch.bfloat16,), (torch.float32,)
_U8 = (torch.uint8, torch.int8, torch.float8_e8m0fnu, torch.float8_e4m3fn)


def tq_quantize_f4(W, fmt, codes_out, scales_out, tensor_scale=None,
                   scale_given=False, dev_status=None, stream=None,
                   check=True):
    """Quantize the rows of a bf16 matrix (row stride free) to 4-bit floats:
    codes_out uint8 [n][k/2], scales_out bytes [n][k/32] (TQ_FMT_MX4) or
    [n][k/16] (TQ_FMT_NV4). NV4: tensor_scale is read when scale_given, else
    written."""
    n, k = W.shape
    dev = _f4_device(W, "tq_quantize_f4: W")
    if W.dtype is not torch.bfloat16 or not W.is_contiguous():
        _f4_tensor(W, _BF16, dev, "tq_quantize_f4: W")
    blocks = n * k // F4_BLOCK.get(fmt, 16)
    if not (_f4_plain(codes_out, torch.uint8, dev, n * k // 2) and
            _f4_plain(scales_out, torch.uint8, dev, blocks)):
        _f4_tensor(codes_out, _U8, dev, "tq_quantize_f4: codes_out")
        _f4_tensor(scales_out, _U8, dev, "tq_quantize_f4: scales_out")
        if codes_out.numel() * 2 < n * k or scales_out.numel() < blocks or \
                not (codes_out.is_contiguous() and scales_out.is_contiguous()):
            raise TqError(TQ_ERR_SHAPE, "tq_quantize_f4: outputs")
    if tensor_scale is not None:
        _f4_tensor(tensor_scale, _F32, dev, "tq_quantize_f4: scale")
    if dev_status is not None:
        _f4_status(dev_status, dev, "tq_quantize_f4: dev_status")
    st = _lib.tq_quantize_f4(W.data_ptr(), n, k, _rows(W), fmt,
                             codes_out.data_ptr(), scales_out.data_ptr(),
                             _ptr(tensor_scale), 1 if scale_given else 0,
                             _ptr(dev_status), _stream(stream, dev))
    if check:
        _check(st, "tq_quantize_f4")
    return st


def tq_linear_f4(w: Weights, x: Weights, y, stream=None, check=True):
    """y = x W^T of two 4-bit matrices of one format; y fp32 or bf16
    [batch][n], row stride free."""
    dev = _f4_device(y, "tq_linear_f4: y")
    _f4_tensor(y, _BF16 + _F32, dev, "tq_linear_f4: y")
    _f4_package(w, dev, "tq_linear_f4: w")
    _f4_package(x, dev, "tq_linear_f4: x")
    if y.dim() != 2 or y.shape[0] < x.n or y.shape[1] < w.n:
        raise TqError(TQ_ERR_SHAPE, "tq_linear_f4: y")
    st = _lib.tq_linear_f4(w.ref, x.ref, y.data_ptr(),
                           _rows(y), TQ_Y_BF16 if y.dtype == torch.bfloat16
                           else TQ_Y_F32, _stream(stream, dev))
    if check:
        _check(st, "tq_linear_f4")
    return st


def tq_linear_experts_f4(w: Weights, n_experts, ids, x, y, status=None,
                         stream=None, check=True):
    """y[t] = x[t] W_e^T with e = ids[t] (int32, device); w holds the stacked
    experts, w.n the rows of one."""
    dev = _f4_device(ids, "tq_linear_experts_f4: ids")
    _f4_tensor(ids, (torch.int32,), dev, "tq_linear_experts_f4: ids")
    _f4_tensor(x, _BF16, dev, "tq_linear_experts_f4: x")
    _f4_tensor(y, _F32, dev, "tq_linear_experts_f4: y")
    _f4_package(w, dev, "tq_linear_experts_f4: weights")
    if status is not None:
        _f4_status(status, dev, "tq_linear_experts_f4: status")
    if ids.dim() != 1 or x.dim() != 2 or y.dim() != 2:
        raise TqError(TQ_ERR_SHAPE, "tq_linear_experts_f4: ids, x, y")
    if w.desc.format in F4_BLOCK:
        _f4_stacked(w.desc.format, *w._keep, n_experts, w.n, w.k,
                    "tq_linear_experts_f4")
    t = ids.shape[0]
    if x.shape[0] < t or y.shape[0] < t or x.shape[1] < w.k or \
            y.shape[1] < w.n:
        raise TqError(TQ_ERR_SHAPE, "tq_linear_experts_f4: x, y")
    st = _lib.tq_linear_experts_f4(w.ref, n_experts, ids.data_ptr(),
                                   t, x.data_ptr(), _rows(x), y.data_ptr(),
                                   _rows(y), _ptr(status),
                                   _stream(stream, dev))
    if check:
        _check(st, "tq_linear_experts_f4")
    return st
