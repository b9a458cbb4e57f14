"""Measured cases of the microscaled 4-bit float operators.

Two formats of 4-bit floats (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
negatives, two codes per byte, the lower k in the low four bits) with one
scale per block of consecutive k of a row:

  mx4   blocks of 32, E8M0 scale (a power of two): w = c 2^(b - 127)
  nv4   blocks of 16, E4M3 scale, one fp32 scale g per tensor: w = c s g

and the operators on them:

  quantize   bf16 matrix -> codes and scales, and back to bf16 (the round trip
             by which a user judges the format on a layer)
  linear     y = x W^T for bf16 x and 4-bit W (decode steps)
  product    y = x W^T with both sides in 4 bits (prompts, large batches)
  experts    y[t] = x[t] W_e^T, e = ids[t], for bf16 x (expert layers)

`own` chooses between plain torch operations and this repository's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = {"mx4": 32, "nv4": 16}
TABLE = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # a gate / up projection packed once when a model is loaded
        dict(name="quantize mx4 21504x5376", op="quantize", fmt="mx4",
             n=21504, k=5376, given=False, acts=False),
        # a q projection packed with a scale of its own, found on the way
        dict(name="quantize nv4 8192x5376", op="quantize", fmt="nv4",
             n=8192, k=5376, given=False, acts=False),
        # the activations of 37 rows before a 4-bit product, calibrated scale
        dict(name="quantize nv4 37x5376 given", op="quantize", fmt="nv4",
             n=37, k=5376, given=True, acts=True),
        # one decode step of one sequence through a q projection
        dict(name="linear mx4 8192x5376 b1", op="linear", fmt="mx4",
             n=8192, k=5376, batch=1),
        # four sequences through a down projection
        dict(name="linear nv4 5376x21504 b4", op="linear", fmt="nv4",
             n=5376, k=21504, batch=4),
        # a full decode batch through an up projection
        dict(name="linear mx4 21504x5376 b64", op="linear", fmt="mx4",
             n=21504, k=5376, batch=64),
        # a ragged layer at an odd batch
        dict(name="linear nv4 1003x4128 b13", op="linear", fmt="nv4",
             n=1003, k=4128, batch=13),
        # a long prompt through an up projection
        dict(name="product mx4 21504x5376 t2048", op="product", fmt="mx4",
             n=21504, k=5376, batch=2048, y="bf16"),
        # an odd prompt length through an o projection
        dict(name="product nv4 5376x8192 t777", op="product", fmt="nv4",
             n=5376, k=8192, batch=777, y="fp32"),
        # a decode batch with quantized activations
        dict(name="product mx4 8192x5376 t16", op="product", fmt="mx4",
             n=8192, k=5376, batch=16, y="fp32"),
        # the routed rows of a decode step over an expert layer
        dict(name="experts mx4 128x768x2048 r64", op="experts", fmt="mx4",
             e=128, n=768, k=2048, rows=64),
        # a larger batch, several rows for each expert
        dict(name="experts nv4 128x768x2048 r500", op="experts", fmt="nv4",
             e=128, n=768, k=2048, rows=500),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "linear", "product", "experts"))
    fmt = rng.choice(("mx4", "nv4"))
    if op == "experts":
        e = _log(rng, 2, 128)
        k = 32 * _log(rng, 2, 64)
        n = _log(rng, 16, 768)
        return dict(op=op, fmt=fmt, e=e, n=n, k=k, rows=_log(rng, 1, 500))
    k = 32 * _log(rng, 2, 672)
    n = _log(rng, 16, min(21504, 21504 * 5376 // k))
    if op == "quantize":
        acts = rng.random() < 0.5
        return dict(op=op, fmt=fmt, n=n, k=k, acts=acts,
                    given=fmt == "nv4" and rng.random() < 0.5)
    if op == "linear":
        return dict(op=op, fmt=fmt, n=n, k=k, batch=_log(rng, 1, 64))
    return dict(op=op, fmt=fmt, n=n, k=k, batch=_log(rng, 1, 2048),
                y=rng.choice(("fp32", "bf16")))


def work(case):
    fmt, n, k = case["fmt"], case["n"], case["k"]
    bits4 = n * k * (0.5 + 1.0 / BLOCK[fmt])  # codes and scales of the matrix
    if case["op"] == "quantize":  # bf16 in, package out; package in, bf16 out
        return {"bytes": 4.0 * n * k + 2 * bits4, "flops": 0.0}
    if case["op"] == "linear":
        b = case["batch"]
        return {"bytes": bits4 + 2.0 * b * k + 4.0 * b * n,
                "flops": 2.0 * b * n * k}
    if case["op"] == "product":
        b = case["batch"]
        return {"bytes": bits4 + b * k * (0.5 + 1.0 / BLOCK[fmt]) +
                (2.0 if case["y"] == "bf16" else 4.0) * b * n,
                "flops": 2.0 * b * n * k}
    t = case["rows"]
    used = case["e"] * (1 - (1 - 1 / case["e"]) ** t)  # distinct experts drawn
    return {"bytes": used * bits4 + 2.0 * t * k + 4.0 * t * n,
            "flops": 2.0 * t * n * k}


# ---- inputs --------------------------------------------------------------------

def _weights(g, n, k):
    """bf16 weights: normal times a heavy-tailed factor of each value."""
    w = torch.randn(n, k, generator=g, device=DEV)
    u = torch.rand(n, k, generator=g, device=DEV)
    return (0.02 * w * (1.0 - u).clamp_min(1e-4).pow(-0.2)).to(torch.bfloat16)


def _acts(g, rows, k):
    """bf16 activations: normal, with a few channels that run hot."""
    x = torch.randn(rows, k, generator=g, device=DEV)
    hot = 1.0 + 15.0 * (torch.rand(k, generator=g, device=DEV) < 0.005)
    return (x * hot).to(torch.bfloat16)


def _tensor_scale(w):
    return (w.abs().max().double() / 2688.0).float().clamp_min(1e-30) \
        .reshape(1)


def _pack(codes):
    """4-bit codes [n][k] uint8 -> [n][k / 2], the lower k in the low bits."""
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _package(w, fmt):
    """(packed codes, scale bytes, g) of a bf16 matrix."""
    g = _tensor_scale(w) if fmt == "nv4" else None
    codes, scales = _quantize(w, fmt, g)
    return _pack(codes), scales, g


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op, fmt, n, k = case["op"], case["fmt"], case["n"], case["k"]
    s = {"op": op, "fmt": fmt, "n": n, "k": k}
    if op == "quantize":
        s["w"] = _acts(gen, n, k) if case["acts"] else _weights(gen, n, k)
        # a calibrated scale is near, but not at, this matrix's own
        s["g"] = _tensor_scale(s["w"]) * 1.07 if case["given"] else None
    elif op == "experts":
        e, t = case["e"], case["rows"]
        w = _weights(gen, e * n, k)
        gs = None
        if fmt == "nv4":
            gs = (w.view(e, -1).abs().amax(1).double() / 2688.0).float()
        codes, scales = _quantize(
            w, fmt, None if gs is None else gs.repeat_interleave(n)[:, None])
        s.update(e=e, codes=_pack(codes), scales=scales, g=gs,
                 x=_acts(gen, t, k),
                 ids=torch.randint(0, e, (t,), generator=gen, device=DEV,
                                   dtype=torch.int32))
    else:
        s["codes"], s["scales"], s["g"] = _package(_weights(gen, n, k), fmt)
        x = _acts(gen, case["batch"], k)
        if op == "linear":
            s["x"] = x
        else:
            s["xcodes"], s["xscales"], s["xg"] = _package(x, fmt)
            s["y"] = case["y"]
    if own:
        _plan(s)
    return s


def _plan(s):
    """The descriptors and buffers that a program using the library keeps."""
    from packed_weight_matmul_b200 import tq
    op, n, k = s["op"], s["n"], s["k"]
    s["tq"] = tq

    def desc(codes, scales, g, rows):
        return (tq.weights_mx4(codes, scales, rows, k) if s["fmt"] == "mx4"
                else tq.weights_nv4(codes, scales, g, rows, k))

    if op == "quantize":
        s["codes"] = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.empty(n, k // BLOCK[s["fmt"]], dtype=torch.uint8,
                                  device=DEV)
        s["out"] = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
        s["gout"] = s["g"] if s["g"] is not None else \
            torch.empty(1, device=DEV)
        s["h"] = desc(s["codes"], s["scales"], s["gout"], n)
        return
    s["h"] = desc(s["codes"], s["scales"], s["g"], n)
    if op == "product":
        t = s["xcodes"].shape[0]
        s["hx"] = desc(s["xcodes"], s["xscales"], s["xg"], t)
        s["out"] = torch.empty(t, n, device=DEV, dtype=torch.bfloat16
                               if s["y"] == "bf16" else torch.float32)
    else:
        s["out"] = torch.empty(s["x"].shape[0], n, device=DEV)


# ---- one pass --------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "quantize":
        g = s["g"]
        if s["fmt"] == "nv4" and g is None:
            g = (s["w"].abs().max().double() / 2688.0).float().reshape(1)
        codes, scales = _quantize(s["w"], s["fmt"], g)
        return [_values(codes, scales, g, s["fmt"]).to(torch.bfloat16),
                _scale_type(scales, s["fmt"])]
    w = _decode(s["codes"], s["scales"], s["g"], s["fmt"], s.get("e"))
    if op == "linear":
        return s["x"].float() @ w.t()
    if op == "product":
        y = _decode(s["xcodes"], s["xscales"], s["xg"], s["fmt"]) @ w.t()
        return y.to(torch.bfloat16) if s["y"] == "bf16" else y
    picked = w.view(s["e"], s["n"], s["k"])[s["ids"].long()]
    return torch.bmm(picked, s["x"].float()[:, :, None])[:, :, 0]


def _run_own(s):
    tq, op = s["tq"], s["op"]
    if op == "quantize":
        fmt = tq.TQ_FMT_MX4 if s["fmt"] == "mx4" else tq.TQ_FMT_NV4
        tq.tq_quantize_f4(s["w"], fmt, s["codes"], s["scales"],
                          tensor_scale=s["gout"] if s["fmt"] == "nv4" else
                          None, scale_given=s["g"] is not None)
        tq.tq_unpack(s["h"], s["out"])
        return [s["out"], _scale_type(s["scales"], s["fmt"])]
    if op == "linear":
        tq.tq_linear(s["h"], s["x"], s["out"])
    elif op == "product":
        tq.tq_linear_f4(s["h"], s["hx"], s["out"])
    else:
        tq.tq_linear_experts_f4(s["h"], s["e"], s["ids"], s["x"], s["out"])
    return s["out"]


def _scale_type(scales, fmt):
    return scales.view(torch.float8_e8m0fnu if fmt == "mx4"
                       else torch.float8_e4m3fn)


# ---- the plain forms ---------------------------------------------------------------

def _e4m3_bytes(r):
    """Non-negative fp64 -> E4M3 byte, nearest even, at most 448."""
    e = (torch.frexp(r)[1] - 1).clamp_min(-6)
    m = torch.round(torch.ldexp(r, 3 - e))  # 8..16 units, below 8 subnormal
    up = m >= 16
    m, e = torch.where(up, m / 2, m), torch.where(up, e + 1, e)
    byte = torch.where(m >= 8, (e + 7) * 8 + (m - 8), m)
    return byte.clamp_max(126).to(torch.uint8)


def _quantize(w, fmt, g):
    """4-bit codes [n][k] and scale bytes of a bf16 matrix. Quotients are
    taken in 64 bits, so that values next to a border fall on its right side."""
    n, k = w.shape
    v = w.view(n, -1, BLOCK[fmt])
    a = v.abs()
    top = a.amax(2)
    if fmt == "mx4":
        e = (torch.frexp(top.float())[1] - 3).clamp(-127, 125)
        e = torch.where(top == 0, torch.full_like(e, -127), e)
        scales = (e + 127).to(torch.uint8)
        d = torch.ldexp(torch.ones_like(e, dtype=torch.float64), e)
    else:
        g64 = g.double()
        scales = _e4m3_bytes(top.double() / (6.0 * g64))
        d = scales.view(torch.float8_e4m3fn).double() * g64
    q = a.double() / d[:, :, None]
    q = torch.where(d[:, :, None] == 0, torch.zeros_like(q), q)
    code = ((q > 0.25).to(torch.uint8) + (q >= 0.75) + (q > 1.25) +
            (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5.0))
    code = code.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    return code.view(n, k), scales


def _values(codes, scales, g, fmt):
    """fp32 weights of 4-bit codes [n][k]."""
    n, k = codes.shape
    table = torch.tensor(TABLE + tuple(-t for t in TABLE), device=codes.device)
    w = table[codes.int()].view(n, -1, BLOCK[fmt])
    w = w * _scale_type(scales, fmt).float()[:, :, None]
    if g is not None:
        w = w * g.view(-1, 1, 1)
    return w.view(n, k)


def _decode(packed, scales, g, fmt, experts=None):
    codes = torch.stack((packed & 15, packed >> 4), 2).view(packed.shape[0],
                                                            -1)
    if experts is not None and g is not None:
        g = g.repeat_interleave(packed.shape[0] // experts)
    return _values(codes, scales, g, fmt)


# ---- 64 bits -----------------------------------------------------------------------

def _exact_weights(packed, scales, g, fmt):
    """Signs, exponents and mantissas put together in fp64."""
    lo_hi = torch.empty(packed.shape[0], packed.shape[1] * 2,
                        dtype=torch.int32, device=packed.device)
    lo_hi[:, 0::2] = packed.int() % 16
    lo_hi[:, 1::2] = packed.int() // 16
    e, m = lo_hi // 2 % 4, lo_hi % 2
    half = torch.where(e > 0, 2 + m, m).double() / 2
    w = torch.ldexp(half, (e - 1).clamp_min(0)) * (1 - lo_hi // 8 * 2)
    b = scales.int()
    if fmt == "mx4":
        s = torch.exp2(b.double() - 127)
    else:
        s = torch.where(b >= 8, torch.ldexp(1 + (b % 8).double() / 8,
                                            b // 8 - 7),
                        (b % 8).double() / 512)
    w = w * s.repeat_interleave(BLOCK[fmt], 1)
    return w if g is None else w * g.double().view(-1, 1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op, fmt = s["op"], s["fmt"]
    if op == "quantize":
        return _exact_quantize(s)
    if op == "experts":
        e, n, t = s["e"], s["n"], s["x"].shape[0]
        y = torch.empty(t, n, dtype=torch.float64, device=DEV)
        for i in range(e):
            at = (s["ids"] == i).nonzero()[:, 0]
            w = _exact_weights(s["codes"][i * n:(i + 1) * n],
                               s["scales"][i * n:(i + 1) * n],
                               None if s["g"] is None else s["g"][i:i + 1],
                               fmt)
            y[at] = s["x"][at].double() @ w.t()
        return y
    w = _exact_weights(s["codes"], s["scales"], s["g"], fmt)
    if op == "linear":
        return s["x"].double() @ w.t()
    return _exact_weights(s["xcodes"], s["xscales"], s["xg"], fmt) @ w.t()


def _exact_quantize(s):
    fmt, w = s["fmt"], s["w"].double()
    n, k = w.shape
    size = BLOCK[fmt]
    v = w.view(n, k // size, size)
    top = v.abs().max(2).values
    if fmt == "mx4":
        e = torch.floor(torch.log2(top))  # may be one off next to a power
        e = e + (torch.exp2(e + 1) <= top) - (torch.exp2(e) > top)
        scale = torch.exp2(e - 2).clamp(2.0 ** -127, 2.0 ** 125)
        unit = scale
    else:
        g = s["g"]
        if g is None:
            g = (w.abs().max() / 2688.0).float().reshape(1)
        g = g.double()
        r = top / (6.0 * g)
        step = torch.exp2(torch.floor(torch.log2(r.clamp_min(2.0 ** -6))) - 3)
        scale = (torch.round(r / step) * step).clamp_max(448.0)
        unit = scale * g
    q = v / unit[:, :, None]
    q = torch.where(unit[:, :, None] == 0, torch.zeros_like(q), q)
    step = torch.where(q.abs() >= 4, 2.0, torch.where(q.abs() >= 2, 1.0, 0.5))
    q = (torch.round(q / step) * step).clamp(-6.0, 6.0)
    return [(q * unit[:, :, None]).view(n, k), scale]
