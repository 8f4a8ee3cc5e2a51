"""The 8-bit operators beside the binary-basis layers, as cases that can be measured.

A case is one call: the 8-bit integer product with a scale for each token and
each channel ("linear"), the residual addition with the RMS normalisation and
an 8-bit output ("rmsnorm"), the MLP gate with an 8-bit output ("silu_mul") and
the plain row quantisation ("quant").  ``run`` computes it with elementary
torch operations, or (``own``) with the library's entry points.

Codes are returned as the values they stand for (code times row scale), in the
16-bit type of the operator's inputs.
"""
import math

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}

_T_MAX, _MN_MIN, _MN_MAX = 4096, 64, 28672
_WORK_MAX = 2048 * 28672 * 8192          # products of the largest listed linear


def listed():
    return [
        # decode of one sequence: a projection left out of binarisation, y chained in fp16
        dict(name="linear_1x4096x4096_fp16", op="linear", T=1, M=4096, N=4096, out="fp16", acc=False),
        # decode of one sequence: a large MLP projection, y in 32 bits
        dict(name="linear_1x28672x8192_fp32", op="linear", T=1, M=28672, N=8192, out="fp32", acc=False),
        # a decode batch at the layer size of the binary MLP
        dict(name="linear_16x11008x4096_fp16", op="linear", T=16, M=11008, N=4096, out="fp16", acc=False),
        # a short prompt of odd length on an odd-sized layer, added to a bf16 residual
        dict(name="linear_77x1003x2050_bf16_acc", op="linear", T=77, M=1003, N=2050, out="bf16", acc=True),
        # a prompt of a few hundred tokens, a ragged last tile
        dict(name="linear_333x4096x11008_fp16", op="linear", T=333, M=4096, N=11008, out="fp16", acc=False),
        # the prompts of a batch, a large MLP projection
        dict(name="linear_2048x28672x8192_bf16", op="linear", T=2048, M=28672, N=8192, out="bf16", acc=False),
        # decode of one sequence: the norm before a layer
        dict(name="rmsnorm_1x4096_fp16", op="rmsnorm", T=1, N=4096, dt="fp16", h="fp16"),
        # a prompt, the residual stream kept in 32 bits
        dict(name="rmsnorm_2048x8192_bf16_h32", op="rmsnorm", T=2048, N=8192, dt="bf16", h="fp32"),
        # a decode batch: the gate before the down projection
        dict(name="silu_mul_16x11008_fp16", op="silu_mul", T=16, N=11008, dt="fp16"),
        # a prompt: the gate of a large MLP
        dict(name="silu_mul_2048x28672_bf16", op="silu_mul", T=2048, N=28672, dt="bf16"),
        # decode batch of odd size: attention output before its projection
        dict(name="quant_7x4099_fp16", op="quant", T=7, N=4099, dt="fp16"),
        # a prompt's attention outputs
        dict(name="quant_4096x8192_fp16", op="quant", T=4096, N=8192, dt="fp16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "rmsnorm", "silu_mul", "quant"])
    T, N = _log_int(rng, 1, _T_MAX), _log_int(rng, _MN_MIN, _MN_MAX)
    if rng.random() < 0.5:
        N = max(_MN_MIN, N // 64 * 64)
    if op == "linear":
        M = _log_int(rng, _MN_MIN, _MN_MAX)
        if rng.random() < 0.5:
            M = max(_MN_MIN, M // 64 * 64)
        T = max(1, min(T, _WORK_MAX // (M * N)))
        return dict(op=op, T=T, M=M, N=N, out=rng.choice(["fp16", "bf16", "fp32"]), acc=rng.random() < 0.5)
    case = dict(op=op, T=min(T, 2048 * 28672 // N), N=N, dt=rng.choice(["fp16", "bf16"]))
    if op == "rmsnorm":
        case["h"] = rng.choice([case["dt"], "fp32"])
    return case


def _pitch(n):
    return -(-n // 16) * 16


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))
    T, N = case["T"], case["N"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def codes(rows):
        # rows of 16-byte pitch; the largest |code| is about four standard deviations
        buf = torch.zeros(rows, _pitch(N), dtype=torch.int8, device="cuda")
        for i in range(0, rows, 4096):
            part = buf[i:i + 4096, :N]
            part.copy_((normal(*part.shape) * 32.0).round_().clamp_(-127, 127))
        return buf[:, :N]

    st = {"case": dict(case)}
    if case["op"] == "linear":
        M, out = case["M"], _DT[case["out"]]
        st["w"] = codes(M)
        st["sw"] = torch.exp(0.3 * normal(M)) * (0.03 / math.sqrt(N))
        st["xq"] = codes(T)
        st["sx"] = torch.exp(0.3 * normal(T)) * 0.03
        st["y0"] = normal(T, M).to(out) if case["acc"] else None
        st["y"] = torch.empty(T, M, dtype=out, device="cuda")
        return st
    dt = _DT[case["dt"]]
    # a few outlier channels, as activations of language models have them
    outlier = torch.where(torch.rand(N, generator=g, device="cuda") < 0.005, 10.0, 1.0)
    if case["op"] == "rmsnorm":
        hd = _DT[case["h"]]
        st["h"] = (normal(T, N) * outlier * 2.0).to(hd)
        st["delta"] = normal(T, N).to(dt)
        st["gamma"] = (0.5 + torch.rand(N, generator=g, device="cuda")).to(dt)
        st["h_out"] = torch.empty(T, N, dtype=hd, device="cuda")
        st["eps"] = 1e-5
    elif case["op"] == "silu_mul":
        gu = normal(T, 2 * N)                       # one projection's output: gate, then up
        gu[:, N:] *= outlier
        gu = gu.to(dt)
        st["gate"], st["up"] = gu[:, :N], gu[:, N:]
    else:
        st["x"] = (normal(T, N) * outlier).to(dt)
    if T > 4:                                       # a padded batch: one row without a token
        row = T // 2
        for k in ("h", "delta", "gate", "up", "x"):
            if k in st:
                st[k][row] = 0
    st["q"] = torch.zeros(T, _pitch(N), dtype=torch.int8, device="cuda")[:, :N]
    st["scale"] = torch.empty(T, dtype=torch.float32, device="cuda")
    st["value"] = torch.empty(T, N, dtype=dt, device="cuda")
    return st


def _quantise(u, factor):
    """Codes and scales of rows of u; the rows stand for u * factor."""
    a = u.abs().amax(dim=1, keepdim=True)
    q = torch.round(u * torch.where(a > 0, 127.0 / a, torch.zeros_like(a)))
    return q, a * factor / 127.0


def _plain(st):
    case = st["case"]
    if case["op"] == "linear":
        acc = st["xq"].float() @ st["w"].float().t()
        y = acc * st["sx"][:, None] * st["sw"]
        if case["acc"]:
            y = st["y0"].float() + y
        return y.to(_DT[case["out"]])
    dt = _DT[case["dt"]]
    if case["op"] == "rmsnorm":
        h = (st["h"].float() + st["delta"].float()).to(_DT[case["h"]])
        f = h.float()
        r = 1.0 / torch.sqrt((f * f).mean(dim=1, keepdim=True) + st["eps"])
        q, s = _quantise(f * st["gamma"].float(), r)
        return h, (q * s).to(dt)
    if case["op"] == "silu_mul":
        gate = st["gate"].float()
        v = gate / (1.0 + torch.exp(-gate)) * st["up"].float()
    else:
        v = st["x"].float()
    q, s = _quantise(v, 1.0)
    return (q * s).to(dt)


def _library(st):
    from lut_binary_basis_b200 import fluxbin

    case = st["case"]
    if case["op"] == "linear":
        layer = st.get("layer")
        if layer is None:                           # pointers and sizes only
            layer = st["layer"] = fluxbin.Int8Layer(st["w"], st["sw"])
            st["rows"] = fluxbin.QuantRows(st["xq"], st["sx"])
        y = st["y"]
        if case["acc"]:
            y.copy_(st["y0"])                       # the residual that the call adds to
        layer.linear(st["rows"], y, fluxbin.FLAG_ACCUMULATE if case["acc"] else 0)
        return y
    rows = st.get("rows")
    if rows is None:
        rows = st["rows"] = fluxbin.QuantRows(st["q"], st["scale"])
    if case["op"] == "rmsnorm":
        rows.rmsnorm(st["h"], st["gamma"], st["eps"], delta=st["delta"], h_out=st["h_out"])
        return st["h_out"], torch.mul(rows.q, rows.scale[:, None], out=st["value"])
    if case["op"] == "silu_mul":
        rows.silu_mul(st["gate"], st["up"])
    else:
        rows.quantize(st["x"])
    return torch.mul(rows.q, rows.scale[:, None], out=st["value"])


def run(state):
    if own:
        return _library(state)
    return _plain(state)


def work(case):
    T, N = case["T"], case["N"]
    size = {"fp16": 2, "bf16": 2, "fp32": 4}
    if case["op"] == "linear":
        M = case["M"]
        return {"bytes": M * N + 4 * M + T * N + 4 * T + T * M * size[case["out"]] * (2 if case["acc"] else 1),
                "flops": 2 * T * M * N}
    # the values that the codes stand for are written in 16 bits beside them
    if case["op"] == "rmsnorm":
        return {"bytes": T * N * (2 * size[case["h"]] + 2 + 1 + 2) + 2 * N + 4 * T, "flops": 6 * T * N}
    if case["op"] == "silu_mul":
        return {"bytes": T * N * (4 + 1 + 2) + 4 * T, "flops": 7 * T * N}
    return {"bytes": T * N * (2 + 1 + 2) + 4 * T, "flops": 3 * T * N}


def exact(case, seed):
    st = prepare(case, seed)
    T, f8 = case["T"], torch.float64
    if case["op"] == "linear":
        w, out = st["w"].to(f8), torch.empty(T, case["M"], dtype=f8, device="cuda")
        for i in range(0, T, 512):
            dot = torch.einsum("tn,mn->tm", st["xq"][i:i + 512].to(f8), w)
            out[i:i + 512] = torch.einsum("tm,t,m->tm", dot, st["sx"][i:i + 512].to(f8), st["sw"].to(f8))
        if case["acc"]:
            out += st["y0"].to(f8)
        return out
    if case["op"] == "rmsnorm":
        h = torch.add(st["h"].to(f8), st["delta"].to(f8)).to(_DT[case["h"]]).to(f8)
        v = h * st["gamma"].to(f8) * torch.rsqrt(h.square().sum(dim=1) / case["N"] + st["eps"])[:, None]
    elif case["op"] == "silu_mul":
        v = st["gate"].to(f8) * torch.sigmoid(st["gate"].to(f8)) * st["up"].to(f8)
    else:
        v = st["x"].to(f8)
    step = v.abs().max(dim=1, keepdim=True).values / 127.0
    value = torch.where(step > 0, torch.round(v / step), 0.0) * step
    return (h, value) if case["op"] == "rmsnorm" else value
