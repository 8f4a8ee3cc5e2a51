"""Plain implementations of the 8-bit operators (numpy, 64 bits unless the
operator's definition fixes the arithmetic), and the inputs of their tests."""
import numpy as np

EPS24 = 2.0 ** -24          # half a step of fp32, relative


def bf16_round(v):
    """fp32/fp64 -> the nearest bf16 value (ties to even), as fp32.  The fp64
    value is rounded once: to odd in fp32 first, then to nearest."""
    v = np.asarray(v, np.float64)
    f = v.astype(np.float32)
    u = f.view(np.uint32).astype(np.int64)
    inexact = f.astype(np.float64) != v
    too_far = np.abs(f.astype(np.float64)) > np.abs(v)      # rounded away: step back towards zero
    u = np.where(inexact & too_far, u - 1, u)
    u = np.where(inexact, u | 1, u)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16) << 16
    out = (r & 0xFFFFFFFF).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(v), out, f)


def round_to(v, kind):
    if kind == "fp32":
        return np.asarray(v, np.float64).astype(np.float32)
    if kind == "fp16":
        with np.errstate(over="ignore"):
            return np.asarray(v, np.float64).astype(np.float16).astype(np.float32)
    return bf16_round(v)


HALF_STEP = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"fp32": 2.0 ** -149, "fp16": 2.0 ** -25, "bf16": 2.0 ** -133}      # of the subnormal range


def codes_fp32(w, finite=None):
    """Codes of rows of fp32 values by the operators' definition, in fp32."""
    w = np.asarray(w, np.float32)
    with np.errstate(all="ignore"):
        a = np.abs(w).max(axis=1, initial=0.0).astype(np.float32)
        ok = np.isfinite(w).all(axis=1) if finite is None else finite
        pre = np.where(a < np.float32(2.0 ** -100), np.float32(2.0 ** 100), np.float32(1))
        inv = np.where(a > 0, np.float32(127) / (a * pre), np.float32(0)).astype(np.float32)
        v = (w * pre[:, None]).astype(np.float32) * inv[:, None]
        q = np.clip(np.rint(np.where(ok[:, None], v, 0)), -127, 127)
    return q.astype(np.int8), a, ok


def quant(x):
    """(codes, scales) of rows of values that fp32 holds exactly."""
    q, a, ok = codes_fp32(x)
    with np.errstate(all="ignore"):
        return q, np.where(ok, a / np.float32(127), np.float32(np.nan)).astype(np.float32)


def silu_mul(g, u):
    g, u = np.asarray(g, np.float64), np.asarray(u, np.float64)
    with np.errstate(all="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def rmsnorm(h, delta, gamma, eps, kind):
    """(h', codes, fp64 scales)."""
    h = np.asarray(h, np.float64)
    if delta is not None:
        with np.errstate(all="ignore"):
            h = round_to(h + np.asarray(delta, np.float64), kind).astype(np.float64)
    with np.errstate(all="ignore"):
        w = (h.astype(np.float32) * np.asarray(gamma, np.float32)).astype(np.float32)
        ms = (h * h).sum(axis=1)
        ok = np.isfinite(w).all(axis=1) & (ms < 3.4028235e38)
        a = np.abs(w).max(axis=1).astype(np.float64)
        s = np.where(ok, a / np.sqrt(ms / h.shape[1] + eps) / 127.0, np.nan)
        ok &= np.isfinite(s)
        q, _, _ = codes_fp32(w, ok)
    return h, q, np.where(ok, s, np.nan)


def linear(w, sw, x, sx):
    """fp64 product (the integer sum is exact: below 2^53)."""
    return (x.astype(np.float64) @ w.astype(np.float64).T) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
