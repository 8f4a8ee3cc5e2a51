"""Refusals of the 8-bit operators (no GPU needed): argument errors come back
as status codes before any CUDA call, and the binding's own checks raise."""
import numpy as np
import pytest

from lut_binary_basis_b200 import fluxbin
import int8_reference as ref

Q, S, X, U, H, G, D, W, WS, Y = (0x10000000 * i for i in range(1, 11))     # far apart, 16-byte aligned
BIG = 131071


def quant(T=4, N=32, x=X, ldx=32, q=Q, ldq=32, s=S, flags=0):
    return fluxbin.lib().fluxbin_quant_rows(T, N, x, ldx, q, ldq, s, flags, None)


def silu(T=4, N=32, g=X, ldg=32, u=U, ldu=32, q=Q, ldq=32, s=S, flags=0):
    return fluxbin.lib().fluxbin_silu_mul_quant(T, N, g, ldg, u, ldu, q, ldq, s, flags, None)


def norm(T=4, N=32, h=H, ldh=32, d=D, ldd=32, g=G, eps=1e-5, o=None, ldo=0, q=Q, ldq=32, s=S, flags=0):
    return fluxbin.lib().fluxbin_rmsnorm_quant(T, N, h, ldh, d, ldd, g, eps, o, ldo, q, ldq, s, flags, None)


def linear(M=32, N=32, w=W, ldw=32, ws=WS, x=Q, ldx=32, xs=S, T=4, y=Y, ldy=32, flags=0):
    return fluxbin.lib().fluxbin_int8_linear(M, N, w, ldw, ws, x, ldx, xs, T, y, ldy, flags, None)


INVALID, SHAPE, MISALIGNED, UNSUPPORTED = -1, -2, -3, -4


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 0), (dict(T=0, x=0, q=0, s=0), 0),
    (dict(T=-1), SHAPE), (dict(N=-1), SHAPE), (dict(ldx=31), SHAPE), (dict(ldq=31), SHAPE), (dict(ldx=-32), SHAPE),
    (dict(ldx=1 << 41), SHAPE), (dict(N=BIG + 1, ldx=BIG + 1, ldq=BIG + 1), UNSUPPORTED),
    (dict(x=0), INVALID), (dict(q=0), INVALID), (dict(s=0), INVALID),
    (dict(flags=fluxbin.FLAG_ACCUMULATE), INVALID), (dict(flags=fluxbin.FLAG_H_FP32), INVALID), (dict(flags=1 << 20), INVALID),
    (dict(x=X + 1), MISALIGNED), (dict(q=Q + 8), MISALIGNED), (dict(s=S + 2), MISALIGNED), (dict(ldq=40), MISALIGNED),
    (dict(q=X), INVALID), (dict(s=X), INVALID), (dict(s=Q + 96), INVALID), (dict(q=X + 240), INVALID),
])
def test_quant_rows_refusals(kw, status):
    assert quant(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 0), (dict(T=-1), SHAPE), (dict(ldg=31), SHAPE), (dict(ldu=31), SHAPE), (dict(ldq=16), SHAPE),
    (dict(g=0), INVALID), (dict(u=0), INVALID), (dict(q=0), INVALID), (dict(s=0), INVALID),
    (dict(u=U + 1), MISALIGNED), (dict(g=X + 1), MISALIGNED), (dict(q=U), INVALID), (dict(q=X), INVALID),
    (dict(flags=fluxbin.FLAG_EARLY_WEIGHTS), INVALID), (dict(N=BIG + 1, ldg=BIG + 1, ldu=BIG + 1, ldq=BIG + 1), UNSUPPORTED),
])
def test_silu_mul_quant_refusals(kw, status):
    assert silu(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 0), (dict(T=-1), SHAPE), (dict(N=0), SHAPE), (dict(ldh=31), SHAPE), (dict(ldd=31), SHAPE),
    (dict(ldd=31, d=None, h=0), INVALID), (dict(o=Y, ldo=31), SHAPE), (dict(h=0), INVALID), (dict(g=0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(flags=fluxbin.FLAG_Y_FP32), INVALID), (dict(h=H + 2, flags=fluxbin.FLAG_H_FP32), MISALIGNED),
    (dict(o=Y + 2, ldo=32, flags=fluxbin.FLAG_H_FP32), MISALIGNED), (dict(o=Y + 1, ldo=32), MISALIGNED),
    (dict(g=G + 1), MISALIGNED), (dict(d=D + 1), MISALIGNED), (dict(q=Q + 4), MISALIGNED),
    (dict(o=H, ldo=48), INVALID), (dict(o=H + 2, ldo=32), INVALID), (dict(o=D, ldo=32), INVALID), (dict(o=G, ldo=32), INVALID),
    (dict(q=H), INVALID), (dict(q=G), INVALID), (dict(o=Q, ldo=32), INVALID), (dict(s=D), INVALID),
    (dict(N=BIG + 1, ldh=BIG + 1, ldd=BIG + 1, ldq=BIG + 1), UNSUPPORTED),
])
def test_rmsnorm_quant_refusals(kw, status):
    assert norm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 0), (dict(M=0), 0), (dict(T=0, x=0, xs=0, y=0), 0),
    (dict(T=-1), SHAPE), (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(ldw=16), SHAPE), (dict(ldx=16), SHAPE), (dict(ldy=31), SHAPE),
    (dict(M=(1 << 31) - 1, ldy=(1 << 31) - 1), UNSUPPORTED), (dict(T=(1 << 31) - 1), UNSUPPORTED),
    (dict(ldy=1 << 41), SHAPE), (dict(N=BIG + 1, ldw=BIG + 1, ldx=BIG + 1), UNSUPPORTED),
    (dict(w=0), INVALID), (dict(ws=0), INVALID), (dict(x=0), INVALID), (dict(xs=0), INVALID), (dict(y=0), INVALID),
    (dict(flags=fluxbin.FLAG_Y_FP32 | fluxbin.FLAG_BF16), INVALID), (dict(flags=fluxbin.FLAG_PATH_TC), INVALID),
    (dict(flags=fluxbin.FLAG_H_FP32), INVALID),
    (dict(w=W + 8), MISALIGNED), (dict(x=Q + 4), MISALIGNED), (dict(ldw=40), MISALIGNED), (dict(ldx=40), MISALIGNED),
    (dict(ws=WS + 2), MISALIGNED), (dict(xs=S + 2), MISALIGNED), (dict(y=Y + 1), MISALIGNED),
    (dict(y=Y + 2, flags=fluxbin.FLAG_Y_FP32), MISALIGNED),
    (dict(y=Q), INVALID), (dict(y=W + 512), INVALID), (dict(y=WS), INVALID), (dict(y=S), INVALID),
])
def test_int8_linear_refusals(kw, status):
    assert linear(**kw) == status


def test_other_entry_points_refuse_the_new_flags():
    desc = fluxbin.LayerDesc(32, 64, 2, 0, 0, 8, 0, 0)
    import ctypes
    for flag in (fluxbin.FLAG_BF16, fluxbin.FLAG_H_FP32):
        assert fluxbin.lib().fluxbin_linear(ctypes.byref(desc), 0x1000, 0x3000, 0x4000, None, None, None, None, 0x2000,
                                            1, 0x5000, flag, None, 0, None) == INVALID


def test_binding_checks_shapes_types_and_devices():
    torch = pytest.importorskip("torch")
    q = torch.zeros(4, 32, dtype=torch.int8)
    rows = fluxbin.QuantRows(q, torch.zeros(4))
    x = torch.zeros(4, 32, dtype=torch.float16)
    with pytest.raises(ValueError, match="not on a CUDA device"):
        rows.quantize(x)
    for bad in (torch.zeros(4, 31, dtype=torch.float16), torch.zeros(4, 32), torch.zeros(32, 4, dtype=torch.float16).t()):
        with pytest.raises(ValueError):
            rows.quantize(bad)
    with pytest.raises(ValueError):
        fluxbin.QuantRows(q, torch.zeros(3))
    with pytest.raises(ValueError):
        fluxbin.QuantRows(q.float(), torch.zeros(4))
    with pytest.raises(ValueError):
        rows.silu_mul(x, x.bfloat16())
    with pytest.raises(ValueError):
        rows.rmsnorm(x.bfloat16(), torch.ones(32, dtype=torch.float16), 1e-5)
    with pytest.raises(ValueError):
        rows.rmsnorm(x, torch.ones(32, dtype=torch.float16), 1e-5, h_out=x.float())
    layer = fluxbin.Int8Layer(torch.zeros(8, 48, dtype=torch.int8), torch.zeros(8))
    with pytest.raises(ValueError):
        layer.linear(rows, torch.zeros(4, 8))
    layer = fluxbin.Int8Layer(torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8))
    for bad in (torch.zeros(3, 8), torch.zeros(4, 8, dtype=torch.float64), torch.zeros(8, 4).t()):
        with pytest.raises(ValueError):
            layer.linear(rows, bad)
    e = fluxbin.QuantRows.empty(3, 21, "cpu")
    assert e.q.shape == (3, 21) and e.ldq == 32 and e.rows(2).T == 2
    for t in (4, -1):
        with pytest.raises(ValueError):
            e.rows(t)


def test_layer_from_host():
    torch = pytest.importorskip("torch")
    g = np.random.default_rng(5)
    W = g.standard_normal((7, 21))
    W[3] = 0
    layer = fluxbin.Int8Layer.from_host(W, "cpu")
    q, s = layer.w.numpy().astype(np.float64), layer.scale.numpy().astype(np.float64)
    # a weight is off by at most half a code, the scale by half a step of fp32
    assert np.all(np.abs(q * s[:, None] - W) <= 0.5 * s[:, None] * (1 + 1e-12) + np.abs(W) * 2.0 ** -23)
    assert layer.ldw == 32 and np.all(q[3] == 0) and s[3] == 0 and np.abs(q).max() == 127
    with pytest.raises(ValueError):
        fluxbin.Int8Layer.from_host(np.array([[np.nan, 1.0]]), "cpu")
    assert fluxbin.Int8Layer.from_host(np.zeros((2, 0)), "cpu").N == 0
    del torch


# --- the plain implementations themselves, with planted mistakes -------------

def test_reference_bf16_rounding():
    torch = pytest.importorskip("torch")
    g = np.random.default_rng(0)
    v = np.concatenate([g.standard_normal(4000) * 10.0 ** g.uniform(-38, 30, 4000), [0.0, -0.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8]])
    f = v.astype(np.float32)
    want = torch.from_numpy(f).bfloat16().float().numpy()
    assert np.array_equal(ref.bf16_round(f), want)
    # a tie that fp32 would have created: 1 + 2^-8 + 2^-30 lies above the midpoint
    assert ref.bf16_round(np.array([1 + 2.0 ** -8 + 2.0 ** -30]))[0] == np.float32(1 + 2.0 ** -7)


def test_reference_codes():
    q, a, ok = ref.codes_fp32(np.array([[1.0, -2.0, 0.5], [0, 0, 0], [np.nan, 1, 2], [np.inf, 1, 2], [1e-42, -2e-42, 0]]))
    assert q[0].tolist() == [64, -127, 32] and q[1].tolist() == [0, 0, 0]      # 63.5 -> 64, 31.75 -> 32
    assert not ok[2] and not ok[3] and q[2].tolist() == [0, 0, 0] and q[4].tolist()[1] == -127
