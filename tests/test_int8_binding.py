"""Checks of the 8-bit layers' Python binding (no GPU needed)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lut_binary_basis_b200 import fluxbin  # noqa: E402


@pytest.mark.parametrize("dtype,flags", [
    (torch.float16, fluxbin.FLAG_Y_FP32), (torch.float16, fluxbin.FLAG_BF16), (torch.bfloat16, fluxbin.FLAG_Y_FP32),
    (torch.float32, fluxbin.FLAG_BF16), (torch.float16, fluxbin.FLAG_Y_FP32 | fluxbin.FLAG_ACCUMULATE),
    (torch.bfloat16, fluxbin.FLAG_Y_FP32 | fluxbin.FLAG_BF16)])
def test_type_flags_that_are_not_ys_type(dtype, flags):
    """FLAG_Y_FP32 with a 16-bit y would write twice y's bytes."""
    layer = fluxbin.Int8Layer(torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8))
    rows = fluxbin.QuantRows(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError, match="flags"):
        layer.linear(rows, torch.zeros(4, 8, dtype=dtype), flags)


@pytest.mark.parametrize("dtype,flags", [(torch.float32, fluxbin.FLAG_Y_FP32), (torch.bfloat16, fluxbin.FLAG_BF16),
                                         (torch.float16, fluxbin.FLAG_ACCUMULATE)])
def test_type_flags_that_are_ys_type(dtype, flags):
    layer = fluxbin.Int8Layer(torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8))
    rows = fluxbin.QuantRows(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError, match="not on a CUDA device"):       # the next check
        layer.linear(rows, torch.zeros(4, 8, dtype=dtype), flags)


@pytest.mark.parametrize("rows", [[[1e39, 0.0], [1.0, 2.0]], [[1.0, 2.0], [-4.4e40, 1.0]], [[1e300, 1.0]]])
def test_from_host_rows_beyond_an_fp32_scale(rows):
    """127 times the largest fp32 is 4.3e40; 1e39 / 127 still has a scale."""
    W = np.array(rows)
    if np.abs(W).max() < 4.3e40:
        layer = fluxbin.Int8Layer.from_host(W, "cpu")
        assert np.isfinite(layer.scale.numpy()).all() and layer.w[0].tolist() == [127, 0]
    else:
        with pytest.raises(ValueError, match="fp32"):
            fluxbin.Int8Layer.from_host(W, "cpu")


@pytest.mark.parametrize("tiny", [5e-324, 1e-310, 1e-300, 1e-45, 8e-44])
def test_from_host_rows_below_fp32(tiny):
    """A row whose scale is 0 in fp32 is a row of zeros (0.7e-45 is half of
    fp32's smallest, times 127 is 8.9e-44); the other row is untouched."""
    with np.errstate(all="raise", under="ignore"):
        layer = fluxbin.Int8Layer.from_host(np.array([[tiny, -tiny, 0.0], [1.0, -2.0, 0.5]]), "cpu")
    assert layer.scale[0].item() == 0 and not layer.w[0].any()
    assert layer.w[1].tolist() == [64, -127, 32] and layer.scale[1].item() == np.float32(2 / 127)


def test_from_host_small_scales():
    """A scale below fp32's normal range is rounded to a multiple of 2^-149: 127
    times half of that comes on top of half a code."""
    g = np.random.default_rng(3)
    W = g.uniform(-1, 1, (64, 33)) * 10.0 ** g.uniform(-43, -36, (64, 1))
    layer = fluxbin.Int8Layer.from_host(W, "cpu")
    q, s = layer.w.numpy().astype(np.float64), layer.scale.numpy().astype(np.float64)
    assert (s > 0).all() and np.abs(q).max() <= 127
    assert np.all(np.abs(q * s[:, None] - W) <= 0.5 * s[:, None] * (1 + 1e-6) + 127 * 2.0 ** -150)
