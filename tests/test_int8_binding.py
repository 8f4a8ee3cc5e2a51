"""Checks of the 8-bit layers' Python binding (no GPU needed)."""
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
