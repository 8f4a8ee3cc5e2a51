"""The package's names for the 8-bit operators (no GPU needed for the names)."""
import numpy as np
import pytest

import lut_binary_basis_b200 as package
from lut_binary_basis_b200 import fluxbin


def test_names():
    for name in ("Int8Layer", "QuantRows", "FLAG_BF16", "FLAG_H_FP32", "fluxbin_int8_linear", "fluxbin_quant_rows",
                 "fluxbin_rmsnorm_quant", "fluxbin_silu_mul_quant"):
        assert getattr(package, name) is getattr(fluxbin, name)


def test_functions_raise_the_library_status():
    for call in (lambda: package.fluxbin_quant_rows(1, 32, 0, 32, 0x1000, 32, 0x2000, 0, 0),
                 lambda: package.fluxbin_silu_mul_quant(1, 32, 0, 32, 0, 32, 0x1000, 32, 0x2000, 0, 0),
                 lambda: package.fluxbin_rmsnorm_quant(1, 32, 0, 32, None, 0, 0x4000, 1e-5, None, 0, 0x1000, 32, 0x2000, 0, 0),
                 lambda: package.fluxbin_int8_linear(8, 32, 0, 32, 0x4000, 0x1000, 32, 0x2000, 1, 0x8000, 8, 0, 0)):
        with pytest.raises(package.FluxbinError, match="INVALID_ARG"):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 33])
def test_functions_as_the_holders(T):
    """The four functions, with tensors and with plain pointers, on another stream."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    N, M = 320, 200
    g = torch.Generator("cuda").manual_seed(T)
    x, u, d = (torch.randn(T, N, generator=g, device="cuda").bfloat16() for _ in range(3))
    h, gamma = torch.randn(T, N, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda").bfloat16()
    h_out, want_h = torch.empty_like(h), torch.empty_like(h)
    layer = package.Int8Layer.from_host(np.random.default_rng(T).standard_normal((M, N)))
    a, b = package.QuantRows.empty(T, N), package.QuantRows.empty(T, N)
    y, want = torch.zeros(T, M, device="cuda"), torch.zeros(T, M, device="cuda")
    s = torch.cuda.Stream()

    def same():
        s.synchronize()
        torch.cuda.synchronize()
        return torch.equal(a.q, b.q) and torch.equal(a.scale, b.scale)

    torch.cuda.synchronize()
    b.quantize(x)
    package.fluxbin_quant_rows(T, N, x, N, a.q, a.ldq, a.scale, package.FLAG_BF16, s)
    assert same()
    b.silu_mul(x, u)
    package.fluxbin_silu_mul_quant(T, N, x.data_ptr(), N, u.data_ptr(), N, a.q.data_ptr(), a.ldq, a.scale.data_ptr(),
                                   package.FLAG_BF16, s.cuda_stream)
    assert same()
    b.rmsnorm(h, gamma, 1e-5, delta=d, h_out=want_h)
    package.fluxbin_rmsnorm_quant(T, N, h, N, d, N, gamma, 1e-5, h_out, N, a.q, a.ldq, a.scale,
                                  package.FLAG_BF16 | package.FLAG_H_FP32, s)
    assert same() and torch.equal(h_out, want_h)
    layer.linear(b, want)
    package.fluxbin_int8_linear(M, N, layer.w, layer.ldw, layer.scale, a.q, a.ldq, a.scale, T, y, M, package.FLAG_Y_FP32, s)
    assert same() and torch.equal(y, want) and bool((y != 0).any())
