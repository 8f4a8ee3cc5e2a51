"""GPU tests of binary layers that read what an 8-bit layer has just written,
with nothing in between: the same array of activations is rewritten before
every call, and each result is that of the same two calls with the GPU idle
between them.

Tolerance.  A layer split through the workspace adds its partial sums in an order
that varies between calls.  Adding P values in any order is off by at most
(P - 1) 2^-24 times the sum of their magnitudes, which is at most
A[m] = sum_k |r_k[m]| sum_n |c_k[n] x[n]| over both branches; here P is below 128
(a unit of the reduction has 64 columns or more, N is 4096), so two calls differ by
at most 2 * 128 * 2^-24 A < 2^-15 A.  (y itself is about A / sqrt(N), and stale
activations give another y altogether.)
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lut_binary_basis_b200 import fluxbin, synth  # noqa: E402
from test_gpu_parity import spec  # noqa: E402

pytestmark = pytest.mark.gpu

TC = fluxbin.FLAG_PATH_TC | fluxbin.FLAG_EARLY_WEIGHTS


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("sp,B,call", [
    (spec(4096, 4096, 2, 2, 123, 4), 16, TC), (spec(1000, 1024, 2, 1, 50, 8), 5, TC),      # tensor cores
    (spec(4096, 4096, 2, 1, 100, 8), 2, fluxbin.FLAG_EARLY_WEIGHTS), (spec(11008, 4096, 2, 1, 100, 8), 1, fluxbin.FLAG_EARLY_WEIGHTS),
    (spec(11008, 4096, 2, 1, 100, 8), 1, "norm")])
def test_activations_of_the_preceding_kernel(sp, B, call):
    host = synth.make_layer(sp, [7, sp.M])
    d = fluxbin.DeviceLayer.from_host(host)
    g = torch.Generator("cuda").manual_seed(sp.M)
    N, K = sp.N, 512
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    layer8 = fluxbin.Int8Layer(w, torch.full((N,), 1e-4, device="cuda"))
    rows = [fluxbin.QuantRows(torch.randint(-127, 128, (B, K), generator=g, device="cuda", dtype=torch.int8),
                              torch.rand(B, generator=g, device="cuda")) for _ in range(3)]
    x = torch.zeros(B, N, dtype=torch.float16, device="cuda")
    gamma = torch.rand(N, generator=g, device="cuda").half()
    ws = d.workspace(B) if call == "norm" else fluxbin.new_workspace(sp.M, B)

    def run(i, y, wait):
        layer8.linear(rows[i], x)
        if wait:
            torch.cuda.synchronize()
        if call == "norm":
            d.linear_rmsnorm(x, gamma, 1e-5, y, fluxbin.FLAG_Y_FP32 | fluxbin.FLAG_EARLY_WEIGHTS, ws)
        else:
            d.linear(x, y, fluxbin.FLAG_Y_FP32 | call, ws)

    def magnitude():
        v = x.double()
        if call == "norm":
            v = v * gamma.double() / torch.sqrt((v * v).mean(dim=1, keepdim=True) + 1e-5)
        v = v.abs().cpu().numpy()
        r, c, rs, cs = (np.abs(t.astype(np.float64)) for t in (host.r, host.c, host.rs, host.cs))
        return torch.from_numpy(v @ c.T @ r + v[:, host.sal_idx] @ cs.T @ rs).cuda()

    want, tol = [torch.zeros(B, sp.M, device="cuda") for _ in rows], []
    for i, y in enumerate(want):
        run(i, y, True)
        torch.cuda.synchronize()
        tol.append(2.0 ** -15 * magnitude())
    assert bool(((want[0] - want[1]).abs() > tol[0] + tol[1]).double().mean() > 0.9)      # it would show
    ys = [torch.zeros(B, sp.M, device="cuda") for _ in range(24)]
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        run(i % 3, y, False)
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        assert bool(((y.double() - want[i % 3].double()).abs() <= tol[i % 3]).all()), i
