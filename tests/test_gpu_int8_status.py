"""GPU tests of the integer product's bounded waits: their limits count the
waits of one call, not the time of the kernels before it or of its own other
tiles, and one call's failure is told once and touches no other call."""
import pytest

torch = pytest.importorskip("torch")

from lut_binary_basis_b200 import fluxbin  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    fluxbin.fluxbin_device_status()


def problem(T, M, N, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)

    def codes(rows):
        return torch.randint(-128, 128, (rows, N), generator=g, device="cuda", dtype=torch.int8)

    layer = fluxbin.Int8Layer(codes(M), torch.exp(0.3 * torch.randn(M, generator=g, device="cuda")))
    rows = fluxbin.QuantRows(codes(T), torch.exp(0.3 * torch.randn(T, generator=g, device="cuda")))
    want = (rows.q.double() @ layer.w.double().t()).float() * (rows.scale[:, None] * layer.scale)
    return layer, rows, want


@pytest.mark.parametrize("T,M,N", [(20, 11008, 4096), (1, 30000, 512), (300, 9024, 512), (448, 14336, 128)])
def test_behind_long_kernels(T, M, N):
    """Products that are launched while kernels of several milliseconds still run."""
    layer, rows, want = problem(T, M, N)
    big, brows = fluxbin.Int8Layer(torch.ones(8192, 8192, dtype=torch.int8, device="cuda"), torch.ones(8192, device="cuda")), \
        fluxbin.QuantRows(torch.ones(65536, 8192, dtype=torch.int8, device="cuda"), torch.ones(65536, device="cuda"))
    by = torch.empty(65536, 8192, dtype=torch.bfloat16, device="cuda")
    ys = [torch.full((T, M), float("nan"), device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        big.linear(brows, by)
        layer.linear(rows, y, fluxbin.FLAG_EARLY_WEIGHTS if i % 2 else 0)
        layer.linear(rows, y)
    torch.cuda.synchronize()
    assert fluxbin.fluxbin_device_status() == 0
    for y in ys:
        assert torch.equal(y, want)
    assert bool((by[::4097] == 8192).all())


@pytest.mark.parametrize("T,M,N", [(20, 300, 4096), (1, 30000, 512), (300, 9024, 512), (448, 14336, 128)])
def test_a_failed_call_between_others(T, M, N):
    """The give-up path (test hook) between ordinary calls on one stream: NaN in
    its own y only, bit 0 alone, and the tensor memory is there for the next."""
    layer, rows, want = problem(T, M, N, 1)
    ys = [torch.zeros(T, M, device="cuda") for _ in range(9)]
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        layer.linear(rows, y, fluxbin.FLAG_TEST_WAIT_TIMEOUT if i % 3 == 1 else 0)
    torch.cuda.synchronize()
    assert fluxbin.fluxbin_device_status() == 1
    assert fluxbin.fluxbin_device_status() == 0
    for i, y in enumerate(ys):
        assert bool(torch.isnan(y).all()) if i % 3 == 1 else torch.equal(y, want)
