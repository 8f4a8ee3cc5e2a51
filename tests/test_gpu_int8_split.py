"""GPU tests of fluxbin_int8_linear where a cluster shares a tile's K and has
fewer tokens than warps, or lanes past the end of M: calls that follow and
overlap each other, so that a CTA's shared memory is taken over as soon as it
ends.  The result is fixed to the bit (see the reference below)."""
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
    yield
    assert fluxbin.fluxbin_device_status() == 0, "a bounded wait gave up"


def problem(T, M, N, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def codes(rows):
        buf = torch.zeros(rows, -(-N // 16) * 16, device="cuda", dtype=torch.int8)
        buf[:, :N] = torch.randint(-128, 128, (rows, N), generator=g, device="cuda", dtype=torch.int8)
        return buf[:, :N]

    layer = fluxbin.Int8Layer(codes(M), torch.exp(0.3 * torch.randn(M, generator=g, device="cuda")))
    rows = fluxbin.QuantRows(codes(T), torch.exp(0.3 * torch.randn(T, generator=g, device="cuda")))
    # the exact sum rounded to fp32, times the product of the scales: one rounding each
    want = (rows.q.double() @ layer.w.double().t()).float() * (rows.scale[:, None] * layer.scale)
    return layer, rows, want


@pytest.mark.parametrize("T", [1, 2, 3, 5, 7, 9, 17, 40])
@pytest.mark.parametrize("M,N", [(5, 12000), (129, 9000), (333, 20000), (4801, 1030), (5000, 4096), (11008, 4096)])
def test_few_tokens_of_a_split_tile(T, M, N):
    layer, rows, want = problem(T, M, N, T + M)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [torch.full((T, M), float("nan"), device="cuda") for _ in range(24)]
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        layer.linear(rows, y, fluxbin.FLAG_EARLY_WEIGHTS if i % 3 else 0, stream=streams[i // 2 % 2])
    torch.cuda.synchronize()
    for y in ys:
        assert torch.equal(y, want)


def test_calls_of_different_splits_in_a_graph():
    calls = [problem(T, M, N, 7) for T, M, N in ((1, 333, 20000), (17, 11008, 4096), (3, 5, 12000), (200, 700, 3000))]
    ys = [torch.full_like(want, float("nan")) for _, _, want in calls]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(4):
            for (layer, rows, _), y in zip(calls, ys):
                layer.linear(rows, y)
    for _ in range(10):
        for y in ys:
            y.fill_(float("nan"))
        graph.replay()
        for (_, _, want), y in zip(calls, ys):
            assert torch.equal(y, want)
