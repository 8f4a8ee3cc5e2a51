"""GPU tests that fluxbin_int8_linear reads what the kernel before it wrote:
the same arrays of codes and scales, of activations and of weights, are
rewritten by a quantiser before every product, with nothing in between (the
product is already running when the quantiser writes them)."""
import pytest

torch = pytest.importorskip("torch")

from lut_binary_basis_b200 import fluxbin  # noqa: E402

pytestmark = pytest.mark.gpu

# the kernel for few tokens, split tiles, whole tiles, pairs (with one tile and with several)
SHAPES = [(1, 700, 1000), (16, 4000, 2048), (9, 300, 9000), (40, 1000, 1500), (1, 30000, 512), (20, 30000, 512), (300, 9000, 500),
          (448, 14336, 128)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    fluxbin.fluxbin_device_status()
    yield
    assert fluxbin.fluxbin_device_status() == 0, "a bounded wait gave up"


def quantised(values):
    rows = fluxbin.QuantRows.empty(*values.shape)
    rows.quantize(values)
    torch.cuda.synchronize()
    return rows


def want(x, w):
    # the exact sum (below 2^53) rounded to fp32, times the product of the scales: one rounding each
    return torch.cat([(x.q[t:t + 64].double() @ w.q.double().t()).float() * (x.scale[t:t + 64, None] * w.scale)
                      for t in range(0, x.T, 64)])


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T,M,N", SHAPES)
def test_codes_and_scales_of_the_preceding_kernel(T, M, N, captured):
    g = torch.Generator("cuda").manual_seed(T)

    def values(rows):
        # every row another scale, every time
        return torch.randn(rows, N, generator=g, device="cuda") * torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))

    xs, ws = [values(T).half() for _ in range(3)], [values(M).half() for _ in range(2)]
    xq, wq = [quantised(x) for x in xs], [quantised(w) for w in ws]
    x, w = fluxbin.QuantRows.empty(T, N), fluxbin.QuantRows.empty(M, N)
    layer = fluxbin.Int8Layer(w.q, w.scale)
    ys = [torch.full((T, M), float("nan"), device="cuda") for _ in range(12)]

    def calls():
        for i, y in enumerate(ys):
            if i % 4 == 0:
                x.quantize(xs[i % 3])
                w.quantize(ws[i // 4 % 2])          # the weights last
            else:
                x.quantize(xs[i % 3])
            layer.linear(x, y)

    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
        graph.replay()
        graph.replay()
    else:
        calls()
    for i, y in enumerate(ys):
        assert torch.equal(y, want(xq[i % 3], wq[i // 4 % 2])), i
