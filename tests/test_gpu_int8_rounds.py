"""GPU tests of fluxbin_int8_linear where every pair of CTAs has several tiles:
the outputs of one tile leave shared memory while the next tile's are staged.

The result is fixed to the bit: the integer sum is exact (below 2^24 at these
N, so fp32 holds it), then one product of the scales, one with the sum, with
accumulation one addition, and one rounding to y's type, each of which torch
does with a single rounding too.

``tile`` and ``rounds`` are what the choice of a token tile gives on 148 SMs
(74 pairs, 256 channels a tile, 222 tiles unless said).  A group of output
warps has half of a tile's chunks, 32 tokens of a 16-bit y or 16 of a 32-bit
one: an odd number at tiles of 96, 160 and 224, in 16 bits at 192 too.
"""
import pytest

torch = pytest.importorskip("torch")

from lut_binary_basis_b200 import fluxbin  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


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
        return torch.randint(-128, 128, (rows, N), generator=g, device="cuda", dtype=torch.int8)

    def scales(n, typical):
        return torch.exp(0.3 * torch.randn(n, generator=g, device="cuda")) * typical

    return fluxbin.Int8Layer(codes(M), scales(M, 1e-3)), fluxbin.QuantRows(codes(T), scales(T, 1e-2)), g


def product(layer, rows):
    """The scaled product in fp32, before any accumulation."""
    total = torch.empty(rows.T, layer.M, dtype=torch.float32, device="cuda")
    for t in range(0, rows.T, 64):
        total[t:t + 64] = rows.q[t:t + 64].double() @ layer.w.double().t()
    return total * (rows.scale[:, None] * layer.scale)


CASES = [  # T, M, tile, rounds
    (96, 56832, 96, 3), (320, 28416, 160, 3), (384, 28416, 192, 3), (448, 28416, 224, 3), (512, 28416, 256, 3),
    (224, 28672, 224, 2), (448, 14336, 224, 2), (640, 8192, 160, 2),       # 112, 112 and 128 tiles
]


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("N", [64, 256])
@pytest.mark.parametrize("T,M,tile,rounds", CASES)
def test_several_tiles_of_a_pair(T, M, tile, rounds, N, kind):
    """y in rows that TMA writes, stored and accumulated, over repeated calls."""
    layer, rows, g = problem(T, M, N, T + N)
    value = product(layer, rows)
    want = value.to(DT[kind])
    y = torch.empty(T, M, dtype=DT[kind], device="cuda")
    for _ in range(8):
        y.fill_(float("nan"))
        layer.linear(rows, y)
        assert torch.equal(y, want)
    y0 = torch.randn(T, M, generator=g, device="cuda").to(DT[kind])
    want = (y0.float() + value).to(DT[kind])
    for _ in range(4):
        y.copy_(y0)
        layer.linear(rows, y, fluxbin.FLAG_ACCUMULATE)
        assert torch.equal(y, want)


@pytest.mark.parametrize("kind", ["fp16", "fp32"])
@pytest.mark.parametrize("T,M", [(96, 56829), (320, 28411), (384, 28411), (448, 28411)])
def test_a_last_tile_that_tma_cannot_write(T, M, kind):
    """M that ends off a 16-byte boundary in aligned rows: a pair's tiles go
    out by TMA but for the last of M, which goes row by row (same tiles)."""
    layer, rows, g = problem(T, M, 128, T)
    value = product(layer, rows)
    buf = torch.full((T, -(-M // 8) * 8), 5.0, dtype=DT[kind], device="cuda")
    y = buf[:, :M]
    for _ in range(4):
        y.fill_(float("nan"))
        layer.linear(rows, y)
        assert torch.equal(y, value.to(DT[kind]))
    y0 = torch.randn(T, M, generator=g, device="cuda").to(DT[kind])
    y.copy_(y0)
    layer.linear(rows, y, fluxbin.FLAG_ACCUMULATE)
    assert torch.equal(y, (y0.float() + value).to(DT[kind]))
    assert bool((buf[:, M:] == 5).all())


@pytest.mark.parametrize("T,M", [(320, 28416), (448, 28416)])
def test_as_a_few_tokens_at_a_time(T, M):
    """The same rows through the kernel for few tokens."""
    layer, rows, _ = problem(T, M, 256, 3)
    y, few = (torch.empty(T, M, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    layer.linear(rows, y)
    for t in range(0, T, 16):
        layer.linear(fluxbin.QuantRows(rows.q[t:t + 16], rows.scale[t:t + 16]), few[t:t + 16])
    assert torch.equal(y, few)


def test_captured_and_replayed_on_new_codes():
    T, M, N = 448, 28416, 128
    layer, rows, g = problem(T, M, N, 4)
    y = torch.empty(T, M, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.linear(rows, y)
    for _ in range(3):
        rows.q.copy_(torch.randint(-128, 128, (T, N), generator=g, device="cuda", dtype=torch.int8))
        rows.scale.mul_(torch.exp(0.3 * torch.randn(T, generator=g, device="cuda")))
        y.fill_(float("nan"))
        graph.replay()
        assert torch.equal(y, product(layer, rows).half())
