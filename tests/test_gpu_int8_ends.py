"""GPU tests of fluxbin_int8_linear added to rows of y at every offset from a
16-byte boundary, by CTAs with a whole tile each, whose last tile has one
channel or a few: the ends of rows, read and written element by element."""
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


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("T,M", [(1, 29953), (20, 29953), (20, 29959), (3, 29966)])      # 234 tiles of 128 channels and 1, 1, 7, 14 more
def test_accumulation_at_every_offset(T, M, kind):
    N = 512
    g = torch.Generator("cuda").manual_seed(T + M)
    w = torch.randint(-128, 128, (M, N), generator=g, device="cuda", dtype=torch.int8)
    x = torch.randint(-128, 128, (T, N), generator=g, device="cuda", dtype=torch.int8)
    layer = fluxbin.Int8Layer(w, torch.exp(0.3 * torch.randn(M, generator=g, device="cuda")) * 1e-3)
    rows = fluxbin.QuantRows(x, torch.exp(0.3 * torch.randn(T, generator=g, device="cuda")) * 1e-2)
    # exact in fp32 (below 2^24), then one rounding a product, the addition and y's type
    value = (x.double() @ w.double().t()).float() * (rows.scale[:, None] * layer.scale)
    for first in range(128 // torch.finfo(DT[kind]).bits):
        buf = torch.full((T, M + 11), 5.0, dtype=DT[kind], device="cuda")       # an odd pitch: rows at every offset
        y = buf[:, first:first + M]
        y0 = torch.randn(T, M, generator=g, device="cuda").to(DT[kind])
        y.copy_(y0)
        layer.linear(rows, y, fluxbin.FLAG_ACCUMULATE)
        assert torch.equal(y, (y0.float() + value).to(DT[kind])), first
        assert bool((buf[:, :first] == 5).all()) and bool((buf[:, first + M:] == 5).all())
