"""GPU tests of fluxbin_int8_linear against the exact integer product.

Tolerance: the integer sum is exact; its conversion to fp32, the product of
the scales and the product of the two are off by half a step (2^-24) each, so
|error| <= 3 * 2^-24 |v| (3.01 with the second-order terms); an accumulation
adds half a step of the sum, the output type half a step of the result (and
half its smallest subnormal).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lut_binary_basis_b200 import fluxbin  # noqa: E402
import int8_reference as ref  # noqa: E402

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


def codes(g, rows, N, extra=0):
    """Random codes of the whole range; the bytes between the rows are 77."""
    pitch = -(-N // 16) * 16 + extra
    buf = torch.full((rows, pitch), 77, dtype=torch.int8)
    c = torch.from_numpy(g.integers(-128, 128, (rows, N)).astype(np.int8))
    buf[:, :N] = c
    return c.numpy(), buf.cuda()[:, :N]


def problem(T, M, N, seed=0, extra=0):
    g = np.random.default_rng([seed, T, M, N])
    w, wd = codes(g, M, N, extra)
    x, xd = codes(g, T, N, extra)
    sw = np.exp(0.3 * g.standard_normal(M)).astype(np.float32) * np.float32(1e-3)
    sx = np.exp(0.3 * g.standard_normal(T)).astype(np.float32) * np.float32(1e-2)
    layer = fluxbin.Int8Layer(wd, torch.from_numpy(sw).cuda())
    rows = fluxbin.QuantRows(xd, torch.from_numpy(sx).cuda())
    return layer, rows, ref.linear(w, sw, x, sx)


def check(y, want, kind, y0=None):
    got = y.float().cpu().numpy().astype(np.float64)
    tol = 3.01 * ref.EPS24 * np.abs(want)
    if y0 is not None:
        want = want + y0
        tol = tol + ref.EPS24 * np.abs(want)
    tol = tol + ref.HALF_STEP[kind] * (np.abs(want) + tol) + ref.TINY[kind]
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}"


def run(layer, rows, kind, y0=None, flags=0):
    """The product into an array with guard columns and a guard row."""
    T, M = rows.T, layer.M
    buf = torch.full((T + 1, M + 3), 5.0, dtype=DT[kind], device="cuda")
    y = buf[:T, :M]
    if y0 is None:
        y.fill_(float("nan"))
    else:
        y.copy_(y0)
        flags |= fluxbin.FLAG_ACCUMULATE
    layer.linear(rows, y, flags)
    torch.cuda.synchronize()
    assert bool((buf[:T, M:] == 5).all()) and bool((buf[T] == 5).all())
    return y


SIZES = [1, 2, 3, 5, 8, 9, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 160, 200, 255, 256, 257, 300, 513]


@pytest.mark.parametrize("T", SIZES)
@pytest.mark.parametrize("M,N", [(128, 128), (256, 512), (200, 272), (77, 33), (513, 1000)])
def test_every_batch_size(T, M, N):
    layer, rows, want = problem(T, M, N)
    check(run(layer, rows, "fp32"), want, "fp32")


@pytest.mark.parametrize("T,M,N", [
    (1, 1, 1), (1, 1, 16), (2, 3, 5), (1, 7, 15), (1, 16, 17), (3, 15, 31), (4, 17, 127), (7, 127, 129), (9, 129, 255),
    (1, 4096, 4096), (1, 1003, 2050), (3, 4736, 8192), (2, 4737, 300), (16, 4736, 4096), (9, 500, 4097), (8, 300, 8193), (4, 11008, 4096), (16, 4096, 11008), (1, 64, 65536), (5, 40, 131071), (70, 40, 131071),
    (20, 4096, 4096), (64, 2048, 4096), (77, 1003, 2050), (333, 1024, 3000), (500, 3001, 777), (1000, 512, 64), (2049, 300, 200),
    (40, 19500, 300), (24, 19001, 640), (60, 40000, 130)])
@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
def test_shapes_and_types(T, M, N, kind):
    layer, rows, want = problem(T, M, N, seed=1, extra=32)
    # fp16 holds up to 65504: bring the largest results below it
    top = np.abs(want).max()
    if kind == "fp16" and top > 6e4:
        k = 2.0 ** np.ceil(np.log2(top / 6e4))
        layer.scale.div_(k)
        want = want / k
    check(run(layer, rows, kind), want, kind)
    y0 = torch.randn(T, M, device="cuda").mul_(float(np.abs(want).mean()) + 1e-3).to(DT[kind])
    check(run(layer, rows, kind, y0, fluxbin.FLAG_EARLY_WEIGHTS), want, kind, y0.float().cpu().numpy().astype(np.float64))


@pytest.mark.parametrize("T", [1, 6, 20, 130, 300])
def test_largest_sums(T):
    """Every product the largest, at the largest N: the 32-bit sums do not overflow."""
    M, N = 130, 131071
    for cw, cx in ((-128, -128), (127, -128), (127, 127)):
        w = torch.full((M, 131072), cw, dtype=torch.int8, device="cuda")[:, :N]
        x = torch.full((T, 131072), cx, dtype=torch.int8, device="cuda")[:, :N]
        layer = fluxbin.Int8Layer(w, torch.ones(M, device="cuda"))
        rows = fluxbin.QuantRows(x, torch.ones(T, device="cuda"))
        want = np.full((T, M), float(cw * cx * N))
        check(run(layer, rows, "fp32"), want, "fp32")


@pytest.mark.parametrize("M,N", [(640, 1024), (999, 2049), (4096, 4096)])
def test_a_token_alone_and_in_a_batch(M, N):
    """A token's row has the same bits whatever batch it is in."""
    layer, rows, _ = problem(300, M, N, seed=2)
    y = run(layer, rows, "fp32")
    for T in (1, 2, 7, 8, 9, 16, 17, 32, 40, 64, 100, 128, 150, 256, 299):
        assert torch.equal(run(layer, rows.rows(T), "fp32"), y[:T]), T
    for t in (0, 131, 299):
        one = fluxbin.QuantRows(rows.q[t:t + 1], rows.scale[t:t + 1])
        assert torch.equal(run(layer, one, "fp32"), y[t:t + 1])


@pytest.mark.parametrize("T", [1, 5, 16, 40, 200])
def test_scales_that_are_not_finite(T):
    """NaN scales (rows that had no finite value) reach their rows only; zero scales give zeros."""
    layer, rows, want = problem(T, 300, 500, seed=3)
    rows.scale[T // 2] = float("nan")
    if T > 2:
        rows.scale[0] = 0
    y = run(layer, rows, "fp32").cpu().numpy()
    assert np.isnan(y[T // 2]).all() and not np.isnan(np.delete(y, T // 2, axis=0)).any()
    if T > 2:
        assert np.all(y[0] == 0)


@pytest.mark.parametrize("T,M", [(1, 5), (33, 130), (200, 257)])
def test_no_input_features(T, M):
    layer = fluxbin.Int8Layer(torch.zeros(M, 0, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"))
    rows = fluxbin.QuantRows(torch.zeros(T, 0, dtype=torch.int8, device="cuda"), torch.ones(T, device="cuda"))
    assert bool((run(layer, rows, "fp16") == 0).all())
    y0 = torch.randn(T, M, device="cuda")
    assert torch.equal(run(layer, rows, "fp32", y0), y0)


def test_empty_calls():
    layer, rows, _ = problem(4, 64, 64)
    y = torch.zeros(0, 64, device="cuda")
    layer.linear(rows.rows(0), y)
    fluxbin.Int8Layer(layer.w[:0], layer.scale[:0]).linear(rows, torch.zeros(4, 0, device="cuda"))


@pytest.mark.parametrize("kind", ["fp16", "fp32"])
@pytest.mark.parametrize("T,M,N", [(33, 19456, 256), (50, 19203, 384), (300, 149, 2000), (17, 640, 9000)])
def test_accumulation_into_any_rows(T, M, N, kind):
    """y's rows at every offset from a 16-byte boundary, accumulated."""
    layer, rows, want = problem(T, M, N, seed=11)
    if kind == "fp16":
        layer.scale.mul_(2.0 ** -6)
        want = want * 2.0 ** -6
    for first in range(0, 8 if kind == "fp16" else 4):
        buf = torch.full((T, M + 8), 5.0, dtype=DT[kind], device="cuda")
        y = buf[:, first:first + M]
        y.copy_(torch.randn(T, M, device="cuda"))
        y0 = y.float().cpu().numpy().astype(np.float64)
        layer.linear(rows, y, fluxbin.FLAG_ACCUMULATE)
        check(y, want, kind, y0)
        assert bool((buf[:, :first] == 5).all()) and bool((buf[:, first + M:] == 5).all())


def test_unaligned_y():
    """y at its own elements' alignment, odd pitch."""
    for T in (1, 20, 260):
        layer, rows, want = problem(T, 301, 320, seed=4)
        for kind in ("fp16", "fp32"):
            buf = torch.full((T, 305), 3.0, dtype=DT[kind], device="cuda")
            layer.linear(rows, buf[:, 1:302])
            check(buf[:, 1:302], want, kind)
            assert bool((buf[:, :1] == 3).all()) and bool((buf[:, 302:] == 3).all())


@pytest.mark.parametrize("kind", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("T,M,N", [(129, 9473, 130), (300, 5000, 400), (700, 3333, 256), (1025, 2600, 1000), (2500, 1100, 300)])
@pytest.mark.parametrize("pad,first", [(0, 0), (8, 8), (3, 0), (8, 1)])
def test_many_tiles(T, M, N, pad, first, kind):
    """Enough tiles for several rounds of every CTA, several groups of token
    tiles, ragged ends; y with rows that allow bulk copies and rows that do
    not, stored and accumulated."""
    layer, rows, want = problem(T, M, N, seed=10)
    if kind == "fp16":
        layer.scale.mul_(2.0 ** -4)
        want = want * 2.0 ** -4
    ld = -(-M // 8) * 8 + pad + first
    buf = torch.full((T + 1, ld), 5.0, dtype=DT[kind], device="cuda")
    y = buf[:T, first:first + M]
    layer.linear(rows, y)
    check(y, want, kind)
    y.copy_(torch.randn(T, M, device="cuda"))
    y0 = y.float().cpu().numpy().astype(np.float64)
    layer.linear(rows, y, fluxbin.FLAG_ACCUMULATE)
    check(y, want, kind, y0)
    assert bool((buf[T] == 5).all()) and bool((buf[:T, :first] == 5).all()) and bool((buf[:T, first + M:] == 5).all())


def test_repeated_calls_and_streams():
    """Calls that overlap on two streams, with no order between them."""
    layer, rows, want = problem(24, 1500, 2000, seed=5)
    big, brows, bwant = problem(200, 700, 3000, seed=6)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ys = [torch.full((24, 1500), float("nan"), device="cuda") for _ in range(8)]
    zs = [torch.full((200, 700), float("nan"), device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    for y, z in zip(ys, zs):
        layer.linear(rows, y, stream=s1)
        big.linear(brows, z, stream=s2)
    torch.cuda.synchronize()
    for y, z in zip(ys, zs):
        check(y, want, "fp32")
        check(z, bwant, "fp32")


def test_many_tokens():
    """More token tiles than a grid dimension of 65,535 of them would take, and offsets beyond 2^31."""
    T, M, N = 70000, 130, 40
    g = np.random.default_rng(8)
    w, wd = codes(g, M, N)
    x, xd = codes(g, T, N)
    layer = fluxbin.Int8Layer(wd, torch.ones(M, device="cuda"))
    rows = fluxbin.QuantRows(xd, torch.ones(T, device="cuda"))
    buf = torch.zeros(T * 32768, dtype=torch.float16, device="cuda").view(T, 32768)   # 4.6 GB, 2.3e9 elements
    y = buf[:, 1000:1000 + M]
    layer.scale.mul_(2.0 ** -8)
    layer.linear(rows, y)
    check(y, ref.linear(w, np.full(M, 2.0 ** -8, np.float32), x, np.ones(T, np.float32)), "fp16")
    assert bool((buf[:, 999] == 0).all()) and bool((buf[:, 1000 + M] == 0).all())


@pytest.mark.parametrize("T,M,N", [(20, 300, 4096), (200, 2000, 1000), (600, 4096, 512), (700, 9000, 300), (64, 20000, 256)])
def test_waits_that_give_up(T, M, N):
    """The bounded waits' give-up path: NaN outputs, the status bit (read and
    cleared), and a correct next call."""
    layer, rows, want = problem(T, M, N, seed=9)
    y = run(layer, rows, "fp32", flags=fluxbin.FLAG_TEST_WAIT_TIMEOUT)
    assert bool(torch.isnan(y).all())
    assert fluxbin.fluxbin_device_status() & 1
    assert fluxbin.fluxbin_device_status() == 0
    check(run(layer, rows, "fp32"), want, "fp32")
