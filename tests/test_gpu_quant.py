"""GPU tests of the operators that write 8-bit rows: fluxbin_quant_rows,
fluxbin_silu_mul_quant, fluxbin_rmsnorm_quant.

Codes.  quant and rmsnorm take their codes from fp32 products that are fixed
by the definition (for rmsnorm the 1/rms cancels), so the codes equal the
numpy ones exactly.  silu_mul holds v = g / (1 + exp(-g)) u to a relative
delta: the device exponential is within 2 + 1.173 |g| units of 2^-23, the sum
1 + e, the reciprocal (1 unit) and two products add 3.5 more, so
delta = (6 + 1.173 |g|) 2^-23; a code is then within 1/2 of v / s up to
127 (delta_row + delta) for its own and the maximum's error.

Scales.  amax / 127 is one fp32 division: equal exactly.  rmsnorm: the sum of
N positive squares is accumulated over at most N / threads + 10 additions, each
half a step (2^-24) off; the root halves that; the mean, + eps, root,
reciprocal, product and division add six half steps.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lut_binary_basis_b200 import fluxbin  # noqa: E402
import int8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SHAPES = [(1, 1), (3, 7), (1, 8), (5, 17), (2, 64), (9, 100), (33, 255), (2, 256), (4, 257), (3, 1000), (1, 4096),
          (6, 4099), (2, 8192), (3, 11008), (1, 16392), (2, 28672), (1, 32768), (2, 32776), (1, 40001), (1, 131071)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def values(g, T, N, kind, spread=1.0):
    """(fp32 numpy array of values of the type, device tensor)."""
    v = ref.round_to(g.standard_normal((T, N)) * spread, kind)
    return v, torch.from_numpy(v).to(DT[kind]).cuda()


def rows_with_guard(T, N):
    """Rows of codes with guard bytes in the pitch and behind the last row."""
    pitch = -(-N // 16) * 16 + 16
    buf = torch.full((T + 1, pitch), 99, dtype=torch.int8, device="cuda")
    sc = torch.full((T + 1,), -5.0, dtype=torch.float32, device="cuda")
    return fluxbin.QuantRows(buf[:T, :N], sc[:T]), buf, sc


def check_guard(buf, sc, T, N):
    assert bool((buf[:T, N:] == 99).all()) and bool((buf[T] == 99).all()) and sc[T].item() == -5.0


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("T,N", SHAPES)
def test_quant_rows(T, N, kind):
    g = np.random.default_rng([1, T, N])
    x, xd = values(g, T, N, kind, 3.0)
    if T > 2:
        x[1] = 0
        xd[1] = 0
    rows, buf, sc = rows_with_guard(T, N)
    rows.quantize(xd)
    q, s = ref.quant(x)
    assert np.array_equal(rows.q.cpu().numpy(), q)
    assert np.array_equal(rows.scale.cpu().numpy(), s)
    check_guard(buf, sc, T, N)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("T,N", SHAPES)
def test_silu_mul_quant(T, N, kind):
    g = np.random.default_rng([2, T, N])
    # gate and up side by side in one array, as a joint projection writes them
    _, gu = values(g, T, 2 * N, kind, 2.0)
    if T > 2:
        gu[1] = 0
    host = gu.float().cpu().numpy()
    rows, buf, sc = rows_with_guard(T, N)
    rows.silu_mul(gu[:, :N], gu[:, N:])
    v = ref.silu_mul(host[:, :N], host[:, N:])
    delta = (6 + 1.173 * np.abs(host[:, :N]).max()) * 2.0 ** -23
    a = np.abs(v).max(axis=1)
    s = rows.scale.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(s - a / 127) <= a / 127 * (delta + 2.0 ** -23))
    q = rows.q.cpu().numpy().astype(np.float64)
    step = np.where(a > 0, a / 127, 1.0)[:, None]
    assert np.all(np.abs(q - v / step) <= 0.5 + 127 * (2 * delta + 4 * 2.0 ** -23))
    check_guard(buf, sc, T, N)


@pytest.mark.parametrize("kind,hkind", [("fp16", "fp16"), ("bf16", "bf16"), ("fp16", "fp32"), ("bf16", "fp32")])
@pytest.mark.parametrize("T,N", SHAPES)
def test_rmsnorm_quant(T, N, kind, hkind):
    g = np.random.default_rng([3, T, N])
    h, hd = values(g, T, N, hkind, 2.5)
    d, dd = values(g, T, N, kind)
    gm, gd = values(g, 1, N, kind)
    gm, gd = gm[0], gd[0]
    rows, buf, sc = rows_with_guard(T, N)
    eps = 1e-5
    for use_delta, out in ((True, "new"), (True, "in place"), (False, None), (True, None), (False, "new")):
        hin = hd.clone()
        ho = None if out is None else hin if out == "in place" else torch.full_like(hd, float("nan"))
        buf.fill_(99)
        rows.rmsnorm(hin, gd, eps, delta=dd if use_delta else None, h_out=ho)
        want_h, q, s = ref.rmsnorm(h, d if use_delta else None, gm, eps, hkind)
        if ho is not None:
            assert np.array_equal(ho.float().cpu().numpy(), want_h.astype(np.float32))
        if out != "in place":
            assert torch.equal(hin, hd)
        got = rows.scale.cpu().numpy().astype(np.float64)
        adds = -(-N // 32) + 10 if N <= 256 else 8 * -(-N // 8192) + 42     # squares a thread adds, then the tree
        assert np.all(np.abs(got - s) <= np.abs(s) * (adds / 2 + 6) * ref.EPS24)
        assert np.array_equal(rows.q.cpu().numpy(), q)
        check_guard(buf, sc, T, N)


def special_rows(kind, N):
    lowest = {"fp16": -65504.0, "bf16": -3.3895313892515355e38}[kind]
    tiny = {"fp16": 2.0 ** -24, "bf16": 2.0 ** -133}[kind]
    rows = [np.zeros(N), np.full(N, np.nan), np.full(N, -np.inf), np.full(N, lowest), np.full(N, tiny), np.full(N, -0.0)]
    for bad in (np.nan, np.inf, -np.inf, lowest):          # in one place only, the last
        r = np.ones(N)
        r[-1] = bad
        rows.append(r)
    r = np.zeros(N)
    r[0] = tiny
    rows.append(r)
    return np.stack(rows).astype(np.float32)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("N", [1, 33, 264, 5000, 40000])
def test_rows_without_a_finite_scale(N, kind):
    x = special_rows(kind, N)
    T = x.shape[0]
    xd = torch.from_numpy(x).to(DT[kind]).cuda()
    rows, buf, sc = rows_with_guard(T, N)
    rows.quantize(xd)
    q, s = ref.quant(x)
    assert np.array_equal(rows.q.cpu().numpy(), q)
    assert np.array_equal(rows.scale.cpu().numpy(), s, equal_nan=True)
    # the same rows as `up` of the gate: silu(1) is a positive factor, so the
    # kinds of scale (0, NaN, finite) are the same
    rows.silu_mul(torch.ones_like(xd), xd)
    got = rows.scale.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(s)) and np.array_equal(got == 0, s == 0)
    assert np.all(rows.q.cpu().numpy()[np.isnan(s)] == 0)
    # and as h of the norm, with and without eps: no code survives a row
    # without a scale (the squares of bf16's lowest are beyond fp32)
    for eps in (1e-5, 0.0):
        rows.rmsnorm(xd, torch.ones(N, dtype=DT[kind], device="cuda"), eps)
        _, q, s = ref.rmsnorm(x, None, np.ones(N), eps, kind)
        if kind == "bf16" and eps == 0.0:
            # bf16's smallest values square to less than fp32 holds: 1/rms is infinite, no finite scale
            small = (np.abs(x).max(axis=1) < 1e-30) & ~np.isnan(s)
            s[small], q[small] = np.nan, 0
        got = rows.scale.cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(s))
        ok = ~np.isnan(s)
        assert np.all(np.abs(got[ok] - s[ok]) <= np.abs(s[ok]) * 200 * ref.EPS24 + 2.0 ** -149)
        assert np.array_equal(rows.q.cpu().numpy(), q)
    check_guard(buf, sc, T, N)


def test_gate_limits():
    """Large negative gates give silu's limit (0), large positive ones the gate itself."""
    g = torch.tensor([[-60000.0, -100.0, -90.0, 0.0, 90.0, 100.0, 500.0, -0.0]], device="cuda").bfloat16()
    u = torch.ones_like(g)
    rows = fluxbin.QuantRows.empty(1, 8)
    rows.silu_mul(g, u)
    v = ref.silu_mul(g.float().cpu().numpy(), u.float().cpu().numpy())
    assert np.array_equal(rows.q.cpu().numpy(), np.rint(v * 127 / 500).astype(np.int8))
    assert rows.scale.item() == np.float32(500) / np.float32(127)


@pytest.mark.parametrize("N", [512, 515])
def test_strided_and_unaligned_rows(N):
    """Pitches and first elements that forbid 16-byte accesses give the same
    codes as aligned ones."""
    g = np.random.default_rng(7)
    x, _ = values(g, 6, N + 3, "fp16")
    xd = torch.from_numpy(x).half().cuda()
    want, s = ref.quant(x[:, 3:])
    rows = fluxbin.QuantRows.empty(6, N)
    rows.quantize(xd[:, 3:])
    assert np.array_equal(rows.q.cpu().numpy(), want) and np.array_equal(rows.scale.cpu().numpy(), s)
    every2 = torch.zeros(12, N + 3, dtype=torch.float16, device="cuda")
    every2[::2] = xd
    rows.quantize(every2[::2, 3:])
    assert np.array_equal(rows.q.cpu().numpy(), want)
    out = torch.full((6, N + 5), 7.0, dtype=torch.float16, device="cuda")
    gm = torch.ones(N + 1, dtype=torch.float16, device="cuda")[1:]
    rows.rmsnorm(xd[:, 3:], gm, 1e-5, h_out=out[:, 2:2 + N])
    _, q, _ = ref.rmsnorm(x[:, 3:], None, np.ones(N), 1e-5, "fp16")
    assert np.array_equal(rows.q.cpu().numpy(), q)
    assert torch.equal(out[:, 2:2 + N], xd[:, 3:]) and bool((out[:, :2] == 7).all()) and bool((out[:, 2 + N:] == 7).all())


@pytest.mark.parametrize("kind,hkind", [("fp16", "fp16"), ("bf16", "fp32")])
@pytest.mark.parametrize("N", [5, 40, 515, 2050, 9001, 33001])
def test_every_array_at_its_own_offset(N, kind, hkind):
    """h, delta, gamma and h_out each at another offset from a 16-byte boundary."""
    g = np.random.default_rng([8, N])
    T, W = 3, N + 8
    for a, b, c, d in ((1, 2, 3, 0), (0, 1, 5, 2), (3, 0, 0, 1), (2, 7, 6, 3)):
        h, hd = values(g, T, W, hkind, 2.0)
        dl, dd = values(g, T, W, kind)
        gm, gd = values(g, 1, W, kind)
        out = torch.full((T, W), 7.0, dtype=DT[hkind], device="cuda")
        rows, buf, sc = rows_with_guard(T, N)
        rows.rmsnorm(hd[:, a:a + N], gd[0, c:c + N], 1e-5, delta=dd[:, b:b + N], h_out=out[:, d:d + N])
        want, q, _ = ref.rmsnorm(h[:, a:a + N], dl[:, b:b + N], gm[0, c:c + N], 1e-5, hkind)
        assert np.array_equal(out[:, d:d + N].float().cpu().numpy(), want.astype(np.float32))
        assert bool((out[:, :d] == 7).all()) and bool((out[:, d + N:] == 7).all())
        assert np.array_equal(rows.q.cpu().numpy(), q)
        check_guard(buf, sc, T, N)


def test_empty_rows():
    rows = fluxbin.QuantRows.empty(3, 0)
    rows.scale.fill_(7)
    rows.quantize(torch.zeros(3, 0, dtype=torch.float16, device="cuda"))
    assert rows.scale.tolist() == [0, 0, 0]
    rows = fluxbin.QuantRows.empty(0, 32)
    rows.quantize(torch.zeros(0, 32, dtype=torch.float16, device="cuda"))
    rows = fluxbin.QuantRows.empty(3, 0)
    with pytest.raises(fluxbin.FluxbinError) as e:
        rows.rmsnorm(torch.zeros(3, 0, dtype=torch.float16, device="cuda"), torch.zeros(0, dtype=torch.float16, device="cuda"), 1e-5)
    assert e.value.status in (-1, -2)


def test_many_rows():
    """More rows than a grid dimension of 65,535 would take."""
    T, N = 70001, 16
    x = torch.randn(T, N, device="cuda").half()
    rows = fluxbin.QuantRows.empty(T, N)
    rows.quantize(x)
    q, s = ref.quant(x.float().cpu().numpy())
    assert np.array_equal(rows.q.cpu().numpy(), q) and np.array_equal(rows.scale.cpu().numpy(), s)


def in_batches(T, N, run, batch=16):
    """Codes and scales of the same rows, a few at a time."""
    rows = fluxbin.QuantRows.empty(T, N)
    for t in range(0, T, batch):
        run(fluxbin.QuantRows(rows.q[t:t + batch], rows.scale[t:t + batch]), slice(t, t + batch))
    return rows


def same(a, b):
    return torch.equal(a.q, b.q) and torch.equal(a.scale.view(torch.int32), b.scale.view(torch.int32))


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("T,N", [(2371, 4096), (1200, 8200), (1184, 12288), (593, 12296), (300, 20480), (301, 28920),
                                 (296, 28928), (296, 28936), (297, 28671), (1700, 1000)])
def test_gate_of_many_rows(T, N, kind):
    """A row's codes and scale do not depend on how many rows there are, on
    its neighbours (zeros, NaN, infinity among them) or on the kernel."""
    g = torch.Generator(device="cuda").manual_seed(T + N)
    gu = (torch.randn(T, 2 * N, device="cuda", generator=g) * 2).to(DT[kind])
    gu[T // 3] = 0
    gu[T // 2, N - 1] = float("nan")
    gu[T // 2 + 1, N + 3] = float("inf")
    gu[T - 1] *= 2.0 ** -6
    rows, buf, sc = rows_with_guard(T, N)
    rows.silu_mul(gu[:, :N], gu[:, N:])
    few = in_batches(T, N, lambda r, at: r.silu_mul(gu[at, :N], gu[at, N:]))
    assert same(rows, few)
    check_guard(buf, sc, T, N)
    assert rows.scale[T // 3].item() == 0 and bool(torch.isnan(rows.scale[T // 2:T // 2 + 2]).all())
    assert not rows.q[T // 3].any() and not rows.q[T // 2:T // 2 + 2].any()
    for t in (0, T // 3 + 1, T - 2, T - 1):
        host = gu[t:t + 1].float().cpu().numpy()
        v = ref.silu_mul(host[:, :N], host[:, N:])
        delta = (6 + 1.173 * np.abs(host[:, :N]).max()) * 2.0 ** -23
        a = np.abs(v).max()
        assert abs(rows.scale[t].item() * 127.0 / a - 1) <= delta + 2.0 ** -23
        assert np.abs(rows.q[t].cpu().numpy() - v[0] * (127 / a)).max() <= 0.5 + 127 * 2 * delta + 2.0 ** -15


@pytest.mark.parametrize("N", [256, 4096, 8191, 28672])
def test_many_rows_as_in_small_batches(N):
    """What is asked of L2 ahead stays within the rows and changes nothing."""
    T = 1500 if N < 10000 else 400
    x = torch.randn(T, N, device="cuda").bfloat16()
    rows = fluxbin.QuantRows.empty(T, N)
    assert same(rows.quantize(x) or rows, in_batches(T, N, lambda r, at: r.quantize(x[at])))
    h, gamma, h2 = torch.randn(T, N, device="cuda"), torch.rand(N, device="cuda").bfloat16(), torch.empty(T, N, device="cuda")
    rows.rmsnorm(h, gamma, 1e-6, delta=x, h_out=h2)
    assert torch.equal(h2, h + x.float())
    few = in_batches(T, N, lambda r, at: r.rmsnorm(h[at], gamma, 1e-6, delta=x[at]))
    assert torch.equal(rows.q, few.q)
    # the sums of squares may be taken in another order: N / 32 + 16 roundings of half a step at most, each way, halved by the root
    assert bool(((rows.scale - few.scale).abs() <= rows.scale * (N / 32 + 16) * 2.0 ** -24).all())


def test_gate_of_many_rows_in_two_graphs_at_once():
    """Captured calls that run side by side, each with its own rows, replayed
    after the inputs have changed."""
    T, N = 700, 16400
    gu = [torch.randn(T, 2 * N, device="cuda").half() for _ in range(2)]
    rows = [fluxbin.QuantRows.empty(T, N) for _ in range(2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for x, r in zip(gu, rows):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            r.silu_mul(x[:, :N], x[:, N:])
        graphs.append(graph)
    for _ in range(3):
        for x in gu:
            x.copy_(torch.randn(T, 2 * N, device="cuda"))
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for x, r in zip(gu, rows):
            want = fluxbin.QuantRows.empty(T, N)
            want.silu_mul(x[:, :N], x[:, N:])
            assert same(r, want)
