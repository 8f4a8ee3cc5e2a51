"""GPU tests of fluxbin_silu_mul_quant at the most negative gates whose exp(-g)
fp32 holds (down to g = -88.72; 1 + exp(-g) has no normal reciprocal from
-87.33 on), and below, where the value is 0.

Tolerance.  v = g / (1 + exp(-g)) u is held to a relative delta, in units of
2^-23: the exponent's rounded constant and product turn into |g|, the approximate
exponential has 2, the sum, the reciprocal and two products add 3 at most:
delta = (|g| + 5) 2^-23.  A code is within 1/2 of v / s up to 127
times its own error and the maximum's; the scale has the maximum's error and one
rounding.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lut_binary_basis_b200 import fluxbin  # noqa: E402
import int8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
LIMIT = -88.72      # exp(88.7228) is 2^128
# sizes of each kernel: several rows a CTA, one CTA, a cluster, and the one for many aligned rows
SIZES = [(5, 8), (3, 61), (7, 515), (2, 4096), (300, 2050), (1, 11008), (3, 33001), (700, 4096), (300, 20480)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def check(g, u, rows):
    gate, up = (t.float().cpu().numpy().astype(np.float64) for t in (g, u))
    with np.errstate(over="ignore"):
        v = np.where(gate < LIMIT, 0.0, gate / (1.0 + np.exp(-gate)) * up)
    delta = (np.abs(np.maximum(gate, LIMIT)) + 5) * 2.0 ** -23
    a = np.abs(v).max(axis=1)
    delta_max = delta.max(axis=1)
    s = rows.scale.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(s - a / 127) <= a / 127 * (delta_max + ref.EPS24) + 2.0 ** -149)
    q = rows.q.cpu().numpy().astype(np.float64)
    step = np.where(a > 0, a / 127, 1.0)[:, None]
    assert np.all(np.abs(q - v / step) <= 0.5 + 127 * (delta + delta_max[:, None] + 4 * 2.0 ** -23))


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("T,N", SIZES)
def test_rows_of_the_most_negative_gates(T, N, kind):
    """Whole rows of them: the scale is small, not zero, and the codes are theirs."""
    r = np.random.default_rng([T, N])
    g = torch.from_numpy(r.uniform(-88.6, -87.4, (T, N))).to(DT[kind]).cuda()      # (the types' steps here: 1/16, 1/2)
    u = torch.from_numpy(r.uniform(0.1, 1.0, (T, N)) * r.choice([-1.0, 1.0], (T, N)) * 6e4).to(DT[kind]).cuda()
    rows = fluxbin.QuantRows.empty(T, N)
    rows.silu_mul(g, u)
    check(g, u, rows)
    assert bool((rows.scale > 0).all()) and bool((rows.q.abs().amax(dim=1) == 127).all())


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("T,N", SIZES)
def test_a_few_of_them(T, N, kind):
    """Among ordinary gates, where a large `up` makes one of them the maximum, and below the limit."""
    r = np.random.default_rng([T, N, 1])
    gate, up = r.standard_normal((T, N)), r.standard_normal((T, N))
    at = r.random((T, N)) < 0.02
    gate[at] = r.uniform(-95, -80, int(at.sum()))
    if kind == "bf16":
        up[:, N // 2], gate[:, N // 2] = 3e38, -88.0        # v about -160
    gate[:, N - 1] = -60000.0
    g, u = (torch.from_numpy(t).to(DT[kind]).cuda() for t in (gate, up))
    rows = fluxbin.QuantRows.empty(T, N)
    rows.silu_mul(g, u)
    check(g, u, rows)
    if kind == "bf16":
        assert bool((rows.q[:, N // 2] == -127).all())


@pytest.mark.parametrize("T,N", [(4, 40), (700, 4096)])
def test_infinite_gates_and_ups(T, N):
    g, u = torch.full((T, N), -88.0, device="cuda").half(), torch.ones(T, N, device="cuda").half()
    g[1, 3] = float("-inf")
    u[2, N - 1] = float("inf")
    g[3, 0] = float("nan")
    rows = fluxbin.QuantRows.empty(T, N)
    rows.silu_mul(g, u)
    assert torch.isnan(rows.scale).nonzero().flatten().tolist() == [1, 2, 3]
    assert not rows.q[1:4].any() and bool((rows.q[0] == -127).all()) and rows.scale[0].item() > 0


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_smallest_and_largest_gates(kind):
    """A quarter of the smallest value is exact, the largest does not overflow on the way."""
    top, tiny = torch.finfo(DT[kind]).max, {"fp16": 2.0 ** -24, "bf16": 2.0 ** -133}[kind]
    g = torch.tensor([[top, 1.0], [tiny, tiny], [-tiny, 0.0]], device="cuda").to(DT[kind])
    u = torch.ones_like(g)
    if kind == "bf16":
        u[1:] = 2.0 ** 120
    rows = fluxbin.QuantRows.empty(3, 2)
    rows.silu_mul(g, u)
    check(g, u, rows)
    assert rows.scale[0].item() == np.float32(top) / np.float32(127) and rows.q[1].tolist() == [127, 127]
