"""The 8-bit operators together, as a block of a model uses them: residual add
and norm, joint gate/up projection, gate, down projection added to the
residual stream, at a decode batch and at a prompt, eagerly and captured in
CUDA graphs; beside a binary layer that reads the same normalised row.

Each operator is checked by itself elsewhere; here the chain is held to the
same chain of plain implementations, fed with the device's own codes at each
step, so that a difference is one operator's and within its tolerance.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from lut_binary_basis_b200 import fluxbin  # noqa: E402
import int8_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    fluxbin.fluxbin_device_status()
    yield
    assert fluxbin.fluxbin_device_status() == 0, "a bounded wait gave up"


class Block:
    """The MLP half of a block on 8-bit layers; the stream in fp32."""

    def __init__(self, T, N, F, seed):
        g = np.random.default_rng(seed)
        self.gate_up = fluxbin.Int8Layer.from_host(g.standard_normal((2 * F, N)) / np.sqrt(N))
        self.down = fluxbin.Int8Layer.from_host(g.standard_normal((N, F)) / np.sqrt(F))
        self.gamma = torch.from_numpy(g.uniform(0.5, 1.5, N)).half().cuda()
        self.xq, self.aq = fluxbin.QuantRows.empty(T, N), fluxbin.QuantRows.empty(T, F)
        self.gu = torch.empty(T, 2 * F, dtype=torch.float16, device="cuda")
        self.F = F

    def __call__(self, h, delta):
        F = self.F
        self.xq.rmsnorm(h, self.gamma, 1e-5, delta=delta, h_out=h)
        self.gate_up.linear(self.xq, self.gu, fluxbin.FLAG_EARLY_WEIGHTS)
        self.aq.silu_mul(self.gu[:, :F], self.gu[:, F:])
        self.down.linear(self.aq, h, fluxbin.FLAG_ACCUMULATE | fluxbin.FLAG_EARLY_WEIGHTS)


def close(got, want, rel):
    return np.linalg.norm(got - want) <= rel * np.linalg.norm(want)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("T,N,F", [(1, 512, 1376), (5, 1000, 300), (16, 512, 1376), (40, 520, 640), (300, 512, 1000)])
def test_block(T, N, F):
    g = np.random.default_rng([T, N])
    b = Block(T, N, F, [1, T, N])
    h0 = g.standard_normal((T, N)).astype(np.float32)
    d0 = g.standard_normal((T, N)).astype(np.float16)
    h, d = torch.from_numpy(h0).cuda(), torch.from_numpy(d0).cuda()
    b(h, d)
    torch.cuda.synchronize()
    # step by step, each from the device's own input to it
    h1, q, s = ref.rmsnorm(h0, d0, host(b.gamma), 1e-5, "fp32")
    assert np.array_equal(b.xq.q.cpu().numpy(), q)
    gu = ref.linear(b.gate_up.w.cpu().numpy(), host(b.gate_up.scale), q, host(b.xq.scale))
    assert np.all(np.abs(host(b.gu) - gu) <= np.abs(gu) * (2.0 ** -11 + 4 * ref.EPS24) + 2.0 ** -25)
    v = ref.silu_mul(host(b.gu)[:, :F], host(b.gu)[:, F:])
    a = np.abs(v).max(axis=1, keepdims=True) / 127
    assert np.all(np.abs(b.aq.q.cpu().numpy() - v / a) <= 0.5 + 1e-3)     # 1e-3 is 8 delta * 127 at |g| = 6
    y = h1 + ref.linear(b.down.w.cpu().numpy(), host(b.down.scale), b.aq.q.cpu().numpy(), host(b.aq.scale))
    assert np.all(np.abs(host(h) - y) <= 5 * ref.EPS24 * (np.abs(y) + np.abs(y - h1)) + 1e-30)


@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_captured_and_replayed(T):
    """The block in a CUDA graph, replayed on new inputs, beside an eager call
    and a second graph of the same layers."""
    N, F = 512, 1376
    b, c = Block(T, N, F, 3), Block(T, N, F, 3)
    g = torch.Generator("cuda").manual_seed(T)
    h, d = torch.zeros(T, N, device="cuda"), torch.zeros(T, N, device="cuda").half()
    h2, d2 = h.clone(), d.clone()

    def graph_of(block, h, d):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            block(h, d)
        torch.cuda.current_stream().wait_stream(s)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            block(h, d)
            block(h, d)
        return gr

    g1, g2 = graph_of(b, h, d), graph_of(c, h2, d2)
    eager = Block(T, N, F, 3)
    for _ in range(3):
        x, y = torch.randn(T, N, generator=g, device="cuda"), torch.randn(T, N, generator=g, device="cuda").half()
        want = x.clone()
        eager(want, y)
        eager(want, y)
        for t, u in ((h, d), (h2, d2)):
            t.copy_(x)
            u.copy_(y)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            g1.replay()
        with torch.cuda.stream(s2):
            g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, want) and torch.equal(h2, want)


def test_next_to_a_binary_layer():
    """One normalised row through an 8-bit layer and through a binary one."""
    import oracle
    from lut_binary_basis_b200 import synth
    sp = synth.scaled_spec(synth.layer_7b_proj(), M=300, N=520, n_sal=26)
    layer = synth.make_layer(sp, synth.layer_key(9, 0, 0))
    x = synth.make_x(sp, 1, synth.x_key(9, 0, 0, 1))
    want = oracle.linear(layer, x)
    d = fluxbin.DeviceLayer.from_host(layer)
    y = torch.zeros(1, sp.M, device="cuda")
    xd = torch.from_numpy(x).cuda()
    d.linear(xd, y, fluxbin.FLAG_Y_FP32, fluxbin.new_workspace(sp.M, 1))
    # the same layer's response to unit vectors is its dense matrix
    eye = np.eye(sp.N, dtype=np.float16)
    W = np.concatenate([oracle.linear(layer, eye[i:i + 16]) for i in range(0, sp.N, 16)]).T
    layer8 = fluxbin.Int8Layer.from_host(W)
    rows = fluxbin.QuantRows.empty(1, sp.N)
    rows.quantize(xd)
    y8 = torch.zeros(1, sp.M, device="cuda")
    layer8.linear(rows, y8)
    assert close(host(y), want, 2e-3)
    # 8-bit codes: each weight is off by at most s/2 and each activation by
    # s_x/2, so |y8 - y| <= sum |W| s_x/2 + sum |x| s/2 + N s s_x/4
    sx, sw = rows.scale.item(), host(layer8.scale)
    bound = np.abs(W).sum(axis=1) * sx / 2 + np.abs(x.astype(np.float64)).sum() * sw / 2 + sp.N * sw * sx / 4
    assert np.all(np.abs(host(y8)[0] - want[0]) <= bound * (1 + 1e-5))


def test_other_device_and_stream():
    """Tensors used on another stream than the current one; a device that is not the current one where there is one."""
    T, N, F = 4, 512, 640
    b, e = Block(T, N, F, 5), Block(T, N, F, 5)
    h = torch.randn(T, N, device="cuda")
    d = torch.randn(T, N, device="cuda").half()
    want = h.clone()
    e(want, d)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b.xq.rmsnorm(h, b.gamma, 1e-5, delta=d, h_out=h, stream=s)
    b.gate_up.linear(b.xq, b.gu, stream=s)
    b.aq.silu_mul(b.gu[:, :F], b.gu[:, F:], stream=s.cuda_stream)
    b.down.linear(b.aq, h, fluxbin.FLAG_ACCUMULATE, stream=s)
    s.synchronize()
    assert torch.equal(h, want)
    if torch.cuda.device_count() > 1:
        rows = fluxbin.QuantRows.empty(2, 64, "cuda:1")
        rows.quantize(torch.randn(2, 64, device="cuda:1").half())
        torch.cuda.synchronize(1)


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing has to be warmed up: the process's first calls are captured."""
    import os
    import subprocess
    import sys
    code = """
import torch
from lut_binary_basis_b200 import fluxbin
torch.zeros(1, device="cuda")
out = []
for T, M in ((1, 64), (40, 256), (300, 20000)):
    x = torch.ones(T, 96, device="cuda").half()
    rows = fluxbin.QuantRows.empty(T, 96)
    layer = fluxbin.Int8Layer(torch.ones(M, 96, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"))
    y = torch.zeros(T, M, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rows.quantize(x)
        layer.linear(rows, y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.allclose(y, torch.full_like(y, 96.0), rtol=1e-6), (T, M)
assert fluxbin.fluxbin_device_status() == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_host_threads():
    """Calls from two host threads at once, each on its own stream."""
    import threading
    results = {}

    def work(k):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            g = torch.Generator("cuda").manual_seed(k)
            ok = True
            for T, M, N in ((1, 512, 512), (33, 700, 900), (300, 5000, 400)) * 5:
                x = torch.randn(T, N, generator=g, device="cuda").half()
                w = torch.randint(-127, 128, (M, N), generator=g, device="cuda", dtype=torch.int8)
                wp = torch.zeros(M, -(-N // 16) * 16, dtype=torch.int8, device="cuda")[:, :N]
                wp.copy_(w)
                layer = fluxbin.Int8Layer(wp, torch.ones(M, device="cuda"))
                rows = fluxbin.QuantRows.empty(T, N)
                rows.quantize(x)
                y = torch.empty(T, M, device="cuda")
                layer.linear(rows, y)
                want = (rows.q.double() @ w.double().t()) * rows.scale.double()[:, None]
                ok = ok and bool(((y.double() - want).abs() <= want.abs() * 2.0 ** -22).all())
            s.synchronize()
            results[k] = ok

    threads = [threading.Thread(target=work, args=(k,)) for k in (1, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=120)
    assert results == {1: True, 2: True}


@pytest.mark.parametrize("T,M,N", [(1, 700, 1000), (16, 300, 3000), (40, 1000, 1500), (300, 9000, 500)])
def test_weights_written_by_the_preceding_kernel(T, M, N):
    """Without FLAG_EARLY_WEIGHTS the weights may come from the kernel before,
    which a programmatic dependent launch overlaps: new weights every call."""
    g = torch.Generator("cuda").manual_seed(7)
    wrows, xrows = fluxbin.QuantRows.empty(M, N), fluxbin.QuantRows.empty(T, N)
    xrows.quantize(torch.randn(T, N, generator=g, device="cuda").half())
    layer = fluxbin.Int8Layer(wrows.q, wrows.scale)
    dense = [torch.randn(M, N, generator=g, device="cuda").half() for _ in range(4)]
    ys = [torch.empty(T, M, device="cuda") for _ in range(12)]
    want = []
    for d in dense:
        wrows.quantize(d)
        torch.cuda.synchronize()
        want.append((xrows.q.double() @ wrows.q.double().t()) * xrows.scale.double()[:, None] * wrows.scale.double())
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        wrows.quantize(dense[i % 4])
        layer.linear(xrows, y)
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        # three roundings of 2^-24 each, as in the single-operator tests
        assert bool(((y.double() - want[i % 4]).abs() <= 3.01 * ref.EPS24 * want[i % 4].abs()).all()), i
