"""The calls around the estimator on buffers of more than 2^31 elements: what lies behind that offset is checked
against the formulas (in 64 bits where they round), and what has to stay untouched or zero with it."""
import pytest

from tests import _dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as zz
    zz.lib()
    return zz


def test_linear_outputs(z):
    import torch
    N, i, o = 270000, 64, 8192
    assert N * o > 2 ** 31
    x = torch.randn(N, i, device="cuda").bfloat16()
    W = torch.randn(o, i, device="cuda").bfloat16()
    y = z.dust_linear(x, W, act="relu")
    part = slice(N - 4096, N)
    ref = (x[part].double() @ W.double().t()).clamp(min=0)
    assert bool(((y[part].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -16 * (x[part].double().abs() @ W.double().abs().t())).all())
    # backward: dz of a billion-element operand, dx and db
    dx, _, db = z.dust_linear_backward(y, x, W, act="gelu", z=y, dW=None)
    s = y[part].double()
    dz = s * (0.5 * torch.erfc(-s / 2 ** 0.5) + s * torch.exp(-s * s / 2) * 0.3989422804014327)
    got, want = dx[part].double(), dz @ W.double()
    mag = dz.abs() @ W.double().abs()
    assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -7 * mag).all())
    assert bool(torch.isfinite(db).all()) and z.dust_last_device_error()[0] == 0


def test_embedding(z):
    import torch
    V, d = 70000, 32768
    assert V * d > 2 ** 31
    E = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 5, V - 2, V - 1, -1], dtype=torch.int32, device="cuda")
    for r in (5, V - 2, V - 1):
        E[r] = r % 100
    out = z.dust_embedding(ids, E)
    assert torch.equal(out, torch.stack([E[V - 1], E[5], E[V - 2], E[V - 1], E[0]]))
    del E
    g = torch.randn(5, d, device="cuda")
    G = torch.full((V, d), 3.0, device="cuda")  # 9 GB
    z.dust_embedding_grad(ids, g, V, G=G)
    assert torch.equal(G[V - 1], g[0] + g[3]) and torch.equal(G[V - 2], g[2]) and torch.equal(G[5], g[1])
    G[[V - 1, V - 2, 5]] = 0
    assert float(G.abs().max()) == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer(z, bits):
    import torch
    n = 2 ** 31 + 1000
    W, G = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    G[-1000:] = torch.linspace(-1, 1, 1000, device="cuda")
    opt = z.DustOptimizer([W], [G], bits=bits)
    opt.step(z.adam(1e-2, 1))
    w, g = W[-1000:].double(), G[-1000:].double()
    want = -1e-2 * g / (g.abs() + 1e-8)
    assert bool(((w - want).abs() <= 2.0 ** -18 * 1e-2).all())
    assert float(W[:-1000].abs().max()) == 0
