"""The linear layer, the embedding, the estimator and the grouped optimizer step together, as a step uses them:
token ids -> embedding -> linear with GELU (its pre-activation kept) -> linear with the embedding as residual ->
the output-error estimate of the second layer's output -> back through both layers -> the table's gradient ->
one optimizer step over every tensor.  Each stage is checked against the plain 64-bit formula of what it was
given, so the tolerances are those of the single operators; the whole step is captured and replayed."""
import pytest

from tests import _dev  # noqa: F401
from tests.test_gpu_linear import act64, check

pytestmark = pytest.mark.gpu

V, D, H, N, K = 500, 64, 192, 777, 8
SIGMA, GAMMA, SCALE = 1e-2, 0.9, 8.0


@pytest.fixture(scope="module")
def z():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as zz
    zz.lib()
    return zz


class Model:
    def __init__(self, z, bits):
        import torch
        g = torch.Generator(device="cuda").manual_seed(3)
        n = lambda *s, std=1.0: torch.randn(s, device="cuda", generator=g) * std  # noqa: E731
        self.z = z
        self.E, self.W1, self.b1 = n(V, D, std=0.1), n(H, D, std=D ** -0.5), n(H, std=0.02)
        self.W2, self.b2 = n(D, H, std=H ** -0.5), n(D, std=0.02)
        self.params = [self.E, self.W1, self.b1, self.W2, self.b2]
        self.half = [None, self.W1.bfloat16(), None, self.W2.bfloat16(), None]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.opt = z.DustOptimizer(self.params, self.grads, W_bf16=self.half, bits=bits, decay=[1, 1, 0, 1, 0])
        ids = torch.randint(0, V, (N,), device="cuda", generator=g, dtype=torch.int32)
        ids[-30:] = -1  # a padded batch
        self.ids, self.u = ids, n(N, D).bfloat16()
        self.cu = torch.tensor([0, 200, 500, N], dtype=torch.int32, device="cuda")
        self.count = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.per_token = torch.tensor([1.0 / N], device="cuda")
        self.key = z.NoiseKey(0x5EED0055, 2)

    def step(self):
        import torch
        z = self.z
        W1, W2 = self.half[1], self.half[3]
        x0 = z.dust_embedding(self.ids, self.E, scale=SCALE, out_dtype=torch.bfloat16)
        h, pre = z.dust_linear(x0, W1, bias=self.b1, act="gelu", z=True)
        y = z.dust_linear(h, W2, bias=self.b2, residual=x0)
        # the second layer's product is what is perturbed: its output error, and through it the rest
        target = (self.u.float() - y.float() + z.dust_linear(h, W2, out_dtype=torch.float32)).bfloat16()
        dl = z.dust_noisy_linear_fwd(h, W2, target, K, SIGMA, self.key)
        r = z.dust_credit(dl, self.cu, GAMMA)
        _, g2 = z.dust_weight_grad(r, h, D, K, SIGMA, self.key, G_W=self.grads[3], g_out=True)
        dh, _, _ = z.dust_linear_backward(g2, h, W2, dW=None, db=self.grads[4])
        dx, _, _ = z.dust_linear_backward(dh, x0, W1, act="gelu", z=pre, dW=self.grads[1], db=self.grads[2])
        dx0 = dx.float() + g2  # the residual's part
        z.dust_embedding_grad(self.ids, dx0, V, scale=SCALE, G=self.grads[0])
        self.count.add_(1)
        self.opt.step(z.adam(1e-2, 1, weight_decay=0.1), g_scale=self.per_token, step=self.count)
        return x0, h, pre, y, g2, dh, dx, dx0


@pytest.mark.parametrize("bits", [32, 8])
def test_stages(z, bits):
    import torch
    m = Model(z, bits)
    before = [p.double().clone() for p in m.params]
    W1, W2 = m.half[1].double().clone(), m.half[3].double().clone()
    x0, h, pre, y, g2, dh, dx, dx0 = m.step()
    torch.cuda.synchronize()
    E = before[0]
    live = (m.ids >= 0).double()[:, None]
    want = E[m.ids.clamp(min=0).long()] * SCALE * live
    check(x0, want, 2.0 ** -8 * want.abs() + 1e-30, "embedding")

    def sums(a, b, n):
        return (n + 16) * 2.0 ** -23 * (a.abs() @ b.abs())

    zr = x0.double() @ W1.t() + before[2]
    tol = sums(x0.double(), W1.t(), D) + 2.0 ** -23 * zr.abs()
    check(pre, zr, tol + 2.0 ** -8 * (zr.abs() + tol), "pre-activation")
    hr = act64(zr, "gelu")[0]
    tol = 1.2 * tol + 2.0 ** -19 * (1 + zr.abs())
    check(h, hr, tol + 2.0 ** -8 * (hr.abs() + tol), "hidden")
    yr = h.double() @ W2.t() + before[4] + x0.double()
    tol = sums(h.double(), W2.t(), H) + 2.0 ** -22 * (yr.abs() + x0.double().abs())
    check(y, yr, tol + 2.0 ** -8 * (yr.abs() + tol), "output")
    # g2 (fp32) enters as two bf16 terms, a bf16 dx as one
    dhr = g2.double() @ W2
    tol = (g2.double().abs() @ W2.abs()) * (2.0 ** -8 + (D + 16) * 2.0 ** -23)
    check(dh, dhr, tol + 2.0 ** -8 * (dhr.abs() + tol), "dh")
    dz = dh.double() * act64(pre.double(), "gelu")[1]
    e = dh.double().abs() * 2.0 ** -19 * (1 + pre.double().abs())
    tol = (dz.abs() @ W1.abs()) * (2.0 ** -8 + (H + 16) * 2.0 ** -23) + 1.01 * (e @ W1.abs())
    check(dx, dz @ W1, tol + 2.0 ** -8 * ((dz @ W1).abs() + tol), "dx")
    tol = (dz.abs().t() @ x0.double().abs()) * (2.0 ** -16 + (2 * N + 40) * 2.0 ** -23) + 1.01 * (e.t() @ x0.double().abs())
    check(m.grads[1], dz.t() @ x0.double(), tol, "dW1")
    check(m.grads[2], dz.sum(0), dz.abs().sum(0) * (N + 8) * 2.0 ** -23 + 1.01 * e.sum(0), "db1")
    check(m.grads[4], g2.double().sum(0), g2.double().abs().sum(0) * (N + 8) * 2.0 ** -23, "db2")
    rows, part = m.ids[m.ids >= 0].long(), dx0.double()[m.ids >= 0] * SCALE
    ref = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, rows, part)
    mag = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, rows, part.abs())
    cnt = torch.bincount(rows, minlength=V)[:, None].double()
    check(m.grads[0], ref, (cnt + 2) * 2.0 ** -24 * mag * 1.001, "table gradient")
    # Adam's first step from zero moments: m / c1 = g and sqrt(v / c2) = |g|, to the rounding of (1 - beta)
    for p, w0, g, decay in zip(m.params, before, m.grads, [1, 1, 0, 1, 0]):
        g = g.double() / N
        step = 1e-2 * g / (g.abs() + 1e-8)
        want = w0 * (1 - 1e-2 * 0.1 * decay) - step
        assert bool(((p.double() - want).abs() <= 2.0 ** -18 * step.abs() + 2.0 ** -22 * (w0.abs() + 1e-2)).all())
    assert torch.equal(m.half[1], m.W1.bfloat16()) and torch.equal(m.half[3], m.W2.bfloat16())
    assert z.dust_last_device_error()[0] == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_equal_eager_steps(z, bits):
    import torch
    a, b = Model(z, bits), Model(z, bits)
    c = Model(z, bits)
    c.step()  # one-time set-up of every call, outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for _ in range(4):
        graph.replay()
        b.step()
    torch.cuda.synchronize()
    for p, q in zip(a.params + a.opt.m + a.opt.v + a.grads, b.params + b.opt.m + b.opt.v + b.grads):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    assert int(a.count) == 4 and z.dust_last_device_error()[0] == 0


def test_steps_on_two_streams_at_once(z):
    """Two models stepping on streams of their own, interleaved, give what each gives alone."""
    import torch
    alone = [Model(z, 32), Model(z, 8)]
    both = [Model(z, 32), Model(z, 8)]
    for m in alone:
        for _ in range(3):
            m.step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for m, s in zip(both, streams):
            with torch.cuda.stream(s):
                m.step()
    torch.cuda.synchronize()
    for m, n in zip(alone, both):
        for p, q in zip(m.params + m.opt.m + m.opt.v, n.params + n.opt.m + n.opt.v):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    assert z.dust_last_device_error()[0] == 0
