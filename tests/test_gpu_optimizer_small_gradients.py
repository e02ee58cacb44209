"""The Adam step of DustOptimizer where the second moment is subnormal and eps is smaller than its root.

From zero moments m = 0.1 g and v = fl(0.001 fl(g^2)), products of two fp32 numbers rounded once each (half a step of a subnormal
number is not small: v is taken as fp32 arithmetic leaves it, and the step is checked against the formula on that v).  The step
lr (m / c1) / (sqrt(v / c2) + eps) has a root, a quotient, two corrections and three products, each right to a few fp32
steps: within 2^-19 relative, and half a step of the smallest number for the products."""
import pytest

from tests import _dev  # noqa: F401

pytestmark = pytest.mark.gpu
LR = 1e-2


@pytest.fixture(scope="module")
def z():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as zz
    zz.lib()
    return zz


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-8, 1e-20, 1e-22, 1e-30])
def test_subnormal_second_moments(z, bits, eps):
    import numpy as np
    import torch
    f = np.float32
    n = 1024
    g = np.logspace(-20.5, -16, n).astype(f) * np.where(np.arange(n) % 2, f(1), f(-1))
    W = torch.zeros(n, device="cuda")
    opt = z.DustOptimizer([W], [torch.from_numpy(g).cuda()], bits=bits)
    opt.step(z.adam(LR, 1, 0.9, 0.999, eps))
    v = (f(1 - 0.999) * (g * g).astype(f)).astype(f)
    assert int((v > 0).sum()) > n // 2 and int(((v > 0) & (v < 1.17e-38)).sum()) > n // 4
    if bits == 32:
        assert np.array_equal(opt.v[0].cpu().numpy(), v)
    v, g = v.astype(np.float64), g.astype(np.float64)
    step = float(f(LR)) * g / (np.sqrt(v / float(1 - 0.999)) + float(f(eps)))
    off = np.abs(W.cpu().numpy().astype(np.float64) + step) - (2.0 ** -19 * np.abs(step) + 2.0 ** -149)
    assert off.max() <= 0, (float(off.max()), int(off.argmax()), float(step[off.argmax()]))


def test_agrees_with_one_tensor_at_a_time(z):
    """dust_optimizer_step takes 1 - beta2 from the fp32 beta2 (1.3e-5 off in v, which the first step's correction carries too:
    it cancels), so the steps agree to 2^-18 where v is a normal number, and to the rounding of a subnormal one, of
    which v has at least 2^7 steps here: half a step (2^-8) of each call's v, halved again by the root."""
    import torch
    g = torch.logspace(-18.9, -17, 512, device="cuda")
    W = torch.zeros(512, device="cuda")
    opt = z.DustOptimizer([W], [g])
    opt.step(z.adam(LR, 1, eps=1e-25))
    W1, m, v = torch.zeros_like(W), torch.zeros_like(W), torch.zeros_like(W)
    z.dust_optimizer_step(z.adam(LR, 1, eps=1e-25), g, W1, m, v)
    assert float((opt.v[0] / 2.0 ** -149).min()) >= 2 ** 7
    assert bool(((W - W1).abs() <= (2.0 ** -18 + 2.0 ** -8) * W1.abs()).all())
