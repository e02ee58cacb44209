"""Infinite output gradients through dust_linear_backward: what the formula makes infinite is so, with its sign, and not NaN, also
where dz goes to the tensor cores as two bf16 terms."""
import pytest

from tests import _dev  # noqa: F401
from tests.test_gpu_linear import act64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as zz
    zz.lib()
    return zz


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("dy_f32", [False, True])
@pytest.mark.parametrize("terms", [1, 2])
@pytest.mark.parametrize("N", [5, 333])
def test_infinite_gradient(z, act, dy_f32, terms, N):
    import torch
    g = torch.Generator(device="cuda").manual_seed(N)
    d_in, d_out = 80, 144
    dt = torch.float32 if dy_f32 else torch.bfloat16

    def nonzero(*shape):
        t = torch.randn(shape, device="cuda", generator=g)
        return torch.where(t < 0, t - 0.1, t + 0.1)

    x, W = nonzero(N, d_in).bfloat16(), nonzero(d_out, d_in).bfloat16()
    pre = (0.5 + torch.rand(N, d_out, device="cuda", generator=g)).bfloat16()  # where every slope is positive
    dy = nonzero(N, d_out).to(dt)
    inf = float("inf")
    dy[N - 1, 3], dy[0, 17], dy[2, 140] = inf, -inf, inf
    dx, dW, db = z.dust_linear_backward(dy, x, W, act=act, z=pre if act != "none" else None, dx_dtype=torch.float32, g_terms=terms)
    slope = act64(pre.double(), act)[1] if act != "none" else torch.ones(N, d_out, dtype=torch.float64, device="cuda")
    dz = dy.double() * slope

    def kind(t):  # 0 finite, 1 and 2 the infinities, 3 NaN
        return torch.isposinf(t).int() + 2 * torch.isneginf(t).int() + 3 * torch.isnan(t).int()

    # one product at a time: a library product may form 0 times infinity
    for got, want in ((dW, (dz.t()[:, :, None] * x.double()[None]).sum(1)), (dx, (dz[:, :, None] * W.double()[None]).sum(1)),
                      (db, dz.sum(0))):
        assert int((kind(want) > 0).sum()) > 0 and torch.equal(kind(got), kind(want))
    assert z.dust_last_device_error()[0] == 0
