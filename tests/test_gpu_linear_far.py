"""Far pre-activations, infinities and NaN through every form of the product: each column has a value of its own from the bias, so
every form sees all of them.  Where an activation is at its limit, y is the value or zero; in between it is the formula's,
within 2^-19 (1 + |z|), and half a bf16 step where y is bf16."""
import pytest

from tests import _dev  # noqa: F401
from tests.test_gpu_linear import ACTS, act64

pytestmark = pytest.mark.gpu
FAR = [float("-inf"), -3e38, -1e30, -1e4, -200.0, -90.0, -30.0, -3.0, 0.0, 3.0, 30.0, 90.0, 200.0, 1e4, 1e30, 3e38, float("inf"),
       float("nan")]


@pytest.fixture(scope="module")
def z():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as zz
    zz.lib()
    return zz


def limit(v, act):
    import torch
    if act == "none" or v != v or v > 20:
        return v
    return 0.0 if v < -20 else float(act64(torch.tensor(v, dtype=torch.float64), act)[0])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("N,d_in,d_out", [(1, 16, 288), (2, 48, 288), (13, 16, 288), (40, 2048, 288), (600, 16, 288), (1100, 640, 2432),
                                          (1100, 768, 2432)])
def test_outputs(z, N, d_in, d_out, act, out, residual):
    import torch
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    x = torch.zeros(N, d_in, dtype=torch.bfloat16, device="cuda")
    W = torch.ones(d_out, d_in, dtype=torch.bfloat16, device="cuda")
    far = (FAR * (d_out // len(FAR) + 1))[:d_out]
    b = torch.tensor(far, dtype=torch.float32, device="cuda")
    res = torch.full((N, d_out), 0.5, dtype=dt, device="cuda") if residual else None
    y, pre = z.dust_linear(x, W, bias=b, act=act, residual=res, out_dtype=dt, z=True)
    add = 0.5 if residual else 0.0
    want = torch.tensor([limit(v, act) + add for v in far], dtype=torch.float64, device="cuda")
    near = torch.where(b.abs() < 20, 2.0 ** -19 * (1 + b.abs().double()), torch.zeros_like(want))
    half = 2.0 ** -8 if out == "bf16" else 2.0 ** -23
    fin = torch.isfinite(want)
    off = (y.double() - want).abs()[:, fin] - (near + half * (want.abs() + near) + 1e-9)[fin]
    assert float(off.max()) <= 0
    assert bool((torch.nan_to_num(y.double(), nan=7.0)[:, ~fin] == torch.nan_to_num(want, nan=7.0)[~fin]).all())
    assert torch.equal(torch.nan_to_num(pre.double(), nan=7.0),
                       torch.nan_to_num(b.bfloat16().double(), nan=7.0).expand(N, d_out))
    assert z.dust_last_device_error()[0] == 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N", [1, 13, 600])
def test_slopes(z, act, N):
    import torch
    far = [v for v in FAR if v == v]
    d_out = 16 * len(far)
    pre = torch.tensor(far * 16, dtype=torch.float32, device="cuda").bfloat16().expand(N, d_out).contiguous()
    x = torch.ones(N, 32, dtype=torch.bfloat16, device="cuda")
    W = torch.ones(d_out, 32, dtype=torch.bfloat16, device="cuda")
    dy = torch.ones(N, d_out, device="cuda")
    dx, dW, db = z.dust_linear_backward(dy, x, W, act=act, z=pre, dx_dtype=torch.float32)
    slope = torch.tensor([1.0 if act == "none" or v > 20 else 0.0 if v < -20 else float(act64(torch.tensor(v, dtype=torch.float64), act)[1])
                          for v in far * 16], dtype=torch.float64, device="cuda")
    tol = 2.0 ** -19 + 2.0 ** -16  # a slope, and its two bf16 terms
    assert bool(((db.double() - N * slope).abs() <= N * tol).all())
    assert bool(((dW.double() - N * slope[:, None]).abs() <= N * tol).all())
    assert bool(((dx.double() - slope.sum()).abs() <= d_out * tol).all())
