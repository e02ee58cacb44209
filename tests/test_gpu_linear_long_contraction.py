"""bf16 outputs of long contractions.  The tensor cores truncate as they add, which shows most where all products have one sign: a
chain of products that is never handed over loses about 5e-9 of the sum for each of them, 8e-4 over 131072.

Bound: the sum is handed over every 512 products, that is 32 steps of 16, each off by at most two units of 2^-23 of the
chain's sum so far; the K / 512 sums, a bias and a residual are added with half a unit, 2^-24, of the total each.  x and W are positive, so the
sum of magnitudes is the sum.  On top, half a bf16 step: 2^-8 of the value."""
import pytest

from tests import _dev  # noqa: F401
from tests.test_gpu_linear_forms import launched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as zz
    zz.lib()
    return zz


def positive(g, rows, cols):
    """Rows of sizes that differ, so that the sums fall anywhere between two bf16 numbers."""
    import torch
    return (torch.rand(rows, cols, device="cuda", generator=g) * torch.exp2(4 * torch.rand(rows, 1, device="cuda", generator=g))).bfloat16()


def product(a, bt):
    import torch
    out = torch.zeros(a.shape[0], bt.shape[0], dtype=torch.float64, device="cuda")
    for k in range(0, a.shape[1], 16384):
        out += a[:, k:k + 16384].double() @ bt[:, k:k + 16384].double().t()
    return out


def check(got, ref, K):
    off = ref * (64 * 2.0 ** -23 + (K // 512 + 4) * 2.0 ** -24)
    over = ((got.double() - ref).abs() - off - 2.0 ** -8 * (ref + off)).max()
    assert float(over) <= 0, float(over / ref.max())


# the widths that the rule takes: 64, 128 and 256 columns a tile
@pytest.mark.parametrize("N,K,n_out", [(1100, 131088, 1152), (1000, 16400, 1296), (600, 16400, 1808), (5001, 16400, 1040),
                                       (1100, 16400, 2432)])
def test_forward_and_dx(z, N, K, n_out):
    import torch
    g = torch.Generator(device="cuda").manual_seed(K + n_out)
    x, W = positive(g, N, K), positive(g, n_out, K)
    ref = product(x, W)
    b = torch.rand(n_out, device="cuda", generator=g)
    y = torch.full((N + 2, n_out + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    names = launched(z, lambda: z.dust_linear(x, W, y=y[:N, :n_out]))
    assert len(names) == 1 and names[0].startswith("linear_tcgen05_") and "pair" not in names[0]
    check(y[:N, :n_out], ref, K)
    assert bool((y[N:] == 7).all()) and bool((y[:, n_out:] == 7).all())
    # the epilogue: bias, z, activation, residual
    res = torch.rand(N, n_out, device="cuda", generator=g).bfloat16()
    y2, pre = z.dust_linear(x, W, bias=b, act="relu", residual=res, z=True)
    with_b = ref + b.double()
    check(pre, with_b, K)
    check(y2, with_b + res.double(), K)
    # dx = dy W2 with dy = x as the gradient and W2 [K, n_out]: the same sums
    W2 = W.t().contiguous()
    dx, _, _ = z.dust_linear_backward(x, torch.zeros(N, n_out, dtype=torch.bfloat16, device="cuda"), W2, dW=None, db=None)
    check(dx, ref, K)
    assert z.dust_last_device_error()[0] == 0
