"""A padding token's row is zero whatever the scale, an infinite or NaN one among them."""
import pytest

from tests import _dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [float("inf"), float("-inf"), float("nan"), -2.0])
@pytest.mark.parametrize("d", [16, 13])
def test_padding_rows(scale, d):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as z
    ids = torch.tensor([1, -1, 0, 7, -5], dtype=torch.int32, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        E = torch.ones(3, 16, dtype=dt, device="cuda")[:, :d]
        for out_dt in (torch.bfloat16, torch.float32):
            out = z.dust_embedding(ids, E, scale=scale, out_dtype=out_dt).float()
            assert bool((out[[1, 4]] == 0).all()) and bool(torch.isnan(out[3]).all())
            live, want = out[[0, 2]], torch.full((2, d), scale, device="cuda")
            assert bool(torch.isnan(live).all()) if scale != scale else torch.equal(live, want)
