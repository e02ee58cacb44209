"""The table's gradient at the largest number of rows that the call accepts (2^31 - 2; the table is 34 GB)."""
import pytest

from tests import _dev  # noqa: F401

pytestmark = pytest.mark.gpu


def test_most_rows():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as z
    V = 2 ** 31 - 2
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB of device memory")
    G = torch.full((V, 4), 3.0, device="cuda")
    for N in (6, 5000):  # one launch, and the sorted form
        ids = torch.full((N,), -1, dtype=torch.int32, device="cuda")
        ids[:6] = torch.tensor([0, V - 1, 2 ** 30, V - 1, V - 20, 2 ** 31 - 1], dtype=torch.int32)
        g = torch.full((N, 1), float("nan"), device="cuda")
        g[:6, 0] = torch.tensor([1.0, 2.0, 4.0, 8.0, 16.0, 32.0])
        view = torch.zeros(N, 4, device="cuda")
        view[:, :1] = g
        G[:, 0] = 3.0
        z.dust_embedding_grad(ids, view[:, :1], V, G=G[:, :1])
        rows = torch.tensor([0, V - 1, 2 ** 30, V - 20], device="cuda")
        assert G[rows, 0].tolist() == [1.0, 10.0, 4.0, 16.0]
        G[rows, 0] = 0.0
        assert float(G[:, 0].abs().max()) == 0.0 and float(G[::4097, 1:].min()) == 3.0
    del G
    torch.cuda.empty_cache()
