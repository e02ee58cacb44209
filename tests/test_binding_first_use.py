"""The binding's tables are filled at the first use: a second thread that comes in between sees none of a table or all of it (CPU
only)."""
import zeroth_order_transformer_b200 as z


def test_table_of_types_is_never_half_filled(monkeypatch):
    import torch
    seen = []

    class Watched(dict):
        def __setitem__(self, k, v):
            super().__setitem__(k, v)
            seen.append(set(z._dtypes()))  # what a thread that runs now would get

    monkeypatch.setattr(z, "_DT", Watched())
    both = {torch.bfloat16, torch.float32}
    assert set(z._dtypes()) == both and all(s == both for s in seen)
    assert z._dtypes()[torch.bfloat16] == z.DUST_BF16 and z._dtypes()[torch.float32] == z.DUST_F32
