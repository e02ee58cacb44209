"""DustOptimizer refuses gradients that share memory with what a step writes: the kernel would read elements that other threads
have already updated."""
import pytest

from tests import _dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_apart_from_weights_and_moments(bits):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as z
    f = lambda n: torch.zeros(n, device="cuda")  # noqa: E731
    W, G = [f(512), f(256)], [f(512), f(256)]
    half = [torch.zeros(512, dtype=torch.bfloat16, device="cuda"), None]
    opt = z.DustOptimizer(W, G, W_bf16=half, bits=bits)
    held = torch.zeros(1024, device="cuda")
    for bad in ([W[0], G[1]], [G[0], W[0][:256]], [G[0], W[0][256:]]):
        with pytest.raises(ValueError):
            z.DustOptimizer(W, bad, bits=bits)
        with pytest.raises(ValueError):
            opt.set_gradients(bad)
    with pytest.raises(ValueError):  # a weight in the middle of a gradient
        z.DustOptimizer([held[256:512], W[1]], [held[128:384], G[1]], bits=bits)
    with pytest.raises(ValueError):  # the bf16 copy
        opt.set_gradients([half[0], torch.zeros(256, dtype=torch.bfloat16, device="cuda")])
    if bits == 32:
        with pytest.raises(ValueError):
            opt.set_gradients([opt.m[0], G[1]])
        with pytest.raises(ValueError):
            opt.set_gradients([G[0], opt.v[1]])
    # after a refusal the gradients are those that were there
    G[0].fill_(1.0)
    opt.step(z.adam(1e-2, 1))
    assert bool((W[0] < 0).all()) and bool((W[1] == 0).all())
    # neighbours, and one gradient for two tensors, are no overlap
    z.DustOptimizer([held[:256]], [held[256:512]], bits=bits).step(z.adam(1e-2, 1))
    two = z.DustOptimizer([f(256), f(256)], [G[1], G[1]], bits=bits)
    two.step(z.adam(1e-2, 1))
