"""Every form of the linear layer's products, with the form that ran read from the launches' names: tile widths, pairs of CTAs
(an odd count of row tiles leaves the last pair's second CTA without rows; widths that end before the second half of
the last pair's columns), fp32 outputs collected in registers, dW of one and two terms, splits."""
import pytest

from tests import _dev  # noqa: F401
from tests import test_gpu_linear as layer
from tests.test_gpu_linear import _bf, _gen, back_case, fwd_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as zz
    zz.lib()
    return zz


def launched(z, run):
    """The names of the launches that `run` makes."""
    z.dust_profile_enable(64)
    try:
        run()
        return [name for name, _ in z.dust_profile_read()]
    finally:
        z.dust_profile_disable()


# N, d_in, d_out -> forms of y in bf16 and in fp32
FORWARD = [
    (1, 256, 320, "linear_rows", "linear_rows"),
    (2, 256, 320, "linear_rows", "linear_rows"),
    (3, 256, 320, "linear_tokens_tcgen05_16", "linear_tokens_tcgen05_16"),
    (24, 1040, 320, "linear_tokens_tcgen05_32", "linear_tokens_tcgen05_32"),
    (60, 1552, 400, "linear_tokens_tcgen05_64", "linear_tokens_tcgen05_64"),
    (200, 2576, 1296, "linear_tokens_tcgen05_128", "linear_tokens_tcgen05_128"),
    (300, 208, 400, "linear_tcgen05_64", "linear_tcgen05_64"),
    (5001, 1024, 1024, "linear_tcgen05_128", "linear_tcgen05_128"),
    (1100, 640, 2432, "linear_tcgen05_256", "linear_tcgen05_256"),
    (1000, 640, 2576, "linear_tcgen05_256", "linear_tcgen05_256"),
    (1000, 768, 2432, "linear_tcgen05_256_pair", "linear_tcgen05_256"),  # eight row tiles; the last columns end at a half
    (1100, 768, 2432, "linear_tcgen05_256_pair", "linear_tcgen05_256"),  # nine row tiles
    (1000, 784, 2576, "linear_tcgen05_256_pair", "linear_tcgen05_256"),  # sixteen columns in the last tile
    (1100, 800, 2704, "linear_tcgen05_256_pair", "linear_tcgen05_256"),  # sixteen columns in the last tile's second half
    (5000, 768, 2432, "linear_tcgen05_256_pair", "linear_tcgen05_256"),  # several tiles for each pair
]


@pytest.mark.parametrize("N,d_in,d_out,bf16,f32", FORWARD)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("extras", ["none", "bias z", "bias residual", "all, rows apart"])
def test_forward(z, N, d_in, d_out, bf16, f32, out, extras):
    k = (N + d_in + len(extras)) % 4
    act = ["none", "gelu", "silu", "gelu_tanh"][k] if extras != "none" else "none"
    got = launched(z, lambda: fwd_case(z, N, d_in, d_out, act, "bias" in extras or "all" in extras,
                                       "residual" in extras or "all" in extras, "z" in extras or "all" in extras, out, N + k,
                                       ld_extra=8 if "apart" in extras else 0))
    assert got == [bf16 if out == "bf16" else f32]


@pytest.mark.parametrize("N,d_in,d_out,bf16,f32", FORWARD)
def test_residual_buffer_as_output(z, N, d_in, d_out, bf16, f32):
    import torch
    g = _gen(N)
    x, W, b = _bf(g, N, d_in), _bf(g, d_out, d_in, std=d_in ** -0.5), torch.randn(d_out, device="cuda", generator=g)
    for dt in (torch.bfloat16, torch.float32):
        r = torch.randn(N, d_out, device="cuda", generator=g).to(dt)
        want = z.dust_linear(x, W, bias=b, act="silu", residual=r, out_dtype=dt)
        got = z.dust_linear(x, W, bias=b, act="silu", residual=r, y=r)
        assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)


# N, d_in, d_out -> form of dx in bf16, in fp32 with two terms, form of dW, whether dW is split
BACKWARD = [
    (7, 320, 256, "tokens_tcgen05_16", "64", "64", False),
    (60, 400, 1552, "tokens_tcgen05_64", "64", "64", False),
    (1100, 2432, 768, "256_pair", "256", "128", False),
    (1000, 2576, 784, "256_pair", "256", "128", False),
    (1100, 2704, 800, "256_pair", "256", "256", False),
    (1100, 2432, 640, "256", "256", "128", False),
    (230, 1296, 1936, "64", "64", "256", False),
    (4300, 1280, 528, "128", "128", "256", True),
    (5001, 1024, 1024, "128", "128", "128", True),
]


@pytest.mark.parametrize("N,d_in,d_out,dx16,dx32,dw,split", BACKWARD)
@pytest.mark.parametrize("act,dy,dx,terms", [("none", "bf16", "bf16", 2), ("none", "f32", "bf16", 2), ("none", "f32", "f32", 2), ("gelu", "bf16", "f32", 2), ("silu", "f32", "f32", 1),
                                             ("gelu_tanh", "bf16", "bf16", 1)])
def test_backward(z, N, d_in, d_out, dx16, dx32, dw, split, act, dy, dx, terms):
    import torch
    dts = {"bf16": torch.bfloat16, "f32": torch.float32}
    for accumulate in (False, True):
        got = launched(z, lambda: back_case(z, N, d_in, d_out, act, dts[dy], dts[dx], terms, accumulate, N + d_in,
                                            ld_extra=8 * accumulate))
        form = {n[len("linear_"):] for n in got}
        two = terms == 2 and not (act == "none" and dy == "bf16")
        want = dx16 if dx == "bf16" or (not two and "tokens" in dx16) else dx32
        assert "dx_" + (want if "tokens" in want else "tcgen05_" + want) in form, got
        assert f"dw_tcgen05_{dw}" + ("_two_terms" if two else "") in form, got
        assert "join" in form and "dz" in form, got
    # dW alone: the sums of its splits are a launch of their own
    g = _gen(N)
    args = _bf(g, N, d_out), _bf(g, N, d_in), _bf(g, d_out, d_in)
    got = launched(z, lambda: z.dust_linear_backward(*args, dx=None, db=None))
    assert got == [f"linear_dw_tcgen05_{dw}"] + (["linear_join"] if split else []), got


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("outs", ["dx dW db", "dx dW"])
def test_overlapping_launches_of_pairs(z, act, outs):
    """The chain of overlapping backward calls, eager and captured, where dx goes to pairs of CTAs and dW to 256-wide tiles."""
    N, d = 16384, 768
    g = _gen(3)
    dy, x, W = _bf(g, N, d), _bf(g, N, d), _bf(g, d, d, std=d ** -0.5)
    names = launched(z, lambda: z.dust_linear_backward(dy, x, W, act, z=dy if act != "none" else None))
    assert "linear_dx_tcgen05_256_pair" in names and any(n.startswith("linear_dw_tcgen05_256") for n in names), names
    layer.test_calls_in_a_row_equal_calls_waited_for(z, act, N, d, outs)


def test_forward_pairs_repeat_in_a_graph(z):
    """Pairs one after the other, each reading what the one before wrote, eager and captured: bit for bit the results of calls that
    were waited for."""
    import torch
    g = _gen(4)
    N, d = 1100, 2432
    W = _bf(g, d, d, std=d ** -0.5)
    x0, bufs = _bf(g, N, d), [torch.empty(N, d, dtype=torch.bfloat16, device="cuda") for _ in range(5)]
    assert launched(z, lambda: z.dust_linear(x0, W)) == ["linear_tcgen05_256_pair"]

    def chain(wait):
        x = x0
        for y in bufs:
            z.dust_linear(x, W, act="silu", residual=x, y=y)
            if wait:
                torch.cuda.synchronize()
            x = y

    chain(True)
    want = [t.clone() for t in bufs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain(False)
    for run in (lambda: chain(False), graph.replay) * 3:
        for t in bufs:
            t.zero_()
        run()
        assert all(torch.equal(a, b) for a, b in zip(bufs, want))
