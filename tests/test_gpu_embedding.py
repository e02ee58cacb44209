"""dust_embedding and dust_embedding_grad.

The lookup rounds the fp32 product scale E once (and once more to bf16): equal to the same product taken
in 64 bits and rounded the same way.  The gradient's row v is an fp32 sum of n_v terms: off by at most
(n_v + 2) 2^-24 times the sum of their magnitudes (half a step for each addition and for the scaling), and half a
step of the result with a previous value."""
import pytest

from tests import _dev  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def z():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as zz
    zz.lib()
    return zz


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _pitched(rows, cols, dtype, fill, g=None, extra=0):
    """A [rows, cols] view whose rows begin at multiples of 8 elements; all else holds `fill`."""
    import torch
    b = torch.full((rows + 2, -(-cols // 8) * 8 + extra), fill, dtype=dtype, device="cuda")
    if g is not None:
        b[:rows, :cols] = torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
    return b, b[:rows, :cols]


@pytest.mark.parametrize("N,V,d", [(1, 1, 1), (5, 7, 3), (33, 100, 48), (257, 50, 65), (1000, 4096, 256), (3, 9, 2049), (5000, 300, 24)])
@pytest.mark.parametrize("table", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_lookup(z, N, V, d, table, out):
    import torch
    g = torch.Generator(device="cuda").manual_seed(N + d)
    buf, E = _pitched(V, d, _dt(table), 3.0, g, extra=8 * (N & 1))
    ids = torch.randint(-2, V + 1, (N,), device="cuda", generator=g, dtype=torch.int32)
    obuf, o = _pitched(N, d, _dt(out), 7.0)
    scale = 1.0 if N & 1 else 0.37
    z.dust_embedding(ids, E, scale=scale, out=o)
    torch.cuda.synchronize()
    s32 = torch.tensor(scale, dtype=torch.float32).double()
    want = (E[ids.clamp(0, V - 1).long()].double() * s32).float()
    want[ids < 0] = 0
    want[ids >= V] = float("nan")
    assert torch.equal(torch.nan_to_num(o.float(), nan=99.0), torch.nan_to_num(want.to(_dt(out)).float(), nan=99.0))
    assert bool((obuf[N:] == 7).all()) and bool((obuf[:N, d:] == 7).all())


def grad_case(z, ids, V, d, dt, scale, accumulate, seed, extra=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = ids.numel()
    _, gr = _pitched(N, d, _dt(dt), float("nan"), g, extra=extra)
    Gbuf, G = _pitched(V, d, torch.float32, 7.0, g if accumulate else None, extra=extra)
    before = G.double().clone()
    z.dust_embedding_grad(ids, gr, V, scale=scale, G=G, accumulate=accumulate)
    torch.cuda.synchronize()
    live = (ids >= 0) & (ids < V)
    rows, terms = ids[live].long(), gr[live].double() * torch.tensor(scale, dtype=torch.float32).double().cuda()
    ref = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, rows, terms)
    mag = torch.zeros(V, d, dtype=torch.float64, device="cuda").index_add_(0, rows, terms.abs())
    n = torch.bincount(rows, minlength=V)[:, None].double()
    tol = (n + 2) * 2.0 ** -24 * mag * (1 + 1e-3)
    if accumulate:
        ref = ref + before
        tol = tol + 2.0 ** -24 * ref.abs()
        assert torch.equal(G[n[:, 0] == 0].double(), before[n[:, 0] == 0])
    else:
        assert bool((G[n[:, 0] == 0] == 0).all())
    assert bool(torch.isfinite(G).all())
    over = ((G.double() - ref).abs() - tol).max()
    assert float(over) <= 0, float(over)
    assert bool((Gbuf[V:] == 7).all()) and bool((Gbuf[:V, d:] == 7).all())
    return G


@pytest.mark.parametrize("N,V,d", [(1, 1, 1), (1, 5000, 40), (2, 3, 7), (31, 64, 130), (32, 64, 257), (33, 1, 48), (100, 511, 64),
                                   (1000, 512, 96), (4095, 300, 33), (4096, 40000, 16), (4097, 40000, 24), (20000, 70000, 8),
                                   (30000, 1000, 300)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient(z, N, V, d, dt, accumulate):
    import torch
    g = torch.Generator(device="cuda").manual_seed(N)
    ids = torch.randint(-1, V + 1, (N,), device="cuda", generator=g, dtype=torch.int32)
    grad_case(z, ids, V, d, dt, 1.0 if N & 1 else 2.5, accumulate, N + d, extra=8 * (N & 1))


@pytest.mark.parametrize("kind", ["one id", "last row", "all padding", "too large", "runs", "sorted", "reversed", "zipf"])
@pytest.mark.parametrize("N", [40, 3000, 9000])
def test_gradient_of_special_batches(z, kind, N):
    import torch
    V, d = 1030, 72
    at = torch.arange(N, device="cuda", dtype=torch.int32)
    ids = {"one id": at * 0 + 513, "last row": at * 0 + V - 1, "all padding": at * 0 - 1, "too large": at + V,
           "runs": (at // 97) % V, "sorted": (at * V) // N, "reversed": (N - 1 - at) % V,
           "zipf": (torch.exp(torch.rand(N, device="cuda") * 6.9) - 1).int()}[kind].to(torch.int32)
    for dt, accumulate in (("f32", False), ("bf16", True)):
        grad_case(z, ids, V, d, dt, 0.5, accumulate, 5)


@pytest.mark.parametrize("N", [4097, 8192, 8193, 12345, 16384, 16385])
@pytest.mark.parametrize("V", [1, 5, 511, 512, 70001, 1 << 20])
def test_sort_of_middle_batches(z, N, V):
    """Whole-number gradients below 2^24 in sum: every order of the sums gives the same bits, a lost, doubled or
    misplaced token does not."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(N + V)
    d = 12
    ids = torch.randint(-3, V + 3, (N,), device="cuda", dtype=torch.int32, generator=g)
    ids[N // 3: N // 2] = min(V - 1, 77)  # a long run
    gr = torch.randint(-500, 500, (N, d), device="cuda", generator=g).float()
    want = torch.zeros(V, d, dtype=torch.float64, device="cuda")
    ok = (ids >= 0) & (ids < V)
    want.index_add_(0, ids[ok].long(), gr[ok].double())
    for acc in (False, True):
        G = torch.full((V, d), 7.0, device="cuda")
        z.dust_embedding_grad(ids, gr, V, G=G, accumulate=acc)
        assert torch.equal(G.double(), want + (7.0 if acc else 0.0))


def test_long_chunks(z):
    """Enough tokens for chunks longer than 32, with ids that cross many of them."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    N = 300000
    ids = (torch.rand(N, device="cuda", generator=g) ** 4 * 50).to(torch.int32)
    grad_case(z, ids, 64, 40, "f32", 1.0, False, 2)
    grad_case(z, ids * 0 + 7, 64, 24, "bf16", 1.0, True, 3)


def test_three_sort_passes(z):
    import torch
    g = torch.Generator(device="cuda").manual_seed(4)
    V = (1 << 19) + 5
    for N in (700, 6000):
        ids = torch.randint(0, V, (N,), device="cuda", generator=g, dtype=torch.int32)
        ids[5:9] = V - 1
        grad_case(z, ids, V, 8, "f32", 1.0, False, N)


def test_repeats_bit_for_bit_and_in_a_graph(z):
    import torch
    g = torch.Generator(device="cuda").manual_seed(6)
    for N in (900, 30000):
        ids = (torch.rand(N, device="cuda", generator=g) ** 3 * 200).to(torch.int32)
        gr = torch.randn(N, 96, device="cuda", generator=g)
        E = torch.randn(200, 96, device="cuda", generator=g)
        G = z.dust_embedding_grad(ids, gr, 200).clone()
        out = z.dust_embedding(ids, E, scale=2.0).clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        assert torch.equal(z.dust_embedding_grad(ids, gr, 200), G)
        G2, out2 = z.dust_embedding_grad(ids, gr, 200, stream=s), z.dust_embedding(ids, E, scale=2.0, stream=s)
        s.synchronize()
        assert torch.equal(G2, G) and torch.equal(out2, out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            Gc, oc = z.dust_embedding_grad(ids, gr, 200), z.dust_embedding(ids, E, scale=2.0)
        ids.copy_(torch.flip(ids, dims=[0]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Gc, z.dust_embedding_grad(ids, gr, 200))
        assert torch.equal(oc, z.dust_embedding(ids, E, scale=2.0))


def test_a_nan_gradient_stays_in_its_row(z):
    import torch
    ids = torch.tensor([3, 1, 3, 2, -1, 9], dtype=torch.int32, device="cuda")
    gr = torch.ones(6, 16, device="cuda")
    gr[1, 4] = float("nan")
    gr[4] = float("nan")  # padding: not read into any row
    gr[5] = float("inf")  # an id behind the table
    G = z.dust_embedding_grad(ids, gr, 5)
    want = torch.zeros(5, 16, device="cuda")
    want[1], want[2], want[3] = 1, 1, 2
    want[1, 4] = float("nan")
    assert torch.equal(torch.nan_to_num(G, nan=99.0), torch.nan_to_num(want, nan=99.0))


def test_gradient_matches_differences(z):
    """The lookup is linear in E, so a difference along any direction is exact up to the fp32 sums."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(8)
    ids = torch.randint(-1, 30, (200,), device="cuda", generator=g, dtype=torch.int32)
    E, v = torch.randn(30, 40, device="cuda", generator=g), torch.randn(30, 40, device="cuda", generator=g)
    dy = torch.randn(200, 40, device="cuda", generator=g)
    G = z.dust_embedding_grad(ids, dy, 30, scale=1.5)
    num = ((z.dust_embedding(ids, E + v, scale=1.5).double() - z.dust_embedding(ids, E, scale=1.5).double()) * dy.double()).sum()
    have, size = (G.double() * v.double()).sum(), (G.double().abs() * v.double().abs()).sum()
    # E + v, the two lookups and the sums: a few fp32 half steps of terms no larger than a few units
    assert abs(float(num - have)) <= 2.0 ** -24 * (200 + 8) * float(size) + 6 * 2.0 ** -24 * 8 * 1.5 * float(dy.abs().sum())


def test_binding_refuses(z):
    import torch
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    E, gr = torch.zeros(5, 16, device="cuda"), torch.zeros(4, 16, device="cuda")
    for bad in (lambda: z.dust_embedding(ids[::2], E), lambda: z.dust_embedding(ids, E[0]), lambda: z.dust_embedding(ids, E.t()),
                lambda: z.dust_embedding(ids, E, out=gr[:3]), lambda: z.dust_embedding_grad(ids, gr[:3], 5),
                lambda: z.dust_embedding_grad(ids, gr, 5, accumulate=True), lambda: z.dust_embedding_grad(ids, gr, 5, G=E[:4])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: z.dust_embedding(ids.long(), E), lambda: z.dust_embedding(ids, E.half()),
                lambda: z.dust_embedding_grad(ids, gr.half(), 5), lambda: z.dust_embedding_grad(ids, gr, 5, G=E.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(z.DustError):
        z.dust_embedding(ids, torch.zeros(5, 15, device="cuda"))  # rows off the 16-byte grid
    with pytest.raises(z.DustError):
        z.dust_embedding_grad(ids, gr, 0)
