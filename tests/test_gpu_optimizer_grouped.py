"""DustOptimizer (dust_optimizer_step_grouped) against the formulas in 64 bits.

fp32 moments: m and v are each a product and a multiply-add of two terms with fp32 factors beta and 1 - beta
(four half steps, 2^-24, of the terms' magnitudes; one and a half more for the square); w loses half a step for the decay and half for
the update, and the update itself is right to 2^-19 relative (square root, quotient, bias corrections).
8-bit moments: the held value is the moment rounded to e4m3 of its block's scale: off by at most half a step,
2^-4 of the value or 2^-10 of the scale where that is larger, on top of the fp32 error; the weights use the moments
before they are rounded."""
import pytest

from tests import _dev  # noqa: F401

pytestmark = pytest.mark.gpu
SIZES = [1, 3, 4, 255, 256, 257, 1000, 4096, 4099, 20000, 0, 70001]
LR, EPS, WD = 1e-2, 1e-8, 0.1


@pytest.fixture(scope="module")
def z():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as zz
    zz.lib()
    return zz


def f32(x):
    import torch
    return float(torch.tensor(x, dtype=torch.float32))


B1, B2 = 0.9, 0.999


def make(z, sizes, bits, g_dt, seed, kind="adam"):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = [torch.randn(n, device="cuda", generator=g) for n in sizes]
    G = [(torch.randn(n, device="cuda", generator=g) * torch.exp(torch.randn(n, device="cuda", generator=g))).to(g_dt) for n in sizes]
    Wb = [torch.empty(n, dtype=torch.bfloat16, device="cuda") if i % 3 else None for i, n in enumerate(sizes)]
    decay = [float(i % 2) for i in range(len(sizes))]
    lrs = [1.0 if i % 4 else 0.5 for i in range(len(sizes))]
    return z.DustOptimizer(W, G, W_bf16=Wb, bits=bits, lr_scale=lrs, decay=decay), decay, lrs


def held(opt, i, what):
    """The values that tensor i's moment stands for, in 64 bits, and the scale of each element's block."""
    import torch
    n = opt.W[i].numel()
    if opt.bits == 32:
        return getattr(opt, what)[i].double(), None
    s = getattr(opt, what + "_scale")[i].double().repeat_interleave(256)[:n]
    return getattr(opt, what)[i].float().double() * s, s


def steps(z, opt, decay, lrs, n_steps, kind, gs, seed, dev_step=False):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    b1, b2, lr, wd, eps, mu = B1, B2, f32(LR), f32(WD), f32(EPS), f32(0.8)
    scale = torch.tensor([gs], device="cuda") if gs != 1.0 else None
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in range(1, n_steps + 1):
        for G in opt.G:
            G.copy_(torch.randn(G.shape, device="cuda", generator=g) * 0.3)
        before = [(w.double().clone(), held(opt, i, "m")[0].clone(), held(opt, i, "v")[0].clone()) for i, w in enumerate(opt.W)]
        count.fill_(t)
        if kind == "adam":
            opt.step(z.adam(LR, 1 if dev_step else t, B1, B2, EPS, WD), g_scale=scale, step=count if dev_step else None)
        else:
            opt.step(z.sgd_momentum(LR, 0.8, WD), g_scale=scale)
        torch.cuda.synchronize()
        for i, (w0, m0, v0) in enumerate(before):
            if w0.numel() == 0:
                continue
            G = opt.G[i].double() * f32(gs)
            if opt.bits == 8:
                v0 = v0.square()
            l, d = lr * lrs[i], wd * decay[i]
            w = w0 * (1 - l * d)
            if kind == "adam":
                m, v = b1 * m0 + (1 - b1) * G, b2 * v0 + (1 - b2) * G * G
                em = 4 * 2.0 ** -24 * (b1 * m0.abs() + (1 - b1) * G.abs())
                ev = 6 * 2.0 ** -24 * v
                c1, c2 = 1 - b1 ** t, 1 - b2 ** t
                den = (v / c2).sqrt() + eps
                step = l * (m / c1) / den
                es = step.abs() * 2.0 ** -19 + l * em / c1 / den
            else:
                m, v = mu * m0 + G, None
                em = 3 * 2.0 ** -24 * (mu * m0.abs() + G.abs())
                step, es = l * m, l * em
            ref = w - step
            tol = es + 2.0 ** -23 * (w0.abs() + step.abs() + ref.abs())
            assert bool(((opt.W[i].double() - ref).abs() <= tol).all()), (i, t, float(((opt.W[i].double() - ref).abs() - tol).max()))
            for name, x, e in (("m", m, em),) + ((("v", v, ev),) if kind == "adam" else ()):
                got, s = held(opt, i, name)
                if opt.bits == 8:
                    if name == "v":
                        x, e = v.sqrt(), 2.0 ** -21 * v.sqrt()
                    e = e + torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s) * (1 + 1e-5) + 2.0 ** -22 * x.abs()
                    if name == "v":  # a positive value keeps at least the smallest code
                        e = torch.maximum(e, 2.0 ** -9 * s * (1 + 1e-5))
                        assert bool((got[x > 0] > 0).all())
                    # the block's largest magnitude is held as the largest code
                    pad = torch.zeros(-(-x.numel() // 256) * 256, dtype=torch.float64, device="cuda")
                    pad[:x.numel()] = x.abs()
                    top = pad.view(-1, 256).amax(1)
                    have = getattr(opt, name + "_scale")[i].double() * 448
                    assert bool(((have - top).abs() <= 2.0 ** -19 * top).all())
                assert bool(((got - x).abs() <= e + 1e-37).all()), (name, i, t, float(((got - x).abs() - e).max()))
            if opt.W_bf16[i] is not None:
                assert torch.equal(opt.W_bf16[i], opt.W[i].to(torch.bfloat16))


@pytest.mark.parametrize("bits,kind", [(32, "adam"), (32, "sgd"), (8, "adam")])
@pytest.mark.parametrize("grad", ["f32", "bf16"])
@pytest.mark.parametrize("gs", [1.0, 0.125])
def test_steps(z, bits, kind, grad, gs):
    import torch
    opt, decay, lrs = make(z, SIZES, bits, torch.float32 if grad == "f32" else torch.bfloat16, 1)
    steps(z, opt, decay, lrs, 3, kind, gs, 2)


def test_eight_bit_codes_are_those_of_the_fp32_formulas(z):
    """Codes and scales bit for bit, against the formulas evaluated with one fp32 rounding an operation (numpy's
    fp32 arithmetic, and a conversion to e4m3 by rounding to its steps in 64 bits)."""
    import numpy as np
    import torch
    f = np.float32
    n = 256 * 2000
    rng = np.random.default_rng(11)
    size = np.exp(rng.standard_normal(n // 256).repeat(256)).astype(f)
    W = [torch.zeros(n, device="cuda")]
    G = torch.zeros(n, device="cuda")
    opt = z.DustOptimizer(W, [G], bits=8)
    gs = f(0.3)
    m, r = np.zeros(n, f), np.zeros(n, f)

    def hold(x, least):
        b = x.reshape(-1, 256)
        top = np.abs(b).max(1)
        near = (b * (f(448) / top)[:, None]).astype(f)
        near = np.where(near > 0, np.maximum(near, f(least)), near).astype(np.float64)
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(near), 2.0 ** -6))) - 3)
        code = np.rint(near / step) * step
        scale = (top * (f(1) / f(448))).astype(f)
        return code.astype(f), scale, (code.astype(f) * scale[:, None]).astype(f).reshape(-1)

    for t in range(1, 5):
        g = (rng.standard_normal(n).astype(f) * size).astype(f)
        G.copy_(torch.from_numpy(g))
        opt.step(z.adam(1e-3, t), g_scale=torch.tensor([float(gs)], device="cuda"))
        g = (g * gs).astype(f)
        m = m * f(0.9) + g * f(1 - 0.9)
        r = np.sqrt((r * r) * f(0.999) + (g * g) * f(1 - 0.999))
        for name, x, least in (("m", m, 0.0), ("v", r, 2.0 ** -9)):
            code, scale, held_x = hold(x, least)
            assert np.array_equal(getattr(opt, name + "_scale")[0].cpu().numpy(), scale), (name, t)
            assert np.array_equal(getattr(opt, name)[0].float().cpu().numpy(), code.reshape(-1)), (name, t)
            if name == "m":
                m = held_x
            else:
                r = held_x


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [32, 33, 256, 257, 300])
def test_many_tensors(z, bits, count):
    """Table sizes and several launches."""
    import torch
    opt, decay, lrs = make(z, [(7 * i) % 601 for i in range(count)], bits, torch.float32, 3)
    steps(z, opt, decay, lrs, 1, "adam", 1.0, 4)


@pytest.mark.parametrize("bits", [32, 8])
def test_step_count_on_the_device(z, bits):
    import torch
    opt, decay, lrs = make(z, [300, 5000], bits, torch.float32, 5)
    steps(z, opt, decay, lrs, 3, "adam", 1.0, 6, dev_step=True)


def test_same_as_one_tensor_at_a_time(z):
    """The step of dust_optimizer_step, within the two kernels' rounding; v also within 1.3e-5, since that call takes
    1 - beta2 from the fp32 beta2: |fl(0.999) - 0.999| = 1.29e-8, 1.29e-5 of 0.001.  (The bias correction
    1 - beta2^t carries the same factor at small t, so the weights agree to rounding.)"""
    import torch
    opt, _, _ = make(z, [10000, 77], 32, torch.float32, 7)
    opt = z.DustOptimizer(opt.W, opt.G)
    W = [w.clone() for w in opt.W]
    m, v = [torch.zeros_like(w) for w in W], [torch.zeros_like(w) for w in W]
    for t in (1, 2):
        opt.step(z.adam(1e-3, t, weight_decay=0.01))
        for i in range(2):
            z.dust_optimizer_step(z.adam(1e-3, t, weight_decay=0.01), opt.G[i], W[i], m[i], v[i])
    for i in range(2):
        assert torch.allclose(opt.W[i], W[i], rtol=1e-6, atol=1e-7)
        assert torch.allclose(opt.m[i], m[i], rtol=1e-6, atol=0) and torch.allclose(opt.v[i], v[i], rtol=1.4e-5, atol=0)


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_replay(z, bits):
    """A captured step with its count on the device, replayed three times, equals three eager steps."""
    import torch
    a, _, _ = make(z, [1000, 257], bits, torch.float32, 8)
    b, _, _ = make(z, [1000, 257], bits, torch.float32, 8)
    count = torch.ones(1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        a.step(z.adam(1e-3, 1, weight_decay=0.1), step=count)
        count.add_(1)
    for _ in range(3):
        graph.replay()
    cb = torch.ones(1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        b.step(z.adam(1e-3, 1, weight_decay=0.1), step=cb)
        cb.add_(1)
    torch.cuda.synchronize()
    for x, y in zip(a.W + a.m + a.v, b.W + b.m + b.v):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_eight_bit_special_values(z):
    """Zero blocks, tiny blocks, and a non-finite gradient that spoils its own block's moments only."""
    import torch
    n = 1024
    W, G = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    G[300] = 1e-33           # below the smallest magnitude that a block holds
    G[512 + 7] = float("inf")
    G[768:] = torch.linspace(-1, 1, 256, device="cuda")
    opt = z.DustOptimizer([W], [G], bits=8)
    opt.step(z.adam(1e-3, 1))
    torch.cuda.synchronize()
    m, sm = held(opt, 0, "m")
    r, sr = held(opt, 0, "v")
    assert bool((m[:512] == 0).all()) and bool((r[:512] == 0).all()) and bool((opt.m_scale[0][:2] == 0).all())
    assert bool(torch.isfinite(m[768:]).all()) and float(m[768:].abs().max()) > 0.09
    assert not bool(torch.isfinite(opt.m_scale[0][2])) and bool(torch.isfinite(opt.m_scale[0][3]))
    assert bool(torch.isfinite(W[:512 + 7]).all()) and bool(torch.isfinite(W[512 + 8:]).all())
    assert not bool(torch.isfinite(W[512 + 7]))


def test_eight_bit_average_does_not_stick(z):
    """After the gradients shrink tenfold the held sqrt(v) follows the exact average's decay: the median ratio
    stays within 5% (a half step is 6%; a code that could not move would leave it at 2 to 4)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)
    n = 256 * 64
    size = torch.exp(torch.randn(n, device="cuda", generator=g))
    W, G = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    a, b = z.DustOptimizer([W.clone()], [G], bits=8), z.DustOptimizer([W.clone()], [G], bits=32)
    for t in range(1, 601):
        G.copy_(torch.randn(n, device="cuda", generator=g) * size * (1.0 if t <= 200 else 0.1))
        for o in (a, b):
            o.step(z.adam(1e-3, t, beta2=0.99))
        if t in (200, 400, 600):
            ratio = held(a, 0, "v")[0] / b.v[0].double().sqrt()
            assert abs(float(ratio.median()) - 1) < 0.05, t


def test_refuses(z):
    import torch
    W, G = [torch.zeros(64, device="cuda"), torch.zeros(32, device="cuda")], [torch.zeros(64, device="cuda"), torch.zeros(32, device="cuda")]
    z.DustOptimizer(W, G)
    flat = torch.zeros(96, device="cuda")
    for bad in (lambda: z.DustOptimizer(W, G[:1]), lambda: z.DustOptimizer(W, G[::-1]), lambda: z.DustOptimizer(W, G, bits=16),
                lambda: z.DustOptimizer([W[0], W[0]], [G[0], G[0]]), lambda: z.DustOptimizer([flat[:64], flat[32:64]], G),
                lambda: z.DustOptimizer(W, G, m=[W[0], torch.zeros(32, device="cuda")]),
                lambda: z.DustOptimizer(W, G, W_bf16=[None]), lambda: z.DustOptimizer([w.half() for w in W], G),
                lambda: z.DustOptimizer(W, [G[0], G[1].bfloat16()]),
                lambda: z.DustOptimizer(W, G).step(z.adam(1e-3, 1), g_scale=torch.ones(2, device="cuda")),
                lambda: z.DustOptimizer(W, G).step(z.adam(1e-3, 1), step=torch.ones(1, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        z.DustOptimizer(W, [t.half() for t in G])
    with pytest.raises(z.DustError):
        z.DustOptimizer(W, G).step(z.adam(1e-3, 0))
    with pytest.raises(z.DustError):
        z.DustOptimizer(W, G, bits=8).step(z.sgd_momentum(0.1, 0.9))
