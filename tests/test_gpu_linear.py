"""dust_linear and dust_linear_backward against plain 64-bit products.

Tolerances, element by element, with A the same sum taken over magnitudes (|x| |W|^T + |b| and so on): an
fp32 sum of n terms is off by at most n steps of 2^-23 A (one step, not half of one, for each addition: the
tensor cores may truncate).  An output in bf16 adds half its step, 2^-8 relative; an operand dz held as one
bf16 term 2^-8, as two terms 2^-16 relative.  The activations and their slopes are off by at most 2^-19 (1 + |z|)
(a few fp32 steps of each factor, the exponential's argument rounded to 2^-24 relative where |u| exp(-u) <
0.4) and scale an error of z by at most 1.2."""
import math

import pytest

from tests import _dev  # noqa: F401  (lazy torch)

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module")
def z():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import zeroth_order_transformer_b200 as zz
    zz.lib()
    return zz


def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def _bf(g, *shape, std=1.0):
    import torch
    return (torch.randn(shape, device="cuda", generator=g) * std).to(torch.bfloat16)


def act64(x, act):
    """(act, act') in 64 bits."""
    import torch
    if act == "relu":
        return x.clamp(min=0), (x > 0).double()
    if act == "gelu":
        c = 0.5 * torch.erfc(-x / math.sqrt(2))
        return x * c, c + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (x + 0.044715 * x ** 3))
        return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * k * (1 + 0.134145 * x * x)
    if act == "silu":
        p = torch.sigmoid(x)
        return x * p, p * (1 + x * (1 - p))
    return x, torch.ones_like(x)


def check(got, ref, tol, what):
    import torch
    assert got.shape == ref.shape, what
    g = got.double()
    assert bool(torch.isfinite(g).all()), what
    over = ((g - ref).abs() - tol).max()
    assert float(over) <= 0, (what, float(over), float((g - ref).abs().max()))


def fwd_case(z, N, d_in, d_out, act, bias, residual, keep, out, seed, ld_extra=0):
    import torch
    g = _gen(seed)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[out]

    def wide(t):  # the same matrix as a view of a wider buffer
        if not ld_extra:
            return t
        b = torch.full((t.shape[0], t.shape[1] + ld_extra), float("nan"), dtype=t.dtype, device="cuda")
        b[:, :t.shape[1]] = t
        return b[:, :t.shape[1]]

    x, W = wide(_bf(g, N, d_in)), _bf(g, d_out, d_in, std=d_in ** -0.5)
    b = torch.randn(d_out, device="cuda", generator=g) if bias else None
    res = wide(torch.randn(N, d_out, device="cuda", generator=g).to(dt)) if residual else None
    y = torch.full((N + 3, d_out + ld_extra), 7.0, dtype=dt, device="cuda")
    zz = torch.full((N + 3, d_out + ld_extra), 7.0, dtype=torch.bfloat16, device="cuda") if keep else None
    got = z.dust_linear(x, W, bias=b, act=act, residual=res, y=y[:N, :d_out], z=zz[:N, :d_out] if keep else None)
    torch.cuda.synchronize()
    pre = x.double() @ W.double().t()
    A = x.double().abs() @ W.double().abs().t()
    if bias:
        pre, A = pre + b.double(), A + b.double().abs()
    ref = act64(pre, act)[0]
    off = 1.2 * (d_in + 16) * 2.0 ** -23 * A + 2.0 ** -19 * (1 + pre.abs())
    if residual:
        ref = ref + res.double()
        off = off + 2.0 ** -23 * ref.abs()
    half = 2.0 ** -8 if out == "bf16" else 2.0 ** -24
    check(y[:N, :d_out], ref, off + half * (ref.abs() + off), (N, d_in, d_out, act))
    if keep:
        assert got[1].data_ptr() == zz.data_ptr()
        offz = (d_in + 16) * 2.0 ** -23 * A
        check(zz[:N, :d_out], pre, offz + 2.0 ** -8 * (pre.abs() + offz), "z")
        assert bool((zz[N:] == 7).all()) and bool((zz[:, d_out:] == 7).all())
    # nothing behind the last row or column is written
    assert bool((y[N:] == 7).all()) and bool((y[:, d_out:] == 7).all())
    assert z.dust_last_device_error()[0] == 0


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 8, 9, 33])
@pytest.mark.parametrize("d_in,d_out", [(16, 16), (48, 272), (528, 64), (1040, 144)])
def test_few_tokens(z, N, d_in, d_out):
    k = N + d_in
    fwd_case(z, N, d_in, d_out, ACTS[k % 5], bool(k & 1), bool(k & 2), bool(k & 4), ["bf16", "f32"][(k >> 1) & 1], k)


@pytest.mark.parametrize("N,d_in,d_out", [(9, 128, 64), (24, 2048, 512), (128, 4112, 80), (129, 784, 336), (100, 64, 4112), (17, 320, 1040),
                                          (300, 1552, 16), (60, 1552, 400), (200, 2576, 1296), (513, 4112, 272)])
def test_contraction_over_a_cluster(z, N, d_in, d_out):
    """Few output tiles and contractions of one to many blocks, shares that are short or empty among them."""
    for k, out in enumerate(("bf16", "f32")):
        fwd_case(z, N, d_in, d_out, ACTS[(N + k) % 5], True, bool((N + k) & 1), True, out, N + k, ld_extra=8 * k)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_activations(z, act, out):
    fwd_case(z, 200, 112, 320, act, True, False, True, out, 5)


@pytest.mark.parametrize("N,d_in,d_out", [(127, 64, 256), (128, 80, 512), (129, 208, 48), (1000, 256, 784), (300, 1040, 4112),
                                          (5000, 144, 1040)])
@pytest.mark.parametrize("residual", [False, True])
def test_tiles(z, N, d_in, d_out, residual):
    fwd_case(z, N, d_in, d_out, "none", True, residual, False, "bf16", N + d_out)


@pytest.mark.parametrize("N", [1, 6, 150])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_rows_further_apart(z, N, out):
    fwd_case(z, N, 96, 176, "silu", True, True, True, out, N, ld_extra=24)


def test_more_tiles_than_ctas(z):
    """Several tiles for each CTA, so both accumulators are refilled."""
    fwd_case(z, 128 * 40, 256, 256 * 9, "gelu", True, True, True, "bf16", 3)


def test_far_pre_activations(z):
    """Far out the activations and their slopes are at their limits, at infinity too; a NaN stays one."""
    import torch
    inf = float("inf")
    far = torch.tensor([-inf, -1e30, -1e4, -200, -90, -30, 0, 30, 90, 200, 1e4, 1e30, inf], device="cuda")
    W = torch.eye(16, dtype=torch.bfloat16, device="cuda")[:, :16].contiguous()
    for N in (1, 2, 13, 600):  # one for each form of the product
        for k in range(0, 13, max(1, min(N, 13))):
            x = torch.zeros(N, 16, dtype=torch.bfloat16, device="cuda")
            # an infinite input times the zeros of W would be NaN: the bias brings the value
            v = far[(torch.arange(N, device="cuda") + k) % 13]
            for t in range(min(N, 13)):
                b = torch.full((16,), float(v[t]), device="cuda")
                for act in ACTS:
                    y, pre = z.dust_linear(x, W, bias=b, act=act, out_dtype=torch.float32, z=True)
                    lim = float(v[t])
                    want = lim if act == "none" or lim > 20 else 0.0
                    if lim == -30 or lim == 0:
                        want = float(act64(v[t].double(), act)[0])
                    assert torch.allclose(y, torch.full_like(y, want), rtol=1e-6, atol=1e-6), (N, act, lim, y[0, 0])
                    dy = torch.ones(N, 16, device="cuda")
                    _, _, db = z.dust_linear_backward(dy, x, W, act=act, z=pre, dx=None, dW=None)
                    slope = 1.0 if act == "none" or lim > 20 else 0.0 if lim < -20 else float(act64(v[t].double(), act)[1])
                    assert torch.allclose(db, torch.full_like(db, N * slope), rtol=1e-5, atol=1e-6), (N, act, lim, db[0])
                if N > 2:
                    break


def test_residual_buffer_as_output(z):
    import torch
    g = _gen(9)
    for N in (7, 700):
        x, W, r = _bf(g, N, 128), _bf(g, 256, 128, std=0.1), _bf(g, N, 256)
        want = z.dust_linear(x, W, act="gelu", residual=r)
        got = z.dust_linear(x, W, act="gelu", residual=r, y=r)
        assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)


def test_not_a_number_stays_in_its_row(z):
    import torch
    g = _gen(10)
    for N in (8, 300):
        x, W = _bf(g, N, 64), _bf(g, 128, 64)
        x[3, 5] = float("nan")
        for act in ACTS:
            y = z.dust_linear(x, W, act=act)
            bad = torch.isnan(y)
            assert bool(bad[3].all()) and int(bad.sum()) == 128, act


# ------------------------------------------------------------------------------------------ backward

def back_case(z, N, d_in, d_out, act, dy_dt, dx_dt, terms, accumulate, seed, ld_extra=0):
    import torch
    g = _gen(seed)

    def wide(t):
        if not ld_extra:
            return t
        b = torch.full((t.shape[0], t.shape[1] + ld_extra), float("nan"), dtype=t.dtype, device="cuda")
        b[:, :t.shape[1]] = t
        return b[:, :t.shape[1]]

    x, W = wide(_bf(g, N, d_in)), _bf(g, d_out, d_in, std=d_in ** -0.5)
    zz = wide(_bf(g, N, d_out, std=1.5)) if act != "none" else None
    dy = wide((torch.randn(N, d_out, device="cuda", generator=g) * 1e-2).to(dy_dt))
    dx = torch.full((N + 2, d_in + ld_extra), 7.0, dtype=dx_dt, device="cuda")
    dW0, db0 = torch.randn(d_out, d_in, device="cuda", generator=g), torch.randn(d_out, device="cuda", generator=g)
    dW, db = dW0.clone(), db0.clone()
    z.dust_linear_backward(dy, x, W, act=act, z=zz, dx=dx[:N, :d_in], dW=dW, db=db, accumulate=accumulate, g_terms=terms)
    torch.cuda.synchronize()
    slope = act64(zz.double(), act)[1] if zz is not None else 1.0
    dz = dy.double() * slope
    # the slope's own error, and dz rounded to its terms
    e_sl = dy.double().abs() * 2.0 ** -19 * (1 + (zz.double().abs() if zz is not None else 0))
    exact = act == "none" and dy_dt == torch.bfloat16
    held = 0.0 if exact else 2.0 ** -16 if terms == 2 else 2.0 ** -8
    held_dx = 0.0 if exact else 2.0 ** -8 if (terms == 1 or dx_dt == torch.bfloat16) else 2.0 ** -16
    aW, ax = W.double().abs(), x.double().abs()
    ref = dz @ W.double()
    off = (dz.abs() @ aW) * (held_dx + (2 * d_out + 16) * 2.0 ** -23) + 1.01 * (e_sl @ aW)
    half = 2.0 ** -8 if dx_dt == torch.bfloat16 else 2.0 ** -24
    check(dx[:N, :d_in], ref, off + half * (ref.abs() + off) + 1e-30, "dx")
    assert bool((dx[N:] == 7).all()) and bool((dx[:, d_in:] == 7).all())
    ref = dz.t() @ x.double()
    off = (dz.abs().t() @ ax) * (held + (2 * N + 40) * 2.0 ** -23) + 1.01 * (e_sl.t() @ ax)
    if accumulate:
        ref = ref + dW0.double()
        off = off + 2.0 ** -23 * (ref.abs() + dW0.double().abs())
    check(dW, ref, off + 1e-30, "dW")
    ref, off = dz.sum(0), dz.abs().sum(0) * (N + 8) * 2.0 ** -23 + 1.01 * e_sl.sum(0)
    if accumulate:
        ref = ref + db0.double()
        off = off + 2.0 ** -23 * (ref.abs() + db0.double().abs())
    check(db, ref, off + 1e-30, "db")
    assert z.dust_last_device_error()[0] == 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("terms", [1, 2])
@pytest.mark.parametrize("f32", [False, True])
def test_backward(z, act, terms, f32):
    import torch
    dt = torch.float32 if f32 else torch.bfloat16
    back_case(z, 333, 208, 144, act, dt, dt, terms, False, 11)


@pytest.mark.parametrize("N,d_in,d_out", [(1, 16, 16), (7, 48, 272), (16, 208, 1040), (31, 64, 4112), (60, 336, 2064), (130, 272, 2320), (513, 144, 784), (128, 64, 64), (257, 528, 784), (2100, 272, 96), (1111, 1040, 1296)])
def test_backward_sizes(z, N, d_in, d_out):
    import torch
    back_case(z, N, d_in, d_out, ["gelu", "none"][N & 1], torch.bfloat16, torch.bfloat16, 2, bool(N & 2), N)


@pytest.mark.parametrize("act,f32", [("none", False), ("none", True), ("silu", False)])
def test_backward_rows_further_apart(z, act, f32):
    import torch
    back_case(z, 300, 96, 176, act, torch.float32 if f32 else torch.bfloat16, torch.float32, 2, True, 21, ld_extra=24)


@pytest.mark.parametrize("which", ["dx", "dW", "db"])
def test_backward_one_output_alone(z, which):
    import torch
    g = _gen(31)
    dy, x, W, zz = _bf(g, 200, 64), _bf(g, 200, 48), _bf(g, 64, 48), _bf(g, 200, 64)
    for act in ("none", "gelu"):
        every = dict(zip(("dx", "dW", "db"), z.dust_linear_backward(dy, x, W, act=act, z=zz)))
        want = {n: (True if n == which else None) for n in every}
        got = dict(zip(("dx", "dW", "db"), z.dust_linear_backward(dy, x, W, act=act, z=zz, **want)))
        assert torch.equal(got[which], every[which])
        assert all(got[n] is None for n in got if n != which)


def test_backward_matches_differences(z):
    """The derivative of a weighted sum of y along random directions of x, W and b: central differences in
    64 bits of the formula with step h are off by h^2/6 times the third derivative (below 40 for these sizes
    and the GELU's tanh form) and by the outputs' tolerances."""
    import torch
    g = _gen(41)
    N, i, o = 16, 32, 48
    x, W = _bf(g, N, i), _bf(g, o, i, std=i ** -0.5)
    b = torch.zeros(o, device="cuda")
    dy = torch.randn(N, o, device="cuda", generator=g)
    pre = (x.double() @ W.double().t()).to(torch.bfloat16)
    # the backward pass differentiates at the stored z: the difference is taken there too
    shift = pre.double() - x.double() @ W.double().t()
    dx, dW, db = z.dust_linear_backward(dy, x, W, act="gelu_tanh", z=pre, dx_dtype=torch.float32)
    f = lambda xx, ww, bb: (dy.double() * act64(xx @ ww.t() + bb + shift, "gelu_tanh")[0]).sum()  # noqa: E731
    h = 1e-4
    for got, k in ((dx, 0), (dW, 1), (db, 2)):
        base = [x.double(), W.double(), b.double()]
        v = torch.randn(base[k].shape, device="cuda", generator=g, dtype=torch.float64)
        up, dn = list(base), list(base)
        up[k], dn[k] = base[k] + h * v, base[k] - h * v
        num = (f(*up) - f(*dn)) / (2 * h)
        have = (got.double() * v).sum()
        size = (got.double().abs() * v.abs()).sum()
        assert abs(float(num - have)) <= 2.0 ** -14 * float(size) + 40 * h * h * float(dy.abs().sum()), k


def test_backward_repeats_bit_for_bit(z):
    import torch
    g = _gen(51)
    dy, x, W, zz = _bf(g, 3000, 256), _bf(g, 3000, 128), _bf(g, 256, 128), _bf(g, 3000, 256)
    a = z.dust_linear_backward(dy, x, W, act="silu", z=zz)
    b = z.dust_linear_backward(dy, x, W, act="silu", z=zz)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("N,d", [(40, 256), (700, 512), (5001, 1024)])
@pytest.mark.parametrize("outs", ["dx dW db", "dx db", "dx dW"])
def test_calls_in_a_row_equal_calls_waited_for(z, act, N, d, outs):
    """The kernels of a call overlap one another and those of the next call.  A chain in which dx is the next
    call's dy and its x, dW accumulates and one workspace serves all of it gives the bits of a chain with a
    wait after every call, launched eagerly and replayed from a graph."""
    import torch
    g = _gen(23)
    dy0, x0, pre = _bf(g, N, d), _bf(g, N, d), _bf(g, N, d)
    W = _bf(g, d, d, std=d ** -0.5)
    ws = torch.empty(z.dust_workspace_size(z.DUST_OP_LINEAR_BACKWARD, z.DUST_BF16, N, d, d, 0), dtype=torch.uint8,
                     device="cuda")
    bufs = [torch.empty_like(dy0) for _ in range(6)]
    dW = torch.zeros(d, d, device="cuda") if "dW" in outs else None
    db = [torch.zeros(d, device="cuda") for _ in bufs] if "db" in outs else None

    def chain(wait):
        dy, x = dy0, x0
        if dW is not None:
            dW.zero_()
        for i, out in enumerate(bufs):
            if db is not None:
                db[i].zero_()
            z.dust_linear_backward(dy, x, W, act, z=pre if act != "none" else None, dx=out, dW=dW,
                                   db=db[i] if db is not None else None, accumulate=True, workspace=ws)
            if wait:
                torch.cuda.synchronize()
            x, dy = dy, out

    def held():
        return [t.clone() for t in bufs + (db or []) + ([dW] if dW is not None else [])]

    chain(True)
    want = held()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        chain(False)
    for run in (lambda: chain(False), graph.replay) * 3:
        for t in bufs:
            t.zero_()
        run()
        for a, b in zip(held(), want):
            assert torch.equal(a, b)


def test_other_stream_and_graph(z):
    """On a stream of the caller's, and captured: a replay computes from what the buffers then hold."""
    import torch
    g = _gen(61)
    for N in (3, 400):
        x, W, b = _bf(g, N, 128), _bf(g, 192, 128, std=0.1), torch.randn(192, device="cuda", generator=g)
        want, pre = z.dust_linear(x, W, bias=b, act="gelu", z=True)
        grads = z.dust_linear_backward(want, x, W, act="gelu", z=pre)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        got, pre2 = z.dust_linear(x, W, bias=b, act="gelu", z=True, stream=s)
        grads2 = z.dust_linear_backward(got, x, W, act="gelu", z=pre2, stream=s)
        s.synchronize()
        assert torch.equal(got, want) and all(torch.equal(p, q) for p, q in zip(grads, grads2))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, p = z.dust_linear(x, W, bias=b, act="gelu", z=True)
            out = z.dust_linear_backward(y, x, W, act="gelu", z=p)
        x.copy_(torch.flip(x, dims=[1]))
        graph.replay()
        torch.cuda.synchronize()
        want, pre = z.dust_linear(x, W, bias=b, act="gelu", z=True)
        grads = z.dust_linear_backward(want, x, W, act="gelu", z=pre)
        assert torch.equal(y, want) and all(torch.equal(a, c) for a, c in zip(out, grads))


def test_binding_refuses(z):
    import torch
    g = _gen(71)
    x, W = _bf(g, 4, 32), _bf(g, 16, 32)
    y = torch.empty(4, 16, device="cuda")
    for bad in (lambda: z.dust_linear(x, W, act="tanh"), lambda: z.dust_linear(x, _bf(g, 16, 48)),
                lambda: z.dust_linear(x, W, bias=torch.zeros(15, device="cuda")),
                lambda: z.dust_linear(x, W, residual=y[:3].bfloat16()), lambda: z.dust_linear(x, W, y=y[:2]),
                lambda: z.dust_linear(x.t(), W),
                lambda: z.dust_linear_backward(y, x, W, act="gelu"),
                lambda: z.dust_linear_backward(y, x[:3], W),
                lambda: z.dust_linear_backward(y, x, W, accumulate=True)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: z.dust_linear(x.float(), W), lambda: z.dust_linear(x, W, residual=y),
                lambda: z.dust_linear(x, W, out_dtype=torch.float16), lambda: z.dust_linear_backward(y, x, W, dx_dtype=torch.float16),
                lambda: z.dust_linear(x, W, y=y, out_dtype=torch.bfloat16),
                lambda: z.dust_linear_backward(y.half(), x, W)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(z.DustError):
        z.dust_linear(_bf(g, 4, 24), _bf(g, 16, 24))
    with pytest.raises(z.DustError):
        z.dust_linear_backward(y, x, W, g_terms=3)
