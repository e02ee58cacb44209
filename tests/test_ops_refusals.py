"""The linear layer, the embedding and the grouped optimizer step refuse bad arguments before they
touch the device (CPU only: the addresses are made up and never read)."""
import ctypes

import pytest

import zeroth_order_transformer_b200 as z

P = 0x1000  # any 16-byte aligned (and 256-byte aligned) address
BIG = 1 << 40


def _linear(**kw):
    a = dict(x=P, ld_x=64, W=P, bias=P, act=2, res=P, ld_res=64, dt=z.DUST_BF16, N=4, d_in=64, d_out=64, y=P,
             out_dt=z.DUST_BF16, ld_y=64, zz=P, ld_z=64, s=None)
    a.update(kw)
    return z.lib().dust_linear(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(W=None), 1), (dict(y=None), 1), (dict(N=0), 1), (dict(d_in=0), 1), (dict(d_out=-16), 1),
    (dict(act=5), 1), (dict(act=-1), 1), (dict(dt=7), 1), (dict(out_dt=2), 1),
    (dict(x=P + 8), 1), (dict(W=P + 2), 1), (dict(bias=P + 4), 1), (dict(res=P + 8), 1), (dict(y=P + 8), 1),
    (dict(zz=P + 8), 1),
    (dict(ld_x=56), 1), (dict(ld_x=68), 1), (dict(ld_y=48), 1), (dict(ld_y=68), 1), (dict(ld_res=60), 1),
    (dict(ld_z=68), 1), (dict(ld_x=BIG), 1),
    (dict(dt=z.DUST_F32), 2), (dict(d_in=56), 2), (dict(d_out=56), 2), (dict(N=1 << 30), 2),
])
def test_linear_refuses(kw, code):
    assert _linear(**kw) == code


def _back(**kw):
    a = dict(dy=P, dy_dt=z.DUST_BF16, ld_dy=64, zz=P, ld_z=64, x=P, ld_x=64, W=P, act=2, dt=z.DUST_BF16, N=4, d_in=64,
             d_out=64, terms=2, dx=P, dx_dt=z.DUST_BF16, ld_dx=64, dW=P, db=P, acc=0, ws=P, nb=1 << 30, s=None)
    a.update(kw)
    return z.lib().dust_linear_backward(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), 1), (dict(zz=None), 1), (dict(x=None), 1), (dict(W=None), 1),
    (dict(dx=None, dW=None, db=None), 1), (dict(terms=0), 1), (dict(terms=3), 1), (dict(N=0), 1), (dict(act=9), 1),
    (dict(dy=P + 8), 1), (dict(zz=P + 8), 1), (dict(dW=P + 4), 1), (dict(db=P + 4), 1), (dict(dx=P + 8), 1),
    (dict(ld_dy=60), 1), (dict(ld_z=68), 1), (dict(ld_x=60), 1), (dict(ld_dx=62), 1),
    (dict(dt=z.DUST_F32), 2), (dict(d_in=72), 1), (dict(d_in=40, ld_x=64), 2), (dict(N=1 << 23), 2),
    (dict(ws=None), 5), (dict(nb=100), 5), (dict(ws=P + 16), 5),
])
def test_linear_backward_refuses(kw, code):
    assert _back(**kw) == code


def _emb(**kw):
    a = dict(ids=P, E=P, dt=z.DUST_BF16, ld=64, N=4, V=10, d=60, scale=1.0, out=P, out_dt=z.DUST_F32, ld_out=60, s=None)
    a.update(kw)
    return z.lib().dust_embedding(*a.values())


@pytest.mark.parametrize("kw", [
    dict(ids=None), dict(E=None), dict(out=None), dict(N=0), dict(V=0), dict(d=0), dict(dt=5), dict(out_dt=5),
    dict(ids=P + 2), dict(E=P + 8), dict(out=P + 4), dict(ld=56), dict(ld=60), dict(ld_out=62), dict(ld_out=56),
])
def test_embedding_refuses(kw):
    assert _emb(**kw) == 1


def _egrad(**kw):
    a = dict(ids=P, g=P, dt=z.DUST_F32, ld=60, N=4, V=10, d=60, scale=1.0, G=P, ld_G=60, acc=0, ws=P, nb=1 << 30, s=None)
    a.update(kw)
    return z.lib().dust_embedding_grad(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), 1), (dict(g=None), 1), (dict(G=None), 1), (dict(N=0), 1), (dict(V=-1), 1), (dict(d=0), 1),
    (dict(g=P + 8), 1), (dict(G=P + 8), 1), (dict(ld=56), 1), (dict(ld=62), 1), (dict(ld_G=61), 1), (dict(dt=3), 1),
    (dict(dt=z.DUST_BF16, ld=60), 1), (dict(V=2147483647), 2), (dict(N=(1 << 26) + 1), 2), (dict(N=1 << 40), 2), (dict(N=5000, ws=None), 5),
    (dict(N=5000, nb=64), 5),
])
def test_embedding_grad_refuses(kw, code):
    assert _egrad(**kw) == code


def _opt(opt=None, n=1, g_dt=z.DUST_F32, state=z.DUST_STATE_F32, g_scale=None, step=None, **kw):
    a = dict(G=P, W=P, W_bf16=P, m=P, v=P, m_scale=P, v_scale=P, n=100, lr_scale=1.0, decay_scale=1.0)
    a.update(kw)
    d = (z.dust_opt_tensor * 1)(z.dust_opt_tensor(*a.values()))
    o = opt if opt is not None else z.adam(1e-3, 1)
    return z.lib().dust_optimizer_step_grouped(ctypes.byref(o), d, n, g_dt, state, g_scale, step, None)


@pytest.mark.parametrize("kw,code", [
    (dict(opt=z.adam(1e-3, 0)), 1), (dict(opt=z.adam(float("nan"), 1)), 1), (dict(opt=z.sgd_momentum(0.1, 1.0)), 1),
    (dict(opt=z.adam(1e-3, 1, weight_decay=float("inf"))), 1),
    (dict(n=-1), 1), (dict(g_dt=4), 1), (dict(state=2), 1), (dict(g_scale=P + 2), 1), (dict(step=P + 1), 1),
    (dict(G=None), 1), (dict(W=None), 1), (dict(m=None), 1), (dict(v=None), 1),
    (dict(state=1, m_scale=None), 1), (dict(state=1, v_scale=None), 1), (dict(state=1, v_scale=P + 2), 1),
    (dict(G=P + 4), 1), (dict(W=P + 8), 1), (dict(W_bf16=P + 8), 1), (dict(m=P + 4), 1), (dict(v=P + 8), 1),
    (dict(lr_scale=-1.0), 1), (dict(decay_scale=float("nan")), 1), (dict(lr_scale=float("inf")), 1),
    (dict(opt=z.sgd_momentum(0.1, 0.9), state=1), 2),
])
def test_grouped_optimizer_refuses(kw, code):
    # the numbered n of a tensor is set through the descriptor, the count of tensors through n
    assert _opt(**kw) == code


def test_grouped_optimizer_without_work_is_ok():
    o = z.adam(1e-3, 1)
    assert z.lib().dust_optimizer_step_grouped(ctypes.byref(o), None, 0, 0, 0, None, None, None) == 0
    d = (z.dust_opt_tensor * 2)()
    assert z.lib().dust_optimizer_step_grouped(ctypes.byref(o), d, 2, 0, 0, None, None, None) == 0
    d[1].n = -1
    assert z.lib().dust_optimizer_step_grouped(ctypes.byref(o), d, 2, 0, 0, None, None, None) == 1


def test_workspace_sizes():
    lb = lambda N, i, o: z.dust_workspace_size(z.DUST_OP_LINEAR_BACKWARD, z.DUST_BF16, N, i, o, 0)  # noqa: E731
    assert lb(1000, 64, 128) >= 2 * 1000 * 128 * 2
    assert lb(2000, 64, 128) > lb(1000, 64, 128)
    assert lb(10, 0, 128) == 0
    eg = lambda N, V, d: z.dust_workspace_size(z.DUST_OP_EMBEDDING_GRAD, z.DUST_F32, N, V, d, 0)  # noqa: E731
    assert eg(4096, 1, 1) == 0 and eg(4097, 1, 1) > 0  # up to 4096 tokens are sorted in shared memory
    assert eg(100000, 50, 64) >= 4 * 4 * 100000
    assert eg(10, 10, 0) == 0


def test_outputs_that_are_inputs_are_refused():
    """Each buffer at an address of its own but for one pair."""
    q = [P * (i + 1) for i in range(10)]
    at = dict(x=q[0], W=q[1], bias=q[2], res=q[3], y=q[4], zz=q[5])
    for out, others in (("y", ("x", "W", "bias")), ("zz", ("x", "W", "bias", "res", "y"))):
        for o in others:
            assert _linear(**{**at, out: at[o]}) == 1, (out, o)
    assert _linear(**{**at, "y": at["res"], "ld_y": 72}) == 1
    at = dict(dy=q[0], zz=q[1], x=q[2], W=q[3], dx=q[4], dW=q[5], db=q[6])
    for out in ("dx", "dW", "db"):
        for o in at:
            if o != out:
                assert _back(**{**at, out: at[o]}) == 1, (out, o)
    assert _emb(ids=q[0], E=q[1], out=q[1]) == 1 and _emb(ids=q[0], E=q[1], out=q[0]) == 1
    assert _egrad(ids=q[0], g=q[1], G=q[1]) == 1 and _egrad(ids=q[0], g=q[1], G=q[0]) == 1


def test_binding_refuses_cpu_tensors():
    import torch
    x, W = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(16, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        z.dust_linear(x, W)
    with pytest.raises(ValueError):
        z.dust_linear_backward(x, x, W)
    with pytest.raises(ValueError):
        z.dust_embedding(torch.zeros(3, dtype=torch.int32), W)
    with pytest.raises(TypeError):
        z.dust_embedding(torch.zeros(3, dtype=torch.int64), W)
    with pytest.raises(ValueError):
        z.dust_embedding_grad(torch.zeros(3, dtype=torch.int32), x, 8)
    with pytest.raises(ValueError):
        z.DustOptimizer([torch.zeros(8)], [torch.zeros(8)])
    with pytest.raises(ValueError):
        z.DustOptimizer([], [])
