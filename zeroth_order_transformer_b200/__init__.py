"""Python binding of libdust, the B200 implementation of the Dust token-level
node-perturbation gradient estimator for one linear layer.

The binding only marshals arguments: it checks tensors, takes their device pointers and the
current CUDA stream, allocates outputs and workspaces with PyTorch, and calls the C ABI
declared in ``include/dust.h``.  Every step of the estimator runs in the CUDA kernels of
``libdust.so``; there is no other code path.  If the library is missing, every call raises.

Function names follow the C ABI:
  dust_noisy_linear_fwd  per-draw loss change of the noisy layer (noise equation)
  dust_credit            centred loss and discounted credit (centred-loss, credit equations)
  dust_weight_grad       output-error estimate g and weight estimate G_W
and around the estimator, for the rest of a training step:
  dust_linear, dust_linear_backward      the clean layer with its epilogue, and its exact gradients
  dust_embedding, dust_embedding_grad    the token embedding and the gradient of its table
  DustOptimizer (dust_optimizer_step_grouped)   one step over all tensors, moments in 32 or 8 bits
"""
from __future__ import annotations

import bisect
import ctypes
import os
from typing import NamedTuple, Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdust.so")

DUST_OK = 0
DUST_ERR_INVALID_ARG = 1
DUST_ERR_UNSUPPORTED = 2
DUST_ERR_CUDA = 3
DUST_ERR_TIMEOUT = 4
DUST_ERR_WORKSPACE = 5

DUST_F32 = 0
DUST_BF16 = 1

DUST_OP_NOISY_LINEAR_FWD = 0
DUST_OP_CREDIT = 1
DUST_OP_WEIGHT_GRAD = 2
DUST_OP_LOGITS_CE = 3
DUST_OP_SPSA_PROBE = 4
DUST_OP_LINEAR_BACKWARD = 5
DUST_OP_EMBEDDING_GRAD = 6

DUST_ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

DUST_STATE_F32 = 0
DUST_STATE_E4M3 = 1
DUST_STATE_BLOCK = 256
DUST_EMBEDDING_SMALL = 4096

EXPORTED_SYMBOLS = (
    "dust_noisy_linear_fwd", "dust_credit", "dust_weight_grad", "dust_workspace_size",
    "dust_status_string", "dust_last_device_error", "dust_debug_philox",
    "dust_debug_credit_skip_publish", "dust_profile_enable", "dust_profile_disable",
    "dust_profile_read", "dust_credit_no_alloc", "dust_noisy_linear_fwd_grouped",
    "dust_credit_grouped", "dust_weight_grad_grouped", "dust_workspace_size_grouped",
    "dust_optimizer_step", "dust_weight_grad_step", "dust_noisy_logits_ce",
    "dust_debug_normal_sum", "dust_debug_fwd_plan", "dust_attn_reward", "dust_discounted_credit",
    "dust_spsa_probe", "dust_spsa_estimate", "dust_noisy_linear_output", "dust_debug_word_sum",
    "dust_linear", "dust_linear_backward", "dust_embedding", "dust_embedding_grad",
    "dust_optimizer_step_grouped",
)

DUST_OPT_SGD_MOMENTUM = 1
DUST_OPT_ADAM = 2


class DustError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


class dust_noise_key(ctypes.Structure):
    _fields_ = [("seed", ctypes.c_uint64), ("layer_id", ctypes.c_uint32),
                ("draw_offset", ctypes.c_uint32), ("token_offset", ctypes.c_uint32),
                ("channel_offset", ctypes.c_uint32)]


class dust_layer_desc(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("W", ctypes.c_void_p), ("u", ctypes.c_void_p),
                ("d_in", ctypes.c_int32), ("d_out", ctypes.c_int32), ("layer_id", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("dloss", ctypes.c_void_p),
                ("ld_dloss", ctypes.c_int64), ("r", ctypes.c_void_p), ("ld_r", ctypes.c_int64),
                ("G_W", ctypes.c_void_p), ("g_out", ctypes.c_void_p)]


class dust_opt_params(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("step", ctypes.c_int32), ("lr", ctypes.c_float),
                ("momentum", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class dust_opt_tensor(ctypes.Structure):
    _fields_ = [("G", ctypes.c_void_p), ("W", ctypes.c_void_p), ("W_bf16", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("lr_scale", ctypes.c_float),
                ("decay_scale", ctypes.c_float)]


def sgd_momentum(lr: float, momentum: float, weight_decay: float = 0.0) -> dust_opt_params:
    return dust_opt_params(DUST_OPT_SGD_MOMENTUM, 0, lr, momentum, 0.0, 0.0, 0.0, weight_decay)


def adam(lr: float, step: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
         weight_decay: float = 0.0) -> dust_opt_params:
    return dust_opt_params(DUST_OPT_ADAM, step, lr, 0.0, beta1, beta2, eps, weight_decay)


class NoiseKey(NamedTuple):
    seed: int
    layer_id: int = 0
    draw_offset: int = 0
    token_offset: int = 0
    channel_offset: int = 0

    def c(self) -> dust_noise_key:
        return dust_noise_key(self.seed & 0xFFFFFFFFFFFFFFFF, self.layer_id, self.draw_offset,
                              self.token_offset, self.channel_offset)


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libdust.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libdust.so is not built ({LIB_PATH}); run "
                               "`python -m zeroth_order_transformer_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                 ctypes.c_float, ctypes.c_size_t)
        L.dust_noisy_linear_fwd.argtypes = [vp, vp, vp, ctypes.c_int, i64, i32, i32, i32, f32,
                                            dust_noise_key, vp, i64, vp, sz, vp]
        L.dust_credit.argtypes = [vp, i64, i32, i64, vp, i32, f32, vp, i64, vp, sz, vp]
        L.dust_weight_grad.argtypes = [vp, i64, vp, ctypes.c_int, i64, i32, i32, i32, i32, f32,
                                       dust_noise_key, vp, ctypes.c_int, vp, i32, vp, sz, vp]
        L.dust_credit_no_alloc.argtypes = [vp, i64, i32, i64, vp, i32, f32, vp, i64, vp]
        L.dust_credit_no_alloc.restype = ctypes.c_int
        dp = ctypes.POINTER(dust_layer_desc)
        L.dust_noisy_linear_fwd_grouped.argtypes = [dp, i32, i64, i32, f32, dust_noise_key, vp,
                                                    sz, vp]
        L.dust_credit_grouped.argtypes = [dp, i32, i32, i64, vp, i32, f32, vp, sz, vp]
        L.dust_weight_grad_grouped.argtypes = [dp, i32, i64, i32, i32, f32, dust_noise_key,
                                               ctypes.c_int, i32, vp, sz, vp]
        L.dust_workspace_size_grouped.argtypes = [ctypes.c_int, dp, i32, i64, i32]
        L.dust_workspace_size_grouped.restype = sz
        for name in ("dust_noisy_linear_fwd_grouped", "dust_credit_grouped",
                     "dust_weight_grad_grouped"):
            getattr(L, name).restype = ctypes.c_int
        op = ctypes.POINTER(dust_opt_params)
        L.dust_optimizer_step.argtypes = [op, vp, vp, vp, vp, vp, i64, vp]
        L.dust_optimizer_step.restype = ctypes.c_int
        L.dust_weight_grad_step.argtypes = [vp, i64, vp, ctypes.c_int, i64, i32, i32, i32, i32,
                                            f32, dust_noise_key, vp, ctypes.c_int, vp, i32, op, vp,
                                            vp, vp, vp, vp, sz, vp]
        L.dust_weight_grad_step.restype = ctypes.c_int
        L.dust_noisy_logits_ce.argtypes = [vp, i64, ctypes.c_int, vp, i64, i32, i32, i32, i32,
                                           f32, dust_noise_key, vp, i64, vp, sz, vp]
        L.dust_noisy_logits_ce.restype = ctypes.c_int
        L.dust_workspace_size.argtypes = [ctypes.c_int, ctypes.c_int, i64, i32, i32, i32]
        L.dust_workspace_size.restype = sz
        L.dust_status_string.argtypes = [ctypes.c_int]
        L.dust_status_string.restype = ctypes.c_char_p
        L.dust_last_device_error.argtypes = [vp, ctypes.POINTER(i32)]
        L.dust_debug_philox.argtypes = [vp, i64, ctypes.c_uint64, vp, vp, vp]
        L.dust_attn_reward.argtypes = [vp, i64, vp, i64, ctypes.c_int, i64, i32, i32, vp, i64,
                                       vp]
        L.dust_attn_reward.restype = ctypes.c_int
        L.dust_discounted_credit.argtypes = [vp, i64, i32, i64, vp, i32, f32, vp, i64, vp, sz,
                                             vp]
        L.dust_discounted_credit.restype = ctypes.c_int
        L.dust_noisy_linear_output.argtypes = [vp, vp, ctypes.c_int, i64, i32, i32, i32, f32,
                                               dust_noise_key, vp, ctypes.c_int, i64, vp]
        L.dust_noisy_linear_output.restype = ctypes.c_int
        L.dust_spsa_probe.argtypes = [vp, vp, vp, ctypes.c_int, i64, i32, i32, i32, f32,
                                      dust_noise_key, vp, vp, vp, vp, sz, vp]
        L.dust_spsa_probe.restype = ctypes.c_int
        L.dust_spsa_estimate.argtypes = [vp, i32, i32, i32, i32, dust_noise_key, vp, ctypes.c_int,
                                         vp]
        L.dust_spsa_estimate.restype = ctypes.c_int
        L.dust_debug_normal_sum.argtypes = [dust_noise_key, i64, i32, vp, vp]
        L.dust_debug_normal_sum.restype = ctypes.c_int
        L.dust_debug_word_sum.argtypes = [dust_noise_key, i64, i32, vp, vp]
        L.dust_debug_word_sum.restype = ctypes.c_int
        L.dust_linear.argtypes = [vp, i64, vp, vp, ctypes.c_int, vp, i64, ctypes.c_int, i64, i32, i32, vp,
                                  ctypes.c_int, i64, vp, i64, vp]
        L.dust_linear_backward.argtypes = [vp, ctypes.c_int, i64, vp, i64, vp, i64, vp, ctypes.c_int,
                                           ctypes.c_int, i64, i32, i32, i32, vp, ctypes.c_int, i64, vp, vp,
                                           ctypes.c_int, vp, sz, vp]
        L.dust_embedding.argtypes = [vp, vp, ctypes.c_int, i64, i64, i32, i32, f32, vp, ctypes.c_int, i64, vp]
        L.dust_embedding_grad.argtypes = [vp, vp, ctypes.c_int, i64, i64, i32, i32, f32, vp, i64,
                                          ctypes.c_int, vp, sz, vp]
        L.dust_optimizer_step_grouped.argtypes = [op, ctypes.POINTER(dust_opt_tensor), i32, ctypes.c_int,
                                                  ctypes.c_int, vp, vp, vp]
        for name in ("dust_linear", "dust_linear_backward", "dust_embedding", "dust_embedding_grad",
                     "dust_optimizer_step_grouped"):
            getattr(L, name).restype = ctypes.c_int
        L.dust_debug_credit_skip_publish.argtypes = [i32]
        L.dust_debug_credit_skip_publish.restype = None
        L.dust_debug_fwd_plan.argtypes = [i64, i32, i32, vp, i32, ctypes.POINTER(i32),
                                          ctypes.POINTER(i32)]
        L.dust_debug_fwd_plan.restype = ctypes.c_int
        L.dust_profile_enable.argtypes = [i32]
        L.dust_profile_enable.restype = ctypes.c_int
        L.dust_profile_disable.argtypes = []
        L.dust_profile_disable.restype = None
        L.dust_profile_read.argtypes = [ctypes.POINTER(ctypes.c_char_p),
                                        ctypes.POINTER(ctypes.c_float), i32]
        L.dust_profile_read.restype = i32
        for name in ("dust_noisy_linear_fwd", "dust_credit", "dust_weight_grad",
                     "dust_last_device_error", "dust_debug_philox"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().dust_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != DUST_OK:
        raise DustError(status, where)


def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return DUST_BF16
    if t.dtype == torch.float32:
        return DUST_F32
    raise TypeError(f"unsupported dtype {t.dtype}; layers are bf16 or fp32")


def _cuda(t, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _cuda_rows(t, name: str):
    """A CUDA matrix whose rows are contiguous; rows may be further apart (the row stride is
    passed as the leading dimension)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    return t


def _stream(device, stream) -> int:
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream)


def _workspace(ws, nbytes: int, device):
    torch = _torch()
    if nbytes == 0:
        return None, 0
    if ws is None or ws.numel() * ws.element_size() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def dust_workspace_size(op: int, dtype: int, N: int, d_in: int, d_out: int, K: int) -> int:
    return int(lib().dust_workspace_size(op, dtype, N, d_in, d_out, K))


def dust_noisy_linear_fwd(x, W, u, K: int, sigma: float, key: NoiseKey, dloss=None,
                          workspace=None, stream=None):
    """Per-draw loss change dloss[K, N] (fp32) of the layer W x_t + sigma a_t against u_t."""
    torch = _torch()
    _cuda(x, "x"), _cuda(W, "W"), _cuda(u, "u")
    N, d_in = x.shape
    d_out = W.shape[0]
    if W.shape != (d_out, d_in) or u.shape != (N, d_out) or not (x.dtype == W.dtype == u.dtype):
        raise ValueError("shapes/dtypes: x [N, d_in], W [d_out, d_in], u [N, d_out], one dtype")
    dt = _dtype_code(x)
    if dloss is None:
        dloss = torch.empty((K, N), dtype=torch.float32, device=x.device)
    _cuda_rows(dloss, "dloss")
    ws, nb = _workspace(workspace, dust_workspace_size(DUST_OP_NOISY_LINEAR_FWD, dt, N, d_in,
                                                       d_out, K), x.device)
    st = lib().dust_noisy_linear_fwd(x.data_ptr(), W.data_ptr(), u.data_ptr(), dt, N, d_in,
                                     d_out, K, float(sigma), key.c(), dloss.data_ptr(),
                                     dloss.stride(0), ws.data_ptr() if ws is not None else None,
                                     nb, _stream(x.device, stream))
    _check(st, "dust_noisy_linear_fwd")
    return dloss


def dust_noisy_logits_ce(z, y, v0: int, S: int, K: int, sigma: float, key: NoiseKey,
                         dloss=None, workspace=None, stream=None):
    """Per-draw change of the full-vocabulary cross-entropy dloss[K, N] when noise is added to
    the cached logits of the slab [v0, v0 + S) (LM-head perturbation)."""
    torch = _torch()
    _cuda(z, "z"), _cuda(y, "y")
    if y.dtype != torch.int32:
        raise TypeError("y must be int32")
    N, V = z.shape
    dt = _dtype_code(z)
    if dloss is None:
        dloss = torch.empty((K, N), dtype=torch.float32, device=z.device)
    ws, nb = _workspace(workspace, dust_workspace_size(DUST_OP_LOGITS_CE, dt, N, V, S, K),
                        z.device)
    st = lib().dust_noisy_logits_ce(z.data_ptr(), z.stride(0), dt, y.data_ptr(), N, V, v0, S, K,
                                    float(sigma), key.c(), dloss.data_ptr(), dloss.stride(0),
                                    ws.data_ptr() if ws is not None else None, nb,
                                    _stream(z.device, stream))
    _check(st, "dust_noisy_logits_ce")
    return dloss


def dust_credit(loss, cu_seqlens, gamma: float, r=None, workspace=None, stream=None):
    """Credit r[K, N] from losses [K, N] and int32 cu_seqlens [n_seq + 1] (device)."""
    torch = _torch()
    _cuda_rows(loss, "loss"), _cuda(cu_seqlens, "cu_seqlens")
    if loss.dtype != torch.float32 or cu_seqlens.dtype != torch.int32:
        raise TypeError("loss must be float32 and cu_seqlens int32")
    K, N = loss.shape
    if r is None:
        r = torch.empty((K, N), dtype=torch.float32, device=loss.device)
    _cuda_rows(r, "r")
    ws, nb = _workspace(workspace, dust_workspace_size(DUST_OP_CREDIT, DUST_F32, N, 0, 0, K),
                        loss.device)
    st = lib().dust_credit(loss.data_ptr(), loss.stride(0), K, N, cu_seqlens.data_ptr(),
                           cu_seqlens.numel() - 1, float(gamma), r.data_ptr(), r.stride(0),
                           ws.data_ptr() if ws is not None else None, nb,
                           _stream(loss.device, stream))
    _check(st, "dust_credit")
    return r


def dust_attn_reward(ghat, delta_o, c=None, stream=None):
    """Attention-internal reward c[K, N] = -<ghat_t, delta_o[i, t]> from the fp32 output-error
    estimate ghat [N, d] at the attention output and delta_o [K, N, d] (bf16 or fp32)."""
    torch = _torch()
    _cuda(ghat, "ghat")
    if not delta_o.is_cuda:
        raise ValueError("delta_o must be a CUDA tensor")
    if ghat.dtype != torch.float32:
        raise TypeError("ghat must be float32")
    K, N, d = delta_o.shape
    if tuple(ghat.shape) != (N, d) or delta_o.stride(2) != 1 or delta_o.stride(0) != N * delta_o.stride(1):
        raise ValueError("ghat must be [N, d] and delta_o [K, N, d] with rows N * ld apart")
    if c is None:
        c = torch.empty((K, N), dtype=torch.float32, device=ghat.device)
    st = lib().dust_attn_reward(ghat.data_ptr(), ghat.stride(0), delta_o.data_ptr(),
                                delta_o.stride(1), _dtype_code(delta_o), N, d, K, c.data_ptr(),
                                c.stride(0), _stream(ghat.device, stream))
    _check(st, "dust_attn_reward")
    return c


def dust_discounted_credit(c, cu_seqlens, gamma: float, r=None, workspace=None, stream=None):
    """The credit equation on a given reward c [K, N] (no centring): r[K, N]."""
    torch = _torch()
    _cuda(c, "c"), _cuda(cu_seqlens, "cu_seqlens")
    if c.dtype != torch.float32 or cu_seqlens.dtype != torch.int32:
        raise TypeError("c must be float32 and cu_seqlens int32")
    K, N = c.shape
    if r is None:
        r = torch.empty((K, N), dtype=torch.float32, device=c.device)
    _cuda(r, "r")
    ws, nb = _workspace(workspace, dust_workspace_size(DUST_OP_CREDIT, DUST_F32, N, 0, 0, K),
                        c.device)
    st = lib().dust_discounted_credit(c.data_ptr(), c.stride(0), K, N, cu_seqlens.data_ptr(),
                                      cu_seqlens.numel() - 1, float(gamma), r.data_ptr(),
                                      r.stride(0), ws.data_ptr() if ws is not None else None,
                                      nb, _stream(c.device, stream))
    _check(st, "dust_discounted_credit")
    return r


def dust_noisy_linear_output(x, W, K: int, sigma: float, key: NoiseKey, y_out=None,
                             out_dtype=None, stream=None):
    """The perturbed outputs y_out[K, N, d_out] = W x_t + sigma a_t^(i) (fp32 by default, or
    out_dtype=torch.bfloat16), with the noise of dust_noisy_linear_fwd for the same key."""
    torch = _torch()
    _cuda(x, "x"), _cuda(W, "W")
    N, d_in = x.shape
    d_out = W.shape[0]
    if y_out is None:
        y_out = torch.empty((K, N, d_out), dtype=out_dtype or torch.float32, device=x.device)
    _cuda(y_out, "y_out")
    st = lib().dust_noisy_linear_output(x.data_ptr(), W.data_ptr(), _dtype_code(x), N, d_in,
                                        d_out, K, float(sigma), key.c(), y_out.data_ptr(),
                                        _dtype_code(y_out), y_out.stride(1),
                                        _stream(x.device, stream))
    _check(st, "dust_noisy_linear_output")
    return y_out


def dust_spsa_probe(x, W, u, P: int, eps: float, key: NoiseKey, p=None, losses: bool = False,
                    workspace=None, stream=None):
    """SPSA / MeZO probe: p[P] = (L_+ - L_-) / (2 eps) for the weight directions z_j of
    draws key.draw_offset .. + P; with losses=True also returns L_+ and L_- [P]."""
    torch = _torch()
    _cuda(x, "x"), _cuda(W, "W"), _cuda(u, "u")
    N, d_in = x.shape
    d_out = W.shape[0]
    dt = _dtype_code(x)
    if p is None:
        p = torch.empty(P, dtype=torch.float32, device=x.device)
    Lp = torch.empty(P, dtype=torch.float32, device=x.device) if losses else None
    Lm = torch.empty(P, dtype=torch.float32, device=x.device) if losses else None
    ws, nb = _workspace(workspace, dust_workspace_size(DUST_OP_SPSA_PROBE, dt, N, d_in, d_out, P),
                        x.device)
    st = lib().dust_spsa_probe(x.data_ptr(), W.data_ptr(), u.data_ptr(), dt, N, d_in, d_out, P,
                               float(eps), key.c(), p.data_ptr(), _ptr(Lp), _ptr(Lm),
                               ws.data_ptr() if ws is not None else None, nb,
                               _stream(x.device, stream))
    _check(st, "dust_spsa_probe")
    return (p, Lp, Lm) if losses else p


def dust_spsa_estimate(p, P_total: int, d_out: int, d_in: int, key: NoiseKey, G=None,
                       accumulate: bool = False, stream=None):
    """G [d_out, d_in] (+)= (1/P_total) sum_j p[j] z_j."""
    torch = _torch()
    _cuda(p, "p")
    if G is None:
        G = torch.empty((d_out, d_in), dtype=torch.float32, device=p.device)
        accumulate = False
    _cuda(G, "G")
    st = lib().dust_spsa_estimate(p.data_ptr(), p.numel(), P_total, d_in, d_out, key.c(),
                                  G.data_ptr(), 1 if accumulate else 0, _stream(p.device, stream))
    _check(st, "dust_spsa_estimate")
    return G


def dust_credit_no_alloc(loss, cu_seqlens, gamma: float, r, stream=None):
    """dust_credit with the library's static 4 MiB scratch instead of a workspace, for callers
    that cannot allocate device memory; ``r`` must be given (float32 [K, N], rows contiguous,
    rows may be further apart, as may those of ``loss``).  Calls that overlap on the GPU share
    the scratch and race: serialize them."""
    torch = _torch()
    _cuda_rows(loss, "loss"), _cuda(cu_seqlens, "cu_seqlens"), _cuda_rows(r, "r")
    if loss.dtype != torch.float32 or r.dtype != torch.float32 or cu_seqlens.dtype != torch.int32:
        raise TypeError("loss and r must be float32 and cu_seqlens int32")
    K, N = loss.shape
    if tuple(r.shape) != (K, N):
        raise ValueError(f"r must be [K, N] = [{K}, {N}] like loss, got {tuple(r.shape)}")
    st = lib().dust_credit_no_alloc(loss.data_ptr(), loss.stride(0), K, N, cu_seqlens.data_ptr(),
                                    cu_seqlens.numel() - 1, float(gamma), r.data_ptr(),
                                    r.stride(0), _stream(loss.device, stream))
    _check(st, "dust_credit_no_alloc")
    return r


G_TERMS = 2  # default: g enters the bf16 contraction as hi + lo terms


def dust_weight_grad(r, x, d_out: int, K_total: int, sigma: float, key: NoiseKey, G_W=None,
                     accumulate: bool = False, g_out=None, workspace=None, stream=None,
                     g_terms: int = G_TERMS) -> Tuple[object, Optional[object]]:
    """G_W[d_out, d_in] (fp32) and, if g_out is a tensor or True, g[N, d_out] (fp32).  For bf16
    x, g enters the tensor cores as ``g_terms`` bf16 terms (2: hi + lo; 1: rounded once)."""
    torch = _torch()
    _cuda_rows(r, "r"), _cuda(x, "x")
    K_chunk, N = r.shape
    d_in = x.shape[1]
    dt = _dtype_code(x)
    if G_W is None:
        G_W = torch.empty((d_out, d_in), dtype=torch.float32, device=x.device)
        accumulate = False
    _cuda(G_W, "G_W")
    if g_out is True:
        g_out = torch.empty((N, d_out), dtype=torch.float32, device=x.device)
    if g_out is False:
        g_out = None
    need = dust_workspace_size(DUST_OP_WEIGHT_GRAD, dt, N, d_in, d_out, K_chunk)
    if dt == DUST_F32 and g_out is not None:
        need = 0
    ws, nb = _workspace(workspace, need, x.device)
    st = lib().dust_weight_grad(r.data_ptr(), r.stride(0), x.data_ptr(), dt, N, d_in, d_out,
                                K_chunk, K_total, float(sigma), key.c(), G_W.data_ptr(),
                                1 if accumulate else 0,
                                g_out.data_ptr() if g_out is not None else None, int(g_terms),
                                ws.data_ptr() if ws is not None else None, nb,
                                _stream(x.device, stream))
    _check(st, "dust_weight_grad")
    return G_W, g_out


def _ptr(t):
    return t.data_ptr() if t is not None else None


def dust_optimizer_step(opt: dust_opt_params, G, W, m, v=None, W_bf16=None, stream=None):
    """One optimizer step in place on fp32 W, m (and v for Adam) from the estimate G."""
    for t, nm in ((G, "G"), (W, "W"), (m, "m")):
        _cuda(t, nm)
    st = lib().dust_optimizer_step(ctypes.byref(opt), G.data_ptr(), W.data_ptr(), _ptr(W_bf16),
                                   m.data_ptr(), _ptr(v), W.numel(), _stream(W.device, stream))
    _check(st, "dust_optimizer_step")
    return W


def dust_weight_grad_step(r, x, d_out: int, K_total: int, sigma: float, key: NoiseKey,
                          opt: dust_opt_params, W, m, v=None, W_bf16=None, G_W=None,
                          accumulate: bool = False, g_out=None, workspace=None, stream=None,
                          g_terms: int = G_TERMS):
    """dust_weight_grad with the optimizer step fused into the pass that finishes G_W."""
    _cuda(r, "r"), _cuda(x, "x"), _cuda(W, "W"), _cuda(m, "m")
    K_chunk, N = r.shape
    d_in = x.shape[1]
    dt = _dtype_code(x)
    ws, nb = _workspace(workspace, dust_workspace_size(DUST_OP_WEIGHT_GRAD, dt, N, d_in, d_out,
                                                       K_chunk), x.device)
    st = lib().dust_weight_grad_step(r.data_ptr(), r.stride(0), x.data_ptr(), dt, N, d_in, d_out,
                                     K_chunk, K_total, float(sigma), key.c(), _ptr(G_W),
                                     1 if accumulate else 0, _ptr(g_out), int(g_terms),
                                     ctypes.byref(opt),
                                     W.data_ptr(), _ptr(W_bf16), m.data_ptr(), _ptr(v),
                                     ws.data_ptr() if ws is not None else None, nb,
                                     _stream(x.device, stream))
    _check(st, "dust_weight_grad_step")
    return W


# ------------------------------------------------------------------ around the estimator

# Host time counts in these calls (a lookup of a few tokens is 2 us on the device), so they take the
# stream handle and the current device without the objects around them (3 us for a Stream) and check
# each tensor once.
_DT = {}  # torch dtype -> C code, filled at the first use


def _dtypes() -> dict:
    if not _DT:
        torch = _torch()
        _DT.update({torch.bfloat16: DUST_BF16, torch.float32: DUST_F32})  # both at once: another thread may look now
    return _DT


_HOST: list = []


def _host():
    """(current device, raw handle of a device's current stream), as functions, looked up once: the smallest calls take
    as long as the host's part of them."""
    if not _HOST:
        C = _torch()._C
        _HOST[:] = C._cuda_getDevice, C._cuda_getCurrentRawStream
    return _HOST


def _raw_stream(index: int) -> int:
    return _host()[1](index)


def _scope(index: int, stream):
    """What a call has to run under: its tensors' device, and its stream, so that outputs and workspaces
    that the call allocates belong to the stream that uses them.  None if it is current already."""
    if index < 0:
        raise ValueError("the tensors must be CUDA tensors")
    if stream is None:
        return None if index == _host()[0]() else _torch().cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{index}")
    return _torch().cuda.stream(stream)


def _rows(t, name: str, rows: int, cols: int, index: int, only=None) -> int:
    """Checks a CUDA matrix [rows, cols] of bf16 or fp32 (or of the type `only`) with contiguous rows and
    returns its row stride."""
    dtype = t.dtype
    if dtype is not only and (only is not None or dtype not in _dtypes()):
        raise TypeError(f"{name} must be {only or 'bf16 or fp32'}, not {dtype}")
    strides = t.stride()
    if t.get_device() != index or t.shape != (rows, cols) or (strides[1] != 1 and cols > 1):
        raise ValueError(f"{name} must be a [{rows}, {cols}] matrix with contiguous rows on cuda:{index}, got "
                         f"{tuple(t.shape)}, strides {strides}, on {t.device}")
    return strides[0] if rows > 1 else -(-cols // 8) * 8


def _flat(t, name: str, n: int, index: int, dtype):
    if t.get_device() != index or index < 0 or t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of {n} elements on cuda:{index}")
    return t


def _new_rows(like, rows: int, cols: int, dtype, vec: int):
    """A new [rows, cols] matrix whose rows begin at multiples of `vec` elements, and its row stride."""
    if cols % vec == 0:
        return like.new_empty(rows, cols, dtype=dtype), cols
    ld = -(-cols // vec) * vec
    return like.new_empty((rows, ld), dtype=dtype)[:, :cols], ld


def _new_workspace(workspace, nbytes: int, like):
    """(address, bytes, what keeps it alive) of a given workspace that suffices, or of a new one."""
    torch = _torch()
    if nbytes == 0:
        return None, 0, None
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        workspace = like.new_empty(nbytes, dtype=torch.uint8)
    elif workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _act_code(act: str) -> int:
    code = DUST_ACTS.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}; one of {sorted(DUST_ACTS)}")
    return code


def dust_linear(x, W, bias=None, act: str = "none", residual=None, y=None, z=None, out_dtype=None, stream=None):
    """y[N, d_out] = act(x W^T + bias) + residual for bf16 x [N, d_in] and W [d_out, d_in]; bias fp32
    [d_out]; y (and residual) bf16 by default, or out_dtype=torch.float32.  z=True (or a bf16
    tensor) also keeps the pre-activation for dust_linear_backward and returns (y, z).  Rows of
    x, residual, y and z may be further apart than their length."""
    torch = _torch()
    bf, f32 = torch.bfloat16, torch.float32
    dev = x.get_device()
    scope = _scope(dev, stream)
    if scope is not None:
        with scope:
            return dust_linear(x, W, bias, act, residual, y, z, out_dtype)
    if x.dim() != 2 or W.dim() != 2:
        raise ValueError("x must be [N, d_in] and W [d_out, d_in]")
    N, d_in = x.shape
    d_out, k = W.shape
    if k != d_in:
        raise ValueError("x must be [N, d_in] and W [d_out, d_in]")
    ld_x = _rows(x, "x", N, d_in, dev, bf)
    _flat(W, "W", d_out * d_in, dev, bf)
    if bias is not None:
        _flat(bias, "bias", d_out, dev, f32)
    if y is None:
        y = x.new_empty(N, d_out, dtype=out_dtype)  # x's, bf16, by default
        ld_y = d_out
        if y.dtype not in _dtypes():
            raise TypeError(f"out_dtype must be bf16 or fp32, not {out_dtype}")
    else:
        if out_dtype is not None and y.dtype != out_dtype:
            raise TypeError(f"y is {y.dtype}, out_dtype {out_dtype}")
        ld_y = _rows(y, "y", N, d_out, dev)
    ld_res = _rows(residual, "residual", N, d_out, dev, y.dtype) if residual is not None else 0
    keep = z is not None and z is not False
    if z is True:
        z, ld_z = x.new_empty(N, d_out), d_out
    else:
        ld_z = _rows(z, "z", N, d_out, dev, bf) if keep else 0
    st = lib().dust_linear(x.data_ptr(), ld_x, W.data_ptr(), _ptr(bias), _act_code(act), _ptr(residual), ld_res,
                           DUST_BF16, N, d_in, d_out, y.data_ptr(), _dtypes()[y.dtype], ld_y,
                           z.data_ptr() if keep else None, ld_z, _raw_stream(dev))
    _check(st, "dust_linear")
    return (y, z) if keep else y


def dust_linear_backward(dy, x, W, act: str = "none", z=None, dx=True, dW=True, db=True, accumulate: bool = False,
                         dx_dtype=None, workspace=None, stream=None, g_terms: int = G_TERMS):
    """(dx, dW, db) of dust_linear from dy [N, d_out] (bf16 or fp32) and the pre-activation z that it
    kept (not needed for act="none"): dx [N, d_in] bf16 (or dx_dtype=torch.float32), dW fp32
    [d_out, d_in], db fp32 [d_out].  dz = dy act'(z) goes to the tensor cores as g_terms bf16 terms in dW and in
    an fp32 dx, as one in a bf16 dx (a bf16 dy without an activation is exact in one).  Each output is True (allocated), a tensor, or None (skipped);
    accumulate=True adds to the given dW and db."""
    torch = _torch()
    bf, f32 = torch.bfloat16, torch.float32
    dev = dy.get_device()
    scope = _scope(dev, stream)
    if scope is not None:
        with scope:
            return dust_linear_backward(dy, x, W, act, z, dx, dW, db, accumulate, dx_dtype, workspace, None, g_terms)
    if dy.dim() != 2 or x.dim() != 2 or W.dim() != 2:
        raise ValueError("dy must be [N, d_out], x [N, d_in], W [d_out, d_in]")
    N, d_out = dy.shape
    d_in = x.shape[1]
    ld_dy = _rows(dy, "dy", N, d_out, dev)
    ld_x = _rows(x, "x", N, d_in, dev, bf)
    if W.shape != (d_out, d_in):
        raise ValueError("dy must be [N, d_out], x [N, d_in], W [d_out, d_in]")
    _flat(W, "W", d_out * d_in, dev, bf)
    code = _act_code(act)
    if code and z is None:
        raise ValueError(f"act={act!r} needs the pre-activation z that dust_linear kept")
    ld_z = _rows(z, "z", N, d_out, dev, bf) if code else 0
    if accumulate and (dW is True or db is True):
        raise ValueError("accumulate adds to given dW and db tensors; pass them, or None to skip them")
    if dx is True:
        dx, ld_dx = x.new_empty(N, d_in, dtype=dx_dtype), d_in  # x's type, bf16, by default
        if dx.dtype not in _dtypes():
            raise TypeError(f"dx_dtype must be bf16 or fp32, not {dx_dtype}")
    elif dx is None or dx is False:
        dx, ld_dx = None, 0
    else:
        if dx_dtype is not None and dx.dtype != dx_dtype:
            raise TypeError(f"dx is {dx.dtype}, dx_dtype {dx_dtype}")
        ld_dx = _rows(dx, "dx", N, d_in, dev)
    if dW is True:
        dW = x.new_empty(d_out, d_in, dtype=f32)
    elif dW is None or dW is False:
        dW = None
    else:
        _flat(dW, "dW", d_out * d_in, dev, f32)
    if db is True:
        db = x.new_empty(d_out, dtype=f32)
    elif db is None or db is False:
        db = None
    else:
        _flat(db, "db", d_out, dev, f32)
    at, nb, ws = _new_workspace(workspace, dust_workspace_size(DUST_OP_LINEAR_BACKWARD, DUST_BF16, N, d_in, d_out, 0), x)
    st = lib().dust_linear_backward(dy.data_ptr(), _dtypes()[dy.dtype], ld_dy, z.data_ptr() if code else None, ld_z,
                                    x.data_ptr(), ld_x, W.data_ptr(), code, DUST_BF16, N, d_in, d_out,
                                    int(g_terms), _ptr(dx),
                                    DUST_F32 if dx is not None and dx.dtype == f32 else DUST_BF16, ld_dx,
                                    _ptr(dW), _ptr(db), 1 if accumulate else 0, at, nb, _raw_stream(dev))
    _check(st, "dust_linear_backward")
    return dx, dW, db


def _check_ids(ids) -> int:
    torch = _torch()
    if ids.dtype is not torch.int32:
        raise TypeError("ids must be int32")
    if ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous CUDA vector")
    return ids.numel()


def dust_embedding(ids, E, scale: float = 1.0, out=None, out_dtype=None, stream=None):
    """out[N, d] = scale E[ids] for int32 ids [N] and a bf16 or fp32 table E [V, d] (out of E's type, or
    out_dtype).  A negative id gives a zero row, an id >= V a NaN row."""
    N = _check_ids(ids)
    dev = ids.get_device()
    scope = _scope(dev, stream)
    if scope is not None:
        with scope:
            return dust_embedding(ids, E, scale, out, out_dtype)
    if E.dim() != 2:
        raise ValueError("E must be [V, d]")
    V, d = E.shape
    ld_E = _rows(E, "E", V, d, dev)
    codes = _dtypes()
    if out is None:
        out, ld_out = _new_rows(E, N, d, out_dtype or E.dtype, 8)
        if out.dtype not in codes:
            raise TypeError(f"out_dtype must be bf16 or fp32, not {out.dtype}")
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    else:
        ld_out = _rows(out, "out", N, d, dev)
    st = lib().dust_embedding(ids.data_ptr(), E.data_ptr(), codes[E.dtype], ld_E, N, V, d, scale, out.data_ptr(),
                              codes[out.dtype], ld_out, _raw_stream(dev))
    if st:
        _check(st, "dust_embedding")
    return out


def dust_embedding_grad(ids, g, V: int, scale: float = 1.0, G=None, accumulate: bool = False, workspace=None,
                        stream=None):
    """The table's gradient G[v] (+)= scale sum of g[t] over the tokens with ids[t] = v, fp32 [V, d], from g
    [N, d] (bf16 or fp32).  accumulate=True adds to the rows of the given G that have tokens."""
    torch = _torch()
    N = _check_ids(ids)
    dev = ids.get_device()
    scope = _scope(dev, stream)
    if scope is not None:
        with scope:
            return dust_embedding_grad(ids, g, V, scale, G, accumulate, workspace)
    if g.dim() != 2:
        raise ValueError("g must be [N, d]")
    d = g.shape[1]
    ld_g = _rows(g, "g", N, d, dev)
    if G is not None:
        ld_G = _rows(G, "G", V, d, dev, torch.float32)
    elif accumulate:
        raise ValueError("accumulate adds to a given G")
    else:
        G, ld_G = _new_rows(g, V, d, torch.float32, 4)
    dt = _dtypes()[g.dtype]
    nb = 0 if N <= DUST_EMBEDDING_SMALL else dust_workspace_size(DUST_OP_EMBEDDING_GRAD, dt, N, V, d, 0)
    at, nb, ws = _new_workspace(workspace, nb, g)
    st = lib().dust_embedding_grad(ids.data_ptr(), g.data_ptr(), dt, ld_g, N, V, d, scale, G.data_ptr(), ld_G,
                                   1 if accumulate else 0, at, nb, _raw_stream(dev))
    if st:
        _check(st, "dust_embedding_grad")
    return G


class DustOptimizer:
    """One optimizer step over many tensors in one launch (dust_optimizer_step_grouped), with the moments
    in fp32 (bits=32) or e4m3 codes with a scale for each block of 256 elements (bits=8, Adam only).

    W: list of fp32 master weights (any shapes, contiguous); G: list of their gradients (all fp32 or
    all bf16); W_bf16: optional list of bf16 copies to refresh (entries may be None).  lr_scale and
    decay multiply the learning rate and the weight decay tensor by tensor (decay=False: none).
    The moments are the lists ``m`` and ``v`` (bits=8: torch.float8_e4m3fn codes of m and of sqrt(v), with
    ``m_scale`` and ``v_scale``), created as zeros or taken over from m=, v=, m_scale=, v_scale=."""

    def __init__(self, W, G, W_bf16=None, bits: int = 32, lr_scale=None, decay=None, m=None, v=None, m_scale=None,
                 v_scale=None):
        torch = _torch()
        if bits not in (32, 8):
            raise ValueError("bits must be 32 or 8")
        self.W, self.bits = list(W), bits
        k = len(self.W)
        if k == 0:
            raise ValueError("no tensors")
        self.device = self.W[0].device
        self._index = self.W[0].get_device()
        dev, f32 = self.device, torch.float32
        sizes = [t.numel() for t in self.W]
        state = f32 if bits == 32 else torch.float8_e4m3fn

        def take(given, what, dtype, counts, may_skip=False, zeros=False):
            if given is None:
                return [torch.zeros(n, dtype=dtype, device=dev) if zeros else None for n in counts]
            given = list(given)
            if len(given) != k:
                raise ValueError(f"{what} must have one entry for each of the {k} tensors")
            for i, (t, n) in enumerate(zip(given, counts)):
                if t is not None or not may_skip:
                    _flat(t, f"{what}[{i}]", n, self._index, dtype)
            return given

        take(self.W, "W", f32, sizes)
        self.W_bf16 = take(W_bf16, "W_bf16", torch.bfloat16, sizes, may_skip=True)
        self.m = take(m, "m", state, sizes, zeros=True)
        self.v = take(v, "v", state, sizes, zeros=True)
        blocks = [-(-n // DUST_STATE_BLOCK) for n in sizes]
        self.m_scale = take(m_scale, "m_scale", f32, blocks, zeros=True) if bits == 8 else None
        self.v_scale = take(v_scale, "v_scale", f32, blocks, zeros=True) if bits == 8 else None
        held = [t for ts in (self.W, self.W_bf16, self.m, self.v, self.m_scale, self.v_scale) if ts is not None
                for t in ts if t is not None]
        self._written = self._spans(held)
        if any(b[0] < a[1] for a, b in zip(self._written, self._written[1:])):
            raise ValueError("weights and moments must not share memory")
        self._desc = (dust_opt_tensor * k)()
        for i, d in enumerate(self._desc):
            d.W, d.W_bf16, d.m, d.v = (_ptr(t) for t in (self.W[i], self.W_bf16[i], self.m[i], self.v[i]))
            if bits == 8:
                d.m_scale, d.v_scale = self.m_scale[i].data_ptr(), self.v_scale[i].data_ptr()
            d.n = sizes[i]
            d.lr_scale = 1.0 if lr_scale is None else float(lr_scale[i])
            d.decay_scale = 1.0 if decay is None else float(decay[i])
        self.set_gradients(G)

    @staticmethod
    def _spans(tensors):
        """(first byte, byte behind the last) of each tensor that has elements, by address."""
        return sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors if t.numel())

    def set_gradients(self, G) -> None:
        """Takes other gradient tensors for the steps that follow.  They may share memory with one another, not with
        the weights and moments."""
        torch = _torch()
        G = list(G)
        if len(G) != len(self.W):
            raise ValueError(f"G must have one entry for each of the {len(self.W)} tensors")
        dtype = G[0].dtype
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"gradients are fp32 or bf16, not {dtype}")
        for i, (g, w) in enumerate(zip(G, self.W)):
            _flat(g, f"G[{i}]", w.numel(), self._index, dtype)
        # by address, the last span that begins before a gradient's end is the one that can reach into it
        begins = [a for a, _ in self._written]
        for a, b in self._spans(G):
            at = bisect.bisect_left(begins, b) - 1
            if at >= 0 and self._written[at][1] > a:
                raise ValueError("gradients must not share memory with weights or moments")
        self.G, self._g_dt = G, DUST_F32 if dtype == torch.float32 else DUST_BF16
        for d, g in zip(self._desc, G):
            d.G = g.data_ptr()

    def step(self, opt: dust_opt_params, g_scale=None, step=None, stream=None):
        """One step with the hyper-parameters of sgd_momentum(...) or adam(...).  g_scale: optional fp32
        CUDA scalar that multiplies every gradient.  step: optional int32 CUDA scalar with Adam's
        step count, read when the step runs (for captured graphs); None takes opt.step."""
        torch = _torch()
        scope = _scope(self._index, stream)
        if scope is not None:
            with scope:
                return self.step(opt, g_scale, step)
        if g_scale is not None:
            _flat(g_scale, "g_scale", 1, self._index, torch.float32)
        if step is not None:
            _flat(step, "step", 1, self._index, torch.int32)
        st = lib().dust_optimizer_step_grouped(ctypes.byref(opt), self._desc, len(self.W), self._g_dt,
                                               DUST_STATE_F32 if self.bits == 32 else DUST_STATE_E4M3,
                                               _ptr(g_scale), _ptr(step), _raw_stream(self._index))
        _check(st, "dust_optimizer_step_grouped")
        return self.W


def dust_last_device_error(stream=None, device=None) -> Tuple[int, int]:
    """(status, info) of the device error word, which is then cleared."""
    torch = _torch()
    dev = device if device is not None else torch.cuda.current_device()
    info = ctypes.c_int32(0)
    st = lib().dust_last_device_error(_stream(dev, stream), ctypes.byref(info))
    return int(st), int(info.value)


def dust_debug_philox(ctr, seed: int, stream=None):
    """Words (uint32 as int64) and fp32 normals for counters ctr [n, 4] (uint32 as int32)."""
    torch = _torch()
    _cuda(ctr, "ctr")
    n = ctr.shape[0]
    words = torch.empty((n, 4), dtype=torch.int32, device=ctr.device)
    normals = torch.empty((n, 4), dtype=torch.float32, device=ctr.device)
    st = lib().dust_debug_philox(ctr.data_ptr(), n, seed & 0xFFFFFFFFFFFFFFFF, words.data_ptr(),
                                 normals.data_ptr(), _stream(ctr.device, stream))
    _check(st, "dust_debug_philox")
    return words, normals


def dust_debug_normal_sum(key: NoiseKey, n: int, n_quads: int, out=None, device=None,
                          stream=None):
    """out[g] = sum of the 4 n_quads normals of token key.token_offset + g (draw
    key.draw_offset, channels from key.channel_offset): the generator-only throughput probe."""
    torch = _torch()
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=device or "cuda")
    _cuda(out, "out")
    st = lib().dust_debug_normal_sum(key.c(), n, n_quads, out.data_ptr(),
                                     _stream(out.device, stream))
    _check(st, "dust_debug_normal_sum")
    return out


def dust_debug_word_sum(key: NoiseKey, n: int, n_blocks: int, out=None, device=None,
                        stream=None):
    """out[g] (int32 bits of uint32) = XOR of the words of the Philox blocks (channel quad
    key.channel_offset / 4 + j, token key.token_offset + g, draw key.draw_offset), j < n_blocks:
    the generator's integer part alone, as a throughput probe."""
    torch = _torch()
    if out is None:
        out = torch.empty(n, dtype=torch.int32, device=device or "cuda")
    _cuda(out, "out")
    st = lib().dust_debug_word_sum(key.c(), n, n_blocks, out.data_ptr(),
                                   _stream(out.device, stream))
    _check(st, "dust_debug_word_sum")
    return out


def dust_debug_fwd_plan(N: int, K: int, d_outs, sms: int):
    """(persistent, tail split) of the bf16 forward for layers of output widths `d_outs` on a
    device with `sms` SMs (host only; no device needed)."""
    arr = (ctypes.c_int32 * len(d_outs))(*[int(d) for d in d_outs])
    p, sp = ctypes.c_int32(0), ctypes.c_int32(0)
    st = lib().dust_debug_fwd_plan(int(N), int(K), len(d_outs), ctypes.cast(arr, ctypes.c_void_p),
                                   int(sms), ctypes.byref(p), ctypes.byref(sp))
    _check(st, "dust_debug_fwd_plan")
    return bool(p.value), sp.value


def dust_debug_credit_skip_publish(block: int) -> None:
    lib().dust_debug_credit_skip_publish(int(block))


def dust_profile_enable(capacity: int) -> None:
    _check(lib().dust_profile_enable(int(capacity)), "dust_profile_enable")


def dust_profile_disable() -> None:
    lib().dust_profile_disable()


def dust_profile_read(max_records: int = 1 << 16):
    """[(kernel name, milliseconds)] of the launches recorded since enabling (synchronizes)."""
    names = (ctypes.c_char_p * max_records)()
    ms = (ctypes.c_float * max_records)()
    n = lib().dust_profile_read(names, ms, max_records)
    return [(names[i].decode(), float(ms[i])) for i in range(n)]


def _sequence_cuts(cu, N: int, chunks: int):
    """Token cuts [0, ..., N] at sequence ends near k N / chunks, kept at multiples of 4 tokens
    so that every run's row and column views stay 16-byte aligned."""
    import numpy as np
    ends = cu[(cu % 4 == 0) & (cu > 0) & (cu < N)]
    cuts = [0]
    for c in range(1, chunks):
        if ends.size == 0:
            break
        e = int(ends[int(np.argmin(np.abs(ends - N * c / chunks)))])
        if e > cuts[-1]:
            cuts.append(e)
    cuts.append(N)
    return cuts


class DustStack:
    """Many bf16 layers sharing one token batch (a transformer block stack), estimated with the
    grouped calls: one launch per step for up to 64 layers.  ``layers`` is a list of
    (x, W, u, layer_id) device tensors; outputs live in ``dloss[l]``, ``r[l]``, ``G_W[l]``.
    The weight estimates are views of one flat fp32 buffer ``G_W_flat`` (layer l at
    ``layout[l]``), so that consecutive layers can be exchanged between ranks in one call."""

    def __init__(self, layers, K: int, want_g: bool = False, g_terms: int = G_TERMS):
        from . import distributed
        torch = _torch()
        self.K = K
        self.g_terms = g_terms
        self.layers = layers
        x0 = layers[0][0]
        self.N = x0.shape[0]
        dev = x0.device
        n = len(layers)
        self.dloss = [torch.empty((K, self.N), dtype=torch.float32, device=dev) for _ in range(n)]
        self.r = [torch.empty((K, self.N), dtype=torch.float32, device=dev) for _ in range(n)]
        self.layout, total = distributed.flat_layout([(W.shape[0], W.shape[1])
                                                      for (_, W, _, _) in layers])
        self.G_W_flat = torch.empty(total, dtype=torch.float32, device=dev)
        self.G_W = [self.G_W_flat[o:o + m].view(W.shape[0], W.shape[1])
                    for (o, m), (_, W, _, _) in zip(self.layout, layers)]
        self.g = ([torch.empty((self.N, W.shape[0]), dtype=torch.float32, device=dev)
                   for (_, W, _, _) in layers] if want_g else None)
        self.desc = (dust_layer_desc * n)()
        for l, (x, W, u, layer_id) in enumerate(layers):
            for t, nm in ((x, "x"), (W, "W"), (u, "u")):
                _cuda(t, nm)
                if t.dtype != torch.bfloat16:
                    raise TypeError("grouped calls take bf16 layers")
            if x.shape[0] != self.N or u.shape != (self.N, W.shape[0]) or x.shape[1] != W.shape[1]:
                raise ValueError("layer shapes: x [N, d_in], W [d_out, d_in], u [N, d_out]")
            d = self.desc[l]
            d.x, d.W, d.u = x.data_ptr(), W.data_ptr(), u.data_ptr()
            d.d_in, d.d_out = x.shape[1], W.shape[0]
            d.layer_id, d.reserved = layer_id, 0
            d.dloss, d.ld_dloss = self.dloss[l].data_ptr(), self.N
            d.r, d.ld_r = self.r[l].data_ptr(), self.N
            d.G_W = self.G_W[l].data_ptr()
            d.g_out = self.g[l].data_ptr() if want_g else None
        self.ws = torch.empty(max(self._ws_need(self.desc, n, self.N), 256), dtype=torch.uint8,
                              device=dev)
        self._comm = None

    def _ws_need(self, desc, n: int, N: int) -> int:
        return max(int(lib().dust_workspace_size_grouped(op, desc, n, N, self.K))
                   for op in range(3))

    @staticmethod
    def _sub(desc, l0: int):
        """Pointer to descriptor l0 of a descriptor array (a bucket of consecutive layers)."""
        return ctypes.cast(ctypes.addressof(desc) + l0 * ctypes.sizeof(dust_layer_desc),
                           ctypes.POINTER(dust_layer_desc))

    def _weight_grad(self, desc, N: int, key, accumulate: bool, s: int, reduce, buckets: int):
        """The grouped weight estimate; with ``reduce``, in buckets of consecutive layers, each
        bucket's span of G_W_flat handed to ``reduce`` on a side stream as soon as its launch
        is queued, so the exchange overlaps the later buckets' work."""
        from . import distributed
        torch = _torch()
        n = len(self.layers)
        nb = self.ws.numel()
        if reduce is None:
            _check(lib().dust_weight_grad_grouped(desc, n, N, self.K, self.K, float(self.sigma),
                                                  key, 1 if accumulate else 0, self.g_terms,
                                                  self.ws.data_ptr(), nb, s),
                   "dust_weight_grad_grouped")
            return
        dev = self.ws.device
        comp = torch.cuda.current_stream(dev)
        if self._comm is None:
            self._comm = torch.cuda.Stream(device=dev)
        plan = distributed.plan_buckets([m for _, m in self.layout], buckets)
        for l0, l1 in plan:
            sub = self._sub(desc, l0)
            need = int(lib().dust_workspace_size_grouped(DUST_OP_WEIGHT_GRAD, sub, l1 - l0, N,
                                                         self.K))
            if need > nb:
                raise RuntimeError("stack workspace too small for a bucket")
            _check(lib().dust_weight_grad_grouped(sub, l1 - l0, N, self.K, self.K,
                                                  float(self.sigma), key,
                                                  1 if accumulate else 0, self.g_terms,
                                                  self.ws.data_ptr(), nb, s),
                   "dust_weight_grad_grouped")
            ev = torch.cuda.Event()
            ev.record(comp)
            self._comm.wait_event(ev)
            with torch.cuda.stream(self._comm):
                a, b = distributed.bucket_span(self.layout, (l0, l1))
                reduce(self.G_W_flat[a:b])
        comp.wait_stream(self._comm)

    def estimate(self, cu_seqlens, sigma: float, gamma: float, seed: int, draw_offset: int = 0,
                 token_offset: int = 0, stream=None, reduce=None, buckets: int = 12):
        """Forward, credit and weight estimate of every layer on the device inputs.  ``reduce``
        (optional, e.g. a sum over data-parallel ranks) is applied to G_W_flat in ``buckets``
        spans of consecutive layers, overlapped with the remaining weight estimates; it must
        run on the current stream (torch collectives do).  ``stream`` must be None (the
        current stream) when ``reduce`` is given."""
        if reduce is not None and stream is not None:
            raise ValueError("reduce runs against the current stream; pass stream=None")
        n = len(self.layers)
        s = _stream(self.ws.device, stream)
        nb = self.ws.numel()
        self.sigma = sigma
        key = NoiseKey(seed, 0, draw_offset, token_offset).c()
        _check(lib().dust_noisy_linear_fwd_grouped(self.desc, n, self.N, self.K, float(sigma), key,
                                                   self.ws.data_ptr(), nb, s),
               "dust_noisy_linear_fwd_grouped")
        _check(lib().dust_credit_grouped(self.desc, n, self.K, self.N, cu_seqlens.data_ptr(),
                                         cu_seqlens.numel() - 1, float(gamma), self.ws.data_ptr(),
                                         nb, s), "dust_credit_grouped")
        self._weight_grad(self.desc, self.N, key, False, s, reduce, buckets)
        return self.G_W

    def estimate_from_host(self, host_layers, cu_seqlens, sigma: float, gamma: float,
                           seed: int, G_host=None, chunks: int = 12, reduce=None,
                           draw_offset: int = 0, token_offset: int = 0):
        """The estimate from inputs in pinned host memory (``host_layers``: one (x, W, u) per
        layer, the shapes of the stack's device tensors, which receive them), pipelined over
        ``chunks`` buckets of consecutive layers of about equal input bytes: a copy stream
        uploads bucket after bucket; each bucket goes through the grouped forward, credit and
        weight estimate as soon as its inputs are in; its span of G_W_flat is copied back on a
        third stream (into ``G_host``, pinned, allocated if None) while the later buckets are
        uploaded and estimated.  ``reduce`` (optional, e.g. the sum over data-parallel ranks)
        is applied to each bucket's span on a side stream before it is copied back.
        Synchronises."""
        from . import distributed
        import numpy as np
        torch = _torch()
        dev = self.ws.device
        cu = np.asarray(cu_seqlens, dtype=np.int64)
        N = int(cu[-1])
        if N != self.N or len(host_layers) != len(self.layers):
            raise ValueError("host inputs do not match the stack")
        self.sigma = sigma
        if not hasattr(self, "_copy"):
            self._copy = torch.cuda.Stream(device=dev)
            self._back = torch.cuda.Stream(device=dev)
        comp = torch.cuda.current_stream(dev)
        cu_d = torch.from_numpy(cu.astype(np.int32)).pin_memory().to(dev, non_blocking=True)
        sizes = [sum(t.numel() * t.element_size() for t in h) for h in host_layers]
        plan = distributed.plan_buckets(sizes, chunks)
        ready = []
        self._copy.wait_stream(comp)  # the uploads start after the work already queued
        with torch.cuda.stream(self._copy):
            for l0, l1 in plan:
                for (x, W, u, _), (hx, hW, hu) in zip(self.layers[l0:l1], host_layers[l0:l1]):
                    W.copy_(hW, non_blocking=True)
                    x.copy_(hx, non_blocking=True)
                    u.copy_(hu, non_blocking=True)
                ev = torch.cuda.Event()
                ev.record(self._copy)
                ready.append(ev)
        if G_host is None:
            G_host = torch.empty(self.G_W_flat.shape, dtype=torch.float32, pin_memory=True)
        nb = self.ws.numel()
        s = _stream(dev, None)
        key = NoiseKey(seed, 0, draw_offset, token_offset).c()
        if reduce is not None and self._comm is None:
            self._comm = torch.cuda.Stream(device=dev)
        for (l0, l1), ev in zip(plan, ready):
            comp.wait_event(ev)
            n = l1 - l0
            sub = self._sub(self.desc, l0)
            if self._ws_need(sub, n, N) > nb:
                raise RuntimeError("stack workspace too small for a bucket")
            _check(lib().dust_noisy_linear_fwd_grouped(sub, n, N, self.K, float(sigma), key,
                                                       self.ws.data_ptr(), nb, s),
                   "dust_noisy_linear_fwd_grouped")
            _check(lib().dust_credit_grouped(sub, n, self.K, N, cu_d.data_ptr(), cu_d.numel() - 1,
                                             float(gamma), self.ws.data_ptr(), nb, s),
                   "dust_credit_grouped")
            _check(lib().dust_weight_grad_grouped(sub, n, N, self.K, self.K, float(sigma), key, 0,
                                                  self.g_terms, self.ws.data_ptr(), nb, s),
                   "dust_weight_grad_grouped")
            a, b = distributed.bucket_span(self.layout, (l0, l1))
            done = torch.cuda.Event()
            done.record(comp)
            src = comp
            if reduce is not None:
                self._comm.wait_event(done)
                with torch.cuda.stream(self._comm):
                    reduce(self.G_W_flat[a:b])
                src = self._comm
            self._back.wait_stream(src)
            with torch.cuda.stream(self._back):
                G_host[a:b].copy_(self.G_W_flat[a:b], non_blocking=True)
        comp.wait_stream(self._back)
        comp.synchronize()
        return G_host


class DustLayer:
    """One layer's estimator with workspaces kept between calls (fwd -> credit -> weight grad)."""

    def __init__(self, N: int, d_in: int, d_out: int, K: int, dtype, device):
        torch = _torch()
        dt = DUST_BF16 if dtype == torch.bfloat16 else DUST_F32
        self.N, self.d_in, self.d_out, self.K = N, d_in, d_out, K
        nbytes = max(dust_workspace_size(op, dt, N, d_in, d_out, K) for op in range(3))
        self.ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        self.dloss = torch.empty((K, N), dtype=torch.float32, device=device)
        self.r = torch.empty((K, N), dtype=torch.float32, device=device)
        self.G_W = torch.empty((d_out, d_in), dtype=torch.float32, device=device)

    def estimate(self, x, W, u, cu_seqlens, sigma: float, gamma: float, key: NoiseKey,
                 stream=None):
        dust_noisy_linear_fwd(x, W, u, self.K, sigma, key, self.dloss, self.ws, stream)
        dust_credit(self.dloss, cu_seqlens, gamma, self.r, self.ws, stream)
        dust_weight_grad(self.r, x, self.d_out, self.K, sigma, key, self.G_W, False, None,
                         self.ws, stream)
        return self.G_W

    def estimate_from_host(self, hx, hW, hu, cu_seqlens, sigma: float, gamma: float,
                           key: NoiseKey, G_host=None, chunks: int = 4, reduce=None):
        """The estimate from inputs in pinned host memory, with the upload overlapped: the
        tokens are cut into ``chunks`` runs of whole sequences; each run is copied on a copy
        stream while the previous one goes through the forward, the credit and the weight
        estimate (accumulated over the runs, token offsets keeping the noise of the whole
        batch).  ``reduce`` (optional) is applied to the device G_W before it is copied back
        (for instance the all-reduce over data-parallel ranks).  G_W comes back into
        ``G_host`` (pinned, allocated if None).  Synchronises."""
        import numpy as np
        torch = _torch()
        dev = self.ws.device
        cu = np.asarray(cu_seqlens, dtype=np.int64)
        N = int(cu[-1])
        if N != self.N:
            raise ValueError("cu_seqlens does not cover the layer's N tokens")
        if not hasattr(self, "_x"):
            self._x = torch.empty((N, self.d_in), dtype=hx.dtype, device=dev)
            self._u = torch.empty((N, self.d_out), dtype=hu.dtype, device=dev)
            self._W = torch.empty((self.d_out, self.d_in), dtype=hW.dtype, device=dev)
            self._copy = torch.cuda.Stream(device=dev)
        # cuts at sequence ends that keep the per-run views 16-byte aligned
        cuts = _sequence_cuts(cu, N, chunks)
        # every run's local cu_seqlens, uploaded once
        locs = [(cu[(cu >= a) & (cu <= b)] - a).astype(np.int32) for a, b in zip(cuts[:-1], cuts[1:])]
        cu_all = torch.from_numpy(np.concatenate(locs)).pin_memory().to(dev, non_blocking=True)
        offs = np.cumsum([0] + [len(l) for l in locs])
        comp = torch.cuda.current_stream(dev)
        ready = []
        self._copy.wait_stream(comp)  # the uploads start after the work already queued
        with torch.cuda.stream(self._copy):
            self._W.copy_(hW, non_blocking=True)
            for a, b in zip(cuts[:-1], cuts[1:]):
                self._x[a:b].copy_(hx[a:b], non_blocking=True)
                self._u[a:b].copy_(hu[a:b], non_blocking=True)
                ev = torch.cuda.Event()
                ev.record(self._copy)
                ready.append(ev)
        for n, ((a, b), ev) in enumerate(zip(zip(cuts[:-1], cuts[1:]), ready)):
            comp.wait_event(ev)
            cu_d = cu_all[int(offs[n]):int(offs[n + 1])]
            k = key._replace(token_offset=key.token_offset + a)
            x, u = self._x[a:b], self._u[a:b]
            dl, r = self.dloss[:, a:b], self.r[:, a:b]
            dust_noisy_linear_fwd(x, self._W, u, self.K, sigma, k, dl, self.ws)
            dust_credit(dl, cu_d, gamma, r, self.ws)
            dust_weight_grad(r, x, self.d_out, self.K, sigma, k, self.G_W, n > 0, None, self.ws)
        if reduce is not None:
            reduce(self.G_W)
        if G_host is None:
            G_host = torch.empty(self.G_W.shape, dtype=self.G_W.dtype, pin_memory=True)
        G_host.copy_(self.G_W, non_blocking=True)
        torch.cuda.current_stream(dev).synchronize()
        return G_host
