"""Gated DeltaNet-2 token mixer for MI355X (gfx950): Python binding of libgdn2.

A thin ctypes layer over the C ABI in ``include/gdn2.h``: it checks tensor
shapes, dtypes and devices, allocates outputs and workspace with PyTorch, sets
the library's stream to PyTorch's current stream and calls the library. Every
step of the computation runs in the HIP kernels; there is no other code path,
and importing this package fails if the library has not been built.

Recurrence (snilld.dk, "Hvad Gated DeltaNet-2 ændrer", update equation), per
sequence and head, state S in R^{dk x dv}:
    S_t = (I - k_t (b_t * k_t)^T) Diag(exp(log_alpha_t)) S_{t-1} + k_t (w_t * v_t)^T
    o_t = S_t^T q_t

Around it, for a whole layer: ``prologue_fwd`` / ``prologue_bwd`` (short
convolution, unit norm, sigmoid), ``recurrent_fwd`` (the recurrence over a few
tokens a sequence, its states in a pool) and ``layer_norm_fwd`` /
``layer_norm_bwd``; the layer's dense half: ``linear_fwd`` / ``linear_bwd``
(projections with bias, activation and residual, in bf16, fp32 or 8 bits),
``rms_norm_fwd`` / ``rms_norm_bwd`` before them (its output in 8 bits with
scales, if wanted), and ``grad_norm`` / ``clip_grads`` over a model's gradients.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, 'libgdn2.so')

GDN2_OK, GDN2_ERR_INVALID, GDN2_ERR_UNSUPPORTED, GDN2_ERR_WORKSPACE, GDN2_ERR_HIP = range(5)
GDN2_F32, GDN2_BF16, GDN2_E4M3 = 0, 1, 2
ACTIVATIONS = {None: 0, 'none': 0, 'sigmoid': 1, 'silu': 2, 'gelu_tanh': 3}
GDN2_GATES_PER_CHANNEL, GDN2_GATE_B_PER_HEAD, GDN2_GATE_W_PER_HEAD, GDN2_GATE_ALPHA_PER_HEAD = 0, 1, 2, 4
CHUNK = 64

EXPORTS = ('gdn2_set_stream', 'gdn2_get_stream', 'gdn2_status_string',
           'gdn2_chunk_fwd_workspace_bytes', 'gdn2_chunk_fwd', 'gdn2_chunk_fwd_noalloc', 'gdn2_chunk_fwd_gates',
           'gdn2_chunk_fwd_sized_workspace_bytes', 'gdn2_chunk_fwd_sized',
           'gdn2_decode_step', 'gdn2_decode_step_gates',
           'gdn2_chunk_fwd_prologue', 'gdn2_decode_step_prologue',
           'gdn2_chunk_bwd_workspace_bytes', 'gdn2_chunk_bwd', 'gdn2_chunk_fwd_keep', 'gdn2_chunk_bwd_kept',
           'gdn2_recurrent_fwd', 'gdn2_prologue_fwd', 'gdn2_prologue_bwd_workspace_bytes', 'gdn2_prologue_bwd',
           'gdn2_layer_norm_fwd', 'gdn2_layer_norm_bwd_workspace_bytes', 'gdn2_layer_norm_bwd',
           'gdn2_linear_fwd', 'gdn2_linear_bwd_workspace_bytes', 'gdn2_linear_bwd',
           'gdn2_rms_norm_fwd', 'gdn2_rms_norm_bwd_workspace_bytes', 'gdn2_rms_norm_bwd',
           'gdn2_clip_grads_workspace_bytes', 'gdn2_grad_norm', 'gdn2_clip_grads',
           'gdn2_profile_begin', 'gdn2_profile_end', 'gdn2_profile_kernel')


class ShortConv(ctypes.Structure):
    """gdn2_short_conv: taps, biases and history of the three short convolutions."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        'weight_q', 'weight_k', 'weight_v', 'bias_q', 'bias_k', 'bias_v',
        'state_in_q', 'state_in_k', 'state_in_v', 'state_out_q', 'state_out_k', 'state_out_v')]


class Gdn2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f'{where}: {status_string(status)}')
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f'{LIB_PATH} is missing: build it first (python -c "import __graft_entry__ as g; g.build()")')
    lib = ctypes.CDLL(LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.gdn2_set_stream.argtypes = [vp]
    lib.gdn2_set_stream.restype = i
    lib.gdn2_get_stream.argtypes = []
    lib.gdn2_get_stream.restype = vp
    lib.gdn2_status_string.argtypes = [i]
    lib.gdn2_status_string.restype = ctypes.c_char_p
    lib.gdn2_chunk_fwd_workspace_bytes.argtypes = [i] * 8
    lib.gdn2_chunk_fwd_workspace_bytes.restype = sz
    lib.gdn2_chunk_fwd.argtypes = [vp] * 10 + [i] * 8 + [vp, sz]
    lib.gdn2_chunk_fwd.restype = i
    lib.gdn2_chunk_fwd_noalloc.argtypes = [vp] * 10 + [i] * 8
    lib.gdn2_chunk_fwd_noalloc.restype = i
    lib.gdn2_chunk_fwd_gates.argtypes = [vp] * 6 + [i] + [vp] * 4 + [i] * 8 + [vp, sz]
    lib.gdn2_chunk_fwd_gates.restype = i
    lib.gdn2_chunk_fwd_sized_workspace_bytes.argtypes = [i] * 9
    lib.gdn2_chunk_fwd_sized_workspace_bytes.restype = sz
    lib.gdn2_chunk_fwd_sized.argtypes = [vp] * 10 + [i] * 9 + [vp, sz]
    lib.gdn2_chunk_fwd_sized.restype = i
    lib.gdn2_decode_step.argtypes = [vp] * 8 + [i] * 6
    lib.gdn2_decode_step.restype = i
    lib.gdn2_decode_step_gates.argtypes = [vp] * 6 + [i] + [vp] * 2 + [i] * 6
    lib.gdn2_decode_step_gates.restype = i
    pc = ctypes.POINTER(ShortConv)
    lib.gdn2_chunk_fwd_prologue.argtypes = [vp] * 6 + [pc] + [vp] * 4 + [i] * 8 + [vp, sz]
    lib.gdn2_chunk_fwd_prologue.restype = i
    lib.gdn2_decode_step_prologue.argtypes = [vp] * 6 + [pc] + [vp] * 2 + [i] * 6
    lib.gdn2_decode_step_prologue.restype = i
    lib.gdn2_chunk_bwd_workspace_bytes.argtypes = [i] * 8
    lib.gdn2_chunk_bwd_workspace_bytes.restype = sz
    lib.gdn2_chunk_bwd.argtypes = [vp] * 10 + [i] * 7 + [vp] * 7 + [vp, sz]
    lib.gdn2_chunk_bwd.restype = i
    lib.gdn2_chunk_fwd_keep.argtypes = [vp] * 10 + [i] * 8 + [vp, sz]
    lib.gdn2_chunk_fwd_keep.restype = i
    lib.gdn2_chunk_bwd_kept.argtypes = [vp] * 10 + [i] * 7 + [vp] * 7 + [vp, sz]
    lib.gdn2_chunk_bwd_kept.restype = i
    i64, f = ctypes.c_int64, ctypes.c_float
    lib.gdn2_recurrent_fwd.argtypes = [vp] * 6 + [i] + [vp] * 6 + [i] * 10
    lib.gdn2_recurrent_fwd.restype = i
    lib.gdn2_prologue_fwd.argtypes = [vp] * 5 + [i, pc] + [vp] * 9 + [i] * 9
    lib.gdn2_prologue_fwd.restype = i
    lib.gdn2_prologue_bwd_workspace_bytes.argtypes = [i] * 8
    lib.gdn2_prologue_bwd_workspace_bytes.restype = sz
    lib.gdn2_prologue_bwd.argtypes = [vp] * 5 + [i, pc] + [vp] * 18 + [i] * 10 + [vp, sz]
    lib.gdn2_prologue_bwd.restype = i
    lib.gdn2_layer_norm_fwd.argtypes = [vp] * 6 + [i64, i, f, i, i]
    lib.gdn2_layer_norm_fwd.restype = i
    lib.gdn2_layer_norm_bwd_workspace_bytes.argtypes = [i64, i]
    lib.gdn2_layer_norm_bwd_workspace_bytes.restype = sz
    lib.gdn2_layer_norm_bwd.argtypes = [vp] * 7 + [i64, i, f, i, i, vp, sz]
    lib.gdn2_layer_norm_bwd.restype = i
    lib.gdn2_linear_fwd.argtypes = [vp] * 8 + [i64] + [i] * 5
    lib.gdn2_linear_fwd.restype = i
    lib.gdn2_linear_bwd_workspace_bytes.argtypes = [i64] + [i] * 8
    lib.gdn2_linear_bwd_workspace_bytes.restype = sz
    lib.gdn2_linear_bwd.argtypes = [vp] * 7 + [i64] + [i] * 5 + [vp, sz]
    lib.gdn2_linear_bwd.restype = i
    lib.gdn2_rms_norm_fwd.argtypes = [vp] * 6 + [i64, i, f, i, i]
    lib.gdn2_rms_norm_fwd.restype = i
    lib.gdn2_rms_norm_bwd_workspace_bytes.argtypes = [i64, i]
    lib.gdn2_rms_norm_bwd_workspace_bytes.restype = sz
    lib.gdn2_rms_norm_bwd.argtypes = [vp] * 6 + [i64, i, f, i, i, vp, sz]
    lib.gdn2_rms_norm_bwd.restype = i
    lib.gdn2_clip_grads_workspace_bytes.argtypes = []
    lib.gdn2_clip_grads_workspace_bytes.restype = sz
    lib.gdn2_grad_norm.argtypes = [vp, vp, vp, i, vp, vp, sz]
    lib.gdn2_grad_norm.restype = i
    lib.gdn2_clip_grads.argtypes = [vp] * 5 + [i, f, vp, i, vp, sz]
    lib.gdn2_clip_grads.restype = i
    lib.gdn2_profile_begin.argtypes = [i]
    lib.gdn2_profile_begin.restype = i
    lib.gdn2_profile_end.argtypes = []
    lib.gdn2_profile_end.restype = i
    lib.gdn2_profile_kernel.argtypes = [i, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_int),
                                        ctypes.POINTER(ctypes.c_double)]
    lib.gdn2_profile_kernel.restype = i
    return lib


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def status_string(status: int) -> str:
    return _lib.gdn2_status_string(int(status)).decode()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN2_BF16
    if t.dtype == torch.float32:
        return GDN2_F32
    raise TypeError(f'unsupported input dtype {t.dtype} (bfloat16 or float32)')


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t: torch.Tensor, name: str, shape, dtype, device):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f'{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}')
    if t.dtype != dtype:
        raise TypeError(f'{name}: expected {dtype}, got {t.dtype}')
    if t.device != device:
        raise ValueError(f'{name}: expected device {device}, got {t.device}')
    if not t.is_contiguous():
        raise ValueError(f'{name}: must be contiguous')


def set_stream(stream: Optional[torch.cuda.Stream] = None) -> None:
    """Point the library at ``stream`` (default: PyTorch's current stream)."""
    s = torch.cuda.current_stream() if stream is None else stream
    _lib.gdn2_set_stream(ctypes.c_void_p(s.cuda_stream))


def workspace_bytes(B: int, T: int, N: int, H: int, dk: int, dv: int, dtype: torch.dtype,
                    varlen: bool, chunk: int = CHUNK) -> int:
    code = GDN2_BF16 if dtype == torch.bfloat16 else GDN2_F32
    return int(_lib.gdn2_chunk_fwd_sized_workspace_bytes(B, T, N, H, dk, dv, code, int(varlen), int(chunk)))


def profile_begin(max_calls: int) -> None:
    """Time each kernel of this thread's next ``max_calls`` library calls with HIP events."""
    st = _lib.gdn2_profile_begin(int(max_calls))
    if st != GDN2_OK:
        raise Gdn2Error(st, 'gdn2_profile_begin')


def profile_end() -> dict:
    """Stop recording; return {kernel name: (launches, total ms)} for the recorded calls."""
    _lib.gdn2_profile_end()
    out = {}
    idx = 0
    while True:
        name, n, ms = ctypes.c_char_p(), ctypes.c_int(), ctypes.c_double()
        st = _lib.gdn2_profile_kernel(idx, ctypes.byref(name), ctypes.byref(n), ctypes.byref(ms))
        if st == GDN2_ERR_INVALID:
            break
        if st != GDN2_OK:
            raise Gdn2Error(st, 'gdn2_profile_kernel')
        out[name.value.decode()] = (n.value, ms.value)
        idx += 1
    return out


def _gate_layout(lead, H, dk, dv, b, w, log_alpha, dt, dev) -> int:
    """Gate layout bits from the gate shapes: a gate without the channel axis
    ([..., H]) holds one value per token-head (KDA / Gated DeltaNet forms)."""
    gates = 0
    for name, t, d, bit, tdt in (('b', b, dk, GDN2_GATE_B_PER_HEAD, dt), ('w', w, dv, GDN2_GATE_W_PER_HEAD, dt),
                                 ('log_alpha', log_alpha, dk, GDN2_GATE_ALPHA_PER_HEAD, torch.float32)):
        if t.dim() == len(lead) + 1:
            _check(t, name, (*lead, H), tdt, dev)
            gates |= bit
        else:
            _check(t, name, (*lead, H, d), tdt, dev)
    return gates


def chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor,
              b: torch.Tensor, w: torch.Tensor, S0: Optional[torch.Tensor] = None,
              cu_seqlens: Optional[torch.Tensor] = None, *, out: Optional[torch.Tensor] = None,
              final_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
              workspace: Optional[torch.Tensor] = None,
              chunk: int = CHUNK) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunkwise prefill. q, k, b: [B, T, H, dk]; v, w: [B, T, H, dv] (bf16 or
    fp32); log_alpha: [B, T, H, dk] fp32. With ``cu_seqlens`` (int32 [N+1] on
    the device) B must be 1 and the sequences are packed along T. S0: [N, H,
    dk, dv] fp32 or None (zeros). Returns (o [B, T, H, dv] fp32, S_T [N, H, dk,
    dv] fp32 or None). b, w and log_alpha may instead be [B, T, H], one gate
    per token-head (KDA: b = w = beta; Gated DeltaNet: also a scalar decay).
    ``chunk``: tokens per chunk, 64, or 32 / 128 (gdn2_chunk_fwd_sized,
    per-channel gates only)."""
    if q.dim() != 4:
        raise ValueError('q must be [B, T, H, dk]')
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    for name, t, d in (('q', q, dk), ('k', k, dk), ('v', v, dv)):
        _check(t, name, (B, T, H, d), dt, dev)
    gates = _gate_layout((B, T), H, dk, dv, b, w, log_alpha, dt, dev)
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.device != dev:
            raise ValueError('cu_seqlens must be a 1-D int32 tensor on the same device')
        if not cu_seqlens.is_contiguous():
            raise ValueError('cu_seqlens must be contiguous')
        N = cu_seqlens.numel() - 1
    else:
        N = B
    if S0 is not None:
        _check(S0, 'S0', (N, H, dk, dv), torch.float32, dev)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=torch.float32, device=dev)
    else:
        _check(out, 'out', (B, T, H, dv), torch.float32, dev)
    ST = None
    if final_state is not None:
        _check(final_state, 'final_state', (N, H, dk, dv), torch.float32, dev)
        ST = final_state
    elif output_final_state:
        ST = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    varlen = cu_seqlens is not None
    if chunk != CHUNK and gates != GDN2_GATES_PER_CHANNEL:
        raise ValueError(f'chunk = {chunk} takes per-channel gates only')
    need = _lib.gdn2_chunk_fwd_sized_workspace_bytes(B, T, N, H, dk, dv, code, int(varlen), int(chunk))
    if need == 0:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, 'gdn2_chunk_fwd_sized_workspace_bytes')
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    set_stream()
    wsb = workspace.numel() * workspace.element_size()
    if chunk == CHUNK and gates == GDN2_GATES_PER_CHANNEL:
        st = _lib.gdn2_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                 _ptr(S0), _ptr(out), _ptr(ST), _ptr(cu_seqlens),
                                 B, T, N, H, dk, dv, code, GDN2_F32, _ptr(workspace), wsb)
        where = 'gdn2_chunk_fwd'
    elif chunk == CHUNK:
        st = _lib.gdn2_chunk_fwd_gates(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), gates,
                                       _ptr(S0), _ptr(out), _ptr(ST), _ptr(cu_seqlens),
                                       B, T, N, H, dk, dv, code, GDN2_F32, _ptr(workspace), wsb)
        where = 'gdn2_chunk_fwd_gates'
    else:
        st = _lib.gdn2_chunk_fwd_sized(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                       _ptr(S0), _ptr(out), _ptr(ST), _ptr(cu_seqlens),
                                       B, T, N, H, dk, dv, code, GDN2_F32, int(chunk), _ptr(workspace), wsb)
        where = 'gdn2_chunk_fwd_sized'
    if st != GDN2_OK:
        raise Gdn2Error(st, where)
    return out, ST


def decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor,
                b: torch.Tensor, w: torch.Tensor, S: torch.Tensor, *,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token per sequence. q, k, b: [N, H, dk]; v, w: [N, H, dv]; log_alpha
    [N, H, dk] fp32; S: [N, H, dk, dv] fp32, updated in place. Returns o [N, H, dv] fp32.
    b, w and log_alpha may instead be [N, H] (one gate per sequence-head)."""
    if q.dim() != 3:
        raise ValueError('q must be [N, H, dk]')
    N, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    for name, t, d in (('q', q, dk), ('k', k, dk), ('v', v, dv)):
        _check(t, name, (N, H, d), dt, dev)
    gates = _gate_layout((N,), H, dk, dv, b, w, log_alpha, dt, dev)
    _check(S, 'S', (N, H, dk, dv), torch.float32, dev)
    if out is None:
        out = torch.empty((N, H, dv), dtype=torch.float32, device=dev)
    else:
        _check(out, 'out', (N, H, dv), torch.float32, dev)
    set_stream()
    if gates == GDN2_GATES_PER_CHANNEL:
        st = _lib.gdn2_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w),
                                   _ptr(S), _ptr(out), N, H, dk, dv, code, GDN2_F32)
        where = 'gdn2_decode_step'
    else:
        st = _lib.gdn2_decode_step_gates(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), gates,
                                         _ptr(S), _ptr(out), N, H, dk, dv, code, GDN2_F32)
        where = 'gdn2_decode_step_gates'
    if st != GDN2_OK:
        raise Gdn2Error(st, where)
    return out


def _short_conv(H, dk, dv, dev, dt, lead_n, weight, bias, state_in, state_out) -> ShortConv:
    """Marshal (q, k, v) triples of taps, biases and histories into a ShortConv."""
    dims = (dk, dk, dv)
    if weight is None or len(weight) != 3:
        raise ValueError('conv_weight must be a (q, k, v) triple of [H*d, 4] float32 tensors')
    sc = ShortConv()
    for n, t, d in zip('qkv', weight, dims):
        _check(t, f'conv_weight[{n}]', (H * d, 4), torch.float32, dev)
        setattr(sc, f'weight_{n}', t.data_ptr())
    if bias is not None:
        for n, t, d in zip('qkv', bias, dims):
            if t is not None:
                _check(t, f'conv_bias[{n}]', (H * d,), torch.float32, dev)
                setattr(sc, f'bias_{n}', t.data_ptr())
    for label, trip in (('in', state_in), ('out', state_out)):
        if trip is None:
            continue
        for n, t, d in zip('qkv', trip, dims):
            _check(t, f'conv_state_{label}[{n}]', (lead_n, H, 3, d), dt, dev)
            setattr(sc, f'state_{label}_{n}', t.data_ptr())
    return sc


def chunk_fwd_prologue(q_raw: torch.Tensor, k_raw: torch.Tensor, v_raw: torch.Tensor, log_alpha: torch.Tensor,
                       b_logit: torch.Tensor, w_logit: torch.Tensor, conv_weight, conv_bias=None,
                       S0: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
                       conv_state=None, conv_state_out=None, output_conv_state: bool = True,
                       out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                       output_final_state: bool = True, workspace: Optional[torch.Tensor] = None):
    """Prefill on the projections' outputs, with the prologue fused in:
    q = L2Norm(ShortConv(q_raw)), k = L2Norm(ShortConv(k_raw)), v = ShortConv(v_raw),
    b = sigmoid(b_logit), w = sigmoid(w_logit).

    Shapes as in ``chunk_fwd`` (gates per channel). conv_weight: (q, k, v) taps
    [H*dk, 4], [H*dk, 4], [H*dv, 4] float32, tap 3 on the current token;
    conv_bias: such a triple of [H*d] (entries may be None) or None.
    conv_state: (q, k, v) histories [N, H, 3, d] in the input dtype (the
    three raw inputs before each sequence, oldest first) or None for zeros.
    conv_state_out: tensors to receive the new histories (may be conv_state
    itself); allocated when None and ``output_conv_state``.
    Returns (o, S_T or None, conv_state_out triple or None).
    """
    if q_raw.dim() != 4:
        raise ValueError('q_raw must be [B, T, H, dk]')
    B, T, H, dk = q_raw.shape
    dv = v_raw.shape[-1]
    dev, dt = q_raw.device, q_raw.dtype
    code = _dtype_code(q_raw)
    for name, t, d in (('q_raw', q_raw, dk), ('k_raw', k_raw, dk), ('v_raw', v_raw, dv),
                       ('b_logit', b_logit, dk), ('w_logit', w_logit, dv)):
        _check(t, name, (B, T, H, d), dt, dev)
    _check(log_alpha, 'log_alpha', (B, T, H, dk), torch.float32, dev)
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.device != dev:
            raise ValueError('cu_seqlens must be a 1-D int32 tensor on the same device')
        if not cu_seqlens.is_contiguous():
            raise ValueError('cu_seqlens must be contiguous')
        N = cu_seqlens.numel() - 1
    else:
        N = B
    if S0 is not None:
        _check(S0, 'S0', (N, H, dk, dv), torch.float32, dev)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=torch.float32, device=dev)
    else:
        _check(out, 'out', (B, T, H, dv), torch.float32, dev)
    ST = None
    if final_state is not None:
        _check(final_state, 'final_state', (N, H, dk, dv), torch.float32, dev)
        ST = final_state
    elif output_final_state:
        ST = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    if conv_state_out is None and output_conv_state:
        conv_state_out = tuple(torch.empty((N, H, 3, d), dtype=dt, device=dev) for d in (dk, dk, dv))
    sc = _short_conv(H, dk, dv, dev, dt, N, conv_weight, conv_bias, conv_state, conv_state_out)
    varlen = cu_seqlens is not None
    need = _lib.gdn2_chunk_fwd_workspace_bytes(B, T, N, H, dk, dv, code, int(varlen))
    if need == 0:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, 'gdn2_chunk_fwd_workspace_bytes')
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    set_stream()
    st = _lib.gdn2_chunk_fwd_prologue(_ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(log_alpha), _ptr(b_logit),
                                      _ptr(w_logit), ctypes.byref(sc), _ptr(S0), _ptr(out), _ptr(ST),
                                      _ptr(cu_seqlens), B, T, N, H, dk, dv, code, GDN2_F32, _ptr(workspace),
                                      workspace.numel() * workspace.element_size())
    if st != GDN2_OK:
        raise Gdn2Error(st, 'gdn2_chunk_fwd_prologue')
    return out, ST, conv_state_out


def decode_step_prologue(q_raw: torch.Tensor, k_raw: torch.Tensor, v_raw: torch.Tensor, log_alpha: torch.Tensor,
                         b_logit: torch.Tensor, w_logit: torch.Tensor, S: torch.Tensor, conv_weight,
                         conv_bias=None, conv_state=None, *, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token per sequence on raw inputs ([N, H, d]), prologue fused in.
    S [N, H, dk, dv] float32 and the conv_state histories ((q, k, v) triple
    of [N, H, 3, d], or None for zeros) are updated in place. Returns o."""
    if q_raw.dim() != 3:
        raise ValueError('q_raw must be [N, H, dk]')
    N, H, dk = q_raw.shape
    dv = v_raw.shape[-1]
    dev, dt = q_raw.device, q_raw.dtype
    code = _dtype_code(q_raw)
    for name, t, d in (('q_raw', q_raw, dk), ('k_raw', k_raw, dk), ('v_raw', v_raw, dv),
                       ('b_logit', b_logit, dk), ('w_logit', w_logit, dv)):
        _check(t, name, (N, H, d), dt, dev)
    _check(log_alpha, 'log_alpha', (N, H, dk), torch.float32, dev)
    _check(S, 'S', (N, H, dk, dv), torch.float32, dev)
    if out is None:
        out = torch.empty((N, H, dv), dtype=torch.float32, device=dev)
    else:
        _check(out, 'out', (N, H, dv), torch.float32, dev)
    sc = _short_conv(H, dk, dv, dev, dt, N, conv_weight, conv_bias, conv_state, conv_state)
    set_stream()
    st = _lib.gdn2_decode_step_prologue(_ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(log_alpha), _ptr(b_logit),
                                        _ptr(w_logit), ctypes.byref(sc), _ptr(S), _ptr(out), N, H, dk, dv, code,
                                        GDN2_F32)
    if st != GDN2_OK:
        raise Gdn2Error(st, 'gdn2_decode_step_prologue')
    return out


def _seq_count(cu_seqlens, B, dev):
    if cu_seqlens is None:
        return B
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.device != dev:
        raise ValueError('cu_seqlens must be a 1-D int32 tensor on the same device')
    if not cu_seqlens.is_contiguous():
        raise ValueError('cu_seqlens must be contiguous')
    return cu_seqlens.numel() - 1


def bwd_workspace_bytes(B: int, T: int, N: int, H: int, dk: int, dv: int, dtype: torch.dtype, varlen: bool) -> int:
    """Device workspace of chunk_bwd, chunk_fwd_keep and chunk_bwd_kept."""
    code = GDN2_BF16 if dtype == torch.bfloat16 else GDN2_F32
    need = _lib.gdn2_chunk_bwd_workspace_bytes(B, T, N, H, dk, dv, code, int(varlen))
    if need == 0:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, 'gdn2_chunk_bwd_workspace_bytes')
    return need


def _bwd(fn: str, q, k, v, log_alpha, b, w, S0, dO, dST, cu_seqlens, workspace, need_workspace) -> dict:
    if q.dim() != 4:
        raise ValueError('q must be [B, T, H, dk]')
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    for name, t, d in (('q', q, dk), ('k', k, dk), ('v', v, dv), ('b', b, dk), ('w', w, dv)):
        _check(t, name, (B, T, H, d), dt, dev)
    _check(log_alpha, 'log_alpha', (B, T, H, dk), torch.float32, dev)
    _check(dO, 'dO', (B, T, H, dv), torch.float32, dev)
    N = _seq_count(cu_seqlens, B, dev)
    for name, t in (('S0', S0), ('dST', dST)):
        if t is not None:
            _check(t, name, (N, H, dk, dv), torch.float32, dev)
    g = {name: torch.empty((B, T, H, d), dtype=torch.float32, device=dev)
         for name, d in (('q', dk), ('k', dk), ('v', dv), ('log_alpha', dk), ('b', dk), ('w', dv))}
    g['S0'] = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    need = bwd_workspace_bytes(B, T, N, H, dk, dv, dt, cu_seqlens is not None)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        if need_workspace:
            raise ValueError(f'{fn}: pass the workspace of the matching chunk_fwd_keep ({need} bytes)')
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    set_stream()
    st = getattr(_lib, fn)(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0), _ptr(dO),
                           _ptr(dST), _ptr(cu_seqlens), B, T, N, H, dk, dv, code,
                           _ptr(g['q']), _ptr(g['k']), _ptr(g['v']), _ptr(g['log_alpha']), _ptr(g['b']),
                           _ptr(g['w']), _ptr(g['S0']), _ptr(workspace),
                           workspace.numel() * workspace.element_size())
    if st != GDN2_OK:
        raise Gdn2Error(st, fn)
    return g


def chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor,
              b: torch.Tensor, w: torch.Tensor, S0: Optional[torch.Tensor], dO: torch.Tensor,
              dST: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
              workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of a loss through ``chunk_fwd`` (per-channel gates): given
    dO = dL/do [B, T, H, dv] float32 and dST = dL/dS_T [N, H, dk, dv] (or
    None), returns float32 tensors {'q', 'k', 'v', 'log_alpha', 'b', 'w'}
    shaped like those inputs and 'S0' [N, H, dk, dv]."""
    return _bwd('gdn2_chunk_bwd', q, k, v, log_alpha, b, w, S0, dO, dST, cu_seqlens, workspace, False)


def chunk_fwd_keep(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor,
                   b: torch.Tensor, w: torch.Tensor, S0: Optional[torch.Tensor] = None,
                   cu_seqlens: Optional[torch.Tensor] = None, *,
                   workspace: Optional[torch.Tensor] = None):
    """The training forward (gdn2_chunk_fwd_keep): ``chunk_fwd`` with
    per-channel gates that also keeps, in the returned workspace, what
    ``chunk_bwd_kept`` needs. Returns (o [B, T, H, dv] float32,
    S_T [N, H, dk, dv] float32, workspace)."""
    if q.dim() != 4:
        raise ValueError('q must be [B, T, H, dk]')
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    for name, t, d in (('q', q, dk), ('k', k, dk), ('v', v, dv), ('b', b, dk), ('w', w, dv)):
        _check(t, name, (B, T, H, d), dt, dev)
    _check(log_alpha, 'log_alpha', (B, T, H, dk), torch.float32, dev)
    N = _seq_count(cu_seqlens, B, dev)
    if S0 is not None:
        _check(S0, 'S0', (N, H, dk, dv), torch.float32, dev)
    o = torch.empty((B, T, H, dv), dtype=torch.float32, device=dev)
    ST = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    need = bwd_workspace_bytes(B, T, N, H, dk, dv, dt, cu_seqlens is not None)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    set_stream()
    st = _lib.gdn2_chunk_fwd_keep(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0), _ptr(o),
                                  _ptr(ST), _ptr(cu_seqlens), B, T, N, H, dk, dv, code, GDN2_F32, _ptr(workspace),
                                  workspace.numel() * workspace.element_size())
    if st != GDN2_OK:
        raise Gdn2Error(st, 'gdn2_chunk_fwd_keep')
    return o, ST, workspace


def chunk_bwd_kept(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor,
                   b: torch.Tensor, w: torch.Tensor, S0: Optional[torch.Tensor], dO: torch.Tensor,
                   dST: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
                   workspace: torch.Tensor) -> dict:
    """``chunk_bwd`` from what the last ``chunk_fwd_keep`` on the same inputs
    left in ``workspace`` (gdn2_chunk_bwd_kept): the same gradients without
    running the forward again."""
    return _bwd('gdn2_chunk_bwd_kept', q, k, v, log_alpha, b, w, S0, dO, dST, cu_seqlens, workspace, True)


# ---- operators around the mixer: the recurrence on state slots, the prologue
# and the closing layer norm. Their tensors live on one GPU, which need not be
# the current one; work goes to that GPU's current stream.

_CODES = {torch.float32: GDN2_F32, torch.bfloat16: GDN2_BF16}


def _gpu(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f'{name}: must be on the GPU, got {t.device}')
    return t.device


def _need(t: torch.Tensor, name: str, shape, dtype, device):
    """_check, with its messages, at the cost of one comparison each where all is well."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _check(t, name, shape, dtype, device)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


_data_ptr = torch.Tensor.data_ptr


# The current stream's handle: current_stream() builds a Stream object around
# it, most of the host's time of a small call (1.9 of 12 us).
_raw_stream = getattr(torch._C, '_cuda_getCurrentRawStream', None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, where: str, dev: torch.device, *args) -> None:
    """Call the library on ``dev``'s current stream, with ``dev`` current."""
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return _call(fn, where, dev, *args)
    _lib.gdn2_set_stream(_raw_stream(dev.index))
    st = fn(*args)
    if st != GDN2_OK:
        raise Gdn2Error(st, where)


def _index(t: Optional[torch.Tensor], name: str, n: int, dev):
    if t is not None:
        _need(t, name, (n,), torch.int32, dev)


def _gate(t: torch.Tensor, name: str, shape, dtype, dev, bit: int) -> int:
    """Layout bit of a gate: 0 with its channel axis, ``bit`` without."""
    if t.dim() == len(shape):
        _need(t, name, shape, dtype, dev)
        return 0
    _need(t, name, shape[:-1], dtype, dev)
    return bit


def _heads(q, k, v, cu_seqlens, names):
    """Sizes from q, k [B, T, HK, dk] and v [B, T, H, dv], checked."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError(f'{names[0]} and {names[2]} must be [B, T, heads, d]')
    dev, dt = _gpu(q, names[0]), q.dtype
    _dtype_code(q)
    B, T, HK, dk = q.shape
    H, dv = v.shape[2:]
    _need(k, names[1], q.shape, dt, dev)
    if not q.is_contiguous():
        raise ValueError(f'{names[0]}: must be contiguous')
    _need(v, names[2], (B, T, H, dv), dt, dev)
    if HK < 1 or H % HK:
        raise ValueError(f'{names[2]}: its {H} heads are not a multiple of the {HK} of {names[0]}')
    return dev, dt, B, T, _seq_count(cu_seqlens, B, dev), H, HK, dk, dv


def recurrent_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor, b: torch.Tensor,
                  w: torch.Tensor, state: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, *,
                  slot_in: Optional[torch.Tensor] = None, slot_out: Optional[torch.Tensor] = None,
                  commit: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The recurrence token by token over short sequences, their states in a pool
    (gdn2_recurrent_fwd): continuous batching, draft tokens, short prompts.

    q, k: [B, T, HK, dk]; v: [B, T, H, dv] (bf16 or fp32; HK divides H, head h
    uses q/k head h // (H // HK)); b, log_alpha: [B, T, H, dk] and w:
    [B, T, H, dv], or [B, T, H] for one gate per token-head (log_alpha fp32).
    With ``cu_seqlens`` B is 1 and the sequences are packed along T.
    state: [slots, H, dk, dv] fp32, updated in place. slot_in, slot_out, commit:
    int32 [N] on the device, as gdn2.h has them (slot numbers outside the pool:
    zeros in, not kept; commit: leading tokens whose effect is kept). Returns
    o [B, T, H, dv] in ``out_dtype`` (fp32 or bf16)."""
    dev, dt, B, T, N, H, HK, dk, dv = _heads(q, k, v, cu_seqlens, ('q', 'k', 'v'))
    lead = (B, T, H)
    gates = (_gate(b, 'b', (*lead, dk), dt, dev, GDN2_GATE_B_PER_HEAD)
             | _gate(w, 'w', (*lead, dv), dt, dev, GDN2_GATE_W_PER_HEAD)
             | _gate(log_alpha, 'log_alpha', (*lead, dk), torch.float32, dev, GDN2_GATE_ALPHA_PER_HEAD))
    if state.dim() != 4:
        raise ValueError('state must be [slots, H, dk, dv]')
    slots = state.shape[0]
    _need(state, 'state', (slots, H, dk, dv), torch.float32, dev)
    _index(slot_in, 'slot_in', N, dev)
    _index(slot_out, 'slot_out', N, dev)
    _index(commit, 'commit', N, dev)
    if slot_in is None and slots < N:
        raise ValueError(f'state: {slots} slots for {N} sequences (pass slot_in)')
    if out is None:
        if out_dtype not in _CODES:
            raise TypeError(f'unsupported output dtype {out_dtype} (bfloat16 or float32)')
        out = torch.empty((B, T, H, dv), dtype=out_dtype, device=dev)
    else:
        if out.dtype not in _CODES:
            raise TypeError(f'unsupported output dtype {out.dtype} (bfloat16 or float32)')
        _need(out, 'out', (B, T, H, dv), out.dtype, dev)
    _call(_lib.gdn2_recurrent_fwd, 'gdn2_recurrent_fwd', dev, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          log_alpha.data_ptr(), b.data_ptr(), w.data_ptr(), gates, state.data_ptr(), _addr(slot_in), _addr(slot_out),
          _addr(commit), out.data_ptr(), _addr(cu_seqlens), B, T, N, H, HK, slots, dk, dv, _CODES[dt],
          _CODES[out.dtype])
    return out


def _conv_pools(conv_weight, conv_bias, conv_state, conv_state_out, heads, dims, dt, dev):
    """ShortConv of a prologue call whose histories are pools, and their slots."""
    if conv_weight is None or len(conv_weight) != 3:
        raise ValueError('conv_weight must be a (q, k, v) triple of [heads*d, 4] float32 tensors')
    addr = [None] * 12   # the struct's fields in order
    slots, f32 = 0, torch.float32
    for z, (t, h, d) in enumerate(zip(conv_weight, heads, dims)):
        if t is None:
            raise ValueError('conv_weight: none of the triple may be None')
        _need(t, 'conv_weight', (h * d, 4), f32, dev)
        addr[z] = t.data_ptr()
    if conv_bias is not None:
        if len(conv_bias) != 3:
            raise ValueError('conv_bias must be a (q, k, v) triple')
        for z, (t, h, d) in enumerate(zip(conv_bias, heads, dims)):
            if t is not None:
                _need(t, 'conv_bias', (h * d,), f32, dev)
                addr[3 + z] = t.data_ptr()
    for at, trip in ((6, conv_state), (9, conv_state_out)):
        if trip is None:
            continue
        if len(trip) != 3:
            raise ValueError('conv_state must be a (q, k, v) triple')
        if at == 9 and trip is conv_state:
            addr[9:] = addr[6:9]
            continue
        for z, (t, h, d) in enumerate(zip(trip, heads, dims)):
            if t is None:
                raise ValueError('conv_state: all three of the triple or none (None instead of it)')
            slots = slots or (t.shape[0] if t.dim() else 0)
            _need(t, 'conv_state', (slots, h, 3, d), dt, dev)
            addr[at + z] = t.data_ptr()
    return ShortConv(*addr), slots


def _prologue_sizes(q_raw, k_raw, v_raw, b_logit, w_logit, cu_seqlens):
    dev, dt, B, T, N, H, HK, dk, dv = _heads(q_raw, k_raw, v_raw, cu_seqlens, ('q_raw', 'k_raw', 'v_raw'))
    gates = (_gate(b_logit, 'b_logit', (B, T, H, dk), dt, dev, GDN2_GATE_B_PER_HEAD)
             | _gate(w_logit, 'w_logit', (B, T, H, dv), dt, dev, GDN2_GATE_W_PER_HEAD))
    return dev, dt, gates, B, T, N, H, HK, dk, dv


def prologue_fwd(q_raw: torch.Tensor, k_raw: torch.Tensor, v_raw: torch.Tensor, b_logit: torch.Tensor,
                 w_logit: torch.Tensor, conv_weight, conv_bias=None, cu_seqlens: Optional[torch.Tensor] = None, *,
                 conv_state=None, conv_state_out=None, slot_in: Optional[torch.Tensor] = None,
                 slot_out: Optional[torch.Tensor] = None, commit: Optional[torch.Tensor] = None, out=None):
    """The mixer's inputs from the layer's projections (gdn2_prologue_fwd): q and
    k through their short convolutions and to unit norm, v through its own,
    b and w through the sigmoid.

    q_raw, k_raw: [B, T, HK, dk]; v_raw: [B, T, H, dv]; b_logit: [B, T, H, dk] or
    [B, T, H]; w_logit: [B, T, H, dv] or [B, T, H]. conv_weight, conv_bias as in
    ``chunk_fwd_prologue`` (q and k: HK*dk channels). conv_state,
    conv_state_out: (q, k, v) pools of histories, [slots, HK, 3, dk] twice and
    [slots, H, 3, dv], or None for zeros / not written; conv_state_out may be
    conv_state itself. slot_in, slot_out, commit as in ``recurrent_fwd``. out:
    five tensors to write (b and w may be their own logits), or None. Returns (q, k, v, b, w) in the input dtype."""
    dev, dt, gates, B, T, N, H, HK, dk, dv = _prologue_sizes(q_raw, k_raw, v_raw, b_logit, w_logit, cu_seqlens)
    sc, slots = _conv_pools(conv_weight, conv_bias, conv_state, conv_state_out, (HK, HK, H), (dk, dk, dv), dt, dev)
    _index(slot_in, 'slot_in', N, dev)
    _index(slot_out, 'slot_out', N, dev)
    _index(commit, 'commit', N, dev)
    if slots and slot_in is None and slots < N:
        raise ValueError(f'conv_state: {slots} slots for {N} sequences (pass slot_in)')
    raw = (q_raw, k_raw, v_raw, b_logit, w_logit)
    if out is None:
        out = tuple(map(torch.empty_like, raw))
    else:
        if len(out) != 5:
            raise ValueError('out must be (q, k, v, b, w)')
        for n, t, x in zip('qkvbw', out, raw):
            _need(t, f'out[{n}]', x.shape, dt, dev)
    _call(_lib.gdn2_prologue_fwd, 'gdn2_prologue_fwd', dev, *map(_data_ptr, raw), gates, ctypes.byref(sc),
          _addr(slot_in), _addr(slot_out), _addr(commit), *map(_data_ptr, out), _addr(cu_seqlens), B, T, N, H,
          HK, slots, dk, dv, _CODES[dt])
    return tuple(out)


def prologue_bwd(q_raw: torch.Tensor, k_raw: torch.Tensor, v_raw: torch.Tensor, b_logit: torch.Tensor,
                 w_logit: torch.Tensor, conv_weight, conv_bias, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor,
                 db: torch.Tensor, dw: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, *, conv_state=None,
                 slot_in: Optional[torch.Tensor] = None, grad_dtype: Optional[torch.dtype] = None,
                 workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradient of ``prologue_fwd`` (gdn2_prologue_bwd) from dq, dk, dv, db, dw,
    fp32 and shaped like q, k, v, b, w (what ``chunk_bwd`` returns). Returns
    {'q_raw', 'k_raw', 'v_raw', 'b_logit', 'w_logit'} in ``grad_dtype`` (None:
    the inputs'), fp32 {'weight_q', 'weight_k', 'weight_v'} [heads*d, 4] and
    'bias_q', 'bias_k', 'bias_v' for the biases that conv_bias holds."""
    dev, dt, gates, B, T, N, H, HK, Dk, Dv = _prologue_sizes(q_raw, k_raw, v_raw, b_logit, w_logit, cu_seqlens)
    heads, dims = (HK, HK, H), (Dk, Dk, Dv)
    sc, slots = _conv_pools(conv_weight, conv_bias, conv_state, None, heads, dims, dt, dev)
    _index(slot_in, 'slot_in', N, dev)
    if slots and slot_in is None and slots < N:
        raise ValueError(f'conv_state: {slots} slots for {N} sequences (pass slot_in)')
    raw, grads = (q_raw, k_raw, v_raw, b_logit, w_logit), (dq, dk, dv, db, dw)
    for n, t, x in zip(('dq', 'dk', 'dv', 'db', 'dw'), grads, raw):
        _need(t, n, x.shape, torch.float32, dev)
    grad_dtype = dt if grad_dtype is None else grad_dtype
    if grad_dtype not in _CODES:
        raise TypeError(f'unsupported gradient dtype {grad_dtype} (bfloat16 or float32)')
    like = raw if grad_dtype is dt else grads if grad_dtype is torch.float32 else None
    if like is None:
        like = [torch.empty(x.shape, dtype=grad_dtype, device=dev) for x in raw]
    outs = tuple(map(torch.empty_like, like))
    g = dict(zip(('q_raw', 'k_raw', 'v_raw', 'b_logit', 'w_logit'), outs))
    taps = tuple(map(torch.empty_like, conv_weight))
    g.update(zip(('weight_q', 'weight_k', 'weight_v'), taps))
    if conv_bias is not None:
        for n, x in zip(('bias_q', 'bias_k', 'bias_v'), conv_bias):
            if x is not None:
                g[n] = torch.empty_like(x)
    need = _lib.gdn2_prologue_bwd_workspace_bytes(B, T, N, H, HK, Dk, Dv, int(cu_seqlens is not None))
    if need == 0:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, 'gdn2_prologue_bwd_workspace_bytes')
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f'workspace: must be contiguous on {dev}')
    _call(_lib.gdn2_prologue_bwd, 'gdn2_prologue_bwd', dev, *map(_data_ptr, raw), gates, ctypes.byref(sc),
          _addr(slot_in), *map(_data_ptr, grads), *map(_data_ptr, outs), *map(_data_ptr, taps),
          _addr(g.get('bias_q')), _addr(g.get('bias_k')), _addr(g.get('bias_v')), _addr(cu_seqlens), B, T, N, H, HK, slots, Dk, Dv, _CODES[dt], _CODES[grad_dtype], workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return g


def layer_norm_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   residual: Optional[torch.Tensor] = None, *, eps: float = 1e-5, output_sum: bool = False,
                   out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None):
    """LayerNorm(x + residual) over the last axis (gdn2_layer_norm_fwd). x,
    residual: [..., cols], one dtype (bf16 or fp32); weight, bias: [cols] fp32.
    Returns (y in ``out_dtype`` (None: x's), h or None): h = x + residual, what
    ``layer_norm_bwd`` takes, with ``output_sum`` or into ``sum_out`` (which,
    like ``out``, may be x or residual itself)."""
    dev, dt, shape = _gpu(x, 'x'), x.dtype, x.shape
    _dtype_code(x)
    if x.dim() < 1 or shape[-1] < 1:
        raise ValueError('x must be [..., cols] with cols >= 1')
    cols = shape[-1]
    if not x.is_contiguous():
        raise ValueError('x: must be contiguous')
    _need(weight, 'weight', (cols,), torch.float32, dev)
    if bias is not None:
        _need(bias, 'bias', (cols,), torch.float32, dev)
    if residual is not None:
        _need(residual, 'residual', shape, dt, dev)
    if sum_out is not None:
        _need(sum_out, 'sum_out', shape, dt, dev)
    elif output_sum:
        sum_out = torch.empty_like(x)
    out_dtype = out.dtype if out is not None else (dt if out_dtype is None else out_dtype)
    if out_dtype not in _CODES:
        raise TypeError(f'unsupported output dtype {out_dtype} (bfloat16 or float32)')
    if out is None:
        out = torch.empty_like(x) if out_dtype is dt else torch.empty(shape, dtype=out_dtype, device=dev)
    else:
        _need(out, 'out', shape, out_dtype, dev)
    _call(_lib.gdn2_layer_norm_fwd, 'gdn2_layer_norm_fwd', dev, x.data_ptr(), _addr(residual), weight.data_ptr(),
          _addr(bias), out.data_ptr(), _addr(sum_out), x.numel() // cols, cols, eps, _CODES[dt], _CODES[out_dtype])
    return out, sum_out


def layer_norm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, *, dsum: Optional[torch.Tensor] = None,
                   eps: float = 1e-5, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradient of ``layer_norm_fwd`` (gdn2_layer_norm_bwd). h: [..., cols], the
    sum the forward returned (x where there was no residual); dy: shaped like
    it, bf16 or fp32; dsum: a further gradient of h, added on. Returns
    {'x': dL/dh (of x and of residual alike) in h's dtype, 'weight', 'bias':
    fp32 [cols]}."""
    dev, dt, shape = _gpu(h, 'h'), h.dtype, h.shape
    _dtype_code(h)
    if h.dim() < 1 or shape[-1] < 1:
        raise ValueError('h must be [..., cols] with cols >= 1')
    cols = shape[-1]
    rows = h.numel() // cols
    if dy.dtype not in _CODES:
        raise TypeError(f'unsupported gradient dtype {dy.dtype} (bfloat16 or float32)')
    if not h.is_contiguous():
        raise ValueError('h: must be contiguous')
    _need(dy, 'dy', shape, dy.dtype, dev)
    _need(weight, 'weight', (cols,), torch.float32, dev)
    if dsum is not None:
        _need(dsum, 'dsum', shape, dt, dev)
    if out is None:
        out = torch.empty_like(h)
    else:
        _need(out, 'out', shape, dt, dev)
    g = {'x': out, 'weight': torch.empty_like(weight), 'bias': torch.empty_like(weight)}
    need = _lib.gdn2_layer_norm_bwd_workspace_bytes(rows, cols)
    if need == 0:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, 'gdn2_layer_norm_bwd_workspace_bytes')
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f'workspace: must be contiguous on {dev}')
    _call(_lib.gdn2_layer_norm_bwd, 'gdn2_layer_norm_bwd', dev, dy.data_ptr(), h.data_ptr(), weight.data_ptr(),
          _addr(dsum), out.data_ptr(), g['weight'].data_ptr(), g['bias'].data_ptr(), rows, cols, eps, _CODES[dt],
          _CODES[dy.dtype], workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return g


# ---- the layer's dense half: projections, the norm before them, the clipping of their gradients

_E4M3 = torch.float8_e4m3fn


def _act_code(activation) -> int:
    code = ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f'unsupported activation {activation!r} (one of {[a for a in ACTIVATIONS if a]})')
    return code


def _linear_sizes(x, weight, name='x'):
    """Device, dtype, leading shape, rows, in_features and out_features of a linear layer, checked."""
    dev, dt = _gpu(x, name), x.dtype
    if x.dim() < 1 or weight.dim() != 2 or weight.shape[0] < 1 or weight.shape[1] < 1:
        raise ValueError(f'{name} must be [..., in_features] and weight [out_features, in_features], of one at least')
    N, K = weight.shape
    lead = x.shape[:-1]
    if x.shape[-1] != K:
        raise ValueError(f'{name}: expected {K} in_features, got {x.shape[-1]}')
    if not x.is_contiguous():
        raise ValueError(f'{name}: must be contiguous')
    _need(weight, 'weight', (N, K), dt, dev)
    return dev, dt, lead, x.numel() // K, K, N


def linear_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               residual: Optional[torch.Tensor] = None, *, activation: Optional[str] = None,
               x_scale: Optional[torch.Tensor] = None, weight_scale: Optional[torch.Tensor] = None,
               out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None, output_preact: bool = False,
               preact_out: Optional[torch.Tensor] = None):
    """act(x weight^T + bias) + residual (gdn2_linear_fwd). x: [..., in_features],
    weight: [out_features, in_features], one dtype: bf16, fp32, or float8_e4m3fn
    with fp32 x_scale ([...], x's leading shape) and weight_scale [out_features],
    which multiply the product (large ones to bf16 are added with fewer bits than
    fp32's, see gdn2.h; to fp32 they are not). bias: [out_features] fp32. residual:
    [..., out_features] in the output's dtype. activation: None, 'sigmoid',
    'silu' or 'gelu_tanh'. Returns (y in ``out_dtype`` (None: x's; bf16 for 8 bits),
    z or None): z, the activation's argument in x's dtype, is what ``linear_bwd``
    takes, with ``output_preact`` or into ``preact_out``. ``out`` may be the residual."""
    dev, dt, lead, M, K, N = _linear_sizes(x, weight)
    act = _act_code(activation)
    e4m3 = dt is _E4M3
    if not e4m3:
        _dtype_code(x)
        if x_scale is not None or weight_scale is not None:
            raise ValueError('x_scale and weight_scale: only with float8_e4m3fn operands')
    else:
        if x_scale is None or weight_scale is None:
            raise ValueError('float8_e4m3fn operands need x_scale and weight_scale')
        _need(x_scale, 'x_scale', lead, torch.float32, dev)
        _need(weight_scale, 'weight_scale', (N,), torch.float32, dev)
        if output_preact or preact_out is not None:
            raise ValueError('preact: not with float8_e4m3fn operands')
    out_dtype = out.dtype if out is not None else (torch.bfloat16 if e4m3 else dt) if out_dtype is None else out_dtype
    if out_dtype not in _CODES:
        raise TypeError(f'unsupported output dtype {out_dtype} (bfloat16 or float32)')
    shape = (*lead, N)
    if bias is not None:
        _need(bias, 'bias', (N,), torch.float32, dev)
    if residual is not None:
        _need(residual, 'residual', shape, out_dtype, dev)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=dev)
    else:
        _need(out, 'out', shape, out_dtype, dev)
    if preact_out is not None:
        _need(preact_out, 'preact_out', shape, dt, dev)
    elif output_preact:
        preact_out = torch.empty(shape, dtype=dt, device=dev)
    _call(_lib.gdn2_linear_fwd, 'gdn2_linear_fwd', dev, x.data_ptr(), weight.data_ptr(), _addr(bias), _addr(residual),
          _addr(x_scale), _addr(weight_scale), out.data_ptr(), _addr(preact_out), M, K, N, act,
          GDN2_E4M3 if e4m3 else _CODES[dt], _CODES[out_dtype])
    return out, preact_out


def linear_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, preact: Optional[torch.Tensor] = None, *,
               activation: Optional[str] = None, output_x: bool = True, output_weight: bool = True,
               output_bias: bool = True, workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradient of ``linear_fwd`` (gdn2_linear_bwd) from dy: [..., out_features]
    (bf16 or fp32, the forward's output dtype), x, weight and, with an
    activation, the z that the forward returned. Returns {'x': dL/dx, 'weight':
    dL/dweight} in x's dtype (bf16 or fp32) and {'bias': fp32}, each if its
    flag is set. The residual's gradient is dy itself."""
    dev, dt, lead, M, K, N = _linear_sizes(x, weight)
    _dtype_code(x)
    act = _act_code(activation)
    shape = (*lead, N)
    if dy.dtype not in _CODES:
        raise TypeError(f'unsupported gradient dtype {dy.dtype} (bfloat16 or float32)')
    _need(dy, 'dy', shape, dy.dtype, dev)
    if act and preact is None:
        raise ValueError(f'preact: {activation} needs what linear_fwd returned')
    if preact is not None:
        _need(preact, 'preact', shape, dt, dev)
    if not (output_x or output_weight or output_bias):
        raise ValueError('none of the gradients is wanted')
    g = {}
    if output_x:
        g['x'] = torch.empty_like(x)
    if output_weight:
        g['weight'] = torch.empty_like(weight)
    if output_bias:
        g['bias'] = torch.empty(N, dtype=torch.float32, device=dev)
    codes = _CODES[dt], _CODES[dy.dtype]
    need = _lib.gdn2_linear_bwd_workspace_bytes(M, K, N, act, *codes, output_x, output_weight, output_bias)
    if need == 0:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, 'gdn2_linear_bwd_workspace_bytes')
    workspace = _workspace(workspace, need, dev)
    _call(_lib.gdn2_linear_bwd, 'gdn2_linear_bwd', dev, dy.data_ptr(), x.data_ptr(), weight.data_ptr(), _addr(preact),
          _addr(g.get('x')), _addr(g.get('weight')), _addr(g.get('bias')), M, K, N, act, *codes, workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return g


def _workspace(workspace: Optional[torch.Tensor], need: int, dev) -> torch.Tensor:
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f'workspace: must be contiguous on {dev}')
    return workspace


def rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
                 output_sum: bool = False, out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None,
                 scale_out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None):
    """RMS norm of x + residual over the last axis (gdn2_rms_norm_fwd). x,
    residual: [..., cols], one dtype (bf16 or fp32); weight: [cols] fp32. Returns
    (y, h or None, scale or None): y in ``out_dtype`` (None: x's; bf16, fp32 or
    float8_e4m3fn); h = x + residual, what ``rms_norm_bwd`` takes, with
    ``output_sum`` or into ``sum_out``; scale: [...] fp32, with float8_e4m3fn
    alone: y times its row's scale is the norm, and ``linear_fwd`` takes both.
    ``out`` (same dtype) and ``sum_out`` may be x or residual itself."""
    dev, dt, shape = _gpu(x, 'x'), x.dtype, x.shape
    _dtype_code(x)
    if x.dim() < 1 or shape[-1] < 1:
        raise ValueError('x must be [..., cols] with cols >= 1')
    cols = shape[-1]
    if not x.is_contiguous():
        raise ValueError('x: must be contiguous')
    _need(weight, 'weight', (cols,), torch.float32, dev)
    if residual is not None:
        _need(residual, 'residual', shape, dt, dev)
    if sum_out is not None:
        _need(sum_out, 'sum_out', shape, dt, dev)
    elif output_sum:
        sum_out = torch.empty_like(x)
    out_dtype = out.dtype if out is not None else (dt if out_dtype is None else out_dtype)
    e4m3 = out_dtype is _E4M3
    if not e4m3 and out_dtype not in _CODES:
        raise TypeError(f'unsupported output dtype {out_dtype} (bfloat16, float32 or float8_e4m3fn)')
    if out is None:
        out = torch.empty_like(x) if out_dtype is dt else torch.empty(shape, dtype=out_dtype, device=dev)
    else:
        _need(out, 'out', shape, out_dtype, dev)
    if scale_out is not None:
        if not e4m3:
            raise ValueError('scale_out: only with a float8_e4m3fn output')
        _need(scale_out, 'scale_out', shape[:-1], torch.float32, dev)
    elif e4m3:
        scale_out = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    _call(_lib.gdn2_rms_norm_fwd, 'gdn2_rms_norm_fwd', dev, x.data_ptr(), _addr(residual), weight.data_ptr(),
          out.data_ptr(), _addr(scale_out), _addr(sum_out), x.numel() // cols, cols, eps, _CODES[dt],
          GDN2_E4M3 if e4m3 else _CODES[out_dtype])
    return out, sum_out, scale_out


def rms_norm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, *, dsum: Optional[torch.Tensor] = None,
                 eps: float = 1e-5, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradient of ``rms_norm_fwd`` (gdn2_rms_norm_bwd). h: [..., cols], the sum
    the forward returned (x where there was no residual); dy: shaped like it,
    bf16 or fp32; dsum: a further gradient of h, added on. Returns {'x': dL/dh (of
    x and of residual alike) in h's dtype, 'weight': fp32 [cols]}."""
    dev, dt, shape = _gpu(h, 'h'), h.dtype, h.shape
    _dtype_code(h)
    if h.dim() < 1 or shape[-1] < 1:
        raise ValueError('h must be [..., cols] with cols >= 1')
    cols = shape[-1]
    rows = h.numel() // cols
    if dy.dtype not in _CODES:
        raise TypeError(f'unsupported gradient dtype {dy.dtype} (bfloat16 or float32)')
    if not h.is_contiguous():
        raise ValueError('h: must be contiguous')
    _need(dy, 'dy', shape, dy.dtype, dev)
    _need(weight, 'weight', (cols,), torch.float32, dev)
    if dsum is not None:
        _need(dsum, 'dsum', shape, dt, dev)
    if out is None:
        out = torch.empty_like(h)
    else:
        _need(out, 'out', shape, dt, dev)
    g = {'x': out, 'weight': torch.empty_like(weight)}
    need = _lib.gdn2_rms_norm_bwd_workspace_bytes(rows, cols)
    if need == 0:
        raise Gdn2Error(GDN2_ERR_UNSUPPORTED, 'gdn2_rms_norm_bwd_workspace_bytes')
    workspace = _workspace(workspace, need, dev)
    _call(_lib.gdn2_rms_norm_bwd, 'gdn2_rms_norm_bwd', dev, dy.data_ptr(), h.data_ptr(), weight.data_ptr(), _addr(dsum),
          out.data_ptr(), g['weight'].data_ptr(), rows, cols, eps, _CODES[dt], _CODES[dy.dtype], workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return g


def _tensor_list(tensors, name):
    """Addresses, element counts and dtype codes of tensors on one GPU, as ctypes arrays."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError(f'{name}: no tensors')
    n, dev = len(tensors), _gpu(tensors[0], name)
    types = [_CODES.get(t.dtype) for t in tensors]
    if None in types:
        i = types.index(None)
        raise TypeError(f'{name}[{i}]: unsupported dtype {tensors[i].dtype} (bfloat16 or float32)')
    for i, t in enumerate(tensors):
        if t.device != dev:
            raise ValueError(f'{name}[{i}]: expected device {dev}, got {t.device}')
        if not t.is_contiguous():
            raise ValueError(f'{name}[{i}]: must be contiguous')
    return (tensors, dev, (ctypes.c_void_p * n)(*map(_data_ptr, tensors)), (ctypes.c_int64 * n)(*map(torch.Tensor.numel, tensors)),
            (ctypes.c_int32 * n)(*types))


def grad_norm(grads, *, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The norm over all elements of a list of bf16 and fp32 tensors on one GPU
    (gdn2_grad_norm), an fp32 tensor without axes."""
    _, dev, ptrs, sizes, types = _tensor_list(grads, 'grads')
    norm = torch.empty((), dtype=torch.float32, device=dev)
    workspace = _workspace(workspace, _lib.gdn2_clip_grads_workspace_bytes(), dev)
    _call(_lib.gdn2_grad_norm, 'gdn2_grad_norm', dev, ptrs, sizes, types, len(sizes), norm.data_ptr(),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return norm


def clip_grads(grads, max_norm: float, *, out=None, norm: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Scale a list of bf16 and fp32 tensors on one GPU by min(1, max_norm / (norm +
    1e-6)), in place or into the tensors of ``out`` (same shapes, bf16 or fp32;
    each may be its gradient itself, none may overlap another)
    (gdn2_clip_grads). norm: the global norm to go by, an fp32 tensor of one element on the
    device (a norm over several devices' parts, say), or None for that of
    ``grads``. Returns the norm."""
    grads, dev, ptrs, sizes, types = _tensor_list(grads, 'grads')
    optrs, otypes = ptrs, types
    if out is not None:
        out, odev, optrs, osizes, otypes = _tensor_list(out, 'out')
        if len(out) != len(grads) or odev != dev:
            raise ValueError(f'out: expected {len(grads)} tensors on {dev}, got {len(out)} on {odev}')
        for i, (t, o) in enumerate(zip(grads, out)):
            if t.shape != o.shape:
                raise ValueError(f'out[{i}]: expected shape {tuple(t.shape)}, got {tuple(o.shape)}')
    given = norm is not None
    if given:
        if norm.numel() != 1 or norm.dtype != torch.float32 or norm.device != dev:
            raise ValueError(f'norm: expected one float32 on {dev}')
    else:
        norm = torch.empty((), dtype=torch.float32, device=dev)
        workspace = _workspace(workspace, _lib.gdn2_clip_grads_workspace_bytes(), dev)
    _call(_lib.gdn2_clip_grads, 'gdn2_clip_grads', dev, ptrs, optrs, sizes, types, otypes, len(grads), max_norm,
          norm.data_ptr(), given, None if given else workspace.data_ptr(),
          0 if given else workspace.numel() * workspace.element_size())
    return norm
