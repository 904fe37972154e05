"""Python binding of linear attention with a decay for each head (argument marshalling only, as
``api``): the chunked forward and backward and the single-token step.

Layouts: q, k are bf16 ``[T_total, Hk, D]`` and v, dO ``[T_total, H, D]`` (packed sequences through
``cu_seqlens``, int64 ``[N + 1]``) or dense ``[B, T, H, D]``; q, k and v may be columns of a wider
tensor (tokens of one stride).  ``log_decay`` is float32 ``[H]``, states float32 ``[N, H, D, D]``
(row = key channel).  The step takes ``[rows, H, D]`` and a pool of states, with ``slots`` (int64
``[rows]``) naming each row's state and a negative slot marking a padded row.
"""
import ctypes

import torch

from .api import _check, lib
from .block import _need, _opt, _pool, _ptr, _scratch, _stream


class DlaShape(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int64), ("num_heads", ctypes.c_int32),
                ("num_k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("cu_seqlens", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        L = lib()
        vp, sz, i32, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        sp, st = ctypes.POINTER(DlaShape), ctypes.c_int
        for name, res, args in (
                ("dla_workspace_bytes", sz, [sp, i32]),
                ("dla_fwd", st, [sp] + [vp] * 8 + [sz, vp]),
                ("dla_bwd", st, [sp] + [vp] * 8 + [sz] + [vp] * 5),
                ("dla_step", st, [i32] * 5 + [f32] + [vp, i64] * 3 + [vp] * 5)):
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _LIB = L
    return _LIB


def _tokens(t, shape, name):
    """A bf16 tensor [..., heads, D] of tokens of one stride (columns of a wider tensor are fine); returns the stride."""
    if t is None or t.dtype is not torch.bfloat16 or t.shape != shape or not t.is_cuda:
        if t is None:
            raise ValueError("%s is required" % name)
        raise ValueError("%s must be a CUDA bfloat16 tensor of shape %s (got %s %s %s)"
                         % (name, tuple(shape), t.device, t.dtype, tuple(t.shape)))
    heads, D = shape[-2:]
    if t.is_contiguous():
        return heads * D
    st = t.stride()
    many = [i for i in range(len(shape) - 2) if shape[i] > 1]  # strides of single tokens mean nothing
    ld = st[many[-1]] if many else heads * D
    if st[-1] != 1 or (heads > 1 and st[-2] != D) or ld < heads * D or (len(many) == 2 and st[0] != shape[1] * ld):
        raise ValueError("%s must consist of tokens of one stride (got strides %s for shape %s)" % (name, st, tuple(shape)))
    return ld


class _Call:
    """Shape of one call: value heads from v, q / k heads from q."""

    def __init__(self, q, k, v, log_decay, cu_seqlens, num_seqs, scale):
        if q is None or v is None or q.dim() not in (3, 4) or v.dim() != q.dim():
            raise ValueError("q and v must be [T_total, heads, D] or [B, T, heads, D]")
        self.H, self.D, self.Hk = v.shape[-2], v.shape[-1], q.shape[-2]
        self.vshape, self.qshape = v.shape, v.shape[:-2] + (self.Hk, self.D)
        if v.dim() == 4:
            if cu_seqlens is not None:
                raise ValueError("cu_seqlens goes with packed [T_total, heads, D] tensors")
            self.N, self.T = v.shape[0], v.shape[0] * v.shape[1]
        else:
            self.T = v.shape[0]
            self.N = (1 if num_seqs is None else int(num_seqs)) if cu_seqlens is None else cu_seqlens.numel() - 1
        if cu_seqlens is not None:
            _need(cu_seqlens, torch.int64, (self.N + 1,), "cu_seqlens")
        _need(log_decay, torch.float32, (self.H,), "log_decay")
        self.cu, self.states = cu_seqlens, (self.N, self.H, self.D, self.D)
        self.shape = DlaShape(self.N, self.T, self.H, self.Hk, self.D, _ptr(cu_seqlens),
                              self.D ** -0.5 if scale is None else scale, _tokens(q, self.qshape, "q"),
                              _tokens(k, self.qshape, "k"), _tokens(v, self.vshape, "v"))


def dla_workspace_bytes(q, k, v, log_decay, cu_seqlens=None, num_seqs=None, backward=False):
    """Bytes of the workspace of dla_fwd / dla_bwd for these tensors."""
    return int(_lib().dla_workspace_bytes(_Call(q, k, v, log_decay, cu_seqlens, num_seqs, None).shape, bool(backward)))


def dla_fwd(q, k, v, log_decay, h0=None, cu_seqlens=None, num_seqs=None, scale=None, want_ht=True, workspace=None):
    """Linear attention with a decay for each head: S_t = e^log_decay S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t
    (scale None: D^-1/2).  Returns dict(o, ht): the output and (None without ``want_ht``) the states after the
    sequences."""
    P = _Call(q, k, v, log_decay, cu_seqlens, num_seqs, scale)
    _opt(h0, torch.float32, P.states, "h0")
    ws = _scratch(workspace, _lib().dla_workspace_bytes(P.shape, 0), v)
    o = torch.empty(P.vshape, dtype=torch.bfloat16, device=v.device)
    ht = torch.empty(P.states, dtype=torch.float32, device=v.device) if want_ht else None
    rc = _lib().dla_fwd(P.shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(h0), o.data_ptr(),
                        _ptr(ht), ws.data_ptr(), ws.numel(), _stream(v, q, k, log_decay, h0, P.cu, ws))
    if rc:
        _check(rc, "dla_fwd")
    return {"o": o, "ht": ht}


def dla_bwd(q, k, v, log_decay, dO, h0=None, dht=None, cu_seqlens=None, num_seqs=None, scale=None, workspace=None):
    """Backward of dla_fwd for the loss sum <dO, o> + sum <dht, ht>.  Returns dict(dq, dk, dv, dh0); the decay is
    a constant of its head."""
    P = _Call(q, k, v, log_decay, cu_seqlens, num_seqs, scale)
    _need(dO, torch.bfloat16, P.vshape, "dO")
    _opt(h0, torch.float32, P.states, "h0")
    _opt(dht, torch.float32, P.states, "dht")
    ws = _scratch(workspace, _lib().dla_workspace_bytes(P.shape, 1), v)
    bf16 = dict(dtype=torch.bfloat16, device=v.device)
    out = {"dq": torch.empty(P.qshape, **bf16), "dk": torch.empty(P.qshape, **bf16), "dv": torch.empty(P.vshape, **bf16),
           "dh0": torch.empty(P.states, dtype=torch.float32, device=v.device)}
    rc = _lib().dla_bwd(P.shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _ptr(h0), dO.data_ptr(),
                        _ptr(dht), ws.data_ptr(), ws.numel(), out["dq"].data_ptr(), out["dk"].data_ptr(),
                        out["dv"].data_ptr(), out["dh0"].data_ptr(), _stream(v, q, k, log_decay, h0, dO, dht, P.cu, ws))
    if rc:
        _check(rc, "dla_bwd")
    return out


def dla_step(q, k, v, log_decay, state, slots=None, scale=None, out=None):
    """One token of dla_fwd for each row: q, k bf16 [rows, Hk, D], v [rows, H, D]; ``state`` float32
    [pool, H, D, D] is updated in place.  Returns o [rows, H, D] (zero for rows whose slot is negative)."""
    if q is None or v is None or q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and v must be [rows, heads, D]")
    rows, H, D = v.shape
    Hk = q.shape[1]
    _need(log_decay, torch.float32, (H,), "log_decay")
    ld = [_tokens(t, (rows, n, D), name) for t, n, name in ((q, Hk, "q"), (k, Hk, "k"), (v, H, "v"))]
    pool = _pool(state, torch.float32, (H, D, D), slots, rows, "state")
    o = torch.empty((rows, H, D), dtype=torch.bfloat16, device=v.device) if out is None else \
        _need(out, torch.bfloat16, (rows, H, D), "out")
    rc = _lib().dla_step(rows, H, Hk, D, pool, D ** -0.5 if scale is None else scale, q.data_ptr(), ld[0], k.data_ptr(),
                         ld[1], v.data_ptr(), ld[2], log_decay.data_ptr(), _ptr(slots), state.data_ptr(), o.data_ptr(),
                         _stream(v, q, k, log_decay, slots, state, o))
    if rc:
        _check(rc, "dla_step")
    return o
