"""Python binding of the operators around the delta rule in a recurrent block (argument
marshalling only, as ``api``): the causal conv1d's forward and single-token step, the gated
linear recurrence (forward, backward, step) and the RMS norm with the residual's addition
(forward, backward).

Layouts: activations are token-major ``[T_total, C]`` (packed sequences through
``cu_seqlens``, int64 ``[N + 1]``) or dense ``[B, T, C]``; ``x`` and ``g`` may be column
slices of a wider tensor (rows of one stride), everything else is contiguous.  Steps take
``[rows, C]`` and a pool of states, with ``slots`` (int64 ``[rows]``) naming each row's state
and a negative slot marking a padded row.
"""
import ctypes

import torch

from .api import _check, lib

GATES = {"log": 0, "softplus": 1}      # GLR_GATE_LOG / GLR_GATE_SOFTPLUS
QUANTS = {None: 0, "token": 1, "block": 2}  # GDR_QUANT_NONE / GDR_QUANT_ROW / GDR_QUANT_BLOCK
_TYPES = {torch.bfloat16: 0, torch.float32: 1}  # GDR_TYPE_BF16 / GDR_TYPE_F32


class GlrShape(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32), ("total_tokens", ctypes.c_int64), ("channels", ctypes.c_int32),
                ("cu_seqlens", ctypes.c_void_p), ("gate", ctypes.c_int32), ("complement", ctypes.c_int32),
                ("act_type", ctypes.c_int32), ("gate_type", ctypes.c_int32), ("x_stride", ctypes.c_int64),
                ("g_stride", ctypes.c_int64)]


_LIB = None


def _like(t):
    """An uninitialised contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _lib():
    global _LIB
    if _LIB is None:
        L = lib()
        vp, sz, i32, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        sp, st = ctypes.POINTER(GlrShape), ctypes.c_int
        for name, res, args in (
                ("glr_workspace_bytes", sz, [sp]),
                ("glr_fwd", st, [sp] + [vp] * 8 + [sz, vp]),
                ("glr_bwd", st, [sp] + [vp] * 9 + [sz] + [vp] * 6),
                ("glr_step", st, [i32] * 7 + [vp, i64, vp, i64] + [vp] * 6),
                ("gdr_rmsnorm_fwd", st, [i64, i32, vp, i64, vp, i32, vp, f32, i32] + [vp] * 5),
                ("gdr_rmsnorm_workspace_bytes", sz, [i64, i32]),
                ("gdr_rmsnorm_bwd", st, [i64, i32, vp, vp, i32, vp, vp, vp, vp, sz, vp, vp, vp]),
                ("gdr_conv1d_fwd", st, [i32, i64, i32, i32, vp, vp, i64, vp, vp, vp, i32, vp, vp, vp]),
                ("gdr_conv1d_step", st, [i32] * 4 + [vp, i64] + [vp] * 4 + [i32, vp, vp])):
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        L.glr_test_stall_next_call.restype, L.glr_test_stall_next_call.argtypes = None, [ctypes.c_int]
        _LIB = L
    return _LIB


def _ptr(t):
    return None if t is None else t.data_ptr()


_SEVERAL = None  # whether there are several GPUs


def _stream(t, *others):
    """The current stream of t's device, which all tensors of a call are on and which is the current one."""
    global _SEVERAL
    if _SEVERAL is None:
        _SEVERAL = torch.cuda.device_count() > 1
    if _SEVERAL:
        current = torch.cuda.current_device()
        for u in (t,) + others:
            if u is not None and u.get_device() != current:
                raise ValueError("all tensors of a call must be on the current device %d (got %s)" % (current, u.device))
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _scratch(workspace, need, like):
    """A workspace of ``need`` bytes: the caller's, or a new one."""
    if workspace is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=like.device)
    if workspace.dtype is not torch.uint8 or workspace.numel() < need or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA uint8 tensor of at least %d bytes" % need)
    return workspace


def _bad(t, dtype, shape, name):
    if t is None:
        raise ValueError("%s is required" % name)
    raise ValueError("%s must be a contiguous CUDA %s tensor of shape %s (got %s %s %s)"
                     % (name, dtype, tuple(shape), t.device, t.dtype, tuple(t.shape)))


def _need(t, dtype, shape, name):
    if t is None or t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _bad(t, dtype, shape, name)
    return t


def _opt(t, dtype, shape, name):
    return None if t is None else _need(t, dtype, shape, name)


def _rows(t, dtypes, shape, name):
    """A tensor of rows of one stride (a column slice of a wider one is fine); returns the stride."""
    if t is None or t.dtype not in dtypes or t.shape != shape or not t.is_cuda:
        _bad(t, " / ".join(str(d) for d in dtypes), shape, name)
    C = shape[-1]
    if t.is_contiguous():
        return C
    st = t.stride()
    many = [i for i in range(len(shape) - 1) if shape[i] > 1]  # strides of single rows mean nothing
    ld = st[many[-1]] if many else C
    if st[-1] != 1 or ld < C or (len(many) == 2 and st[0] != shape[1] * ld):
        raise ValueError("%s must consist of rows of one stride (got strides %s for shape %s)" % (name, st, tuple(shape)))
    return ld


class _Tokens:
    """Sequences and tokens of one call, from x ([T, C] with cu_seqlens / num_seqs, or [B, T, C])."""

    def __init__(self, x, cu_seqlens, num_seqs):
        if x is None or x.dim() not in (2, 3):
            raise ValueError("x must be [T_total, C] or [B, T, C]")
        self.shape, self.C = x.shape, x.shape[-1]
        if x.dim() == 3:
            if cu_seqlens is not None:
                raise ValueError("cu_seqlens goes with packed [T_total, C] tensors")
            self.N, self.T = x.shape[0], x.shape[0] * x.shape[1]
        else:
            self.T = x.shape[0]
            self.N = (1 if num_seqs is None else int(num_seqs)) if cu_seqlens is None else cu_seqlens.numel() - 1
        if cu_seqlens is not None:
            _need(cu_seqlens, torch.int64, (self.N + 1,), "cu_seqlens")
        self.cu = cu_seqlens


def _gate(gate, A_log, dt_bias, C):
    if gate not in GATES:
        raise ValueError("gate must be one of %s" % sorted(GATES))
    if gate == "softplus":
        _need(A_log, torch.float32, (C,), "A_log")
        _need(dt_bias, torch.float32, (C,), "dt_bias")
        return 1, A_log, dt_bias
    return 0, None, None


def _glr_types(x, g):
    if x.dtype is torch.float32 and g.dtype is torch.bfloat16:
        raise ValueError("float32 activations need a float32 gate")


_ACT = (torch.bfloat16, torch.float32)


def _glr_shape(x, g, cu_seqlens, num_seqs, gate, complement):
    P = _Tokens(x, cu_seqlens, num_seqs)
    ldx = _rows(x, _ACT, P.shape, "x")
    ldg = _rows(g, _ACT, P.shape, "g")
    _glr_types(x, g)
    return P, GlrShape(P.N, P.T, P.C, _ptr(P.cu), gate, bool(complement), _TYPES[x.dtype], _TYPES[g.dtype], ldx, ldg)


def glr_workspace_bytes(x, g, cu_seqlens=None, num_seqs=None, gate="log", complement=False):
    """Bytes of the workspace of glr_fwd / glr_bwd for these tensors."""
    return int(_lib().glr_workspace_bytes(_glr_shape(x, g, cu_seqlens, num_seqs, GATES[gate], complement)[1]))


def glr_fwd(x, g, h0=None, A_log=None, dt_bias=None, cu_seqlens=None, num_seqs=None, gate="log", complement=False,
            want_ht=True, workspace=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + s_t x_t per channel, a = exp(log gate), s = 1 or (with
    ``complement``) 1 - a.  ``gate``: "log" (g is the log gate) or "softplus" (g is g_raw, the log gate
    -exp(A_log) softplus(g_raw + dt_bias)).  x bf16 or float32, g bf16 or float32 (float32 for float32 x),
    A_log, dt_bias float32 [C], h0 float32 [N, C].  Returns dict(h, ht)."""
    gate, A_log, dt_bias = _gate(gate, A_log, dt_bias, x.shape[-1])
    P, sh = _glr_shape(x, g, cu_seqlens, num_seqs, gate, complement)
    _opt(h0, torch.float32, (P.N, P.C), "h0")
    ws = _scratch(workspace, _lib().glr_workspace_bytes(sh), x)
    h = _like(x)
    ht = torch.empty((P.N, P.C), dtype=torch.float32, device=x.device) if want_ht else None
    rc = _lib().glr_fwd(sh, x.data_ptr(), g.data_ptr(), _ptr(A_log), _ptr(dt_bias), _ptr(h0), h.data_ptr(), _ptr(ht),
                        ws.data_ptr(), ws.numel(), _stream(x, g, A_log, dt_bias, h0, P.cu, ws))
    if rc:
        _check(rc, "glr_fwd")
    return {"h": h, "ht": ht}


def glr_bwd(x, g, h, dh, h0=None, dht=None, A_log=None, dt_bias=None, cu_seqlens=None, num_seqs=None, gate="log",
            complement=False, workspace=None):
    """Backward of glr_fwd for the loss sum <dh, h> + sum <dht, ht>; h is the forward's output.  Returns
    dict(dx, dg, dh0) and, with the softplus gate, dA_log and ddt_bias (dg is then with respect to g_raw)."""
    gate, A_log, dt_bias = _gate(gate, A_log, dt_bias, x.shape[-1])
    P, sh = _glr_shape(x, g, cu_seqlens, num_seqs, gate, complement)
    _need(h, x.dtype, P.shape, "h")
    _need(dh, x.dtype, P.shape, "dh")
    _opt(h0, torch.float32, (P.N, P.C), "h0")
    _opt(dht, torch.float32, (P.N, P.C), "dht")
    ws = _scratch(workspace, _lib().glr_workspace_bytes(sh), x)
    out = {"dx": _like(x), "dg": _like(g),
           "dh0": torch.empty((P.N, P.C), dtype=torch.float32, device=x.device)}
    if gate:
        out["dA_log"] = torch.empty(P.C, dtype=torch.float32, device=x.device)
        out["ddt_bias"] = torch.empty(P.C, dtype=torch.float32, device=x.device)
    rc = _lib().glr_bwd(sh, x.data_ptr(), g.data_ptr(), _ptr(A_log), _ptr(dt_bias), h.data_ptr(), _ptr(h0),
                        dh.data_ptr(), _ptr(dht), ws.data_ptr(), ws.numel(), out["dx"].data_ptr(),
                        out["dg"].data_ptr(), out["dh0"].data_ptr(), _ptr(out.get("dA_log")),
                        _ptr(out.get("ddt_bias")), _stream(x, g, A_log, dt_bias, h, h0, dh, dht, P.cu, ws))
    if rc:
        _check(rc, "glr_bwd")
    return out


def _pool(state, dtype, tail, slots, rows, name):
    if state is None or state.dim() != len(tail) + 1 or state.shape[1:] != tail or state.dtype is not dtype or \
            not state.is_cuda or not state.is_contiguous():
        _bad(state, dtype, (rows if slots is None else "pool",) + tuple(tail), name)
    if slots is not None:
        _need(slots, torch.int64, (rows,), "slots")
    elif state.shape[0] < rows:
        raise ValueError("%s holds fewer states than there are rows" % name)
    return state.shape[0]


def glr_step(x, g, state, slots=None, A_log=None, dt_bias=None, gate="log", complement=False, out=None):
    """One token of glr_fwd for each row: x, g [rows, C]; ``state`` float32 [pool, C] is updated in place.
    Returns y [rows, C] (the new state in x's type; zero for rows whose slot is negative)."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, C]")
    rows, C = shape = x.shape
    gate, A_log, dt_bias = _gate(gate, A_log, dt_bias, C)
    ldx = _rows(x, _ACT, shape, "x")
    ldg = _rows(g, _ACT, shape, "g")
    _glr_types(x, g)
    pool = _pool(state, torch.float32, (C,), slots, rows, "state")
    y = _like(x) if out is None else _need(out, x.dtype, shape, "out")
    rc = _lib().glr_step(rows, C, pool, gate, bool(complement), _TYPES[x.dtype], _TYPES[g.dtype], x.data_ptr(), ldx,
                         g.data_ptr(), ldg, _ptr(A_log), _ptr(dt_bias), _ptr(slots), state.data_ptr(), y.data_ptr(),
                         _stream(x, g, A_log, dt_bias, slots, state, y))
    if rc:
        _check(rc, "glr_step")
    return y


def rmsnorm_fwd(x, weight, residual=None, eps=1e-6, quant=None):
    """RMS norm of s = x + residual over the last dimension: x bf16 [..., C], residual bf16 or float32 of x's
    shape or None, weight float32 [C].  ``quant``: None (y bf16), "token" or "block" (y float8_e4m3fn with a
    float32 scale for each row, or for each 128 channels of it).  Returns dict(y, rstd), with ``residual``
    (the stored sum s) if one was given and ``scale`` with quant."""
    if quant not in QUANTS:
        raise ValueError("quant must be None, 'token' or 'block'")
    if x.dim() < 1:
        raise ValueError("x must be [..., C]")
    shape = x.shape
    C = shape[-1]
    if x.dim() != 2:
        x = x.reshape(-1, C)
    rows = x.shape[0]
    ldx = _rows(x, (torch.bfloat16,), (rows, C), "x")
    _need(weight, torch.float32, (C,), "weight")
    if quant:
        y = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
    else:
        y = _like(x) if x.shape == shape else torch.empty(shape, dtype=torch.bfloat16, device=x.device)
    out = {"y": y, "rstd": torch.empty(shape[:-1], dtype=torch.float32, device=x.device)}
    res_type = 0
    if residual is not None:
        if residual.dtype not in _TYPES:
            _bad(residual, "bfloat16 / float32", shape, "residual")
        _need(residual, residual.dtype, shape, "residual")
        res_type = _TYPES[residual.dtype]
        out["residual"] = torch.empty_like(residual)
    if quant:
        out["scale"] = torch.empty((rows, 1 if quant == "token" else (C + 127) // 128), dtype=torch.float32,
                                   device=x.device)
    rc = _lib().gdr_rmsnorm_fwd(rows, C, x.data_ptr(), ldx, _ptr(residual), res_type, weight.data_ptr(), eps,
                                QUANTS[quant], out["y"].data_ptr(), _ptr(out.get("scale")), _ptr(out.get("residual")),
                                out["rstd"].data_ptr(), _stream(x, weight, residual))
    if rc:
        _check(rc, "gdr_rmsnorm_fwd")
    return out


def rmsnorm_bwd(dy, s, weight, rstd, dres=None, workspace=None):
    """Backward of rmsnorm_fwd: dy bf16 [..., C]; s the stored sum (the forward's ``residual``, or its x);
    dres (s's type) the gradient that reaches s directly.  Returns dict(dx, dweight); dx, in s's type, is the
    gradient of s, hence of both x and the residual."""
    if s is None or s.dim() < 1 or s.dtype not in _TYPES:
        raise ValueError("s must be a bfloat16 or float32 tensor [..., C]")
    shape = s.shape
    C = shape[-1]
    _need(s, s.dtype, shape, "s")
    _need(dy, torch.bfloat16, shape, "dy")
    _need(weight, torch.float32, (C,), "weight")
    _need(rstd, torch.float32, shape[:-1], "rstd")
    _opt(dres, s.dtype, shape, "dres")
    rows = rstd.numel()
    need = _lib().gdr_rmsnorm_workspace_bytes(rows, C)
    workspace = _scratch(workspace, need, s)
    out = {"dx": torch.empty_like(s),
           "dweight": torch.empty(C, dtype=torch.float32, device=s.device)}
    rc = _lib().gdr_rmsnorm_bwd(rows, C, dy.data_ptr(), s.data_ptr(), _TYPES[s.dtype], weight.data_ptr(),
                                rstd.data_ptr(), _ptr(dres), workspace.data_ptr(), workspace.numel(),
                                out["dx"].data_ptr(), out["dweight"].data_ptr(), _stream(s, dy, weight, rstd, dres, workspace))
    if rc:
        _check(rc, "gdr_rmsnorm_bwd")
    return out


def _conv_weights(weight, bias, C):
    K = weight.shape[1] if weight is not None and weight.dim() == 2 else -1
    _need(weight, torch.float32, (C, K), "weight")
    _opt(bias, torch.float32, (C,), "bias")
    return K


def conv1d_fwd(x, weight, bias=None, state=None, cu_seqlens=None, num_seqs=None, silu=True, want_state=False):
    """Causal depthwise conv1d (+ SiLU): x bf16 [T, C] (or [B, T, C]), weight float32 [C, K], bias float32 [C]
    or None; ``state`` bf16 [N, K - 1, C] holds the inputs before each sequence (oldest first; None: zero).
    Returns dict(y, state): the last K - 1 inputs of each sequence with ``want_state``, else None."""
    P = _Tokens(x, cu_seqlens, num_seqs)
    ldx = _rows(x, (torch.bfloat16,), P.shape, "x")
    K = _conv_weights(weight, bias, P.C)
    _opt(state, torch.bfloat16, (P.N, K - 1, P.C), "state")
    y = _like(x)
    new = torch.empty((P.N, K - 1, P.C), dtype=torch.bfloat16, device=x.device) if want_state else None
    rc = _lib().gdr_conv1d_fwd(P.N, P.T, P.C, K, _ptr(P.cu), x.data_ptr(), ldx, weight.data_ptr(), _ptr(bias),
                               _ptr(state), bool(silu), y.data_ptr(), _ptr(new), _stream(x, weight, bias, state, P.cu))
    if rc:
        _check(rc, "gdr_conv1d_fwd")
    return {"y": y, "state": new}


def conv1d_step(x, state, weight, bias=None, slots=None, silu=True, out=None):
    """One token of conv1d_fwd for each row: x bf16 [rows, C]; ``state`` bf16 [pool, K - 1, C] is shifted in
    place.  Returns y [rows, C] (zero for rows whose slot is negative)."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, C]")
    rows, C = shape = x.shape
    ldx = _rows(x, (torch.bfloat16,), shape, "x")
    K = _conv_weights(weight, bias, C)
    pool = _pool(state, torch.bfloat16, (K - 1, C), slots, rows, "state")
    y = _like(x) if out is None else \
        _need(out, torch.bfloat16, shape, "out")
    rc = _lib().gdr_conv1d_step(rows, C, K, pool, x.data_ptr(), ldx, state.data_ptr(), weight.data_ptr(), _ptr(bias),
                                _ptr(slots), bool(silu), y.data_ptr(), _stream(x, state, weight, bias, slots, y))
    if rc:
        _check(rc, "gdr_conv1d_step")
    return y


def test_stall_next_glr(block: int):
    """Test hook: block ``block`` of the next glr_fwd / glr_bwd gives up at its second tile, as after a
    wait that ran out (GDR_DEV_TIMEOUT)."""
    _lib().glr_test_stall_next_call(int(block))
