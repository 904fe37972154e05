"""The operators around the delta rule in a recurrent block, float64, from their definitions
(TEST INFRASTRUCTURE ONLY; shares no code with the CUDA path).

* gated linear recurrence: h_t = a_t h_{t-1} + s_t x_t token by token, a = exp(g), s = 1 or
  1 - a, g given or -exp(A_log) softplus(g_raw + dt_bias); its gradients by the chain rule
  walked backwards through the same tokens;
* RMS norm with the residual's addition (the sum rounded as it is stored), and its gradients;
* causal conv1d forward with states (``oracle.conv`` has the stateless forward and the backward).
"""
import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def softplus(z):
    return np.logaddexp(z, 0.0)


def sigmoid(z):
    return np.exp(-np.logaddexp(0.0, -z))


def log_gate(g, A_log, dt_bias):
    return g if A_log is None else -np.exp(A_log) * softplus(g + dt_bias)


def glr_fwd(x, g, cu, h0=None, A_log=None, dt_bias=None, complement=False):
    """x, g [T, C], cu [N + 1] -> h [T, C], ht [N, C]."""
    x, g, h0, A_log, dt_bias = (_f64(v) for v in (x, g, h0, A_log, dt_bias))
    lg = log_gate(g, A_log, dt_bias)
    T, C = x.shape
    N = len(cu) - 1
    h, ht = np.zeros((T, C)), np.zeros((N, C))
    for n in range(N):
        s = np.zeros(C) if h0 is None else h0[n].copy()
        for t in range(cu[n], cu[n + 1]):
            s = np.exp(lg[t]) * s + (-np.expm1(lg[t]) if complement else 1.0) * x[t]
            h[t] = s
        ht[n] = s
    return h, ht


def glr_bwd(x, g, h, dh, cu, h0=None, dht=None, A_log=None, dt_bias=None, complement=False):
    """Gradients of sum <dh, h> + sum <dht, ht>, with h_{t-1} read from ``h``.  Returns dict(dx, dg, dh0,
    dA_log, ddt_bias, and the magnitudes sum |terms| of the last two as mA_log, mdt_bias)."""
    x, g, h, dh, h0, dht, A_log, dt_bias = (_f64(v) for v in (x, g, h, dh, h0, dht, A_log, dt_bias))
    lg = log_gate(g, A_log, dt_bias)
    T, C = x.shape
    N = len(cu) - 1
    dx, dlg = np.zeros((T, C)), np.zeros((T, C))
    dh0 = np.zeros((N, C)) if dht is None else dht.copy()
    for n in range(N):
        back = dh0[n].copy()
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            a = np.exp(lg[t])
            prev = h[t - 1] if t > cu[n] else (np.zeros(C) if h0 is None else h0[n])
            lam = dh[t] + back
            dx[t] = lam * (-np.expm1(lg[t]) if complement else 1.0)
            dlg[t] = lam * a * (prev - x[t] if complement else prev)
            back = a * lam
        dh0[n] = back
    out = {"dx": dx, "dg": dlg, "dh0": dh0}
    if A_log is not None:
        out["dg"] = dlg * -np.exp(A_log) * sigmoid(g + dt_bias)
        out["dA_log"], out["mA_log"] = (dlg * lg).sum(0), np.abs(dlg * lg).sum(0)
        out["ddt_bias"], out["mdt_bias"] = out["dg"].sum(0), np.abs(out["dg"]).sum(0)
    return out


def rmsnorm(s, weight, eps):
    """s [R, C] (the stored sum) -> y, rstd."""
    s, weight = _f64(s), _f64(weight)
    rstd = 1.0 / np.sqrt((s * s).mean(1) + eps)
    return s * rstd[:, None] * weight, rstd


def rmsnorm_bwd(dy, s, weight, eps, dres=None):
    """Gradients of sum <dy, y> + sum <dres, s>: dx [R, C], dweight [C] and sum |terms| of dweight."""
    dy, s, weight, dres = (_f64(v) for v in (dy, s, weight, dres))
    rstd = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    n, u = s * rstd, weight * dy
    dx = rstd * (u - n * (u * n).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + dres
    return dx, (dy * n).sum(0), np.abs(dy * n).sum(0)


def block_scales(y, block):
    """max |y| / 448 of each ``block`` channels (1 where they are all zero) [R, ceil(C / block)]."""
    y = _f64(y)
    R, C = y.shape
    nb = -(-C // block)
    pad = np.zeros((R, nb * block))
    pad[:, :C] = np.abs(y)
    most = pad.reshape(R, nb, block).max(2)
    return np.where(most > 0, most / 448.0, 1.0)


def conv1d_fwd(x, w, bias, cu, silu, state=None):
    """x [T, C], w [C, K], state [N, K - 1, C] -> y [T, C], the states after the sequences [N, K - 1, C]."""
    x, w, bias, state = (_f64(v) for v in (x, w, bias, state))
    T, C = x.shape
    K, N = w.shape[1], len(cu) - 1
    y, new = np.zeros((T, C)), np.zeros((N, K - 1, C))
    for n in range(N):
        L = cu[n + 1] - cu[n]
        line = np.concatenate([np.zeros((K - 1, C)) if state is None else state[n], x[cu[n]:cu[n + 1]]])
        z = sum(w[:, k] * line[k:k + L] for k in range(K)) + (0.0 if bias is None else bias)
        y[cu[n]:cu[n + 1]] = z * sigmoid(z) if silu else z
        new[n] = line[L:]
    return y, new
