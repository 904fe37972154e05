"""Linear attention with a decay for each head and the 8-bit products around it, float64, from their
definitions (TEST INFRASTRUCTURE ONLY; shares no code with the CUDA path).

* S_t = e^g S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t token by token, and its gradients by the chain rule
  walked backwards through the same tokens;
* codes and scales of e4m3 blocks, and the product of such operands.

With ``magnitudes=True`` the recurrences run on absolute values: sums of the terms' magnitudes, which
bound what rounding the terms can do.
"""
import numpy as np


def _f64(a):
    return None if a is None else np.asarray(a, dtype=np.float64)


def _prepared(arrays, magnitudes):
    arrays = [_f64(a) for a in arrays]
    return [None if a is None else np.abs(a) for a in arrays] if magnitudes else arrays


def dla_fwd(q, k, v, g, cu, h0=None, scale=1.0, magnitudes=False):
    """q, k [T, Hk, D], v [T, H, D], g [H], cu [N + 1], h0 [N, H, D, D] -> o [T, H, D], ht [N, H, D, D]."""
    q, k, v, h0 = _prepared((q, k, v, h0), magnitudes)
    T, H, D = v.shape
    group, N = H // q.shape[1], len(cu) - 1
    a = np.exp(_f64(g))[:, None, None]
    scale = abs(scale) if magnitudes else scale
    o, ht = np.zeros((T, H, D)), np.zeros((N, H, D, D))
    for n in range(N):
        S = np.zeros((H, D, D)) if h0 is None else h0[n].copy()
        for t in range(cu[n], cu[n + 1]):
            S = a * S + np.repeat(k[t], group, axis=0)[:, :, None] * v[t][:, None, :]
            o[t] = scale * np.matmul(np.repeat(q[t], group, axis=0)[:, None, :], S)[:, 0]
        ht[n] = S
    return o, ht


def dla_bwd(q, k, v, g, dO, cu, h0=None, dht=None, scale=1.0, magnitudes=False):
    """Gradients of sum <dO, o> + sum <dht, ht>: dict(dq, dk, dv, dh0)."""
    q, k, v, dO, h0, dht = _prepared((q, k, v, dO, h0, dht), magnitudes)
    T, H, D = v.shape
    Hk, N = q.shape[1], len(cu) - 1
    group = H // Hk
    a = np.exp(_f64(g))[:, None, None]
    scale = abs(scale) if magnitudes else scale
    dq, dk, dv = np.zeros((T, H, D)), np.zeros((T, H, D)), np.zeros((T, H, D))
    dh0 = np.zeros((N, H, D, D))
    wide = lambda x: np.repeat(x, group, axis=0)  # noqa: E731
    for n in range(N):
        S = np.zeros((H, D, D)) if h0 is None else h0[n].copy()
        for t in range(cu[n], cu[n + 1]):
            S = a * S + wide(k[t])[:, :, None] * v[t][:, None, :]
            dq[t] = scale * np.matmul(S, dO[t][:, :, None])[:, :, 0]
        R = np.zeros((H, D, D)) if dht is None else dht[n].copy()
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            R = R + scale * wide(q[t])[:, :, None] * dO[t][:, None, :]
            dk[t] = np.matmul(R, v[t][:, :, None])[:, :, 0]
            dv[t] = np.matmul(wide(k[t])[:, None, :], R)[:, 0]
            R = a * R
        dh0[n] = R
    shared = lambda x: x.reshape(T, Hk, group, D).sum(2)  # noqa: E731
    return {"dq": shared(dq), "dk": shared(dk), "dv": dv, "dh0": dh0}


def tile_scales(x, rows, cols=128):
    """max |x| / 448 of each rows x cols tile of a matrix (1 where it is all zero)."""
    x = np.abs(_f64(x))
    R, C = x.shape
    nr, nc = -(-R // rows), -(-C // cols)
    pad = np.zeros((nr * rows, nc * cols))
    pad[:R, :C] = x
    most = pad.reshape(nr, rows, nc, cols).max((1, 3))
    return np.where(most > 0, most / 448.0, 1.0)


def spread(scale, rows, cols, shape):
    """A scale for each element of a matrix of ``shape`` from those of its rows x cols tiles."""
    return np.repeat(np.repeat(_f64(scale), rows, axis=0), cols, axis=1)[:shape[0], :shape[1]]


def linear(x, xs, w, ws, bias=None, magnitudes=False):
    """x [M, K], w [N, K]: the values of e4m3 codes; xs [M, ceil(K / 128)] or [M, 1], ws [ceil(N / 128), ceil(K / 128)]."""
    x, w, bias = _f64(x), _f64(w), _f64(bias)
    x = x * (spread(xs, 1, 128, x.shape) if xs.shape[1] > 1 else _f64(xs))
    w = w * spread(ws, 128, 128, w.shape)
    if magnitudes:
        x, w, bias = np.abs(x), np.abs(w), None if bias is None else np.abs(bias)
    y = x @ w.T
    return y if bias is None else y + bias
