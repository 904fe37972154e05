"""Pins of the float64 oracle of the recurrent block's operators (oracle/block.py): gradients
against central differences, the conv against oracle/conv.py, closed forms."""
import numpy as np
import pytest

from oracle import block, conv


def _diff(f, v, d, eps=1e-6):
    return (f(v + eps * d) - f(v - eps * d)) / (2 * eps)


@pytest.mark.parametrize("soft", [False, True])
@pytest.mark.parametrize("comp", [False, True])
def test_glr_gradients_against_differences(soft, comp):
    r = np.random.RandomState(3)
    lens = [5, 0, 1, 9]
    cu = np.concatenate([[0], np.cumsum(lens)])
    T, C, N = cu[-1], 4, len(lens)
    v = {"x": r.randn(T, C), "g": r.randn(T, C) * 0.5 - (0.0 if soft else 1.0), "h0": r.randn(N, C)}
    if soft:
        v["A_log"], v["dt_bias"] = r.randn(C) * 0.3, r.randn(C)
    dh, dht = r.randn(T, C), r.randn(N, C)

    def loss(**over):
        h, ht = block.glr_fwd(cu=cu, complement=comp, **{**v, **over})
        return (h * dh).sum() + (ht * dht).sum()

    h, _ = block.glr_fwd(cu=cu, complement=comp, **v)
    out = block.glr_bwd(v["x"], v["g"], h, dh, cu, v["h0"], dht, v.get("A_log"), v.get("dt_bias"), comp)
    for name in v:
        d = r.randn(*v[name].shape)
        want = _diff(lambda p: loss(**{name: p}), v[name], d)
        # central differences of O(1) values at eps 1e-6: truncation ~1e-12, rounding ~1e-16 T C / 1e-6
        assert abs((out["d" + name] * d).sum() - want) < 1e-7 * max(1.0, abs(want)), name


def test_glr_closed_form():
    # constant decay a and input 1: h_t = sum_{i<=t} a^i; with the complement 1 - a^{t+1}
    a, T = 0.7, 12
    g, x = np.full((T, 2), np.log(a)), np.ones((T, 2))
    t = np.arange(1, T + 1)[:, None]
    assert np.allclose(block.glr_fwd(x, g, [0, T])[0], (1 - a ** t) / (1 - a), atol=1e-13)
    assert np.allclose(block.glr_fwd(x, g, [0, T], complement=True)[0], 1 - a ** t, atol=1e-13)


def test_rmsnorm_gradients_against_differences():
    r = np.random.RandomState(4)
    s, w, dy, dres = r.randn(3, 10), r.randn(10), r.randn(3, 10), r.randn(3, 10)
    dx, dw, _ = block.rmsnorm_bwd(dy, s, w, 1e-6, dres)
    d = r.randn(3, 10)
    want = _diff(lambda p: (block.rmsnorm(p, w, 1e-6)[0] * dy).sum() + (p * dres).sum(), s, d)
    assert abs((dx * d).sum() - want) < 1e-7
    d = r.randn(10)
    want = _diff(lambda p: (block.rmsnorm(s, p, 1e-6)[0] * dy).sum(), w, d)
    assert abs((dw * d).sum() - want) < 1e-7


@pytest.mark.parametrize("width", [1, 2, 4])
def test_conv_forward_agrees_and_continues(width):
    r = np.random.RandomState(5)
    cu = np.array([0, 7, 7, 9])
    x, w, b = r.randn(9, 3), r.randn(3, width), r.randn(3)
    y, new = block.conv1d_fwd(x, w, b, cu, True)
    assert np.allclose(y, conv.conv1d_fwd(x, w, b, cu, True)[0], atol=1e-13)
    # a sequence cut in two, the second part from the first one's state, gives the same outputs
    y1, st = block.conv1d_fwd(x[:2], w, b, [0, 2], True)
    y2, st2 = block.conv1d_fwd(x[2:7], w, b, [0, 5], True, state=st)
    assert np.allclose(np.concatenate([y1, y2]), y[:7], atol=1e-13) and np.allclose(st2[0], new[0])


def test_block_scales():
    y = np.zeros((2, 130))
    y[0, 5], y[0, 129] = -448.0, 4.48
    assert np.allclose(block.block_scales(y, 128), [[1.0, 0.01], [1.0, 1.0]])
