"""Pins of the float64 oracle of linear attention with a decay for each head (oracle/dla.py): worked
values, the closed form of the sums, and its gradients against central differences."""
import numpy as np
import pytest

from oracle import dla as ref


def _inputs(T, H, Hk, D, N, seed=0):
    r = np.random.default_rng(seed)
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    cu = [0] + sorted(r.integers(0, T + 1, N - 1).tolist()) + [T]
    return dict(q=n(T, Hk, D), k=n(T, Hk, D), v=n(T, H, D), g=-np.abs(n(H)) * 0.3, cu=cu, h0=n(N, H, D, D)), n(T, H, D), n(N, H, D, D)


def test_two_tokens_by_hand():
    one = np.ones((2, 1, 1))
    o, ht = ref.dla_fwd(2 * one, 3 * one, np.array([[[5.0]], [[7.0]]]), [np.log(0.5)], [0, 2], scale=0.1)
    # S_1 = 15, S_2 = 7.5 + 21
    assert np.allclose(o[:, 0, 0], [0.1 * 2 * 15, 0.1 * 2 * 28.5], rtol=1e-15) and np.allclose(ht, 28.5, rtol=1e-15)


def test_closed_form():
    x, _, _ = _inputs(9, 4, 2, 3, 2)
    o, ht = ref.dla_fwd(**x, scale=0.7)
    for n in range(2):
        b, e = x["cu"][n], x["cu"][n + 1]
        for h in range(4):
            for t in range(b, e):
                want = sum(np.exp(x["g"][h] * (t - s)) * (x["q"][t, h // 2] @ x["k"][s, h // 2]) * x["v"][s, h] for s in range(b, t + 1))
                want = want + np.exp(x["g"][h] * (t - b + 1)) * x["q"][t, h // 2] @ x["h0"][n, h]
                assert np.allclose(o[t, h], 0.7 * want, rtol=1e-12)


@pytest.mark.parametrize("name", ["q", "k", "v", "h0"])
def test_gradients_against_differences(name):
    x, dO, dht = _inputs(8, 4, 2, 3, 3, seed=3)
    grads = ref.dla_bwd(**{k: v for k, v in x.items()}, dO=dO, dht=dht, scale=0.6)

    def loss(y):
        o, ht = ref.dla_fwd(**{**x, name: y}, scale=0.6)
        return (o * dO).sum() + (ht * dht).sum()

    grad = np.zeros_like(x[name])
    for i in np.ndindex(x[name].shape):  # the loss is linear in each of them: differences are exact but for rounding
        step = np.zeros_like(grad)
        step[i] = 0.5
        grad[i] = loss(x[name] + step) - loss(x[name] - step)
    assert np.allclose(grads["d" + name], grad, rtol=1e-10, atol=1e-11)


def test_tile_scales_and_product():
    x = np.zeros((3, 130))
    x[0, 5], x[2, 129], x[1, 7] = -448.0, 4.48, 44.8
    s = ref.tile_scales(x, 1)
    assert np.allclose(s, [[1, 1], [0.1, 1], [1, 0.01]]) and np.allclose(ref.tile_scales(x, 128), [[1, 0.01]])
    w = np.ones((129, 130))
    ws = np.array([[1.0, 2.0], [3.0, 4.0]])
    y = ref.linear(x, s, w, ws, bias=np.arange(129.0))
    assert np.allclose(y[2, :128], 4.48 * 0.01 * 2 + np.arange(128.0)) and np.isclose(y[0, 128], -448 * 3 + 128)
