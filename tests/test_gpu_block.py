"""GPU parity of the recurrent block's operators against the float64 oracle (oracle/block.py).

Tolerances, relative L2 of a tensor unless said otherwise:
* bf16 results, element by element: half a bf16 step of the exact value (8 significant bits:
  2^(e-8) for |v| in [2^e, 2^(e+1))) for the one rounding at the end, and the bound of the
  operator's fp32 results for the arithmetic before it, of the larger of |v| and the tensor's
  root mean square (a sum that cancels keeps the error of its terms).
* fp32 results of the recurrence: one rounding of the decay (2^-24) and one of the state per
  token, over a memory of at most the longest test sequence, 650 tokens, all of one sign in the
  worst case: 650 * 2 * 2^-24 = 7.8e-5.  The softplus gate adds 3e-6 of the log gate, which a
  memory of 1 / |g| tokens turns into 3e-6 of the state.  8e-5.
* sums over tokens or rows whose terms cancel (dA_log, ddt_bias, dweight): 8e-5 of the sum of
  the terms' magnitudes, per channel.
* RMS norm: a sum of C squares is off by at most the depth of its longest chain of additions,
  below C / 64 + 12 roundings, half of which reach rstd: (C / 64 + 12) 2^-25 + 2^-22 (rsqrt).
* e4m3 codes: within half a step of the exact quotient (2^-4 of it, or 2^-10 among the
  subnormals), and 1e-4 of it for the fp32 arithmetic that chose the side; scales as rstd
  plus two roundings.
"""
import numpy as np
import pytest
import torch

import chunked_gated_delta_bwd_gb300 as gdr
from oracle import block as ref
from tests.helpers import f64, rel_l2

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TOL_STATE = 8e-5
TOL_TWO_ROUNDINGS = 2.0 ** -8  # two bf16 results of the same exact values, relative L2


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from chunked_gated_delta_bwd_gb300 import build
    build.build()


def _close(got, want, dtype, tol=TOL_STATE):
    """``got`` (float64 values of a tensor of ``dtype``) against the exact values."""
    if dtype == F32:
        return rel_l2(got, want) <= tol
    rms = np.sqrt(np.mean(want ** 2))
    half = np.where(want == 0, 0.0, 2.0 ** (np.floor(np.log2(np.where(want == 0, 1.0, np.abs(want)))) - 8))
    return bool(np.all(np.abs(got - want) <= half + tol * np.maximum(np.abs(want), rms)))


def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int64)


def _glr_inputs(lens, C, seed, act=BF16, gate_t=BF16, gate="log", states=True, split=False):
    gen = torch.Generator().manual_seed(seed)
    T, N = int(sum(lens)), len(lens)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = n(T, C).to(act)
    d = {"cu": _cu(lens)}
    if gate == "softplus":
        g = n(T, C).to(gate_t)
        d["A_log"], d["dt_bias"] = torch.rand(C, generator=gen) - 1.0, -5.0 * torch.rand(C, generator=gen)
    else:
        g = (-torch.nn.functional.softplus(n(T, C) - 6.0 * torch.rand(C, generator=gen))).to(gate_t)
    if split and act == gate_t:
        both = torch.cat([x, g, x], 1).cuda()
        d["x"], d["g"] = both[:, :C], both[:, C:2 * C]
    else:
        d["x"], d["g"] = x.cuda(), g.cuda()
    d["dh"] = n(T, C).to(act).cuda()
    if states:
        d["h0"], d["dht"] = n(N, C).cuda(), n(N, C).cuda()
    return d


def _params(d):
    return {k: d[k].cuda() for k in ("A_log", "dt_bias") if k in d}


def _ref_params(d):
    return {k: f64(d[k]) for k in ("A_log", "dt_bias") if k in d}


def _check_glr(d, gate, comp, dense=None, stream=None):
    """Forward and backward of one problem against the oracle; the backward takes the forward's h."""
    how = dict(gate=gate, complement=comp, **_params(d))
    h0, dht = d.get("h0"), d.get("dht")
    if dense:
        lay = lambda t: t.unflatten(0, dense)  # noqa: E731
        seqs = {}
    else:
        lay = lambda t: t  # noqa: E731
        seqs = {"cu_seqlens": d["cu"].cuda()}
    out = gdr.glr_fwd(lay(d["x"]), lay(d["g"]), h0=h0, **seqs, **how)
    assert out["h"].shape == lay(d["x"]).shape
    T, C = d["x"].shape
    h = out["h"].reshape(T, C)
    cu = d["cu"].tolist()
    want, want_t = ref.glr_fwd(f64(d["x"]), f64(d["g"]), cu, f64(h0), complement=comp, **_ref_params(d))
    act = d["x"].dtype
    assert _close(f64(h), want, act)
    assert rel_l2(f64(out["ht"]), want_t) <= TOL_STATE
    grad = gdr.glr_bwd(lay(d["x"]), lay(d["g"]), out["h"], lay(d["dh"]), h0=h0, dht=dht, **seqs, **how)
    back = ref.glr_bwd(f64(d["x"]), f64(d["g"]), f64(h), f64(d["dh"]), cu, f64(h0), f64(dht), complement=comp,
                       **_ref_params(d))
    assert _close(f64(grad["dx"]).reshape(T, C), back["dx"], act)
    assert _close(f64(grad["dg"]).reshape(T, C), back["dg"], d["g"].dtype)
    assert rel_l2(f64(grad["dh0"]), back["dh0"]) <= TOL_STATE
    if gate == "softplus":
        assert np.all(np.abs(f64(grad["dA_log"]) - back["dA_log"]) <= TOL_STATE * back["mA_log"] + 1e-30)
        assert np.all(np.abs(f64(grad["ddt_bias"]) - back["ddt_bias"]) <= TOL_STATE * back["mdt_bias"] + 1e-30)


TYPES = [(BF16, BF16), (BF16, F32), (F32, F32)]


@pytest.mark.parametrize("gate", ["log", "softplus"])
@pytest.mark.parametrize("comp", [False, True])
@pytest.mark.parametrize("types", range(3))
def test_glr_packed_sequences(gate, comp, types):
    # sequences of zero and one token, around multiples of 16 and 128, one over several hundred
    act, gt = TYPES[types]
    lens = [1, 0, 127, 128, 129, 0, 0, 15, 17, 1, 1, 650, 3, 16, 0]
    _check_glr(_glr_inputs(lens, 130, 10 + types, act, gt, gate), gate, comp)


@pytest.mark.parametrize("lens", [[1], [2], [0, 0, 1], [1] * 300, [128], [129], [300, 0], [64, 64, 64, 64]])
@pytest.mark.parametrize("C", [2, 64, 66])
def test_glr_lengths(lens, C):
    _check_glr(_glr_inputs(lens, C, 40 + C), "log", False)
    _check_glr(_glr_inputs(lens, C, 41 + C, states=False, gate="softplus"), "softplus", True)


@pytest.mark.parametrize("dense", [(1, 1), (1, 333), (3, 200), (5, 1), (2, 128), (40, 3)])
def test_glr_dense_layout_and_column_slices(dense):
    d = _glr_inputs([dense[1]] * dense[0], 96, 60, split=True)
    _check_glr(d, "log", True, dense=dense)
    d = _glr_inputs([dense[1]] * dense[0], 96, 61, F32, F32, "softplus", split=True)
    _check_glr(d, "softplus", False, dense=dense)


def test_glr_wide_channels():
    _check_glr(_glr_inputs([257, 100], 2050, 62, gate="softplus"), "softplus", True)


# Sequences far past one block's reach, where states travel through runs of chunks and of groups of
# chunks and through the stored states: log gates between 1 / 650 and 2 / 650, whose memory of at most
# 650 tokens is the one that the tolerances are derived for and carries a state over many chunks
# (C = 72: whole 16-byte pieces of a row; 66: not; 520: more tiles than are resident).
LONG = [([9000], 72, 0), ([9000], 66, 2), ([4096, 4096, 64], 72, 1), ([10, 8300, 0, 5, 63, 4097, 1], 66, 0),
        ([30, 4161, 1, 700, 0, 4099], 72, 2), ([9000], 520, 0), ([1] * 70 + [5000] + [9] * 130 + [2600], 520, 1)]


def _long_inputs(lens, C, types, gate):
    act, gt = TYPES[types]
    d = _glr_inputs(lens, C, 500 + C + len(lens), act, gt, gate)
    if gate == "log":
        gen = torch.Generator().manual_seed(C)
        d["g"] = (-(1.0 + 1.0 / 64 + 0.9 * torch.rand(sum(lens), C, generator=gen)) / 650.0).to(gt).cuda()
    return d


@pytest.mark.parametrize("gate", ["log", "softplus"])
@pytest.mark.parametrize("comp", [False, True])
@pytest.mark.parametrize("lens,C,types", LONG)
def test_glr_long_sequences(gate, comp, lens, C, types):
    _check_glr(_long_inputs(lens, C, types, gate), gate, comp)


@pytest.mark.parametrize("C", [512, 514])
def test_glr_calls_on_two_streams_at_once(C):
    """Two streams, each its own workspace (the second one's blocks wait for room behind the first's)."""
    ds = [_long_inputs([6000, 200, 3000], C, 0, gate) for gate in ("log", "softplus")]

    def run(d, gate):
        how = dict(gate=gate, cu_seqlens=d["cu_dev"], h0=d["h0"], **d["par"])
        f = gdr.glr_fwd(d["x"], d["g"], **how)
        b = gdr.glr_bwd(d["x"], d["g"], f["h"], d["dh"], dht=d["dht"], **how)
        return [f["h"], f["ht"]] + [b[k] for k in sorted(b) if b[k] is not None]

    for d in ds:
        d["cu_dev"], d["par"] = d["cu"].cuda(), _params(d)
    want = [run(d, gate) for d, gate in zip(ds, ("log", "softplus"))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(6):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(ds[i], ("log", "softplus")[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for outs in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


# Slow channels, each by itself, over 5000 tokens.  The state is rounded twice a token, at random:
# sqrt(5000) 2^-24 = 4.2e-6 of it; 1 - a is off by a few 2^-24 of itself (the softplus gate's polynomial:
# 2e-7), which the state follows, 6e-7.  1e-5.
def _slow(gate, C):
    gen = torch.Generator().manual_seed(400 + C)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    slow = torch.tensor([1e-2, 1e-3, 1e-4, 1e-5])[torch.arange(C) % 4]
    x, h0 = n(5000, C), n(1, C)
    if gate == "log":
        return x, h0, -slow * torch.exp(0.3 * n(5000, C)), {}
    # (softplus(z) is near e^z here)
    g = 0.3 * n(5000, C)
    return x, h0, g, {"A_log": torch.rand(C, generator=gen) - 0.5, "dt_bias": torch.log(slow)}


def _off(got, want):
    return np.sqrt(((f64(got) - want) ** 2).sum(0) / (want ** 2).sum(0))


@pytest.mark.parametrize("gate", ["log", "softplus"])
@pytest.mark.parametrize("C", [64, 66])
def test_glr_decay_of_slow_channels(gate, C):
    """The decay of h0 over many tokens, forward and (of dht) backward."""
    _, h0, g, par = _slow(gate, C)
    zero, par_gpu = torch.zeros_like(g), {k: v.cuda() for k, v in par.items()}
    out = gdr.glr_fwd(zero.cuda(), g.cuda(), h0=h0.cuda(), gate=gate, **par_gpu)
    want, _ = ref.glr_fwd(f64(zero), f64(g), [0, 5000], f64(h0), **{k: f64(v) for k, v in par.items()})
    assert _off(out["h"], want).max() <= 1e-5
    back = gdr.glr_bwd(zero.cuda(), g.cuda(), out["h"], zero.cuda(), dht=h0.cuda(), gate=gate, **par_gpu)
    want = ref.glr_bwd(f64(zero), f64(g), want, f64(zero), [0, 5000], None, f64(h0), **{k: f64(v) for k, v in par.items()})
    assert _off(back["dx"], want["dx"]).max() <= 1e-5


@pytest.mark.parametrize("gate", ["log", "softplus"])
@pytest.mark.parametrize("C", [64, 66])
def test_glr_complement_of_slow_channels(gate, C):
    """The input scale 1 - a to its own precision."""
    x, h0, g, par = _slow(gate, C)
    par_gpu, par = {k: v.cuda() for k, v in par.items()}, {k: f64(v) for k, v in par.items()}
    out = gdr.glr_fwd(x.cuda(), g.cuda(), h0=h0.cuda(), gate=gate, complement=True, **par_gpu)
    want, _ = ref.glr_fwd(f64(x), f64(g), [0, 5000], f64(h0), complement=True, **par)
    assert _off(out["h"], want).max() <= 1e-5
    # one token on a state of zero: y = (1 - a) x (the gate and three roundings)
    y = gdr.glr_step(x[:1].cuda(), g[:1].cuda(), torch.zeros(1, C, device="cuda"), gate=gate, complement=True, **par_gpu)
    want, _ = ref.glr_fwd(f64(x[:1]), f64(g[:1]), [0, 1], complement=True, **par)
    assert np.all(np.abs(f64(y) - want) <= 1e-6 * np.abs(want))


@pytest.mark.parametrize("types", range(3))
def test_glr_complement_keeps_the_state_at_decay_one(types):
    """A log gate of zero (either sign) passes the state on to the last bit, however large x is."""
    act, gt = TYPES[types]
    gen = torch.Generator().manual_seed(17)
    h0 = torch.randn(2, 72, generator=gen).to(act).float().cuda()
    x = (1e6 * torch.randn(300, 72, generator=gen)).to(act).cuda()
    g = torch.zeros(300, 72, dtype=gt, device="cuda")
    g[::2] = -0.0
    out = gdr.glr_fwd(x, g, h0=h0, cu_seqlens=_cu([130, 170]).cuda(), complement=True)
    assert torch.equal(out["ht"], h0)
    assert torch.equal(out["h"].float(), torch.cat([h0[:1].expand(130, 72), h0[1:].expand(170, 72)]))
    state = h0.clone()
    gdr.glr_step(x[:2], g[:2], state, complement=True)
    assert torch.equal(state, h0)


@pytest.mark.parametrize("gate", ["log", "softplus"])
@pytest.mark.parametrize("comp", [False, True])
def test_glr_every_channel_by_itself(gate, comp):
    """Relative L2 per channel, where the tests above take all channels together."""
    d = _glr_inputs([700, 0, 1, 1300], 130, 72, F32, F32, gate)
    how = dict(gate=gate, complement=comp, cu_seqlens=d["cu"].cuda(), h0=d["h0"], **_params(d))
    out = gdr.glr_fwd(d["x"], d["g"], **how)
    want, _ = ref.glr_fwd(f64(d["x"]), f64(d["g"]), d["cu"].tolist(), f64(d["h0"]), complement=comp, **_ref_params(d))
    assert _off(out["h"], want).max() <= TOL_STATE
    grad = gdr.glr_bwd(d["x"], d["g"], out["h"], d["dh"], dht=d["dht"], **how)
    back = ref.glr_bwd(f64(d["x"]), f64(d["g"]), f64(out["h"]), f64(d["dh"]), d["cu"].tolist(), f64(d["h0"]), f64(d["dht"]),
                       complement=comp, **_ref_params(d))
    for k in ("dx", "dg"):
        assert _off(grad[k], back[k]).max() <= TOL_STATE, k


def test_glr_gates_of_zero_and_infinity():
    # log gate 0 (nothing forgotten), -inf (everything forgotten) and large positive is not used;
    # the state stays finite and follows the definition exactly enough
    d = _glr_inputs([200, 130], 64, 63, F32, F32)
    d["g"][::7] = 0.0
    d["g"][5::50] = float("-inf")
    d["g"][3::9] = -200.0
    out = gdr.glr_fwd(d["x"], d["g"], h0=d["h0"], cu_seqlens=d["cu"].cuda())
    want, want_t = ref.glr_fwd(f64(d["x"]), f64(d["g"]), d["cu"].tolist(), f64(d["h0"]))
    assert rel_l2(f64(out["h"]), want) <= TOL_STATE and rel_l2(f64(out["ht"]), want_t) <= TOL_STATE


@pytest.mark.parametrize("g", [60.0, 88.0, 89.0, 100.0, 177.0, 1e4, float("inf")])
@pytest.mark.parametrize("types", range(3))
def test_glr_growth_keeps_its_sign(g, types):
    """A positive log gate multiplies the state by e^g, or by 2^127 where that is more; never by a wrapped exponent."""
    act, gt = TYPES[types]
    h0 = torch.tensor([[1e-30, -1e-30, 2e-30, 0.0]], device="cuda")
    x = torch.zeros(1, 4, dtype=act, device="cuda")
    gg = torch.full((1, 4), g, device="cuda").to(gt)
    want = f64(h0) * min(np.exp(float(gg[0, 0])) if g < 700 else np.inf, 2.0 ** 127)
    out = gdr.glr_fwd(x, gg, h0=h0)
    assert rel_l2(f64(out["ht"]), want) <= 1e-5  # a log gate of 88 is off by up to 2^-24 of itself, the decay by that of 88
    state = h0.clone()
    gdr.glr_step(x, gg, state)
    assert rel_l2(f64(state), want) <= 1e-5
    back = gdr.glr_bwd(x, gg, out["h"], x, h0=h0, dht=h0)
    assert rel_l2(f64(back["dh0"]), want) <= 1e-5


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_glr_one_sequence_does_not_reach_another(bad):
    # a NaN or an infinity in one packed sequence leaves every other sequence's results untouched
    lens = [200, 0, 300, 5, 150]
    d = _glr_inputs(lens, 66, 64, gate="softplus")
    seqs = dict(cu_seqlens=d["cu"].cuda(), gate="softplus", **_params(d))

    def both():
        f = gdr.glr_fwd(d["x"], d["g"], h0=d["h0"], **seqs)
        b = gdr.glr_bwd(d["x"], d["g"], f["h"], d["dh"], h0=d["h0"], dht=d["dht"], **seqs)
        return f, b

    f0, b0 = both()
    d["x"][300:310], d["dh"][400:403], d["h0"][2, 3], d["dht"][2] = bad, bad, bad, bad
    f1, b1 = both()
    keep = torch.ones(sum(lens), dtype=torch.bool)
    keep[200:500] = False
    for a, b in ((f0["h"], f1["h"]), (b0["dx"], b1["dx"]), (b0["dg"], b1["dg"])):
        assert torch.equal(a[keep], b[keep])
    others = [0, 1, 3, 4]
    assert torch.equal(f0["ht"][others], f1["ht"][others]) and torch.equal(b0["dh0"][others], b1["dh0"][others])
    assert not torch.isfinite(f1["h"][299:310].float()).all()


def test_glr_directional_differences():
    # the kernels alone: the loss of the float32 forward moved along a direction by +-eps against
    # the backward.  Central differences of a loss L with eps = 1/64: truncation of relative order
    # eps^2 (2.4e-4 times third derivatives of order one), rounding 2^-24 |terms| / eps ~ 4e-6
    d = _glr_inputs([140, 33], 64, 65, F32, F32, "softplus")
    how = dict(cu_seqlens=d["cu"].cuda(), gate="softplus", complement=True)
    base = {"x": d["x"], "g": d["g"], "h0": d["h0"], **_params(d)}

    def loss(v):
        o = gdr.glr_fwd(v["x"], v["g"], h0=v["h0"], A_log=v["A_log"], dt_bias=v["dt_bias"], **how)
        return float((o["h"].double() * d["dh"].double()).sum() + (o["ht"].double() * d["dht"].double()).sum())

    h = gdr.glr_fwd(base["x"], base["g"], h0=base["h0"], A_log=base["A_log"], dt_bias=base["dt_bias"], **how)["h"]
    grads = gdr.glr_bwd(base["x"], base["g"], h, d["dh"], h0=base["h0"], dht=d["dht"], A_log=base["A_log"],
                        dt_bias=base["dt_bias"], **how)
    eps = 1.0 / 64
    for name in base:
        grad = grads["d" + name].double()
        step = grad / grad.norm()  # along the gradient: the derivative is its norm, nothing cancels
        moved = [loss({**base, name: (base[name].double() + s * eps * step).float()}) for s in (1, -1)]
        got = (moved[0] - moved[1]) / (2 * eps)
        assert abs(got - float(grad.norm())) <= 2e-3 * float(grad.norm()), (name, got, float(grad.norm()))


def test_glr_bitwise_repeatable_and_other_stream():
    d = _glr_inputs([700, 1, 900], 192, 66, gate="softplus")
    seqs = dict(cu_seqlens=d["cu"].cuda(), gate="softplus", **_params(d))

    def both():
        f = gdr.glr_fwd(d["x"], d["g"], h0=d["h0"], **seqs)
        return {**f, **gdr.glr_bwd(d["x"], d["g"], f["h"], d["dh"], h0=d["h0"], dht=d["dht"], **seqs)}

    first = both()
    torch.cuda.synchronize()
    for _ in range(20):
        again = both()
        for k, v in first.items():
            assert torch.equal(v, again[k]), k
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = both()
    side.synchronize()
    for k, v in first.items():
        assert torch.equal(v, again[k]), k


def test_glr_graph_replay():
    d = _glr_inputs([600, 41], 128, 67)
    cu = d["cu"].cuda()
    ws = torch.empty(gdr.glr_workspace_bytes(d["x"], d["g"], cu_seqlens=cu), dtype=torch.uint8, device="cuda")
    want = gdr.glr_fwd(d["x"], d["g"], h0=d["h0"], cu_seqlens=cu, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gdr.glr_fwd(d["x"], d["g"], h0=d["h0"], cu_seqlens=cu, workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got["h"], want["h"]) and torch.equal(got["ht"], want["ht"])


def test_backward_and_steps_in_a_graph():
    """Captured calls replayed on new inputs: kernels launched ahead of the one before, steps in place."""
    d = _glr_inputs([600, 41], 128, 73, gate="softplus")
    how = dict(gate="softplus", complement=True, **_params(d))
    cu, s = d["cu"].cuda(), d["x"]
    w, rstd = torch.ones(128, device="cuda"), torch.ones(641, device="cuda")
    conv_w, conv_b = torch.full((128, 4), 0.25, device="cuda"), torch.zeros(128, device="cuda")
    taps, state = torch.zeros(8, 3, 128, dtype=BF16, device="cuda"), torch.zeros(8, 128, device="cuda")
    h = gdr.glr_fwd(d["x"], d["g"], cu_seqlens=cu, **how)["h"]

    def calls():
        out = dict(gdr.glr_bwd(d["x"], d["g"], h, d["dh"], cu_seqlens=cu, **how))
        out.update({"n" + k: v for k, v in gdr.rmsnorm_bwd(d["dh"], s, w, rstd).items()})
        out["c"] = gdr.conv1d_step(d["x"][:8], taps, conv_w, conv_b)
        out["y"] = gdr.glr_step(out["c"], d["g"][:8], state, **how)
        return out

    calls()  # (once outside the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for seed in (1, 2):
        d["x"].copy_(torch.randn(641, 128, generator=torch.Generator().manual_seed(seed)))
        d["dh"].copy_(d["dh"].flip(0))
        taps.zero_(), state.zero_()
        graph.replay()
        torch.cuda.synchronize()
        after = {k: v.clone() for k, v in got.items()}, taps.clone(), state.clone()
        taps.zero_(), state.zero_()
        want = calls()
        assert all(torch.equal(after[0][k], want[k]) for k in want) and torch.equal(after[1], taps) and torch.equal(after[2], state)


def test_glr_inconsistent_cu_seqlens_reported():
    d = _glr_inputs([100, 200], 64, 68)
    for cu in ([0, 200, 100], [0, 100, 299], [1, 100, 300], [0, 400, 300], [0, -5, 300]):
        ws = torch.zeros(gdr.glr_workspace_bytes(d["x"], d["g"], num_seqs=2), dtype=torch.uint8, device="cuda")
        if ws.numel() < (need := gdr.glr_workspace_bytes(d["x"], d["g"], cu_seqlens=d["cu"].cuda())):
            ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        bad = torch.tensor(cu, dtype=torch.int64, device="cuda")
        gdr.glr_fwd(d["x"], d["g"], cu_seqlens=bad, workspace=ws)
        assert gdr.workspace_status(ws) == 1, cu  # GDR_DEV_BAD_SEQLENS
        gdr.glr_bwd(d["x"], d["g"], d["x"], d["dh"], cu_seqlens=bad, workspace=ws)
        assert gdr.workspace_status(ws) == 1, cu
    gdr.glr_fwd(d["x"], d["g"], cu_seqlens=d["cu"].cuda(), workspace=ws)
    assert gdr.workspace_status(ws) == 0


@pytest.mark.parametrize("C", [1024, 1026])  # copies by tensor maps, by pairs of channels
@pytest.mark.parametrize("types", [0, 2])
@pytest.mark.parametrize("block", [0, 100])
def test_glr_wait_that_runs_out_is_reported(C, types, block):
    """A block that gives up stops those that wait for it; the status word says so, and the next call on
    the same workspace is right."""
    from chunked_gated_delta_bwd_gb300.block import test_stall_next_glr as stall_next
    act, gt = TYPES[types]
    d = _glr_inputs([3000, 64 * 80 - 3000], C, 71, act, gt, "softplus")
    how = dict(gate="softplus", cu_seqlens=d["cu"].cuda(), h0=d["h0"], **_params(d))
    ws = torch.empty(gdr.glr_workspace_bytes(d["x"], d["g"], cu_seqlens=how["cu_seqlens"], gate="softplus"), dtype=torch.uint8,
                     device="cuda")
    fwd = lambda: gdr.glr_fwd(d["x"], d["g"], workspace=ws, **how)  # noqa: E731
    want = fwd()
    bwd = lambda: gdr.glr_bwd(d["x"], d["g"], want["h"], d["dh"], dht=d["dht"], workspace=ws, **how)  # noqa: E731
    for call in (fwd, bwd):
        first = call()
        assert gdr.workspace_status(ws) == 0
        stall_next(block)
        call()
        assert gdr.workspace_status(ws) == 4  # GDR_DEV_TIMEOUT
        again = call()
        assert gdr.workspace_status(ws) == 0
        assert all(torch.equal(again[k], first[k]) for k in first)


def test_glr_no_tokens():
    x = torch.empty(0, 8, dtype=BF16, device="cuda")
    h0 = torch.randn(3, 8, device="cuda")
    cu = torch.zeros(4, dtype=torch.int64, device="cuda")
    out = gdr.glr_fwd(x, x, h0=h0, cu_seqlens=cu)
    assert out["h"].shape == (0, 8) and torch.equal(out["ht"], h0)
    p = torch.zeros(8, device="cuda")
    g = gdr.glr_bwd(x, x, x, x, dht=h0, cu_seqlens=cu, gate="softplus", A_log=p, dt_bias=p)
    assert torch.equal(g["dh0"], h0) and not g["dA_log"].any() and not g["ddt_bias"].any()


def test_glr_offsets_past_32_bits():
    # 2^20 + 77 tokens of 2050 channels: the last rows lie past 2^31 elements.  A tail of 2000
    # tokens computed alone, from a zero state 2000 tokens before its checked part, agrees: the
    # log gate -0.05 forgets e^-100 over it
    T, C = (1 << 20) + 77, 2050
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(T, C, generator=gen, device="cuda", dtype=BF16)
    g = torch.full((T, C), -0.05, dtype=BF16, device="cuda")
    out = gdr.glr_fwd(x, g)
    tail = gdr.glr_fwd(x[-4000:].clone(), g[-4000:].clone())
    assert rel_l2(f64(out["h"][-2000:]), f64(tail["h"][-2000:])) <= TOL_TWO_ROUNDINGS
    assert rel_l2(f64(out["ht"]), f64(tail["ht"])) <= TOL_STATE
    back = gdr.glr_bwd(x, g, out["h"], x)
    head = gdr.glr_bwd(x[:4000].clone(), g[:4000].clone(), out["h"][:4000].clone(), x[:4000].clone())
    assert rel_l2(f64(back["dx"][:2000]), f64(head["dx"][:2000])) <= TOL_TWO_ROUNDINGS
    assert rel_l2(f64(back["dh0"]), f64(head["dh0"])) <= TOL_STATE
    last = gdr.glr_bwd(x[-500:].clone(), g[-500:].clone(), out["h"][-500:].clone(), x[-500:].clone())
    assert rel_l2(f64(back["dg"][-499:]), f64(last["dg"][1:])) <= TOL_TWO_ROUNDINGS


@pytest.mark.parametrize("gate", ["log", "softplus"])
@pytest.mark.parametrize("comp", [False, True])
@pytest.mark.parametrize("act", [BF16, F32])
@pytest.mark.parametrize("rows,C", [(1, 2), (3, 130), (70, 512)])
def test_glr_step_on_a_pool(gate, comp, act, rows, C):
    d = _glr_inputs([1] * rows, C, 80, act, act, gate, split=True)
    pool = torch.randn(2 * rows + 1, C, device="cuda")
    slots = torch.randperm(2 * rows + 1, generator=torch.Generator().manual_seed(1))[:rows]
    slots[1::5] = -1
    slots[2::7] = 2 * rows + 1  # past the pool: treated as padding
    on = (slots >= 0) & (slots <= 2 * rows)
    state = pool.clone()
    y = gdr.glr_step(d["x"], d["g"], state, slots=slots.cuda(), gate=gate, complement=comp, **_params(d))
    want = f64(pool).copy()
    for i in np.nonzero(on.numpy())[0]:
        h, _ = ref.glr_fwd(f64(d["x"][i:i + 1]), f64(d["g"][i:i + 1]), [0, 1], want[slots[i]][None], complement=comp,
                           **_ref_params(d))
        want[slots[i]] = h[0]
    touched = slots[on].tolist()
    assert rel_l2(f64(state)[touched], want[touched]) <= 5e-6  # one token: the gate's 3e-6 and roundings
    rest = [i for i in range(2 * rows + 1) if i not in touched]
    assert torch.equal(state[rest], pool[rest])
    assert torch.equal(y[on.cuda()], state[slots[on].cuda()].to(act)) and not y[~on.cuda()].any()


def test_steps_continue_a_prefill():
    # prefill then single tokens gives the tail of one long prefill: conv -> recurrence
    gen = torch.Generator().manual_seed(9)
    N, P, S, C = 3, 37, 9, 64
    x = torch.randn(N, P + S, C, generator=gen).to(BF16).cuda()
    g = -torch.rand(N, P + S, C, generator=gen).to(BF16).cuda()
    w, b = torch.randn(C, 4, generator=gen).cuda() * 0.5, torch.randn(C, generator=gen).cuda()
    y = gdr.conv1d_fwd(x, w, b, want_state=True)
    whole = gdr.glr_fwd(y["y"], g)
    pre = gdr.conv1d_fwd(x[:, :P].contiguous(), w, b, want_state=True)
    st = gdr.glr_fwd(pre["y"], g[:, :P].contiguous())
    conv, state = pre["state"], st["ht"]
    for t in range(P, P + S):
        yt = gdr.conv1d_step(x[:, t], conv, w, b)
        assert torch.equal(yt, y["y"][:, t])
        ht = gdr.glr_step(yt, g[:, t], state)
        assert rel_l2(f64(ht), f64(whole["h"][:, t])) <= TOL_TWO_ROUNDINGS
    assert torch.equal(conv, y["state"]) and rel_l2(f64(state), f64(whole["ht"])) <= TOL_STATE


# ---------------------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------------------

def _tol_rstd(C):
    return (C / 64 + 12) * 2.0 ** -25 + 2.0 ** -22


def _norm_inputs(R, C, res, seed):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=gen).to(BF16).cuda()
    w = (1.0 + 0.2 * torch.randn(C, generator=gen)).cuda()
    r = None if res is None else (3.0 * torch.randn(R, C, generator=gen)).to(res).cuda()
    return x, w, r


NORM_SIZES = [(1, 2), (5, 64), (3, 66), (129, 128), (7, 130), (33, 512), (4, 1000), (2, 2048), (3, 4098), (2, 12290),
              (1, 40000)]


@pytest.mark.parametrize("R,C", NORM_SIZES)
@pytest.mark.parametrize("res", [None, BF16, F32])
def test_rmsnorm_forward(R, C, res):
    x, w, r = _norm_inputs(R, C, res, C)
    for quant in (None, "token", "block"):
        out = gdr.rmsnorm_fwd(x, w, residual=r, quant=quant)
        if r is None:
            s = x
        else:
            s = (x.float() + r.float()).to(res)
            assert torch.equal(out["residual"], s)
        y, rstd = ref.rmsnorm(f64(s), f64(w), 1e-6)
        assert np.max(np.abs(f64(out["rstd"]) / rstd - 1)) <= _tol_rstd(C)
        if quant is None:
            assert _close(f64(out["y"]), y, BF16)
            continue
        block = C if quant == "token" else 128
        scale = ref.block_scales(y, block)
        assert out["y"].dtype == torch.float8_e4m3fn and out["scale"].shape == scale.shape
        assert np.max(np.abs(f64(out["scale"]) / scale - 1)) <= _tol_rstd(C) + 4 * 2.0 ** -24
        v = y / np.repeat(scale, block, axis=1)[:, :C]
        err = np.abs(f64(out["y"].float()) - v)
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10) + 1e-4 * np.abs(v))


def test_rmsnorm_rows_of_zero_and_huge():
    # a zero row: y 0, scale 1; rows whose squares overflow to infinity give y 0 with finite
    # scales; a NaN stays in its row
    x, w, _ = _norm_inputs(6, 256, None, 3)
    x[1] = 0
    x[3] = 1e30
    x[4, 7] = float("nan")
    for quant in (None, "token", "block"):
        out = gdr.rmsnorm_fwd(x, w, quant=quant)
        y = out["y"].float()
        assert not y[1].any() and not y[3].any() and torch.isnan(y[4]).all() and torch.isfinite(y[[0, 2, 5]]).all()
        if quant:
            assert (out["scale"][1] == 1).all() and (out["scale"][3] == 1).all()
            assert torch.isfinite(out["scale"][[0, 2, 5]]).all()


@pytest.mark.parametrize("C", [64, 256, 1000, 12290, 40000])
@pytest.mark.parametrize("quant", ["token", "block"])
def test_rmsnorm_codes_of_tiny_values(C, quant):
    """Rows around the smallest floats, zeros among them: max |y| / 448 is subnormal or rounds to zero,
    and 448 / max |y| overflows.  Zeros are code 0, no code is NaN, and codes times scale are y to
    e4m3's half step and the subnormal scale's (2^-150 of up to 448 each)."""
    tiny = torch.tensor([1e-37, 1e-38, 1e-39, 1e-40, 0.0], dtype=F32)
    gen = torch.Generator().manual_seed(C)
    x = (torch.rand(5, C, generator=gen) + 0.5) * torch.sign(torch.randn(5, C, generator=gen)) * tiny[:, None]
    x[:, ::3] = 0
    x[:, 0] = tiny
    w = 1.0 + 0.2 * torch.randn(C, generator=gen)
    w[C // 2:] *= 1e-6  # blocks whose values are a millionth of the others': scales below the floats
    x, w = x.to(BF16).cuda(), w.cuda()
    out = gdr.rmsnorm_fwd(x, w, quant=quant)
    code, scale = f64(out["y"].float()), f64(out["scale"])
    assert np.isfinite(code).all() and np.isfinite(scale).all() and (scale > 0).all()
    y, _ = ref.rmsnorm(f64(x), f64(w), 1e-6)
    assert (code[y == 0] == 0).all()
    block = C if quant == "token" else 128
    scale = np.repeat(scale, block, axis=1)[:, :C]
    assert np.all(np.abs(code * scale - y) <= 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * scale + 1e-4 * np.abs(y) + 450 * 2.0 ** -150)


@pytest.mark.parametrize("R,C", [(40, 64), (9, 2048), (5, 8192), (3, 20000)])
@pytest.mark.parametrize("quant", ["token", "block"])
def test_rmsnorm_codes_are_of_the_quotient(R, C, quant):
    """The scale is max |y| / 448 and the code e4m3(y / scale), both to the last bit, for the float32 y
    = s rstd w of the returned rstd: also where the quotient lies next to the middle of two codes."""
    gen = torch.Generator().manual_seed(R)
    x = torch.sign(torch.randn(R, C, generator=gen))
    codes = torch.arange(1, 126, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    middle = (codes[1:] + codes[:-1]) / 2
    w = middle[torch.randint(0, 124, (C,), generator=gen)] * (447.0 + torch.rand(1, generator=gen)) / 448.0
    w[::64] = 447.7
    w = w * (1 + torch.randint(-2, 3, (C,), generator=gen) * 2.0 ** -23)
    x, w = x.to(BF16).cuda(), w.cuda()
    out = gdr.rmsnorm_fwd(x, w, quant=quant)
    y = (x.float() * out["rstd"][:, None] * w).cpu()
    block = C if quant == "token" else 128
    nb = -(-C // block)
    most = torch.nn.functional.pad(y.abs(), (0, nb * block - C)).view(R, nb, block).amax(2)
    scale = most / 448.0
    assert torch.equal(out["scale"].cpu(), scale)
    want = (y / scale.repeat_interleave(block, dim=1)[:, :C]).to(torch.float8_e4m3fn)
    assert torch.equal(out["y"].cpu().view(torch.uint8), want.view(torch.uint8))


def test_rmsnorm_layouts():
    # [B, T, H, D] per head, column slices of a wider tensor, no rows
    x, w, _ = _norm_inputs(24, 64, None, 8)
    whole = gdr.rmsnorm_fwd(x, w)
    heads = gdr.rmsnorm_fwd(x.reshape(2, 3, 4, 64), w)
    assert heads["y"].shape == (2, 3, 4, 64) and heads["rstd"].shape == (2, 3, 4)
    assert torch.equal(heads["y"].reshape(24, 64), whole["y"])
    wide = torch.zeros(24, 200, dtype=BF16, device="cuda")
    for at in (0, 2, 6, 64):
        wide[:, at:at + 64] = x
        assert torch.equal(gdr.rmsnorm_fwd(wide[:, at:at + 64], w)["y"], whole["y"])
    none = gdr.rmsnorm_fwd(x[:0], w, quant="block")
    assert none["y"].shape == (0, 64)
    back = gdr.rmsnorm_bwd(x[:0], x[:0], w, none["rstd"])
    assert back["dx"].shape == (0, 64) and not back["dweight"].any()


@pytest.mark.parametrize("R,C", NORM_SIZES + [(1031, 128), (2500, 66)])
@pytest.mark.parametrize("res", [None, BF16, F32])
def test_rmsnorm_backward(R, C, res):
    dy, w, s = _norm_inputs(R, C, res or BF16, C + 1)
    dres = None if res is None else torch.randn(R, C, generator=torch.Generator().manual_seed(2)).to(res).cuda()
    _, rstd = ref.rmsnorm(f64(s), f64(w), 1e-6)
    r32 = torch.tensor(rstd, dtype=F32, device="cuda")
    out = gdr.rmsnorm_bwd(dy, s, w, r32, dres=dres)
    dx, dw, mw = ref.rmsnorm_bwd(f64(dy), f64(s), f64(w), 1e-6, f64(dres))
    # fp32: the projection sum's chain, as rstd's, of terms that may cancel: at most sqrt(C) of
    # their size in dx's own scale; in practice a few roundings.  2e-5 for float32
    assert out["dx"].dtype == s.dtype and _close(f64(out["dx"]), dx, s.dtype, 2e-5)
    assert np.all(np.abs(f64(out["dweight"]) - dw) <= TOL_STATE * mw + 1e-30)
    again = gdr.rmsnorm_bwd(dy, s, w, r32, dres=dres)
    assert torch.equal(again["dx"], out["dx"]) and torch.equal(again["dweight"], out["dweight"])


@pytest.mark.parametrize("C", [2048, 4098, 5120, 8192, 12290, 16384, 20000])
@pytest.mark.parametrize("res", [None, BF16, F32])
def test_rmsnorm_rows_in_turn(C, res):
    """More rows than blocks, so that each walks several (one or more pieces a thread, rows past registers):
    every row as when it is alone, and dweight of every channel by itself."""
    R = 1300
    x, w, r = _norm_inputs(R, C, res, C)
    pick = [0, 1, 151, 152, 303, 304, 607, 608, 760, 1299]
    for quant in (None, "token", "block"):
        out = gdr.rmsnorm_fwd(x, w, residual=r, quant=quant)
        for i in pick:
            one = gdr.rmsnorm_fwd(x[i:i + 1].clone(), w, residual=None if r is None else r[i:i + 1].clone(), quant=quant)
            for k in one:
                assert torch.equal(out[k][i:i + 1].view(torch.uint8), one[k].view(torch.uint8)), (k, i)
    s = x if r is None else out["residual"]
    dy, dres = _norm_inputs(R, C, None, C + 3)[0], None if r is None else r.flip(0).contiguous()
    back = gdr.rmsnorm_bwd(dy, s, w, out["rstd"], dres=dres)
    for i in pick:
        one = gdr.rmsnorm_bwd(dy[i:i + 1].clone(), s[i:i + 1].clone(), w, out["rstd"][i:i + 1].clone(),
                              dres=None if dres is None else dres[i:i + 1].clone())
        assert torch.equal(back["dx"][i:i + 1], one["dx"]), i
    # float32 sums of 1300 terms: below 1300 / (number of partial sums) + 16 roundings, 2^-24 each, of the terms' magnitudes
    n = dy.double() * s.double() * out["rstd"].double()[:, None]
    assert ((back["dweight"].double() - n.sum(0)).abs() <= TOL_STATE * n.abs().sum(0)).all()


def test_rmsnorm_backward_of_no_rows():
    """Nothing but dweight and the workspace is needed, and nothing else is read."""
    from chunked_gated_delta_bwd_gb300 import block
    dw = torch.full((24,), 7.0, device="cuda")
    ws = torch.empty(block._lib().gdr_rmsnorm_workspace_bytes(0, 24), dtype=torch.uint8, device="cuda")
    rc = block._lib().gdr_rmsnorm_bwd(0, 24, None, None, 0, None, None, None, ws.data_ptr(), ws.numel(), None, dw.data_ptr(),
                                      torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and not dw.any()


@pytest.mark.parametrize("R,C", [(0, 64), (5, 64), (3, 40000)])
def test_rmsnorm_backward_leaves_a_clear_status_word(R, C):
    """gdr_workspace_status tells of the last call that used the workspace, not of an earlier one."""
    from chunked_gated_delta_bwd_gb300 import block
    dy, w, s = _norm_inputs(R, C, BF16, 12)
    ws = torch.full((block._lib().gdr_rmsnorm_workspace_bytes(R, C),), 255, dtype=torch.uint8, device="cuda")
    gdr.rmsnorm_bwd(dy, s, w, torch.ones(R, device="cuda"), workspace=ws)
    assert gdr.workspace_status(ws) == 0


def test_rmsnorm_offsets_past_32_bits():
    R, C = (1 << 20) + 3, 2050
    gen = torch.Generator("cuda").manual_seed(6)
    x = torch.randn(R, C, generator=gen, device="cuda", dtype=BF16)
    w = torch.rand(C, generator=gen, device="cuda") + 0.5
    out, tail = gdr.rmsnorm_fwd(x, w, quant="block"), gdr.rmsnorm_fwd(x[-9:].clone(), w, quant="block")
    assert torch.equal(out["y"][-9:].float(), tail["y"].float()) and torch.equal(out["scale"][-9:], tail["scale"])
    back, last = gdr.rmsnorm_bwd(x, x, w, out["rstd"]), gdr.rmsnorm_bwd(x[-9:].clone(), x[-9:].clone(), w, tail["rstd"])
    assert torch.equal(back["dx"][-9:], last["dx"])


# ---------------------------------------------------------------------------------------
# conv1d
# ---------------------------------------------------------------------------------------

def _conv_inputs(lens, C, K, seed, states):
    gen = torch.Generator().manual_seed(seed)
    T, N = int(sum(lens)), len(lens)
    return {"x": torch.randn(T, C, generator=gen).to(BF16).cuda(), "cu": _cu(lens),
            "w": (0.5 * torch.randn(C, K, generator=gen)).cuda(), "b": (0.1 * torch.randn(C, generator=gen)).cuda(),
            "state": torch.randn(N, K - 1, C, generator=gen).to(BF16).cuda() if states else None}


# z is a sum of K + 1 fp32 products of O(1) terms that may cancel; y is rounded once
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("states", [False, True])
@pytest.mark.parametrize("C", [2, 66, 516])
def test_conv_forward(K, silu, states, C):
    lens = [1, 0, 127, 129, 2, 3, 0, 1, 260, 64, 0]
    d = _conv_inputs(lens, C, K, 90 + K, states)
    out = gdr.conv1d_fwd(d["x"], d["w"], d["b"], state=d["state"], cu_seqlens=d["cu"].cuda(), silu=silu, want_state=True)
    y, new = ref.conv1d_fwd(f64(d["x"]), f64(d["w"]), f64(d["b"]), d["cu"].tolist(), silu, f64(d["state"]))
    assert _close(f64(out["y"]), y, BF16)
    assert np.array_equal(f64(out["state"]), new)


@pytest.mark.parametrize("dense", [(1, 1), (3, 2), (2, 300), (70, 1)])
def test_conv_forward_dense_slices_and_no_bias(dense):
    B, T = dense
    d = _conv_inputs([T] * B, 72, 4, 95, False)
    wide = torch.zeros(B * T, 200, dtype=BF16, device="cuda")
    wide[:, 6:78] = d["x"]
    out = gdr.conv1d_fwd(wide.reshape(B, T, 200)[..., 6:78], d["w"], silu=True)
    y, _ = ref.conv1d_fwd(f64(d["x"]), f64(d["w"]), None, d["cu"].tolist(), True)
    assert out["state"] is None and _close(f64(out["y"]).reshape(B * T, 72), y, BF16)


def test_conv_forward_inconsistent_cu_seqlens_stays_inside():
    d = _conv_inputs([100, 200], 64, 4, 96, True)
    for cu in ([0, 250, 100], [5, 100, 300], [0, 400, 300], [-3, -2, -1], [0, 1 << 40, 300]):
        out = gdr.conv1d_fwd(d["x"], d["w"], d["b"], state=d["state"], want_state=True,
                             cu_seqlens=torch.tensor(cu, dtype=torch.int64, device="cuda"))
        torch.cuda.synchronize()
        assert out["y"].shape == d["x"].shape


def test_conv_no_tokens_passes_the_state():
    d = _conv_inputs([0, 0], 8, 4, 97, True)
    out = gdr.conv1d_fwd(d["x"], d["w"], d["b"], state=d["state"], cu_seqlens=d["cu"].cuda(), want_state=True)
    assert torch.equal(out["state"], d["state"])


def test_conv_forward_offsets_past_32_bits():
    T, C = (1 << 20) + 5, 2050
    gen = torch.Generator("cuda").manual_seed(7)
    x = torch.randn(T, C, generator=gen, device="cuda", dtype=BF16)
    w = torch.randn(C, 4, generator=gen, device="cuda")
    out = gdr.conv1d_fwd(x, w, want_state=True)
    tail = gdr.conv1d_fwd(x[-50:].clone(), w, want_state=True)
    assert torch.equal(out["y"][-47:], tail["y"][3:]) and torch.equal(out["state"], tail["state"])


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("rows,C", [(1, 2), (37, 130)])
def test_conv_step_on_a_pool(K, rows, C):
    d = _conv_inputs([1] * rows, C, K, 98, False)
    pool = torch.randn(2 * rows, K - 1, C).to(BF16).cuda()
    slots = torch.randperm(2 * rows, generator=torch.Generator().manual_seed(2))[:rows]
    slots[1::5], slots[2::7] = -1, 2 * rows
    on = (slots >= 0) & (slots < 2 * rows)
    state = pool.clone()
    y = gdr.conv1d_step(d["x"], state, d["w"], d["b"], slots=slots.cuda())
    want = pool.clone()
    for i in torch.nonzero(on)[:, 0].tolist():
        s = int(slots[i])
        yi, new = ref.conv1d_fwd(f64(d["x"][i:i + 1]), f64(d["w"]), f64(d["b"]), [0, 1], True, f64(pool[s:s + 1]))
        want[s] = torch.tensor(new[0]).to(BF16)
        assert _close(f64(y[i]), yi[0], BF16)
    assert torch.equal(state, want) and not y[~on.cuda()].any()


# Steps of four channels a thread (rows of whole aligned pieces) and of two (all others).
@pytest.mark.parametrize("shift", [0, 2, 4])
@pytest.mark.parametrize("C", [4, 516, 518])
def test_steps_on_column_slices(shift, C):
    """x and g as slices at an offset of `shift` columns of wider rows, against the contiguous step's answer."""
    gen = torch.Generator().manual_seed(300 + C)
    rows, wide = 9, C + 12
    both = torch.randn(rows, 2 * wide, generator=gen).to(BF16).cuda()
    x, g = both[:, shift:shift + C], both[:, wide + shift:wide + shift + C]
    pool = torch.randn(rows, C, generator=gen).cuda()
    A_log, dt_bias = torch.rand(C, generator=gen).cuda() - 1.0, torch.randn(C, generator=gen).cuda()
    how = dict(gate="softplus", complement=True, A_log=A_log, dt_bias=dt_bias)
    state, again = pool.clone(), pool.clone()
    y = gdr.glr_step(x, g, state, **how)
    assert torch.equal(y, gdr.glr_step(x.contiguous(), g.contiguous(), again, **how)) and torch.equal(state, again)
    for i in range(rows):
        want, _ = ref.glr_fwd(f64(x[i:i + 1]), f64(g[i:i + 1]), [0, 1], f64(pool[i:i + 1]), complement=True,
                              A_log=f64(A_log), dt_bias=f64(dt_bias))
        assert rel_l2(f64(state[i]), want[0]) <= 5e-6  # one token: the gate's 3e-6 and roundings
    w, b = torch.randn(C, 4, generator=gen).cuda(), torch.randn(C, generator=gen).cuda()
    taps = torch.randn(rows, 3, C, generator=gen).to(BF16).cuda()
    state = taps.clone()
    y = gdr.conv1d_step(x, state, w, b)
    want, new = ref.conv1d_fwd(f64(x), f64(w), f64(b), list(range(rows + 1)), True, f64(taps))
    assert _close(f64(y), want, BF16)
    assert torch.equal(state, torch.tensor(new).to(BF16).cuda())
