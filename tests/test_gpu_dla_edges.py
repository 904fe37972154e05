"""Linear attention with a decay for each head at the edges of what its header allows.  Inputs as in test_gpu_dla.py."""
import pytest
import torch

import chunked_gated_delta_bwd_gb300 as gdr
from chunked_gated_delta_bwd_gb300 import api, dla
from tests.test_gpu_dla import _built, _inputs  # noqa: F401  (the fixture builds the library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hk", [4, 2, 1])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cu", [[0, 10, 5, 300], [1, 10, 20, 300], [0, 10, 20, 299], [0] + [9] * 40 + [301], [0] + [9, 8] * 20 + [300]])
def test_bad_sequence_borders_write_nothing(cu, D, Hk):
    """No output is touched, the gradients of shared heads among them; the workspace holds what an earlier call might have left."""
    H, N, T = 4, len(cu) - 1, 300
    d = _inputs([T], H, Hk, D, 94, states=False)
    cu = torch.tensor(cu, device="cuda")
    args = [d["q"], d["k"], d["v"], d["g"]]
    ws = torch.full((gdr.dla_workspace_bytes(*args, cu_seqlens=cu, backward=True),), 0x41, dtype=torch.uint8, device="cuda")
    states = torch.ones(N, H, D, D, device="cuda")
    out = {n: torch.full_like(t, 7.0) for n, t in dict(o=d["v"], ht=states, dq=d["q"], dk=d["k"], dv=d["v"], dh0=states).items()}
    P, L = dla._Call(*args, cu, None, None), dla._lib()
    at = lambda *names: [out[n].data_ptr() for n in names]  # noqa: E731
    plain, stream = [t.data_ptr() for t in args], torch.cuda.current_stream().cuda_stream
    assert L.dla_fwd(P.shape, *plain, states.data_ptr(), *at("o", "ht"), ws.data_ptr(), ws.numel(), stream) == 0
    assert api.workspace_status(ws) == api.GDR_DEV_BAD_SEQLENS
    ws.fill_(0x41)
    assert L.dla_bwd(P.shape, *plain, states.data_ptr(), d["dO"].data_ptr(), states.data_ptr(), ws.data_ptr(), ws.numel(),
                     *at("dq", "dk", "dv", "dh0"), stream) == 0
    assert api.workspace_status(ws) == api.GDR_DEV_BAD_SEQLENS
    for n, t in out.items():
        assert (t == 7.0).all(), n


@pytest.mark.parametrize("pooled", [False, True])
def test_steps_of_more_rows_than_a_grid(pooled):
    """The rows go out in two kernels, which are counted, and are those of two smaller calls."""
    rows, first, D = 65535 + 6, 65000, 64
    pool = rows + 3
    gen = torch.Generator("cuda").manual_seed(95)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v = (n(rows, 1, D).to(torch.bfloat16) for _ in range(3))
    g, state = torch.tensor([-0.1], device="cuda"), n(pool, 1, D, D)
    slots = None
    if pooled:
        slots = torch.randperm(pool, generator=gen, device="cuda")[:rows]
        slots[[5, rows - 2]] = torch.tensor([-1, pool], device="cuda")
    want = state.clone()
    parts = []
    for a, b in ((0, first), (first, rows)):
        mine = dict(slots=slots[a:b].clone()) if pooled else {}
        parts.append(gdr.dla_step(q[a:b].clone(), k[a:b].clone(), v[a:b].clone(), g, want if pooled else want[a:], **mine))
    api.profile_begin(2)
    o = gdr.dla_step(q, k, v, g, state, slots=slots)
    assert api.profile_end()["dla"][1] == 2
    assert torch.equal(o, torch.cat(parts)) and torch.equal(state, want)
    assert o[-1].any() and (not pooled or not o[rows - 2].any())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [5, 1000, 5003])
def test_what_is_not_finite_is_carried_along_a_shared_sequence(D, at):
    """One sequence, long enough that several blocks share it: a token's NaN reaches all that its decay reaches in
    fp32; where the decay is zero it is either carried on or gone, and nothing else comes of it."""
    T, decays = 9000, [0.0, -1e-3, -0.02, -0.05, -2.0]
    H = len(decays)
    d = _inputs([T], H, H, D, 96, decays=decays)
    call = lambda: {**gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"]),  # noqa: E731
                    **gdr.dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], h0=d["h0"], dht=d["dht"])}
    clean = call()
    keep = {n: d[n].clone() for n in ("v", "dO")}
    first = at // 128 * 128  # of the token's chunk
    rows = torch.arange(T, device="cuda")[:, None]
    for name, ahead, hit, state in (("v", rows - at, ("o", "dq"), "ht"), ("dO", at - rows, ("dk", "dv"), "dh0")):
        d[name][at] = float("nan")
        out = call()
        d[name].copy_(keep[name])
        # e^-100 = 3.7e-44, a subnormal number that is not zero; e^-104 rounds to zero
        reached = (ahead >= 0) & (ahead * -d["g"] < 100)
        before = rows < first if name == "v" else rows >= first + 128
        for n in hit:
            bad = torch.isnan(out[n])
            assert bad[reached.expand(T, H)].all(), (name, n)
            same = (out[n] == clean[n]).all(2)
            assert same[before.expand(T, H)].all(), (name, n)
            assert (bad.all(2) | same | ((rows >= first) & (rows < first + 128))).all(), (name, n)
        end = torch.isnan(out[state])[0].flatten(1)
        far = (T - at if name == "v" else at) * -d["g"]
        assert end[far < 100].all() and (end.all(1) | (out[state][0] == clean[state][0]).flatten(1).all(1)).all(), name


def test_states_past_32_bits():
    """More than 2^32 numbers of states, in sequences and in a pool: the last ones are those of a call of their own."""
    N, H, D = 70_000, 4, 128
    assert N * H * D * D > 1 << 32
    gen = torch.Generator("cuda").manual_seed(97)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, dO = (n(2 * N, H, D).to(torch.bfloat16) for _ in range(4))
    g, some = torch.tensor([-0.1, -0.01, -1.0, 0.0], device="cuda"), n(7, H, D, D)
    h0 = some.repeat(N // 7, 1, 1, 1)
    out = gdr.dla_fwd(q, k, v, g, h0=h0, num_seqs=N)
    grad = gdr.dla_bwd(q, k, v, g, dO, h0=h0, dht=h0, num_seqs=N)
    for s in (0, 33_000, N - 7):  # (a multiple of 7 beyond 2^31 numbers is near the second)
        s = s // 7 * 7
        tail = lambda t: t[2 * s:2 * s + 14].clone()  # noqa: E731
        a = gdr.dla_fwd(tail(q), tail(k), tail(v), g, h0=some, num_seqs=7)
        b = gdr.dla_bwd(tail(q), tail(k), tail(v), g, tail(dO), h0=some, dht=some, num_seqs=7)
        assert torch.equal(out["o"][2 * s:2 * s + 14], a["o"]) and torch.equal(out["ht"][s:s + 7], a["ht"])
        for name in ("dq", "dk", "dv"):
            assert torch.equal(grad[name][2 * s:2 * s + 14], b[name]), name
        assert torch.equal(grad["dh0"][s:s + 7], b["dh0"])
    del out, grad
    slots = torch.tensor([N - 1, 0, 40_000], device="cuda")
    part = h0[slots].clone()
    o = gdr.dla_step(q[:3], k[:3], v[:3], g, h0, slots=slots)
    assert torch.equal(o, gdr.dla_step(q[:3], k[:3], v[:3], g, part)) and torch.equal(h0[slots], part)
    assert torch.equal(h0[N - 2], some[5]) and torch.equal(h0[40_001], some[40_001 % 7])
