"""GPU parity of linear attention with a decay for each head against the float64 oracle (oracle/dla.py).

Tolerances.  A bf16 rounding is off by at most u = 2^-8 of the value.
* o, dq, dk, dv, element by element: q k^T with its decays and the state are rounded to bf16 as the
  products' operands, u of each term's magnitude, and the result once more, u of its own; where value heads
  share q and k their gradients are summed in fp32.  The terms' magnitudes come from the oracle run on
  absolute values (which also bounds fp32's 2^-24 per operation, a few hundred of them at most: 2^-15).
  In the 2-norm over many elements a rounding counts with its root mean square, at most u / sqrt 3; three
  of them are u.
* ht, dh0: the tokens' terms are held in two bf16 numbers, u^2 = 2^-16 of a term's magnitude at most, and
  what fp32 adds: 2^-23 for each of at most a few hundred operations, below 2^-16: 2^-15 of the magnitudes
  element by element; 2^-16 in the 2-norm, where errors of either sign count with their root mean square.
* the step: the state is one multiply-add in fp32 (decay 2^-22, sum 2^-24 of the magnitudes: 2^-21), its
  output a sum of D terms and one rounding.
"""
import numpy as np
import pytest
import torch

import chunked_gated_delta_bwd_gb300 as gdr
from chunked_gated_delta_bwd_gb300 import api
from oracle import dla as ref
from tests.helpers import f64, rel_l2

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from chunked_gated_delta_bwd_gb300 import build
    build.build()


def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int64)


DECAYS = [-1e-4, -0.7, -0.01, 0.0, -1e-6, -3.0, -0.1, -40.0]


def _inputs(lens, H, Hk, D, seed, states=True, split=False, decays=None):
    gen = torch.Generator().manual_seed(seed)
    T, N = int(sum(lens)), len(lens)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = {"cu": _cu(lens), "g": torch.tensor((decays or DECAYS * 8)[:H], dtype=F32).cuda()}
    if split:
        both = n(T, (2 * Hk + H) * D + 8).to(BF16).cuda()
        d["q"], d["k"], d["v"] = (both[:, a:a + h * D].unflatten(1, (h, D)) for a, h in
                                  ((0, Hk), (Hk * D, Hk), (2 * Hk * D + 8, H)))
    else:
        d["q"], d["k"], d["v"] = (n(T, h, D).to(BF16).cuda() for h in (Hk, Hk, H))
    d["dO"] = n(T, H, D).to(BF16).cuda()
    d["h0"], d["dht"] = (n(N, H, D, D).cuda(), n(N, H, D, D).cuda()) if states else (None, None)
    return d


def _close(got, want, size, what, many=True):
    """A bf16 result against the exact values; ``size``: the sums of its terms' magnitudes."""
    err = np.abs(got - want)
    bad = err > U * np.abs(want) * (1 + U) + (2 * U + U * U + 2.0 ** -15) * size
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.nanmax(err)))
    assert np.isfinite(got).all(), what
    if many:
        assert rel_l2(got, want) <= U, (what, rel_l2(got, want))


def _close32(got, want, size, what):
    err = np.abs(got - want)
    # (a decay below 2^-126 is no normal fp32 number and may count as zero: e^-104 = 6.8e-46; the terms without
    # their decays sum to less than 2^16 here)
    assert np.all(err <= 2.0 ** -15 * size + 2.0 ** -110), (what, float((err / np.maximum(size, 1e-300)).max()))
    assert rel_l2(got, want) <= 2.0 ** -16, (what, rel_l2(got, want))


def _check(d, dense=None, scale=None, backward=True):
    """Forward and backward of one problem against the oracle."""
    D = d["v"].shape[-1]
    lay = (lambda t: t.unflatten(0, dense)) if dense else (lambda t: t)
    seqs = {} if dense else {"cu_seqlens": d["cu"].cuda()}
    cu = d["cu"].tolist()
    s = D ** -0.5 if scale is None else scale
    args = [lay(d[n]) for n in ("q", "k", "v")] + [d["g"]]
    plain = [f64(d[n]) for n in ("q", "k", "v", "g")]
    T = plain[2].shape[0]
    many = T * plain[2].shape[1] >= 64
    ws = torch.full((gdr.dla_workspace_bytes(*args, **seqs, backward=True),), 255, dtype=torch.uint8, device="cuda")
    out = gdr.dla_fwd(*args, h0=d["h0"], scale=scale, workspace=ws, **seqs)
    assert api.workspace_status(ws) == 0
    assert out["o"].shape == args[2].shape
    want, size = (ref.dla_fwd(*plain, cu, f64(d["h0"]), s, magnitudes=m) for m in (False, True))
    _close(f64(out["o"]).reshape(want[0].shape), want[0], size[0], "o", many)
    _close32(f64(out["ht"]), want[1], size[1], "ht")
    if not backward:
        return out
    grad = gdr.dla_bwd(*args, lay(d["dO"]), h0=d["h0"], dht=d["dht"], scale=scale, workspace=ws, **seqs)
    assert api.workspace_status(ws) == 0
    want, size = (ref.dla_bwd(*plain, f64(d["dO"]), cu, f64(d["h0"]), f64(d["dht"]), s, magnitudes=m) for m in (False, True))
    for n in ("dq", "dk", "dv"):
        assert grad[n].shape == args["qkv".index(n[1])].shape
        _close(f64(grad[n]).reshape(want[n].shape), want[n], size[n], n, many)
    _close32(f64(grad["dh0"]), want["dh0"], size["dh0"], "dh0")
    return {**out, **grad}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(3, 3), (4, 2), (4, 1)])
@pytest.mark.parametrize("states", [True, False])
def test_packed_sequences(D, heads, states):
    # sequences of zero and one token, around multiples of 16 and of the chunk of 128, and longer ones
    lens = [1, 0, 127, 128, 129, 0, 0, 15, 17, 1, 1, 650, 3, 256, 0]
    _check(_inputs(lens, *heads, D, 10, states=states))


@pytest.mark.parametrize("lens", [[1], [2], [0, 0, 1], [1] * 40, [128], [129], [300, 0], [64, 64, 64, 64], [0, 257]])
@pytest.mark.parametrize("D", [64, 128])
def test_lengths(lens, D):
    _check(_inputs(lens, 2, 2, D, 40))
    _check(_inputs(lens, 1, 1, D, 41, states=False), scale=-0.3)


@pytest.mark.parametrize("dense", [(1, 1), (1, 333), (3, 200), (5, 1), (2, 128), (40, 3), (2, 1025)])
@pytest.mark.parametrize("D", [64, 128])
def test_dense_layout_and_column_slices(dense, D):
    _check(_inputs([dense[1]] * dense[0], 2, 1, D, 60, split=True), dense=dense)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[9000], [5000, 1, 3999, 0, 130], [700] * 13])
def test_long_sequences(lens, D):
    """Sequences that are split over multiprocessors, at memories that end inside a part and that span all of it."""
    _check(_inputs(lens, 5, 5, D, 70, decays=[0.0, -1e-4, -0.05, -1.0, -0.003]))


@pytest.mark.parametrize("heads,D,dense", [((16, 4), 64, (19, 300)), ((6, 6), 128, (25, 260)), ((40, 40), 64, (1, 1300)),
                                           ((76, 2), 128, (1, 520)), ((150, 1), 64, (1, 640))])
def test_whole_chains_of_one_length(heads, D, dense):
    """As many chains as the blocks share evenly, or nearly: each block walks whole ones."""
    _check(_inputs([dense[1]] * dense[0], *heads, D, 70 + D, decays=DECAYS * 19), dense=dense)


# sequences too long to be walked whole beside many short ones, and empty ones
MIXED = [3000, 0, 129, 1, 700, 128, 127, 0, 640, 1300, 513, 2]


@pytest.mark.parametrize("lens,heads,D", [(MIXED, (12, 3), 64), (MIXED[::-1], (10, 10), 128),
                                          ([900, 0, 905, 1023, 1024, 1025, 130, 7], (30, 10), 64),
                                          ([5000] + [300] * 31, (6, 3), 64), ([300] * 31 + [3000], (6, 6), 128),
                                          ([130, 7, 513, 128, 300] * 8, (9, 3), 64), ([257, 1, 300] * 12 + [700], (12, 12), 64),
                                          ([257, 1, 300] * 12 + [700, 0], (12, 12), 64)])
def test_whole_chains_beside_ranges(lens, heads, D):
    _check(_inputs(lens, *heads, D, len(lens) + D, decays=DECAYS * 4))


def test_whole_chains_without_states_and_column_slices():
    _check(_inputs(MIXED, 10, 5, 128, 75, states=False, split=True, decays=DECAYS * 3))


@pytest.mark.parametrize("D", [64, 128])
def test_whole_chains_keep_what_is_not_finite(D):
    """The blocks that walk a chain of NaN go on with other chains, whose results are those of a clean call."""
    H = 12
    d = _inputs(MIXED, H, H, D, 76 + D, decays=DECAYS * 2)
    cu = d["cu"].cuda()
    call = lambda: {**gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], cu_seqlens=cu),  # noqa: E731
                    **gdr.dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], h0=d["h0"], dht=d["dht"], cu_seqlens=cu)}
    clean = call()
    hit = torch.zeros(len(MIXED), H, dtype=torch.bool)
    for seq, head, bad in ((0, 2, float("nan")), (4, 5, float("inf")), (9, 0, float("nan"))):
        hit[seq, head] = True
        a, b = d["cu"][seq].item(), d["cu"][seq + 1].item()
        for n in ("q", "k", "v", "dO"):
            d[n][a:b, head] = bad
        d["h0"][seq, head], d["dht"][seq, head] = bad, -bad
    rows = torch.repeat_interleave(~hit, torch.tensor(MIXED), dim=0).cuda()
    out = call()
    for n, t in out.items():
        keep = ~hit.cuda() if n in ("ht", "dh0") else rows
        assert torch.equal(t[keep], clean[n][keep]), n


def test_many_heads():
    _check(_inputs([300, 5, 129], 40, 8, 64, 75, decays=[-0.02 * i for i in range(40)]))


def test_many_sequences():
    _check(_inputs([3, 0, 1, 130] * 200, 1, 1, 64, 76))


@pytest.mark.parametrize("n", [31, 32, 33, 64])
def test_sequences_around_a_warp(n):
    _check(_inputs([(37 * i) % 150 for i in range(n)], 2, 2, 64, 77))


def test_very_many_sequences():
    """Tens of thousands of sequences of zero to two tokens, against the closed form."""
    lens = [1, 0, 2] * 15000
    d = _inputs(lens, 2, 2, 64, 78, states=False, decays=[-0.5, -0.1])
    cu = d["cu"].cuda()
    out = gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=cu)
    q, k, v = (d[n].double() for n in ("q", "k", "v"))
    first = torch.zeros(v.shape[0], dtype=torch.bool, device="cuda")
    first[cu[:-1][cu[1:] > cu[:-1]]] = True
    own = (q * k).sum(2, keepdim=True) * v
    before = torch.exp(d["g"].double())[:, None] * (q[1:] * k[:-1]).sum(2, keepdim=True) * v[:-1]
    own[1:] += torch.where(first[1:, None, None], 0.0, before)
    assert rel_l2(f64(out["o"]), f64(own * 64 ** -0.5)) <= U
    last = torch.cat([first[1:], torch.ones(1, dtype=torch.bool, device="cuda")])
    state = k[:, :, :, None] * v[:, :, None, :]
    state[1:] += torch.where(first[1:, None, None, None], 0.0, torch.exp(d["g"].double())[:, None, None] * state[:-1])
    assert not out["ht"][1::3].any()
    full = torch.ones(len(lens), dtype=torch.bool, device="cuda")
    full[1::3] = False
    assert rel_l2(f64(out["ht"][full]), f64(state[last])) <= 2.0 ** -16


def test_sequences_of_one_length_given_by_their_number():
    d = _inputs([200, 200, 200], 2, 1, 128, 79)
    a = gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], cu_seqlens=d["cu"].cuda())
    b = gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], num_seqs=3)
    assert _same(a, b)
    a = gdr.dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], h0=d["h0"], dht=d["dht"], cu_seqlens=d["cu"].cuda())
    b = gdr.dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], h0=d["h0"], dht=d["dht"], num_seqs=3)
    assert _same(a, b)


def test_offsets_past_32_bits():
    """v, o and the gradients beyond 2^32 elements: the last tokens, whose memory is short, are those of a call of their own."""
    H, D, T, tail = 40, 128, 850_000, 1500
    assert T * H * D > 1 << 32
    gen = torch.Generator("cuda").manual_seed(93)
    n = lambda t, h: torch.randn(t, h, D, generator=gen, device="cuda", dtype=BF16)  # noqa: E731
    q, k = n(T, 1), n(T, 1)
    v, dO = n(20_000, H).repeat(T // 20_000 + 1, 1, 1)[:T], n(10_000, H).repeat(T // 10_000, 1, 1)
    g = torch.full((H,), -0.3, device="cuda")
    out = gdr.dla_fwd(q, k, v, g)["o"]
    assert torch.isfinite(out[::997]).all()
    part = gdr.dla_fwd(q[-tail:], k[-tail:], v[-tail:].contiguous(), g)["o"]
    assert rel_l2(f64(out[-500:]), f64(part[-500:])) <= U
    del out, part
    cu = torch.tensor([0, 1000, T - 3000, T], device="cuda")
    grad = gdr.dla_bwd(q, k, v, g, dO, cu_seqlens=cu)
    part = gdr.dla_bwd(q[-3000:], k[-3000:], v[-3000:].contiguous(), g, dO[-3000:].contiguous())
    for name in ("dq", "dk", "dv"):
        assert rel_l2(f64(grad[name][-3000:]), f64(part[name])) <= U, name


def test_extreme_decays():
    """No memory at all (also by an infinite log decay), growth, a state that has to survive many tokens."""
    d = _inputs([200, 77], 6, 6, 64, 80, decays=[float("-inf"), -1e30, -104.0, 0.02, -1e-9, -20.0])
    out = _check(d, scale=1.0)
    assert torch.isfinite(out["dh0"]).all()


def test_scale_zero_and_large():
    d = _inputs([150], 2, 2, 64, 81)
    out = gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], scale=0.0)
    assert not out["o"].any() and out["ht"].any()
    _check(d, scale=1e4)


def test_no_tokens():
    e = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    g, h0 = torch.zeros(2, device="cuda"), torch.randn(3, 2, 64, 64, device="cuda")
    cu = torch.zeros(4, dtype=torch.int64, device="cuda")
    out = gdr.dla_fwd(e, e, e, g, h0=h0, cu_seqlens=cu)
    assert out["o"].shape == e.shape and torch.equal(out["ht"], h0)
    assert torch.equal(gdr.dla_bwd(e, e, e, g, e, dht=h0, cu_seqlens=cu)["dh0"], h0)
    assert not gdr.dla_bwd(e, e, e, g, e, h0=h0, cu_seqlens=cu)["dh0"].any()


def test_without_final_states():
    d = _inputs([300, 20], 2, 2, 128, 82)
    cu = d["cu"].cuda()
    a = gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], cu_seqlens=cu)
    b = gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], cu_seqlens=cu, want_ht=False)
    assert b["ht"] is None and torch.equal(a["o"], b["o"])


@pytest.mark.parametrize("D", [64, 128])
def test_what_is_not_finite_stays_in_its_sequence(D):
    """NaN and infinities of a neighbour inside the same chunk of memory reach nothing of another sequence."""
    lens = [70, 60, 130, 5, 200]
    d = _inputs(lens, 2, 2, D, 83)
    cu = d["cu"].cuda()
    call = lambda: {**gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], cu_seqlens=cu),  # noqa: E731
                    **gdr.dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], h0=d["h0"], dht=d["dht"], cu_seqlens=cu)}
    clean = call()
    bad = [1, 3]
    for i in bad:
        b, e = int(d["cu"][i]), int(d["cu"][i + 1])
        for n, x in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("dO", float("-inf"))):
            d[n][b:e] = x
        d["h0"][i], d["dht"][i] = float("nan"), float("inf")
    dirty = call()
    for i in set(range(len(lens))) - set(bad):
        b, e = int(d["cu"][i]), int(d["cu"][i + 1])
        for n in ("o", "dq", "dk", "dv"):
            assert torch.equal(clean[n][b:e], dirty[n][b:e]), (n, i)
        for n in ("ht", "dh0"):
            assert torch.equal(clean[n][i], dirty[n][i]), (n, i)


def test_causality_inside_a_chunk():
    """Finite changes to later tokens leave o of earlier ones as it was, bit for bit; to earlier tokens' dO
    the gradients dk, dv of later ones."""
    d = _inputs([400], 2, 2, 128, 84)
    fwd = lambda: gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"])["o"]  # noqa: E731
    bwd = lambda: gdr.dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"])  # noqa: E731
    o, grad = fwd(), bwd()
    keep = {n: d[n].clone() for n in ("q", "k", "v", "dO")}
    for n in ("k", "v"):
        d[n][173:] = 1e4
    assert torch.equal(fwd()[:173], o[:173])
    for n in keep:
        d[n].copy_(keep[n])
    d["q"][:230] = 1e4
    d["dO"][:230] = -1e4
    new = bwd()
    assert torch.equal(new["dk"][230:], grad["dk"][230:]) and torch.equal(new["dv"][230:], grad["dv"][230:])


@pytest.mark.parametrize("cu", [[0, 10, 5, 300], [1, 10, 20, 300], [0, 10, 20, 299], [0, -5, 20, 300], [0, 1 << 40, 20, 300]])
def test_bad_sequence_borders(cu):
    d = _inputs([300], 2, 2, 64, 85, states=False)
    cu = torch.tensor(cu, device="cuda")
    ws = torch.empty(gdr.dla_workspace_bytes(d["q"], d["k"], d["v"], d["g"], cu_seqlens=cu, backward=True), dtype=torch.uint8, device="cuda")
    gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=cu, workspace=ws)
    assert api.workspace_status(ws) == api.GDR_DEV_BAD_SEQLENS
    gdr.dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu_seqlens=cu, workspace=ws)
    assert api.workspace_status(ws) == api.GDR_DEV_BAD_SEQLENS
    many = torch.cat([cu[:-1], cu[-2:-1].clamp(0, 300).repeat(40), cu[-1:]])  # (more sequences than a warp has lanes)
    if (many[1:] < many[:-1]).any() or many[0] != 0 or many[-1] != 300:
        wide = torch.empty(gdr.dla_workspace_bytes(d["q"], d["k"], d["v"], d["g"], cu_seqlens=many, backward=True), dtype=torch.uint8, device="cuda")
        gdr.dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], cu_seqlens=many, workspace=wide)
        assert api.workspace_status(wide) == api.GDR_DEV_BAD_SEQLENS
    good = torch.tensor([0, 10, 20, 300], device="cuda")
    gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=good, workspace=ws)
    assert api.workspace_status(ws) == 0


def _same(a, b):
    return all(torch.equal(a[n], b[n]) for n in a if a[n] is not None)


@pytest.mark.parametrize("lens,H", [([300, 7], 2), ([9000, 40], 3), (MIXED, 16)])
def test_same_results_every_time_and_in_a_graph(lens, H):
    d = _inputs(lens, H, 1, 64, 86)
    cu = d["cu"].cuda()

    def call():
        return {**gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], cu_seqlens=cu),
                **gdr.dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], h0=d["h0"], dht=d["dht"], cu_seqlens=cu)}

    first = call()
    assert all(_same(first, call()) for _ in range(4))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(2):
        for t in out.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(first, out)
    d["v"].mul_(2)
    graph.replay()
    assert _same(call(), out)


def test_two_streams_at_once():
    ds = [_inputs([5000, 3], 4, 4, 64, 87), _inputs([77, 2000], 4, 4, 64, 88)]
    run = lambda d: {**gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], cu_seqlens=d["cu"].cuda()),  # noqa: E731
                     **gdr.dla_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], dht=d["dht"], cu_seqlens=d["cu"].cuda())}
    alone = [run(d) for d in ds]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                got.append(run(d))
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(alone, got))


# ------------------------------------------------------------------ single tokens

def _step_inputs(rows, H, Hk, D, pool, seed):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return [n(rows, h, D).to(BF16).cuda() for h in (Hk, Hk, H)] + [torch.tensor((DECAYS * 8)[:H]).cuda(), n(pool, H, D, D).cuda()], gen


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,H,Hk", [(1, 1, 1), (3, 4, 2), (5, 3, 3), (130, 8, 1)])
@pytest.mark.parametrize("pooled", [False, True])
def test_step(D, rows, H, Hk, pooled):
    pool = rows + 4
    (q, k, v, g, state), gen = _step_inputs(rows, H, Hk, D, pool, 90)
    slots = None
    at = list(range(rows))
    if pooled:
        at = torch.randperm(pool, generator=gen)[:rows].tolist()
        for i in range(1, rows, 3):
            at[i] = [-1, pool, -(1 << 40), 1 << 40][i % 4]
        slots = torch.tensor(at, device="cuda")
    old = state.clone()
    o = gdr.dla_step(q, k, v, g, state, slots=slots, scale=0.3)
    touched = set()
    for n, s in enumerate(at):
        if not 0 <= s < pool:
            assert not o[n].any()
            continue
        touched.add(s)
        args = [f64(t[n:n + 1]) for t in (q, k, v)] + [f64(g), [0, 1], f64(old[s:s + 1]), 0.3]
        (wo, ws), (mo, ms) = (ref.dla_fwd(*args, magnitudes=m) for m in (False, True))
        assert np.all(np.abs(f64(state[s]) - ws[0]) <= 2.0 ** -21 * ms[0])
        assert np.all(np.abs(f64(o[n]) - wo[0]) <= U * np.abs(wo[0]) * (1 + U) + 2.0 ** -16 * mo[0])
    for s in set(range(pool)) - touched:
        assert torch.equal(state[s], old[s])


def test_step_out_slices_and_graph():
    (q, k, v, g, state), _ = _step_inputs(6, 4, 4, 128, 6, 91)
    both = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
    sl = [t.unflatten(1, (4, 128)) for t in both.split(512, dim=1)]
    s1, s2 = state.clone(), state.clone()
    a = gdr.dla_step(q, k, v, g, s1)
    out = torch.empty_like(v)
    assert gdr.dla_step(*sl, g, s2, out=out) is out and torch.equal(a, out) and torch.equal(s1, s2)
    s3 = state.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = gdr.dla_step(*sl, g, s3)
    for _ in range(2):
        graph.replay()
    gdr.dla_step(q, k, v, g, s1)
    torch.cuda.synchronize()
    assert torch.equal(s1, s3) and torch.isfinite(b).all()


def test_steps_continue_a_prefill():
    lens, more = [130, 1, 40], 5
    d = _inputs([n + more for n in lens], 4, 2, 128, 92, states=False)
    cu = d["cu"].tolist()
    whole = gdr.dla_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=d["cu"].cuda())
    head = torch.cat([torch.arange(b, e - more) for b, e in zip(cu[:-1], cu[1:])]).cuda()
    out = gdr.dla_fwd(d["q"][head], d["k"][head], d["v"][head], d["g"], cu_seqlens=_cu(lens).cuda())
    state = out["ht"]
    for j in range(more):
        at = torch.tensor([e - more + j for e in cu[1:]]).cuda()
        o = gdr.dla_step(d["q"][at], d["k"][at], d["v"][at], d["g"], state)
        assert rel_l2(f64(o), f64(whole["o"][at])) <= 2 * U
    assert rel_l2(f64(state), f64(whole["ht"])) <= 2.0 ** -15
