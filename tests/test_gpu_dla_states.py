"""How exactly linear attention's fp32 states leave (ht of the forward, dh0 of the backward), state by state, against
the closed form of their sums in float64, for memories from one token to all of a sequence.

Tolerance, in the 2-norm of a state.  With f = w y in [2^E, 2^(E+1)), its bf16 rounding leaves r, evenly spread over +-2^(E-8), and
r's rounding is off by half a step of r's own binade, 2^(E-17) at most: 2^(2E-34) (1/2 + 1/16 + ...) / 3 in the mean square,
2^(E-17) 0.44 in the root, 2^-17 0.31 = 2.4e-6 of f (whose root mean square is 1.4 2^E).  fp32 adds up to 2^-23 for each addition of
the products of 16 tokens and a part to a sum (the tensor cores cut off; 16 for each chunk, of which the later ones count fully):
1.2e-7 sqrt 16 = 4.8e-7 in the root mean square.  Together 2.5e-6; 2^-18 = 3.8e-6 leaves half of it again for states whose f lie low
in their binades (0.44 2^-17 = 3.4e-6 where all do).  The terms of a few tokens share a few weights, whose products with y need not
spread evenly: below 32 tokens the bound of every term counts, 2^-17, and 2^-20 for fp32.  With growth the first tokens count most, and a chunk's growth (expf and its
argument: 2^-23 together) multiplies them once for each chunk that follows.
"""
import numpy as np
import pytest
import torch

import chunked_gated_delta_bwd_gb300 as gdr
from tests.test_gpu_dla import _built  # noqa: F401  (the fixture builds the library)

pytestmark = pytest.mark.gpu

DECAYS = [0.0, -1e-5, -1e-4, -1e-3, -4e-3, -0.008, -0.0117, -0.02, -0.05, -0.3, -1.0, -20.0, 1e-3, 0.01]
LENS = [[9000], [5000, 1, 3999, 0, 130], [128], [127, 129, 256, 3], [640, 5] * 20, [700] * 13 + [0], [130, 2000, 1, 128] * 4]


def _sums(a, b, n, g, init):
    """sum_t e^(g n_t) a_t b_t^T + e^(g len) init in float64: a, b [T, H, D], n [T], g [H], init [H, D, D]."""
    w = torch.exp(g[None, :] * n[:, None])
    return torch.einsum("thi,thj->hij", a * w[:, :, None], b) + torch.exp(g * len(n))[:, None, None] * init


@pytest.mark.parametrize("states", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "%dx%d" % (len(x), max(x)))
def test_states_one_by_one(lens, D, states):
    H, T, N = len(DECAYS), sum(lens), len(lens)
    gen = torch.Generator("cuda").manual_seed(D + T)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, dO = (n(T, H, D).to(torch.bfloat16) for _ in range(4))
    h0, dht = n(N, H, D, D), n(N, H, D, D)
    g = torch.tensor(DECAYS, device="cuda")
    ends = np.cumsum([0] + lens).tolist()
    cu = torch.tensor(ends, device="cuda")
    first = dict(h0=h0) if states else {}
    ht = gdr.dla_fwd(q, k, v, g, cu_seqlens=cu, **first)["ht"].double()
    dh0 = gdr.dla_bwd(q, k, v, g, dO, cu_seqlens=cu, scale=0.3, dht=dht if states else None, **first)["dh0"].double()
    q, k, v, dO, h0, dht = (t.double() for t in (q, k, v, dO, h0 * states, dht * states))
    scale = float(torch.tensor(0.3))  # (as the call's float32 has it)
    for s, (b, e) in enumerate(zip(ends[:-1], ends[1:])):
        at = torch.arange(e - b, device="cuda", dtype=torch.float64)
        for name, got, want in (("ht", ht[s], _sums(k[b:e], v[b:e], (e - b - 1) - at, g.double(), h0[s])),
                                ("dh0", dh0[s], _sums(scale * q[b:e], dO[b:e], at + 1, g.double(), dht[s]))):
            off = (got - want).flatten(1).norm(dim=1)
            size = want.flatten(1).norm(dim=1)
            # (where nothing but what has decayed to nothing is left, e^-104 and below counts as zero)
            growth = torch.where(g > 0, (e - b) / 128 * 2.0 ** -23, 0.0)
            bad = off > ((2.0 ** -18 if e - b >= 32 else 2.0 ** -17 + 2.0 ** -20) + growth) * size + 2.0 ** -140
            assert not bad.any(), (name, s, [(DECAYS[i], float(off[i] / size[i])) for i in bad.nonzero().flatten().tolist()])
