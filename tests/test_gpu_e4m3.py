"""GPU parity of the 8-bit products against their definitions in float64 (oracle/dla.py), and the run of the
operators as a layer uses them: norm, 8-bit projection, linear attention, norm of each head, 8-bit projection.

Tolerances.
* scales: max / 448 rounded once: 2^-24.  Codes: within half a step of the exact quotient (2^-4 of it, or
  2^-10 among the subnormals) and 2^-22 for the rounded scale.
* the product: the sums of a block of 128 and of the blocks are held in fp32: exact products of e4m3, at most
  128 additions in a block, two roundings for the scales and one addition for each block: with the tensor
  cores' additions taken as off by up to 2^-22 of the terms' magnitudes each, 130 * 2^-22 < 2^-14 of the
  magnitudes; then one bf16 rounding, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import chunked_gated_delta_bwd_gb300 as gdr
from oracle import block as ref_block
from oracle import dla as ref
from tests.helpers import f64, rel_l2

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from chunked_gated_delta_bwd_gb300 import build
    build.build()


def _matrix(R, C, seed, dtype=F32):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(R, C, generator=gen) * torch.exp(3 * torch.randn(R, 1, generator=gen))
    return x.to(dtype).cuda()


def _check_codes(x, out, rows):
    x = f64(x)
    scale = ref.tile_scales(x, rows)
    assert out["scale"].shape == scale.shape
    assert np.all(np.abs(f64(out["scale"]) - scale) <= 2.0 ** -24 * scale)
    want = x / ref.spread(scale, rows, 128, x.shape)
    err = np.abs(f64(out["y"].float()).reshape(x.shape) - want)
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 2.0 ** -22 * np.abs(want))
    # the codes are those of the division by the stored scale, ties to even
    exact = torch.tensor(x / ref.spread(f64(out["scale"]), rows, 128, x.shape)).float().to(E4M3)
    far = f64(exact.float()) != f64(out["y"].float()).reshape(x.shape)
    assert far.mean() <= 1e-4, far.mean()  # (fp32 quotients next to a tie)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R,C", [(1, 2), (3, 128), (5, 130), (1, 6144), (129, 126), (127, 2048), (65, 258), (300, 200), (2, 4104)])
def test_quant_rows_and_tiles(R, C, dtype):
    x = _matrix(R, C, R + C, dtype)
    _check_codes(x, gdr.quant_e4m3(x), 1)
    a, b = gdr.quant_e4m3(x, tiles=True), gdr.quant_e4m3(x, tiles=True, transposed=True)
    _check_codes(x, a, 128)
    assert torch.equal(a["y"].view(torch.uint8), b["y"].view(torch.uint8)) and torch.equal(a["scale"], b["scale"])
    assert torch.equal(b["y_t"].view(torch.uint8), b["y"].view(torch.uint8).t()) and torch.equal(b["scale_t"], b["scale"].t())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quant_codes_are_those_of_the_division(dtype):
    """Code for code, also on ties (which ratios of bf16 numbers often are): the fp32 quotient, rounded to e4m3; scales
    of every size, down to where quotients of subnormal numbers are taken."""
    gen = torch.Generator().manual_seed(9)
    x = torch.randn(4096, 256, generator=gen) * torch.exp2(torch.linspace(-140, 110, 4096))[:, None]
    x[::7] = torch.round(x[::7] / x[::7].abs().amax(1, keepdim=True) * 64)
    x = x.to(dtype).cuda()
    for tiles in (False, True):
        q = gdr.quant_e4m3(x, tiles=tiles)
        s = q["scale"].repeat_interleave(128, dim=1)
        s = s.repeat_interleave(128, dim=0) if tiles else s
        # (float64 division of float32 numbers, rounded to float32, is the float32 division; scales that are subnormal
        # numbers are rounded so far that quotients pass 448, where the codes end)
        want = (x.double() / s.double()).float().clamp(-448, 448).to(E4M3)
        assert torch.equal(q["y"].view(torch.uint8), want.view(torch.uint8))


def test_quant_slices_shapes_and_zeros():
    wide = _matrix(40, 500, 1, BF16)
    for a, b in ((0, 256), (6, 300), (2, 4)):
        s, c = wide[:, a:b], wide[:, a:b].contiguous()
        for tiles in (False, True):
            x, y = gdr.quant_e4m3(s, tiles=tiles), gdr.quant_e4m3(c, tiles=tiles)
            assert torch.equal(x["y"].view(torch.uint8), y["y"].view(torch.uint8)) and torch.equal(x["scale"], y["scale"])
    t = gdr.quant_e4m3(wide.view(4, 10, 500))
    assert t["y"].shape == (4, 10, 500) and t["scale"].shape == (40, 4)
    assert gdr.quant_e4m3(wide[:0])["y"].shape == (0, 500) and gdr.quant_e4m3(wide[:0], tiles=True)["scale"].shape == (0, 4)
    z = torch.zeros(130, 200, device="cuda")
    z[0, 0], z[129, 199] = 1e-45, -3e38  # the smallest float32, nearly the largest
    for tiles in (False, True):
        q = gdr.quant_e4m3(z, tiles=tiles)
        assert float(q["y"][0, 0].float()) == 1.0 and float(q["y"][129, 199].float()) == -448.0
        assert (q["scale"] > 0).all() and float(q["scale"].flatten()[1]) == 1.0
    z[3, 5], z[4, 150] = float("inf"), float("nan")
    q = gdr.quant_e4m3(z)
    assert torch.isinf(q["scale"][3, 0]) and torch.isnan(q["y"][4, 150].float()) and torch.isfinite(q["scale"][4]).all()


def _operands(M, K, N, seed, blocks=True, bias=True):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x, w = gdr.quant_e4m3(_matrix(M, K, seed)), gdr.quant_e4m3(_matrix(N, K, seed + 1), tiles=True)
    xs = x["scale"] if blocks else torch.exp(n(M, 1)).cuda()
    return x["y"], xs.contiguous(), w["y"], w["scale"], n(N).cuda() if bias else None


def _check_linear(ops):
    y = f64(gdr.linear_e4m3(*ops))
    plain = [f64(t.float()) if t is not None else None for t in ops]
    want, size = ref.linear(*plain), ref.linear(*plain, magnitudes=True)
    assert y.shape == want.shape
    err = np.abs(y - want)
    assert np.all(err <= U * np.abs(want) * (1 + U) + 2.0 ** -14 * size), float((err / size).max())


@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 33, 64, 65, 128, 129, 200, 257, 500])
@pytest.mark.parametrize("K,N", [(16, 8), (128, 128), (144, 136), (512, 256), (912, 120), (2048, 264)])
def test_linear(M, K, N):
    _check_linear(_operands(M, K, N, M + K + N, blocks=(M + N // 8) % 3 != 0, bias=M % 2 == 0))


@pytest.mark.parametrize("M,K,N", [(1, 4096, 2048), (5, 2048, 6144), (3000, 256, 1032), (1500, 2064, 520), (4111, 128, 128), (40, 8192, 128)])
def test_linear_larger(M, K, N):
    _check_linear(_operands(M, K, N, 7))


def test_linear_shapes_out_and_specials():
    x, xs, w, ws, b = _operands(12, 256, 128, 3)
    y = gdr.linear_e4m3(x, xs, w, ws, bias=b)
    out = torch.empty(3, 4, 128, dtype=BF16, device="cuda")
    assert gdr.linear_e4m3(x.view(3, 4, 256), xs, w, ws, bias=b, out=out) is out and torch.equal(out.view(12, 128), y)
    assert gdr.linear_e4m3(x[:0], xs[:0], w, ws).shape == (0, 128)
    # a NaN code reaches its own row (of x) or column (of w) alone
    x, w = x.clone(), w.clone()
    x.view(torch.uint8)[5, 100] = 0x7F
    w.view(torch.uint8)[77, 3] = 0xFF
    bad = torch.isnan(gdr.linear_e4m3(x, xs, w, ws, bias=b))
    want = torch.zeros(12, 128, dtype=torch.bool, device="cuda")
    want[5], want[:, 77] = True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("M,K,N", [(5, 2048, 1024), (300, 1024, 384), (2000, 512, 512)])
def test_linear_same_every_time_in_graphs_and_on_streams(M, K, N):
    ops = _operands(M, K, N, 11)
    first = gdr.linear_e4m3(*ops)
    assert all(torch.equal(first, gdr.linear_e4m3(*ops)) for _ in range(5))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = gdr.linear_e4m3(*ops)
    y.zero_()
    graph.replay()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(first, y)
    got = []
    for s in streams * 2:
        with torch.cuda.stream(s):
            got.append(gdr.linear_e4m3(*ops))
    torch.cuda.synchronize()
    assert all(torch.equal(first, t) for t in got)


def test_gradient_through_a_projection():
    """dx = dy W with the weight's transposed codes: the product's own backward."""
    M, K, N = 130, 384, 256
    w = _matrix(N, K, 5)
    dy = _matrix(M, N, 6, BF16)
    wq, dq = gdr.quant_e4m3(w, tiles=True, transposed=True), gdr.quant_e4m3(dy)
    dx = f64(gdr.linear_e4m3(dq["y"], dq["scale"], wq["y_t"], wq["scale_t"]))
    values = lambda codes, scale, rows: f64(codes.float()) * ref.spread(f64(scale), rows, 128, codes.shape)  # noqa: E731
    vd, vw = values(dq["y"], dq["scale"], 1), values(wq["y"], wq["scale"], 128)
    want, size = vd @ vw, np.abs(vd) @ np.abs(vw)
    assert np.all(np.abs(dx - want) <= U * np.abs(want) * (1 + U) + 2.0 ** -14 * size)


def test_a_layer():
    """Norm, 8-bit projection, linear attention, the norm of each head, 8-bit projection; a prefill and its
    continuation by single tokens, against float64 from the same codes and the values that are handed on."""
    C, H, D, lens = 256, 4, 128, [200, 1, 140]
    gen = torch.Generator().manual_seed(17)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    T = sum(lens)
    x, res = n(T, C).to(BF16).cuda(), n(T, C).to(BF16).cuda()
    w1, w2 = torch.ones(C).cuda(), torch.ones(D).cuda()
    w_in = gdr.quant_e4m3((n(3 * H * D, C) * C ** -0.5).cuda(), tiles=True)
    w_out = gdr.quant_e4m3((n(C, H * D) * (H * D) ** -0.5).cuda(), tiles=True)
    g = torch.tensor([-0.5, -0.1, -0.02, -0.004]).cuda()
    cu = torch.tensor([0] + list(np.cumsum(lens)), device="cuda")

    def layer(x, res, attend):
        a = gdr.rmsnorm_fwd(x, w1, residual=res, quant="block")
        qkv = gdr.linear_e4m3(a["y"], a["scale"], w_in["y"], w_in["scale"])
        q, k, v = (t.unflatten(1, (H, D)) for t in qkv.split(H * D, dim=1))
        o = attend(q, k, v)
        b = gdr.rmsnorm_fwd(o.view(-1, D), w2, quant="token")
        y8, s8 = b["y"].view(-1, H * D), b["scale"].view(-1, H)
        return gdr.linear_e4m3(y8, s8, w_out["y"], w_out["scale"]), (a, qkv, o, y8, s8)

    kept = {}

    def attend(q, k, v):
        kept.update(gdr.dla_fwd(q, k, v, g, cu_seqlens=cu))
        return kept["o"]

    y, (a, qkv, o, y8, s8) = layer(x, res, attend)
    want_qkv = ref.linear(f64(a["y"].float()), f64(a["scale"]), f64(w_in["y"].float()), f64(w_in["scale"]))
    assert rel_l2(f64(qkv), want_qkv) <= U
    q, k, v = (t.reshape(T, H, D) for t in np.split(f64(qkv), 3, axis=1))
    want_o, want_t = ref.dla_fwd(q, k, v, f64(g), cu.tolist(), scale=D ** -0.5)
    assert rel_l2(f64(o), want_o) <= U and rel_l2(f64(kept["ht"]), want_t) <= 2.0 ** -16
    normed, _ = ref_block.rmsnorm(f64(o).reshape(-1, D), np.ones(D), 1e-6)
    got = f64(y8.float()).reshape(-1, D) * f64(s8).reshape(-1, 1)
    assert rel_l2(got, normed) <= 2.0 ** -4
    assert rel_l2(f64(y), ref.linear(f64(y8.float()), f64(s8), f64(w_out["y"].float()), f64(w_out["scale"]))) <= U
    # single tokens from the states: as a prefill that is one token longer
    x1, r1 = n(3, C).to(BF16).cuda(), n(3, C).to(BF16).cuda()
    pool = torch.zeros(5, H, D, D, device="cuda")
    slots = torch.tensor([4, 0, 2], device="cuda")
    pool[slots] = kept["ht"]
    y1, (_, qkv1, o1, _, _) = layer(x1, r1, lambda q, k, v: gdr.dla_step(q, k, v, g, pool, slots=slots))
    q, k, v = (t.reshape(3, H, D) for t in np.split(f64(qkv1), 3, axis=1))
    want_1, _ = ref.dla_fwd(q, k, v, f64(g), [0, 1, 2, 3], want_t, D ** -0.5)
    assert rel_l2(f64(o1), want_1) <= U and torch.isfinite(y1).all()
