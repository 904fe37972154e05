"""The 8-bit products at the edges of what their header allows.  Operands and tolerances as in test_gpu_e4m3.py."""
import pytest
import torch

import chunked_gated_delta_bwd_gb300 as gdr
from tests.test_gpu_e4m3 import _built, _check_linear, _operands  # noqa: F401  (the fixture builds the library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [3, 16, 29, 64])
@pytest.mark.parametrize("K,N,blocks", [(4096, 152 * 128, True), (4112, 153 * 128, True), (2048 + 16, 20000, False)])
def test_few_rows_through_many_turns_of_the_scales(M, K, N, blocks):
    """More tiles than multiprocessors, so that one block walks the whole inner dimension and its two halves of the
    scales' buffer are each filled again and again; the same bits every time."""
    ops = _operands(M, K, N, 21, blocks=blocks)
    _check_linear(ops)
    first = gdr.linear_e4m3(*ops)
    assert all(torch.equal(first, gdr.linear_e4m3(*ops)) for _ in range(20))


def _codes(t):
    return t.view(torch.uint8)


def test_quant_offsets_past_32_bits():
    """Matrices of more than 2^32 values: rows from all over are those of a call of their own, in every form."""
    R, C = 600_005, 8192
    assert R * C > 1 << 32
    x = torch.randn(20_000, C, device="cuda", generator=torch.Generator("cuda").manual_seed(5)).to(torch.bfloat16).repeat(R // 20_000 + 1, 1)[:R]
    x[-300:] *= 3
    rows = gdr.quant_e4m3(x)
    for a, b in ((0, 130), (262_100, 262_300), (R - 133, R)):  # (2^31 values before the second)
        part = gdr.quant_e4m3(x[a:b].clone())
        assert torch.equal(_codes(rows["y"][a:b]), _codes(part["y"])) and torch.equal(rows["scale"][a:b], part["scale"])
    del rows
    tiles = gdr.quant_e4m3(x, tiles=True, transposed=True)
    for a, b in ((0, 128), (262_144, 262_400), (R // 128 * 128, R)):  # (whole tiles)
        part = gdr.quant_e4m3(x[a:b].clone(), tiles=True, transposed=True)
        assert torch.equal(_codes(tiles["y"][a:b]), _codes(part["y"])) and torch.equal(_codes(tiles["y_t"])[:, a:b], _codes(part["y_t"]))
        s = slice(a // 128, -(-b // 128))
        assert torch.equal(tiles["scale"][s], part["scale"]) and torch.equal(tiles["scale_t"][:, s], part["scale_t"])


@pytest.mark.parametrize("tiles", [False, True])
def test_quant_of_the_most_rows(tiles):
    R = (1 << 31) - 1
    x = torch.zeros(R, 2, dtype=torch.bfloat16, device="cuda")
    x[-200:] = torch.randn(200, 2, device="cuda", generator=torch.Generator("cuda").manual_seed(6)).to(torch.bfloat16)
    q = gdr.quant_e4m3(x, tiles=tiles)
    n = 127 + (0 if tiles else 73)  # (the last tile has 127 rows)
    part = gdr.quant_e4m3(x[-n:].clone(), tiles=tiles)
    assert torch.equal(_codes(q["y"][-n:]), _codes(part["y"])) and torch.equal(q["scale"][-len(part["scale"]):], part["scale"])
    assert (q["scale"][::9_999_991] == 1).all() and not _codes(q["y"][::9_999_991]).any()


def test_linear_offsets_past_32_bits():
    """An output and a first operand of more than 2^32 values."""
    M, K, N = 750_001, 5760, 5768
    assert M * K > 1 << 32 and M * N > 1 << 32
    x, xs, w, ws, b = _operands(5000, K, N, 31)
    x, xs = x.view(torch.uint8).repeat(M // 5000 + 1, 1)[:M].view(x.dtype), xs.repeat(M // 5000 + 1, 1)[:M].contiguous()
    y = gdr.linear_e4m3(x, xs, w, ws, bias=b)
    first = y[:5000].clone()
    for a in (370_000, 745_000):
        assert torch.equal(y[a:a + 5000], first)
    assert torch.equal(y[750_000], first[0])
    _check_linear((x[:300].clone(), xs[:300].clone(), w, ws, b))


def test_linear_of_the_most_rows():
    M, K, N = (1 << 31) - 128, 16, 8
    x, xs, w, ws, b = _operands(1024, K, N, 33)
    want = gdr.linear_e4m3(x, xs, w, ws, bias=b)
    many, scales = torch.zeros(M, K, dtype=torch.uint8, device="cuda"), torch.ones(M, 1, device="cuda")
    for at in (0, 1 << 30, M - 1024):  # (blocks of 1024 rows from a tile's first row on)
        many[at:at + 1024], scales[at:at + 1024] = _codes(x), xs
    y = gdr.linear_e4m3(many.view(x.dtype), scales, w, ws, bias=b)
    for at in (0, 1 << 30, M - 1024):
        assert torch.equal(y[at:at + 1024], want)
    assert torch.equal(y[2048::7_000_003], b.to(torch.bfloat16).expand(len(y[2048::7_000_003]), N))
