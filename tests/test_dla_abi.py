"""Refusals of linear attention with a decay for each head and of the 8-bit products, on the host: the C
ABI's argument checks (the pointers here are not device memory, so every call must be refused before any
launch) and the binding's checks."""
import pytest
import torch

import chunked_gated_delta_bwd_gb300 as gdr
from chunked_gated_delta_bwd_gb300 import build, dla, e4m3

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
MB = 1 << 20


def at(i):
    """Aligned addresses, far apart, that are never dereferenced."""
    return (i + 1) * 64 * MB


@pytest.fixture(scope="module")
def L():
    build.build()
    return dla._lib()


@pytest.fixture(scope="module")
def E(L):
    return e4m3._lib()


def _shape(**over):
    sh = dla.DlaShape(2, 256, 4, 2, 64, None, 0.125, 0, 0, 0)
    for k, v in over.items():
        setattr(sh, k, v)
    return sh


def _fwd(sh, need=1 << 24):
    return [sh, at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7), need, None]


def _bwd(sh, need=1 << 24):
    return [sh, at(0), at(1), at(2), at(3), at(4), at(5), at(6), at(7), need, at(8), at(9), at(10), at(11), None]


@pytest.mark.parametrize("over,code", [
    (dict(num_seqs=0), INVALID), (dict(total_tokens=-2), INVALID), (dict(total_tokens=255), INVALID),
    (dict(num_heads=0), INVALID), (dict(num_heads=3), INVALID), (dict(num_k_heads=3), INVALID), (dict(num_k_heads=-1), INVALID),
    (dict(num_heads=1 << 17), INVALID), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED),
    (dict(cu_seqlens=4100), INVALID), (dict(total_tokens=(1 << 30) + 2), INVALID), (dict(num_seqs=1 << 23), INVALID),
    (dict(total_tokens=1 << 30, num_heads=256), INVALID), (dict(total_tokens=1 << 62), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q_stride=120), INVALID), (dict(k_stride=132), INVALID), (dict(v_stride=248), INVALID), (dict(q_stride=-128), INVALID),
    (dict(v_stride=1 << 33), INVALID)])
def test_shapes_refused(L, over, code):
    sh = _shape(**over)
    assert L.dla_workspace_bytes(sh, 0) == 0 and L.dla_workspace_bytes(sh, 1) == 0
    assert L.dla_fwd(*_fwd(sh)) == code
    assert L.dla_bwd(*_bwd(sh)) == code
    assert L.gdr_last_error()


def test_pointers_refused(L):
    sh = _shape()
    need = L.dla_workspace_bytes(sh, 0)
    assert 0 < need <= L.dla_workspace_bytes(sh, 1)
    ok = _fwd(sh, need)
    for i in (1, 2, 3, 4, 6, 8):
        for bad in (None, at(40) + 2):
            assert L.dla_fwd(*ok[:i], bad, *ok[i + 1:]) == INVALID, (i, bad)
    for i in (5, 7):  # h0, ht may be NULL but not misaligned
        assert L.dla_fwd(*ok[:i], at(40) + 4, *ok[i + 1:]) == INVALID, i
    assert L.dla_fwd(*ok[:9], need - 1, None) == WORKSPACE
    need = L.dla_workspace_bytes(sh, 1)
    ok = _bwd(sh, need)
    for i in (1, 2, 3, 4, 6, 8, 10, 11, 12, 13):
        for bad in (None, at(40) + 2):
            assert L.dla_bwd(*ok[:i], bad, *ok[i + 1:]) == INVALID, (i, bad)
    for i in (5, 7):
        assert L.dla_bwd(*ok[:i], at(40) + 4, *ok[i + 1:]) == INVALID, i
    assert L.dla_bwd(*ok[:9], need - 1, *ok[10:]) == WORKSPACE


def test_shared_memory_refused(L):
    sh = _shape()  # q, k: 256 x 2 x 64 bf16 (64 KB), v, o: 128 KB, states: 128 KB
    ok = _fwd(sh)
    for i, bad in ((6, at(2)), (6, at(0) + 65520), (6, at(1) - 16), (7, at(4)), (7, at(4) + 131056), (8, at(6) + 16), (7, at(5)), (8, at(4)), (6, at(3))):
        assert L.dla_fwd(*ok[:i], bad, *ok[i + 1:]) == INVALID, i
        assert b"share" in L.gdr_last_error()
    wide = _shape(q_stride=1024)  # (the last token ends the extent)
    ok = _fwd(wide)
    assert L.dla_fwd(*ok[:6], at(0) + 2 * (255 * 1024 + 128) - 16, *ok[7:]) == INVALID
    ok = _bwd(sh)
    for i, bad in ((10, at(0)), (11, at(1)), (12, at(6) + 16), (13, at(7)), (13, at(4) - 16), (11, at(8)), (8, at(9)), (12, at(2))):
        assert L.dla_bwd(*ok[:i], bad, *ok[i + 1:]) == INVALID, i
        assert b"share" in L.gdr_last_error()


def test_steps_refused(L):
    ok = [3, 4, 2, 64, 5, 0.5, at(0), 0, at(1), 0, at(2), 0, at(3), at(4), at(5), at(6), None]
    for i, v, code in ((0, -1, INVALID), (1, 0, INVALID), (1, 5, INVALID), (2, 3, INVALID), (3, 32, UNSUPPORTED), (4, -1, INVALID),
                       (5, float("inf"), INVALID), (6, None, INVALID), (6, at(9) + 8, INVALID), (7, 100, INVALID), (8, None, INVALID),
                       (9, 130, INVALID), (10, at(9) + 4, INVALID), (11, 8, INVALID), (12, None, INVALID), (13, at(9) + 4, INVALID),
                       (14, None, INVALID), (14, at(9) + 8, INVALID), (15, None, INVALID), (15, at(2), INVALID), (14, at(6) + 16, INVALID)):
        assert L.dla_step(*ok[:i], v, *ok[i + 1:]) == code, (i, v)
    assert L.dla_step(6, 4, 2, 64, 5, 0.5, at(0), 0, at(1), 0, at(2), 0, at(3), None, at(5), at(6), None) == INVALID  # pool < rows
    assert L.dla_step(1 << 30, 4, 2, 64, 5, 0.5, at(0), 0, at(1), 0, at(2), 0, at(3), at(4), at(5), at(6), None) == INVALID


def test_quant_refused(E):
    ok = [3, 130, at(0), 0, 0, 1, at(1), at(2), at(3), at(4), None]
    for i, v, code in ((0, -1, INVALID), (0, 1 << 31, INVALID), (1, 0, INVALID), (1, 129, INVALID), (1, (1 << 28) + 2, INVALID),
                       (2, None, INVALID), (2, at(9) + 2, INVALID), (3, 128, INVALID), (3, 131, INVALID), (3, 1 << 39, INVALID),
                       (4, 2, UNSUPPORTED), (5, 0, INVALID), (6, None, INVALID), (6, at(9) + 8, INVALID), (7, None, INVALID),
                       (8, None, INVALID), (8, at(9) + 4, INVALID), (9, None, INVALID), (9, at(9) + 4, INVALID)):
        assert E.gdr_quant_e4m3(*ok[:i], v, *ok[i + 1:]) == code, (i, v)
    assert E.gdr_quant_e4m3((1 << 31) - 1, 1 << 20, *ok[2:]) == INVALID
    assert E.gdr_quant_e4m3(3, 130, at(0) + 4, 0, 1, 0, at(1), at(2), None, None, None) == INVALID


def test_linear_refused(E):
    ok = [3, 256, 128, at(0), at(1), 2, at(2), at(3), at(4), at(5), None]
    for i, v, code in ((0, -1, INVALID), (0, 1 << 31, INVALID), (1, 0, INVALID), (1, 264, INVALID), (1, 1 << 25, INVALID),
                       (2, 0, INVALID), (2, 132, INVALID), (2, 1 << 25, INVALID), (3, None, INVALID), (3, at(9) + 8, INVALID),
                       (4, None, INVALID), (4, at(9) + 4, INVALID), (5, 0, INVALID), (5, 3, INVALID), (6, None, INVALID),
                       (7, None, INVALID), (8, at(9) + 4, INVALID), (9, None, INVALID), (9, at(9) + 8, INVALID)):
        assert E.gdr_linear_e4m3(*ok[:i], v, *ok[i + 1:]) == code, (i, v)


def test_binding_refuses():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    g, s = torch.zeros(2), torch.zeros(4, 2, 64, 64)
    c = torch.zeros(4, 128).to(torch.float8_e4m3fn)
    for call in (lambda: gdr.dla_fwd(x, x, x, g), lambda: gdr.dla_bwd(x, x, x, g, x), lambda: gdr.dla_step(x, x, x, g, s),
                 lambda: gdr.dla_fwd(x[0], x[0], x[0], g), lambda: gdr.dla_step(x[0], x[0], x[0], g, s),
                 lambda: gdr.dla_fwd(None, x, x, g), lambda: gdr.dla_fwd(x.repeat(1, 1, 2), x.repeat(1, 1, 2), x, g), lambda: gdr.quant_e4m3(x.to(torch.float16)), lambda: gdr.quant_e4m3(x),
                 lambda: gdr.quant_e4m3(x, tiles=True), lambda: gdr.quant_e4m3(x[0], transposed=True), lambda: gdr.quant_e4m3(None),
                 lambda: gdr.linear_e4m3(c, torch.ones(4, 1), c, torch.ones(1, 1)), lambda: gdr.linear_e4m3(c, None, None, None)):
        with pytest.raises(ValueError):
            call()


def test_token_strides():
    class T:
        """A stand-in with the attributes the rule reads."""
        def __init__(self, t):
            self.t, self.dtype, self.shape, self.is_cuda, self.device = t, t.dtype, t.shape, True, "cuda"
        def is_contiguous(self):
            return self.t.is_contiguous()
        def stride(self):
            return self.t.stride()

    rule = lambda t: dla._tokens(T(t), t.shape, "q")  # noqa: E731
    wide = torch.zeros(2, 6, 512, dtype=torch.bfloat16)
    cut = lambda t, a, b: t[..., a:b].unflatten(-1, (-1, 64))  # noqa: E731
    assert rule(cut(wide, 0, 512)) == 512 and rule(cut(wide, 64, 192)) == 512 and rule(cut(wide[0], 8, 72)) == 512
    assert rule(cut(wide[:, :1], 0, 64)) == 6 * 512 and rule(cut(wide[:1, :1], 64, 192)) == 128
    for bad in (cut(wide[:, ::2][:, :2], 0, 64), cut(wide[:, :3], 0, 64), cut(wide, 0, 512)[:, :, ::2],
                cut(wide, 0, 512).transpose(1, 2), cut(wide[0, :1], 0, 64).expand(4, 1, 64), cut(wide, 0, 512)[..., ::2]):
        with pytest.raises(ValueError):
            rule(bad)
