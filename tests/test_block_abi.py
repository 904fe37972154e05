"""Refusals of the recurrent block's operators, on the host: the C ABI's argument checks (the
pointers here are not device memory, so every call must be refused before any launch) and the
binding's checks of types, shapes and strides."""
import ctypes

import pytest
import torch

import chunked_gated_delta_bwd_gb300 as gdr
from chunked_gated_delta_bwd_gb300 import block, build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
A = 4096  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return block._lib()


def _shape(**over):
    sh = block.GlrShape(2, 256, 8, None, 0, 0, 0, 0, 0, 0)
    for k, v in over.items():
        setattr(sh, k, v)
    return sh


@pytest.mark.parametrize("over,code", [
    (dict(num_seqs=0), INVALID), (dict(total_tokens=-2), INVALID), (dict(total_tokens=255), INVALID),
    (dict(channels=0), INVALID), (dict(channels=7), INVALID), (dict(gate=2), INVALID),
    (dict(act_type=2), UNSUPPORTED), (dict(gate_type=-1), UNSUPPORTED),
    (dict(act_type=1, gate_type=0), UNSUPPORTED), (dict(x_stride=6), INVALID), (dict(g_stride=9), INVALID),
    (dict(total_tokens=1 << 38), INVALID)])
def test_glr_shapes_refused(L, over, code):
    sh = _shape(**over)
    assert L.glr_workspace_bytes(sh) == 0
    assert L.glr_fwd(sh, A, A, A, A, None, A, None, A, 1 << 40, None) == code
    assert L.glr_bwd(sh, A, A, A, A, A, None, A, None, A, 1 << 40, A, A, A, A, A, None) == code
    assert L.gdr_last_error()


def test_glr_pointers_refused(L):
    sh = _shape(gate=1, complement=1)
    need = L.glr_workspace_bytes(sh)
    assert need > 0
    args = [sh, A, A, A, A, None, A, None, A, need, None]
    for i in (1, 2, 3, 4, 6, 8):
        for bad in (None, A + 2):
            assert L.glr_fwd(*args[:i], bad, *args[i + 1:]) == INVALID, (i, bad)
    for i in (5, 7):  # h0, ht may be NULL but not misaligned
        assert L.glr_fwd(*args[:i], A + 4, *args[i + 1:]) == INVALID, i
    assert L.glr_fwd(*args[:9], need - 1, None) == WORKSPACE
    args = [sh, A, A, A, A, A, None, A, None, A, need, A, A, A, A, A, None]
    for i in (1, 2, 3, 4, 5, 7, 9, 11, 12, 13, 14, 15):
        for bad in (None, A + 2):
            assert L.glr_bwd(*args[:i], bad, *args[i + 1:]) == INVALID, (i, bad)
    assert L.glr_bwd(*args[:10], need - 1, *args[11:]) == WORKSPACE


@pytest.mark.parametrize("tokens,channels,seqs", [
    (1 << 36, 1 << 30, 1), (1 << 36, 1 << 28, 1), (1 << 20, (1 << 20) + 2, 1), (1 << 36, 32, 1), (1 << 37, 2, 1),
    (2, (1 << 28) + 2, 1), (0, 1 << 28, 1 << 30)])
def test_sizes_past_the_limits_refused(L, tokens, channels, seqs):
    """Also where the product of the sizes leaves 64 bits."""
    sh = _shape(total_tokens=tokens, channels=channels, num_seqs=seqs)
    assert L.glr_workspace_bytes(sh) == 0
    assert L.glr_fwd(sh, A, A, None, None, None, A, None, A, (1 << 63) - 1, None) == INVALID
    assert L.glr_bwd(sh, A, A, None, None, A, None, A, None, A, (1 << 63) - 1, A, A, A, None, None, None) == INVALID
    assert L.gdr_conv1d_fwd(seqs, tokens, channels, 4, None, A, 0, A, None, None, 1, A, None, None) == INVALID


def test_channels_and_strides_past_the_limits_refused(L):
    C = (1 << 28) + 2
    assert L.glr_step(3, C, 3, 0, 0, 0, 0, A, 0, A, 0, None, None, None, A, A, None) == INVALID
    assert L.gdr_conv1d_step(3, C, 4, 3, A, 0, A, A, None, None, 1, A, None) == INVALID
    assert L.gdr_rmsnorm_fwd(3, C, A, 0, None, 0, A, 1e-6, 0, A, None, None, A, None) == INVALID
    assert L.gdr_rmsnorm_workspace_bytes(3, C) == 0
    assert L.gdr_rmsnorm_bwd(3, C, A, A, 0, A, A, None, A, 1 << 62, A, A, None) == INVALID
    assert L.glr_fwd(_shape(x_stride=1 << 62), A, A, None, None, None, A, None, A, 1 << 62, None) == INVALID
    assert L.glr_workspace_bytes(_shape(total_tokens=1 << 20, channels=1 << 20)) > 0


def test_states_that_share_memory_refused(L):
    """Buffers of two sequences' states (2 x 8 float32) and of 256 x 8 bf16 tokens, at distinct addresses but
    for the pair in question."""
    sh = _shape()
    need = L.glr_workspace_bytes(sh)
    at = lambda i: A + i * (1 << 20)  # noqa: E731
    for ht in (at(2), at(2) + 32, at(2) - 48):
        assert L.glr_fwd(sh, at(0), at(1), None, None, at(2), at(3), ht, at(4), need, None) == INVALID, ht
        assert b"share" in L.gdr_last_error()
    call = lambda dx, dg, dh0: L.glr_bwd(sh, at(0), at(1), None, None, at(2), at(3), at(4), at(5), at(6), need,  # noqa: E731
                                         dx, dg, dh0, None, None, None)
    for bad in ((at(7), at(8), at(3)), (at(7), at(8), at(5)), (at(7), at(8), at(5) + 16), (at(2), at(8), at(9)),
                (at(7), at(2), at(9)), (at(2) + 4080, at(8), at(9)), (at(7), at(2) - 16, at(9))):
        assert call(*bad) == INVALID, bad
        assert b"share" in L.gdr_last_error()
    for new in (at(3), at(3) + 80, at(3) - 80):  # states: 2 x 3 x 8 bf16
        assert L.gdr_conv1d_fwd(2, 256, 8, 4, None, at(0), 0, at(1), None, at(3), 1, at(2), new, None) == INVALID
        assert b"share" in L.gdr_last_error()


def test_steps_refused(L):
    ok = [3, 8, 5, 1, 0, 0, 0, A, 0, A, 0, A, A, A, A, A, None]
    for i, v, code in ((0, -1, INVALID), (1, 5, INVALID), (2, -1, INVALID), (3, 7, INVALID), (5, 3, UNSUPPORTED),
                       (7, None, INVALID), (7, A + 2, INVALID), (8, 4, INVALID), (9, None, INVALID), (10, 11, INVALID),
                       (11, None, INVALID), (12, None, INVALID), (13, A + 4, INVALID), (14, None, INVALID),
                       (15, None, INVALID), (15, A + 8, INVALID)):
        assert L.glr_step(*ok[:i], v, *ok[i + 1:]) == code, (i, v)
    assert L.glr_step(9, 8, 5, 0, 0, 0, 0, A, 0, A, 0, None, None, None, A, A, None) == INVALID  # pool < rows
    ok = [3, 8, 4, 5, A, 0, A, A, A, A, 1, A, None]
    for i, v, code in ((0, -1, INVALID), (1, 5, INVALID), (2, 0, UNSUPPORTED), (2, 5, UNSUPPORTED), (3, -1, INVALID),
                       (4, None, INVALID), (4, A + 2, INVALID), (5, 4, INVALID), (6, None, INVALID),
                       (7, None, INVALID), (8, A + 4, INVALID), (9, A + 4, INVALID), (11, None, INVALID)):
        assert L.gdr_conv1d_step(*ok[:i], v, *ok[i + 1:]) == code, (i, v)


def test_conv_forward_refused(L):
    ok = [2, 256, 8, 4, None, A, 0, A, A, A, 1, A, A + 64, None]
    for i, v, code in ((0, 0, INVALID), (1, 255, INVALID), (1, -2, INVALID), (2, 7, INVALID), (3, 0, UNSUPPORTED),
                       (3, 5, UNSUPPORTED), (5, None, INVALID), (5, A + 2, INVALID), (6, 7, INVALID),
                       (7, None, INVALID), (8, A + 4, INVALID), (9, A + 4, INVALID), (9, A + 64, INVALID),
                       (11, None, INVALID), (12, A + 4, INVALID)):
        assert L.gdr_conv1d_fwd(*ok[:i], v, *ok[i + 1:]) == code, (i, v)


def test_norm_refused(L):
    ok = [3, 8, A, 0, A, 0, A, 1e-6, 2, A, A, A, A, None]
    for i, v, code in ((0, -1, INVALID), (0, 1 << 31, INVALID), (1, 0, INVALID), (1, 9, INVALID), (2, None, INVALID),
                       (2, A + 2, INVALID), (3, 6, INVALID), (4, A + 4, INVALID), (5, 2, UNSUPPORTED),
                       (6, None, INVALID), (7, -1.0, INVALID), (7, float("nan"), INVALID), (8, 3, INVALID),
                       (9, None, INVALID), (10, None, INVALID), (11, None, INVALID), (12, None, INVALID)):
        assert L.gdr_rmsnorm_fwd(*ok[:i], v, *ok[i + 1:]) == code, (i, v)
    need = L.gdr_rmsnorm_workspace_bytes(3, 8)
    assert need > 0 and L.gdr_rmsnorm_workspace_bytes(3, 7) == 0
    ok = [3, 8, A, A, 1, A, A, A, A, need, A, A, None]
    for i, v, code in ((0, -1, INVALID), (1, 3, INVALID), (2, None, INVALID), (3, None, INVALID), (4, 5, UNSUPPORTED),
                       (5, None, INVALID), (6, None, INVALID), (7, A + 4, INVALID), (8, None, INVALID),
                       (9, need - 1, WORKSPACE), (10, None, INVALID), (11, None, INVALID)):
        assert L.gdr_rmsnorm_bwd(*ok[:i], v, *ok[i + 1:]) == code, (i, v)


def test_binding_refuses_what_is_not_on_the_gpu():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8)
    for call in (lambda: gdr.glr_fwd(x, x), lambda: gdr.glr_bwd(x, x, x, x),
                 lambda: gdr.glr_step(x, x, torch.zeros(4, 8)), lambda: gdr.rmsnorm_fwd(x, w),
                 lambda: gdr.rmsnorm_bwd(x, x, w, torch.zeros(4)), lambda: gdr.conv1d_fwd(x, torch.zeros(8, 4)),
                 lambda: gdr.conv1d_step(x, torch.zeros(4, 3, 8, dtype=torch.bfloat16), torch.zeros(8, 4)),
                 lambda: gdr.glr_fwd(x, x, gate="tanh"), lambda: gdr.rmsnorm_fwd(x, w, quant="int4")):
        with pytest.raises(ValueError):
            call()


def test_row_strides():
    # the stride rule itself, on the host: slices of one row stride pass, others are refused
    class T:
        """A stand-in with the attributes the rule reads."""
        def __init__(self, t):
            self.t, self.dtype, self.shape, self.is_cuda, self.device = t, t.dtype, t.shape, True, "cuda"
        def is_contiguous(self):
            return self.t.is_contiguous()
        def stride(self):
            return self.t.stride()

    rule = lambda t: block._rows(T(t), (torch.bfloat16,), t.shape, "x")  # noqa: E731
    wide = torch.zeros(2, 6, 32, dtype=torch.bfloat16)
    assert rule(wide) == 32 and rule(wide[..., 8:16]) == 32 and rule(wide[0, :, 4:8]) == 32
    assert rule(wide[:, :1, :8]) == 6 * 32       # one token per sequence: the rows are the sequences
    assert rule(wide[:1, 1:3, :8]) == 32 and rule(wide[:1, :1, :8]) == 8
    for bad in (wide[:, ::2][:, :2], wide[:, :3], wide[..., ::2], wide[0].t(), wide[0, :1].expand(4, 32)):
        with pytest.raises(ValueError):
            rule(bad)


def test_workspaces_and_devices_refused(monkeypatch):
    """A workspace that the kernels could not write as given; tensors of another GPU than the current one."""
    from types import SimpleNamespace

    def ws(**over):
        d = dict(dtype=torch.uint8, numel=lambda: 512, is_cuda=True, is_contiguous=lambda: True)
        return SimpleNamespace(**{**d, **over})

    like = torch.zeros(1)
    good = ws()
    assert block._scratch(good, 512, like) is good and block._scratch(None, 100, like).numel() == 100
    for bad in (ws(dtype=torch.int8), ws(numel=lambda: 511), ws(is_cuda=False), ws(is_contiguous=lambda: False)):
        with pytest.raises(ValueError):
            block._scratch(bad, 512, like)
    on = lambda i: SimpleNamespace(get_device=lambda: i, device="cuda:%d" % i)  # noqa: E731
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 40 + d, raising=False)
    monkeypatch.setattr(block, "_SEVERAL", True)
    assert block._stream(on(0), None, on(0)) == 40
    for tensors in ((on(1),), (on(0), on(1)), (on(0), None, on(1))):
        with pytest.raises(ValueError):
            block._stream(*tensors)
