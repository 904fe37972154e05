"""The recurrent block example on the GPU: its gradients against torch autograd of the same block in
float32, a falling loss, and decoding that continues a prefill."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from chunked_gated_delta_bwd_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_block.py")
    spec = importlib.util.spec_from_file_location("recurrent_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _plain(block, p, x, residual, cu):
    """The block in float32 with autograd, token by token."""
    C, K = block.channels, block.width
    s = x + residual
    y = s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-6) * p["norm"]
    u, g = (y @ p["w_in"]).split(C, dim=1)
    out = []
    for b, e in zip(cu[:-1], cu[1:]):
        line = torch.cat([torch.zeros(K - 1, C, device=x.device), u[b:e]])
        z = sum(p["conv"][:, k] * line[k:k + e - b] for k in range(K)) + p["conv_bias"]
        c = torch.nn.functional.silu(z)
        a = torch.exp(-torch.exp(p["A_log"]) * torch.nn.functional.softplus(g[b:e] + p["dt_bias"]))
        h = torch.zeros(C, device=x.device)
        for t in range(e - b):
            h = a[t] * h + (1 - a[t]) * c[t]
            out.append(h)
    return torch.stack(out) @ p["w_out"], s


def test_gradients_against_autograd(ex):
    block = ex.RecurrentBlock(64, seed=4)
    gen = torch.Generator("cuda").manual_seed(4)
    cu = [0, 30, 31, 100]
    x = torch.randn(100, 64, generator=gen, device="cuda").to(torch.bfloat16)
    residual = torch.randn(100, 64, generator=gen, device="cuda").to(torch.bfloat16)
    dout = torch.randn(100, 64, generator=gen, device="cuda").to(torch.bfloat16)
    dres = torch.randn(100, 64, generator=gen, device="cuda").to(torch.bfloat16)
    out, new, _, saved = block.forward(x, residual, torch.tensor(cu, device="cuda"))
    dx, grads = block.backward(saved, dout, dres)
    p = {k: v.clone().requires_grad_() for k, v in block.p.items()}
    xf = x.float().requires_grad_()
    ref, s = _plain(block, p, xf, residual.float(), cu)
    ((ref * dout.float()).sum() + (s * dres.float()).sum()).backward()
    rel = lambda a, b: float(((a.float() - b.float()).norm() / b.float().norm()).detach())  # noqa: E731
    # every tensor between the operators is rounded to bf16 (2^-8 each, half a dozen on the longest
    # path, partly amplified by the projections' cancelling sums): 6 * 2^-8
    tol = 6 * 2.0 ** -8
    assert rel(out, ref) <= tol and rel(new, s) <= 2.0 ** -8
    assert rel(dx, xf.grad) <= tol
    for name, grad in grads.items():
        assert rel(grad, p[name].grad) <= tol, name


def test_training_lowers_the_loss(ex):
    losses = ex.train(steps=40)
    assert all(v == v for v in losses) and losses[-1] < 0.5 * losses[0]


@pytest.mark.parametrize("eight_bit", [False, True])
def test_decoding_continues_a_prefill(ex, eight_bit):
    # bf16 roundings on both ways (6 * 2^-8 as above); the 8-bit prefill adds e4m3's 2^-4 to the
    # projection's inputs, half of which a sum of random signs passes on, and the states forget
    assert ex.serve(eight_bit=eight_bit) <= (2.0 ** -4 if eight_bit else 6 * 2.0 ** -8)
