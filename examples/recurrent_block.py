"""A gated recurrent block, trained, prefilled and served with the library's operators.

    s = x + residual;  y = RMSnorm(s);  u, g = y W_in;  c = SiLU(conv1d(u));  h = recurrence(c, g);  out = h W_out

The norm, the conv and the recurrence are the library's calls (with their backward and their
single-token forms); the two projections are torch products, or for an 8-bit prefill the first is the
library's product of the norm's e4m3 codes with those of the weight.  Run as a program it trains the
block for a few steps to remember tokens, and checks that decoding token by token continues a
prefill:

    python examples/recurrent_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_bwd_gb300 as gdr  # noqa: E402


class RecurrentBlock:
    """Packed sequences of ``channels`` channels; parameters in float32, products in bf16."""

    def __init__(self, channels, width=4, seed=0, device="cuda"):
        gen = torch.Generator(device).manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(*shape, generator=gen, device=device) * std

        C = channels
        self.p = {
            "norm": torch.ones(C, device=device),
            "w_in": normal(C, 2 * C, std=C ** -0.5),
            "conv": normal(C, width, std=width ** -0.5),
            "conv_bias": torch.zeros(C, device=device),
            # memories of one to a few hundred tokens: softplus(dt_bias) of 1 down to e^-5
            "A_log": torch.zeros(C, device=device),
            "dt_bias": -5.0 * torch.rand(C, generator=gen, device=device),
            "w_out": normal(C, C, std=C ** -0.5),
        }
        self.channels, self.width = C, width

    def _gate(self):
        return dict(A_log=self.p["A_log"], dt_bias=self.p["dt_bias"], gate="softplus", complement=True)

    def _project(self, normed, weight):
        """y W for y as rmsnorm_fwd gives it: bf16, or e4m3 with a scale for each 128 channels (a multiple of 16)."""
        if "scale" in normed:  # (a server whose weights stay would keep w)
            w = gdr.quant_e4m3(weight, tiles=True, transposed=True)  # (weight is [in, out], the product's [out, in])
            return gdr.linear_e4m3(normed["y"], normed["scale"], w["y_t"], w["scale_t"])
        return normed["y"] @ weight.to(torch.bfloat16)

    def forward(self, x, residual, cu_seqlens, states=None, eight_bit=False):
        """x, residual bf16 [T, C]; ``states``: a pool's (conv, recurrence) states before the sequences.
        Returns the output, the new residual, the states after the sequences and what backward needs."""
        conv0, h0 = states if states is not None else (None, None)
        n = gdr.rmsnorm_fwd(x, self.p["norm"], residual=residual, quant="block" if eight_bit else None)
        ug = self._project(n, self.p["w_in"])
        u, g = ug[:, :self.channels], ug[:, self.channels:]  # column slices, taken as they are
        c = gdr.conv1d_fwd(u, self.p["conv"], self.p["conv_bias"], state=conv0, cu_seqlens=cu_seqlens, want_state=True)
        r = gdr.glr_fwd(c["y"], g, h0=h0, cu_seqlens=cu_seqlens, **self._gate())
        out = r["h"] @ self.p["w_out"].to(torch.bfloat16)
        return out, n["residual"], (c["state"], r["ht"]), (n, u, g, c["y"], r["h"], cu_seqlens)

    def backward(self, saved, dout, dresidual=None):
        """Gradients of x (and the residual, which has the same) and of the parameters, from those of the
        output and of the new residual; the sequences began from zero states."""
        n, u, g, c, h, cu = saved
        grads = {"w_out": (h.t() @ dout).float()}
        r = gdr.glr_bwd(c, g, h, dout @ self.p["w_out"].to(torch.bfloat16).t(), cu_seqlens=cu, **self._gate())
        grads["A_log"], grads["dt_bias"] = r["dA_log"], r["ddt_bias"]
        v = gdr.conv1d_bwd(u.contiguous(), self.p["conv"], self.p["conv_bias"], r["dx"], cu_seqlens=cu)
        grads["conv"], grads["conv_bias"] = v["dweight"], v["dbias"]
        dug = torch.cat([v["dx"], r["dg"]], 1)
        grads["w_in"] = (n["y"].t() @ dug).float()
        d = gdr.rmsnorm_bwd(dug @ self.p["w_in"].to(torch.bfloat16).t(), n["residual"], self.p["norm"], n["rstd"],
                            dres=dresidual)
        grads["norm"] = d["dweight"]
        return d["dx"], grads

    def step(self, x, residual, states, slots=None):
        """One token of each row (x, residual bf16 [rows, C]) on a pool of states, updated in place."""
        conv, state = states
        n = gdr.rmsnorm_fwd(x, self.p["norm"], residual=residual)
        ug = self._project(n, self.p["w_in"])
        c = gdr.conv1d_step(ug[:, :self.channels], conv, self.p["conv"], self.p["conv_bias"], slots=slots)
        h = gdr.glr_step(c, ug[:, self.channels:], state, slots=slots, **self._gate())
        return h @ self.p["w_out"].to(torch.bfloat16), n["residual"]


def train(steps=60, channels=256, lengths=(300, 17, 1, 450), seed=1, lr=0.12):
    """Learns to repeat the token before (and to pass nothing where there is none); returns the losses."""
    block = RecurrentBlock(channels, seed=seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    cu = torch.tensor([0] + torch.tensor(lengths).cumsum(0).tolist(), device="cuda")
    T = int(sum(lengths))
    x = torch.randn(T, channels, generator=gen, device="cuda").to(torch.bfloat16)
    target = torch.cat([x[:1], x[:-1]]).float()
    target[cu[:-1]] = 0
    residual = torch.zeros_like(x)
    losses = []
    for _ in range(steps):
        out, _, _, saved = block.forward(x, residual, cu)
        diff = out.float() - target
        losses.append(float(diff.square().mean()))
        _, grads = block.backward(saved, (diff * (2.0 / channels)).to(torch.bfloat16))
        for name, grad in grads.items():
            p = block.p[name]
            p -= lr * grad * (p.norm() + 1.0) / (grad.norm() + 1e-6)  # normalised steps: one rate for all
    return losses


def serve(channels=256, prompts=(40, 7, 129), tokens=12, seed=2, eight_bit=False):
    """Prefills prompts, decodes more tokens from a pool of states, and returns how far the decoded
    outputs are from those of one long prefill (relative to their size)."""
    block = RecurrentBlock(channels, seed=seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    whole = [torch.randn(n + tokens, channels, generator=gen, device="cuda").to(torch.bfloat16) for n in prompts]

    def packed(parts):
        cu = torch.tensor([0] + torch.tensor([len(p) for p in parts]).cumsum(0).tolist(), device="cuda")
        return torch.cat(parts), cu

    x, cu = packed(whole)
    want, _, _, _ = block.forward(x, torch.zeros_like(x), cu)
    x, cu = packed([w[:n] for w, n in zip(whole, prompts)])
    _, _, states, _ = block.forward(x, torch.zeros_like(x), cu, eight_bit=eight_bit)
    rows, pool = len(prompts), 2 * len(prompts)
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(seed))[:rows].cuda()
    conv = torch.zeros(pool, block.width - 1, channels, dtype=torch.bfloat16, device="cuda")
    state = torch.zeros(pool, channels, device="cuda")
    conv[slots], state[slots] = states
    ends = torch.tensor([n + tokens for n in prompts]).cumsum(0).tolist()
    worst = 0.0
    for t in range(tokens):
        xt = torch.stack([w[n + t] for w, n in zip(whole, prompts)])
        out, _ = block.step(xt, torch.zeros_like(xt), (conv, state), slots=slots)
        ref = torch.stack([want[e - tokens + t] for e in ends])
        worst = max(worst, float((out.float() - ref.float()).norm() / ref.float().norm()))
    return worst


if __name__ == "__main__":
    losses = train()
    print("training: loss %.3f -> %.3f" % (losses[0], losses[-1]))
    print("serving: decoded outputs within %.1e of the long prefill, after an 8-bit prefill %.1e"
          % (serve(), serve(eight_bit=True)))
