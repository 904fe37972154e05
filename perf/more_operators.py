"""Linear attention with a decay for each head, and the 8-bit product of the projections around it.

Five calls, measured as a user makes them: linear attention's chunked forward and backward and its
single-token step (``dla_fwd``, ``dla_bwd``, ``dla_step``), the product of e4m3 operands with a scale
for each block of 128 (``linear_e4m3``), and the quantisation that brings weights, activations and
gradients into its form (``quant_e4m3``).

``own`` selects the framework's kernels; otherwise ``run`` computes the same results from
elementary torch operations in 32 bits.  ``exact`` restates the definitions in 64 bits, token by
token for the attention.
"""
import math

import torch

own = False

_E4M3_MAX = 448.0
_CHUNK = 128  # of the plain form


# --------------------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------------------

def _dla(name, op, tokens, seqs, ragged, heads, k_heads, dim, states, split):
    return {"name": name, "op": op, "tokens": tokens, "seqs": seqs, "ragged": ragged, "heads": heads,
            "k_heads": k_heads, "dim": dim, "states": states, "split": split}


def _linear(name, rows, inner, outer, scales, bias):
    return {"name": name, "op": "linear", "rows": rows, "inner": inner, "outer": outer, "scales": scales, "bias": bias}


def listed():
    return [
        # one short prompt of odd length, small heads, q and k shared by two value heads: latency counts
        _dla("dla_fwd_t509_h8_k4_d64", "dla_fwd", 509, 1, True, 8, 4, 64, True, False),
        # prefill of packed prompts of very different lengths; q, k, v are column slices of one projection
        _dla("dla_fwd_ragged16_h32", "dla_fwd", 30011, 16, True, 32, 32, 128, True, True),
        # training on one long sequence
        _dla("dla_fwd_t32k_h16", "dla_fwd", 32768, 1, False, 16, 16, 128, False, False),
        # backward of two dense sequences of odd length, grouped heads, states and their gradients
        _dla("dla_bwd_b2_t4095_h16_k4_d64", "dla_bwd", 8190, 2, False, 16, 4, 64, True, False),
        # backward of one long sequence
        _dla("dla_bwd_t32k_h16", "dla_bwd", 32768, 1, False, 16, 16, 128, False, False),
        # decoding three sequences: latency
        {"name": "dla_step_3_h16", "op": "dla_step", "rows": 3, "heads": 16, "k_heads": 16, "dim": 128, "pool": 0},
        # decoding a batch of a serving program: states in a pool, some rows of the batch padding
        {"name": "dla_step_257_h16_pool", "op": "dla_step", "rows": 257, "heads": 16, "k_heads": 16, "dim": 128,
         "pool": 300},
        # the q, k, v projection of five decoded tokens: the weights are read once
        _linear("linear_5x2048x6144", 5, 2048, 6144, "block", False),
        # the output projection of a decoding batch, odd rows, a bias
        _linear("linear_509x4096x2048_bias", 509, 4096, 2048, "block", True),
        # the q, k, v projection of a long prefill
        _linear("linear_32768x2048x6144", 32768, 2048, 6144, "block", False),
        # gradients on their way back through a projection, an odd number of tokens
        {"name": "quant_rows_8191x6144", "op": "quant", "rows": 8191, "channels": 6144, "type": "bf16", "form": "rows"},
        # a weight from its float32 master copy, for the forward and (transposed) for the backward
        {"name": "quant_tiles_6144x2048_f32", "op": "quant", "rows": 6144, "channels": 2048, "type": "f32",
         "form": "tiles_both"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MOST = 1 << 26  # elements (tokens x channels) of one drawn case


def _heads(rng):
    heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 16, 24, 32])
    return heads, rng.choice([d for d in range(1, heads + 1) if heads % d == 0]) if rng.random() < 0.4 else heads


def _width(rng):
    """The width of a projection: heads of 64 or 128 channels, or odd multiples of 16."""
    return rng.choice([1, 2, 3, 5, 8, 11, 16, 32, 48]) * 128 if rng.random() < 0.6 else 16 * (_log_int(rng, 4, 400) | 1)


def draw(rng):
    op = rng.choice(["dla_fwd", "dla_fwd", "dla_bwd", "dla_bwd", "dla_step", "linear", "linear", "linear", "quant"])
    if op in ("dla_fwd", "dla_bwd"):
        (heads, k_heads), dim = _heads(rng), rng.choice([64, 128, 128])
        # a drawn pass moves no more than the largest listed one
        tokens = _log_int(rng, 1, min(65536, _MOST // (heads * dim)))
        seqs = min(tokens, _log_int(rng, 1, 64))
        ragged = rng.random() < 0.6
        if not ragged:
            tokens = seqs * max(1, tokens // seqs)
        return {"op": op, "tokens": tokens, "seqs": seqs, "ragged": ragged, "heads": heads, "k_heads": k_heads,
                "dim": dim, "states": rng.random() < 0.6, "split": rng.random() < 0.4}
    if op == "dla_step":
        (heads, k_heads), dim = _heads(rng), rng.choice([64, 128])
        rows = _log_int(rng, 1, min(512, (257 * 16 << 14) // (heads * dim * dim)))
        return {"op": op, "rows": rows, "heads": heads, "k_heads": k_heads, "dim": dim,
                "pool": rows + rng.randrange(0, rows // 4 + 2) if rng.random() < 0.6 else 0}
    if op == "linear":
        inner, outer = _width(rng), _width(rng)
        most = (32768 * 2048 * 6144) // (inner * outer)
        return {"op": op, "rows": _log_int(rng, 1, min(32768, most)), "inner": inner, "outer": outer,
                "scales": rng.choice(["block", "block", "token"]), "bias": rng.random() < 0.4}
    channels = _width(rng) if rng.random() < 0.7 else 2 * (_log_int(rng, 32, 3000) | 1)
    rows = _log_int(rng, 1, min(1 << 16, _MOST // (2 * channels)))
    return {"op": op, "rows": rows, "channels": channels, "type": rng.choice(["bf16", "f32"]),
            "form": rng.choice(["rows", "tiles", "tiles_both"])}


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------

def _lengths(case, gen):
    """The sequences' borders on the host: random cuts, empty sequences among them, or equal lengths."""
    T, N = case["tokens"], case["seqs"]
    if case["ragged"]:
        return [0] + sorted(torch.randint(0, T + 1, (N - 1,), generator=gen).tolist()) + [T]
    return [n * (T // N) for n in range(N + 1)]


def _slots(case, host):
    """Which state of the pool each row of the batch has; every 16th row is padding (-1).  None without a pool."""
    if not case["pool"]:
        return None
    slots = torch.randperm(case["pool"], generator=host)[:case["rows"]]
    slots[15::16] = -1
    return slots.cuda()


def _codes(values, block):
    """(e4m3 codes, scale of each ``block`` columns) of a float32 matrix."""
    R, C = values.shape
    nb = -(-C // block)
    parts = torch.nn.functional.pad(values, (0, nb * block - C)).view(R, nb, block)
    scale = parts.abs().amax(2) / _E4M3_MAX
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    return (parts / scale[:, :, None]).view(R, -1)[:, :C].to(torch.float8_e4m3fn), scale


def _tile_codes(w):
    """(e4m3 codes, scale of each 128 x 128 tile) of a float32 matrix."""
    N, K = w.shape
    n, k = -(-N // 128), -(-K // 128)
    tiles = torch.nn.functional.pad(w, (0, 128 * k - K, 0, 128 * n - N)).view(n, 128, k, 128)
    scale = tiles.abs().amax((1, 3)) / _E4M3_MAX
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    codes = (tiles / scale[:, None, :, None]).view(128 * n, 128 * k)[:N, :K]
    return codes.contiguous().to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    st = {"case": dict(case)}
    op = case["op"]
    if op in ("dla_fwd", "dla_bwd", "dla_step"):
        H, Hk, D = case["heads"], case["k_heads"], case["dim"]
        st["scale"] = D ** -0.5
        # memories of one token up to ten thousand, another one for each head
        u = torch.rand(H, generator=gen, device="cuda")
        st["g"] = -torch.exp(math.log(1e-4) * u)
    if op in ("dla_fwd", "dla_bwd"):
        T, N = case["tokens"], case["seqs"]
        st["ends"] = _lengths(case, host)
        st["cu"] = torch.tensor(st["ends"], dtype=torch.int64, device="cuda")
        st["chunks"] = _Chunks(st["ends"], st["cu"].device)
        if case["split"]:  # columns of one projection's output
            both = normal(T, (2 * Hk + H) * D)
            q, k, v = both.split([Hk * D, Hk * D, H * D], dim=1)
            st["q"], st["k"], st["v"] = q.unflatten(1, (Hk, D)), k.unflatten(1, (Hk, D)), v.unflatten(1, (H, D))
        else:
            st["q"], st["k"], st["v"] = normal(T, Hk, D), normal(T, Hk, D), normal(T, H, D)
        st["h0"] = normal(N, H, D, D, dtype=torch.float32, std=0.5) if case["states"] else None
        if op == "dla_bwd":
            st["dO"] = normal(T, H, D)
            st["dht"] = normal(N, H, D, D, dtype=torch.float32, std=0.5) if case["states"] else None
        if not case["ragged"]:  # the dense layout
            for name in ("q", "k", "v", "dO"):
                if name in st:
                    st[name] = st[name].unflatten(0, (N, T // N))
    elif op == "dla_step":
        R = case["rows"]
        st["q"], st["k"], st["v"] = normal(R, Hk, D), normal(R, Hk, D), normal(R, H, D)
        st["slots"] = _slots(case, host)
        st["state"] = normal(case["pool"] or R, H, D, D, dtype=torch.float32)
    elif op == "linear":
        M, K, N = case["rows"], case["inner"], case["outer"]
        # a norm's output: channels of different sizes
        x = torch.randn(M, K, generator=gen, device="cuda") * torch.exp(torch.randn(K, generator=gen, device="cuda") * 0.5)
        st["x"], st["x_scale"] = _codes(x, 128 if case["scales"] == "block" else K)
        st["w"], st["w_scale"] = _tile_codes(torch.randn(N, K, generator=gen, device="cuda") * K ** -0.5)
        st["bias"] = normal(N, dtype=torch.float32, std=0.1) if case["bias"] else None
    else:
        R, C = case["rows"], case["channels"]
        size = torch.exp(torch.randn(R, 1, generator=gen, device="cuda") * 2.0)  # rows of very different sizes
        x = torch.randn(R, C, generator=gen, device="cuda") * (size if case["form"] == "rows" else C ** -0.5)
        st["x"] = x.to(torch.bfloat16) if case["type"] == "bf16" else x
    return st


# --------------------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------------------

def _flat(st, name):
    t = st[name]
    return t.flatten(0, 1) if t.dim() == 4 else t


class _Chunks:
    """The plain forms' plan: the sequences cut into chunks of _CHUNK tokens, the last of each shorter."""

    def __init__(self, ends, dev):
        lens = torch.tensor([b - a for a, b in zip(ends[:-1], ends[1:])])
        count = (lens + _CHUNK - 1) // _CHUNK
        self.seq = torch.repeat_interleave(torch.arange(len(lens)), count)
        first = torch.cumsum(count, 0) - count
        local = torch.arange(len(self.seq)) - first[self.seq]
        begin = torch.tensor(ends[:-1])
        start = begin[self.seq] + _CHUNK * local
        length = torch.minimum(lens[self.seq] - _CHUNK * local, torch.tensor(_CHUNK))
        token = start[:, None] + torch.arange(_CHUNK)
        inside = torch.arange(_CHUNK) < length[:, None]
        self.rows, self.of_rows = inside.flatten().nonzero().flatten().to(dev), token[inside].to(dev)
        self.outside = ~inside[:, :, None, None].to(dev)
        self.token = token.clamp(max=max(0, ends[-1] - 1)).to(dev)
        self.lens, self.begin, self.seq = lens.to(dev), begin.to(dev), self.seq.to(dev)
        self.start, self.length = start.to(dev), length.to(dev)
        self.end = self.start + self.length

    def take(self, t):
        """[T, H, D] -> float32 [H, chunks, _CHUNK, D], zero past a sequence's end."""
        return t.float()[self.token].masked_fill_(self.outside, 0).permute(2, 0, 1, 3)

    def put(self, x, like):
        """[H, chunks, _CHUNK, D] -> [T, H, D]."""
        out = torch.empty(like.shape[0], x.shape[0], x.shape[3], device=x.device)
        out[self.of_rows] = x.permute(1, 2, 0, 3).flatten(0, 1)[self.rows]
        return out


def _power(g, n):
    """e^(g n) of every head for whole numbers n: [H, *n.shape], the angle in 64 bits."""
    return torch.exp(g.double().view(-1, *[1] * n.dim()) * n).float()


def _carried(ch, g, sums, init, back):
    """The state before each chunk (after it, ``back``) [H, chunks, D, D], and after the whole sequence
    [N, H, D, D], from each chunk's sum [H, chunks, D, D] and the sequences' initial states."""
    same = ch.seq[:, None] == ch.seq[None, :]
    at = torch.arange(len(ch.seq), device=ch.seq.device)
    if back:
        away, order = ch.start[None, :] - ch.end[:, None], at[None, :] > at[:, None]
        from_init = (ch.begin + ch.lens)[ch.seq] - ch.end
        reach = ch.start - ch.begin[ch.seq]
    else:
        away, order = ch.start[:, None] - ch.end[None, :], at[None, :] < at[:, None]
        from_init = ch.start - ch.begin[ch.seq]
        reach = (ch.begin + ch.lens)[ch.seq] - ch.end
    H, D = sums.shape[0], sums.shape[-1]
    W = torch.where(same & order, _power(g, away.clamp(min=0)), torch.zeros((), device=g.device))
    state = torch.matmul(W, sums.flatten(2)).unflatten(2, (D, D))
    pick = torch.zeros(ch.lens.numel(), len(ch.seq), device=g.device)
    pick[ch.seq, at] = 1
    final = torch.matmul(pick * _power(g, reach)[:, None, :], sums.flatten(2)).unflatten(2, (D, D)).transpose(0, 1)
    if init is not None:
        state = state + _power(g, from_init)[:, :, None, None] * init.transpose(0, 1)[:, ch.seq]
        final = final + _power(g, ch.lens).t()[:, :, None, None] * init
    return state, final


def _decays(ch, g):
    """D_ij = e^(g (i - j)) for i >= j [H, 1, C, C]; the weights of a chunk's rows against the state before it
    [H, 1, C, 1], and of its tokens in the state after it [H, chunks, C, 1]."""
    i = torch.arange(_CHUNK, device=g.device)
    away = i[:, None] - i[None, :]
    D = torch.where(away >= 0, _power(g, away.clamp(min=0)), torch.zeros((), device=g.device))[:, None]
    left = ch.length[:, None] - 1 - i
    after = torch.where(left >= 0, _power(g, left.clamp(min=0)), torch.zeros((), device=g.device))
    return D, _power(g, i + 1)[:, None, :, None], after[:, :, :, None]


def _grouped(st, name):
    """q or k with a copy for each value head."""
    return _flat(st, name).repeat_interleave(st["case"]["heads"] // st["case"]["k_heads"], dim=1)


def _plain_dla_fwd(st):
    ch, g, scale = st["chunks"], st["g"], st["scale"]
    q, k, v = (ch.take(t) for t in (_grouped(st, "q"), _grouped(st, "k"), _flat(st, "v")))
    D, before, after = _decays(ch, g)
    state, ht = _carried(ch, g, torch.matmul((k * after).transpose(2, 3), v), st["h0"], False)
    o = torch.matmul(torch.matmul(q, k.transpose(2, 3)) * D, v) + before * torch.matmul(q, state)
    v = st["v"]
    return {"o": ch.put(o * scale, _flat(st, "v")).reshape(v.shape).to(v.dtype), "ht": ht}


def _plain_dla_bwd(st):
    case, ch, g, scale = st["case"], st["chunks"], st["g"], st["scale"]
    q, k, v, dO = (ch.take(t) for t in (_grouped(st, "q"), _grouped(st, "k"), _flat(st, "v"), _flat(st, "dO")))
    dO = dO * scale
    D, before, after = _decays(ch, g)
    state, _ = _carried(ch, g, torch.matmul((k * after).transpose(2, 3), v), st["h0"], False)
    carry, dh0 = _carried(ch, g, torch.matmul((q * before).transpose(2, 3), dO), st["dht"], True)
    P = torch.matmul(q, k.transpose(2, 3)) * D
    dP = torch.matmul(dO, v.transpose(2, 3)) * D
    dq = torch.matmul(dP, k) + before * torch.matmul(dO, state.transpose(2, 3))
    dk = torch.matmul(dP.transpose(2, 3), q) + after * torch.matmul(v, carry.transpose(2, 3))
    dv = torch.matmul(P.transpose(2, 3), dO) + after * torch.matmul(k, carry)

    def out(x, name):
        like = st[name]
        x = ch.put(x, _flat(st, name))
        if name != "v":
            x = x.unflatten(1, (case["k_heads"], -1)).sum(2)
        return x.reshape(like.shape).to(like.dtype)

    return {"dq": out(dq, "q"), "dk": out(dk, "k"), "dv": out(dv, "v"), "dh0": dh0}


def _plain_dla_step(st):
    state, slots, v = st["state"], st["slots"], st["v"]
    q, k = _grouped(st, "q").float(), _grouped(st, "k").float()
    decay = torch.exp(st["g"])[:, None, None]
    if slots is None:
        state.copy_(decay * state + k[..., None] * v.float()[:, :, None, :])
        new, keep = state, None
    else:
        keep = slots >= 0
        at = slots.clamp(min=0)
        new = decay * state[at] + k[..., None] * v.float()[:, :, None, :]
        state[slots[keep]] = new[keep]
    o = (q[..., None] * new).sum(2) * st["scale"]
    if keep is not None:
        o = torch.where(keep[:, None, None], o, torch.zeros_like(o))
    return {"o": o.to(v.dtype), "state": state}


def _spread(scale, block, size):
    return scale.repeat_interleave(block, dim=1)[:, :size]


def _plain_linear(st):
    x, w = st["x"].float(), st["w"].float()
    N, K = w.shape
    x = x * (_spread(st["x_scale"], 128, K) if st["case"]["scales"] == "block" else st["x_scale"])
    w = w * _spread(st["w_scale"], 128, K).repeat_interleave(128, dim=0)[:N]
    y = torch.matmul(x, w.t())
    return {"y": (y if st["bias"] is None else y + st["bias"]).to(torch.bfloat16)}


def _plain_quant(st):
    x, form = st["x"].float(), st["case"]["form"]
    y, scale = _codes(x, 128) if form == "rows" else _tile_codes(x)
    out = {"y": y, "scale": scale}
    if form == "tiles_both":
        out["y_t"], out["scale_t"] = y.t().contiguous(), scale.t().contiguous()
    return out


_PLAIN = {"dla_fwd": _plain_dla_fwd, "dla_bwd": _plain_dla_bwd, "dla_step": _plain_dla_step, "linear": _plain_linear,
          "quant": _plain_quant}


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------

def run(st):
    case = st["case"]
    if not own:
        return _PLAIN[case["op"]](st)
    import chunked_gated_delta_bwd_gb300 as gdr
    op = case["op"]
    if op == "dla_fwd":
        return gdr.dla_fwd(st["q"], st["k"], st["v"], st["g"], h0=st["h0"], scale=st["scale"],
                           cu_seqlens=st["cu"] if case["ragged"] else None)
    if op == "dla_bwd":
        return gdr.dla_bwd(st["q"], st["k"], st["v"], st["g"], st["dO"], h0=st["h0"], dht=st["dht"], scale=st["scale"],
                           cu_seqlens=st["cu"] if case["ragged"] else None)
    if op == "dla_step":
        return {"o": gdr.dla_step(st["q"], st["k"], st["v"], st["g"], st["state"], slots=st["slots"], scale=st["scale"]),
                "state": st["state"]}
    if op == "linear":
        return {"y": gdr.linear_e4m3(st["x"], st["x_scale"], st["w"], st["w_scale"], bias=st["bias"])}
    return gdr.quant_e4m3(st["x"], tiles=case["form"] != "rows", transposed=case["form"] == "tiles_both")


# --------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("dla_fwd", "dla_bwd"):
        T, H, Hk, D, N = (case[n] for n in ("tokens", "heads", "k_heads", "dim", "seqs"))
        state = 4 * N * H * D * D
        if op == "dla_fwd":  # q, k, v in, o and the final states out
            return {"bytes": 4 * T * D * (H + Hk) + state * (1 + case["states"]), "flops": 4 * T * H * D * D}
        # q, k, v, dO in, dq, dk, dv and dh0 out
        return {"bytes": 2 * T * D * (4 * Hk + 3 * H) + state * (1 + 2 * case["states"]), "flops": 10 * T * H * D * D}
    if op == "dla_step":
        rows, H, Hk, D = (case[n] for n in ("rows", "heads", "k_heads", "dim"))
        live = rows - (rows // 16 if case["pool"] else 0)
        return {"bytes": live * (8 * H * D * D + 2 * D * (2 * Hk + H)) + 2 * rows * H * D, "flops": 5 * live * H * D * D}
    if op == "linear":
        M, K, N = case["rows"], case["inner"], case["outer"]
        nb = -(-K // 128)
        scales = 4 * M * (nb if case["scales"] == "block" else 1) + 4 * nb * -(-N // 128)
        return {"bytes": M * K + N * K + 2 * M * N + scales + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    R, C, form = case["rows"], case["channels"], case["form"]
    size, nb = (2 if case["type"] == "bf16" else 4), -(-C // 128)
    scales = 4 * nb * (R if form == "rows" else -(-R // 128))
    both = 1 + (form == "tiles_both")
    return {"bytes": R * C * (size + both) + scales * both, "flops": 3 * R * C}


# --------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------

def _wide(t):
    return None if t is None else t.to(torch.float64)


def _exact_dla(st, case, forward):
    H, D, ends = case["heads"], case["dim"], st["ends"]
    group = H // case["k_heads"]
    q, k, v = (_wide(_flat(st, n)) for n in ("q", "k", "v"))
    q, k = (t.repeat_interleave(group, dim=1) for t in (q, k))
    decay = torch.exp(_wide(st["g"]))[:, None, None]
    state = torch.zeros(case["seqs"], H, D, D, dtype=torch.float64, device="cuda") if st["h0"] is None else _wide(st["h0"])
    rows, cols = (lambda t: t[:, :, None, :]), (lambda t: t[:, :, :, None])
    if forward:
        o, ht = torch.empty_like(v), state.clone()
        kc, vr, qr = cols(k), rows(v), rows(q * st["scale"])
        for n in range(case["seqs"]):
            for t in range(ends[n], ends[n + 1]):
                ht[n].mul_(decay).baddbmm_(kc[t], vr[t])
                torch.bmm(qr[t], ht[n], out=rows(o)[t])
        return {"o": o.reshape(st["v"].shape), "ht": ht}
    dO = _wide(_flat(st, "dO")) * st["scale"]
    back = torch.zeros_like(state) if st["dht"] is None else _wide(st["dht"]).clone()
    dq, dk, dv = torch.empty_like(v), torch.empty_like(v), torch.empty_like(v)
    kc, vr, qc, kr, dOr, dOc, vc = cols(k), rows(v), cols(q), rows(k), rows(dO), cols(dO), cols(v)
    for n in range(case["seqs"]):
        S, R = state[n].clone(), back[n]
        for t in range(ends[n], ends[n + 1]):
            S.mul_(decay).baddbmm_(kc[t], vr[t])
            torch.bmm(S, dOc[t], out=cols(dq)[t])
        for t in range(ends[n + 1] - 1, ends[n] - 1, -1):
            R.baddbmm_(qc[t], dOr[t])
            torch.bmm(R, vc[t], out=cols(dk)[t])
            torch.bmm(kr[t], R, out=rows(dv)[t])
            R.mul_(decay)
    dq, dk = (t.unflatten(1, (case["k_heads"], group)).sum(2) for t in (dq, dk))
    return {"dq": dq.reshape(st["q"].shape), "dk": dk.reshape(st["k"].shape), "dv": dv.reshape(st["v"].shape), "dh0": back}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("dla_fwd", "dla_bwd"):
        return _exact_dla(st, case, op == "dla_fwd")
    if op == "dla_step":
        group = case["heads"] // case["k_heads"]
        slots = list(range(case["rows"])) if st["slots"] is None else st["slots"].tolist()
        state = _wide(st["state"])
        rows = torch.tensor([i for i, s in enumerate(slots) if s >= 0], device="cuda", dtype=torch.int64)
        at = torch.tensor([s for s in slots if s >= 0], device="cuda", dtype=torch.int64)
        q, k, v = (_wide(st[n])[rows] for n in ("q", "k", "v"))
        q, k = (t.repeat_interleave(group, dim=1) for t in (q, k))
        new = torch.exp(_wide(st["g"]))[:, None, None] * state[at] + torch.einsum("rhd,rhe->rhde", k, v)
        state[at] = new
        o = torch.zeros(st["v"].shape, dtype=torch.float64, device="cuda")
        o[rows] = st["scale"] * torch.einsum("rhd,rhde->rhe", q, new)
        return {"o": o, "state": state}
    if op == "linear":
        x, w, xs, ws = (_wide(st[n]) for n in ("x", "w", "x_scale", "w_scale"))
        K, N = case["inner"], case["outer"]
        block = torch.arange(K, device="cuda") // 128
        x = x * (xs[:, block] if case["scales"] == "block" else xs)
        w = w * ws[(torch.arange(N, device="cuda") // 128)[:, None], block[None, :]]
        y = torch.mm(x, w.t())
        return {"y": y if st["bias"] is None else y + _wide(st["bias"])}
    x, form = _wide(st["x"]), case["form"]
    R, C = x.shape
    of_row = torch.arange(R, device="cuda") // (1 if form == "rows" else 128)
    of_col = torch.arange(C, device="cuda") // 128
    most = torch.zeros(int(of_row[-1]) + 1, int(of_col[-1]) + 1, dtype=torch.float64, device="cuda")
    wide = torch.zeros(R, most.shape[1], dtype=torch.float64, device="cuda")
    wide.scatter_reduce_(1, of_col.expand(R, C), x.abs(), "amax")
    most.scatter_reduce_(0, of_row[:, None].expand(R, most.shape[1]), wide, "amax")
    scale = torch.where(most > 0, most / _E4M3_MAX, torch.ones_like(most))
    out = {"y": x / scale[of_row[:, None], of_col[None, :]], "scale": scale}
    if form == "tiles_both":
        out["y_t"], out["scale_t"] = out["y"].t().contiguous(), scale.t().contiguous()
    return out
