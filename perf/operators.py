"""The operators of a gated recurrent block, measured as a user calls them.

Seven calls: the gated linear recurrence's forward, backward and single-token step
(``glr_fwd``, ``glr_bwd``, ``glr_step``), the RMS norm with the residual's addition and its
backward (``rmsnorm_fwd``, ``rmsnorm_bwd``; bf16, or e4m3 with scales), and the causal
conv1d's forward and single-token step (``conv1d_fwd``, ``conv1d_step``).

``own`` selects the framework's kernels; otherwise ``run`` computes the same results from
elementary torch operations in 32 bits.  ``exact`` restates the definitions in 64 bits,
token by token for the recurrence.
"""
import math

import torch

own = False

_E4M3_MAX = 448.0


# --------------------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------------------

def _glr(name, op, tokens, seqs, ragged, channels, gate, complement, types, split, states):
    return {"name": name, "op": op, "tokens": tokens, "seqs": seqs, "ragged": ragged, "channels": channels,
            "gate": gate, "complement": complement, "types": types, "split": split, "states": states}


def _norm(name, op, rows, channels, residual, quant):
    return {"name": name, "op": op, "rows": rows, "channels": channels, "residual": residual, "quant": quant}


def listed():
    return [
        # decoding three sequences: a call bound by its latency
        {"name": "glr_step_3x2048", "op": "glr_step", "rows": 3, "channels": 2048, "gate": "log",
         "complement": False, "types": "bf16", "pool": 0},
        # decoding a full batch of a serving program: states in a pool, some rows of the batch padding
        {"name": "glr_step_509x4096_pool", "op": "glr_step", "rows": 509, "channels": 4096, "gate": "softplus",
         "complement": True, "types": "bf16", "pool": 700},
        # prefill of packed prompts of very different lengths (32 heads of 128); x and the gate are
        # column slices of one projection
        _glr("glr_fwd_ragged16_h32", "glr_fwd", 30011, 16, True, 4096, "softplus", True, "bf16", True, True),
        # training on one long sequence (16 heads of 128) with a float32 log gate
        _glr("glr_fwd_t32k_h16", "glr_fwd", 32768, 1, False, 2048, "log", False, "bf16_f32", False, False),
        # backward in float32 throughout, two dense sequences, states' gradients
        _glr("glr_bwd_b2_t4k_f32", "glr_bwd", 8192, 2, False, 2048, "log", False, "f32", False, True),
        # backward of one long sequence, the gate's parameters' gradients among the outputs
        _glr("glr_bwd_t32k_h16", "glr_bwd", 32768, 1, False, 2048, "softplus", True, "bf16", False, False),
        # the norm of five decoded tokens: latency again
        _norm("norm_fwd_5x2048", "norm_fwd", 5, 2048, "bf16", "none"),
        # the norm before an 8-bit projection, a long prefill
        _norm("norm_fwd_32768x2048_e4m3", "norm_fwd", 32768, 2048, "bf16", "block"),
        # per head on the recurrence's output: 4095 tokens of 16 heads, one scale for each row
        _norm("norm_fwd_heads_65520x128", "norm_fwd", 65520, 128, "none", "token"),
        # backward over an odd number of tokens, the residual kept in float32
        _norm("norm_bwd_8191x2048", "norm_bwd", 8191, 2048, "f32", "none"),
        # the q, k, v channels of 16 heads of 128 over one long sequence
        {"name": "conv_fwd_t32k_c6144", "op": "conv_fwd", "tokens": 32768, "seqs": 1, "ragged": False,
         "channels": 6144, "width": 4, "silu": True, "states": False},
        # their single-token form for a decoding batch
        {"name": "conv_step_257x6144", "op": "conv_step", "rows": 257, "channels": 6144, "width": 4, "silu": True,
         "pool": 300},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MOST = 1 << 26  # elements (tokens x channels) of one drawn case


def _channels(rng):
    """Heads of 64 or 128 channels, or any even number, down to where no wide load is aligned."""
    if rng.random() < 0.5:
        return rng.choice([1, 2, 3, 5, 8, 11, 16, 22, 32]) * rng.choice([64, 128])
    return 2 * (_log_int(rng, 32, 4096) | 1)


def draw(rng):
    op = rng.choice(["glr_fwd", "glr_fwd", "glr_bwd", "glr_bwd", "glr_step", "norm_fwd", "norm_fwd", "norm_bwd",
                     "conv_fwd", "conv_step"])
    if op in ("glr_fwd", "glr_bwd", "conv_fwd"):
        channels = _channels(rng)
        # a drawn pass moves no more than the largest listed one (float32 counts twice)
        types = rng.choice(["bf16", "bf16", "bf16_f32", "f32"])
        most = _MOST if op == "conv_fwd" or types != "f32" else _MOST // 2
        tokens = _log_int(rng, 1, max(2, min(65536, most // (2 * channels))))
        seqs = min(tokens, _log_int(rng, 1, 64))
        ragged = rng.random() < 0.6
        if not ragged:
            tokens = seqs * max(1, tokens // seqs)
        if op == "conv_fwd":
            return {"op": op, "tokens": tokens, "seqs": seqs, "ragged": ragged, "channels": channels,
                    "width": rng.choice([2, 3, 4]), "silu": rng.random() < 0.7, "states": rng.random() < 0.5}
        gate = "log" if types == "bf16_f32" else rng.choice(["log", "softplus"])
        return {"op": op, "tokens": tokens, "seqs": seqs, "ragged": ragged, "channels": channels, "gate": gate,
                "complement": rng.random() < 0.5, "types": types,
                "split": types != "bf16_f32" and rng.random() < 0.4, "states": rng.random() < 0.6}
    if op in ("glr_step", "conv_step"):
        rows, channels = _log_int(rng, 1, 1024), _channels(rng)
        pool = rows + rng.randrange(0, rows + 1) if rng.random() < 0.6 else 0
        if op == "conv_step":
            return {"op": op, "rows": rows, "channels": channels, "width": rng.choice([2, 3, 4]),
                    "silu": rng.random() < 0.7, "pool": pool}
        return {"op": op, "rows": rows, "channels": channels, "gate": rng.choice(["log", "softplus"]),
                "complement": rng.random() < 0.5, "types": rng.choice(["bf16", "f32"]), "pool": pool}
    channels = rng.choice([64, 128, _channels(rng), _channels(rng)])
    rows = _log_int(rng, 1, max(2, min(1 << 17, (1 << 26) // channels)))
    residual = rng.choice(["none", "bf16", "f32"])
    if op == "norm_bwd":
        return {"op": op, "rows": rows, "channels": channels, "residual": residual, "quant": "none"}
    return {"op": op, "rows": rows, "channels": channels, "residual": residual,
            "quant": rng.choice(["none", "token", "block"])}


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------

def _types(case):
    act = torch.float32 if case["types"] == "f32" else torch.bfloat16
    gate = torch.bfloat16 if case["types"] == "bf16" else torch.float32
    return act, gate


def _lengths(case, gen):
    """cu_seqlens (int64, on the GPU) and the lengths: random cuts, empty sequences among them, or equal ones."""
    T, N = case["tokens"], case["seqs"]
    if case["ragged"]:
        cuts = torch.randint(0, T + 1, (N - 1,), generator=gen).tolist()
        ends = sorted(cuts) + [T]
    else:
        ends = [(n + 1) * (T // N) for n in range(N)]
    cu = [0] + ends
    return torch.tensor(cu, dtype=torch.int64, device="cuda"), [b - a for a, b in zip(cu[:-1], cu[1:])]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    host = torch.Generator().manual_seed(int(seed))

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo

    st = {"case": dict(case)}
    op, C = case["op"], case["channels"]

    def gate_inputs(rows):
        """The gate's input and its parameters: memories of a few tokens up to hundreds."""
        _, tg = _types(case)
        if case["gate"] == "softplus":  # the framework's recipe, with biases that give long memories too
            st["A_log"], st["dt_bias"] = uniform(-1.0, 0.0, C), uniform(-5.0, 0.0, C)
            return normal(rows, C, dtype=tg)
        z = torch.randn(rows, C, generator=gen, device="cuda") + uniform(-6.0, 0.0, C)
        return (-torch.log1p(torch.exp(z))).to(tg)

    if op in ("glr_fwd", "glr_bwd"):
        T, N = case["tokens"], case["seqs"]
        act, _ = _types(case)
        st["cu"], lens = _lengths(case, host)
        st["longest"] = max(lens)
        x, g = normal(T, C, dtype=act), gate_inputs(T)
        if case["split"]:  # x and the gate as columns of one projection's output
            both = torch.cat([x, g], 1)
            x, g = both[:, :C], both[:, C:]
        st["x"], st["g"] = x, g
        st["h0"] = normal(N, C, dtype=torch.float32, std=0.5) if case["states"] else None
        if op == "glr_bwd":
            st["dh"] = normal(T, C, dtype=act)
            st["dht"] = normal(N, C, dtype=torch.float32, std=0.5) if case["states"] else None
            h, _ = _plain_scan(*_gate(st)[1:], st, st["h0"])  # what the forward kept
            st["h"] = h.to(act)
        if not case["ragged"]:  # the dense layout
            for k in ("x", "g", "dh", "h"):
                if k in st:
                    st[k] = st[k].unflatten(0, (N, T // N))
    elif op == "glr_step":
        act, _ = _types(case)
        st["x"], st["g"] = normal(case["rows"], C, dtype=act), gate_inputs(case["rows"])
        st["slots"] = _slots(case, host)
        st["state"] = normal(case["pool"] or case["rows"], C, dtype=torch.float32)
    elif op in ("norm_fwd", "norm_bwd"):
        R = case["rows"]
        st["weight"] = 1.0 + normal(C, dtype=torch.float32, std=0.2)
        res = {"none": None, "bf16": torch.bfloat16, "f32": torch.float32}[case["residual"]]
        if op == "norm_fwd":
            st["x"] = normal(R, C)
            # a residual stream is larger than what one block adds to it
            st["residual"] = None if res is None else normal(R, C, dtype=res, std=3.0)
        else:
            st["s"] = normal(R, C, dtype=torch.bfloat16 if res is None else res, std=3.0)
            st["rstd"] = torch.rsqrt(st["s"].float().square().mean(1) + 1e-6)
            st["dy"] = normal(R, C)
            st["dres"] = None if res is None else normal(R, C, dtype=res)
    else:
        K = case["width"]
        st["weight"], st["bias"] = normal(C, K, dtype=torch.float32, std=0.5), normal(C, dtype=torch.float32, std=0.1)
        if op == "conv_fwd":
            T, N = case["tokens"], case["seqs"]
            st["cu"], _ = _lengths(case, host)
            st["x"] = normal(T, C)
            st["state"] = normal(N, K - 1, C) if case["states"] else None
            if not case["ragged"]:
                st["x"] = st["x"].unflatten(0, (N, T // N))
        else:
            st["x"] = normal(case["rows"], C)
            st["slots"] = _slots(case, host)
            st["state"] = normal(case["pool"] or case["rows"], K - 1, C)
    return st


def _slots(case, host):
    """Which state of the pool each row of the batch has; every 16th row is padding (-1).  None without a pool."""
    if not case["pool"]:
        return None
    slots = torch.randperm(case["pool"], generator=host)[:case["rows"]]
    slots[15::16] = -1
    return slots.cuda()


# --------------------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------------------

def _flat(st, key):
    t = st[key]
    return t.flatten(0, 1) if t.dim() == 3 else t


def _softplus(z):
    return z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))


def _gate(st):
    """(log gate, decay, x scaled as the recurrence adds it), in 32 bits."""
    g = _flat(st, "g").float()
    if st["case"]["gate"] == "softplus":
        g = -torch.exp(st["A_log"]) * _softplus(g + st["dt_bias"])
    x = _flat(st, "x").float()
    return g, torch.exp(g), (-torch.expm1(g) * x if st["case"]["complement"] else x)


def _sequence_of(cu, T):
    """The sequence of each token, and whether the token is its first one."""
    at = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu, at, right=True) - 1
    return seq, cu[seq] == at


def _doubled(a, b, longest):
    """y_t = a_t y_{t-1} + b_t down the first axis by doubling (a is zero where a sequence starts)."""
    d = 1
    while d < longest:
        b = torch.cat([b[:d], b[d:] + a[d:] * b[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _plain_scan(a, b, st, h0):
    T, cu = a.shape[0], st["cu"]
    seq, first = _sequence_of(cu, T)
    first = first[:, None]
    if h0 is not None:
        b = torch.where(first, b + a * h0[seq], b)
    h = _doubled(torch.where(first, torch.zeros_like(a), a), b, st["longest"])
    start = torch.zeros(cu.numel() - 1, a.shape[1], device=a.device) if h0 is None else h0
    ht = torch.where((cu[1:] > cu[:-1])[:, None], h[(cu[1:] - 1).clamp(min=0)], start)
    return h, ht


def _like(t, st):
    """`t` in the layout of the call's x."""
    return t.reshape(st["x"].shape)


def _plain_glr_fwd(st):
    _, a, b = _gate(st)
    h, ht = _plain_scan(a, b, st, st["h0"])
    return {"h": _like(h, st).to(st["x"].dtype), "ht": ht}


def _plain_glr_bwd(st):
    cu, comp, soft = st["cu"], st["case"]["complement"], st["case"]["gate"] == "softplus"
    g, a, _ = _gate(st)
    x, h, dh = _flat(st, "x").float(), _flat(st, "h").float(), _flat(st, "dh").float()
    T, C = a.shape
    seq, first = _sequence_of(cu, T)
    h0 = torch.zeros(cu.numel() - 1, C, device=a.device) if st["h0"] is None else st["h0"]
    dht = torch.zeros_like(h0) if st["dht"] is None else st["dht"]
    last = torch.cat([first[1:], first.new_ones(1)])[:, None]
    dh = torch.where(last, dh + dht[seq], dh)
    nxt = torch.where(last, torch.zeros_like(a), torch.cat([a[1:], a[:1]]))
    lam = _doubled(nxt.flip(0), dh.flip(0), st["longest"]).flip(0)
    prev = torch.where(first[:, None], h0[seq], torch.cat([h[:1], h[:-1]]))
    dg = lam * a * (prev - x if comp else prev)
    dx = lam * -torch.expm1(g) if comp else lam
    begin = cu[:-1].clamp(max=T - 1)
    dh0 = torch.where((cu[1:] > cu[:-1])[:, None], (a * lam)[begin], dht)
    out = {"dx": _like(dx, st).to(st["x"].dtype), "dh0": dh0}
    if soft:
        z = _flat(st, "g").float() + st["dt_bias"]
        out["dA_log"] = (dg * g).sum(0)
        dg = dg * -torch.exp(st["A_log"]) / (1 + torch.exp(-z))
        out["ddt_bias"] = dg.sum(0)
    out["dg"] = _like(dg, st).to(st["g"].dtype)
    return out


def _plain_glr_step(st):
    _, a, b = _gate(st)
    state, slots = st["state"], st["slots"]
    if slots is None:
        state.copy_(a * state + b)
        return {"y": state.to(st["x"].dtype), "state": state}
    on = (slots >= 0)[:, None]
    at = slots.clamp(min=0)
    h = torch.where(on, a * state[at] + b, torch.zeros_like(a))
    keep = slots >= 0
    state[slots[keep]] = h[keep]
    return {"y": h.to(st["x"].dtype), "state": state}


def _plain_norm_fwd(st):
    case, x, r = st["case"], st["x"], st["residual"]
    s = x if r is None else (x.float() + r.float()).to(r.dtype)
    f = s.float()
    rstd = torch.rsqrt(f.square().mean(1) + 1e-6)
    y = f * rstd[:, None] * st["weight"]
    out = {"rstd": rstd}
    if r is not None:
        out["residual"] = s
    if case["quant"] == "none":
        out["y"] = y.to(x.dtype)
        return out
    R, C = y.shape
    block = C if case["quant"] == "token" else 128
    nb = (C + block - 1) // block
    blocks = torch.zeros(R, nb * block, device=y.device)
    blocks[:, :C] = y
    blocks = blocks.view(R, nb, block)
    most = blocks.abs().amax(2)
    scale = torch.where(most > 0, most / _E4M3_MAX, torch.ones_like(most))
    out["y"] = (blocks / scale[:, :, None]).view(R, -1)[:, :C].to(torch.float8_e4m3fn)
    out["scale"] = scale
    return out


def _plain_norm_bwd(st):
    s, dy, rstd = st["s"].float(), st["dy"].float(), st["rstd"][:, None]
    n, u = s * rstd, dy * st["weight"]
    dx = rstd * (u - n * (u * n).mean(1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return {"dx": dx.to(st["s"].dtype), "dweight": (dy * n).sum(0)}


def _taps(st):
    """x of each token's last K tokens (0 or the state before the sequence), oldest first."""
    x, cu, K = _flat(st, "x").float(), st["cu"], st["case"]["width"]
    T = x.shape[0]
    seq, _ = _sequence_of(cu, T)
    local = torch.arange(T, device=x.device) - cu[seq]

    def tap(back):
        if back == 0:
            return x
        v = torch.cat([x[:back], x[:-back]])[:T] if back < T else x
        before = (local < back)[:, None]
        old = torch.zeros_like(x) if st["state"] is None else \
            st["state"][seq, (K - 1 - back + local).clamp(max=K - 2)].float()
        return torch.where(before, old, v)

    return [tap(K - 1 - k) for k in range(K)]


def _activated(z, silu):
    return z / (1 + torch.exp(-z)) if silu else z


def _plain_conv_fwd(st):
    case, w, cu = st["case"], st["weight"], st["cu"]
    z = sum(w[:, k] * t for k, t in enumerate(_taps(st))) + st["bias"]
    x, K = _flat(st, "x"), case["width"]
    back = torch.arange(K - 1, device=x.device)[None, :] - (K - 1)  # tokens before the sequence's end
    lens = (cu[1:] - cu[:-1])[:, None]
    inside = (lens + back >= 0)[:, :, None]
    old = torch.zeros(lens.shape[0], K - 1, x.shape[1], dtype=x.dtype, device=x.device) if st["state"] is None else \
        st["state"].gather(1, (lens + back + K - 1).clamp(max=K - 2)[:, :, None].expand(-1, -1, x.shape[1]))
    new = torch.where(inside, x[(cu[1:, None] + back).clamp(min=0)], old)
    return {"y": _like(_activated(z, case["silu"]), st).to(x.dtype), "state": new}


def _plain_conv_step(st):
    case, w, x, slots = st["case"], st["weight"], st["x"], st["slots"]
    state = st["state"]
    at = torch.arange(x.shape[0], device=x.device) if slots is None else slots.clamp(min=0)
    taps = torch.cat([state[at], x[:, None]], 1)
    z = (taps.float() * w.t()).sum(1) + st["bias"]
    y = _activated(z, case["silu"]).to(x.dtype)
    if slots is None:
        state.copy_(taps[:, 1:])
        return {"y": y, "state": state}
    keep = slots >= 0
    state[slots[keep]] = taps[keep, 1:]
    return {"y": torch.where(keep[:, None], y, torch.zeros_like(y)), "state": state}


_PLAIN = {"glr_fwd": _plain_glr_fwd, "glr_bwd": _plain_glr_bwd, "glr_step": _plain_glr_step,
          "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "conv_fwd": _plain_conv_fwd,
          "conv_step": _plain_conv_step}


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------

def run(st):
    case = st["case"]
    if not own:
        return _PLAIN[case["op"]](st)
    import chunked_gated_delta_bwd_gb300 as gdr
    op = case["op"]
    if op in ("glr_fwd", "glr_bwd", "glr_step"):
        how = {"gate": case["gate"], "complement": case["complement"], "A_log": st.get("A_log"),
               "dt_bias": st.get("dt_bias")}
        if op == "glr_step":
            return {"y": gdr.glr_step(st["x"], st["g"], st["state"], slots=st["slots"], **how), "state": st["state"]}
        cu = st["cu"] if case["ragged"] else None
        if op == "glr_fwd":
            return gdr.glr_fwd(st["x"], st["g"], h0=st["h0"], cu_seqlens=cu, **how)
        return gdr.glr_bwd(st["x"], st["g"], st["h"], st["dh"], h0=st["h0"], dht=st["dht"], cu_seqlens=cu, **how)
    if op == "norm_fwd":
        quant = None if case["quant"] == "none" else case["quant"]
        return gdr.rmsnorm_fwd(st["x"], st["weight"], residual=st["residual"], quant=quant)
    if op == "norm_bwd":
        return gdr.rmsnorm_bwd(st["dy"], st["s"], st["weight"], st["rstd"], dres=st["dres"])
    if op == "conv_fwd":
        return gdr.conv1d_fwd(st["x"], st["weight"], st["bias"], state=st["state"],
                              cu_seqlens=st["cu"] if case["ragged"] else None, silu=case["silu"], want_state=True)
    return {"y": gdr.conv1d_step(st["x"], st["state"], st["weight"], st["bias"], slots=st["slots"],
                                 silu=case["silu"]), "state": st["state"]}


# --------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------

def work(case):
    op, C = case["op"], case["channels"]
    size = {"bf16": 2, "f32": 4, "none": 0}
    if op in ("glr_fwd", "glr_bwd"):
        n, N = case["tokens"] * C, case["seqs"] * C
        act, tg = (4 if case["types"] == "f32" else 2), (2 if case["types"] == "bf16" else 4)
        par = 8 * C if case["gate"] == "softplus" else 0
        states = 4 * N * (2 if case["states"] else 1)  # ht (dh0) out, h0 in
        more = 8 if case["gate"] == "softplus" else 0  # the gate's function of one element
        if op == "glr_fwd":
            return {"bytes": n * (2 * act + tg) + states + par, "flops": n * (3 + 2 * case["complement"] + more)}
        reads = act * (2 + case["complement"])  # h, dh, and x where the gate's gradient needs it
        return {"bytes": n * (reads + act + 2 * tg) + states + (4 * N if case["states"] else 0) + 2 * par,
                "flops": n * (6 + 3 * case["complement"] + 2 * more)}
    if op in ("glr_step", "conv_step"):
        rows, pad = case["rows"], case["rows"] // 16 if case["pool"] else 0
        live = (rows - pad) * C
        if op == "conv_step":
            K = case["width"]
            return {"bytes": live * (2 + 4 * (K - 1)) + 2 * rows * C + 4 * C * (K + 1) + 8 * rows,
                    "flops": live * (2 * K + 4)}
        s = size[case["types"]]
        return {"bytes": live * (2 * s + 8) + s * rows * C + (8 * C if case["gate"] == "softplus" else 0),
                "flops": live * 12}
    if op in ("norm_fwd", "norm_bwd"):
        R = case["rows"]
        n, r = R * C, size[case["residual"]]
        if op == "norm_bwd":
            s = r or 2
            return {"bytes": n * (2 + s + r + s) + 4 * R + 8 * C, "flops": 12 * n}
        y = 2 if case["quant"] == "none" else 1
        scales = {"none": 0, "token": 1, "block": (C + 127) // 128}[case["quant"]]
        return {"bytes": n * (2 + 2 * r + y) + 4 * R * (1 + scales) + 4 * C, "flops": 8 * n}
    n, K = case["tokens"] * C, case["width"]
    return {"bytes": 4 * n + 2 * case["seqs"] * (K - 1) * C * (2 if case["states"] else 1) + 4 * C * (K + 1),
            "flops": n * (2 * K + 4)}


# --------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------

def _wide(t):
    return None if t is None else t.to(torch.float64)


def _exact_gate(st):
    raw = _wide(st["g"]).reshape(-1, st["case"]["channels"])
    if st["case"]["gate"] == "log":
        return raw, None
    z = raw + _wide(st["dt_bias"])
    return -torch.exp(_wide(st["A_log"])) * torch.logaddexp(z, torch.zeros_like(z)), z


def exact(case, seed):
    st = prepare(case, seed)
    op, C = case["op"], case["channels"]
    if op in ("glr_fwd", "glr_bwd"):
        cu = st["cu"].tolist()
        g, z = _exact_gate(st)
        x = _wide(st["x"]).reshape(-1, C)
        decay, give = torch.exp(g), (-torch.expm1(g) if case["complement"] else torch.ones_like(g))
        state = torch.zeros(case["seqs"], C, dtype=torch.float64, device="cuda") if st["h0"] is None else _wide(st["h0"])
        if op == "glr_fwd":
            into = give * x
            out, ht = torch.empty_like(x), state.clone()
            for n in range(case["seqs"]):
                h = state[n]
                for t in range(cu[n], cu[n + 1]):
                    h = torch.addcmul(into[t], decay[t], h, out=out[t])
                ht[n] = h
            return {"h": out.reshape(st["x"].shape), "ht": ht}
        h, dh = _wide(st["h"]).reshape(-1, C), _wide(st["dh"]).reshape(-1, C)
        grad, before = torch.empty_like(x), torch.empty_like(x)
        dh0 = torch.zeros_like(state) if st["dht"] is None else _wide(st["dht"]).clone()
        for n in range(case["seqs"]):
            b, e = cu[n], cu[n + 1]
            if b == e:
                continue
            before[b] = state[n]
            before[b + 1:e] = h[b:e - 1]
            carry = dh0[n]
            for t in range(e - 1, b - 1, -1):
                torch.add(dh[t], carry, out=grad[t])
                carry = decay[t] * grad[t]
            dh0[n] = carry
        dg = grad * decay * (before - x if case["complement"] else before)
        res = {"dx": (give * grad).reshape(st["x"].shape), "dh0": dh0}
        if z is not None:
            res["dA_log"] = (dg * g).sum(0)
            dg = -dg * torch.exp(_wide(st["A_log"])) * torch.sigmoid(z)
            res["ddt_bias"] = dg.sum(0)
        res["dg"] = dg.reshape(st["g"].shape)
        return res
    if op in ("glr_step", "conv_step"):
        slots = list(range(case["rows"])) if st["slots"] is None else st["slots"].tolist()
        state = _wide(st["state"])
        rows = torch.tensor([i for i, s in enumerate(slots) if s >= 0], device="cuda", dtype=torch.int64)
        at = torch.tensor([s for s in slots if s >= 0], device="cuda", dtype=torch.int64)
        x = _wide(st["x"])
        y = torch.zeros_like(x)
        if op == "glr_step":
            g, _ = _exact_gate(st)
            s = -torch.expm1(g) if case["complement"] else torch.ones_like(g)
            y[rows] = torch.exp(g[rows]) * state[at] + s[rows] * x[rows]
            state[at] = y[rows]
            return {"y": y, "state": state}
        line = torch.cat([state[at], x[rows][:, None]], 1)
        z = torch.einsum("nkc,ck->nc", line, _wide(st["weight"])) + _wide(st["bias"])
        y[rows] = z * torch.sigmoid(z) if case["silu"] else z
        state[at] = line[:, 1:]
        return {"y": y, "state": state}
    if op == "norm_fwd":
        s = st["x"] if st["residual"] is None else (_wide(st["x"]) + _wide(st["residual"])).to(st["residual"].dtype)
        f = _wide(s)
        mean = (f * f).sum(1) / C
        y = f / torch.sqrt(mean + 1e-6)[:, None] * _wide(st["weight"])
        res = {"rstd": 1 / torch.sqrt(mean + 1e-6), "y": y}
        if st["residual"] is not None:
            res["residual"] = _wide(s)
        if case["quant"] != "none":
            parts = [y] if case["quant"] == "token" else list(torch.split(y, 128, dim=1))
            most = [p.abs().amax(1, keepdim=True) for p in parts]
            scale = [torch.where(m > 0, m / _E4M3_MAX, torch.ones_like(m)) for m in most]
            res["y"] = torch.cat([p / s for p, s in zip(parts, scale)], 1)
            res["scale"] = torch.cat(scale, 1)
        return res
    if op == "norm_bwd":
        s, dy, w = _wide(st["s"]), _wide(st["dy"]), _wide(st["weight"])
        inv = _wide(st["rstd"])[:, None]
        inner = (w * dy * s).sum(1, keepdim=True) / C
        dx = inv * w * dy - inv ** 3 * inner * s
        if st["dres"] is not None:
            dx = dx + _wide(st["dres"])
        return {"dx": dx, "dweight": (dy * s * inv).sum(0)}
    cu, K = st["cu"].tolist(), case["width"]
    x, w = _wide(st["x"]).reshape(-1, C), _wide(st["weight"])
    z = torch.empty_like(x)
    state = torch.zeros(case["seqs"], K - 1, C, dtype=torch.float64, device="cuda") if st["state"] is None else \
        _wide(st["state"]).clone()
    for n in range(case["seqs"]):
        line = torch.cat([state[n], x[cu[n]:cu[n + 1]]])
        L = cu[n + 1] - cu[n]
        z[cu[n]:cu[n + 1]] = _wide(st["bias"]) + sum(w[:, k] * line[k:k + L] for k in range(K))
        state[n] = line[L:]
    return {"y": (z * torch.sigmoid(z) if case["silu"] else z).reshape(st["x"].shape), "state": state}
