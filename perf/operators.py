"""The state-space and rotary operators as they are measured: cases, inputs, plain forms, definitions.

With ``own`` false, ``run`` computes each operator in elementary torch operations in 32 bits
(the rotary angles in 64); with ``own`` true it makes the calls a user makes of
recurrent_state_scan_gb300.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases
def _prompt(name, dtype, lens, heads, head_dim, groups, d_state, kernel, z, initial, packed=True):
    return {"name": name, "op": "ssm_prefill", "dtype": dtype, "lens": ",".join(map(str, lens)), "heads": heads,
            "head_dim": head_dim, "groups": groups, "d_state": d_state, "kernel": kernel, "z": z, "initial": initial,
            "packed": packed}


def _token(name, dtype, batch, heads, head_dim, groups, d_state, kernel, z, slots):
    return {"name": name, "op": "ssm_decode", "dtype": dtype, "batch": batch, "heads": heads, "head_dim": head_dim,
            "groups": groups, "d_state": d_state, "kernel": kernel, "z": z, "slots": slots}


def _rotary(name, dtype, tokens, hq, hk, dim, rot, offset, interleaved, far, inverse, mixed):
    return {"name": name, "op": "rotary", "dtype": dtype, "tokens": tokens, "hq": hq, "hk": hk, "dim": dim,
            "rot": rot, "offset": offset, "interleaved": interleaved, "far": far, "inverse": inverse, "mixed": mixed}


def listed():
    return [
        # One long prompt of a state-space layer: conv, gate, no earlier state.
        _prompt("prompt_8k", "bf16", [8192], 64, 64, 1, 128, 4, True, False, False),
        # A server's packed prefill: ragged prompts, each resuming from a state, B and C in groups.
        _prompt("prompts_packed", "bf16", [4001, 17, 2900, 1, 650, 3333, 128, 1200, 63, 2048, 900, 1143], 64, 64, 8, 128, 4,
                False, True),
        # The largest: a full batch of long prompts, already convolved.
        _prompt("prompts_64k", "bf16", [16384, 8192, 12288, 4096, 20480, 4096], 64, 64, 8, 128, 0, False, True),
        # One short prompt: latency.
        _prompt("prompt_short", "bf16", [37], 32, 64, 1, 64, 4, True, False, False),
        # 16-bit floats, a batch of equal rows with an odd length.
        _prompt("prompt_f16", "f16", [1001, 1001], 24, 64, 1, 128, 4, False, True, False),
        # 32-bit, a smaller state.
        _prompt("prompt_f32", "f32", [700, 45, 300], 16, 32, 2, 48, 3, True, True),
        # Continuous batching: 256 requests' next tokens against pools of states.
        _token("tokens_256_slots", "bf16", 256, 64, 64, 8, 128, 4, True, True),
        # A single request's next token: latency.
        _token("token_1", "bf16", 1, 64, 64, 1, 128, 4, True, False),
        # 32-bit, odd sizes, already convolved.
        _token("tokens_f32_odd", "f32", 33, 20, 52, 4, 90, 0, False, False),
        # Queries and keys of a long prompt, half layout, the whole head.
        _rotary("rotary_32k", "bf16", 32768, 32, 8, 128, 128, 0, False, False, False, False),
        # The next tokens of 64 far-advanced requests: interleaved, part of the head.
        _rotary("rotary_tokens", "bf16", 64, 16, 2, 128, 64, 64, True, True, False, False),
        # C and B inside the mixed row of a state-space layer, in place there; the turn's inverse.
        _rotary("rotary_mixed_row", "f16", 5003, 8, 8, 96, 80, 0, False, False, True, True),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["ssm_prefill", "ssm_prefill", "ssm_decode", "rotary"])
    if op == "ssm_prefill":
        dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
        groups = rng.choice([1, 1, 2, 4, 8])
        heads = groups * rng.randint(max(1, 8 // groups), 64 // groups)
        head_dim = rng.choice([32, 48, 64, 64, 64, 80, 128])
        d_state = rng.choice([16, 48, 64, 100, 128, 128])
        total = log(1, 32768 if dtype == "bf16" else 2048)
        total = max(1, min(total, 65536 * 64 // (heads * max(1, head_dim // 64) * 2)))
        packed = rng.random() < 0.6
        if packed:
            n = rng.randint(1, 12)
            cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        else:
            n = min(total, rng.choice([1, 1, 2, 3, 5]))
            lens = [max(1, total // n)] * n
        c = _prompt("", dtype, lens, heads, head_dim, groups, d_state, rng.choice([0, 2, 3, 4, 4, 4]), rng.random() < 0.5,
                    rng.random() < 0.5, packed)
    elif op == "ssm_decode":
        groups = rng.choice([1, 1, 2, 4, 8])
        c = _token("", rng.choice(["bf16", "bf16", "f16", "f32"]), log(1, 256), groups * rng.randint(max(1, 8 // groups), 64 // groups),
                   rng.choice([32, 48, 64, 64, 64, 80]), groups, rng.choice([16, 64, 100, 128, 128]), rng.choice([0, 2, 3, 4, 4]),
                   rng.random() < 0.5, rng.random() < 0.5)
    else:
        dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        rot = rng.choice([dim, dim, dim // 2 // 2 * 2, 64])
        c = _rotary("", rng.choice(["bf16", "bf16", "f16", "f32"]), log(1, 16384), rng.choice([1, 4, 8, 16, 28, 32]),
                    rng.choice([1, 2, 4, 8]), dim, rot, rng.choice([0, dim - rot]), rng.random() < 0.5, rng.random() < 0.5,
                    rng.random() < 0.3, rng.random() < 0.3)
    del c["name"]
    return c


# ---------------------------------------------------------------------------- inputs
def _lens(case):
    return [int(s) for s in case["lens"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    io = _DT[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    s = {"case": dict(case)}
    if case["op"] == "rotary":
        T, hq, hk, D = case["tokens"], case["hq"], case["hk"], case["dim"]
        if case["mixed"]:   # [other | k | q], as B and C stand behind x in a layer's mixed row
            row = normal(1, T, 256 + (hk + hq) * D).to(io)
            s["k"] = row[:, :, 256:256 + hk * D].unflatten(2, (hk, D))
            s["q"] = row[:, :, 256 + hk * D:].unflatten(2, (hq, D))
        else:
            s["q"], s["k"] = normal(1, T, hq, D).to(io), normal(1, T, hk, D).to(io)
        s["inv_freq"] = (1e4 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])).float()
        top = 1 << 20 if case["far"] else 4096
        pos = torch.randint(0, top, (1, T), generator=g, device="cuda", dtype=torch.int32) if case["far"] \
            else torch.arange(T, device="cuda", dtype=torch.int32)[None] + 7
        s["positions"], s["scale"] = pos, 1.1 if case["far"] else 1.0
        return s
    H, P, G, N, K = (case[k] for k in ("heads", "head_dim", "groups", "d_state", "kernel"))
    C = H * P + 2 * G * N
    if case["op"] == "ssm_prefill":
        lens = _lens(case)
        B, T, n = (1, sum(lens), len(lens)) if case["packed"] else (len(lens), lens[0], len(lens))
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda") if case["packed"] else None
    else:
        B, T, n = case["batch"], 1, case["batch"]
    # The layer's projection lays z, the mixed row and dt out beside one another.
    width = (H * P if case["z"] else 0) + C + H
    width += -width % 8
    row = normal(B, T, width).to(io)
    at = H * P if case["z"] else 0
    s["z"] = row[:, :, :at].unflatten(2, (H, P)) if case["z"] else None
    s["xbc"], s["dt"] = row[:, :, at:at + C], row[:, :, at + C:at + C + H]
    s["A_log"] = torch.log(uniform(1.0, 16.0, H))
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), H))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["D"] = uniform(0.5, 1.5, H)
    s["w"] = uniform(-K ** -0.5, K ** -0.5, C, 1, K).to(io) if K else None
    s["bias"] = normal(C, std=0.1).to(io) if K else None
    if case["op"] == "ssm_prefill":
        s["state"] = normal(n, H, N, P, std=0.3) if case["initial"] else None
        s["conv_state"] = normal(n, K - 1, C).to(io) if K and case["initial"] else None
    else:
        pool = B + B // 4 + 1 if case["slots"] else B
        s["state"] = normal(pool, H, N, P, std=0.3)
        s["conv_state"] = normal(pool, K - 1, C).to(io) if K else None
        s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:B].to(torch.int32) if case["slots"] else None
    return s


# ---------------------------------------------------------------------------- the framework's calls
def _own(s):
    import recurrent_state_scan_gb300 as lib
    c = s["case"]
    if c["op"] == "rotary":
        q, k = lib.gdn_rotary(s["q"], s["k"], s["inv_freq"], positions=s["positions"], rot_offset=c["offset"],
                              interleaved=c["interleaved"], inverse=c["inverse"], scale=s["scale"])
        return {"q": q, "k": k}
    kw = dict(heads=c["heads"], head_dim=c["head_dim"], groups=c["groups"], d_state=c["d_state"], D=s["D"], dt_bias=s["dt_bias"],
              z=s["z"], conv_weight=s["w"], conv_bias=s["bias"])
    if c["op"] == "ssm_prefill":
        y, state, conv = lib.gdn_ssm_prefill(s["xbc"], s["dt"], s["A_log"], state_in=s["state"], conv_state_in=s["conv_state"],
                                             cu_seqlens=s["cu"], **kw)
        return {"y": y, "state": state, "conv_state": conv}
    y = lib.gdn_ssm_decode(s["xbc"], s["dt"], s["A_log"], s["state"], conv_state=s["conv_state"], slots=s["slots"], **kw)
    return {"y": y, "state": s["state"], "conv_state": s["conv_state"]}


# ---------------------------------------------------------------------------- the plain forms (32 bits)
CHUNK = 64


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"].double()[..., None, None] * s["inv_freq"].double()
    cos, sin = (angle.cos() * s["scale"]).float(), (angle.sin() * s["scale"]).float()
    sin = -sin if c["inverse"] else sin

    def turn(t):
        part = t[..., c["offset"]:c["offset"] + c["rot"]].float()
        pair = part.unflatten(-1, (-1, 2)).transpose(-1, -2) if c["interleaved"] else part.unflatten(-1, (2, -1))
        a, b = pair[..., 0, :], pair[..., 1, :]
        pair = torch.stack((a * cos - b * sin, b * cos + a * sin), -2)
        out = t.clone()
        out[..., c["offset"]:c["offset"] + c["rot"]] = \
            (pair.transpose(-1, -2) if c["interleaved"] else pair).flatten(-2).to(t.dtype)
        return out

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _conv(s, pad, T):
    """The causal convolution over pad [n, K - 1 + T, C] and silu, rounded to the I/O type as the layer's conv stores it."""
    w = s["w"].float()
    u = sum((w[:, 0, j] * pad[:, j:j + T] for j in range(w.shape[2])), s["bias"].float())
    return (u / (1 + torch.exp(-u))).to(s["xbc"].dtype).float()


def _gates(s, dt):
    """(step, log decay) of dt [..., H]: the step is softplus(dt + dt_bias)."""
    d = dt.float() + s["dt_bias"]
    d = d.clamp_min(0) + torch.log1p(torch.exp(-d.abs()))
    return d, -torch.exp(s["A_log"]) * d


def _finish(s, y, x, io):
    """The skip D x, the gate silu(z), and the one rounding to the I/O type."""
    y = y + s["D"][:, None] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z / (1 + torch.exp(-z)))
    return y.to(io)


def _plain_prefill(s):
    c, io = s["case"], s["xbc"].dtype
    H, P, G, N, K = (c[k] for k in ("heads", "head_dim", "groups", "d_state", "kernel"))
    B, tokens, C = s["xbc"].shape
    lens = _lens(c)
    x, dt = s["xbc"].float(), s["dt"].float()
    at = None
    if s["cu"] is not None:
        place = torch.arange(max(lens), device=x.device)
        ends = s["cu"].long()
        at = torch.where(place < (ends[1:] - ends[:-1])[:, None], ends[:-1, None] + place, tokens)   # [n, Tmax]
        x = torch.cat([x[0], x.new_zeros(1, C)])[at]
        dt = torch.cat([dt[0], dt.new_zeros(1, H)])[at]
    n, T = x.shape[:2]
    conv_state = None
    if K:
        past = s["conv_state"].float() if s["conv_state"] is not None else x.new_zeros(n, K - 1, C)
        pad = torch.cat([past, x], 1)
        last = torch.tensor(lens, device=x.device)[:, None] + torch.arange(K - 1, device=x.device)
        conv_state = pad.gather(1, last[..., None].expand(-1, -1, C)).to(io)
        x = _conv(s, pad, T)
    d, la = _gates(s, dt)
    if at is not None:
        d, la = d * (at < tokens)[..., None], la * (at < tokens)[..., None]
    # Chunks of L tokens: inside one by its decay matrix, across them by the chunks' decay matrix.
    L = min(CHUNK, max(T, 1))
    nc = -(-T // L)
    x, d, la = (torch.cat([t, t.new_zeros(n, nc * L - T, t.shape[2])], 1).unflatten(1, (nc, L)) for t in (x, d, la))
    u = x[..., :H * P].unflatten(3, (H, P)).permute(0, 1, 3, 2, 4)                            # [n, nc, H, L, P]
    b = x[..., H * P:H * P + G * N].unflatten(3, (G, N)).permute(0, 1, 3, 2, 4)               # [n, nc, G, L, N]
    q = x[..., H * P + G * N:].unflatten(3, (G, N)).permute(0, 1, 3, 2, 4)
    d, cum = d.transpose(2, 3), la.transpose(2, 3).double().cumsum(-1)                        # [n, nc, H, L]
    within = torch.exp((cum[..., :, None] - cum[..., None, :]).float().masked_fill(
        ~torch.ones(L, L, dtype=torch.bool, device=x.device).tril(), -math.inf))
    m = within.unflatten(2, (G, H // G)) * (q @ b.transpose(-1, -2))[:, :, :, None]
    y = (m.flatten(2, 3) * d[..., None, :]) @ u
    left = d * torch.exp((cum[..., -1:] - cum).float())
    local = b.transpose(-1, -2)[:, :, :, None] @ (left[..., None] * u).unflatten(2, (G, H // G))
    local = local.flatten(2, 3).permute(0, 2, 1, 3, 4).flatten(3)                             # [n, H, nc, N P]
    ends = torch.cat([cum.new_zeros(n, H, 1), cum[..., -1].transpose(1, 2).cumsum(-1)], -1)  # [n, H, nc + 1]
    # State before chunk i (i = nc: the last): sum over j < i of e^(ends_i - ends_{j+1}) local_j, and the first state's part.
    over = torch.exp((ends[..., :, None] - ends[..., None, 1:]).float().masked_fill(
        ~torch.ones(nc + 1, nc, dtype=torch.bool, device=x.device).tril(-1), -math.inf))
    states = over @ local
    if s["state"] is not None:
        states = states + torch.exp(ends.float())[..., None] * s["state"].flatten(2)[:, :, None]
    states = states.unflatten(3, (N, P)).permute(0, 2, 1, 3, 4)                               # [n, nc + 1, H, N, P]
    reach = (q[:, :, :, None] * torch.exp(cum.float()).unflatten(2, (G, H // G))[..., None]).flatten(2, 3)
    y = y + reach @ states[:, :-1]

    def back(t):   # [n, nc, H, L, P] as the tokens lie
        t = t.permute(0, 1, 3, 2, 4).flatten(1, 2)[:, :T]
        return t if at is None else t[at < tokens][None]

    return {"y": _finish(s, back(y), back(u), io), "state": states[:, -1].contiguous(), "conv_state": conv_state}


def _plain_decode(s):
    c, io = s["case"], s["xbc"].dtype
    H, P, G, N, K = (c[k] for k in ("heads", "head_dim", "groups", "d_state", "kernel"))
    x = s["xbc"].float()
    at = s["slots"].long() if s["slots"] is not None else torch.arange(x.shape[0], device=x.device)
    if K:
        pad = torch.cat([s["conv_state"][at].float(), x], 1)
        s["conv_state"][at] = pad[:, 1:].to(io)
        x = _conv(s, pad, 1)
    d, la = _gates(s, s["dt"][:, 0])                                                          # [B, H]
    u = x[:, 0, :H * P].unflatten(1, (H, P))
    b = x[:, 0, H * P:H * P + G * N].unflatten(1, (G, N)).repeat_interleave(H // G, 1)
    q = x[:, 0, H * P + G * N:].unflatten(1, (G, N)).repeat_interleave(H // G, 1)
    state = s["state"][at] * torch.exp(la)[..., None, None] + b[..., None] * (d[..., None] * u)[:, :, None, :]
    s["state"][at] = state
    y = (q[..., None] * state).sum(2)
    return {"y": _finish(s, y[:, None], u[:, None], io), "state": s["state"], "conv_state": s["conv_state"]}


def run(state):
    if own:
        return _own(state)
    return {"rotary": _plain_rotary, "ssm_prefill": _plain_prefill, "ssm_decode": _plain_decode}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------- the work of one pass
def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rotary":
        values = case["tokens"] * (case["hq"] + case["hk"])
        return {"bytes": 2 * es * values * case["dim"] + 4 * case["tokens"] + 2 * case["rot"], "flops": 3 * values * case["rot"]}
    H, P, G, N, K = (case[k] for k in ("heads", "head_dim", "groups", "d_state", "kernel"))
    C = H * P + 2 * G * N
    lens = _lens(case) if case["op"] == "ssm_prefill" else [1] * case["batch"]
    tokens, n = sum(lens), len(lens)
    both = case["op"] == "ssm_decode" or case["initial"]
    bytes_ = tokens * es * (C + H + H * P * (2 if case["z"] else 1)) + 4 * n * H * N * P * (2 if both else 1)
    bytes_ += (es * C * (K + 1) + es * n * (K - 1) * C * (2 if both else 1)) if K else 0
    # The state's update and its readout; the convolution.
    return {"bytes": bytes_ + 12 * H, "flops": tokens * (4 * H * N * P + 2 * C * K)}


# ---------------------------------------------------------------------------- the definitions (64 bits)
def _exact_sequence(s, x, dt, z, past, state):
    """The recurrence as it is defined, token by token: x [n, T, C], dt [n, T, H], past [n, K - 1, C], state [n, H, N, P]."""
    c, io = s["case"], s["xbc"].dtype
    H, P, G, N, K = (c[k] for k in ("heads", "head_dim", "groups", "d_state", "kernel"))
    n, T, C = x.shape
    if K:
        taps = torch.cat([past, x], 1).unfold(1, K, 1)                                        # [n, T, C, K]
        u = torch.einsum("ntck,ck->ntc", taps, s["w"][:, 0].double()) + s["bias"].double()
        x = (u * torch.sigmoid(u)).to(io).double()
    step = torch.logaddexp(torch.zeros((), dtype=torch.float64, device=x.device), dt + s["dt_bias"].double())
    keep = torch.exp(-step * torch.exp(s["A_log"].double()))
    share = torch.arange(H, device=x.device) // (H // G)
    ys = x.new_empty(n, T, H, P)
    for t in range(T):
        u = x[:, t, :H * P].view(n, H, P)
        b = x[:, t, H * P:H * P + G * N].view(n, G, N)[:, share]
        q = x[:, t, H * P + G * N:].view(n, G, N)[:, share]
        state = state * keep[:, t, :, None, None]
        state += (step[:, t, :, None] * b)[..., None] * u[:, :, None]
        ys[:, t] = (q[:, :, None] @ state)[:, :, 0]
    ys += s["D"].double()[:, None] * x[..., :H * P].unflatten(2, (H, P))
    if z is not None:
        ys = ys * (z * torch.sigmoid(z))
    return ys, state


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        turn = torch.polar(torch.full((), s["scale"], dtype=torch.float64, device="cuda"),
                           s["positions"].double()[..., None, None] * s["inv_freq"].double() * (-1.0 if case["inverse"] else 1.0))
        out = {}
        for name in ("q", "k"):
            t, r, o = s[name].double(), case["rot"], case["offset"]
            first = torch.arange(0, r, 2, device="cuda") if case["interleaved"] else torch.arange(r // 2, device="cuda")
            second = o + first + (1 if case["interleaved"] else r // 2)
            v = torch.complex(t[..., o + first], t[..., second]) * turn
            t[..., o + first], t[..., second] = v.real, v.imag
            out[name] = t
        return out
    H, N, P, K = (case[k] for k in ("heads", "d_state", "head_dim", "kernel"))
    C = s["xbc"].shape[2]
    if case["op"] == "ssm_decode":
        at = s["slots"].long() if case["slots"] else torch.arange(case["batch"], device="cuda")
        past = s["conv_state"][at].double() if K else None
        z = s["z"].double() if case["z"] else None
        y, state = _exact_sequence(s, s["xbc"].double(), s["dt"].double(), z, past, s["state"][at].double())
        pool = s["state"].double()
        pool[at] = state
        conv = None
        if K:
            conv = s["conv_state"].double()
            conv[at] = torch.cat([past, s["xbc"].double()], 1)[:, 1:]
        return {"y": y, "state": pool, "conv_state": conv}
    lens = _lens(case)
    tokens, n = sum(lens), len(lens)
    spans = [(sum(lens[:i]), sum(lens[:i + 1])) for i in range(n)]
    x, dt = s["xbc"].reshape(tokens, C).double(), s["dt"].reshape(tokens, H).double()
    z = s["z"].reshape(tokens, H, P).double() if case["z"] else None
    first = s["state"].double() if case["initial"] else x.new_zeros(n, H, N, P)
    past = (s["conv_state"].double() if case["initial"] else x.new_zeros(n, K - 1, C)) if K else None
    y, state, conv = x.new_empty(tokens, H, P), first.clone(), None if past is None else past.clone()
    # Sequences of one length together.
    for length in sorted(set(lens) - {0}):
        of = [i for i in range(n) if lens[i] == length]
        rows = torch.stack([torch.arange(*spans[i], device="cuda") for i in of])
        got, last = _exact_sequence(s, x[rows], dt[rows], None if z is None else z[rows], None if past is None else past[of], first[of])
        y[rows], state[of] = got, last
        if K:
            conv[of] = torch.cat([past[of], x[rows]], 1)[:, length:]
    return {"y": y.view(s["xbc"].shape[0], -1, H, P), "state": state, "conv_state": conv}
