"""The diagonal recurrence and its 8-bit checkpoints as they are measured: cases, inputs, plain forms, definitions.

With ``own`` false, ``run`` computes each operator in elementary torch operations in 32 bits; with
``own`` true it makes the calls a user makes of recurrent_state_scan_gb300.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CHUNK = 64      # rows between the states that a training step keeps
BLOCK = 64      # channels that share a step of the 8-bit codes


# ---------------------------------------------------------------------------- cases
def _rows(name, op, dtype, lens, channels, gate, weighting, b, initial, packed=True, bits=0, tight=False):
    return {"name": name, "op": op, "dtype": dtype, "lens": ",".join(map(str, lens)), "channels": channels, "gate": gate,
            "weighting": weighting, "b": b, "initial": initial, "packed": packed, "bits": bits, "tight": tight}


def _token(name, dtype, batch, channels, gate, weighting, b, slots):
    return {"name": name, "op": "decode", "dtype": dtype, "batch": batch, "channels": channels, "gate": gate, "weighting": weighting,
            "b": b, "slots": slots, "tight": False}


def _codes(name, dtype, rows, channels):
    return {"name": name, "op": "codes", "dtype": dtype, "rows": rows, "channels": channels}


def listed():
    return [
        # One long prompt of a recurrent layer with both gates, no earlier state.
        _rows("prompt_8k", "prefill", "bf16", [8192], 4096, "sigmoid", "norm", True, False, False),
        # A server's packed prefill: ragged prompts, each resuming from a state, the layer's own softplus gate.
        _rows("prompts_packed", "prefill", "bf16", [4001, 17, 2900, 1, 650, 3333, 128, 1200, 63, 2048, 900, 1143], 2560, "softplus",
              "complement", True, True),
        # One short prompt: latency.
        _rows("prompt_short", "prefill", "bf16", [37], 2048, "sigmoid", "norm", True, False, False),
        # 32-bit, an odd width, no input gate.
        _rows("prompts_f32_odd", "prefill", "f32", [700, 45, 300], 1001, "softplus", "plain", False, True),
        # A training step's share of this layer: the forward pass and the backward pass of a batch, the largest case.
        _rows("train_16k", "train", "bf16", [4096] * 4, 4096, "sigmoid", "norm", True, False, False),
        # The same, the inputs kept for the backward pass in 8 bits.
        _rows("train_16k_8bit", "train", "bf16", [4096] * 4, 4096, "sigmoid", "norm", True, False, False, 8),
        # Packed documents, some of them continued from an earlier part (their gradients handed back), 16-bit floats, 8-bit checkpoints.
        _rows("train_packed_f16", "train", "f16", [1500, 3, 700, 64, 1201, 1, 0, 627], 1536, "softplus", "complement", True, True, True, 8),
        # 32-bit training, small.
        _rows("train_f32", "train", "f32", [500, 77, 1, 423], 640, "sigmoid", "plain", True, True),
        # Continuous batching: 256 requests' next tokens against a pool of states.
        _token("tokens_256_slots", "bf16", 256, 4096, "sigmoid", "norm", True, True),
        # A single request's next token: latency.
        _token("token_1", "bf16", 1, 2560, "softplus", "complement", True, False),
        # Any other activation of a layer kept in 8 bits and read back: long rows, and an odd width.
        _codes("codes_16k", "bf16", 16384, 4096),
        _codes("codes_f16_odd", "f16", 1001, 1111),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["prefill", "prefill", "train", "train", "train", "decode", "codes"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    channels = log(64, 5120)
    channels = channels if rng.random() < 0.3 else max(64, channels // 64 * 64)
    gate, weighting = rng.choice(["softplus", "sigmoid"]), rng.choice(["norm", "norm", "complement", "plain"])
    if op == "codes":
        c = _codes("", dtype, log(1, 16384), channels)
    elif op == "decode":
        c = _token("", dtype, log(1, 512), channels, gate, weighting, rng.random() < 0.8, rng.random() < 0.5)
        c["tight"] = rng.random() < 0.2
    else:
        total = log(1, 16384 if dtype != "f32" else 6000)
        packed = rng.random() < 0.6
        if packed:
            n = rng.randint(1, 12)
            cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        else:
            n = min(total, rng.choice([1, 1, 2, 3, 5]))
            lens = [max(1, total // n)] * n
        c = _rows("", op, dtype, lens, min(channels, 4096), gate, weighting, rng.random() < 0.8, rng.random() < 0.5, packed,
                  rng.choice([0, 8]) if op == "train" else 0, rng.random() < 0.2)
    del c["name"]
    return c


# ---------------------------------------------------------------------------- inputs
def _lens(case):
    return [int(s) for s in case["lens"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    io, C = _DT[case["dtype"]], case["channels"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    s = {"case": dict(case)}
    if case["op"] == "codes":
        # Activations: a few channels far larger than the others, as trained layers have them.
        s["x"] = (normal(1, case["rows"], C) * torch.exp(normal(C))).to(io)
        return s
    if case["op"] == "decode":
        B, T, n = case["batch"], 1, case["batch"]
    else:
        lens = _lens(case)
        B, T, n = (1, sum(lens), len(lens)) if case["packed"] else (len(lens), lens[0], len(lens))
        ends = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
        s["cu"] = ends if case["packed"] else None
        # The rows that begin and end a sequence, and the sequences that have any.
        some = torch.tensor([i for i in range(n) if lens[i]], dtype=torch.long, device="cuda")
        s["edges"] = ends[:-1][some].long(), ends[1:][some].long() - 1, some
    # x, a and b are parts of one projection's rows.
    part = C if case["tight"] else C + -C % 8
    row = normal(B, T, part * (3 if case["b"] else 2)).to(io)
    s["x"], s["a"] = row[:, :, :C], row[:, :, part:part + C]
    s["b"] = row[:, :, 2 * part:2 * part + C] if case["b"] else None
    if case["gate"] == "sigmoid":     # decays of 0.9 to 0.999 where the gate is open
        s["A_log"], s["a_bias"] = torch.log(-torch.log(uniform(0.9, 0.999, C))), normal(C, std=0.5)
    else:                             # the layer's usual rates and steps
        s["A_log"] = torch.log(uniform(1.0, 16.0, C))
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), C))
        s["a_bias"] = step + torch.log(-torch.expm1(-step))
    s["b_bias"] = normal(C, std=0.5) if case["b"] else None
    if case["op"] == "decode":
        pool = B + B // 4 + 1 if case["slots"] else B
        s["state"] = normal(pool, C)
        s["slots"] = torch.randperm(pool, generator=g, device="cuda")[:B].to(torch.int32) if case["slots"] else None
        return s
    s["state"] = normal(n, C) if case["initial"] else None
    if case["op"] == "train":
        s["dy"] = normal(B, T, C).to(io)
        s["dstate"] = normal(n, C) if case["initial"] else None
    return s


# ---------------------------------------------------------------------------- the framework's calls
def _own(s):
    import recurrent_state_scan_gb300 as lib
    c = s["case"]
    if c["op"] == "codes":
        codes, steps = lib.gdn_checkpoint_pack(s["x"])
        return {"x": lib.gdn_checkpoint_unpack(codes, steps, s["x"].dtype)}
    kw = dict(a_bias=s["a_bias"], b_bias=s["b_bias"], gate=c["gate"], weighting=c["weighting"])
    if c["op"] == "decode":
        y = lib.gdn_diag_decode(s["x"], s["a"], s["b"], s["A_log"], s["state"], slots=s["slots"], **kw)
        return {"y": y, "state": s["state"]}
    keep = None if c["op"] == "prefill" else "8bit" if c["bits"] else "states"
    y, state, kept = lib.gdn_diag_prefill(s["x"], s["a"], s["b"], s["A_log"], state_in=s["state"], cu_seqlens=s["cu"], keep=keep, **kw)
    if c["op"] == "prefill":
        return {"y": y, "state": state}
    held = {} if c["bits"] else dict(x=s["x"], a=s["a"], b=s["b"])
    dx, da, db, dA_log, da_bias, db_bias, dstate = lib.gdn_diag_backward(
        s["dy"], kept, s["A_log"], a_bias=s["a_bias"], b_bias=s["b_bias"], state_in=s["state"], cu_seqlens=s["cu"],
        dstate_out=s["dstate"], **held)
    return {"y": y, "state": state, "dx": dx, "da": da, "db": db, "dA_log": dA_log, "da_bias": da_bias, "db_bias": db_bias,
            "dstate": dstate}


# ---------------------------------------------------------------------------- the plain forms (32 bits)
def _gates(s, x, a, b):
    """(decay, weight of the gated input, gated input, log decay, open gate, input gate) of rows [n, C]."""
    c = s["case"]
    z = a + s["a_bias"]
    gate = 1 / (1 + torch.exp(-z))
    opening = gate if c["gate"] == "sigmoid" else z.clamp_min(0) + torch.log1p(torch.exp(-z.abs()))
    g = -torch.exp(s["A_log"]) * opening
    i = 1 / (1 + torch.exp(-(b + s["b_bias"]))) if b is not None else torch.ones_like(x)
    w = torch.sqrt(-torch.expm1(2 * g)) if c["weighting"] == "norm" else -torch.expm1(g) if c["weighting"] == "complement" else torch.ones_like(g)
    return torch.exp(g), w, i * x, g, gate, i


def _scan(keep, add):
    """h_t = keep_t h_(t-1) + add_t down the rows, in doubling steps."""
    keep, add, d = keep.clone(), add.clone(), 1
    while d < add.shape[0]:
        add[d:] += keep[d:] * add[:-d]
        keep[d:] *= keep[:-d].clone()
        d *= 2
    return add


def _stored(x):
    """x [rows, C] as 8-bit codes with a step per row and BLOCK channels hold it."""
    rows, C = x.shape
    v = torch.cat([x, x.new_zeros(rows, -C % BLOCK)], 1).view(rows, -1, BLOCK)
    m, e = torch.frexp(v.abs().amax(-1, keepdim=True))
    step = ((e - 7 + (m >= 255 / 256)).clamp_min(-117).int() + 127 << 23).view(torch.float32)     # that power of two
    return (torch.round(v / step).clamp(-127, 127) * step).view(rows, -1)[:, :C]


def _plain_rows(s):
    c, io = s["case"], s["x"].dtype
    B, T, C = s["x"].shape
    rows = B * T
    flat = lambda t: None if t is None else t.reshape(rows, C).float()  # noqa: E731
    x, a, b = flat(s["x"]), flat(s["a"]), flat(s["b"])
    first, last, some = s["edges"]
    start = s["state"] if s["state"] is not None else x.new_zeros(len(_lens(c)), C)
    keep, w, v, *_ = _gates(s, x, a, b)
    inner, add = keep.clone(), w * v
    inner[first] = 0
    add[first] += keep[first] * start[some]
    h = _scan(inner, add)
    state = start.clone()
    state[some] = h[last]
    out = {"y": h.to(io).view(B, T, C), "state": state}
    if c["op"] == "prefill":
        return out
    past = torch.cat([h.new_zeros(1, C), h[:-1]])
    past[first] = start[some]
    if c["bits"]:       # what the codes hold, from the kept states on
        x, a, b = _stored(x), _stored(a), None if b is None else _stored(b)
        keep, w, v, *_ = _gates(s, x, a, b)
        inner, add = keep.clone(), w * v
        begin = torch.cat([first, torch.arange(0, rows, CHUNK, device="cuda")]).unique()
        inner[begin] = 0
        add[begin] += keep[begin] * past[begin]
        again = _scan(inner, add)
        again = torch.cat([again.new_zeros(1, C), again[:-1]])
        again[begin] = past[begin]
        past = again
    keep, w, v, g, gate, i = _gates(s, x, a, b)
    inner = keep.clone()
    inner[first] = 0
    add = s["dy"].reshape(rows, C).float()
    if s["dstate"] is not None:
        add = add.index_add(0, last, s["dstate"][some])
    back = torch.cat([inner[1:], inner.new_zeros(1, C)]).flip(0)
    G = _scan(back, add.flip(0)).flip(0)
    turn = -torch.exp(2 * g) / w if c["weighting"] == "norm" else -keep if c["weighting"] == "complement" else torch.zeros_like(g)
    dg = G * (keep * past + v * turn)
    dx = G * w * i
    da = dg * g * (1 - gate) if c["gate"] == "sigmoid" else -dg * torch.exp(s["A_log"]) * gate
    db = dx * x * (1 - i) if b is not None else None
    dstate = None
    if s["state"] is not None:
        dstate = torch.zeros_like(start) if s["dstate"] is None else s["dstate"].clone()
        dstate[some] = keep[first] * G[first]
    shaped = lambda t: None if t is None else t.to(io).view(B, T, C)  # noqa: E731
    return {**out, "dx": shaped(dx), "da": shaped(da), "db": shaped(db), "dA_log": (dg * g).sum(0), "da_bias": da.sum(0),
            "db_bias": None if db is None else db.sum(0), "dstate": dstate}


def _plain_decode(s):
    at = s["slots"].long() if s["slots"] is not None else torch.arange(s["x"].shape[0], device="cuda")
    x, a = s["x"][:, 0].float(), s["a"][:, 0].float()
    keep, w, v, *_ = _gates(s, x, a, None if s["b"] is None else s["b"][:, 0].float())
    h = keep * s["state"][at] + w * v
    s["state"][at] = h
    return {"y": h.to(s["x"].dtype)[:, None], "state": s["state"]}


def run(state):
    if own:
        return _own(state)
    if state["case"]["op"] == "codes":
        return {"x": _stored(state["x"][0].float()).to(state["x"].dtype)[None]}
    return _plain_decode(state) if state["case"]["op"] == "decode" else _plain_rows(state)


# ---------------------------------------------------------------------------- the work of one pass
def work(case):
    es, C = 4 if case["dtype"] == "f32" else 2, case["channels"]
    if case["op"] == "codes":           # x, the codes out and in, x again
        blocks = -(-C // BLOCK)
        return {"bytes": case["rows"] * (2 * es * C + 2 * C + 2 * blocks), "flops": 3 * case["rows"] * C}
    ins = 3 if case["b"] else 2
    params = 4 * C * ins
    if case["op"] == "decode":
        return {"bytes": case["batch"] * C * (es * (ins + 1) + 8) + params, "flops": case["batch"] * C * 14}
    lens = _lens(case)
    n, rows = len(lens), sum(lens)
    states = 4 * n * C * (2 if case["initial"] else 1)
    if case["op"] == "prefill":
        return {"bytes": rows * C * es * (ins + 1) + states + params, "flops": rows * C * 14}
    # x, a, b and dy in, y, dx, da and db out, each once, although the backward pass has to meet x, a and b (or their codes) again.
    return {"bytes": rows * C * es * (2 * ins + 2) + 2 * states + 2 * params, "flops": rows * C * 45}


# ---------------------------------------------------------------------------- the definitions (64 bits)
def _decay_and_input(case, x, a, b, A_log, a_bias, b_bias):
    z = a + a_bias
    amount = torch.sigmoid(z) if case["gate"] == "sigmoid" else torch.logaddexp(torch.zeros_like(z), z)
    g = -A_log.exp() * amount
    v = x if b is None else torch.sigmoid(b + b_bias) * x
    if case["weighting"] == "norm":
        v = v * (-torch.expm1(2 * g)) ** 0.5
    elif case["weighting"] == "complement":
        v = v * -torch.expm1(g)
    return g.exp(), v


def _held(t):
    """What 8 bits hold: the nearest multiple of the least power of two that keeps a block's values below 127.5 of it."""
    rows, C = t.shape
    out = torch.empty_like(t)
    for lo in range(0, C, BLOCK):
        v = t[:, lo:lo + BLOCK]
        most = v.abs().max(1, keepdim=True).values
        e = torch.where(most > 0, torch.floor(torch.log2(most / 127.5)) + 1, torch.full_like(most, -117)).clamp_min(-117)
        step = (e.long() + 1023 << 52).view(torch.float64)       # 2^e
        out[:, lo:lo + BLOCK] = torch.round(v / step).clamp(-127, 127) * step
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "codes":
        return {"x": _held(s["x"][0].double())[None]}
    wide = {k: None if s.get(k) is None else s[k].double() for k in ("x", "a", "b", "A_log", "a_bias", "b_bias", "state", "dy", "dstate")}
    B, T, C = s["x"].shape
    if case["op"] == "decode":
        at = s["slots"].long() if case["slots"] else torch.arange(B, device="cuda")
        alpha, v = _decay_and_input(case, wide["x"], wide["a"], wide["b"], wide["A_log"], wide["a_bias"], wide["b_bias"])
        h = alpha[:, 0] * wide["state"][at] + v[:, 0]
        wide["state"][at] = h
        return {"y": h[:, None], "state": wide["state"]}
    rows, lens = B * T, _lens(case)
    begin = [sum(lens[:i]) for i in range(len(lens))]
    # Sequences in lockstep: at step t the rows of those that are longer.
    steps, of = [], []
    for t in range(max(lens)):
        alive = [i for i, length in enumerate(lens) if length > t]
        if t == 0 or len(alive) != len(of[-1]):
            of.append(torch.tensor(alive, device="cuda"))
            base = torch.tensor([begin[i] for i in alive], device="cuda")
        else:
            of.append(of[-1])
        steps.append(base + t)
    flat = lambda t: None if t is None else t.reshape(rows, C)  # noqa: E731
    leaves = [flat(wide["x"]), flat(wide["a"]), flat(wide["b"]), wide["A_log"], wide["a_bias"], wide["b_bias"]]
    alpha, v = _decay_and_input(case, *leaves)
    first = wide["state"] if case["initial"] else v.new_zeros(len(lens), C)
    state, h, past = first.clone(), torch.empty_like(v), torch.empty_like(v)
    for at, seqs in zip(steps, of):
        past[at] = state[seqs]
        state[seqs] = alpha[at] * state[seqs] + v[at]
        h[at] = state[seqs]
    out = {"y": h.view(B, T, C), "state": state}
    if case["op"] == "prefill":
        return out
    if case["bits"]:
        leaves[:3] = [None if t is None else _held(t) for t in leaves[:3]]
    leaves = [None if t is None else t.clone().requires_grad_() for t in leaves]
    alpha, v = _decay_and_input(case, *leaves)
    fixed, add = alpha.detach(), v.detach()
    if case["bits"]:    # the states again, from the kept ones at every CHUNK-th row
        for lo in range(1, min(CHUNK, rows)):
            at = torch.arange(lo, rows, CHUNK, device="cuda")
            at = at[~torch.isin(at, torch.tensor(begin, device="cuda"))]
            past[at] = fixed[at - 1] * past[at - 1] + add[at - 1]
    G, carry = torch.empty_like(add), wide["dstate"].clone() if case["initial"] else add.new_zeros(len(lens), C)
    dy = flat(wide["dy"])
    for at, seqs in zip(reversed(steps), reversed(of)):
        G[at] = dy[at] + carry[seqs]
        carry[seqs] = fixed[at] * G[at]
    wanted = [t for t in leaves if t is not None]
    grads = iter(torch.autograd.grad([alpha, v], wanted, [G * past, G]))
    dx, da, db, dA_log, da_bias, db_bias = (None if t is None else next(grads) for t in leaves)
    shaped = lambda t: None if t is None else t.view(B, T, C)  # noqa: E731
    return {**out, "dx": shaped(dx), "da": shaped(da), "db": shaped(db), "dA_log": dA_log, "da_bias": da_bias, "db_bias": db_bias,
            "dstate": carry if case["initial"] else None}
