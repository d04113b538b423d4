"""The diagonal recurrence (gdn_diag_prefill, gdn_diag_backward, gdn_diag_decode) and the 8-bit checkpoints
(gdn_checkpoint_pack, gdn_checkpoint_unpack) against the plain 64-bit definition, their refusals (on the CPU), and a run of
them together.

Tolerances, relative in the 2-norm.  A rounding to a 16-bit type is off by at most u = finfo(t).eps / 2 of its value, so a
rounded tensor by u of its norm.  What is computed in fp32 is off by F = 1e-5 of the norm of its terms (where these cancel,
of their magnitudes' sum): a gate's argument z rounds |z| 2^-23 into its exponential, which with the quotient, the weight and
the products is off by some 6 x 2^-23 more, 16 x 2^-23 = 2e-6 in all for |z| up to 10; sums that run over up to 2,000 tokens
round each 2^-24, at random signs, 2.7e-6; and G and h, each off by that much, meet in one product, twice (2 + 2.7) 1e-6.
"""
import ctypes
import math

import pytest
import torch

import recurrent_state_scan_gb300 as lib
from recurrent_state_scan_gb300 import gdn

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F = 1e-5
KINDS = [("softplus", "norm"), ("softplus", "complement"), ("softplus", "plain"), ("sigmoid", "norm"), ("sigmoid", "complement"),
         ("sigmoid", "plain")]


def u(dtype):
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ inputs and definitions
def draw(io, lens, C, *, gate="sigmoid", weighting="norm", b=True, packed=True, initial=True, seed=0, device="cuda", gap=0, z=1.0):
    """A call's tensors; x, a, b and dy are slices of one row with `gap` unused values behind each."""
    g = torch.Generator().manual_seed(seed)
    B, T, n = (1, sum(lens), len(lens)) if packed else (len(lens), lens[0] if lens else 0, len(lens))
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    row = rnd(B, T, 4, C + gap).clamp(-4, 4).to(DT[io]).to(device)
    m = {"lens": lens, "C": C, "gate": gate, "weighting": weighting, "packed": packed, "io": DT[io], "x": row[:, :, 0, :C],
         "a": z * row[:, :, 1, :C] if z != 1.0 else row[:, :, 1, :C], "b": row[:, :, 2, :C] if b else None, "dy": row[:, :, 3, :C],
         "A_log": (rnd(C).clamp(-2, 2) - 2).to(device), "a_bias": rnd(C).clamp(-3, 3).to(device),
         "b_bias": rnd(C).clamp(-3, 3).to(device) if b else None, "state": rnd(n, C).to(device) if initial else None,
         "dstate": rnd(n, C).to(device) if initial else None, "cu": None}
    if packed:
        m["cu"] = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device=device)
    return m


def kinds(m):
    return dict(a_bias=m["a_bias"], b_bias=m["b_bias"], gate=m["gate"], weighting=m["weighting"])


def prefill(m, keep=None, **kw):
    out = lib.gdn_diag_prefill(m["x"], m["a"], m["b"], m["A_log"], state_in=m["state"], cu_seqlens=m["cu"], keep=keep, **kinds(m), **kw)
    assert lib.gdn_last_device_status() == 0
    return out


def backward(m, kept, **kw):
    held = dict(x=m["x"], a=m["a"], b=m["b"]) if kept.keep == "states" else {}
    out = lib.gdn_diag_backward(m["dy"], kept, m["A_log"], a_bias=m["a_bias"], b_bias=m["b_bias"], state_in=m["state"],
                                cu_seqlens=m["cu"], dstate_out=m["dstate"], **held, **kw)
    assert lib.gdn_last_device_status() == 0
    return out


def wide(m):
    """The call's tensors in 64 bits on the CPU, rows flat."""
    w = {k: None if m[k] is None else m[k].double().cpu() for k in ("x", "a", "b", "dy", "A_log", "a_bias", "b_bias", "state", "dstate")}
    for k in ("x", "a", "b", "dy"):
        w[k] = None if w[k] is None else w[k].reshape(-1, m["C"])
    return w


def gates(m, w):
    z = w["a"] + (w["a_bias"] if w["a_bias"] is not None else 0)
    s = torch.sigmoid(z)
    g = -torch.exp(w["A_log"]) * (s if m["gate"] == "sigmoid" else torch.logaddexp(torch.zeros_like(z), z))
    i = torch.ones_like(g) if w["b"] is None else torch.sigmoid(w["b"] + (w["b_bias"] if w["b_bias"] is not None else 0))
    alpha = torch.exp(g)
    weight = {"norm": (-torch.expm1(2 * g)).sqrt(), "complement": -torch.expm1(g), "plain": torch.ones_like(g)}[m["weighting"]]
    slope = {"norm": -alpha ** 2 / weight.clamp_min(1e-300), "complement": -alpha, "plain": torch.zeros_like(g)}[m["weighting"]]
    return g, alpha, s, i, weight, slope


def define(m, w=None):
    """(y, final states, h before each row), token by token."""
    w = w or wide(m)
    g, alpha, _, i, weight, _ = gates(m, w)
    add = weight * i * w["x"]
    h, past, states, r = torch.empty_like(add), torch.empty_like(add), [], 0
    for n, L in enumerate(m["lens"]):
        s = w["state"][n].clone() if w["state"] is not None else torch.zeros(m["C"], dtype=torch.float64)
        for t in range(r, r + L):
            past[t] = s
            s = alpha[t] * s + add[t]
            h[t] = s
        states.append(s)
        r += L
    return h, torch.stack(states) if states else torch.zeros(0, m["C"], dtype=torch.float64), past


def stored(x):
    """What 8 bits hold of x [rows, C] (64 bits), by the definition."""
    out = x.clone()
    for lo in range(0, x.shape[1], 64):
        for r in range(x.shape[0]):
            v = x[r, lo:lo + 64]
            if not torch.isfinite(v).all():
                out[r, lo:lo + 64] = math.nan
                continue
            top = float(v.abs().max())
            e = -117
            while top >= 127.5 * 2.0 ** e and e < 121:
                e += max(1, math.frexp(top / (127.5 * 2.0 ** e))[1] - 1)
            out[r, lo:lo + 64] = (v / 2.0 ** e).round().clamp(-127, 127) * 2.0 ** e
    return out


def define_gradients(m, bits=False):
    """{name: (gradient, magnitude of its terms)}."""
    w = wide(m)
    _, _, past = define(m, w)
    if bits:
        w = dict(w, **{k: None if w[k] is None else stored(w[k]) for k in ("x", "a", "b")})
    g, alpha, s, i, weight, slope = gates(m, w)
    if bits:                        # h again from each 64th row, at the values that the codes hold
        add, first = weight * i * w["x"], {sum(m["lens"][:n]) for n in range(len(m["lens"]))}
        for t in range(1, len(past)):
            if t % 64 and t not in first:
                past[t] = alpha[t - 1] * past[t - 1] + add[t - 1]
    G, size, r = torch.empty_like(g), torch.empty_like(g), 0
    dstate = torch.zeros(len(m["lens"]), m["C"], dtype=torch.float64)
    for n, L in enumerate(m["lens"]):
        c = w["dstate"][n].clone() if w["dstate"] is not None else torch.zeros(m["C"], dtype=torch.float64)
        cs = c.abs()
        for t in range(r + L - 1, r - 1, -1):
            G[t], size[t] = w["dy"][t] + c, w["dy"][t].abs() + cs
            c, cs = alpha[t] * G[t], alpha[t] * size[t]
        dstate[n] = c
        r += L
    v = i * w["x"]
    dg, dgs = G * (alpha * past + v * slope), size * (alpha * past.abs() + (v * slope).abs())
    open_ = g * (1 - s) if m["gate"] == "sigmoid" else -torch.exp(w["A_log"]) * s
    dx, da, db = G * weight * i, dg * open_, G * weight * i * w["x"] * (1 - i)
    dxs, das = size * weight * i, dgs * open_.abs()
    dbs = dxs * (w["x"] * (1 - i)).abs()
    out = {"dx": (dx, dxs), "da": (da, das), "db": (db, dbs), "dA_log": ((dg * g).sum(0), (dgs * g.abs()).sum(0)),
           "da_bias": (da.sum(0), das.sum(0)), "db_bias": (db.sum(0), dbs.sum(0)), "dstate": (dstate, dstate.abs() + 1)}
    if w["b"] is None:
        out["db"] = out["db_bias"] = None
    if w["b_bias"] is None:
        out["db_bias"] = None
    if w["state"] is None:
        out["dstate"] = None
    return out


NAMES = ("dx", "da", "db", "dA_log", "da_bias", "db_bias", "dstate")


def near(got, want, size=None, dtype=torch.float32, what=""):
    got = got.double().cpu().reshape(want.shape)
    size = want if size is None else size
    assert torch.isfinite(got).all() or not torch.isfinite(want).all(), what
    off, may = float((got - want).norm()), u(dtype) * float(want.norm()) + F * float(size.norm())
    # (values below 2^-14 of f16 lose up to half of 2^-24 each)
    may += want.numel() ** 0.5 * 2.0 ** -25 if dtype == torch.float16 else 0.0
    assert off <= may, (what, off, may)


def check(m, got, want=None):
    y, state = got[0], got[1]
    h, states, _ = want or define(m)
    near(y, h, None, m["io"], "y")
    near(state, states, None, torch.float32, "state")


def check_gradients(m, got, bits=False):
    for name, t, want in zip(NAMES, got, define_gradients(m, bits).values()):
        assert (t is None) == (want is None), name
        if t is not None:
            near(t, *want, m["io"] if name in ("dx", "da", "db") else torch.float32, name)


# ------------------------------------------------------------------ the definition itself, on the CPU
@pytest.mark.parametrize("gate,weighting", KINDS)
@pytest.mark.parametrize("b", [True, False])
def test_the_gradient_formulas_against_differences(gate, weighting, b):
    """Central differences over 2e-6 in 64 bits: 2^-53 / 1e-6 of the loss's terms, and the third derivative's 1e-12."""
    m = draw("f32", [5, 0, 1, 9], 3, gate=gate, weighting=weighting, b=b, device="cpu", seed=3)
    w = wide(m)

    def loss(w):
        h, states, _ = define(m, w)
        return float((h * w["dy"]).sum() + (states * w["dstate"]).sum())

    want = define_gradients(m)
    for name, key in (("dx", "x"), ("da", "a"), ("db", "b"), ("dA_log", "A_log"), ("da_bias", "a_bias"), ("db_bias", "b_bias"), ("dstate", "state")):
        if want[name] is None:
            continue
        got = torch.empty_like(w[key]).view(-1)
        for k in range(got.numel()):
            sides = []
            for d in (1e-6, -1e-6):
                moved = dict(w, **{key: w[key].clone()})
                moved[key].view(-1)[k] += d
                sides.append(loss(moved))
            got[k] = (sides[0] - sides[1]) / 2e-6
        assert (got.view_as(w[key]) - want[name][0]).abs().max() <= 1e-7, name


# ------------------------------------------------------------------ refusals, on the CPU
GOOD = dict(io_dtype=gdn.GDN_BF16, batch=2, seqlen=8, num_seqs=2, channels=64, gate=1, weighting=2, input_gate=1, keep=1)
WHERE = {name: 0x100000 * (k + 1) for k, name in enumerate(
    ("x", "a", "b", "A_log", "a_bias", "b_bias", "state_in", "y", "state_out", "kept", "dy", "dstate_out", "dx", "da", "db", "dA_log", "da_bias",
     "db_bias", "dstate_in", "workspace", "state"))}
CALLS = {"prefill": ("x", "a", "b", "A_log", "a_bias", "b_bias", "state_in", "cu", "y", "state_out", "kept", "kept_bytes", "workspace", "workspace_bytes", "stream"),
         "backward": ("x", "a", "b", "A_log", "a_bias", "b_bias", "state_in", "cu", "kept", "kept_bytes", "dy", "dstate_out", "dx", "da", "db",
                      "dA_log", "da_bias", "db_bias", "dstate_in", "workspace", "workspace_bytes", "stream"),
         "decode": ("x", "a", "b", "A_log", "a_bias", "b_bias", "state", "pool_size", "slots", "y", "stream")}


def call(which, shape=None, **where):
    """The C call at addresses that no one owns: only refusals come back from it."""
    fields = {**GOOD, **(dict(seqlen=1) if which == "decode" else {}), **(shape or {})}
    at = {**WHERE, "kept_bytes": 1 << 30, "workspace_bytes": 1 << 20, "pool_size": 4, **where}
    return getattr(gdn.load(), "gdn_diag_" + which)(ctypes.byref(gdn.GdnDiagShape(**fields)), *(at.get(k) for k in CALLS[which]))


@pytest.mark.parametrize("which", ["prefill", "backward", "decode"])
@pytest.mark.parametrize("shape,status", [
    (dict(io_dtype=3), 1), (dict(seqlen=-1), 1), (dict(batch=-2, num_seqs=-2), 1), (dict(num_seqs=3), 1), (dict(channels=0), 1),
    (dict(channels=-5), 1), (dict(channels=65535 * 64 + 1), 2), (dict(gate=2), 1), (dict(gate=-1), 1), (dict(weighting=3), 1),
    (dict(input_gate=2), 1), (dict(keep=3), 1), (dict(x_stride=63), 1), (dict(b_stride=1), 1), (dict(y_stride=-64), 1), (dict(dx_stride=2), 1),
    (dict(seqlen=1 << 30), 2), (dict(seqlen=1 << 62), 2), (dict(x_stride=1 << 62), 2), (dict(seqlen=1 << 29, channels=1 << 20), 2)])
def test_refused_shapes(which, shape, status):
    assert call(which, shape) == status
    assert gdn.load().gdn_last_error_message().decode()


@pytest.mark.parametrize("which,where", [
    *[("prefill", {k: None}) for k in ("x", "a", "b", "A_log", "y", "state_out", "kept")],
    *[("backward", {k: None}) for k in ("x", "a", "b", "A_log", "kept", "dy", "dx", "da", "db")],
    *[("decode", {k: None}) for k in ("x", "a", "b", "A_log", "y", "state")],
    *[("prefill", {k: WHERE[k] + 1}) for k in ("x", "y", "A_log", "a_bias", "state_in", "state_out", "kept")],
    *[("backward", {k: WHERE[k] + 1}) for k in ("dy", "db", "dA_log", "dstate_in", "dstate_out", "kept")],
    *[("decode", {k: WHERE[k] + 1}) for k in ("x", "y", "state")], ("decode", dict(slots=0x3001)), ("prefill", dict(cu=0x3001)),
    ("prefill", dict(kept=WHERE["kept"] + 8)), ("prefill", dict(kept_bytes=255)), ("backward", dict(kept_bytes=255)),
    ("prefill", dict(y=WHERE["x"])), ("prefill", dict(y=WHERE["a"] + 64)), ("prefill", dict(state_out=WHERE["state_in"] + 64)),
    ("prefill", dict(kept=WHERE["y"])), ("prefill", dict(state_out=WHERE["y"])), ("prefill", dict(cu=0x3000)),
    ("backward", dict(dx=WHERE["x"])), ("backward", dict(da=WHERE["dx"] + 128)), ("backward", dict(db=WHERE["dy"])),
    ("backward", dict(dstate_in=WHERE["state_in"])), ("backward", dict(dstate_in=WHERE["dstate_out"])), ("backward", dict(dA_log=WHERE["A_log"])),
    ("backward", dict(dx=WHERE["kept"])), ("decode", dict(y=WHERE["x"])), ("decode", dict(y=WHERE["state"])), ("decode", dict(state=WHERE["b"])),
    *[("prefill", {o: WHERE[k] + 16 * (o != "y")}) for o in ("y", "state_out", "kept") for k in ("A_log", "a_bias", "b_bias")],
    *[("decode", {o: WHERE[k]}) for o in ("y", "state") for k in ("A_log", "a_bias", "b_bias")], ("decode", dict(slots=WHERE["y"])),
    ("decode", dict(slots=WHERE["state"] + 512)), ("decode", dict(slots=0x3000, pool_size=0)), ("decode", dict(slots=0x3000, pool_size=-4))])
def test_refused_pointers(which, where):
    assert call(which, None, **where) == gdn.GDN_ERR_INVALID_ARG
    assert gdn.load().gdn_last_error_message().decode()


@pytest.mark.parametrize("which", ["prefill", "backward"])
@pytest.mark.parametrize("num_seqs", [2 ** 30, 2 ** 31 - 200, 2 ** 31 - 1])
def test_refused_numbers_of_sequences(which, num_seqs):
    """More than the search through cu_seqlens can count to."""
    assert call(which, dict(batch=1, num_seqs=num_seqs, seqlen=16), cu=1 << 40) == gdn.GDN_ERR_UNSUPPORTED
    assert "sequences" in gdn.load().gdn_last_error_message().decode()


@pytest.mark.parametrize("B,n,C", [((1 << 32) + 1, (1 << 32) + 1, 64), (1, (1 << 32) + 3, 64), (1, 1, (1 << 32) + 64), (1 << 31, 1 << 31, 1)])
def test_the_binding_refuses_sizes_beyond_32_bits(B, n, C):
    """Their low 32 bits would be another call's."""
    with pytest.raises(gdn.GdnError) as refused:
        gdn._diag_shape(torch.bfloat16, B, 1, n, C, "sigmoid", "norm", True, None, C, C, C, C)
    assert refused.value.status == gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("which,out", [("prefill", "y"), ("prefill", "state_out"), ("backward", "dx"), ("backward", "dstate_in")])
def test_refused_offsets(which, out):
    packed = dict(batch=1, num_seqs=3, seqlen=16)
    assert call(which, packed, cu=WHERE[out] + 16) == gdn.GDN_ERR_INVALID_ARG
    assert "cu_seqlens" in gdn.load().gdn_last_error_message().decode()


def test_refused_workspaces():
    assert call("backward", dict(keep=0)) == gdn.GDN_ERR_INVALID_ARG
    long = dict(batch=4, num_seqs=4, seqlen=20)
    for which, size in (("prefill", gdn.gdn_diag_prefill_workspace_bytes), ("backward", gdn.gdn_diag_backward_workspace_bytes)):
        assert size(gdn.GdnDiagShape(**GOOD)) == 0 < (need := size(gdn.GdnDiagShape(**dict(GOOD, **long))))
        for bad in (dict(workspace_bytes=need - 1), dict(workspace=None), dict(workspace=WHERE["workspace"] + 4), dict(workspace=WHERE["a"])):
            assert call(which, long, **bad) == gdn.GDN_ERR_INVALID_ARG, (which, bad)


def test_slices_of_one_row_lie_beside_one_another():
    """Rows of 3 x 64 channels: dx, da and db in turn are taken; one channel over another's is refused.  (The call that is taken ends
    at the device, which the CPU does not have.)"""
    apart = dict(dx_stride=192, da_stride=192, db_stride=192)
    at = WHERE["dx"]
    for first, second, third, taken in ((0, 64, 128, True), (128, 0, 64, True), (0, 63, 128, False), (0, 64, 129, False), (2, 64, 128, False)):
        if taken and torch.cuda.is_available():
            continue
        status = call("backward", apart, dx=at + 2 * first, da=at + 2 * second, db=at + 2 * third)
        message = gdn.load().gdn_last_error_message().decode()
        assert (status != gdn.GDN_OK and "overlaps" in message) != taken, (first, second, third, message)


@pytest.mark.parametrize("which", ["pack", "unpack"])
def test_refused_codes(which):
    fn = getattr(gdn.load(), "gdn_checkpoint_" + which)

    def go(io=1, rows=4, channels=70, x=0x100000, stride=0, codes=0x200000, steps=0x300000):
        return fn(io, rows, channels, x, stride, codes, steps, None) if which == "pack" else fn(io, rows, channels, codes, steps, x, stride, None)

    for bad in (dict(io=5), dict(rows=-1), dict(channels=-1), dict(x=None), dict(x=0x100001), dict(stride=69), dict(codes=None), dict(steps=None),
                dict(codes=0x100010), dict(steps=0x100000)):
        assert go(**bad) == gdn.GDN_ERR_INVALID_ARG, bad
    assert go(stride=1 << 62) == gdn.GDN_ERR_UNSUPPORTED
    assert go(rows=0, x=None, codes=None, steps=None) == gdn.GDN_OK


def test_the_binding_refuses():
    x = torch.zeros(1, 4, 8)
    for bad in (lambda: lib.gdn_diag_prefill(x, x, x, x[0, 0]), lambda: lib.gdn_diag_decode(x, x, x, x[0, 0], x[0]),
                lambda: lib.gdn_checkpoint_pack(x), lambda: lib.gdn_checkpoint_unpack(x.char(), x.byte()),
                lambda: lib.gdn_diag_backward(x, (x,), x[0, 0])):
        with pytest.raises(gdn.GdnError):
            bad()


@pytest.mark.gpu
def test_the_binding_refuses_on_the_device():
    m = draw("bf16", [5, 3], 64, seed=1)
    _, _, kept = prefill(m, "states")
    args = (m["x"], m["a"], m["b"], m["A_log"])
    held = dict(x=m["x"], a=m["a"], b=m["b"], cu_seqlens=m["cu"])
    for bad in (lambda: lib.gdn_diag_prefill(*args, gate="tanh"), lambda: lib.gdn_diag_prefill(*args, weighting="sum"),
                lambda: lib.gdn_diag_prefill(*args, keep="4bit"), lambda: lib.gdn_diag_prefill(m["x"], m["a"], None, m["A_log"], b_bias=m["b_bias"]),
                lambda: lib.gdn_diag_prefill(m["x"], m["a"].float(), m["b"], m["A_log"]), lambda: lib.gdn_diag_prefill(*args[:3], m["A_log"][:9]),
                lambda: lib.gdn_diag_prefill(m["x"][:, :1].expand(1, 8, 64), *args[1:]), lambda: lib.gdn_diag_prefill(*args[:3], None),
                lambda: lib.gdn_diag_prefill(*args, cu_seqlens=m["cu"].long()), lambda: lib.gdn_diag_prefill(*args, cu_seqlens=m["cu"], state_in=m["state"][:1]),
                lambda: lib.gdn_diag_prefill(*args, y=m["x"]), lambda: lib.gdn_diag_prefill(*args, keep="8bit", kept=kept.data[:16]),
                lambda: lib.gdn_diag_backward(m["dy"], kept, m["A_log"], x=m["x"], a=m["a"], cu_seqlens=m["cu"]),
                lambda: lib.gdn_diag_backward(m["dy"], kept, m["A_log"], **dict(held, cu_seqlens=None)),
                lambda: lib.gdn_diag_backward(m["dy"][:, :7], kept, m["A_log"], **held),
                lambda: lib.gdn_diag_backward(m["dy"].float(), kept, m["A_log"], **held),
                lambda: lib.gdn_diag_backward(m["dy"], kept, m["A_log"], **held, dx=m["x"]),
                lambda: lib.gdn_diag_backward(m["dy"], kept._replace(data=kept.data[:16]), m["A_log"], **held),
                lambda: lib.gdn_diag_decode(*(t[:, :2] for t in args[:3]), m["A_log"], m["state"][:1]),
                lambda: lib.gdn_diag_decode(*(t[:, :1] for t in args[:3]), m["A_log"], m["state"]),
                lambda: lib.gdn_checkpoint_pack(m["x"].int())):
        with pytest.raises(gdn.GdnError):
            bad()
    assert lib.gdn_last_device_status() == 0


# ------------------------------------------------------------------ prompts
@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gate,weighting", KINDS)
@pytest.mark.parametrize("b", [True, False])
def test_prompts_match_the_definition(io, gate, weighting, b):
    m = draw(io, [63, 1, 0, 200, 64, 2, 129], 130, gate=gate, weighting=weighting, b=b, seed=len(gate) + b)
    check(m, prefill(m))


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,packed", [([1], False), ([3, 3], False), ([65] * 3, False), ([700], True), ([0, 0, 5], True), ([0], True),
                                         ([], True), ([0, 0], False), ([1] * 300, True), ([129, 0, 0, 0, 511, 1, 1, 64, 64], True),
                                         ([8] * 70, False), ([0] * 70 + [3, 0, 0] * 40, True)])
@pytest.mark.parametrize("initial", [False, True])
def test_lengths(io, lens, packed, initial):
    """Forward and backward, sequences shorter and longer than a warp's rows and a tile, and empty ones."""
    m = draw(io, lens, 70, packed=packed, initial=initial, seed=len(lens))
    y, state, kept = prefill(m, "states")
    check(m, (y, state))
    check_gradients(m, backward(m, kept))


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("C", [1, 2, 63, 64, 65, 127, 192, 257])
@pytest.mark.parametrize("gap", [0, 1, 2, 8])
def test_widths_and_strides(io, C, gap):
    m = draw(io, [90, 40], C, gap=gap, seed=C)
    wide_ = lambda: torch.full((1, 130, 4, C + gap), 3.0, dtype=DT[io], device="cuda")  # noqa: E731
    ys, ds = wide_(), wide_()
    y, state, kept = prefill(m, "states", y=ys[:, :, 1, :C])
    check(m, (y, state))
    got = backward(m, kept, dx=ds[:, :, 0, :C], da=ds[:, :, 2, :C], db=ds[:, :, 3, :C])
    check_gradients(m, got)
    ys[:, :, 1, :C], ds[:, :, 0, :C], ds[:, :, 2:, :C] = 3, 3, 3
    assert (ys == 3).all() and (ds == 3).all()          # (nothing beside the rows that were asked for)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,packed,C", [([2000], False, 64), ([1999, 2001], True, 40), ([600] * 9, False, 64), ([1300, 5, 2500, 0, 700], True, 128)])
@pytest.mark.parametrize("keep", ["states", "8bit"])
def test_long_rows(lens, packed, C, keep):
    """Many tiles, each waiting for what the one before it hands on."""
    m = draw("f32", lens, C, packed=packed, seed=11)
    shape = gdn.GdnDiagShape(0, 1 if packed else len(lens), sum(lens) if packed else lens[0], len(lens), C, 1, 2, 1, 1)
    assert gdn.gdn_diag_backward_workspace_bytes(shape) > gdn.gdn_diag_prefill_workspace_bytes(shape) > 0
    y, state, kept = prefill(m, keep)
    check(m, (y, state))
    check_gradients(m, backward(m, kept), keep == "8bit")


@pytest.mark.gpu
def test_optional_parameters():
    m = draw("f32", [50, 3], 30, seed=4)
    m["a_bias"] = m["b_bias"] = None
    y, state, kept = prefill(m, "states")
    check(m, (y, state))
    got = backward(m, kept)
    assert got[4] is None and got[5] is None
    for name, t in zip(NAMES, got):
        if t is not None:
            near(t, *define_gradients(m)[name], m["io"], name)


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["softplus", "sigmoid"])
@pytest.mark.parametrize("weighting", ["norm", "complement", "plain"])
def test_gates_far_out(gate, weighting):
    """Shut gates keep the state bit for bit, wide open ones and rates beyond fp32's range clear it; no NaN in results or
    gradients of finite inputs, and none from infinite gates."""
    m = draw("f32", [150], 64, gate=gate, weighting=weighting, seed=5)
    m["a"], m["A_log"] = m["a"].clone(), m["A_log"].clone()
    m["a"][:, 10:100] = -math.inf
    m["a"][:, 120] = 3e38
    m["A_log"][:4] = torch.tensor([95.0, 88.5, 30.0, -60.0])
    m["b"] = m["b"].clone()
    m["b"][:, 40], m["b"][:, 41] = 1e30, -1e30
    y, state, kept = prefill(m, "states")
    if weighting != "plain":
        assert torch.equal(y[:, 99], y[:, 16])
    assert all(torch.isfinite(t).all() for t in (y, state) + backward(m, kept))
    m["a"] = m["a"].clamp(-3e38, 3e38)
    rows = define(m)[0]
    near(y[0, :10], rows[:10], what="before")
    near(y[0, 100:], rows[100:], what="behind")


@pytest.mark.gpu
@pytest.mark.parametrize("gate,weighting", KINDS)
@pytest.mark.parametrize("keep", ["states", "8bit"])
@pytest.mark.parametrize("lens", [[7], [20, 50], [64, 65]])
def test_infinite_biases(gate, weighting, keep, lens):
    """A gate that its bias holds open or shut, in rows that do not fill their tiles: the gradients are those of biases so far
    out that in 64 bits nothing is left of the gate's other side (e^-800 is 0)."""
    m = draw("f32", lens, 64, gate=gate, weighting=weighting, seed=25)
    m["a_bias"], m["b_bias"] = m["a_bias"].clone(), m["b_bias"].clone()
    m["A_log"][3] = 0.0
    m["a_bias"][3], m["a_bias"][4], m["b_bias"][5], m["b_bias"][6] = math.inf, -math.inf, math.inf, -math.inf
    y, state, kept = prefill(m, keep)
    got = backward(m, kept)
    assert all(torch.isfinite(t).all() for t in (y, state, *got))
    far = dict(m, a_bias=m["a_bias"].clamp(-800, 800), b_bias=m["b_bias"].clamp(-800, 800))
    check(far, (y, state))
    check_gradients(far, got, keep == "8bit")


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["softplus", "sigmoid"])
def test_fast_decays_keep_their_digits(gate):
    """Tokens that write nothing: h = h0 e^(sum g), every value on its own.  A token's g rounds (|z| + 8) 2^-23 of itself,
    and its decay 3 units of 2^-23."""
    for T in (1, 8, 70):
        m = draw("f32", [T], 64, gate=gate, weighting="plain", seed=6)
        m["x"] = torch.zeros_like(m["x"])
        m["A_log"] = torch.log(torch.linspace(0.01, 60.0 / T, 64)).cuda()
        y, state, _ = prefill(m)
        w = wide(m)
        G = gates(m, w)[0].cumsum(0)
        want = w["state"] * torch.exp(G)
        off = (8 + 8 + 1) * 2.0 ** -23 * G.abs() + 3 * torch.arange(1, T + 1)[:, None] * 2.0 ** -23
        assert ((y[0].double().cpu() - want).abs() <= off * want.abs() + 2.0 ** -126).all()
        assert torch.equal(state[0], y[0, -1])


@pytest.mark.gpu
@pytest.mark.parametrize("keep", ["states", "8bit"])
@pytest.mark.parametrize("rate", [1e-3, 3e-5, 2e-7])
def test_slow_decays_do_not_drift(keep, rate):
    """65,536 equal tokens that forget next to nothing: h = h0 e^(t g), and G the same way back.  Each of the 1,024 tiles rounds h
    once, by half a unit in the last place (2^-24 of it) at most; equal tokens take nearly equal steps, whose roundings can all
    fall the same way, so they add up as they are.  The exponents (6 x 2^-23 of g, alike in all) add 65,536 g 7e-7, the rows inside
    a tile 16 x 2^-24.  (A product of 65,536 decays in fp32 could be off by 65,536 x 2^-25 = 2e-3.)"""
    T = 65536
    m = draw("f32", [T], 64, weighting="plain", initial=True, seed=7)
    m["x"], m["dy"] = torch.zeros_like(m["x"]), torch.zeros_like(m["dy"])
    m["a"] = (torch.linspace(-1, 1, 64)).expand(1, T, 64).contiguous().cuda()
    m["a_bias"] = torch.zeros(64, device="cuda")
    m["A_log"] = torch.full((64,), math.log(rate), device="cuda")
    if keep == "8bit":
        m["a"] = m["a"].bfloat16().float() * 0 + 0.5       # (a value that the codes hold)
    y, state, kept = prefill(m, keep)
    w = wide(dict(m, a=m["a"][:, :1], x=m["x"][:, :1], b=m["b"][:, :1], dy=m["dy"][:, :1]))
    g = gates(m, w)[0][0]
    far = 1024 * 2.0 ** -24 + 16 * 2.0 ** -24 + T * float(g.abs().max()) * 7e-7
    want = w["state"][0] * torch.exp(T * g)
    assert ((state[0].double().cpu() - want).abs() <= far * want.abs() + 1e-30).all()
    back = backward(m, kept)[6][0].double().cpu()
    want = w["dstate"][0] * torch.exp(T * g)
    assert ((back - want).abs() <= far * want.abs() + 1e-30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("keep", ["states", "8bit"])
def test_a_sequence_does_not_see_its_neighbours(io, keep):
    """Infinities and NaN in the other sequences leave a packed sequence's results and gradients bit for bit."""
    m = draw(io, [70, 33, 90, 6, 700], 64, seed=6)
    y, state, kept = prefill(m, keep)
    before = backward(m, kept)
    for name in ("x", "a", "b", "dy"):
        m[name] = m[name].clone()
        m[name][:, :70], m[name][:, 103:193], m[name][:, 199:] = math.nan, math.inf, math.nan
    for name in ("state", "dstate"):
        m[name] = m[name].clone()
        m[name][0], m[name][2], m[name][4] = math.nan, -math.inf, math.nan
    y2, state2, kept2 = prefill(m, keep)
    after = backward(m, kept2)
    for rows, n in ((slice(70, 103), 1), (slice(193, 199), 3)):
        assert torch.equal(y[:, rows], y2[:, rows]) and torch.equal(state[n], state2[n])
        assert all(torch.equal(s[:, rows], t[:, rows]) for s, t in zip(before[:3], after[:3])) and torch.equal(before[6][n], after[6][n])
    # and one bad value its own channel only
    m = draw(io, [200], 64, seed=8)
    good = prefill(m, "states")
    m["x"] = m["x"].clone()
    m["x"][0, 60, 5] = math.nan
    bad = prefill(m, "states")
    keep_ = torch.arange(64) != 5
    assert torch.equal(good[0][..., keep_], bad[0][..., keep_]) and bad[0][0, 60:, 5].isnan().all() and torch.equal(good[0][:, :60], bad[0][:, :60])


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rate", [-4.0, 0.5, 2.0])
def test_an_infinite_state_stays_infinite(io, rate):
    """Behind warps' rows and tiles too, where decays' products have long become 0."""
    m = draw(io, [400, 9, 200], 130, gate="softplus", weighting="complement", seed=37)
    m["A_log"] = torch.full((130,), rate, device="cuda")
    m["x"], m["state"] = m["x"].clone(), m["state"].clone()
    m["state"][0, 3], m["state"][0, 70], m["state"][2, 5] = math.inf, -math.inf, math.inf
    m["x"][0, 101, 9], m["x"][0, 63, 129], m["x"][0, 350, 3] = -math.inf, math.inf, -math.inf
    y, state, _ = prefill(m)
    h, states, _ = define(m)
    assert h.isinf().sum() > 1000
    for got, want in ((y[0], h), (state, states)):
        got = got.double().cpu()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
        assert torch.equal(got[want.isinf()], want[want.isinf()])


@pytest.mark.gpu
def test_an_infinite_state_ends_at_a_decay_of_0():
    """e^-100 of it is 0 in fp32: NaN from there on, in one call, in two and token by token."""
    m = draw("f32", [200], 64, gate="softplus", weighting="plain", packed=False, seed=38)
    m["A_log"], m["state"], m["a"] = torch.zeros(64, device="cuda"), m["state"].clone(), m["a"].clone()
    m["state"][0, 7], m["a"][0, 90] = math.inf, 110.0
    y, state, _ = prefill(m)
    assert y[0, :90, 7].isinf().all() and y[0, 90:, 7].isnan().all() and state[0, 7].isnan()
    cut = lambda lo, hi: dict(m, **{k: m[k][:, lo:hi].contiguous() for k in ("x", "a", "b")})  # noqa: E731
    for at in (50, 90, 91, 130):
        y0, s, _ = prefill(cut(0, at))
        y1, s, _ = prefill(dict(cut(at, 200), state=s))
        assert torch.equal(torch.cat([y0, y1], 1).isnan(), y.isnan()) and s[0, 7].isnan()
    s, rows = m["state"].clone(), []
    for t in range(200):
        rows.append(lib.gdn_diag_decode(*(m[k][:, t:t + 1] for k in ("x", "a", "b")), m["A_log"], s, **kinds(m)))
    assert torch.equal(torch.cat(rows, 1).isnan(), y.isnan())


@pytest.mark.gpu
def test_chained_calls_and_states_in_place():
    m = draw("bf16", [300], 96, packed=False, seed=7)
    y, state, _ = prefill(m)
    parts, s = [], m["state"].clone()
    for lo, hi in ((0, 101), (101, 165), (165, 300)):
        part = dict(m, state=s, **{k: m[k][:, lo:hi] for k in ("x", "a", "b")})
        parts.append(prefill(part, state_out=s)[0])
    near(torch.cat(parts, 1), y.double().cpu(), None, torch.bfloat16)
    near(s, state.double().cpu())
    m = draw("f32", [700, 0, 3, 64, 0], 96, seed=8)
    y, state, _ = prefill(m)
    s = m["state"].clone()
    again = prefill(dict(m, state=s), state_out=s)
    assert torch.equal(again[0], y) and torch.equal(s, state)


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 100, 90, 200], [1, 100, 150, 200], [0, 50, 100, 199], [0, 300, 100, 200], [0, -5, 100, 200], [0, 50, 60, 2 ** 31 - 1]])
def test_bad_offsets_are_reported_and_nothing_is_written(cu):
    m = draw("bf16", [100, 60, 40], 64, seed=8)
    y, state, kept = prefill(m, "states")
    good = backward(m, kept)
    m["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    outs = [torch.full_like(t, 7.0) for t in (y, state)]
    lib.gdn_diag_prefill(m["x"], m["a"], m["b"], m["A_log"], state_in=m["state"], cu_seqlens=m["cu"], y=outs[0], state_out=outs[1], **kinds(m))
    assert lib.gdn_last_device_status() == gdn.GDN_ERR_DEVICE_CHECK and all((t == 7).all() for t in outs)
    grads = [torch.full_like(t, 7.0) for t in good[:3]]
    lib.gdn_diag_backward(m["dy"], kept, m["A_log"], x=m["x"], a=m["a"], b=m["b"], state_in=m["state"], cu_seqlens=m["cu"],
                          dx=grads[0], da=grads[1], db=grads[2])
    assert lib.gdn_last_device_status() == gdn.GDN_ERR_DEVICE_CHECK and all((t == 7).all() for t in grads)


# ------------------------------------------------------------------ gradients
@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gate,weighting", KINDS)
@pytest.mark.parametrize("b", [True, False])
@pytest.mark.parametrize("keep", ["states", "8bit"])
def test_gradients_match_the_definition(io, gate, weighting, b, keep):
    m = draw(io, [63, 1, 0, 200, 64, 2, 129], 130, gate=gate, weighting=weighting, b=b, seed=len(weighting) + b)
    _, _, kept = prefill(m, keep)
    check_gradients(m, backward(m, kept), keep == "8bit")


def slow_rates(C, seed):
    """A_log of sigmoid gates whose decays are 0.9 to 0.999 where they are open."""
    return torch.log(-torch.log(0.9 + 0.099 * torch.rand(C, generator=torch.Generator().manual_seed(seed)))).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("weighting", ["norm", "complement", "plain"])
@pytest.mark.parametrize("keep", ["states", "8bit"])
@pytest.mark.parametrize("C,lens", [(64, [300]), (128, [70, 0, 261, 33]), (130, [200])])
def test_slow_sigmoid_gates(io, weighting, keep, C, lens):
    """No rate above 1/4 in a slice of 64 channels: decays without an exponential, forward and backward."""
    m = draw(io, lens, C, weighting=weighting, seed=C)
    m["A_log"] = slow_rates(C, C + 1)
    y, state, kept = prefill(m, keep)
    check(m, (y, state))
    check_gradients(m, backward(m, kept), keep == "8bit")


def on_the_codes(m):
    """The call with x, a and b rounded to what 8 bits hold of them, so that codes lose nothing."""
    return dict(m, **{k: stored(m[k].double().cpu().view(-1, m["C"])).to(m["io"]).view(m[k].shape).cuda() for k in ("x", "a", "b")})


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gate,weighting", KINDS)
@pytest.mark.parametrize("keep", ["states", "8bit"])
def test_masked_gates(io, gate, weighting, keep):
    """-infinity in a and b, in whole rows, parts of a block of 64 channels and single values: the definition's results and gradients
    at arguments so low that in 64 bits nothing is left of the gate (e^-800 is 0)."""
    m = on_the_codes(draw(io, [150, 3, 90], 130, gate=gate, weighting=weighting, seed=31))
    g = torch.Generator().manual_seed(32)
    shut, closed = ((torch.rand(1, 243, 130, generator=g) < 0.1).cuda() for _ in range(2))
    shut[:, 20:60], shut[:, 64, 64:], shut[:, 70:80, 7], closed[:, 30:70] = True, True, True, True
    m["a"], m["b"] = m["a"].masked_fill(shut, -math.inf), m["b"].masked_fill(closed, -math.inf)
    y, state, kept = prefill(m, keep)
    got = backward(m, kept)
    assert all(torch.isfinite(t).all() for t in (y, state, *got))
    far = dict(m, a=m["a"].float().clamp_min(-800), b=m["b"].float().clamp_min(-800))
    check(far, (y, state))
    check_gradients(far, got)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
def test_a_masked_gate_leaves_its_block(io):
    """One channel's mask, and codes that are not exact: the others' gradients are the same bits.  (The masked entries are 0 before, so
    they are no block's largest.)  Another infinity, or a NaN, makes its block NaN."""
    m = draw(io, [90], 128, seed=33)
    m["a"], m["b"] = m["a"].clone(), m["b"].clone()
    m["a"][:, 10:30, 5], m["b"][:, 20, 100] = 0, 0
    before = backward(m, prefill(m, "8bit")[2])
    m["a"][:, 10:30, 5], m["b"][:, 20, 100] = -math.inf, -math.inf
    after = backward(m, prefill(m, "8bit")[2])
    others = [c for c in range(128) if c not in (5, 100)]
    assert all(torch.equal(s[..., others], t[..., others]) and torch.isfinite(t).all() for s, t in zip(before, after))
    for bad in (math.inf, math.nan):
        m["a"][:, 40, 70] = bad
        assert backward(m, prefill(m, "8bit")[2])[1][0, 40, 64:].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("gate,weighting", KINDS)
@pytest.mark.parametrize("keep", ["states", "8bit"])
@pytest.mark.parametrize("slow", [False, True])
def test_open_gates_keep_their_digits(gate, weighting, keep, slow):
    """Gates open by z of 5 to 19, every gradient on its own.  1 - s = e s has e^-z off by the argument's roundings, 3 x 2^-24 log2 e
    (16 + 3) ln 2 = 3.4e-6, and by 4 x 2^-23 of the exponential, the quotient and the product: inside F.  The other factors are off by F of
    their terms: x and the states are positive, so that h has no cancellation.  (Multiples of 1/4 that the codes hold.)"""
    T, C = 48, 64
    m = draw("f32", [T], C, gate=gate, weighting=weighting, seed=33)
    g = torch.Generator().manual_seed(34)
    quarters = lambda lo, hi: (torch.randint(4 * lo, 4 * hi + 1, (1, T, C), generator=g) / 4).cuda()  # noqa: E731
    m.update(a=quarters(8, 16), b=quarters(8, 16), x=quarters(1, 4), state=m["state"].abs())
    if slow:
        m["A_log"] = slow_rates(C, 35)
    _, _, kept = prefill(m, keep)
    want = define_gradients(m)
    for name, t in zip(NAMES, backward(m, kept)):
        off = (t.double().cpu().view(want[name][0].shape) - want[name][0]).abs()
        assert (off <= 2 * F * want[name][1]).all(), (name, float((off / want[name][1]).max()))


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("gate", ["softplus", "sigmoid"])
@pytest.mark.parametrize("weighting", ["norm", "complement"])
@pytest.mark.parametrize("keep", ["states", "8bit"])
@pytest.mark.parametrize("slow", [False, True])
def test_large_values_behind_a_mask(io, gate, weighting, keep, slow):
    """A shut gate's token has the weight 0: what finite x it brings reaches nothing."""
    m = draw(io, [150], 64, gate=gate, weighting=weighting, seed=35)
    if slow:
        m["A_log"] = slow_rates(64, 36)
    m["a"], m["x"] = m["a"].clone(), m["x"].clone()
    m["a"][:, 40:75] = -math.inf
    outs = []
    for value in (0.0, 1e30, -torch.finfo(m["io"]).max):
        m["x"][:, 40:75] = value
        y, state, kept = prefill(m, keep)
        outs.append((y, state, *backward(m, kept)))
    for out in outs[1:]:
        assert all(torch.equal(s, t) for s, t in zip(outs[0], out))


@pytest.mark.gpu
@pytest.mark.parametrize("gate,weighting", KINDS)
@pytest.mark.parametrize("keep", ["states", "8bit"])
def test_rates_below_the_normal_range(gate, weighting, keep):
    """e^A_log down to 0, some gates shut: decays of 1 in fp32, and no gradient is NaN or infinite."""
    m = on_the_codes(draw("f32", [100], 64, gate=gate, weighting=weighting, seed=36))
    m["A_log"] = m["A_log"].clone()
    m["A_log"][:8] = torch.tensor([-87.0, -87.5, -88.5, -90.0, -95.0, -103.0, -110.0, -math.inf])
    m["a"] = m["a"].clone()
    m["a"][:, 10:20] = -math.inf
    y, state, kept = prefill(m, keep)
    got = backward(m, kept)
    assert all(torch.isfinite(t).all() for t in (y, state, *got))
    far = dict(m, a=m["a"].clamp_min(-800))
    check(far, (y, state))
    check_gradients(far, got)
    states = m["state"].clone()
    lib.gdn_diag_decode(*(m[k][:, :1] for k in ("x", "a", "b")), m["A_log"], states, **kinds(m))
    assert torch.isfinite(states).all() and (weighting == "plain" or torch.equal(states[:, 1:8], m["state"][:, 1:8]))


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens", [[90], [64, 7]])
def test_the_kept_codes_of_masked_gates(io, lens):
    """-128 where -infinity was, beside the codes and steps of the row with 0 in its place: up to the type's largest values, in rows that
    are masked altogether, and in the rows of a tile's end."""
    C, rows = 130, sum(lens)
    m = draw(io, lens, C, seed=34)
    shut = (torch.rand(1, rows, C, generator=torch.Generator().manual_seed(35)) < 0.2).cuda()
    shut[:, 20:40], shut[:, 3] = True, False
    for name in ("a", "b"):
        m[name] = m[name].clone()
        m[name][:, 5], m[name][:, 6, ::2] = torch.finfo(m["io"]).max, -torch.finfo(m["io"]).max
        m[name] = m[name].masked_fill(shut, -math.inf)
    kept = prefill(m, "8bit")[2]
    slices, tiles = -(-C // 64), -(-rows // 64)
    data = kept.data[tiles * slices * 256:]
    codes = data[:3 * slices * tiles * 4096].view(torch.int8).view(3, slices, tiles * 64, 64)
    steps = data[3 * slices * tiles * 4096:].view(3, slices, tiles * 64)
    for k, name in enumerate(("a", "b")):
        want, want_steps = lib.gdn_checkpoint_pack(m[name].masked_fill(shut, 0))
        assert torch.equal(codes[k + 1, :, :rows].transpose(0, 1).reshape(rows, -1)[:, :C], want[0].masked_fill(shut[0], -128))
        assert torch.equal(steps[k + 1, :, :rows].T, want_steps[0])


@pytest.mark.gpu
@pytest.mark.parametrize("gate,weighting", KINDS)
def test_masked_tokens(gate, weighting):
    """A token whose gates are shut: with COMPLEMENT and NORM, or with both shut, the states stay bit for bit."""
    m = draw("bf16", [1] * 5, 130, gate=gate, weighting=weighting, packed=False, seed=36)
    m["a"], m["b"] = torch.full_like(m["a"], -math.inf), m["b"].clone()
    if weighting == "plain":
        m["b"].fill_(-math.inf)
    state = m["state"].clone()
    y = lib.gdn_diag_decode(m["x"], m["a"], m["b"], m["A_log"], state, **kinds(m))
    assert torch.equal(state, m["state"]) and torch.equal(y[:, 0], state.bfloat16())


@pytest.mark.gpu
def test_gradients_without_a_final_states_gradient():
    for keep in ("states", "8bit"):
        m = draw("f32", [63, 0, 200], 70, seed=2)
        m["dstate"] = None
        _, _, kept = prefill(m, keep)
        check_gradients(m, backward(m, kept), keep == "8bit")


@pytest.mark.gpu
@pytest.mark.parametrize("gate,weighting", KINDS)
def test_gradients_against_differences(gate, weighting):
    """The kernels' own forward pass, a step of 2^-5 either way along one direction of all inputs.  The definition's difference
    along it is off from its slope by the step's square; the kernel's by F of the terms over the step besides."""
    m = draw("f32", [40, 90], 64, gate=gate, weighting=weighting, seed=9)
    _, _, kept = prefill(m, "states")
    grads = dict(zip(NAMES, backward(m, kept)))
    g = torch.Generator().manual_seed(1)
    along = {k: (torch.randn(m[k].shape, generator=g) / 16).cuda() for k in ("x", "a", "b", "A_log", "a_bias", "b_bias", "state")}
    slope = sum(float((grads["d" + k].double() * d.double()).sum()) for k, d in along.items())

    def loss(e, run):
        h, s = run(dict(m, **{k: m[k] + e * d for k, d in along.items()}))[:2]
        return float((h.double().cpu().reshape(-1, 64) * wide(m)["dy"]).sum() + (s.double().cpu() * wide(m)["dstate"]).sum())

    step = 2.0 ** -5
    ours, exact = ((loss(step, run) - loss(-step, run)) / (2 * step) for run in (prefill, define))
    h, s, _ = define(m)
    terms = float((h * wide(m)["dy"]).norm() + (s * wide(m)["dstate"]).norm())
    want = define_gradients(m)
    true = sum(float((want["d" + k][0].view(d.shape) * d.double().cpu()).sum()) for k, d in along.items())
    size = sum(float((want["d" + k][1].view(d.shape) * d.double().cpu()).norm()) for k, d in along.items())
    assert abs(slope - ours) <= abs(exact - true) + F * terms / step + F * size


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("C,lens", [(130, [63, 1, 0, 200, 64]), (64, [1500])])
def test_the_kept_codes_are_those_of_pack(io, C, lens):
    """Bit for bit, [x | a | b][slice of 64 channels][rows in whole tiles of 64][64] behind h before every 64th row; what else the
    forward pass returns does not change with what it keeps."""
    m = draw(io, lens, C, seed=12)
    y, state, kept = prefill(m, "8bit")
    for keep in (None, "states"):
        other = prefill(m, keep)
        assert torch.equal(y, other[0]) and torch.equal(state, other[1])
    rows, slices = sum(lens), -(-C // 64)
    tiles = -(-rows // 64)
    data = kept.data[tiles * slices * 256:]
    codes = data[:3 * slices * tiles * 4096].view(torch.int8).view(3, slices, tiles * 64, 64)
    steps = data[3 * slices * tiles * 4096:].view(3, slices, tiles * 64)
    for k, name in enumerate(("x", "a", "b")):
        want, want_steps = lib.gdn_checkpoint_pack(m[name])
        assert torch.equal(codes[k, :, :rows].transpose(0, 1).reshape(rows, -1)[:, :C], want[0])
        assert torch.equal(steps[k, :, :rows].T, want_steps[0])


@pytest.mark.gpu
def test_results_repeat_bit_for_bit():
    for io, keep in (("bf16", "states"), ("f32", "8bit")):
        m = draw(io, [3000, 41, 999], 200, seed=13)
        first = None
        for _ in range(4):
            y, state, kept = prefill(m, keep)
            now = (y, state, *backward(m, kept))
            first = first or [t.clone() for t in now]
            assert all(torch.equal(s, t) for s, t in zip(first, now))


# ------------------------------------------------------------------ single tokens
@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,C,gap,kind", [(1, 64, 0, 0), (9, 130, 0, 1), (5, 257, 1, 2), (3, 1, 0, 3), (33, 512, 4, 4), (4, 516, 2, 5), (300, 64, 0, 3)])
@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("b", [True, False])
def test_tokens_match_the_definition(io, B, C, gap, kind, slots, b):
    gate, weighting = KINDS[kind]
    m = draw(io, [1] * B, C, gate=gate, weighting=weighting, b=b, packed=False, gap=gap, seed=B)
    E = B + 3 if slots else B
    at = torch.randperm(E, generator=torch.Generator().manual_seed(B))[:B].cuda() if slots else torch.arange(B, device="cuda")
    state = torch.full((E, C), 9.0, device="cuda")
    state[at] = m["state"]
    y = lib.gdn_diag_decode(m["x"], m["a"], m["b"], m["A_log"], state, slots=at.int() if slots else None, **kinds(m))
    assert lib.gdn_last_device_status() == 0
    check(m, (y, state[at]))
    assert (state[[e for e in range(E) if e not in at.tolist()]] == 9).all()


@pytest.mark.gpu
def test_tokens_continue_a_prompt():
    m = draw("bf16", [90, 90], 128, packed=False, seed=9)
    want = define(m)
    _, state, _ = prefill(dict(m, **{k: m[k][:, :84].contiguous() for k in ("x", "a", "b")}))
    ys = [lib.gdn_diag_decode(*(m[k][:, t:t + 1] for k in ("x", "a", "b")), m["A_log"], state, **kinds(m)) for t in range(84, 90)]
    near(torch.cat(ys, 1), want[0].view(2, 90, 128)[:, 84:], None, torch.bfloat16)
    near(state, want[1])


@pytest.mark.gpu
def test_a_slot_outside_the_pool_skips_its_row():
    m = draw("bf16", [1, 1, 1], 64, packed=False, seed=10)
    state = m["state"].clone()
    y = torch.full((3, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([2, 3, -1], dtype=torch.int32, device="cuda")
    lib.gdn_diag_decode(m["x"], m["a"], m["b"], m["A_log"], state, slots=slots, y=y, **kinds(m))
    assert lib.gdn_last_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    assert (y[1:] == 5).all() and torch.equal(state[:2], m["state"][:2]) and not torch.equal(state[2], m["state"][2])


# ------------------------------------------------------------------ 8-bit checkpoints
@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,C,gap", [(1, 1, 0), (5, 64, 0), (7, 130, 1), (9, 200, 8), (33, 257, 0), (3, 1024, 0), (40, 72, 0)])
def test_codes_match_the_definition(io, rows, C, gap):
    g = torch.Generator().manual_seed(rows)
    row = (torch.randn(1, rows, C + gap, generator=g) * torch.exp(3 * torch.randn(1, rows, C + gap, generator=g))).clamp(-6e4, 6e4).to(DT[io]).cuda()
    x = row[..., :C]
    codes, steps = lib.gdn_checkpoint_pack(x)
    assert codes.dtype == torch.int8 and steps.shape == (1, rows, -(-C // 64))
    want = stored(x[0].double().cpu())
    scale = 2.0 ** (steps[0].double().cpu() - 133).repeat_interleave(64, 1)[:, :C]
    assert torch.equal(codes[0].double().cpu() * scale, want)
    for dtype in DT.values():
        wide_ = torch.full((1, rows, C + gap), 3.0, dtype=dtype, device="cuda")
        y = lib.gdn_checkpoint_unpack(codes, steps, dtype, y=wide_[..., :C])
        assert torch.equal(y[0].cpu(), want.clamp(-65504, 65504).to(dtype) if dtype == torch.float16 else want.to(dtype))
        assert (wide_[..., C:] == 3).all()


@pytest.mark.gpu
def test_codes_at_the_ends_of_the_range():
    rows = [[0.0] * 4, [1.0, 127 / 128, 0.5 / 128, 1.5 / 128], [127.4, 1.0, 2.5, 3.5], [127.5, 1.0, 3.0, -5.0], [2.0 ** -126, 2.0 ** -117, 2.0 ** -118, 0.0],
            [2.0 ** -149, 0.0, 0.0, 0.0], [torch.finfo(torch.float32).max, -torch.finfo(torch.float32).max, 2.0 ** 127, 1.0],
            [torch.finfo(torch.bfloat16).max, 2.0 ** 121, 2.0 ** 120, 0.0], [-127.49, 127.49, 126.5, -0.0]]
    x = torch.zeros(1, len(rows), 70)
    x[0, :, :4] = torch.tensor(rows)
    got = lib.gdn_checkpoint_unpack(*lib.gdn_checkpoint_pack(x.cuda()), torch.float32)
    assert torch.equal(got[0].double().cpu(), stored(x[0].double())) and torch.isfinite(got).all()
    bad = torch.ones(1, 3, 130, dtype=torch.float16, device="cuda")
    bad[0, 0, 70], bad[0, 1, 129], bad[0, 2, 3] = math.inf, math.nan, -math.inf
    got = lib.gdn_checkpoint_unpack(*lib.gdn_checkpoint_pack(bad), torch.float16)[0]
    want = torch.ones(3, 130, device="cuda")
    want[0, 64:128], want[1, 128:], want[2, :64] = math.nan, math.nan, math.nan
    assert torch.equal(got.isnan(), want.isnan()) and (got[~got.isnan()] == 1).all()
    top = torch.full((1, 1, 64), 65504.0, dtype=torch.float16, device="cuda")
    assert torch.equal(lib.gdn_checkpoint_unpack(*lib.gdn_checkpoint_pack(top), torch.float16), top)


# ------------------------------------------------------------------ rows and entries far apart
@pytest.mark.gpu
def test_rows_beyond_32_bits():
    """Rows 2^25 elements apart: the last ones start behind 2^31 elements and 2^32 bytes."""
    m = draw("bf16", [60, 10], 64, seed=16)
    want, grads = define(m), define_gradients(m)
    big = torch.empty(70, 1 << 25, dtype=torch.bfloat16, device="cuda")
    for k, name in enumerate(("x", "a", "b", "dy")):
        part = big[None, :, 128 * k:128 * k + 64]
        part.copy_(m[name])
        m[name] = part
    outs = [big[None, :, 128 * k:128 * k + 64] for k in range(4, 8)]
    y, state, kept = prefill(m, "states", y=outs[0])
    check(m, (y, state), want)
    for name, t in zip(NAMES, backward(m, kept, dx=outs[1], da=outs[2], db=outs[3])):
        near(t, *grads[name], torch.bfloat16 if name in ("dx", "da", "db") else torch.float32, name)
    codes, steps = lib.gdn_checkpoint_pack(m["x"])
    assert torch.equal(lib.gdn_checkpoint_unpack(codes, steps, y=outs[0])[0].double().cpu(), stored(m["x"][0].double().cpu()))


@pytest.mark.gpu
def test_kept_codes_beyond_32_bits():
    """2^21 rows of 512 channels: the codes of x, a and b take 3 x 2^30 bytes.  The last rows against the same ones alone."""
    T, C = 1 << 21, 512
    g = torch.Generator(device="cuda").manual_seed(1)
    row = torch.randn(1, T, 3 * C, generator=g, device="cuda", dtype=torch.bfloat16)
    cu = torch.tensor([0, T - 1024, T], dtype=torch.int32, device="cuda")
    A_log, dy = torch.full((C,), -1.0, device="cuda"), torch.randn(1, T, C, generator=g, device="cuda", dtype=torch.bfloat16)
    x, a, b = (row[..., k * C:(k + 1) * C] for k in range(3))
    y, state, kept = lib.gdn_diag_prefill(x, a, b, A_log, cu_seqlens=cu, keep="8bit")
    got = lib.gdn_diag_backward(dy, kept, A_log, cu_seqlens=cu)
    tail = lambda t: t[:, T - 1024:].contiguous()  # noqa: E731
    y1, state1, kept1 = lib.gdn_diag_prefill(tail(x), tail(a), tail(b), A_log, keep="8bit")
    alone = lib.gdn_diag_backward(tail(dy), kept1, A_log)
    assert torch.equal(tail(y), y1) and all(torch.equal(tail(s), t) for s, t in zip(got[:3], alone[:3]))


@pytest.mark.gpu
def test_a_pool_beyond_32_bits():
    C, E = 1 << 19, 4400
    m = draw("bf16", [1, 1, 1], C, packed=False, seed=17)
    state = torch.empty(E, C, device="cuda")
    at = torch.tensor([E - 1, 0, E - 7], device="cuda")
    state[at] = m["state"]
    y = lib.gdn_diag_decode(m["x"], m["a"], m["b"], m["A_log"], state, slots=at.int(), **kinds(m))
    check(m, (y, state[at]))


# ------------------------------------------------------------------ streams, graphs
@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported():
    """A budget below one poll of an earlier tile: the call says so, ends, and the next ones are as before."""
    m = draw("bf16", [5300, 300], 256, seed=14)
    y, state, kept = prefill(m, "states")
    want = (y, state, *backward(m, kept))
    gdn.gdn_set_wait_budget(1)
    try:
        lib.gdn_diag_prefill(m["x"], m["a"], m["b"], m["A_log"], state_in=m["state"], cu_seqlens=m["cu"], keep="states", **kinds(m))
        assert lib.gdn_last_device_status() == gdn.GDN_ERR_TIMEOUT
        lib.gdn_diag_backward(m["dy"], kept, m["A_log"], x=m["x"], a=m["a"], b=m["b"], a_bias=m["a_bias"], b_bias=m["b_bias"],
                              state_in=m["state"], cu_seqlens=m["cu"])
        assert lib.gdn_last_device_status() == gdn.GDN_ERR_TIMEOUT
    finally:
        gdn.gdn_set_wait_budget(0)
    y, state, kept = prefill(m, "states")
    assert all(torch.equal(s, t) for s, t in zip((y, state, *backward(m, kept)), want))


@pytest.mark.gpu
def test_one_workspace_for_calls_in_turn():
    """Whatever an earlier call, or nothing, left in it."""
    m = draw("f32", [700, 500], 130, seed=15)
    shape = gdn.GdnDiagShape(0, 1, 1200, 2, 130, 1, 2, 1, 1)
    work = torch.full((gdn.gdn_diag_backward_workspace_bytes(shape),), 255, dtype=torch.uint8, device="cuda")
    y, state, kept = prefill(m, "states")
    want = backward(m, kept)
    for _ in range(3):
        y2, state2, kept2 = prefill(m, "states", workspace=work)
        got = backward(m, kept2, workspace=work)
        assert torch.equal(y, y2) and torch.equal(state, state2) and all(torch.equal(s, t) for s, t in zip(want, got))


@pytest.mark.gpu
@pytest.mark.parametrize("keep", ["states", "8bit"])
def test_two_graphs_and_an_eager_call(keep):
    """Two captured training steps and an eager one, replayed in turn: none keeps anything from another."""
    runs = []
    for lens, seed in (([500, 3, 200], 21), ([1300, 900, 600], 22)):
        m = draw("bf16", lens, 96, seed=seed)
        step = lambda m=m: (lambda y, s, k: (y, s, *lib.gdn_diag_backward(  # noqa: E731
            m["dy"], k, m["A_log"], a_bias=m["a_bias"], b_bias=m["b_bias"], state_in=m["state"], cu_seqlens=m["cu"], dstate_out=m["dstate"],
            **(dict(x=m["x"], a=m["a"], b=m["b"]) if keep == "states" else {}))))(
            *lib.gdn_diag_prefill(m["x"], m["a"], m["b"], m["A_log"], state_in=m["state"], cu_seqlens=m["cu"], keep=keep, **kinds(m)))
        want = [t.clone() for t in step()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        runs.append((step, want, graph, out))
    for i in (0, 1, 1, 0):
        _, want, graph, out = runs[i]
        for t in out:
            t.zero_()
        graph.replay()
        eager = runs[1 - i][0]()
        torch.cuda.synchronize()
        assert all(torch.equal(s, t) for s, t in zip(out, want)) and all(torch.equal(s, t) for s, t in zip(eager, runs[1 - i][1]))
    assert lib.gdn_last_device_status() == 0


@pytest.mark.gpu
def test_on_another_stream():
    m = draw("bf16", [900, 64], 128, seed=23)
    want = prefill(m, "8bit")
    grads = backward(m, want[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, state, kept = lib.gdn_diag_prefill(m["x"], m["a"], m["b"], m["A_log"], state_in=m["state"], cu_seqlens=m["cu"], keep="8bit",
                                          stream=side, **kinds(m))
    got = lib.gdn_diag_backward(m["dy"], kept, m["A_log"], a_bias=m["a_bias"], b_bias=m["b_bias"], state_in=m["state"], cu_seqlens=m["cu"],
                                dstate_out=m["dstate"], stream=side)
    codes = lib.gdn_checkpoint_unpack(*lib.gdn_checkpoint_pack(m["x"], stream=side), m["io"], stream=side)
    step = lib.gdn_diag_decode(*(m[k][:, :1] for k in ("x", "a", "b")), m["A_log"], m["state"][:1].clone(), stream=side, **kinds(m))
    side.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(state, want[1]) and all(torch.equal(s, t) for s, t in zip(got, grads))
    assert torch.equal(codes, lib.gdn_checkpoint_unpack(*lib.gdn_checkpoint_pack(m["x"]), m["io"])) and step.shape == (1, 1, 128)


@pytest.mark.gpu
def test_calls_on_two_streams_at_once():
    """Each has its own workspace, and its tiles wait for its own alone."""
    m = [draw("bf16", lens, 1024, seed=24) for lens in ([2000, 1], [900, 1200, 300])]
    want = [(lambda y, s, k: (y, s, *backward(q, k)))(*prefill(q, "states")) for q in m]
    sides = [torch.cuda.Stream() for _ in m]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for q, side, outs in zip(m, sides, got):
            y, s, kept = lib.gdn_diag_prefill(q["x"], q["a"], q["b"], q["A_log"], state_in=q["state"], cu_seqlens=q["cu"], keep="states",
                                              stream=side, **kinds(q))
            outs.append((y, s, *lib.gdn_diag_backward(q["dy"], kept, q["A_log"], x=q["x"], a=q["a"], b=q["b"], a_bias=q["a_bias"],
                                                      b_bias=q["b_bias"], state_in=q["state"], cu_seqlens=q["cu"], dstate_out=q["dstate"],
                                                      stream=side)))
    torch.cuda.synchronize()
    assert lib.gdn_last_device_status() == 0
    assert all(torch.equal(s, t) for w, outs in zip(want, got) for out in outs for s, t in zip(w, out))


# ------------------------------------------------------------------ a run of them together
@pytest.mark.gpu
def test_a_layer_trains_and_serves():
    """Projection, convolution, recurrence and gated norm as a layer has them: a training step whose checkpoints are 8 bits, its
    gradient through the projection, then the trained layer on a prompt and its next tokens."""
    g = torch.Generator().manual_seed(30)
    D, C, T, K = 64, 128, 150, 4
    rnd = lambda *s, std=1.0: (std * torch.randn(*s, generator=g)).cuda()  # noqa: E731
    weight, conv = rnd(3 * C, D, std=D ** -0.5).bfloat16(), rnd(C, 1, K, std=K ** -0.5).bfloat16()
    A_log, a_bias, b_bias = rnd(C) - 2, rnd(C), rnd(C)
    inputs, dy = rnd(2, T, D).bfloat16(), rnd(2, T, C).bfloat16()
    kw = dict(a_bias=a_bias, b_bias=b_bias, gate="sigmoid")
    past = torch.zeros(2, K - 1, C, dtype=torch.bfloat16, device="cuda")

    def layer(rows, state, past, keep=None):
        row = rows @ weight.T
        x, after = lib.gdn_causal_conv(row[..., :C].contiguous(), conv, None, past, activation="silu")
        return (row, x, after, *lib.gdn_diag_prefill(x, row[..., C:2 * C], row[..., 2 * C:], A_log, state_in=state, keep=keep, **kw))

    row, x, _, y, _, kept = layer(inputs, None, past, "8bit")
    drow = torch.empty_like(row)
    got = lib.gdn_diag_backward(dy, kept, A_log, a_bias=a_bias, b_bias=b_bias, dx=drow[..., :C], da=drow[..., C:2 * C], db=drow[..., 2 * C:])
    m = {"lens": [T, T], "C": C, "gate": "sigmoid", "weighting": "norm", "packed": False, "io": torch.bfloat16, "x": x, "a": row[..., C:2 * C],
         "b": row[..., 2 * C:], "dy": dy, "A_log": A_log, "a_bias": a_bias, "b_bias": b_bias, "state": None, "dstate": None, "cu": None}
    check_gradients(m, got, bits=True)
    grad = drow.flatten(0, 1).T @ inputs.flatten(0, 1)
    assert grad.shape == weight.shape and torch.isfinite(grad.float()).all()
    _, _, past84, y84, state, _ = layer(inputs[:, :84], None, past)
    parts = [y84]
    for t in range(84, 90):
        row = inputs[:, t:t + 1] @ weight.T
        xt, past84 = lib.gdn_causal_conv(row[..., :C].contiguous(), conv, None, past84, activation="silu")
        parts.append(lib.gdn_diag_decode(xt, row[..., C:2 * C], row[..., 2 * C:], A_log, state, **kw))
    near(torch.cat(parts, 1), define(m)[0].view(2, T, C)[:, :90], None, torch.bfloat16)
