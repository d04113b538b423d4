"""The state-space layer (gdn_ssm_prefill, gdn_ssm_decode) against the plain 64-bit definition, its
refusals (on the CPU), and a run of it with the rotary positions and the layer ops around it.

Tolerances, relative in the 2-norm unless said otherwise, count roundings of half a step,
u = finfo(t).eps / 2 (bf16 2^-8, f16 2^-11, f32 2^-24).  With q = u / sqrt(3), the root mean square of
a rounding spread evenly over half a step each way:
* y of 16-bit types is rounded once, and on the tensor cores its two parts meet one more
  rounding each (the decay-weighted scores, the state); three independent ones and a margin of
  two: 2 sqrt(3) q = 2 u.
* The fp32 state and fp32 y: sums of up to T = 700 terms in fp32 whose errors add as at most
  T u = 4e-5 in the worst case and sqrt(T) u = 1.6e-6 as they fall; exp and log1p add 2 ulp a
  step on exponents up to 16: 1e-5 bounds both, and the three-term bf16 split of the tensor
  cores (2^-24 of each product) stays inside it.
* Behind a convolution in a 16-bit type, x and B are roundings of an fp32 value whose own error, some
  8 x 2^-24 of it, puts it on the other side of a rounding's border than the 64-bit value with
  probability 2 x 8 x 2^-24 over a step (bf16 2^-8, f16 2^-11 at least): p = 2^-12, 2^-9.  It is then
  off by a whole step (2^-7, 2^-10 at most), so the state's mean square error is 2 p step^2 = 2^-25,
  2^-28 of its square, the few values of a small case seeing up to four times its root: 2^-10.5, 2^-12.
"""
import ctypes
import math

import pytest
import torch

import recurrent_state_scan_gb300 as lib
from recurrent_state_scan_gb300 import gdn
from test_rotary import rel, turn

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
STATE_TOL = 1e-5


def state_tol(m):
    return {torch.bfloat16: 2.0 ** -10.5, torch.float16: 2.0 ** -12}.get(m["io"], STATE_TOL) if m["K"] else STATE_TOL


def y_tol(dtype):
    return 1e-5 if dtype == torch.float32 else 2 * torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ inputs and definitions
def draw(io, lens, H, P, G, N, K, *, packed=True, z=True, initial=True, seed=0, device="cuda", gap=5):
    """A layer's tensors; x, dt and z are slices of one row with `gap` unused values behind them."""
    g = torch.Generator().manual_seed(seed)
    dt_ = DT[io]
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0] if lens else 0)
    C, n = H * P + 2 * G * N, len(lens)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    row = rnd(B, T, 2 * H * P + 2 * G * N + H + gap).to(dt_).to(device)
    hp = H * P
    m = {"lens": lens, "H": H, "P": P, "G": G, "N": N, "K": K, "packed": packed, "io": dt_,
         "z": row[..., :hp].unflatten(2, (H, P)) if z else None, "xbc": row[..., hp:hp + C], "dt": row[..., hp + C:hp + C + H],
         "A_log": torch.log(1 + 15 * torch.rand(H, generator=g)).to(device), "dt_bias": (rnd(H) - 3).to(device),
         "D": rnd(H).to(device), "w": None, "b": None, "conv": None, "state": None, "cu": None}
    if K:
        m["w"], m["b"] = (rnd(C, 1, K) * K ** -0.5).to(dt_).to(device), (0.1 * rnd(C)).to(dt_).to(device)
        m["conv"] = rnd(n, K - 1, C).to(dt_).to(device) if initial else None
    if initial:
        m["state"] = (0.5 * rnd(n, H, N, P)).to(device)
    if packed:
        m["cu"] = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device=device)
    return m


def kwargs(m):
    return dict(heads=m["H"], head_dim=m["P"], groups=m["G"], d_state=m["N"], D=m["D"], dt_bias=m["dt_bias"], z=m["z"],
                conv_weight=m["w"], conv_bias=m["b"])


def prefill(m, **kw):
    out = lib.gdn_ssm_prefill(m["xbc"], m["dt"], m["A_log"], state_in=m["state"], conv_state_in=m["conv"], cu_seqlens=m["cu"],
                              **kwargs(m), **kw)
    torch.cuda.synchronize()
    assert lib.gdn_last_device_status() == 0
    return out


def define(m, dt_min=0.0, dt_max=math.inf, silu=True):
    """(y, state, conv state) token by token in 64 bits."""
    H, P, G, N, K, io = (m[k] for k in ("H", "P", "G", "N", "K", "io"))
    C = H * P + 2 * G * N
    x = m["xbc"].reshape(-1, C).double().cpu()
    dt = m["dt"].reshape(-1, H).double().cpu()
    z = m["z"].reshape(-1, H, P).double().cpu() if m["z"] is not None else None
    A, bias, D = (m[k].double().cpu() for k in ("A_log", "dt_bias", "D"))
    y, states, convs, r = torch.zeros(x.shape[0], H, P, dtype=torch.float64), [], [], 0
    for i, L in enumerate(m["lens"]):
        S = m["state"][i].double().cpu().clone() if m["state"] is not None else torch.zeros(H, N, P, dtype=torch.float64)
        past = m["conv"][i].double().cpu() if m["conv"] is not None else torch.zeros(max(K - 1, 0), C, dtype=torch.float64)
        pad = torch.cat([past, x[r:r + L]])
        u = x[r:r + L]
        if K and L:
            w = m["w"].double().cpu()[:, 0]
            u = m["b"].double().cpu() + sum(w[:, j] * pad[j:j + L] for j in range(K))
            u = (u * torch.sigmoid(u) if silu else u).to(io).double()
        for t in range(L):
            d = torch.nn.functional.softplus(dt[r + t] + bias, threshold=100).clamp(dt_min, dt_max)
            xt = u[t, :H * P].view(H, P)
            b, c = (u[t, H * P + k * G * N:H * P + (k + 1) * G * N].view(G, N).repeat_interleave(H // G, 0) for k in (0, 1))
            S = S * torch.exp(-torch.exp(A) * d)[:, None, None] + (d[:, None] * b)[..., None] * xt[:, None]
            out = (c[..., None] * S).sum(1) + D[:, None] * xt
            y[r + t] = out * z[r + t] * torch.sigmoid(z[r + t]) if z is not None else out
        states.append(S)
        convs.append(pad[L:])
        r += L
    empty = torch.zeros(0, max(K - 1, 0), C, dtype=torch.float64)
    return (y.view(m["xbc"].shape[0], -1, H, P) if y.numel() else y, torch.stack(states) if states else torch.zeros(0, H, N, P),
            (torch.stack(convs) if convs else empty) if K else None)


def check(m, got, want):
    y, state, conv = got
    if y.numel():
        assert rel(y, want[0]) <= y_tol(m["io"]), ("y", rel(y, want[0]))
    if not want[1].numel():
        assert state.shape == want[1].shape
    elif want[1].abs().max() > 0:
        assert rel(state, want[1]) <= state_tol(m), ("state", rel(state, want[1]))
    else:
        assert torch.count_nonzero(state) == 0
    if m["K"]:
        assert torch.equal(conv.double().cpu(), want[2])


# ------------------------------------------------------------------ prompts
@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H,P,G,N,K", [(4, 64, 1, 128, 4), (4, 64, 2, 64, 4), (6, 32, 3, 16, 2), (2, 48, 2, 100, 3),
                                       (2, 128, 1, 128, 0), (3, 4, 1, 1, 1), (2, 52, 1, 90, 4), (1, 256, 1, 256, 0),
                                       (2, 80, 2, 33, 4)])
def test_prompts_match_the_definition(io, H, P, G, N, K):
    m = draw(io, [63, 1, 0, 200, 64, 2, 129], H, P, G, N, K, seed=H * P + N)
    check(m, prefill(m), define(m))


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens,packed", [([1], False), ([3, 3], False), ([65, 65, 65], False), ([700], True), ([0, 0, 5], True),
                                         ([0], True), ([], True)])
@pytest.mark.parametrize("initial,z", [(False, False), (True, True)])
def test_prompt_lengths(io, lens, packed, initial, z):
    m = draw(io, lens, 4, 64, 2, 128, 4, packed=packed, initial=initial, z=z, seed=len(lens), gap=8)
    check(m, prefill(m), define(m))


@pytest.mark.gpu
@pytest.mark.parametrize("gap", [0, 1, 8])
def test_rows_may_be_slices_at_any_stride(gap):
    m = draw("bf16", [150, 20], 4, 64, 1, 128, 0, gap=gap, seed=3)
    want = define(m)
    check(m, prefill(m), want)
    for name in ("xbc", "dt", "z"):
        m[name] = m[name].contiguous()
    check(m, prefill(m), want)


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16"])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
def test_convolved_rows_on_16_bytes(io, K):
    """Rows that bulk copies can take, in runs that hold several sequences, a sequence several runs."""
    H, P, G, N = 9, 64, 1, 40
    m = draw(io, [1, 2, 0, 3, 150, 70, 1, 1, 77, 5], H, P, G, N, K, seed=K, gap=(-(2 * H * P + 2 * G * N + H)) % 8)
    assert m["xbc"].stride(1) % 8 == 0 and m["xbc"].data_ptr() % 16 == 0
    check(m, prefill(m), define(m))


@pytest.mark.gpu
@pytest.mark.parametrize("io,T,K,gap", [("bf16", 4000, 4, 0), ("bf16", 4000, 3, 0), ("bf16", 4001, 2, 8), ("bf16", 3999, 1, 0),
                                        ("f16", 4000, 4, 0), ("f16", 4003, 2, 8), ("bf16", 4000, 4, 1), ("f16", 4000, 3, 2),
                                        ("f32", 4000, 4, 0), ("f32", 4002, 2, 4), ("f32", 4000, 3, 1)])
def test_convolved_rows_in_long_runs(io, T, K, gap):
    """Runs of many stages (rows on 16 bytes: 42 rows in stages of 6, four at a time), sequences that begin and end inside them.
    With C's taps 0, D 1 and no earlier state y is the convolved x: against the definition, within its one rounding (and 16 x 2^-24
    of the sum's, the exponential's and the quotient's in fp32), and bit for bit against every row as a single token."""
    H, P, N = 64, 64, 16
    lens = [1000, 41, 1, 0, 7, 1500, 3, 42, 84]
    lens.append(T - sum(lens))
    C, hp, n = H * P + 2 * N, H * P, len(lens)
    g = torch.Generator().manual_seed(T + K)
    row = (3 * torch.randn(1, T, C + H + (-(C + H)) % 8 + gap, generator=g)).to(DT[io]).cuda()
    x, dt = row[..., :C], row[..., C:C + H]
    w = (torch.randn(C, 1, K, generator=g) * K ** -0.5).to(DT[io])
    b = (0.1 * torch.randn(C, generator=g)).to(DT[io])
    w[hp + N:], b[hp + N:] = 0, 0
    w, b, past = w.cuda(), b.cuda(), torch.randn(n, K - 1, C, generator=g).to(DT[io]).cuda()
    cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    layer = dict(heads=H, head_dim=P, d_state=N, D=torch.ones(H, device="cuda"), conv_weight=w, conv_bias=b)
    A_log = torch.zeros(H, device="cuda")
    y, _, conv = lib.gdn_ssm_prefill(x, dt, A_log, conv_state_in=past, cu_seqlens=cu, **layer)
    assert lib.gdn_last_device_status() == 0
    before, pads = [], []
    for i, L in enumerate(lens):
        pads.append(torch.cat([past[i], x[0, cu[i]:cu[i + 1]]]))
        before.append(torch.stack([pads[-1][j:j + L] for j in range(K)], 1))       # [L, K, C]
    rows = torch.cat(before)
    assert torch.equal(conv, torch.stack([p[len(p) - (K - 1):] for p in pads]))
    u, size = b.double().expand(T, C)[:, :hp], b.double().abs().expand(T, C)[:, :hp]
    for j in range(K):
        u = u + w[:hp, 0, j].double() * rows[:, j, :hp].double()
        size = size + (w[:hp, 0, j].double() * rows[:, j, :hp].double()).abs()
    want = (u * torch.sigmoid(u)).view(1, T, H, P)
    off = (want.abs() * torch.finfo(DT[io]).eps / 2 + 16 * 2.0 ** -24 * (size.view_as(want) + want.abs()) + torch.finfo(DT[io]).tiny)
    assert ((y.double() - want).abs() <= off).all()
    del u, size, want, off
    state = torch.zeros(T, H, N, P, device="cuda")
    tokens = lib.gdn_ssm_decode(x.transpose(0, 1), dt.transpose(0, 1), A_log, state, conv_state=rows[:, :-1].contiguous(), **layer)
    assert lib.gdn_last_device_status() == 0 and torch.equal(tokens.view_as(y), y)


@pytest.mark.gpu
def test_optional_operands_and_bounds_on_the_step():
    m = draw("f32", [40, 3], 4, 32, 2, 16, 3, seed=4)
    args = dict(kwargs(m), D=None, dt_bias=None, conv_bias=None)
    got = lib.gdn_ssm_prefill(m["xbc"], m["dt"], m["A_log"], state_in=m["state"], conv_state_in=m["conv"], cu_seqlens=m["cu"],
                              dt_min=0.3, dt_max=0.8, conv_activation="none", **args)
    m["D"], m["dt_bias"], m["b"] = torch.zeros_like(m["D"]), torch.zeros_like(m["D"]), torch.zeros_like(m["b"])
    check(m, got, define(m, 0.3, 0.8, silu=False))


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_extreme_steps(io):
    """Steps of zero (dt = -inf) leave the state alone; huge decays clear it without NaN."""
    m = draw(io, [150], 2, 64, 1, 128, 0, z=False, seed=5)
    dt = m["dt"].clone()
    dt[:, 10:30] = -math.inf
    dt[:, 70] = 3e4
    dt[:, 100:140:7] = 60.0
    m["dt"] = dt
    m["A_log"] = torch.tensor([2.5, 0.0], device="cuda")
    check(m, prefill(m), define(m))
    m["lens"], m["xbc"], m["dt"], m["cu"] = [20], m["xbc"][:, 10:30], dt[:, 10:30], torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    _, state, _ = prefill(m)
    assert torch.equal(state, m["state"])


@pytest.mark.gpu
@pytest.mark.parametrize("io,P", [("bf16", 64), ("bf16", 52), ("f32", 64)])
def test_rates_beyond_fp32(io, P):
    """e^A_log above fp32's range: every token with a step clears the state, one without (dt = -inf) leaves it, the last of a tile too."""
    m = draw(io, [75, 5, 1], 2, P, 1, 64, 0, z=False, seed=32)
    m["A_log"] = torch.tensor([95.0, 88.5], device="cuda")
    m["dt"] = m["dt"].clone()
    m["dt"][:, 60:75], m["dt"][:, 80] = -math.inf, -math.inf
    got = prefill(m)
    check(m, got, define(m))
    assert torch.equal(got[1][2], m["state"][2])
    wide = draw(io, [1, 1], 2, 128, 1, 128, 0, packed=False, z=False, seed=33)
    for m in (draw(io, [1, 1], 2, P, 1, 64, 0, packed=False, z=False, seed=33), wide):
        m["A_log"], m["dt"] = torch.tensor([95.0, 88.5], device="cuda"), m["dt"].clone()
        m["dt"][1] = -math.inf
        state = m["state"].clone()
        y = lib.gdn_ssm_decode(m["xbc"], m["dt"], m["A_log"], state, **kwargs(m))
        check(m, (y, state, None), define(m))
        assert torch.equal(state[1], m["state"][1])


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("gap", [0, 1])
def test_gates_far_out(io, gap):
    """A gate far below zero shuts, one far above passes, a NaN stays."""
    m = draw(io, [70], 2, 64, 1, 64, 0, seed=25, gap=gap)
    z = m["z"].clone() if gap == 0 else torch.empty(1, 70, 129, dtype=DT[io], device="cuda")[..., 1:].unflatten(2, (2, 64)).copy_(m["z"])
    z[:, 10], z[:, 66], z[:, 20], z[:, 30, 0, 3] = -3e38, -100.0, 1000.0, math.nan
    m["z"] = z
    y, want = prefill(m)[0], define(m)[0]
    plain = prefill(dict(m, z=None))[0]
    assert (y[:, 10].abs() <= 2.0 ** -50 * plain[:, 10].abs()).all() and (y[:, 66].abs() <= 2.0 ** -50 * plain[:, 66].abs()).all()
    assert rel(y[:, 20], want[:, 20]) <= y_tol(DT[io]) and y[0, 30, 0, 3].isnan() and int(y.isnan().sum()) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gates_keep_their_digits(io):
    """Each value against the ungated one times silu(z) in 64 bits, on the FP32 cores.  The exponential is off by 2 units in the
    last place, the sum, the quotient and the two products by half a one each: 4 x 2^-23.  In bf16 by fast intrinsics, |z| + 8
    times 2^-23 at most, and two roundings more."""
    far = torch.tensor([-0.5, -5.0, -20.0, -40.0, -60.0, -80.0, -86.0, -88.0, 0.0, 0.25, 5.0, 60.0, 100.0])
    m = draw(io, [1] * 26, 2, 52, 1, 33, 0, packed=False, seed=29)
    m["z"] = (far.repeat(2)[:, None, None, None] + 0.125 * torch.rand(26, 1, 2, 52, generator=torch.Generator().manual_seed(1))).to(DT[io]).cuda()
    silu = m["z"].double() * torch.sigmoid(m["z"].double())
    off = 2.0 ** -16 + 2 * 2.0 ** -8 if io == "bf16" else 4 * 2.0 ** -23

    def near(gated, plain):
        want = plain.double() * silu
        assert ((gated.double() - want).abs() <= off * want.abs() + 2.0 ** -133).all()

    near(prefill(m)[0], prefill(dict(m, z=None))[0])
    token = lambda z: lib.gdn_ssm_decode(m["xbc"], m["dt"], m["A_log"], m["state"].clone(), **dict(kwargs(m), z=z))  # noqa: E731
    near(token(m["z"]), token(None))
    wide = dict(draw(io, [1] * 26, 2, 128, 1, 128, 0, packed=False, seed=30), z=None)       # (the step of larger states)
    token = lambda z: lib.gdn_ssm_decode(wide["xbc"], wide["dt"], wide["A_log"], wide["state"].clone(), **dict(kwargs(wide), z=z))  # noqa: E731
    m["z"] = torch.cat([m["z"], m["z"], m["z"][..., :24]], 3)
    silu = m["z"].double() * torch.sigmoid(m["z"].double())
    near(token(m["z"]), token(None))


@pytest.mark.gpu
@pytest.mark.parametrize("gap", [0, 1])
def test_gates_keep_their_digits_on_the_tensor_cores(gap):
    """Each value against the ungated one times silu(z) in 64 bits: two roundings to bf16, and |z| + 8 times 2^-23 of fast
    intrinsics at most.  (Off 16 bytes z comes by plain loads.)"""
    far = torch.tensor([-0.5, -5.0, -20.0, -40.0, -41.5, -44.0, -50.0, -60.0, -70.0, -80.0, -86.0, 0.0, 0.25, 5.0, 60.0, 100.0])
    m = draw("bf16", [80], 2, 64, 1, 64, 0, seed=31, gap=(-(2 * 2 * 64 + 2 * 64 + 2)) % 8)
    rows = far.repeat(5)[None, :, None, None] + 0.125 * torch.rand(1, 80, 2, 64, generator=torch.Generator().manual_seed(1))
    wide = torch.empty(1, 80, 128 + gap, dtype=torch.bfloat16, device="cuda")
    m["z"] = wide[..., gap:].unflatten(2, (2, 64)).copy_(rows)
    silu = m["z"].double() * torch.sigmoid(m["z"].double())
    want = prefill(dict(m, z=None))[0].double() * silu
    assert ((prefill(m)[0].double() - want).abs() <= (2 * 2.0 ** -8 + 2.0 ** -16) * want.abs() + 2.0 ** -133).all()


@pytest.mark.gpu
@pytest.mark.parametrize("lens,packed", [([700, 64, 130, 1], True), ([1600], False)])
def test_states_of_the_tensor_cores_are_fp32(lens, packed):
    """bf16 prompts return a state that is carried on, so its products w x B keep fp32's digits.  A token's weight w = d e^{G - G_j} is
    off by two units of 2^-23 for its step, as much for the logarithm, log2 w's roundings (half a unit of 2^-20 below 16, times
    ln 2) and the exponential: 8.2 x 2^-23 at most, and the products and their sums some 2^-24 at random signs."""
    m = draw("bf16", lens, 4, 64, 2, 128, 0, packed=packed, initial=False, seed=34, gap=(-(2 * 4 * 64 + 512 + 4)) % 8)
    shape = gdn.GdnSsmShape(1, 1, sum(lens), len(lens), 4, 64, 2, 128, m["xbc"].stride(1), 0, 0)
    assert gdn.gdn_ssm_prefill_plan(shape, gdn.GdnSsmParams(0, 0, 0.0, 1.0))[0] in (gdn.PATH_TC, gdn.PATH_TC_TP)
    assert rel(prefill(m)[1], define(m)[1]) <= 2.0 ** -20


@pytest.mark.gpu
def test_slow_decays_do_not_drift():
    """2,000 tokens that forget next to nothing.  Each rounds its decay (half a step below 1: 2^-25), the state's update
    (2^-24) and its own share (twice 2^-24, of a small part): at random, so they add up to sqrt(2000) times 2 * 2^-24 at most."""
    m = draw("f32", [2000], 4, 32, 1, 16, 0, z=False, seed=24)
    m["A_log"] = torch.full((4,), -6.0, device="cuda")
    _, state, _ = prefill(m)
    assert rel(state, define(m)[1]) <= 2000 ** 0.5 * 2 * 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("H,n,T,path", [(64, 3, 65536, gdn.PATH_TC), (2, 1, 65536, gdn.PATH_TC_TP)])
@pytest.mark.parametrize("A_log", [-10.0, -8.0])
def test_slow_decays_do_not_drift_over_chunks(H, n, T, path, A_log):
    """1,024 chunks (or 128 segments of 8) that forget next to nothing and write nothing.  Each chunk rounds its decay (2^-25) and
    the state (2^-24), at random: sqrt(1024) times 1.5 * 2^-24; the exponent's own roundings are 2^-22 of it."""
    m = draw("bf16", [T] * n, H, 8, 1, 16, 0, packed=False, z=False, seed=28)
    shape = gdn.GdnSsmShape(1, n, T, n, H, 8, 1, 16, 0, 0, 0)
    assert gdn.gdn_ssm_prefill_plan(shape, gdn.GdnSsmParams(0, 0, 0.0, 1.0))[0] == path
    m["A_log"], m["xbc"] = torch.full((H,), A_log, device="cuda"), torch.zeros_like(m["xbc"])
    steps = torch.nn.functional.softplus(m["dt"].double() + m["dt_bias"].double(), threshold=100).sum(1)
    g = math.exp(A_log) * steps
    state = prefill(m)[1].double()
    want = m["state"].double() * torch.exp(-g)[:, :, None, None]
    assert rel(state, want) <= 1024 ** 0.5 * 1.5 * 2.0 ** -24 + float(g.max()) * 2.0 ** -22


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 2])
def test_fast_decays_keep_their_digits(io, T):
    """Tokens that write nothing: the state is S0 e^g, g = -sum of steps.  The step, A and their product round 2 x 2^-23 of g in
    all, the exponential 2 units in the last place and the product half a one, to each token: T (2 |g| + 3) 2^-23."""
    m = draw(io, [T], 9, 64, 1, 64, 0, packed=False, z=False, seed=27)
    m["dt"] = torch.tensor([0.0, 1.0, 3.0, 6.0, 10.0, 14.0, 17.0, 20.0, 40.0], dtype=DT[io], device="cuda").repeat(T, 1)[None]
    m["A_log"], m["dt_bias"], m["xbc"] = torch.zeros(9, device="cuda"), torch.zeros(9, device="cuda"), torch.zeros_like(m["xbc"])
    g = T * torch.nn.functional.softplus(m["dt"][0, 0].double().cpu(), threshold=100)
    want = m["state"].double().cpu() * torch.exp(-g)[:, None, None]
    stepped = m["state"].clone()
    for t in range(T):
        lib.gdn_ssm_decode(m["xbc"][:, t:t + 1], m["dt"][:, t:t + 1], m["A_log"], stepped, **kwargs(m))
    for state in (prefill(m)[1], stepped):
        for h in range(9):
            assert rel(state[:, h], want[:, h]) <= T * (2 * float(g[h]) + 3) * 2.0 ** -23, (h, rel(state[:, h], want[:, h]))


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_a_sequence_does_not_see_its_neighbours(io):
    """Rows of another sequence, infinities and NaN among them, leave a packed sequence's results bit for bit."""
    m = draw(io, [70, 33, 90], 4, 64, 2, 128, 4, seed=6)
    y, state, conv = prefill(m)
    m["xbc"] = m["xbc"].clone()
    m["xbc"][:, :70] = math.nan
    m["xbc"][:, 103:] = math.inf
    y2, state2, conv2 = prefill(m)
    assert torch.equal(y[:, 70:103], y2[:, 70:103]) and torch.equal(state[1], state2[1]) and torch.equal(conv[1], conv2[1])


@pytest.mark.gpu
def test_chained_calls_and_states_in_place():
    m = draw("bf16", [300], 4, 64, 1, 128, 4, packed=False, seed=7)
    y, state, conv = prefill(m)
    parts = []
    for a, b in ((0, 101), (101, 165), (165, 300)):
        p = dict(m, lens=[b - a], **{k: m[k][:, a:b] for k in ("xbc", "dt", "z")})
        yp, p["state"], p["conv"] = prefill(p, state_out=None if a == 0 else p["state"])
        m["state"], m["conv"] = p["state"], p["conv"]
        parts.append(yp)
    assert rel(torch.cat(parts, 1), y) <= 2 * y_tol(torch.bfloat16)
    assert rel(m["state"], state) <= 2 * STATE_TOL and torch.equal(m["conv"], conv)


@pytest.mark.gpu
def test_bad_offsets_are_reported_and_skipped():
    m = draw("bf16", [100, 60, 40], 2, 64, 1, 128, 4, seed=8)
    good = prefill(m)
    m["cu"] = torch.tensor([0, 100, 90, 200], dtype=torch.int32, device="cuda")
    y, state, conv = (torch.full_like(t, 7.0) for t in good)
    lib.gdn_ssm_prefill(m["xbc"], m["dt"], m["A_log"], state_in=m["state"], conv_state_in=m["conv"], cu_seqlens=m["cu"],
                        y=y, state_out=state, conv_state_out=conv, **kwargs(m))
    assert lib.gdn_last_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    assert torch.equal(state[0], good[1][0]) and (state[1] == 7).all() and (conv[1] == 7).all()
    assert torch.equal(y[:, :90], good[0][:, :90])


@pytest.mark.gpu
@pytest.mark.parametrize("H,P,G,N", [(2, 64, 1, 128), (3, 64, 1, 100), (6, 128, 2, 64), (5, 80, 1, 16)])
@pytest.mark.parametrize("lens,packed", [([3000], False), ([1500, 1500], False), ([2100, 5, 0, 1400, 513], True)])
def test_long_prompts_in_time_segments(H, P, G, N, lens, packed):
    """Odd unit counts and lengths over several segments, against the fp32 cores' scan of the same values."""
    m = draw("bf16", lens, H, P, G, N, 0, packed=packed, seed=N + len(lens), gap=(-(2 * H * P + 2 * G * N + H)) % 8)
    shape = gdn.GdnSsmShape(1, len(lens) if not packed else 1, sum(lens) if packed else lens[0], len(lens), H, P, G, N, 0, 0, 0)
    assert gdn.gdn_ssm_prefill_plan(shape, gdn.GdnSsmParams(0, 0, 0.0, 1.0))[0] == gdn.PATH_TC_TP
    wide = dict(m, io=torch.float32, **{k: m[k].float() for k in ("xbc", "dt", "z")})
    check(m, prefill(m), prefill(wide))


@pytest.mark.gpu
@pytest.mark.parametrize("H,lens", [
    (64, [700, 3, 650, 0, 690, 64, 65, 2]),                              # long enough to cut, but none worth it
    (64, [1800, 3, 650, 0, 90, 64, 65, 2]),                              # one that is
    (2, [(37 * i * i) % 150 for i in range(1300)]),                      # more sequences than threads, some empty
    (4, [64] * 700 + [0] * 5 + [1] * 40),
])
def test_packed_prompts_by_length(H, lens):
    """The long ones are taken first: each sequence is still computed, once, wherever it stands."""
    m = draw("bf16", lens, H, 64, 1, 32, 0, seed=len(lens), gap=(-(2 * H * 64 + 64 + H)) % 8)
    wide = dict(m, io=torch.float32, **{k: m[k].float() for k in ("xbc", "dt", "z")})
    check(m, prefill(m), prefill(wide))


@pytest.mark.gpu
def test_bad_offsets_among_long_sequences():
    """An offset far too high makes two sequences overlap and one bad: the others are as they were (uncut, where they were cut)."""
    lens = [1500, 40, 1500, 900]
    m = draw("bf16", lens, 4, 64, 1, 64, 0, seed=26, gap=(-(2 * 4 * 64 + 128 + 4)) % 8)
    good = prefill(m)
    m["cu"][1] = 3900                                    # sequence 0 runs into the others, 1 ends before it begins
    y, state = (torch.full_like(t, 7.0) for t in good[:2])
    lib.gdn_ssm_prefill(m["xbc"], m["dt"], m["A_log"], state_in=m["state"], cu_seqlens=m["cu"], y=y, state_out=state, **kwargs(m))
    assert lib.gdn_last_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    assert rel(state[2:], good[1][2:]) <= 2 * STATE_TOL and (state[1] == 7).all()


@pytest.mark.gpu
def test_bad_offsets_among_many_sequences():
    """Sequences of bad offsets are left alone, the others computed."""
    lens = [70] * 400
    m = draw("bf16", lens, 4, 64, 1, 16, 0, seed=5)
    good = prefill(m)
    m["cu"][200] = 20000
    y, state = (torch.full_like(t, 7.0) for t in good[:2])
    lib.gdn_ssm_prefill(m["xbc"], m["dt"], m["A_log"], state_in=m["state"], cu_seqlens=m["cu"], y=y, state_out=state, **kwargs(m))
    assert lib.gdn_last_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    assert torch.equal(state[:199], good[1][:199]) and torch.equal(state[201:], good[1][201:]) and (state[200] == 7).all()
    assert torch.equal(y[:, :199 * 70], good[0][:, :199 * 70])


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported():
    m = draw("bf16", [300, 1400], 4, 64, 1, 128, 0, seed=14)
    want = prefill(m)
    gdn.gdn_set_wait_budget(50)          # far below one tile load
    try:
        lib.gdn_ssm_prefill(m["xbc"], m["dt"], m["A_log"], state_in=m["state"], cu_seqlens=m["cu"], **kwargs(m))
        torch.cuda.synchronize()
        assert lib.gdn_last_device_status() == gdn.GDN_ERR_TIMEOUT
    finally:
        gdn.gdn_set_wait_budget(0)
    assert all(torch.equal(a, b) for a, b in zip(prefill(m)[:2], want[:2]))


# ------------------------------------------------------------------ single tokens
@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,H,P,G,N,K", [(1, 4, 64, 1, 128, 4), (9, 6, 48, 3, 100, 4), (5, 2, 256, 1, 256, 2), (3, 2, 4, 1, 1, 1),
                                         (4, 4, 52, 2, 33, 0), (2, 3, 80, 1, 16, 3)])
@pytest.mark.parametrize("slots", [False, True])
def test_tokens_match_the_definition(io, B, H, P, G, N, K, slots):
    m = draw(io, [1] * B, H, P, G, N, K, packed=False, seed=B)
    want = define(m)
    E = B + 3 if slots else B
    at = torch.randperm(E, generator=torch.Generator().manual_seed(B))[:B].cuda() if slots else torch.arange(B, device="cuda")
    state = torch.full((E, H, N, P), 9.0, device="cuda")
    state[at] = m["state"]
    conv = None
    if K:
        conv = torch.full((E, K - 1, H * P + 2 * G * N), 9.0, device="cuda", dtype=DT[io])
        conv[at] = m["conv"]
    y = lib.gdn_ssm_decode(m["xbc"], m["dt"], m["A_log"], state, conv_state=conv, slots=at.int() if slots else None, **kwargs(m))
    assert lib.gdn_last_device_status() == 0
    check(m, (y, state[at], conv[at] if K else None), want)
    rest = [e for e in range(E) if e not in at.tolist()]
    assert (state[rest] == 9).all() and (conv is None or (conv[rest] == 9).all())


@pytest.mark.gpu
def test_tokens_continue_a_prompt():
    m = draw("bf16", [90, 90], 4, 64, 2, 128, 4, packed=False, seed=9)
    want = define(m)
    head = dict(m, lens=[84, 84], **{k: m[k][:, :84].contiguous() for k in ("xbc", "dt", "z")})
    _, state, conv = prefill(head)
    ys = []
    for t in range(84, 90):
        step = dict(m, **{k: m[k][:, t:t + 1] for k in ("xbc", "dt", "z")})
        ys.append(lib.gdn_ssm_decode(step["xbc"], step["dt"], step["A_log"], state, conv_state=conv, **kwargs(step)))
    assert rel(torch.cat(ys, 1), want[0][:, 84:]) <= y_tol(torch.bfloat16)
    assert rel(state, want[1]) <= state_tol(m) and torch.equal(conv.double().cpu(), want[2])


@pytest.mark.gpu
def test_a_slot_outside_the_pool_skips_its_row():
    m = draw("bf16", [1, 1, 1], 2, 64, 1, 128, 4, packed=False, seed=10)
    state, conv = m["state"].clone(), m["conv"].clone()
    y = torch.full((3, 1, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([2, 3, -1], dtype=torch.int32, device="cuda")
    lib.gdn_ssm_decode(m["xbc"], m["dt"], m["A_log"], state, conv_state=conv, slots=slots, y=y, **kwargs(m))
    assert lib.gdn_last_device_status() == gdn.GDN_ERR_DEVICE_CHECK
    assert (y[1:] == 5).all() and torch.equal(state[:2], m["state"][:2]) and torch.equal(conv[:2], m["conv"][:2])
    assert not torch.equal(state[2], m["state"][2])


@pytest.mark.gpu
@pytest.mark.parametrize("K,gap", [(2, 0), (3, 0), (4, 0), (4, 5)])
@pytest.mark.parametrize("slots", [False, True])
def test_many_tokens(slots, K, gap):
    """More rows and heads than a launch holds blocks for; mixed rows on 16 bytes and off them."""
    B = 150
    m = draw("bf16", [1] * B, 8, 64, 2, 64, K, packed=False, seed=15, gap=gap)
    at = torch.randperm(B, generator=torch.Generator().manual_seed(1)).cuda() if slots else torch.arange(B, device="cuda")
    state, conv = torch.empty_like(m["state"]), torch.empty_like(m["conv"])
    state[at], conv[at] = m["state"], m["conv"]
    y = lib.gdn_ssm_decode(m["xbc"], m["dt"], m["A_log"], state, conv_state=conv, slots=at.int() if slots else None, **kwargs(m))
    check(m, (y, state[at], conv[at]), define(m))


# ------------------------------------------------------------------ rows and entries far apart
@pytest.mark.gpu
@pytest.mark.parametrize("io,K", [("bf16", 0), ("bf16", 4), ("f16", 4)])
def test_rows_beyond_32_bits(io, K):
    """Rows 2^25 elements apart: the last ones start behind 2^31 elements and 2^32 bytes."""
    m = draw(io, [60, 10], 4, 64, 1, 64, K, seed=16)
    want = define(m)
    for name in ("xbc", "dt", "z"):
        wide = torch.empty(70, 1 << 25, dtype=DT[io], device="cuda")
        rows = m[name].flatten(2)
        part = wide[None, :, 64:64 + rows.shape[2]]
        part.copy_(rows)
        m[name] = part.unflatten(2, m[name].shape[2:])
    check(m, prefill(m), want)
    last = {k: m[k][:, 69:] for k in ("xbc", "dt", "z")}
    one = dict(m, lens=[1], packed=False, state=m["state"][:1], conv=m["conv"][:1] if K else None, **last)
    state, conv = one["state"].clone(), one["conv"].clone() if K else None
    y = lib.gdn_ssm_decode(one["xbc"], one["dt"], one["A_log"], state, conv_state=conv, **kwargs(one))
    check(one, (y, state, conv), define(one))


@pytest.mark.gpu
@pytest.mark.parametrize("H,P", [(64, 64), (32, 128)])
def test_a_pool_beyond_32_bits(H, P):
    m = draw("bf16", [1, 1, 1], H, P, 1, 128, 4, packed=False, seed=17)
    E = 4400                                             # of 2^19 fp32 values each
    state = torch.empty(E, H, 128, P, device="cuda")
    conv = torch.empty(E, 3, m["xbc"].shape[2], dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([E - 1, 0, E - 7], device="cuda")
    state[at], conv[at] = m["state"], m["conv"]
    y = lib.gdn_ssm_decode(m["xbc"], m["dt"], m["A_log"], state, conv_state=conv, slots=at.int(), **kwargs(m))
    assert lib.gdn_last_device_status() == 0
    check(m, (y, state[at], conv[at]), define(m))


# ------------------------------------------------------------------ streams, graphs
@pytest.mark.gpu
def test_two_graphs_and_an_eager_call():
    """Two captured calls and an eager one, replayed in turn: none keeps anything from another."""
    runs = []
    for lens, seed in (([500, 3, 200], 21), ([1300, 900], 22)):
        m = draw("bf16", lens, 64, 64, 2, 64, 4, seed=seed, gap=(-(2 * 4096 + 256 + 64)) % 8)
        want = prefill(m)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = lib.gdn_ssm_prefill(m["xbc"], m["dt"], m["A_log"], state_in=m["state"], conv_state_in=m["conv"],
                                      cu_seqlens=m["cu"], **kwargs(m))
        runs.append((m, want, graph, out))
    for i in (0, 1, 1, 0):
        m, want, graph, out = runs[i]
        for t in out:
            t.zero_()
        graph.replay()
        eager = prefill(runs[1 - i][0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for a, b in zip(eager, runs[1 - i][1]))


@pytest.mark.gpu
def test_captured_tokens_advance_the_states():
    m = draw("bf16", [6, 6], 4, 64, 1, 128, 4, packed=False, seed=23)
    want = define(m)
    state, conv = m["state"].clone(), m["conv"].clone()
    step = {k: m[k][:, :1].clone() for k in ("xbc", "dt", "z")}
    call = lambda **kw: lib.gdn_ssm_decode(step["xbc"], step["dt"], m["A_log"], state, conv_state=conv,  # noqa: E731
                                           **dict(kwargs(m), z=step["z"]), **kw)
    call()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        y = call()
    state.copy_(m["state"])
    conv.copy_(m["conv"])
    ys = []
    for t in range(6):
        for k in step:
            step[k].copy_(m[k][:, t:t + 1])
        graph.replay()
        ys.append(y.clone())
    assert rel(torch.cat(ys, 1), want[0]) <= y_tol(torch.bfloat16)
    assert rel(state, want[1]) <= state_tol(m) and torch.equal(conv.double().cpu(), want[2])


@pytest.mark.gpu
def test_another_stream_and_a_captured_graph():
    m = draw("bf16", [200, 50], 4, 64, 1, 128, 4, seed=11)
    want = prefill(m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = prefill(m, stream=side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = lib.gdn_ssm_prefill(m["xbc"], m["dt"], m["A_log"], state_in=m["state"], conv_state_in=m["conv"],
                                  cu_seqlens=m["cu"], **kwargs(m))
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


# ------------------------------------------------------------------ the operators together
@pytest.mark.gpu
def test_convolution_turn_scan_norm():
    """A layer whose B and C turn with the position: conv, rotary in place on the mixed row, scan, gated norm."""
    H, P, G, N, K, lens = 4, 64, 2, 128, 4, [90, 37]
    m = draw("bf16", lens, H, P, G, N, 0, z=False, initial=False, seed=12)
    C = H * P + 2 * G * N
    w = (torch.randn(C, 1, K, generator=torch.Generator().manual_seed(1)) * 0.5).bfloat16().cuda()
    u = torch.cat([lib.gdn_causal_conv(part.contiguous(), w, activation="silu")[0] for part in m["xbc"].split(lens, 1)], 1)
    inv_freq, _ = lib.gdn_rotary_frequencies(64, device="cuda")
    c, b = (u[..., H * P + i * G * N:H * P + (i + 1) * G * N].unflatten(2, (G, N)) for i in (1, 0))
    pos = torch.cat([torch.arange(n) for n in lens])[None].int().cuda()
    want_c, want_b = (turn(t, pos, inv_freq, 64, True, False, 1.0).bfloat16() for t in (c, b))
    lib.gdn_rotary(c, b, inv_freq, cu_seqlens=m["cu"], rot_offset=64, interleaved=True, q_out=c, k_out=b)
    assert rel(c, want_c) <= 2 ** -8 and rel(b, want_b) <= 2 ** -8
    m["xbc"] = u
    got = prefill(m)
    check(m, got, define(m))
    gate = torch.randn(got[0].shape, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    y = lib.gdn_gated_rmsnorm(got[0], torch.ones(P, dtype=torch.bfloat16, device="cuda"), gate)
    o, gt = got[0].double(), gate.double()
    assert rel(y, o * (o.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * gt * torch.sigmoid(gt)) <= 2 ** -8


# ------------------------------------------------------------------ refusals (no GPU)
def _ssm(**kw):
    d = dict(io_dtype=1, batch=1, seqlen=4, num_seqs=1, heads=4, head_dim=64, groups=2, d_state=16, xbc_stride=0, dt_stride=0,
             z_stride=0)
    return gdn.GdnSsmShape(**dict(d, **kw))


def _params(**kw):
    return gdn.GdnSsmParams(**dict(dict(conv_kernel=4, conv_activation=1, dt_min=0.0, dt_max=1.0), **kw))


BAD_SHAPES = [dict(io_dtype=5), dict(batch=-1, num_seqs=-1), dict(seqlen=-1), dict(num_seqs=2), dict(heads=0), dict(groups=3),
              dict(groups=0), dict(head_dim=0), dict(head_dim=6), dict(head_dim=260), dict(d_state=0), dict(d_state=257),
              dict(xbc_stride=5), dict(dt_stride=3), dict(z_stride=1), dict(heads=65536, groups=1), dict(seqlen=2 ** 31),
              dict(heads=65535, groups=65535, head_dim=64, d_state=128)]
BAD_PARAMS = [dict(conv_kernel=5), dict(conv_kernel=-1), dict(conv_activation=2), dict(dt_min=-1.0), dict(dt_min=math.nan),
              dict(dt_max=math.nan), dict(dt_min=2.0), dict(dt_min=math.inf, dt_max=math.inf)]
P64 = [ctypes.c_void_p(1 << 40 | i << 32) for i in range(16)]     # addresses that are never read: every call is refused
off = lambda i, d: ctypes.c_void_p(P64[i].value + d)  # noqa: E731


def call_prefill(shape, params, **over):
    names = ["xbc", "dt", "z", "w", "b", "conv_in", "conv_out", "A_log", "dt_bias", "D", "state_in", "cu", "y", "state_out", "ws"]
    a = dict(zip(names, P64), cu=None)
    a.update(over)
    return lib.load().gdn_ssm_prefill(ctypes.byref(shape) if shape else None, ctypes.byref(params) if params else None,
                                      *[a[n] for n in names], a.get("ws_bytes", 1 << 30), None)


def call_decode(shape, params, **over):
    names = ["xbc", "dt", "z", "w", "b", "conv", "A_log", "dt_bias", "D", "state"]
    a = dict(zip(names, P64), pool=4, slots=None, y=P64[12])
    a.update(over)
    return lib.load().gdn_ssm_decode(ctypes.byref(shape) if shape else None, ctypes.byref(params) if params else None,
                                     *[a[n] for n in names], a["pool"], a["slots"], a["y"], None)


@pytest.mark.parametrize("shape,params", [(s, {}) for s in BAD_SHAPES] + [({}, p) for p in BAD_PARAMS])
def test_bad_geometry_is_refused(shape, params):
    for call, t in ((call_prefill, 4), (call_decode, 1)):
        s = _ssm(**dict(dict(seqlen=t), **shape))
        assert call(s, _params(**params)) in (gdn.GDN_ERR_INVALID_ARG, gdn.GDN_ERR_UNSUPPORTED)
    if "num_seqs" not in shape or "batch" in shape:      # (batch 1 and two sequences: packed, to the query)
        assert lib.load().gdn_ssm_prefill_workspace_bytes(ctypes.byref(_ssm(**shape)), ctypes.byref(_params(**params))) == 0


@pytest.mark.parametrize("over", [dict(xbc=None), dict(dt=None), dict(w=None), dict(A_log=None), dict(y=None), dict(state_out=None),
                                  dict(conv_out=None), dict(ws=None), dict(ws_bytes=100), dict(ws=off(14, 8)), dict(xbc=off(0, 1)),
                                  dict(A_log=off(7, 2)), dict(state_in=off(10, 4)), dict(state_out=off(13, 8)),
                                  dict(y=P64[0]), dict(y=P64[2]), dict(conv_out=P64[5]), dict(state_out=off(10, 16))])
def test_bad_prefill_pointers_are_refused(over):
    assert call_prefill(_ssm(), _params(), **over) == gdn.GDN_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(xbc=None), dict(dt=None), dict(w=None), dict(A_log=None), dict(y=None), dict(state=None),
                                  dict(conv=None), dict(state=off(9, 4)), dict(slots=P64[14], pool=0), dict(slots=off(14, 2)),
                                  dict(y=P64[0]), dict(z=off(2, 1))])
def test_bad_decode_pointers_are_refused(over):
    assert call_decode(_ssm(seqlen=1), _params(), **over) == gdn.GDN_ERR_INVALID_ARG
    assert call_decode(_ssm(seqlen=2), _params()) == gdn.GDN_ERR_INVALID_ARG
    assert call_prefill(None, _params()) == call_prefill(_ssm(), None) == gdn.GDN_ERR_INVALID_ARG


@pytest.mark.parametrize("shape,params,want", [
    (dict(seqlen=8192, heads=64, groups=1, d_state=128), {}, (gdn.PATH_TC_TP, 4)),
    (dict(seqlen=8192, heads=64, groups=1, d_state=128), dict(conv_kernel=0), (gdn.PATH_TC_TP, 3)),
    (dict(seqlen=8192, heads=64, groups=1, d_state=100), dict(conv_kernel=0), (gdn.PATH_TC_TP, 4)),
    (dict(seqlen=100, heads=64, groups=8), {}, (gdn.PATH_TC, 2)), (dict(seqlen=100, batch=64, num_seqs=64), dict(conv_kernel=0), (gdn.PATH_TC, 1)),
    (dict(seqlen=16384, num_seqs=12, heads=64, groups=8, d_state=128), {}, (gdn.PATH_TC_TP, 5)),
    (dict(seqlen=16384, num_seqs=12, heads=512, groups=8, d_state=128), dict(conv_kernel=0), (gdn.PATH_TC, 2)),
    (dict(io_dtype=0), {}, (gdn.PATH_SIMT, 2)), (dict(io_dtype=2), dict(conv_kernel=0), (gdn.PATH_SIMT, 1)),
    (dict(d_state=129), {}, (gdn.PATH_SIMT, 2)), (dict(head_dim=52), {}, (gdn.PATH_SIMT, 2)), (dict(batch=0, num_seqs=0), {}, (gdn.PATH_SIMT, 0))])
def test_plans(shape, params, want):
    assert gdn.gdn_ssm_prefill_plan(_ssm(**shape), _params(**params)) == want


def test_nothing_to_do_is_no_error():
    assert call_prefill(_ssm(batch=0, num_seqs=0), _params()) == gdn.GDN_OK
    assert call_decode(_ssm(batch=0, num_seqs=0, seqlen=1), _params()) == gdn.GDN_OK


def test_binding_refuses_cpu_tensors():
    m = draw("f32", [4], 2, 32, 1, 16, 2, device="cpu")
    for call in (lambda: lib.gdn_ssm_prefill(m["xbc"], m["dt"], m["A_log"], state_in=m["state"], conv_state_in=m["conv"], **kwargs(m)),
                 lambda: lib.gdn_ssm_decode(m["xbc"][:, :1], m["dt"][:, :1], m["A_log"], m["state"], conv_state=m["conv"],
                                            **dict(kwargs(m), z=None))):
        with pytest.raises(lib.GdnError):
            call()


@pytest.mark.parametrize("name,row", [("xbc", (24,)), ("dt", (4,)), ("z", (4, 4)), ("dt", (1,))])
@pytest.mark.parametrize("B,T", [(1, 512), (32, 1), (3, 7)])
def test_expanded_rows_are_refused(name, row, B, T):
    """A stride of 0 over several rows is not the C calls' 0 for contiguous rows: they would read what the tensor does not hold."""
    t = torch.zeros(1, 1, *row).expand(B, T, *row)
    with pytest.raises(lib.GdnError, match="overlap"):
        gdn._rows(name, t, B, T, row, torch.float32, t.get_device())
    copied = t.contiguous()
    assert gdn._rows(name, copied, B, T, row, torch.float32, copied.get_device()) == (copied.data_ptr(), math.prod(row))


def test_rows_closer_than_their_width_are_refused():
    for B, T, strides in ((1, 8, (0, 2, 1)), (8, 1, (2, 0, 1)), (2, 4, (8, 2, 1))):
        t = torch.zeros(64).as_strided((B, T, 4), strides)
        with pytest.raises(lib.GdnError, match="overlap"):
            gdn._rows("dt", t, B, T, (4,), torch.float32, t.get_device())


def test_rows_of_any_wider_stride_are_taken():
    wide = torch.zeros(2, 6, 9)
    for t, want in ((wide[..., 2:6], 9), (wide[:, :1, 2:6], 54), (wide[:1, :1, 2:6], 4), (wide[:1, :, 2:6], 9),
                    (wide[:, :0, 2:6], 54), (torch.zeros(1, 1, 4).expand(1, 1, 4), 4)):
        assert gdn._rows("dt", t, *t.shape[:2], (4,), torch.float32, t.get_device()) == (t.data_ptr(), want)


@pytest.mark.parametrize("batch,seqlen", [(4, 2 ** 62), (2, 2 ** 63 - 1), (65536, 2 ** 48), (3, 2 ** 31), (2 ** 31 - 1, 2)])
def test_token_counts_beyond_64_bits_are_refused(batch, seqlen):
    """batch x seqlen is 0 or small modulo 2^64 in some of these."""
    shape = _ssm(batch=batch, num_seqs=batch, seqlen=seqlen)
    assert call_prefill(shape, _params()) == gdn.GDN_ERR_UNSUPPORTED
    assert call_decode(shape, _params()) == gdn.GDN_ERR_UNSUPPORTED
    assert lib.load().gdn_ssm_prefill_workspace_bytes(ctypes.byref(shape), ctypes.byref(_params())) == 0
    with pytest.raises(lib.GdnError):
        gdn.gdn_ssm_prefill_plan(shape, _params())


@pytest.mark.parametrize("d,stride", [(0, 0), (-8, 0), (1024, 600), (-2 * 600 * 3, 600)])
def test_y_over_dt_is_refused(d, stride):
    """Steps are read while other heads' results are being stored.  y holds 4 x 256 values of 2 bytes; dt 4 x 4, or rows of 600."""
    call = lambda fn, t: fn(_ssm(seqlen=t, batch=4 // t, num_seqs=4 // t, dt_stride=stride), _params(), y=off(1, -d))  # noqa: E731
    assert call(call_prefill, 4) == call(call_decode, 1) == gdn.GDN_ERR_INVALID_ARG
    assert b"dt" in lib.load().gdn_last_error_message()


@pytest.mark.parametrize("io_dtype", [0, 1])
@pytest.mark.parametrize("kernel,want", [(0, 1), (1, 1), (2, 2), (4, 2)])
def test_plans_without_tokens(io_dtype, kernel, want):
    """Sequences without tokens hand their conv states on by the convolution's launch, where there are any (K > 1)."""
    for shape in (dict(seqlen=0), dict(seqlen=0, num_seqs=3), dict(seqlen=0, batch=5, num_seqs=5)):
        assert gdn.gdn_ssm_prefill_plan(_ssm(io_dtype=io_dtype, **shape), _params(conv_kernel=kernel)) == (gdn.PATH_SIMT, want)


def test_rows_wider_than_a_grid_are_refused():
    """The step would have run, and the launch behind it, which moves the conv states on, failed."""
    for call, t in ((call_prefill, 4), (call_decode, 1)):      # rows of 2^24 elements
        assert call(_ssm(heads=65535, head_dim=256, groups=1, d_state=128, seqlen=t), _params()) == gdn.GDN_ERR_UNSUPPORTED


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """(Torch would have made it current on its own device, and the call have run on this one's default stream.)"""
    class Stream:
        device_index = 1
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    with pytest.raises(lib.GdnError, match="stream must be on cuda:0"):
        with gdn._on(0, Stream()):
            pass
