"""Rotary positions (gdn_rotary, gdn_rotary_frequencies) against the plain 64-bit definition, their
refusals (on the CPU), and runs with the operators that read their results.

Tolerances (relative, 2-norm): in a 16-bit type the result's one rounding of half a step,
finfo.eps / 2; in fp32 three roundings of 2^-24 (products, sum) and the table's cosine and sine
(2^-23 of a turn), 8 x 2^-24 in all.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import recurrent_state_scan_gb300 as lib
from recurrent_state_scan_gb300 import gdn

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def rel(a, b):
    a, b = a.double().cpu(), b.double().cpu()
    assert torch.isfinite(a).all()
    return float((a - b).norm() / b.norm().clamp_min(1e-300))


def tol(dtype):
    return torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 8 * 2.0 ** -24


def turn(t, pos, inv_freq, offset, interleaved, inverse, scale):
    t = t.double().cpu().clone()
    ang = pos.double().cpu()[..., None, None] * inv_freq.double().cpu() * (-1 if inverse else 1)
    rot = 2 * inv_freq.numel()
    first = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    second = first + (1 if interleaved else rot // 2)
    a, b = t[..., offset + first].clone(), t[..., offset + second].clone()
    t[..., offset + first] = scale * (a * ang.cos() - b * ang.sin())
    t[..., offset + second] = scale * (b * ang.cos() + a * ang.sin())
    return t


@pytest.mark.gpu
@pytest.mark.parametrize("io", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,rot,offset", [(1, 1, 1, 128, 128, 0), (5, 3, 1, 64, 32, 32), (33, 4, 2, 96, 80, 0),
                                                  (7, 2, 0, 50, 18, 5), (4100, 2, 1, 64, 64, 0), (3, 5, 2, 256, 256, 0)])
def test_matches_the_definition(io, interleaved, T, hq, hk, D, rot, offset):
    g = torch.Generator().manual_seed(T + D)
    row = torch.randn(2, T, 3 + (hq + hk) * D + 5, generator=g).to(DT[io]).cuda()
    q = row[..., 3:3 + hq * D].unflatten(2, (hq, D))
    k = row[..., 3 + hq * D:3 + (hq + hk) * D].unflatten(2, (hk, D)) if hk else None
    inv_freq, _ = lib.gdn_rotary_frequencies(rot, device="cuda")
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, T), generator=g).int().cuda()
    for inverse in (False, True):
        for x, dense in ((q, False), (q.contiguous(), True)):
            got = lib.gdn_rotary(x, k, inv_freq, positions=pos, rot_offset=offset, interleaved=interleaved, inverse=inverse,
                                 scale=1.25)
            for t, y in zip((x, k), got):
                if t is not None:
                    assert rel(y, turn(t, pos, inv_freq, offset, interleaved, inverse, 1.25)) <= tol(DT[io])
                    rest = [d for d in range(D) if not offset <= d < offset + rot]
                    assert torch.equal(y[..., rest], t[..., rest])


@pytest.mark.gpu
@pytest.mark.parametrize("io,T,hq,hk,D,rot,offset", [("bf16", 80003, 3, 1, 128, 128, 0), ("f16", 78000, 2, 2, 96, 32, 64),
                                                     ("f32", 40001, 4, 1, 64, 64, 0), ("bf16", 80003, 3, 2, 42, 18, 5)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_rows(io, T, hq, hk, D, rot, offset, interleaved):
    """So many rows that a CTA takes up to 32 of them and goes over its threads' rows several times."""
    g = torch.Generator().manual_seed(T)
    q, k = (torch.randn(1, T, h, D, generator=g).to(DT[io]).cuda() for h in (hq, hk))
    inv_freq, _ = lib.gdn_rotary_frequencies(rot, device="cuda")
    got = lib.gdn_rotary(q, k, inv_freq, rot_offset=offset, interleaved=interleaved)
    for t, y in zip((q, k), got):
        assert rel(y, turn(t, torch.arange(T)[None], inv_freq, offset, interleaved, False, 1.0)) <= tol(DT[io])
        for r in (0, 31, 32, T // 2, T - 1):
            assert rel(y[:, r], turn(t[:, r:r + 1], torch.tensor([[r]]), inv_freq, offset, interleaved, False, 1.0)[:, 0]) <= 2 * tol(DT[io])


@pytest.mark.gpu
def test_places_in_packed_rows_and_in_place():
    g = torch.Generator().manual_seed(1)
    lens = [3, 0, 70, 1]
    cu = torch.tensor([0, 3, 3, 73, 74], dtype=torch.int32, device="cuda")
    row = torch.randn(1, 74, 6 * 64, generator=g).bfloat16().cuda()
    q, k = row[..., :256].unflatten(2, (4, 64)), row[..., 256:].unflatten(2, (2, 64))
    inv_freq, _ = lib.gdn_rotary_frequencies(64, device="cuda")
    pos = torch.cat([torch.arange(n) for n in lens])[None].int().cuda()
    want = lib.gdn_rotary(q, k, inv_freq, positions=pos)
    got = lib.gdn_rotary(q, k, inv_freq, cu_seqlens=cu)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    lib.gdn_rotary(q, k, inv_freq, cu_seqlens=cu, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    batch = row.view(2, 37, -1)[..., :256].unflatten(2, (4, 64))
    got, _ = lib.gdn_rotary(batch, None, inv_freq)
    assert rel(got, turn(batch, torch.arange(37).expand(2, 37), inv_freq, 0, False, False, 1.0)) <= tol(torch.bfloat16)


@pytest.mark.gpu
def test_empty_and_one_sided_calls():
    inv_freq, _ = lib.gdn_rotary_frequencies(64, device="cuda")
    q = torch.randn(2, 0, 4, 64, device="cuda")
    assert lib.gdn_rotary(q, None, inv_freq)[0].shape == q.shape
    none, k = torch.randn(1, 5, 0, 64, device="cuda"), torch.randn(1, 5, 2, 64, device="cuda")
    pos = torch.arange(5, dtype=torch.int32, device="cuda")[None]
    _, got = lib.gdn_rotary(none, k, inv_freq, positions=pos)
    assert rel(got, turn(k, pos, inv_freq, 0, False, False, 1.0)) <= tol(torch.float32)


@pytest.mark.gpu
def test_bad_offsets_are_reported():
    q = torch.randn(1, 8, 1, 64, device="cuda")
    inv_freq, _ = lib.gdn_rotary_frequencies(64, device="cuda")
    lib.gdn_rotary(q, None, inv_freq, cu_seqlens=torch.tensor([0, 5, 4, 9], dtype=torch.int32, device="cuda"))
    assert lib.gdn_last_device_status() == gdn.GDN_ERR_DEVICE_CHECK


@pytest.mark.gpu
def test_inverse_is_the_gradient():
    """The transpose of the turn, against the definition's differences."""
    g = torch.Generator().manual_seed(2)
    inv_freq, scale = lib.gdn_rotary_frequencies(32, kind="bands", factor=4.0, trained_length=512, device="cuda")
    pos = torch.randint(0, 4096, (1, 6), generator=g).int().cuda()
    x, dy, step = (torch.randn(1, 6, 2, 48, generator=g) for _ in range(3))
    dx, _ = lib.gdn_rotary(dy.cuda(), None, inv_freq, positions=pos, inverse=True, scale=scale)
    f = lambda v: (turn(v, pos, inv_freq, 0, False, False, scale) * dy.double()).sum()  # noqa: E731
    e = 1e-4
    slope = (f(x.double() + e * step.double()) - f(x.double() - e * step.double())) / (2 * e)
    assert abs(float((dx.double().cpu() * step.double()).sum() - slope)) <= 8 * 2.0 ** -24 * float(dx.cpu().norm() * step.norm())


@pytest.mark.gpu
def test_turned_queries_and_keys_through_the_linear_rule():
    """q and k turned by position, then the framework's linear rule: its scores depend on distances alone."""
    g = torch.Generator().manual_seed(13)
    q, k, v = (torch.randn(1, 100, 2, 128, generator=g).bfloat16().cuda() for _ in range(3))
    inv_freq, _ = lib.gdn_rotary_frequencies(128, device="cuda")
    outs = []
    for start in (0, 1 << 20):
        pos = (torch.arange(100, dtype=torch.int32) + start)[None].cuda()
        a, b = lib.gdn_rotary(q.float(), k.float(), inv_freq, positions=pos)
        outs.append(lib.gdn_prefill_variant(a, b, v.float(), rule="linear")[0])
    # fp32 throughout: the turns differ by their table's rounding, 2^-22 of each value at most.
    assert rel(outs[1], outs[0]) <= 2.0 ** -20


@pytest.mark.gpu
def test_rows_beyond_32_bits():
    g = torch.Generator().manual_seed(14)
    wide = torch.empty(1, 70, 1 << 25, dtype=torch.bfloat16, device="cuda")
    q = wide[..., 64:64 + 3 * 64].unflatten(2, (3, 64))
    q.copy_(torch.randn(1, 70, 3, 64, generator=g))
    inv_freq, _ = lib.gdn_rotary_frequencies(64, device="cuda")
    want = turn(q, torch.arange(70)[None], inv_freq, 0, False, False, 1.0)
    lib.gdn_rotary(q, None, inv_freq, q_out=q)
    assert rel(q, want) <= 2 ** -8


@pytest.mark.gpu
def test_another_stream_and_a_captured_graph():
    g = torch.Generator().manual_seed(15)
    q, k = torch.randn(2, 37, 4, 128, generator=g).half().cuda(), torch.randn(2, 37, 1, 128, generator=g).half().cuda()
    inv_freq, _ = lib.gdn_rotary_frequencies(128, device="cuda")
    want = lib.gdn_rotary(q, k, inv_freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lib.gdn_rotary(q, k, inv_freq, stream=side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = lib.gdn_rotary(q, k, inv_freq)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(got, want, out))


# ------------------------------------------------------------------ frequencies and refusals (no GPU)
def test_frequencies():
    f = lib.gdn_rotary_frequencies
    i = np.arange(0, 64, 2) / 64
    plain = 1e4 ** -i
    got = {k: f(64, 1e4, k, factor=8.0, trained_length=2048, low=1.0, high=32.0) for k in gdn.ROTARY_KINDS}
    half = 2.0 ** -24      # one rounding to fp32
    near = lambda a, b: np.testing.assert_allclose(a.numpy(), b, rtol=2 * half)  # noqa: E731
    near(got["plain"][0], plain)
    near(got["linear"][0], plain / 8)
    near(got["base"][0], (1e4 * 8 ** (64 / 62)) ** -i)
    turns = 2048 * plain / (2 * math.pi)
    keep = np.clip((turns - 1) / 31, 0, 1)
    near(got["wavelength"][0], plain * (keep + (1 - keep) / 8))
    lo, hi = (64 * math.log(2048 / (t * 2 * math.pi)) / (2 * math.log(1e4)) for t in (32.0, 1.0))
    keep = 1 - np.clip((np.arange(32) - math.floor(lo)) / (math.ceil(hi) - math.floor(lo)), 0, 1)
    near(got["bands"][0], plain * (keep + (1 - keep) / 8))
    assert [got[k][1] for k in ("plain", "linear", "base", "wavelength")] == [1.0] * 4
    assert abs(got["bands"][1] - (0.1 * math.log(8) + 1)) <= 2 * half


@pytest.mark.parametrize("bad", [dict(kind="other"), dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=258), dict(base=1.0),
                                 dict(base=math.inf), dict(kind="linear", factor=0.5), dict(kind="base", rot_dim=2, factor=2.0),
                                 dict(kind="bands", factor=2.0), dict(kind="wavelength", factor=2.0, trained_length=99, low=2.0, high=2.0),
                                 dict(kind="linear", factor=math.nan), dict(kind="bands", factor=2.0, trained_length=math.inf)])
def test_frequency_refusals(bad):
    with pytest.raises(lib.GdnError):
        lib.gdn_rotary_frequencies(**dict(dict(rot_dim=64), **bad))


P64 = [ctypes.c_void_p(1 << 40 | i << 32) for i in range(8)]     # addresses that are never read: every call is refused
off = lambda i, d: ctypes.c_void_p(P64[i].value + d)  # noqa: E731


@pytest.mark.parametrize("bad", [dict(io_dtype=4), dict(num_seqs=2), dict(heads_q=-1), dict(head_dim=1), dict(head_dim=2000),
                                 dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(rot_offset=1), dict(rot_offset=-2),
                                 dict(rot_offset=2 ** 31 - 1), dict(scale=math.nan), dict(q_head_stride=32), dict(k_row_stride=1),
                                 dict(k_out_row_stride=64), dict(seqlen=-1), dict(seqlen=2 ** 31), dict(inv=None), dict(q=None),
                                 dict(k_out=None), dict(q=off(0, 1)), dict(inv=off(2, 2)), dict(q_out=P64[0], q_out_row_stride=512)])
def test_refusals(bad):
    d = dict(io_dtype=1, batch=1, seqlen=4, num_seqs=1, heads_q=4, heads_k=2, head_dim=64, rot_dim=64, rot_offset=0, interleaved=0,
             inverse=0, scale=1.0, q_row_stride=256, q_head_stride=64, k_row_stride=128, k_head_stride=64, q_out_row_stride=256,
             q_out_head_stride=64, k_out_row_stride=128, k_out_head_stride=64)
    ptr = dict(q=P64[0], k=P64[1], inv=P64[2], pos=None, cu=None, q_out=P64[5], k_out=P64[6])
    for key, v in bad.items():
        (ptr if key in ptr else d)[key] = v
    assert lib.load().gdn_rotary(ctypes.byref(gdn.GdnRotaryShape(**d)), *ptr.values(), None) == gdn.GDN_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors():
    with pytest.raises(lib.GdnError):
        lib.gdn_rotary(torch.randn(1, 2, 3, 16), None, torch.ones(8))


@pytest.mark.parametrize("batch,seqlen", [(4, 2 ** 62), (2, 2 ** 63 - 1), (65536, 2 ** 48), (2 ** 31 - 1, 2)])
def test_token_counts_beyond_64_bits_are_refused(batch, seqlen):
    """batch x seqlen is 0 or small modulo 2^64 in some of these."""
    test_refusals(dict(batch=batch, num_seqs=batch, seqlen=seqlen))
