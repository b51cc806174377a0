"""Rotary positions with the cache write (pa_rope_frequencies, pa_rope_and_cache) against the
formula in 64 bits."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_350_b200 as pa
from paged_kv_cache_350_b200 import binding as B

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rotate(x, positions, inv_freq, factor, interleaved):
    """x [T, H, D] (64 bits) with its first 2 * len(inv_freq) elements rotated, one complex
    product per pair; also |a| + |b| per element, for the tolerance."""
    y, size = x.clone(), x.abs().clone()
    half = len(inv_freq)
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    angle = positions.double()[:, None] * torch.from_numpy(inv_freq)[None, :]
    unit = torch.polar(torch.full_like(angle, factor), angle)[:, None, :]
    z = torch.complex(x[..., a], x[..., b]) * unit
    y[..., a], y[..., b] = z.real, z.imag
    size[..., a] = size[..., b] = (x[..., a].abs() + x[..., b].abs()) * factor
    return y, size


def tolerance(ref, size, dtype):
    # The fraction of a turn is rounded to 32 bits (|frac| <= 1/2: 2^-26 turns = 9.4e-8 rad), sin
    # and cos are off by 2 ulp of at most 1 (2.4e-7), their product with the factor and the two
    # products and one sum of the rotation each by 2^-24 (2.4e-7 in all): below 6e-7 of |a| + |b|.
    # The result's rounding to its type adds half a step.
    return size * 6e-7 + (ref.abs() * torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 0)


# ---- frequencies ---------------------------------------------------------------------------

def test_frequencies_plain_and_linear():
    f, a = pa.pa_rope_frequencies(64, 10000.0)
    assert f.shape == (32,) and a == 1.0 and f[0] == 1.0
    np.testing.assert_allclose(f, 10000.0 ** (-np.arange(32) / 32.0), rtol=1e-14)
    g, a = pa.pa_rope_frequencies(64, 10000.0, pa.PA_ROPE_SCALE_LINEAR, 4.0)
    np.testing.assert_allclose(g, f / 4.0, rtol=1e-14)
    assert a == 1.0


@pytest.mark.parametrize("R", [2, 16, 128])
def test_frequencies_stretched_base(R):
    f, _ = pa.pa_rope_frequencies(R, 500.0)
    g, _ = pa.pa_rope_frequencies(R, 500.0, pa.PA_ROPE_SCALE_BASE, 8.0)
    assert g[0] == 1.0
    if R > 2:  # the slowest pair is interpolated by the factor
        np.testing.assert_allclose(g[-1], f[-1] / 8.0, rtol=1e-12)
    assert np.all(np.diff(f / g) >= -1e-12)


def test_frequencies_ramp_and_bands():
    R, base, s, old = 128, 10000.0, 16.0, 4096
    f, _ = pa.pa_rope_frequencies(R, base)
    turns = old * f / (2 * math.pi)
    for kind in (pa.PA_ROPE_SCALE_RAMP, pa.PA_ROPE_SCALE_BANDS):
        g, a = pa.pa_rope_frequencies(R, base, kind, s, old, 32.0, 1.0)
        ratio = f / g
        assert np.all(np.diff(ratio) >= -1e-12)
        # (the ramp's ends are whole indexes: one pair to either side)
        np.testing.assert_allclose(ratio[np.flatnonzero(turns > 32)[:-1]], 1.0, rtol=1e-12)
        np.testing.assert_allclose(ratio[np.flatnonzero(turns < 1)[1:]], s, rtol=1e-12)
        if kind == pa.PA_ROPE_SCALE_RAMP:
            assert a == pytest.approx(0.1 * math.log(s) + 1.0, rel=1e-6)
        else:
            keep = np.clip((turns - 1.0) / 31.0, 0, 1)
            np.testing.assert_allclose(g, f * keep + f / s * (1 - keep), rtol=1e-12)
            assert a == 1.0


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, base=1.0),
                                dict(rotary_dim=8, base=float("inf")),
                                dict(rotary_dim=8, scaling=pa.PA_ROPE_SCALE_LINEAR, factor=0.5),
                                dict(rotary_dim=8, scaling=pa.PA_ROPE_SCALE_RAMP, factor=2.0),
                                dict(rotary_dim=8, scaling=pa.PA_ROPE_SCALE_BANDS, factor=2.0, original_len=64,
                                     fast=1.0, slow=1.0), dict(rotary_dim=8, scaling=9)])
def test_frequencies_refusals(kw):
    with pytest.raises(pa.PAError) as e:
        pa.pa_rope_frequencies(**kw)
    assert e.value.status == B.PA_ERR_INVALID_ARG


def test_rope_refusals_on_the_host():
    """The C entry refuses bad sizes before it touches a pointer or the device."""
    def call(**kw):
        a = dict(T=4, Hq=4, Hkv=2, D=64, bs=16, NB=4, qs=256, ks=128, vs=128, R=64, layout=0, f=1.0, dt=B.PA_BF16,
                 q_out=0x1000, q=0x2000)
        a.update(kw)
        p = 0x10000
        return B.lib.pa_rope_and_cache(a["q_out"], a["q"], p, p, p, p, p, p, p, a["T"], a["Hq"], a["Hkv"], a["D"],
                                       a["bs"], a["NB"], a["qs"], a["ks"], a["vs"], a["R"], a["layout"], a["f"],
                                       a["dt"], None, None)
    for bad in (dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(NB=0), dict(R=0), dict(R=63), dict(R=66), dict(layout=2),
                dict(f=float("nan")), dict(dt=7), dict(qs=255), dict(ks=127), dict(vs=0), dict(q_out=None),
                dict(q_out=0x1001), dict(q_out=0x2000, qs=512), dict(q_out=0x2010), dict(q_out=0x1810)):
        assert call(**bad) == B.PA_ERR_INVALID_ARG, bad
    for bad in (dict(D=96), dict(bs=5)):
        assert call(**bad) == B.PA_ERR_UNSUPPORTED, bad
    assert call(T=0) == B.PA_OK


# ---- on the GPU ------------------------------------------------------------------------------

def run_case(dtype, T, Hq, Hkv, D, bs, R, interleaved, far=4096, pad=0, offset=0, extra=0, factor=1.0, seed=0,
             in_place=False):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    width = (Hq + 2 * Hkv) * D + extra
    buf = torch.randn(offset + T * width, generator=g).to(dt)
    row = buf[offset:].view(T, width)
    cut = lambda t, a, h: t[:, a:a + h * D].view(T, h, D)  # noqa: E731
    NB = (T + bs - 1) // bs + 2
    kp, vp = (torch.randn(NB, bs, Hkv, D, generator=g).to(dt) for _ in range(2))
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32)
    if T:
        pos[0], pos[-1] = far - 1, 0
    slots = torch.randperm(NB * bs, generator=g)[:T].contiguous()
    slots[T - pad:] = -1
    inv, _ = pa.pa_rope_frequencies(R, 10000.0)
    rk, rv = kp.double().view(-1, Hkv, D).clone(), vp.double().view(-1, Hkv, D).clone()
    sk = torch.zeros_like(rk)
    q, k, v = cut(row, 0, Hq), cut(row, Hq * D, Hkv), cut(row, (Hq + Hkv) * D, Hkv)
    rq, sq = rotate(q.double(), pos, inv, factor, interleaved)
    ry, sy = rotate(k.double(), pos, inv, factor, interleaved)
    live = slots >= 0
    rk[slots[live]], sk[slots[live]], rv[slots[live]] = ry[live], sy[live], v.double()[live]

    dev_buf = buf.cuda()
    drow = dev_buf[offset:].view(T, width)
    dq = cut(drow, 0, Hq)
    if in_place:
        dq = dq.contiguous()
    out = dq if in_place else torch.full((T, Hq, D), float("nan"), dtype=dt, device="cuda")
    dk, dv = kp.cuda(), vp.cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_rope_and_cache(out, dq, cut(drow, Hq * D, Hkv), cut(drow, (Hq + Hkv) * D, Hkv), dk, dv, pos.cuda(),
                         slots.cuda(), torch.from_numpy(inv).cuda(),
                         layout=pa.PA_ROPE_INTERLEAVED if interleaved else pa.PA_ROPE_HALF, attn_factor=factor,
                         err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    got_q, got_k = out.cpu().double(), dk.cpu().double().view(-1, Hkv, D)
    assert bool(((got_q - rq).abs() <= tolerance(rq, sq, dt)).all())
    assert bool(((got_k - rk).abs() <= torch.where(sk > 0, tolerance(rk, sk, dt), 0.0)).all())
    assert torch.equal(dv.cpu().double().view(-1, Hkv, D), rv)
    if R < D:  # what is not rotated passes through
        assert torch.equal(got_q[..., R:], rq[..., R:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,bs,R", [
    (1, 32, 8, 128, 16, 128), (1, 1, 1, 64, 4, 64), (257, 8, 2, 64, 8, 32), (33, 6, 3, 128, 32, 2),
    (40, 14, 2, 64, 16, 48), (17, 5, 5, 128, 16, 126), (19, 7, 1, 64, 16, 22), (3, 64, 64, 128, 4, 16),
    (5, 3, 1, 128, 16, 100), (1000, 1, 1, 64, 16, 62)])
def test_rope_matches_formula(dtype, interleaved, T, Hq, Hkv, D, bs, R):
    run_case(dtype, T, Hq, Hkv, D, bs, R, interleaved, pad=T // 5, factor=1.0 if T % 2 else 1.2, seed=T + R)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_far_positions(dtype, interleaved):
    run_case(dtype, 300, 4, 2, 128, 16, 128, interleaved, far=(1 << 31) - 1, seed=5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset,extra", [(0, 1), (1, 0), (3, 5), (8, 8), (4, 4), (2, 2)])
def test_rope_strides_and_offsets(dtype, offset, extra):
    run_case(dtype, 29, 4, 2, 64, 16, 64, False, offset=offset, extra=extra, seed=offset)
    run_case(dtype, 29, 4, 2, 64, 16, 20, True, offset=offset, extra=extra, seed=offset)


@pytest.mark.gpu
def test_rope_in_place_and_all_padded():
    run_case("bf16", 31, 4, 2, 128, 16, 64, False, in_place=True)
    run_case("bf16", 31, 4, 2, 128, 16, 50, False, in_place=True)
    run_case("f32", 31, 4, 2, 128, 16, 64, True, in_place=True)
    run_case("bf16", 12, 4, 2, 64, 16, 64, False, pad=12)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("R", [64, 50])
def test_rope_in_a_graph_on_another_stream(layout, R):
    """Captured and replayed: it follows its inputs, and the same inputs give the same bits."""
    T, Hq, Hkv, D, bs = 40, 6, 2, 64, 8
    q, k, v = (torch.randn(T, h, D, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    kp, vp = (torch.zeros(8, bs, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.randperm(64, device="cuda")[:T]
    inv = torch.from_numpy(pa.pa_rope_frequencies(R)[0]).cuda()
    out = torch.empty_like(q)
    call = lambda s=None: pa.pa_rope_and_cache(out, q, k, v, kp, vp, pos, slots, inv, layout=layout, stream=s)  # noqa: E731
    torch.cuda.synchronize()
    call(torch.cuda.Stream())
    torch.cuda.synchronize()
    first = out.clone(), kp.clone(), vp.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in (out, kp, vp):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (out, kp, vp)))
    pos.add_(7)
    graph.replay()
    torch.cuda.synchronize()
    ref, size = rotate(q.cpu().double(), pos.cpu(), inv.cpu().numpy(), 1.0, layout == 1)
    assert bool(((out.cpu().double() - ref).abs() <= tolerance(ref, size, torch.bfloat16)).all())


@pytest.mark.gpu
def test_rope_bad_slot_is_flagged_and_skipped():
    T, Hq, Hkv, D, bs, NB = 4, 2, 1, 64, 16, 2
    q, k, v = (torch.randn(T, h, D, device="cuda") for h in (Hq, Hkv, Hkv))
    kp, vp = (torch.zeros(NB, bs, Hkv, D, device="cuda") for _ in range(2))
    slots = torch.tensor([0, 32, 1 << 40, 5], device="cuda")
    inv = torch.from_numpy(pa.pa_rope_frequencies(D)[0]).cuda()
    for R in (64, 6):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)
        pa.pa_rope_and_cache(out, q, k, v, kp, vp, torch.arange(T, dtype=torch.int32, device="cuda"), slots,
                             inv[:R // 2].contiguous(), err_flag=err)
        assert int(err.item()) == B.PA_DEVERR_BAD_SLOT
        assert pa.pa_status_from_device_flag(int(err.item())) == B.PA_ERR_BAD_SLOT
        rows = vp.view(-1, Hkv, D)
        assert torch.equal(rows[0], v[0]) and torch.equal(rows[5], v[3])
        assert int((rows != 0).any(-1).sum()) == 2
        assert bool(torch.isfinite(out).all())


@pytest.mark.gpu
def test_rope_binding_refusals():
    q = torch.zeros(3, 4, 64, device="cuda")
    k = torch.zeros(3, 2, 64, device="cuda")
    kp = torch.zeros(2, 16, 2, 64, device="cuda")
    pos, slots = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.arange(3, device="cuda")
    inv = torch.ones(32, dtype=torch.float64, device="cuda")
    ok = [q.clone(), q, k, k, kp, kp.clone(), pos, slots, inv]
    pa.pa_rope_and_cache(*ok)
    for i, bad in [(1, q.bfloat16()), (1, q.transpose(0, 1)), (2, k[:2]), (4, kp[:, :8]), (6, pos.long()),
                   (6, pos[:2]), (7, slots.int()), (8, inv.float()), (0, q.cpu()), (8, inv.cpu())]:
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            pa.pa_rope_and_cache(*args)
