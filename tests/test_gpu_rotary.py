"""Rotary positions fused with the KV write, element by element against the
formula in extended precision, and against the plain KV writes where no pair
turns."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_123_gb300 as pa
from paged_kv_cache_123_gb300 import workloads
from tests.helpers import np_

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = workloads.DTYPES
# Error of a rotated value before its rounding, in units of |a| + |b|: the
# angle's rounding to fp32 half turns (2^-24 pi = 1.9e-7) and its truncation
# to 2^-32 turn (1.5e-9), sincospi (2 ulp of at most 1: 1.2e-7), and two
# fp32 roundings in the product sum (1.2e-7): 4.3e-7.
D_REL = 5e-7


def make(T, hq, hkv, D, rot, axes, B, dtype, seed, far=False, pad=0, fused=True):
    gen = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    if fused:                                         # slices of one projection
        qkv = torch.randn(T, (hq + 2 * hkv) * D, generator=gen).to(dt).to(DEV)
        q = qkv[:, :hq * D].view(T, hq, D)
        k = qkv[:, hq * D:(hq + hkv) * D].view(T, hkv, D)
        v = qkv[:, (hq + hkv) * D:].view(T, hkv, D)
    else:
        q, k, v = (torch.randn(T, h, D, generator=gen).to(dt).to(DEV) for h in (hq, hkv, hkv))
    hi = 1 << 31 if far else 1 << 15
    pos = torch.randint(-hi if far else 0, hi, (axes, T), generator=gen)
    half = rot // 2
    inv = 1.0 / (10000.0 ** (torch.arange(half, dtype=torch.float64) / half))
    axis = torch.randint(0, axes, (half,), generator=gen, dtype=torch.int32)
    NB = -(-T // B) + 3
    slots = torch.randperm(NB * B, generator=gen)[:T]
    slots[torch.randperm(T, generator=gen)[:pad]] = -1
    return dict(q=q, k=k, v=v, pos=pos, inv=inv, axis=axis, slots=slots, NB=NB, B=B, D=D, hkv=hkv,
                dtype=dtype)


def formula(x, c, interleaved):
    """Rotated x [T, H, D] in float64 and the scale of its error, |a| + |b|."""
    x64 = torch.from_numpy(oracle.upcast(np_(x), c["dtype"])).numpy()
    half = c["inv"].numel()
    p = c["pos"].numpy()[c["axis"].numpy()].T.astype(np.longdouble)       # [T, half]
    ang = p * c["inv"].numpy().astype(np.longdouble)[None]
    cos, sin = np.cos(ang).astype(np.float64)[:, None], np.sin(ang).astype(np.float64)[:, None]
    y, mag = x64.copy(), np.zeros_like(x64)
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x64[..., ia], x64[..., ib]
    y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


def close(got, want, mag, dtype):
    """One rounding to the stored type after an error of D_REL * mag."""
    got = oracle.upcast(np_(got), dtype)
    half_step = torch.finfo(DT[dtype]).eps / 2
    tiny = 2.0 ** -25 if dtype == "f16" else 0.0
    d = D_REL * mag
    bad = np.abs(got - want) > half_step * (np.abs(want) + d) + d + tiny
    assert not bad.any(), (np.abs(got - want) * bad).max()


def dev(c):
    return {k: c[k].to(DEV) for k in ("pos", "inv", "axis", "slots")}


def run(c, interleaved, kc, vc, *scales, q_out=None):
    g = dev(c)
    call = {0: pa.pa_rotary_reshape_and_cache, 2: pa.pa_rotary_reshape_and_cache_fp8}[len(scales)]
    if scales and torch.is_tensor(scales[0]):
        call = pa.pa_rotary_reshape_and_cache_fp8_scaled
    return call(c["q"], c["k"], c["v"], g["pos"], g["inv"], g["slots"], kc, vc, *scales,
                axis_of_pair=g["axis"], interleaved=interleaved, q_out=q_out)


def gather(cache, slots, B):
    """Rows [n, Hkv, D] of the pool at slots."""
    s = slots.to(cache.device)
    return cache[s // B, :, s % B]


CASES = [("bf16", 1, 4, 1, 64, 64, 1, 16), ("f16", 5, 32, 32, 128, 128, 1, 16),
         ("f32", 130, 6, 2, 64, 32, 2, 4), ("bf16", 1031, 8, 8, 128, 64, 3, 8),
         ("f16", 3000, 16, 2, 128, 128, 4, 64), ("f32", 40, 3, 1, 256, 256, 1, 1),
         ("bf16", 77, 2, 1, 80, 48, 3, 16), ("bf16", 2000, 1, 1, 16, 16, 2, 7),
         ("f16", 9, 5, 5, 96, 96, 8, 32)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("dtype,T,hq,hkv,D,rot,axes,B", CASES)
def test_matches_the_formula(dtype, T, hq, hkv, D, rot, axes, B, far, interleaved):
    c = make(T, hq, hkv, D, rot, axes, B, dtype, 7 * T + D + rot, far=far, pad=min(2, T - 1),
             fused=T % 2 == 1)
    kc = torch.full((c["NB"], hkv, B, D), 7.0, dtype=DT[dtype], device=DEV)
    vc = kc.clone()
    q = run(c, interleaved, kc, vc)
    yq, mq = formula(c["q"], c, interleaved)
    yk, mk = formula(c["k"], c, interleaved)
    close(q, yq, mq, dtype)
    ok = c["slots"] >= 0
    close(gather(kc, c["slots"][ok], B), yk[ok.numpy()], mk[ok.numpy()], dtype)
    assert torch.equal(gather(vc, c["slots"][ok], B), c["v"][ok.to(DEV)])
    untouched = torch.ones(c["NB"] * B, dtype=torch.bool)
    untouched[c["slots"][ok]] = False
    for cache in (kc, vc):
        assert (cache.transpose(1, 2).reshape(c["NB"] * B, -1)[untouched.to(DEV)] == 7.0).all()
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype,T,hq,hkv,D,rot,axes,B", CASES)
def test_fp8_pool_quantises_the_rotated_value_once(dtype, T, hq, hkv, D, rot, axes, B):
    c = make(T, hq, hkv, D, rot, axes, B, dtype, 11 * T + D)
    kc = torch.zeros(c["NB"], hkv, B, D, dtype=torch.uint8, device=DEV)
    vc, ko, vo = kc.clone(), kc.clone(), kc.clone()
    ks, vs = 0.031, 0.02
    run(c, False, kc, vc, ks, vs)
    y, mag = formula(c["k"], c, False)
    got = oracle.e4m3_decode(np_(gather(kc, c["slots"], B)))
    w = np.clip(y / np.float64(np.float32(ks)), -448, 448)
    # half a step of E4M3 (2^-4 relative, 2^-10 below 2^-6), after the error
    # of the value and of the fp32 division (2^-24 relative)
    d = D_REL * mag / ks + 2.0 ** -24 * np.abs(w)
    assert (np.abs(got - w) <= np.maximum(2.0 ** -4 * (np.abs(w) + d), 2.0 ** -10) + d).all()
    pa.pa_reshape_and_cache_fp8(c["k"].contiguous(), c["v"].contiguous(), dev(c)["slots"], ko, vo,
                                ks, vs)
    assert torch.equal(vc, vo)


def run_batch(counts, hkv, B, dtype, seed):
    """Requests whose tokens continue half-filled blocks and open new ones."""
    gen = torch.Generator().manual_seed(seed)
    T = sum(n for _, n in counts)
    c = make(T, 2 * hkv, hkv, 128, 128, 3, B, dtype, seed)
    nblk = [-(-(a + n) // B) for a, n in counts]
    c["NB"] = sum(nblk) + 2
    perm = torch.randperm(c["NB"], generator=gen)
    slots, off = [], 0
    for (a, n), k in zip(counts, nblk):
        p = torch.arange(a, a + n)
        slots.append(perm[off:off + k][p // B] * B + p % B)
        off += k
    c["slots"] = torch.cat(slots)
    return c


def test_block_scales_with_many_heads_and_odd_blocks():
    """More KV heads than a CTA's warps take at once, one-token blocks, a
    block longer than a round of tokens, pairs next to each other."""
    for hkv, D, B, dtype, inter in ((70, 16, 1, "bf16", False), (9, 256, 48, "f32", True),
                                    (3, 96, 256, "f16", False)):
        gen = torch.Generator().manual_seed(B)
        T = 61
        c = make(T, hkv, hkv, D, D, 2, B, dtype, 40 + B)
        nb = -(-T // B)
        perm = torch.randperm(nb + 2, generator=gen)
        c["NB"] = nb + 2
        c["slots"] = perm[:nb][torch.arange(T) // B] * B + torch.arange(T) % B
        kc = torch.zeros(c["NB"], hkv, B, D, dtype=torch.uint8, device=DEV)
        vc, ks = kc.clone(), torch.full((c["NB"], hkv), 3.0, device=DEV)
        vs = ks.clone()
        run(c, inter, kc, vc, ks, vs)
        y, _ = formula(c["k"], c, inter)
        v = oracle.upcast(np_(c["v"]), dtype)
        blk = (c["slots"] // B).numpy()
        for b in range(c["NB"]):
            for h in range(hkv):
                if not (blk == b).any():
                    assert float(ks[b, h]) == 3.0
                    continue
                amax = np.abs(y[blk == b, h]).max()
                near = [oracle.block_scale_e4m3(amax * f) for f in (1 - 2e-6, 1, 1 + 2e-6)]
                assert float(ks[b, h]) in near
                assert float(vs[b, h]) == oracle.block_scale_e4m3(np.abs(v[blk == b, h]).max())
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B", [4, 16, 64])
def test_block_scales_come_from_the_rotated_values(dtype, B):
    c = run_batch([(0, 40), (5, 1), (16, 1), (15, 3), (130, 100), (64, 64)], 2, B, dtype, 3 + B)
    kc = torch.zeros(c["NB"], 2, B, 128, dtype=torch.uint8, device=DEV)
    vc = kc.clone()
    ks = torch.full((c["NB"], 2), 2.0 ** -5, device=DEV)
    vs = torch.full((c["NB"], 2), 2.0 ** -4, device=DEV)
    run(c, False, kc, vc, ks, vs)
    y, mag = formula(c["k"], c, False)
    s = c["slots"].numpy()
    opened = set((s[s % B == 0] // B).tolist())
    for b in range(c["NB"]):
        t = np.nonzero(s // B == b)[0]
        for h in range(2):
            got = float(ks[b, h])
            if b not in opened:
                assert got == 2.0 ** -5 and float(vs[b, h]) == 2.0 ** -4
                continue
            amax = np.abs(y[t, h]).max()
            near = [oracle.block_scale_e4m3(amax * f) for f in (1 - 2e-6, 1, 1 + 2e-6)]
            assert got in near, (got, near)
            assert float(vs[b, h]) == oracle.block_scale_e4m3(
                np.abs(oracle.upcast(np_(c["v"][t.tolist(), h]), dtype)).max())
    sc = ks.cpu().numpy()[s // B].astype(np.float64)[..., None]
    got = oracle.e4m3_decode(np_(gather(kc, c["slots"], B)))
    w = np.clip(y / sc, -448, 448)
    d = D_REL * mag / sc + 2.0 ** -24 * np.abs(w)
    assert (np.abs(got - w) <= np.maximum(2.0 ** -4 * (np.abs(w) + d), 2.0 ** -10) + d).all()
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("pool", ["same", "fp8", "blocks"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_position_zero_is_the_plain_write(dtype, pool):
    """cos 0 = 1 and sin 0 = 0 exactly: the pools must equal the plain
    write's bit for bit, and q passes."""
    c = run_batch([(0, 33), (3, 7), (16, 20)], 2, 16, dtype, 77)
    c["pos"].zero_()
    pdt = DT[dtype] if pool == "same" else torch.uint8
    pools = [torch.zeros(c["NB"], 2, 16, 128, dtype=pdt, device=DEV) for _ in range(4)]
    scales = [torch.full((c["NB"], 2), 0.125, device=DEV) for _ in range(4)]
    k, v, slots = c["k"].contiguous(), c["v"].contiguous(), c["slots"].to(DEV)
    if pool == "same":
        q = run(c, True, pools[0], pools[1])
        pa.pa_reshape_and_cache(k, v, slots, pools[2], pools[3])
    elif pool == "fp8":
        q = run(c, True, pools[0], pools[1], 0.05, 0.07)
        pa.pa_reshape_and_cache_fp8(k, v, slots, pools[2], pools[3], 0.05, 0.07)
    else:
        q = run(c, True, pools[0], pools[1], scales[0], scales[1])
        pa.pa_reshape_and_cache_fp8_scaled(k, v, slots, pools[2], pools[3], scales[2], scales[3])
        assert torch.equal(scales[0], scales[2]) and torch.equal(scales[1], scales[3])
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    assert torch.equal(q, c["q"])


def test_in_place_on_a_slice_of_the_projection():
    c = make(300, 8, 2, 128, 64, 1, 16, "bf16", 5)
    kc = torch.zeros(c["NB"], 2, 16, 128, dtype=torch.bfloat16, device=DEV)
    k0, v0 = c["k"].clone(), c["v"].clone()
    want = run(c, False, kc, kc.clone())
    got = run(c, False, kc, kc.clone(), q_out=c["q"])
    assert got.data_ptr() == c["q"].data_ptr() and torch.equal(got, want)
    assert torch.equal(c["k"], k0) and torch.equal(c["v"], v0)


def test_slots_and_axes_outside_are_reported():
    c = make(20, 2, 1, 64, 64, 2, 16, "f16", 6)
    kc = torch.zeros(c["NB"], 1, 16, 64, dtype=torch.float16, device=DEV)
    vc = kc.clone()
    pa.pa_get_device_error()
    c["slots"][4] = c["NB"] * 16
    run(c, False, kc, vc)
    assert pa.pa_get_device_error() == -5
    ok = torch.arange(20) != 4
    assert torch.equal(gather(vc, c["slots"][ok], 16), c["v"][ok.to(DEV)])
    c["slots"][4] = -1
    c["axis"][3] = 2
    run(c, False, kc, vc)
    assert pa.pa_get_device_error() == -5


def test_no_tokens():
    c = make(1, 2, 1, 64, 64, 1, 16, "f16", 6)
    kc = torch.zeros(2, 1, 16, 64, dtype=torch.float16, device=DEV)
    e = lambda h: torch.empty(0, h, 64, dtype=torch.float16, device=DEV)  # noqa: E731
    i = torch.empty(0, dtype=torch.int64, device=DEV)
    q = pa.pa_rotary_reshape_and_cache(e(2), e(1), e(1), i, c["inv"].to(DEV), i, kc, kc)
    assert q.shape == (0, 2, 64)


def test_python_refusals():
    c = make(4, 2, 1, 64, 64, 1, 16, "bf16", 8)
    g = dev(c)
    kc = torch.zeros(c["NB"], 1, 16, 64, dtype=torch.bfloat16, device=DEV)
    good = [c["q"], c["k"], c["v"], g["pos"], g["inv"], g["slots"], kc, kc]
    bad = [(0, c["q"].transpose(0, 1).contiguous().transpose(0, 1)), (1, c["k"][:2]),
           (2, c["v"].half()), (3, g["pos"].int()), (3, g["pos"][:, :2].contiguous()),
           (4, g["inv"].float()), (5, g["slots"].int()), (6, kc.half()), (7, kc[:1])]
    for i, t in bad:
        with pytest.raises(ValueError):
            pa.pa_rotary_reshape_and_cache(*good[:i], t, *good[i + 1:])
    with pytest.raises(ValueError):
        pa.pa_rotary_reshape_and_cache(*good, axis_of_pair=g["axis"].long())
    with pytest.raises(ValueError):
        pa.pa_rotary_reshape_and_cache_fp8(*good, 1.0, 1.0)      # 16-bit pools
