"""Refusals of the step bookkeeping and rotary calls that need no device: bad
sizes, missing and misaligned pointers are answered before any CUDA call, and
the Python entry points refuse tensors they cannot take."""
import os

import pytest
import torch

import paged_kv_cache_123_gb300 as pa

SHAPE, NULL, DTYPE, ALIAS, ALIGN = -2, -1, -3, -7, -8
P = 1 << 20          # an address that is never read: every call below is refused


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_123_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


EXTEND = dict(ctx=P, new=P, S=4, tables=P, stride=8, B=16, NB=10, ring=P, ring_size=10, state=P,
              state_out=P, T=4, qsl=P, bsl=P, lens=P, pos=P, slots=P, stream=None)
RELEASE = dict(fin=P, lens=P, S=4, tables=P, stride=8, B=16, NB=10, ring=P, ring_size=10, state=P,
               state_out=P, rsl=P, lens_out=P, stream=None)
ROTARY = dict(q=P, qs=256, k=P, ks=128, v=P, vs=128, T=3, Hq=2, Hkv=1, D=128, dtype=2, pos=P,
              pos_stride=3, axes=1, inv=P, axis=None, rot=128, inter=0, slots=P, q_out=2 * P,
              qos=256, kc=P, vc=P, NB=4, B=16)


@pytest.mark.parametrize("change,status", [
    (dict(S=-1), SHAPE), (dict(S=0x7fffffff), SHAPE), (dict(B=0), SHAPE), (dict(NB=-1), SHAPE),
    (dict(stride=-1), SHAPE), (dict(ring_size=-1), SHAPE), (dict(ring_size=1 << 31), SHAPE),
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(ctx=None), NULL), (dict(new=None), NULL),
    (dict(tables=None), NULL), (dict(ring=None), NULL), (dict(state=None), NULL),
    (dict(state_out=None), NULL), (dict(qsl=None), NULL), (dict(bsl=None), NULL),
    (dict(lens=None), NULL), (dict(pos=None), NULL), (dict(slots=None), NULL),
    (dict(pos=P + 4), ALIGN), (dict(state=P + 4), ALIGN), (dict(ctx=P + 2), ALIGN)])
def test_extend_refusals(lib, change, status):
    assert lib.pa_extend_block_tables(*{**EXTEND, **change}.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(S=-1), SHAPE), (dict(B=-3), SHAPE), (dict(NB=-1), SHAPE), (dict(stride=-1), SHAPE),
    (dict(ring_size=1 << 31), SHAPE), (dict(fin=None), NULL), (dict(lens=None), NULL),
    (dict(tables=None), NULL), (dict(ring=None), NULL), (dict(state=None), NULL),
    (dict(state_out=None), NULL), (dict(rsl=None), NULL), (dict(lens_out=None), NULL),
    (dict(rsl=P + 1), ALIGN), (dict(state_out=P + 4), ALIGN)])
def test_release_refusals(lib, change, status):
    assert lib.pa_release_block_tables(*{**RELEASE, **change}.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=9), DTYPE), (dict(T=-1), SHAPE), (dict(Hq=0), SHAPE), (dict(Hkv=0), SHAPE),
    (dict(D=120), SHAPE), (dict(D=272), SHAPE), (dict(rot=24), SHAPE), (dict(rot=0), SHAPE),
    (dict(rot=144), SHAPE), (dict(axes=0), SHAPE), (dict(axes=9), SHAPE), (dict(B=0), SHAPE),
    (dict(axes=2, pos_stride=2), SHAPE), (dict(qs=248), SHAPE), (dict(ks=120), SHAPE),
    (dict(vs=0), SHAPE), (dict(qos=128), SHAPE), (dict(q=None), NULL), (dict(inv=None), NULL),
    (dict(pos=None), NULL), (dict(slots=None), NULL), (dict(kc=None), NULL),
    (dict(q_out=None), NULL), (dict(q=P + 2), ALIGN), (dict(qs=260), ALIGN), (dict(ks=132), ALIGN),
    (dict(vc=P + 8), ALIGN), (dict(inv=P + 4), ALIGN),
    (dict(q_out=P, qos=512), ALIAS)])
def test_rotary_refusals(lib, change, status):
    args = list({**ROTARY, **change}.values())
    assert lib.pa_rotary_reshape_and_cache(*args, None) == status
    assert lib.pa_rotary_reshape_and_cache_fp8(*args, 1.0, 1.0, None) == status
    assert lib.pa_rotary_reshape_and_cache_fp8_scaled(*args, P, P, None) == status


def test_rotary_scale_refusals(lib):
    args = list(ROTARY.values())
    for ks, vs in ((0.0, 1.0), (1.0, -1.0), (float("nan"), 1.0)):
        assert lib.pa_rotary_reshape_and_cache_fp8(*args, ks, vs, None) == SHAPE
    assert lib.pa_rotary_reshape_and_cache_fp8_scaled(*args, None, P, None) == NULL
    assert lib.pa_rotary_reshape_and_cache_fp8_scaled(*args, P, P + 4, None) == ALIGN


def test_no_tokens_need_no_device(lib):
    args = list({**ROTARY, "T": 0}.values())
    assert lib.pa_rotary_reshape_and_cache(*args, None) == 0


def test_python_entry_points_want_cuda_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    st = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_extend_block_tables(i, i, torch.zeros(4, 2, dtype=torch.int32), 16, i, st, 4, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_release_block_tables(i.bool(), i, torch.zeros(4, 2, dtype=torch.int32), 16, i, st, 4)
    q = torch.zeros(4, 2, 64)
    kc = torch.zeros(2, 1, 16, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_rotary_reshape_and_cache(q, q[:, :1], q[:, :1], st, torch.zeros(32).double(), st, kc,
                                       kc)
    with pytest.raises(ValueError, match="head_size"):
        pa.pa_rotary_reshape_and_cache(q[0], q, q, st, st, st, kc, kc)


CHUNK = dict(q=P, qsl=P, S=2, T=4, kc=P, vc=P, tables=P, stride=8, lens=P, Hq=8, Hkv=2, D=128,
             B=16, NB=10, dtype=2, scale=0.1, k_scale=0.5, v_scale=0.5, window=0, max_q=4,
             max_len=128, partition=0, out=P, ws=None, ws_bytes=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=0), SHAPE), (dict(dtype=7), DTYPE), (dict(S=-1), SHAPE), (dict(T=-1), SHAPE),
    (dict(T=1 << 31), SHAPE), (dict(Hq=6), SHAPE), (dict(Hq=32), SHAPE), (dict(D=96), SHAPE),
    (dict(B=4), SHAPE), (dict(B=24), SHAPE), (dict(B=512), SHAPE), (dict(NB=-1), SHAPE),
    (dict(NB=1 << 31), SHAPE), (dict(NB=0), SHAPE), (dict(window=-1), SHAPE),
    (dict(max_q=-1), SHAPE), (dict(max_len=-1), SHAPE), (dict(partition=-1), SHAPE),
    (dict(k_scale=0.0), SHAPE), (dict(v_scale=float("nan")), SHAPE), (dict(max_len=129), -5),
    (dict(max_len=0x7fffffff, stride=1 << 40), SHAPE),
    (dict(q=None), NULL), (dict(qsl=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL),
    (dict(tables=None), NULL), (dict(lens=None), NULL), (dict(out=None), NULL),
    (dict(q=P + 8), ALIGN), (dict(kc=P + 1), ALIGN), (dict(out=P + 2), ALIGN),
    (dict(qsl=P + 2), ALIGN)])
def test_chunk_refusals(lib, change, status):
    args = {**CHUNK, **change}
    assert lib.pa_multi_query_attention_fp8(*args.values()) == status
    if "k_scale" in change or "v_scale" in change:
        return
    vals = [v for k, v in args.items() if k not in ("k_scale", "v_scale")]
    vals[6:6] = [P, P]
    assert lib.pa_multi_query_attention_fp8_scaled(*vals) == status


def test_chunk_needs_scales_and_nothing_for_no_rows(lib):
    vals = [v for k, v in CHUNK.items() if k not in ("k_scale", "v_scale")]
    assert lib.pa_multi_query_attention_fp8_scaled(*vals[:6], None, P, *vals[6:]) == NULL
    assert lib.pa_multi_query_attention_fp8_scaled(*vals[:6], P, P + 4, *vals[6:]) == ALIGN
    for change in (dict(S=0), dict(T=0), dict(max_q=0)):
        assert lib.pa_multi_query_attention_fp8(*{**CHUNK, **change}.values()) == 0


def test_chunk_workspace_refusals(lib):
    good = [4, 2, 8, 2, 128, 16, 4, 128, 0, 0]
    for at, bad in ((0, -1), (1, -1), (2, 6), (4, 100), (5, 4), (6, -1), (7, -1), (8, -1), (9, -1)):
        args = list(good)
        args[at] = bad
        assert lib.pa_multi_query_fp8_workspace_bytes(*args) == SHAPE, at
