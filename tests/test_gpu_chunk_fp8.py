"""Chunks of new tokens over fp8 pools (one scale per pool, or per block),
with and without a sliding window, element by element against the definition
in 64 bits.

Tolerance of an output o = sum_j w_j V_j (weights w_j normalised), derived
from the kernel's roundings:
  * a weight is rounded once to fp16: half a step, 2^-11 relative, or half
    the smallest subnormal, 2^-25 of a value whose largest in the row is at
    least 1: A * 2^-11 + n * 2^-25 * Vmax, with A = sum_j w_j |V_j|;
  * a logit's error dx moves its weight by dx relatively (and the sum by at
    most as much): 2 A dx, with dx <= 2^-20 * max_j sum_d |scale q_d K_jd|
    (fp32 accumulation of up to 128 products and the fp32 exponent
    arithmetic: at most 16 roundings of 2^-24 of the partial sums) + 2^-20;
  * the products P V accumulate in fp32: A * 2^-20;
  * the output's own rounding: eps / 2.
"""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_123_gb300 as pa
from paged_kv_cache_123_gb300 import workloads
from tests.helpers import np_

pytestmark = pytest.mark.gpu
DEV = "cuda"
POOLS = ("pool", "blocks")


def make(dtype, D, hq, hkv, B, ctx, n_new, pool, seed, window=0, junk=True, scale=None):
    """Scattered blocks; rows that belong to no sequence hold NaN codes."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    lens = [c + n for c, n in zip(ctx, n_new)]
    nblk = [-(-L // B) for L in lens]
    NB = sum(nblk) + 3
    perm = rng.permutation(NB)
    tables = np.full((len(lens), max(max(nblk), 1) + 1), -1, np.int32)
    off = 0
    for s, k in enumerate(nblk):
        tables[s, :k] = perm[off:off + k]
        off += k

    def codes():
        x = torch.randn(NB, hkv, B, D, generator=gen) * 16
        c = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
        if junk:
            keep = np.zeros((NB, B), bool)
            for s, L in enumerate(lens):
                j = np.arange(L)
                keep[tables[s, j // B], j % B] = True
            c.transpose(0, 2, 1, 3)[~keep] = 0x7f
        return c

    q = torch.randn(sum(n_new), hq, D, generator=gen).to(workloads.DTYPES[dtype])
    c = dict(q=q, kc=codes(), vc=codes(), tables=tables, B=B, hkv=hkv, dtype=dtype,
             qsl=np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32),
             lens=np.array(lens, np.int32), scale=D ** -0.5 if scale is None else scale,
             window=window, max_q=max(n_new), max_len=max(lens), pool=pool)
    if pool == "pool":
        c["ks"], c["vs"] = 1 / 16, 0.07
    else:
        c["ks"] = np.exp2(rng.integers(-7, -1, (NB, hkv))).astype(np.float32)
        c["vs"] = np.exp2(rng.integers(-9, 0, (NB, hkv))).astype(np.float32)
    return c


def reference(c, rows=None):
    """(out, tolerance) in float64; NaN codes only count where they are seen."""
    q = oracle.upcast(np_(c["q"]), c["dtype"])
    T, hq, D = q.shape
    G, B, NB = hq // c["hkv"], c["B"], c["kc"].shape[0]
    out, tol = np.zeros((T, hq, D)), np.zeros((T, hq, D))
    eps = torch.finfo(workloads.DTYPES[c["dtype"]]).eps / 2
    for s, L in enumerate(c["lens"]):
        a, n = int(c["qsl"][s]), int(c["qsl"][s + 1] - c["qsl"][s])
        if n == 0:
            continue
        first = max(0, L - n + 1 - c["window"]) if c["window"] else 0
        j = np.arange(first, L)
        blk = c["tables"][s, j // B].astype(np.int64)
        j, blk = j[(blk >= 0) & (blk < NB)], blk[(blk >= 0) & (blk < NB)]
        for h in range(c["hkv"]):
            K = oracle.e4m3_decode(c["kc"][blk, h, j % B])
            V = oracle.e4m3_decode(c["vc"][blk, h, j % B])
            if c["pool"] == "pool":
                K, V = K * np.float64(np.float32(c["ks"])), V * np.float64(np.float32(c["vs"]))
                top = 448 * c["vs"]
            else:
                K, V = K * c["ks"][blk, h, None], V * c["vs"][blk, h, None]
                top = 448 * c["vs"][blk, h].max(initial=0)
            for i in range(n):
                if rows is not None and a + i not in rows:
                    continue
                p = L - n + i
                see = j <= p
                if c["window"]:
                    see &= j > p - c["window"]
                k, v = K[see], V[see]
                if not len(k):
                    continue
                qi = q[a + i, h * G:(h + 1) * G]
                x = c["scale"] * (qi @ k.T)
                w = np.exp(x - x.max(-1, keepdims=True))
                w /= w.sum(-1, keepdims=True)
                o, A = w @ v, w @ np.abs(v)
                mag = abs(c["scale"]) * (np.abs(qi) @ np.abs(k).T).max(-1, keepdims=True)
                dx = 2.0 ** -20 * (mag + 1)
                t = A * (2.0 ** -11 + 2 * dx + 2.0 ** -20) + len(k) * 2.0 ** -25 * top
                out[a + i, h * G:(h + 1) * G] = o
                tol[a + i, h * G:(h + 1) * G] = t + eps * (np.abs(o) + t) + 2.0 ** -25
    return out, tol


def on_gpu(c):
    g = {k: torch.from_numpy(c[k]).to(DEV) for k in ("kc", "vc", "tables", "qsl", "lens")}
    g["q"] = c["q"].to(DEV)
    for k in ("ks", "vs"):
        g[k] = c[k] if c["pool"] == "pool" else torch.from_numpy(c[k]).to(DEV)
    return g


def call(c, g, **more):
    more = {**dict(max_query_len=c["max_q"], max_seq_len=c["max_len"], window=c["window"]), **more}
    if c["pool"] == "pool":
        return pa.pa_multi_query_attention_fp8(g["q"], g["qsl"], g["kc"], g["vc"], g["tables"],
                                               g["lens"], c["scale"], c["hkv"], g["ks"], g["vs"],
                                               **more)
    return pa.pa_multi_query_attention_fp8_scaled(g["q"], g["qsl"], g["kc"], g["vc"], g["ks"],
                                                  g["vs"], g["tables"], g["lens"], c["scale"],
                                                  c["hkv"], **more)


def close(got, ref, keep=None):
    want, tol = ref
    got = got.double().cpu().numpy()
    if keep is not None:
        got, want, tol = got[keep], want[keep], tol[keep]
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), ((np.abs(got - want) / tol).max(), np.argwhere(bad)[:4])


def check(c, **more):
    g = on_gpu(c)
    out = call(c, g, **more)
    close(out, reference(c))
    assert pa.pa_get_device_error() == 0
    return out


CTX, NEW = [0, 5, 100, 300, 0, 64, 9], [1, 3, 17, 40, 130, 64, 0]
CASES = [(dt, D, G, 16) for dt in ("bf16", "f16") for D in (64, 128) for G in (1, 2, 4, 8)]
CASES += [("bf16", 128, 8, B) for B in (8, 32, 64, 128, 256)]
CASES += [("f16", 64, 1, B) for B in (8, 64, 256)]


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("dtype,D,G,B", CASES)
def test_matches_the_definition(dtype, D, G, B, pool):
    check(make(dtype, D, 2 * G, 2, B, CTX, NEW, pool, 17 * D + 7 * G + B))


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("B,G", [(16, 8), (8, 4), (64, 1), (256, 2)])
@pytest.mark.parametrize("window", [1, 5, 64, 128, 129, 300, 5000])
def test_window_never_looks_behind_it(window, B, G, pool):
    """Blocks that no new token's window reaches are released (-1)."""
    ctx, new = [0, 700, 1000, 257, 128], [200, 33, 1, 90, 128]
    c = make("bf16", 128, G, 1, B, ctx, new, pool, 3 * window + B, window=window)
    for s, (a, n) in enumerate(zip(ctx, new)):
        c["tables"][s, :max(0, a + 1 - window) // B] = -1
    check(c)
    check(c, partition_size=128)


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("partition", [128, 300, 1024])
@pytest.mark.parametrize("dtype,G,n_new", [("bf16", 8, [4, 1, 3, 2]), ("f16", 1, [7, 1, 30, 2]),
                                           ("bf16", 4, [40, 1, 100, 9])])
def test_partitions_meet(partition, dtype, G, n_new, pool):
    c = make(dtype, 128, 2 * G, 2, 16, [900, 0, 2000, 63], n_new, pool, 71)
    need = pa.pa_multi_query_fp8_workspace_bytes(sum(n_new), 4, 2 * G, 2, 128, 16, c["max_q"],
                                                 c["max_len"], 0, partition)
    assert need > 0
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device=DEV)     # NaN everywhere
    check(c, partition_size=partition, workspace=ws)
    with pytest.raises(pa.PagedAttnError) as e:
        call(c, on_gpu(c), partition_size=partition, workspace=ws[:need - 8])
    assert e.value.status == -4


@pytest.mark.parametrize("pool", POOLS)
def test_many_ragged_sequences(pool):
    """Enough CTAs for several waves: sequences are taken by falling length,
    equal lengths and empty ones among them."""
    rng = np.random.default_rng(8)
    ctx = rng.integers(0, 260, 100).tolist()
    ctx[7] = ctx[8] = ctx[90]
    new = rng.integers(1, 4, 100).tolist()
    new[0] = new[55] = 0
    ctx[55] = 0
    check(make("bf16", 64, 4, 2, 16, ctx, new, pool, 91))


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("S", [77, 80, 128, 129])
def test_long_sequences_are_taken_first(S, pool):
    """Up to 128 sequences with more CTAs than SMs and lengths past 2,048 are
    taken by falling length: equal lengths and empty sequences among them, the
    longest ones last in the batch."""
    rng = np.random.default_rng(S)
    ctx = rng.integers(0, 300, S).tolist()
    ctx[-1], ctx[-2], ctx[5] = 2101, 2101, 2200
    ctx[9] = ctx[10] = ctx[60]
    new = rng.integers(1, 4, S).tolist()
    new[0] = new[55] = 0
    ctx[55] = 0
    check(make("bf16", 64, 8, 4, 16, ctx, new, pool, 93))


def test_positions_next_to_the_largest_length():
    """A window at the end of 2^31 - 1,024 tokens, whose earlier blocks are
    released; one partition and several."""
    B, D, w, n, L = 256, 64, 300, 5, 0x7fffffff - 1023
    c = make("bf16", D, 2, 1, B, [600], [n], "blocks", 94, window=w)
    g = on_gpu(c)
    near = c["lens"][0]
    shift = (L - int(near)) // B * B              # the same place in its block
    want = reference(c)
    cols = (int(near) + shift + B - 1) // B
    t = torch.full((1, cols), -1, dtype=torch.int32, device=DEV)
    t[0, shift // B:] = g["tables"][0, :cols - shift // B]
    g["tables"] = t
    g["lens"] = g["lens"] + shift
    for part in (0, 128):
        close(call(c, g, max_seq_len=L - L % B, partition_size=part), want)
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("n", [31, 32, 33, 64])
def test_rows_around_two_tiles(n):
    """255 to 264 rows per KV head: whole pairs of row tiles and one more."""
    check(make("f16", 128, 8, 1, 32, [0, 150, 400], [n, n, 1], "blocks", 300 + n))


def test_block_scales_far_apart():
    """Scales from 2^-12 to 2^12 in one sequence: what a small one loses is
    counted with the reference, the largest scale (half of fp16's smallest
    step, 2^-25, of each code)."""
    c = make("bf16", 128, 8, 1, 16, [500], [40], "blocks", 92)
    rng = np.random.default_rng(3)
    for k in ("ks", "vs"):
        c[k] = np.exp2(rng.integers(-12, 13, c[k].shape)).astype(np.float32)
    c["scale"] = 2.0 ** -12 * 128 ** -0.5
    out = call(c, on_gpu(c)).double().cpu().numpy()
    want, tol = reference(c)
    q = np.abs(oracle.upcast(np_(c["q"]), "bf16")).sum(-1, keepdims=True)
    dx = c["scale"] * q * 2.0 ** -25 * c["ks"].max()
    extra = 2 * dx * 448 * c["vs"].max() + 2.0 ** -25 * c["vs"].max()
    assert (np.abs(out - want) <= tol + extra).all()
    # and it is the large blocks that are right to the usual tolerance
    assert (np.abs(out - want) <= tol + 2.0 ** -20 * np.abs(want).max()).mean() > 0.99


@pytest.mark.parametrize("pool", POOLS)
def test_single_tokens_split_by_themselves_and_agree_with_decode(pool):
    c = make("bf16", 128, 16, 2, 16, [10, 4999, 2000, 0], [1, 1, 1, 1], pool, 31)
    g = on_gpu(c)
    assert pa.pa_multi_query_fp8_workspace_bytes(4, 4, 16, 2, 128, 16, 1, 5000) > 0
    out = check(c)
    more = dict(max_seq_len=c["max_len"])
    if pool == "pool":
        dec = pa.pa_decode_attention_fp8(g["q"], g["kc"], g["vc"], g["tables"], g["lens"],
                                         c["scale"], 2, g["ks"], g["vs"], **more)
    else:
        dec = pa.pa_decode_attention_fp8_scaled(g["q"], g["kc"], g["vc"], g["ks"], g["vs"],
                                                g["tables"], g["lens"], c["scale"], 2, **more)
    # each call is within its own tolerance; decode's weights are fp16 too
    _, tol = reference(c)
    assert (np.abs((out.double() - dec.double()).cpu().numpy()) <= 2 * tol).all()


@pytest.mark.parametrize("n", [1, 3, 5, 7, 15, 16, 17])
def test_partly_filled_row_tiles(n):
    c = make("bf16", 128, 16, 2, 8, [0, 5, 130, 700, 1029], [n] * 5, "blocks", 1200 + 7 * n)
    check(c)


@pytest.mark.parametrize("scale", [0.0, -0.11, 3.0])
def test_scales_of_any_sign(scale):
    check(make("bf16", 64, 4, 2, 16, [40, 200], [9, 50], "pool", 5, scale=scale))
    check(make("f16", 128, 8, 2, 16, [40, 200], [9, 50], "blocks", 6, scale=scale))


def test_large_and_small_queries_keep_their_bits():
    """bf16 rows far outside fp16's range, and rows of mixed magnitude."""
    c = make("bf16", 128, 8, 2, 16, [300], [64], "pool", 9, scale=1.0)
    e = torch.arange(64) % 8
    q = c["q"].float() * torch.exp2(-(e[:, None, None] * 2.0)) * 0.05
    q[..., 1] *= 2.0 ** -9
    c["q"] = q.to(torch.bfloat16)
    base = check(c)
    for shift in (-90, 60):                     # the same problem in another unit
        d = dict(c, q=(c["q"].float() * 2.0 ** shift).to(torch.bfloat16), scale=2.0 ** -shift)
        assert torch.equal(call(d, on_gpu(d)), base)
    z = dict(c, q=torch.zeros_like(c["q"]))
    check(z)


@pytest.mark.parametrize("pool", POOLS)
@pytest.mark.parametrize("window", [0, 70])
def test_nan_codes_reach_exactly_the_rows_that_see_them(pool, window):
    B, ctx, new = 16, [300, 40], [150, 30]
    c = make("bf16", 128, 8, 1, B, ctx, new, pool, 13, window=window)
    at = {0: [2, 310, 333, 449], 1: [3, 69]}    # cached, and among the new tokens
    for s, js in at.items():
        for j in js:
            c["vc"][c["tables"][s, j // B], 0, j % B, (5 * j) % 128] = 0x7f if j % 2 else 0xff
    g = on_gpu(c)
    for part in (0, 128):
        got = call(c, g, partition_size=part).double().cpu().numpy()
        want, tol = reference(c)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert 0 < np.isnan(want).sum() < want.size / 4
        ok = ~np.isnan(want)
        assert (np.abs(got - want)[ok] <= tol[ok]).all()
    # a NaN key: rows that see it are NaN, the others do not notice
    c = make("bf16", 128, 8, 1, B, ctx, new, pool, 14, window=window)
    c["kc"][c["tables"][0, 320 // B], 0, 320 % B, 7] = 0x7f
    got = call(c, on_gpu(c)).double().cpu().numpy()
    want, tol = reference(c)
    rows = np.zeros(len(got), bool)
    rows[20:150 if not window else min(150, 20 + window)] = True
    assert np.isnan(got[rows]).all() and np.isfinite(got[~rows]).all()
    assert (np.abs(got - want)[~rows] <= tol[~rows]).all()


def test_bad_blocks_are_left_out_and_reported():
    c = make("bf16", 128, 8, 1, 16, [200, 30, 100], [20, 4, 3], "pool", 15)
    c["tables"][0, 3], c["tables"][0, 9] = -7, c["kc"].shape[0]
    c["tables"][1, :] = -1                      # nothing left to attend to: zeros
    pa.pa_get_device_error()
    out = call(c, on_gpu(c))
    assert pa.pa_get_device_error() == -5
    close(out, reference(c))
    assert not out[20:24].any()


def test_bad_lengths_leave_their_rows_alone():
    c = make("f16", 64, 4, 4, 16, [0, 8, 20, 30], [4, 4, 6, 2], "blocks", 51)
    c["lens"][0], c["lens"][2] = 2, c["max_len"] + 1     # shorter than its new tokens; too long
    g = on_gpu(c)
    out = torch.full_like(g["q"], 5.0)
    out = torch.cat([out, out[:3]])                      # rows behind the last sequence
    g["q"] = torch.cat([g["q"], g["q"][:3]])
    pa.pa_get_device_error()
    call(c, g, out=out)
    assert pa.pa_get_device_error() == -5
    assert (out[:4] == 5).all() and (out[8:14] == 5).all() and (out[16:] == 5).all()
    want, tol = reference(c)
    got = out.double().cpu().numpy()
    for a, b in ((4, 8), (14, 16)):
        assert (np.abs(got[a:b] - want[a:b]) <= tol[a:b]).all()
    # a row past the query tensor is never touched
    g["qsl"][4] = 25
    call(c, g, out=out, max_query_len=20)
    assert pa.pa_get_device_error() == -5


def test_same_bits_again_and_through_another_table():
    c = make("bf16", 128, 16, 2, 16, [2000, 100], [100, 9], "blocks", 61)
    g = on_gpu(c)
    a = call(c, g)
    assert torch.equal(a, call(c, g))
    NB = c["kc"].shape[0]
    perm = np.random.default_rng(1).permutation(NB)
    d = dict(c, tables=np.where(c["tables"] >= 0, perm[c["tables"]], -1).astype(np.int32))
    inv = np.argsort(perm)
    for k in ("kc", "vc", "ks", "vs"):
        d[k] = c[k][inv]
    assert torch.equal(a, call(d, on_gpu(d)))


def test_captured_and_replayed_with_new_lengths():
    c = make("bf16", 128, 16, 2, 16, [900, 50], [20, 4], "pool", 62)
    g = on_gpu(c)
    more = dict(max_query_len=40, max_seq_len=2000 if g["tables"].shape[1] * 16 >= 2000 else
                g["tables"].shape[1] * 16)
    out = torch.empty_like(g["q"])
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=DEV)
    call(c, g, out=out, workspace=ws, **more)            # set-up outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(c, g, out=out, workspace=ws, **more)
    for lens, qsl in ((c["lens"], c["qsl"]), (np.array([500, 24], np.int32),
                                              np.array([0, 3, 24], np.int32))):
        g["lens"].copy_(torch.from_numpy(lens))
        g["qsl"].copy_(torch.from_numpy(qsl))
        graph.replay()
        close(out, reference(dict(c, lens=lens, qsl=qsl)))


def test_two_streams_at_once():
    cs = [make("bf16", 128, 8, 1, 16, [1500, 3], [5, 60], "pool", s) for s in (1, 2)]
    gs = [on_gpu(c) for c in cs]
    torch.cuda.synchronize()
    outs = []
    for c, g in zip(cs, gs):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            outs.append(call(c, g))
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        close(o, reference(c))


def test_blocks_past_four_gigabytes_of_codes():
    B, hkv, D = 256, 8, 128
    NB = (1 << 32) // (B * hkv * D) + 9
    small = make("bf16", D, 64, hkv, B, [700, 20], [9, 2], "pool", 63)
    n = small["kc"].shape[0]
    g = on_gpu(small)
    for k in ("kc", "vc"):
        big = torch.empty(NB, hkv, B, D, dtype=torch.uint8, device=DEV)
        big[NB - n:] = g[k]
        g[k] = big
    g["tables"] = torch.where(g["tables"] >= 0, g["tables"] + (NB - n), g["tables"])
    close(call(small, g), reference(small))


def test_refusals():
    c = make("bf16", 128, 8, 2, 16, [40], [4], "pool", 64)
    g = on_gpu(c)

    def status(**change):
        with pytest.raises(pa.PagedAttnError) as e:
            call(dict(c, **{k: v for k, v in change.items() if k in c}),
                 {**g, **{k: v for k, v in change.items() if k in g}},
                 **{k: v for k, v in change.items() if k in ("max_query_len", "max_seq_len",
                                                             "partition_size", "window")})
        return e.value.status

    assert status(ks=0.0) == -2 and status(vs=-1.0) == -2
    assert status(partition_size=-1) == -2 and status(max_query_len=-1) == -2
    assert status(max_seq_len=10 ** 6) == -5
    assert status(q=g["q"].float()) == -2
    c2 = make("bf16", 128, 6, 2, 16, [40], [4], "pool", 64)      # group 3
    with pytest.raises(pa.PagedAttnError):
        call(c2, on_gpu(c2))
    c3 = make("bf16", 128, 8, 2, 4, [40], [4], "pool", 64)       # blocks of 4
    with pytest.raises(pa.PagedAttnError):
        call(c3, on_gpu(c3))
    with pytest.raises(ValueError):
        call(c, {**g, "kc": g["kc"].view(torch.int8)})
    with pytest.raises(ValueError):
        call(c, {**g, "q": g["q"].transpose(0, 1)})
    with pytest.raises(ValueError):
        call(c, {**g, "lens": g["lens"].long()})
    with pytest.raises(ValueError):
        call(c, {**g, "tables": g["tables"][:0]})
    b = make("bf16", 128, 8, 2, 16, [40], [4], "blocks", 64)
    gb = on_gpu(b)
    with pytest.raises(ValueError):
        call(b, {**gb, "ks": gb["ks"][:1]})


def test_nothing_to_do():
    c = make("bf16", 128, 8, 2, 16, [40, 3], [4, 1], "pool", 65)
    g = on_gpu(c)
    g["qsl"].zero_()
    out = torch.full_like(g["q"], 3.0)
    call(c, g, out=out)
    assert (out == 3).all()
    e = {**g, "q": g["q"][:0]}
    assert call(c, e).shape == (0, 8, 128)
    assert pa.pa_get_device_error() == 0
