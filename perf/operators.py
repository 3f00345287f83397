"""Measured cases of the serving-step operators around the paged KV cache.

Four operators, in the order a step uses them:
  extend   block tables, positions and slot maps of a step built on the GPU
           from request lengths, the new blocks taken from a free ring;
  rotary   rotary positions (one or several axes) of q and k fused with the
           KV write into 16/32-bit, fp8 or per-block-scaled fp8 pools;
  chunk    causal attention of chunks of new tokens over fp8 pools, with an
           optional sliding window;
  release  the blocks of finished requests returned to the free ring.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of the GQA-72B-shape batch: one token per request
        dict(name="extend decode S128", op="extend", seqs=128, ctx_lo=1024, ctx_hi=8192, new_lo=1,
             new_hi=1, block=16, pad=0),
        # a large mixed step: thousands of requests, prompts and single tokens
        dict(name="extend mixed S8192", op="extend", seqs=8192, ctx_lo=0, ctx_hi=2048, new_lo=0,
             new_hi=256, block=16, pad=500),
        # a few requests of the GQA batch finish
        dict(name="release S128", op="release", seqs=128, ctx_lo=1024, ctx_hi=8192, block=16,
             part=0.25, holes=0),
        # half of a large long-context batch finishes, some with released windows
        dict(name="release S8192 long", op="release", seqs=8192, ctx_lo=1, ctx_hi=32768, block=16,
             part=0.5, holes=1),
        # decode step of the Llama-7B-shape layer
        dict(name="rotary decode llama7b f16", op="rotary", seqs=64, new_lo=1, new_hi=1, hq=32,
             hkv=32, dim=128, rot=128, axes=1, interleaved=False, block=16, dtype="f16",
             pool="same", pad=0),
        # a prefill chunk with image positions (time, height, width), fp8
        # blocks with their own scales
        dict(name="rotary chunk 3 axes fp8 blocks", op="rotary", seqs=8, new_lo=300, new_hi=700,
             hq=64, hkv=8, dim=128, rot=128, axes=3, interleaved=False, block=16, dtype="bf16",
             pool="fp8_blocks", pad=5),
        # a large prompt batch with image positions, 16-bit pools
        dict(name="rotary prompts 3 axes bf16", op="rotary", seqs=32, new_lo=900, new_hi=1148,
             hq=64, hkv=8, dim=128, rot=128, axes=3, interleaved=False, block=16, dtype="bf16",
             pool="same", pad=0),
        # two short requests, three speculative tokens at most: latency
        dict(name="chunk tiny f16 d64", op="chunk", seqs=2, ctx_lo=7, ctx_hi=40, new_lo=1, new_hi=3,
             hq=4, hkv=4, dim=64, block=16, dtype="f16", pool="fp8", window=0),
        # four speculative tokens per request over the GQA-72B-shape batch
        dict(name="chunk 4 tokens gqa72b", op="chunk", seqs=128, ctx_lo=1024, ctx_hi=8192, new_lo=4,
             new_hi=4, hq=64, hkv=8, dim=128, block=16, dtype="bf16", pool="fp8", window=0),
        # prefill chunks of 512 tokens after a cached context
        dict(name="chunk 8x512 gqa72b", op="chunk", seqs=8, ctx_lo=4096, ctx_hi=4096, new_lo=512,
             new_hi=512, hq=64, hkv=8, dim=128, block=16, dtype="bf16", pool="fp8", window=0),
        # prefill chunks over 32k contexts, blocks with their own scales
        dict(name="chunk 4x256 ctx 32768 blocks", op="chunk", seqs=4, ctx_lo=32768, ctx_hi=32768,
             new_lo=256, new_hi=256, hq=32, hkv=8, dim=128, block=32, dtype="f16",
             pool="fp8_blocks", window=0),
        # a mixed batch (single tokens beside chunks) with a sliding window
        dict(name="chunk mixed window 1000", op="chunk", seqs=16, ctx_lo=0, ctx_hi=8192, new_lo=1,
             new_hi=511, hq=64, hkv=8, dim=128, block=64, dtype="bf16", pool="fp8_blocks",
             window=1000),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend", "release", "rotary", "rotary", "chunk", "chunk"])
    block = rng.choice([8, 16, 32, 64, 128])
    if op == "extend":
        lo = rng.choice([0, 1, 1])
        new_hi = max(lo, _log_int(rng, 1, 256))
        return dict(op=op, seqs=_log_int(rng, 1, 8192), ctx_lo=0, ctx_hi=_log_int(rng, 1, 2048),
                    new_lo=lo, new_hi=max(1, new_hi), block=block, pad=rng.choice([0, 1, 77]))
    if op == "release":
        return dict(op=op, seqs=_log_int(rng, 1, 8000), ctx_lo=1, ctx_hi=_log_int(rng, 10, 32768),
                    block=max(16, block), part=round(rng.uniform(0.1, 0.5), 3),
                    holes=rng.choice([0, 1]))
    dtype = rng.choice(["bf16", "f16"])
    pool = rng.choice(["fp8", "fp8_blocks"])
    hkv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128])
    group = rng.choice([1, 2, 4, 8])
    if op == "rotary":
        tokens = _log_int(rng, 1, 10000)
        seqs = min(tokens, rng.choice([1, 3, 8, 32, 100]))
        per = tokens // seqs
        return dict(op=op, seqs=seqs, new_lo=max(1, per // 2), new_hi=max(1, per + per // 2),
                    hq=hkv * group, hkv=hkv, dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                    axes=rng.choice([1, 2, 3, 4]), interleaved=rng.choice([False, True]),
                    block=block, dtype=rng.choice([dtype, dtype, "f32"]),
                    pool=rng.choice([pool, "same"]), pad=rng.choice([0, 1, 9]))
    new_hi = _log_int(rng, 1, 512)
    ctx_hi = _log_int(rng, 1, 8192)
    # the padded plain form's products stay within the largest listed case's
    seqs = max(1, min(_log_int(rng, 1, 64), (1 << 24) // ((new_hi + 8) * (ctx_hi + new_hi))))
    return dict(op=op, seqs=seqs, ctx_lo=0, ctx_hi=ctx_hi, new_lo=rng.choice([1, max(1, new_hi // 2)]),
                new_hi=new_hi, hq=hkv * group, hkv=hkv, dim=dim, block=block, dtype=dtype,
                pool=pool, window=rng.choice([0, 0, _log_int(rng, 1, 2000)]))


# ---------------------------------------------------------------------------
# lengths: from the case's own values, so that work() knows them
# ---------------------------------------------------------------------------
def _lengths(case):
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    S = case["seqs"]
    ctx = np.array([r.randint(case.get("ctx_lo", 0), case.get("ctx_hi", 200)) for _ in range(S)],
                   dtype=np.int64)
    new = np.array([r.randint(case.get("new_lo", 0), case.get("new_hi", 0)) for _ in range(S)],
                   dtype=np.int64)
    flag = np.array([r.random() < case.get("part", 0.0) for _ in range(S)])
    if case["op"] == "release" and not flag.any():
        flag[r.randrange(S)] = True
    return ctx, new, flag


def _ceil(a, b):
    return -(-a // b)


def _rows_table(nblk, cols, perm):
    """int32 [S, cols] table: row r holds its nblk[r] next ids of perm, -1 behind."""
    start = torch.cumsum(nblk, 0) - nblk
    j = torch.arange(cols, device=DEV)
    idx = (start[:, None] + j[None]).clamp(max=max(0, perm.numel() - 1))
    return torch.where(j[None] < nblk[:, None], perm[idx], -1).to(torch.int32)


def _randn(shape, dtype, gen):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    step = max(1, (1 << 26) // max(1, out[0].numel()))
    for i in range(0, shape[0], step):
        out[i:i + step] = torch.randn(out[i:i + step].shape, generator=gen, device=DEV)
    return out


def _fp8(shape, gen):
    """E4M3 codes (uint8) of N(0, 1) values times 16, as a quantising write leaves them."""
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 26) // max(1, out[0].numel()))
    for i in range(0, shape[0], step):
        x = torch.randn(out[i:i + step].shape, generator=gen, device=DEV) * 16.0
        out[i:i + step] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


# ---------------------------------------------------------------------------
# prepare
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    return globals()["_prepare_" + case["op"]](case, gen)


def _prepare_extend(case, gen):
    ctx, new, _ = _lengths(case)
    B = case["block"]
    held, total = _ceil(ctx, B), _ceil(ctx + new, B)
    cols = int(total.max()) + 1
    taken = int((total - held).sum())
    NB = int(total.sum()) + 64
    perm = torch.randperm(NB, generator=gen, device=DEV)
    nheld = int(held.sum())
    # a full-size ring whose head has moved on: it wraps
    ring = torch.full((NB,), -1, dtype=torch.int32, device=DEV)
    head = NB - min(NB, taken) // 2
    free = perm[nheld:].to(torch.int32)
    ring[(head + torch.arange(free.numel(), device=DEV)) % NB] = free
    tables = _rows_table(torch.from_numpy(held).to(DEV), cols, perm)
    T = int(new.sum()) + case["pad"]
    S = case["seqs"]
    i32, i64 = torch.int32, torch.int64
    return dict(op="extend", B=B, NB=NB, T=T, ctx=torch.from_numpy(ctx).to(DEV, i32),
                new=torch.from_numpy(new).to(DEV, i32), tables=tables, ring=ring,
                state=torch.tensor([head, head + free.numel()], dtype=i64, device=DEV),
                state_out=torch.empty(2, dtype=i64, device=DEV),
                qsl=torch.empty(S + 1, dtype=i32, device=DEV),
                bsl=torch.empty(S + 1, dtype=i32, device=DEV),
                lens=torch.empty(S, dtype=i32, device=DEV),
                pos=torch.empty(T, dtype=i64, device=DEV),
                slots=torch.empty(T, dtype=i64, device=DEV))


def _prepare_release(case, gen):
    ctx, _, flag = _lengths(case)
    B, S = case["block"], case["seqs"]
    held = _ceil(ctx, B)
    NB = int(held.sum()) + 64
    perm = torch.randperm(NB, generator=gen, device=DEV)
    tables = _rows_table(torch.from_numpy(held).to(DEV), int(held.max()) + 1, perm)
    if case["holes"]:  # every third request has released the blocks before a window
        cut = torch.from_numpy(np.where(np.arange(S) % 3 == 0, held // 2, 0)).to(DEV)
        tables[torch.arange(tables.shape[1], device=DEV)[None] < cut[:, None]] = -1
    ring = torch.full((NB,), -1, dtype=torch.int32, device=DEV)
    free = perm[int(held.sum()):].to(torch.int32)
    head = NB - 7
    ring[(head + torch.arange(free.numel(), device=DEV)) % NB] = free
    i32, i64 = torch.int32, torch.int64
    return dict(op="release", B=B, NB=NB, tables=tables, ring=ring,
                fin=torch.from_numpy(flag).to(DEV, torch.uint8),
                lens=torch.from_numpy(ctx).to(DEV, i32),
                state=torch.tensor([head, head + free.numel()], dtype=i64, device=DEV),
                state_out=torch.empty(2, dtype=i64, device=DEV),
                rsl=torch.empty(S + 1, dtype=i32, device=DEV),
                lens_out=torch.empty(S, dtype=i32, device=DEV))


def _prepare_rotary(case, gen):
    ctx, new, _ = _lengths(case)
    B, Hq, Hkv, D = case["block"], case["hq"], case["hkv"], case["dim"]
    nblk = torch.from_numpy(_ceil(ctx + new, B)).to(DEV)
    NB = int(nblk.sum()) + 3
    perm = torch.randperm(NB, generator=gen, device=DEV)
    tables = _rows_table(nblk, int(nblk.max()), perm).long()
    qsl = np.concatenate([[0], np.cumsum(new)])
    req = torch.from_numpy(np.repeat(np.arange(len(new)), new)).to(DEV)
    pos = torch.from_numpy(np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, new)])).to(DEV)
    slots = tables[req, pos // B] * B + pos % B
    pad = case["pad"]
    T = int(qsl[-1]) + pad
    slots = torch.cat([slots, torch.full((pad,), -1, dtype=torch.int64, device=DEV)])
    pos = torch.cat([pos, torch.zeros(pad, dtype=torch.int64, device=DEV)])
    # axis 0 the text position, the others grid positions of images
    positions = torch.stack([pos] + [torch.randint(0, 1 << (6 + 4 * a), (T,), generator=gen, device=DEV)
                                     for a in range(1, case["axes"])])
    half = case["rot"] // 2
    inv = 1.0 / (10000.0 ** (torch.arange(half, dtype=torch.float64, device=DEV) / half))
    axis = (torch.arange(half, device=DEV) * case["axes"] // half).to(torch.int32)
    dt = DT[case["dtype"]]
    qkv = _randn((T, (Hq + 2 * Hkv) * D), dt, gen)  # one fused projection
    q = qkv[:, :Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    v = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    s = dict(op="rotary", B=B, q=q, k=k, v=v, positions=positions, inv=inv, axis=axis,
             slots=slots, interleaved=case["interleaved"], pool=case["pool"],
             q_out=torch.empty(T, Hq, D, dtype=dt, device=DEV))
    pdt = dt if case["pool"] == "same" else torch.uint8
    s["kc"] = torch.zeros(NB, Hkv, B, D, dtype=pdt, device=DEV)
    s["vc"] = torch.zeros(NB, Hkv, B, D, dtype=pdt, device=DEV)
    if case["pool"] == "fp8":
        s["ks"], s["vs"] = 1 / 32, 1 / 24
    if case["pool"] == "fp8_blocks":
        s["ks"] = torch.full((NB, Hkv), 2.0 ** -5, device=DEV)
        s["vs"] = torch.full((NB, Hkv), 2.0 ** -4, device=DEV)
    return s


def _prepare_chunk(case, gen):
    ctx, new, _ = _lengths(case)
    B, Hq, Hkv, D = case["block"], case["hq"], case["hkv"], case["dim"]
    lens = ctx + new
    nblk = torch.from_numpy(_ceil(lens, B)).to(DEV)
    NB = int(nblk.sum()) + 3
    perm = torch.randperm(NB, generator=gen, device=DEV)
    tables = _rows_table(nblk, int(nblk.max()), perm)
    if case["window"]:  # blocks wholly before the first new token's window are released
        gone = torch.from_numpy(np.maximum(0, ctx + 1 - case["window"]) // B).to(DEV)
        tables[torch.arange(tables.shape[1], device=DEV)[None] < gone[:, None]] = -1
    T = int(new.sum())
    s = dict(op="chunk", B=B, Hkv=Hkv, scale=D ** -0.5, window=case["window"], pool=case["pool"],
             q=_randn((T, Hq, D), DT[case["dtype"]], gen), tables=tables,
             kc=_fp8((NB, Hkv, B, D), gen), vc=_fp8((NB, Hkv, B, D), gen),
             qsl=torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).to(DEV, torch.int32),
             lens=torch.from_numpy(lens).to(DEV, torch.int32), max_q=int(new.max()),
             max_len=int(lens.max()), out=torch.empty(T, Hq, D, dtype=DT[case["dtype"]], device=DEV),
             workspace=None)
    if case["pool"] == "fp8":
        s["ks"], s["vs"] = 1 / 16, 1 / 16
    else:  # power-of-two scales around 1/16, as blocks of different magnitude have
        for n in ("ks", "vs"):
            e = torch.randint(-6, -2, (NB, Hkv), generator=gen, device=DEV)
            s[n] = torch.exp2(e.float())
    return s


# ---------------------------------------------------------------------------
# run: the framework's operators, or their plain forms
# ---------------------------------------------------------------------------
def run(s):
    return globals()[("_own_" if own else "_plain_") + s["op"]](s)


def _own_extend(s):
    import paged_kv_cache_123_gb300 as pa
    pa.pa_extend_block_tables(s["ctx"], s["new"], s["tables"], s["B"], s["ring"], s["state"],
                              s["NB"], s["T"], ring_state_out=s["state_out"],
                              query_start_loc=s["qsl"], block_start_loc=s["bsl"],
                              seq_lens=s["lens"], positions=s["pos"], slot_mapping=s["slots"])
    return dict(tables=s["tables"], qsl=s["qsl"], bsl=s["bsl"], lens=s["lens"], pos=s["pos"],
                slots=s["slots"], state=s["state_out"])


def _plain_extend(s):
    ctx, new, B = s["ctx"].long(), s["new"].long(), s["B"]
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    qsl = torch.cat([zero, torch.cumsum(new, 0)])
    first = (ctx + B - 1) // B
    blocks = (ctx + new + B - 1) // B - first
    bsl = torch.cat([zero, torch.cumsum(blocks, 0)])
    t = torch.arange(s["T"], device=DEV)
    live = t < qsl[-1]
    r = (torch.searchsorted(qsl, t, right=True) - 1).clamp(max=ctx.numel() - 1)
    pos = torch.where(live, ctx[r] + t - qsl[r], 0)
    lb = pos // B
    fresh = lb >= first[r]
    at = (s["state"][0] + bsl[r] + lb - first[r]) % s["ring"].numel()
    blk = torch.where(fresh, s["ring"][at], s["tables"][r, lb]).long()
    opens = live & fresh & (pos % B == 0)
    s["tables"][r[opens], lb[opens]] = blk[opens].to(torch.int32)
    slots = torch.where(live, blk * B + pos % B, -1)
    state = s["state"] + torch.cat([bsl[-1:], zero])
    return dict(tables=s["tables"], qsl=qsl.to(torch.int32), bsl=bsl.to(torch.int32),
                lens=(ctx + new).to(torch.int32), pos=pos, slots=slots, state=state)


def _own_release(s):
    import paged_kv_cache_123_gb300 as pa
    pa.pa_release_block_tables(s["fin"], s["lens"], s["tables"], s["B"], s["ring"], s["state"],
                               s["NB"], ring_state_out=s["state_out"], release_start_loc=s["rsl"],
                               seq_lens_out=s["lens_out"])
    return dict(ring=s["ring"], rsl=s["rsl"], lens=s["lens_out"], state=s["state_out"])


def _plain_release(s):
    fin, lens, B = s["fin"] != 0, s["lens"].long(), s["B"]
    held = torch.where(fin, (lens + B - 1) // B, 0)
    j = torch.arange(s["tables"].shape[1], device=DEV)
    out = (j[None] < held[:, None]) & (s["tables"] >= 0)
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    rsl = torch.cat([zero, torch.cumsum(out.sum(1), 0)])
    ids = s["tables"][out]
    s["ring"][(s["state"][1] + torch.arange(ids.numel(), device=DEV)) % s["ring"].numel()] = ids
    return dict(ring=s["ring"], rsl=rsl.to(torch.int32),
                lens=torch.where(fin, 0, lens).to(torch.int32),
                state=s["state"] + torch.cat([zero, rsl[-1:]]))


def _own_rotary(s):
    import paged_kv_cache_123_gb300 as pa
    more = dict(axis_of_pair=s["axis"], interleaved=s["interleaved"], q_out=s["q_out"])
    call = {"same": pa.pa_rotary_reshape_and_cache, "fp8": pa.pa_rotary_reshape_and_cache_fp8,
            "fp8_blocks": pa.pa_rotary_reshape_and_cache_fp8_scaled}[s["pool"]]
    scales = () if s["pool"] == "same" else (s["ks"], s["vs"])
    call(s["q"], s["k"], s["v"], s["positions"], s["inv"], s["slots"], s["kc"], s["vc"], *scales,
         **more)
    return _rotary_outputs(s, s["q_out"])


def _rotary_outputs(s, q):
    if s["pool"] == "same":
        return dict(q=q, kc=s["kc"], vc=s["vc"])
    f8 = torch.float8_e4m3fn
    res = dict(q=q, kc=s["kc"].view(f8), vc=s["vc"].view(f8))
    if s["pool"] == "fp8_blocks":
        res.update(ks=s["ks"], vs=s["vs"])
    return res


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] in fp32; cos, sin [T, 1, half]."""
    half = cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _scale_of(amax):
    """2^(ceil(log2(amax)) - 7) kept in [2^-126, 2^127]; 1 for 0."""
    m, e = torch.frexp(amax)
    e = torch.where(m == 0.5, e - 1, e).double() - 7
    return torch.where(amax == 0, 1.0, torch.exp2(e.clamp(-126, 127))).float()


def _plain_rotary(s):
    angle = (s["positions"].double()[s["axis"].long()] * s["inv"][:, None]).t()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _rotate(s["q"].float(), cos, sin, s["interleaved"]).to(s["q"].dtype)
    k, v = _rotate(s["k"].float(), cos, sin, s["interleaved"]), s["v"].float()
    ok = s["slots"] >= 0
    B = s["B"]
    blk, row, k, v = s["slots"][ok] // B, s["slots"][ok] % B, k[ok], v[ok]
    if s["pool"] == "fp8_blocks":
        opened = torch.zeros(s["kc"].shape[0], dtype=torch.bool, device=DEV)
        opened[blk[row == 0]] = True
        for x, sc in ((k, s["ks"]), (v, s["vs"])):
            amax = torch.zeros_like(sc).index_reduce_(0, blk, x.abs().amax(-1), "amax")
            sc.copy_(torch.where(opened[:, None], _scale_of(amax), sc))
        k, v = k / s["ks"][blk][..., None], v / s["vs"][blk][..., None]
    elif s["pool"] == "fp8":
        k, v = k / s["ks"], v / s["vs"]
    for x, cache in ((k, s["kc"]), (v, s["vc"])):
        if s["pool"] != "same":
            x = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[blk, :, row] = x.to(cache.dtype)
    return _rotary_outputs(s, q)


def _own_chunk(s):
    import paged_kv_cache_123_gb300 as pa
    T, Hq, D = s["q"].shape
    more = dict(max_query_len=s["max_q"], max_seq_len=s["max_len"], window=s["window"],
                out=s["out"])
    if s["workspace"] is None:  # scratch that the program keeps
        need = pa.pa_multi_query_fp8_workspace_bytes(T, s["lens"].numel(), Hq, s["Hkv"], D, s["B"],
                                                     s["max_q"], s["max_len"], s["window"])
        s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
    more["workspace"] = s["workspace"]
    if s["pool"] == "fp8":
        return pa.pa_multi_query_attention_fp8(s["q"], s["qsl"], s["kc"], s["vc"], s["tables"],
                                               s["lens"], s["scale"], s["Hkv"], s["ks"], s["vs"],
                                               **more)
    return pa.pa_multi_query_attention_fp8_scaled(s["q"], s["qsl"], s["kc"], s["vc"], s["ks"],
                                                  s["vs"], s["tables"], s["lens"], s["scale"],
                                                  s["Hkv"], **more)


def _plain_chunk(s):
    q, qsl, lens, B, Hkv = s["q"], s["qsl"].long(), s["lens"].long(), s["B"], s["Hkv"]
    T, Hq, D = q.shape
    S, G, N = lens.numel(), Hq // Hkv, s["max_q"]
    n = qsl[1:] - qsl[:-1]
    i = torch.arange(N, device=DEV)
    rows = (qsl[:-1, None] + i[None]).clamp(max=T - 1)
    live = i[None] < n[:, None]
    qp = q.float()[rows].view(S, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, N * G, D)
    tab = s["tables"].long().clamp(min=0)

    def dense(codes, scale):
        x = codes[tab].view(torch.float8_e4m3fn).float()  # [S, MB, Hkv, B, D]
        x = x * (scale[tab][..., None, None] if torch.is_tensor(scale) else scale)
        return x.transpose(1, 2).reshape(S, Hkv, -1, D)

    x = torch.matmul(qp, dense(s["kc"], s["ks"]).transpose(2, 3)) * s["scale"]
    pos = (lens - n)[:, None] + i[None]
    j = torch.arange(x.shape[-1], device=DEV)
    see = (j <= pos[..., None]) & (j < lens[:, None, None])
    if s["window"]:
        see &= j > pos[..., None] - s["window"]
    see = see[:, None, :, None].expand(S, 1, N, G, j.numel()).reshape(S, 1, N * G, j.numel())
    x = torch.where(see, x, float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.matmul(p, dense(s["vc"], s["vs"])) / p.sum(-1, keepdim=True)
    o = o.view(S, Hkv, N, G, D).permute(0, 2, 1, 3, 4).reshape(S, N, Hq, D)
    out = torch.empty_like(q)
    out[rows[live]] = o[live].to(q.dtype)
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    ctx, new, flag = _lengths(case)
    B, S = case["block"], case["seqs"]
    if case["op"] == "extend":
        T = int(new.sum()) + case["pad"]
        blocks = int((_ceil(ctx + new, B) - _ceil(ctx, B)).sum())
        return {"bytes": 8 * S + 12 * S + 8 * blocks + 16 * T, "flops": 0}
    if case["op"] == "release":
        held = _ceil(ctx, B)[flag].sum()
        return {"bytes": int(5 * S + 8 * S + 8 * held), "flops": 0}
    Hq, Hkv, D = case["hq"], case["hkv"], case["dim"]
    e = DT[case["dtype"]].itemsize
    if case["op"] == "rotary":
        T = int(new.sum())
        pe = e if case["pool"] == "same" else 1
        return {"bytes": T * (2 * Hq * D * e + 2 * Hkv * D * (e + pe) + 8 * case["axes"] + 8),
                "flops": 3 * T * (Hq + Hkv) * case["rot"]}
    lo = np.maximum(0, ctx + 1 - case["window"]) if case["window"] else np.zeros_like(ctx)
    keys = int((ctx + new - lo).sum())
    pairs = 0
    for c, n in zip(ctx.tolist(), new.tolist()):
        full = c + 1 + np.arange(n)
        pairs += int((np.minimum(full, case["window"]) if case["window"] else full).sum())
    scales = 8 * (keys // B) * Hkv if case["pool"] == "fp8_blocks" else 0
    return {"bytes": 2 * keys * Hkv * D + 2 * int(new.sum()) * Hq * D * e + 4 * (keys // B) + scales,
            "flops": 4 * D * Hq * pairs}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("extend", "release"):
        return None
    s = prepare(case, seed)
    return _exact_rotary(s) if case["op"] == "rotary" else _exact_chunk(s)


def _exact_rotary(s):
    q64, k64 = s["q"].double().clone(), s["k"].double().clone()
    half = s["inv"].numel()
    for p in range(half):
        ang = s["positions"][int(s["axis"][p])].double() * s["inv"][p]
        c, sn = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        i, j = (2 * p, 2 * p + 1) if s["interleaved"] else (p, p + half)
        for x in (q64, k64):
            a, b = x[:, :, i].clone(), x[:, :, j].clone()
            x[:, :, i] = a * c - b * sn
            x[:, :, j] = a * sn + b * c
    if s["pool"] != "same":  # the stored codes are rounded values, not computed ones
        return dict(q=q64)
    kc, vc = s["kc"].double(), s["vc"].double()
    t = torch.nonzero(s["slots"] >= 0)[:, 0]
    b, r = s["slots"][t] // s["B"], s["slots"][t] % s["B"]
    kc[b, :, r] = k64[t]
    vc[b, :, r] = s["v"][t].double()
    return dict(q=q64, kc=kc, vc=vc)


def _e4m3_values():
    c = np.arange(256)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    return torch.from_numpy(np.where(c & 128, -v, v)).to(DEV)


def _exact_chunk(s):
    val, B, Hkv = _e4m3_values(), s["B"], s["Hkv"]
    T, Hq, D = s["q"].shape
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=DEV)
    qsl, lens = s["qsl"].tolist(), s["lens"].tolist()
    for r, L in enumerate(lens):
        a, n = qsl[r], qsl[r + 1] - qsl[r]
        if n == 0:
            continue
        first = max(0, L - n + 1 - s["window"]) if s["window"] else 0
        j = torch.arange(first, L, device=DEV)
        blk = s["tables"][r].long()[j // B]
        K = val[s["kc"][blk, :, j % B].long()].transpose(0, 1)
        V = val[s["vc"][blk, :, j % B].long()].transpose(0, 1)
        if torch.is_tensor(s["ks"]):
            K = K * s["ks"][blk].double().t()[..., None]
            V = V * s["vs"][blk].double().t()[..., None]
        else:
            K, V = K * float(np.float32(s["ks"])), V * float(np.float32(s["vs"]))
        for h in range(Hkv):
            qh = s["q"][a:a + n, h * G:(h + 1) * G].double()
            x = torch.einsum("igd,jd->igj", qh, K[h]) * s["scale"]
            last = L - n + torch.arange(n, device=DEV)
            bad = j[None] > last[:, None]
            if s["window"]:
                bad |= j[None] <= last[:, None] - s["window"]
            x.masked_fill_(bad[:, None], -math.inf)
            out[a:a + n, h * G:(h + 1) * G] = torch.einsum("igj,jd->igd", torch.softmax(x, -1), V[h])
    return out
