"""Block tables, positions and slot maps built on the GPU from request
lengths, and the release of finished requests, against a sequential host
restatement, the host block pool and the slot-mapping oracle. Everything is
integers: results must be equal."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_123_gb300 as pa

pytestmark = pytest.mark.gpu
DEV = "cuda"
NO_BLOCKS, OUT_OF_RANGE = -11, -5


def ref_extend(ctx, new, tables, B, ring, head, tail, T):
    """One request after the other, as the host pool does it."""
    tables, S = tables.copy(), len(ctx)
    qsl, bsl = np.zeros(S + 1, np.int64), np.zeros(S + 1, np.int64)
    pos, slots = np.zeros(T, np.int64), np.full(T, -1, np.int64)
    t = 0
    for r in range(S):
        n, c = int(new[r]), int(ctx[r])
        if c < 0 or n < 0 or c + n > tables.shape[1] * B:
            n = 0
        k = 0
        for p in range(c, c + n):
            if p % B == 0:
                tables[r, p // B] = ring[head % len(ring)]
                head, k = head + 1, k + 1
            pos[t], slots[t] = p, int(tables[r, p // B]) * B + p % B
            t += 1
        qsl[r + 1], bsl[r + 1] = t, bsl[r] + k
    lens = np.asarray(ctx) + np.diff(qsl)
    assert head <= tail
    return dict(qsl=qsl, bsl=bsl, lens=lens, pos=pos, slots=slots, tables=tables,
                state=np.array([head, tail]))


def make(S, B, ctx_hi, new_hi, seed, new_lo=0, pad=0, head=0, spare=3):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, S)
    new = rng.integers(new_lo, new_hi + 1, S)
    held, total = -(-ctx // B), -(-(ctx + new) // B)
    NB = int(total.sum()) + spare
    perm = rng.permutation(NB)
    tables = np.full((S, max(1, int(total.max(initial=0)))), -1, np.int32)
    off = 0
    for r in range(S):
        tables[r, :held[r]] = perm[off:off + held[r]]
        off += held[r]
    ring = np.full(NB, -1, np.int32)
    free = perm[off:]
    ring[(head + np.arange(len(free))) % NB] = free
    return dict(ctx=ctx, new=new, tables=tables, ring=ring, head=head, tail=head + len(free),
                B=B, NB=NB, T=int(new.sum()) + pad)


def gpu(c):
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(ctx=i32(c["ctx"]), new=i32(c["new"]), tables=i32(c["tables"]), ring=i32(c["ring"]),
                state=torch.tensor([c["head"], c["tail"]], dtype=torch.int64, device=DEV))


def extend(c, g, T=None, **more):
    qsl, bsl, lens, pos, slots = pa.pa_extend_block_tables(
        g["ctx"], g["new"], g["tables"], c["B"], g["ring"], g["state"], c["NB"],
        c["T"] if T is None else T, **more)
    state = more.get("ring_state_out", g["state"])
    return dict(qsl=qsl, bsl=bsl, lens=lens, pos=pos, slots=slots, tables=g["tables"], state=state)


def same(got, want):
    for k, w in want.items():
        g = got[k].cpu().numpy()
        assert g.shape == w.shape and np.array_equal(g, w), k


# one CTA, a whole cluster, several tiles per CTA, and the two-launch form
# (more token rows than 24,576 and two per request)
SHAPES = [(1, 16, 0, 1), (2, 1, 5, 3), (3, 3, 40, 9), (127, 16, 500, 1), (1024, 8, 30, 2),
          (1025, 16, 100, 40), (5000, 256, 700, 5), (8192, 16, 40, 3), (20000, 4, 9, 1),
          (9000, 16, 20, 30), (64, 128, 2000, 900), (1, 16, 7, 50000)]


@pytest.mark.parametrize("S,B,ctx_hi,new_hi", SHAPES)
@pytest.mark.parametrize("head,pad", [(0, 0), (7, 13), ((1 << 40) + 5, 1)])
def test_extend_matches_the_sequential_rule(S, B, ctx_hi, new_hi, head, pad):
    c = make(S, B, ctx_hi, new_hi, 17 * S + B + pad, pad=pad, head=head)
    g = gpu(c)
    want = ref_extend(c["ctx"], c["new"], c["tables"], B, c["ring"], c["head"], c["tail"], c["T"])
    got = extend(c, g)
    same(got, want)
    assert pa.pa_get_device_error() == 0
    n = int(want["qsl"][-1])
    if n:
        o = oracle.slot_mapping(want["qsl"], want["pos"][:n], want["tables"], B)
        assert np.array_equal(got["slots"].cpu().numpy()[:n], o)


def test_extend_agrees_with_the_slot_mapping_call_and_the_host_pool():
    rng = np.random.default_rng(5)
    B, NB, S = 8, 400, 9
    order = rng.permutation(NB)
    pool = pa.BlockPool(NB, B, free_order=order)
    ctx = rng.integers(0, 60, S)
    for s in range(S):
        pool.add_sequence(s, int(ctx[s]))
    taken = sum(len(pool.blocks[s]) for s in range(S))
    c = dict(ctx=ctx, new=np.ones(S, int), tables=pool.table_rows(range(S), 40), ring=order,
             head=taken, tail=NB, B=B, NB=NB, T=S)
    g = gpu(c)
    for step in range(20):
        positions, pairs = pool.prepare_decode_step(range(S))
        assert not pairs
        got = extend(c, g, seq_lens=g["ctx"])        # lengths and ring state in place
        assert np.array_equal(got["pos"].cpu().numpy(), positions)
        rows = g["tables"].cpu().numpy()
        assert np.array_equal(rows, pool.table_rows(range(S), 40))
        slots = pa.pa_compute_slot_mapping(got["qsl"], got["pos"], g["tables"], B)
        assert torch.equal(slots, got["slots"])
        if step == 11:                               # three requests end
            fin = torch.zeros(S, dtype=torch.bool, device=DEV)
            for s in (1, 4, 8):
                fin[s] = True
                pool.release(s)
                pool.add_sequence(s, 0)
            pa.pa_release_block_tables(fin, g["ctx"], g["tables"], B, g["ring"], g["state"], NB)
            assert (g["ctx"][fin] == 0).all()
            g["tables"][fin] = -1
            head, tail = g["state"].tolist()
            ring = g["ring"].cpu().numpy()
            assert [int(ring[i % NB]) for i in range(head, tail)] == list(pool._free)
    assert pa.pa_get_device_error() == 0


def test_out_of_place_call_leaves_its_inputs():
    c = make(50, 16, 300, 40, 3, head=9)
    g = gpu(c)
    out = torch.empty(2, dtype=torch.int64, device=DEV)
    a = extend(c, g, ring_state_out=out)
    assert g["state"].tolist() == [c["head"], c["tail"]]
    assert np.array_equal(g["ctx"].cpu().numpy(), c["ctx"])
    first = {k: v.clone() for k, v in a.items()}
    b = extend(c, g, ring_state_out=out)             # the same call again gives the same
    for k in first:
        assert torch.equal(first[k], b[k]), k


@pytest.mark.parametrize("S,new_hi", [(40, 30), (3000, 40)])
def test_a_step_that_lacks_blocks_changes_nothing(S, new_hi):
    c = make(S, 4, 50, new_hi, 8, new_lo=1, pad=2, spare=0)
    c["tail"] -= 1                                   # one block too few
    g = gpu(c)
    pa.pa_get_device_error()
    got = extend(c, g)
    assert pa.pa_get_device_error() == NO_BLOCKS
    assert not got["qsl"].any() and not got["bsl"].any() and not got["pos"].any()
    assert (got["slots"] == -1).all()
    assert g["state"].tolist() == [c["head"], c["tail"]]
    assert np.array_equal(got["lens"].cpu().numpy(), c["ctx"])
    assert np.array_equal(g["tables"].cpu().numpy(), c["tables"])
    with pytest.raises(pa.PagedAttnError, match="NO_BLOCKS"):
        from paged_kv_cache_123_gb300._lib import check
        check("pa_extend_block_tables", NO_BLOCKS)


@pytest.mark.parametrize("what", ["rows", "state"])
def test_too_few_rows_or_a_broken_ring_state_change_nothing(what):
    c = make(30, 8, 50, 20, 9, new_lo=1)
    g = gpu(c)
    if what == "state":
        g["state"][0] = c["tail"] + 1                # head behind tail
    state = g["state"].tolist()
    pa.pa_get_device_error()
    got = extend(c, g, T=c["T"] - (1 if what == "rows" else 0))
    assert pa.pa_get_device_error() == OUT_OF_RANGE
    assert not got["qsl"].any() and (got["slots"] == -1).all()
    assert g["state"].tolist() == state


def test_bad_requests_get_nothing_and_the_others_are_served():
    c = make(12, 16, 100, 20, 10, new_lo=1, pad=40)
    cols = c["tables"].shape[1]
    c["ctx"][3], c["new"][5], c["new"][7] = -4, -1, cols * 16 + 1
    want = ref_extend(c["ctx"], c["new"], c["tables"], 16, c["ring"], 0, c["tail"], c["T"])
    g = gpu(c)
    pa.pa_get_device_error()
    same(extend(c, g), want)
    assert pa.pa_get_device_error() == OUT_OF_RANGE


def test_blocks_outside_the_pool_give_no_slot():
    c = make(4, 8, 0, 20, 11, new_lo=9)
    g = gpu(c)
    g["ring"][2] = c["NB"]
    pa.pa_get_device_error()
    got = extend(c, g)
    assert pa.pa_get_device_error() == OUT_OF_RANGE
    assert (got["slots"] < c["NB"] * 8).all() and int((got["slots"] == -1).sum()) > 0


def test_no_requests_and_no_rows():
    empty = np.zeros(0, np.int64)
    c = dict(ctx=empty, new=empty, tables=np.zeros((0, 4), np.int32), ring=np.arange(5), head=0,
             tail=5, B=16, NB=5, T=3)
    g = gpu(c)
    got = extend(c, g)
    assert got["qsl"].tolist() == [0] and got["slots"].tolist() == [-1] * 3
    assert g["state"].tolist() == [0, 5]
    c["T"] = 0
    assert extend(c, g)["pos"].numel() == 0
    assert pa.pa_get_device_error() == 0


def test_extend_captured_and_replayed_in_place():
    """A decode loop as one graph: lengths, tables and ring state advance on
    the device, across block borders, with padding rows."""
    c = make(6, 4, 20, 1, 12, new_lo=1, spare=200)
    c["tables"] = np.pad(c["tables"], ((0, 0), (0, 20)), constant_values=-1)
    g = gpu(c)
    g["new"].fill_(1)
    bufs = dict(query_start_loc=torch.empty(7, dtype=torch.int32, device=DEV),
                block_start_loc=torch.empty(7, dtype=torch.int32, device=DEV),
                positions=torch.empty(9, dtype=torch.int64, device=DEV),
                slot_mapping=torch.empty(9, dtype=torch.int64, device=DEV), seq_lens=g["ctx"])
    call = lambda: pa.pa_extend_block_tables(  # noqa: E731
        g["ctx"], g["new"], g["tables"], 4, g["ring"], g["state"], c["NB"], 9, **bufs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    ctx, tables, head = c["ctx"].copy(), c["tables"].copy(), c["head"]
    for _ in range(30):
        graph.replay()
        w = ref_extend(ctx, np.ones(6, int), tables, 4, c["ring"], head, c["tail"], 9)
        ctx, tables, head = w["lens"], w["tables"], int(w["state"][0])
        assert np.array_equal(bufs["slot_mapping"].cpu().numpy(), w["slots"])
        assert np.array_equal(g["tables"].cpu().numpy(), tables)
        assert g["state"].tolist() == [head, c["tail"]]
    assert pa.pa_get_device_error() == 0


# ---- release ---------------------------------------------------------------
def ref_release(fin, lens, tables, B, ring, head, tail, NB):
    ring, S = ring.copy(), len(lens)
    rsl, out = np.zeros(S + 1, np.int64), np.asarray(lens).copy()
    for r in range(S):
        n = 0
        L = int(lens[r])
        if fin[r] and 0 <= L <= tables.shape[1] * B:
            for b in tables[r, :-(-L // B)]:
                if 0 <= b < NB:
                    ring[tail % len(ring)] = b
                    tail, n = tail + 1, n + 1
            out[r] = 0
        rsl[r + 1] = rsl[r] + n
    return dict(rsl=rsl, lens=out, ring=ring, state=np.array([head, tail]))


def release(c, g, fin, **more):
    rsl = pa.pa_release_block_tables(fin, g["ctx"], g["tables"], c["B"], g["ring"], g["state"],
                                     c["NB"], **more)
    return dict(rsl=rsl, lens=more.get("seq_lens_out", g["ctx"]), ring=g["ring"],
                state=more.get("ring_state_out", g["state"]))


@pytest.mark.parametrize("S,B,ctx_hi", [(1, 16, 0), (1, 16, 90), (5, 1, 40), (128, 16, 2000),
                                        (33, 256, 9000), (1000, 8, 300), (3000, 16, 900),
                                        (9000, 4, 60)])
@pytest.mark.parametrize("holes", [False, True])
def test_release_matches_the_sequential_rule(S, B, ctx_hi, holes):
    c = make(S, B, ctx_hi, 0, S + B, head=23)
    rng = np.random.default_rng(S)
    if holes:
        c["tables"][rng.random(c["tables"].shape) < 0.3] = -1
    fin = rng.random(S) < 0.4
    fin[0] = True
    g = gpu(c)
    want = ref_release(fin, c["ctx"], c["tables"], B, c["ring"], c["head"], c["tail"], c["NB"])
    got = release(c, g, torch.tensor(fin, device=DEV))
    same(got, want)
    assert np.array_equal(g["tables"].cpu().numpy(), c["tables"])
    again = release(c, g, torch.tensor(fin, device=DEV))     # their length is 0: nothing twice
    assert not again["rsl"].any() and again["state"].tolist() == want["state"].tolist()
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("S", [1, 31, 32, 33, 255, 256, 257])
def test_release_of_long_rows_around_a_cluster(S):
    """Rows of more than 512 and 1,024 entries, entries of other pools and
    released ones among them; one launch up to 256 requests."""
    c = make(S, 4, 5000, 0, 7 * S, head=11)
    rng = np.random.default_rng(S + 1)
    c["ctx"][S // 2] = 4 * 1200 if c["tables"].shape[1] >= 1200 else c["ctx"][S // 2]
    c["tables"][rng.random(c["tables"].shape) < 0.2] = -1
    fin = np.ones(S, bool)
    fin[1::5] = False
    g = gpu(c)
    want = ref_release(fin, c["ctx"], c["tables"], 4, c["ring"], c["head"], c["tail"], c["NB"])
    same(release(c, g, torch.tensor(fin, device=DEV)), want)
    assert pa.pa_get_device_error() == 0
    # the same into other arrays: lengths and state are kept
    g = gpu(c)
    out = dict(seq_lens_out=torch.empty(S, dtype=torch.int32, device=DEV),
               ring_state_out=torch.empty(2, dtype=torch.int64, device=DEV))
    same(release(c, g, torch.tensor(fin, device=DEV), **out), want)
    assert np.array_equal(g["ctx"].cpu().numpy(), c["ctx"])
    assert g["state"].tolist() == [c["head"], c["tail"]]


@pytest.mark.parametrize("S", [12031, 12032, 12155, 12156, 12287, 12288])
@pytest.mark.parametrize("new", [1, 5])
def test_extend_around_the_shared_memory_of_a_launch(S, new):
    """Where query_start_loc stops fitting beside the kernels' own shared
    memory, in one launch and in two."""
    c = make(S, 16, 50, new, S + new, new_lo=new)
    same(extend(c, gpu(c)), ref_extend(c["ctx"], c["new"], c["tables"], 16, c["ring"], c["head"],
                                       c["tail"], c["T"]))
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("S", [3, 900])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_extend_around_the_rows_of_one_launch(S, more):
    c = make(S, 16, 500, 24 * 1024 // S, S + more + 5)
    rows = 24 * 1024 + 2 * S + more
    assert c["T"] <= rows
    c["T"] = rows
    g = gpu(c)
    same(extend(c, g), ref_extend(c["ctx"], c["new"], c["tables"], 16, c["ring"], c["head"],
                                  c["tail"], rows))
    assert pa.pa_get_device_error() == 0


@pytest.mark.parametrize("S", [20, 4000])
def test_release_refusals_on_the_device(S):
    c = make(S, 16, 600, 0, 31, spare=0)
    g = gpu(c)
    g["state"][1] += 1                               # a ring with one place too few
    state, ring = g["state"].tolist(), g["ring"].clone()
    fin = torch.ones(S, dtype=torch.uint8, device=DEV)
    pa.pa_get_device_error()
    got = release(c, g, fin)
    assert pa.pa_get_device_error() == OUT_OF_RANGE
    assert not got["rsl"].any() and g["state"].tolist() == state
    assert torch.equal(g["ring"], ring) and np.array_equal(got["lens"].cpu().numpy(), c["ctx"])
    # bad lengths and ids: those rows or entries are left out
    c["ctx"][2], c["ctx"][5] = -1, c["tables"].shape[1] * 16 + 1
    c["tables"][7, 0] = c["NB"] + 4
    c["ctx"][7] = max(c["ctx"][7], 1)
    g = gpu(c)
    want = ref_release(fin.cpu().numpy(), c["ctx"], c["tables"], 16, c["ring"], c["head"],
                       c["tail"], c["NB"])
    same(release(c, g, fin), want)
    assert pa.pa_get_device_error() == OUT_OF_RANGE


def test_two_streams_with_their_own_rings():
    cases = [make(700, 16, 400, 30, s, head=s) for s in (1, 2)]
    gs = [gpu(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for c, g, st in zip(cases, gs, streams):
        with torch.cuda.stream(st):
            outs.append(extend(c, g))
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        same(o, ref_extend(c["ctx"], c["new"], c["tables"], 16, c["ring"], c["head"], c["tail"],
                           c["T"]))
