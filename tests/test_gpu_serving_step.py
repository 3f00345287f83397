"""Whole serving steps on the device, as a user runs them: extend the block
tables, rotate and write, attend over the fp8 pool, release finished
requests; against a host that keeps every request's tokens in plain arrays."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_123_gb300 as pa
from paged_kv_cache_123_gb300 import workloads
from tests.helpers import np_

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D, B, NB, S, COLS = 16, 2, 128, 16, 220, 5, 60
INV = 1.0 / (10000.0 ** (torch.arange(D // 2, dtype=torch.float64) / (D // 2)))


def turned(x, pos):
    """The formula, on float64 [T, H, D]."""
    ang = pos.astype(np.longdouble)[:, None] * INV.numpy().astype(np.longdouble)
    c, s = np.cos(ang).astype(float)[:, None], np.sin(ang).astype(float)[:, None]
    a, b = x[..., :D // 2], x[..., D // 2:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


class Server:
    """Device state of a small server; plan, write, attend, release."""

    def __init__(self, pool, window):
        self.pool, self.window = pool, window
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
        self.lens, self.tables = i32(S), torch.full((S, COLS), -1, dtype=torch.int32, device=DEV)
        self.ring = torch.randperm(NB, generator=torch.Generator().manual_seed(4)).to(
            DEV, torch.int32)
        self.state = torch.tensor([0, NB], dtype=torch.int64, device=DEV)
        self.kc = torch.full((NB, HKV, B, D), 0x7f, dtype=torch.uint8, device=DEV)
        self.vc = self.kc.clone()
        self.scales = ((0.03, 0.04) if pool == "pool" else
                       tuple(torch.ones(NB, HKV, device=DEV) for _ in range(2)))
        self.inv = INV.to(DEV)

    def step(self, new, q, k, v):
        T = q.shape[0]
        qsl, _, _, pos, slots = pa.pa_extend_block_tables(
            self.lens, new, self.tables, B, self.ring, self.state, NB, T, seq_lens=self.lens)
        write = (pa.pa_rotary_reshape_and_cache_fp8 if self.pool == "pool" else
                 pa.pa_rotary_reshape_and_cache_fp8_scaled)
        q = write(q, k, v, pos, self.inv, slots, self.kc, self.vc, *self.scales)
        more = dict(max_query_len=T, max_seq_len=COLS * B, window=self.window)
        if self.pool == "pool":
            out = pa.pa_multi_query_attention_fp8(q, qsl, self.kc, self.vc, self.tables, self.lens,
                                                  D ** -0.5, HKV, *self.scales, **more)
        else:
            out = pa.pa_multi_query_attention_fp8_scaled(q, qsl, self.kc, self.vc, *self.scales,
                                                         self.tables, self.lens, D ** -0.5, HKV,
                                                         **more)
        return q, out, pos


@pytest.mark.parametrize("pool,window", [("pool", 0), ("blocks", 0), ("pool", 50),
                                         ("blocks", 130)])
def test_steps_of_a_small_server(pool, window):
    gen = torch.Generator().manual_seed(11)
    srv = Server(pool, window)
    kv = [[np.zeros((0, HKV, D))] * 2 for _ in range(S)]     # what the pool should hold
    plan = [[100, 7, 0, 33, 1], [1, 1, 1, 1, 1], [4, 1, 60, 1, 300], [1, 0, 1, 16, 1],
            "release", [20, 90, 1, 1, 1], [1, 1, 1, 1, 1]]
    for new in plan:
        if new == "release":
            fin = torch.tensor([0, 1, 0, 1, 0], dtype=torch.bool, device=DEV)
            held = [int(x) for x in srv.lens.cpu()]
            pa.pa_release_block_tables(fin, srv.lens, srv.tables, B, srv.ring, srv.state, NB)
            head, tail = srv.state.tolist()
            assert tail - NB == sum(-(-held[s] // B) for s in (1, 3))
            for s in (1, 3):
                kv[s] = [np.zeros((0, HKV, D))] * 2
            assert srv.lens.tolist() == [0 if s in (1, 3) else held[s] for s in range(S)]
            continue
        T = sum(new) + 3                                     # three padding rows
        qkv = torch.randn(T, (HQ + 2 * HKV) * D, generator=gen).to(torch.bfloat16).to(DEV)
        q, k, v = (qkv[:, a:b].view(T, -1, D) for a, b in
                   ((0, HQ * D), (HQ * D, (HQ + HKV) * D), ((HQ + HKV) * D, None)))
        qr, out, pos = srv.step(torch.tensor(new, dtype=torch.int32, device=DEV), q, k, v)
        assert pa.pa_get_device_error() == 0
        kd, vd = (x.double().cpu().numpy() for x in (k, v))
        p, t = pos.cpu().numpy(), 0
        qh = oracle.upcast(np_(qr), "bf16")                  # q as rotated: its own test
        kr = turned(kd, p)
        for s, n in enumerate(new):
            L0 = len(kv[s][0])
            assert p[t:t + n].tolist() == list(range(L0, L0 + n))
            kv[s] = [np.concatenate([kv[s][0], kr[t:t + n]]),
                     np.concatenate([kv[s][1], vd[t:t + n]])]
            K, V = kv[s]
            for i in range(n):
                lo = max(0, L0 + i + 1 - window) if window else 0
                for h in range(HQ):
                    kh, vh = K[lo:L0 + i + 1, h // 8], V[lo:L0 + i + 1, h // 8]
                    x = (kh @ qh[t + i, h]) * D ** -0.5
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    got = out[t + i, h].double().cpu().numpy() if h % 7 == 0 else None
                    if got is None:
                        continue
                    # E4M3 keeps half a step, 2^-4 relative, of K and V: a
                    # logit moves by at most 2^-4 sum |q k| scale, in practice
                    # by its random sum, sqrt(sum (q k)^2) * 2^-4 / sqrt(3)
                    # per standard deviation; five of them bound the weights'
                    # change exp(2 d) - 1, and V's own half step adds 2^-4
                    sd = (np.sqrt(((kh * qh[t + i, h]) ** 2).sum(-1)) * D ** -0.5).max()
                    d = 5 * sd * 2.0 ** -4 / np.sqrt(3)
                    A = w @ np.abs(vh)
                    tol = A * (2.0 ** -4 + (np.exp(2 * d) - 1)) + 2.0 ** -8 * A + 1e-3
                    assert (np.abs(got - w @ vh) <= tol).all(), (s, i, h)
            t += n
    head, tail = srv.state.tolist()
    rows = srv.tables.cpu().numpy()
    lens = srv.lens.tolist()
    owned = [b for s in range(S) for b in rows[s, :-(-lens[s] // B)]]
    ring = srv.ring.cpu().numpy()
    free = [int(ring[i % NB]) for i in range(head, tail)]
    assert sorted(owned + free) == list(range(NB))           # no block lost or owned twice


def test_a_decode_loop_in_one_graph():
    """extend, rotary write and attention captured once and replayed: the
    same numbers as the calls one by one."""
    gen = torch.Generator().manual_seed(21)
    new = torch.ones(S, dtype=torch.int32, device=DEV)
    qkv = [torch.randn(S, (HQ + 2 * HKV) * D, generator=gen).to(torch.bfloat16).to(DEV)
           for _ in range(20)]
    split = lambda x: [x[:, a:b].view(S, -1, D) for a, b in  # noqa: E731
                       ((0, HQ * D), (HQ * D, (HQ + HKV) * D), ((HQ + HKV) * D, None))]
    plain = Server("blocks", 0)
    want = [plain.step(new, *split(x))[1].clone() for x in qkv]
    srv = Server("blocks", 0)
    x0 = qkv[0].clone()
    warm = Server("blocks", 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm.step(new, *split(x0))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, out, _ = srv.step(new, *split(x0))
    for x, w in zip(qkv, want):
        x0.copy_(x)
        graph.replay()
        assert torch.equal(out, w)
    assert torch.equal(srv.lens, plain.lens) and torch.equal(srv.tables, plain.tables)
    assert pa.pa_get_device_error() == 0
