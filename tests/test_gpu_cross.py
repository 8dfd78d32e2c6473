"""GPU tests of mac_cross_attention against 64 bits.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value.  With x the
scores, P the normalised weights and A = sum P |v|: scores are fp32 sums of d
products, off by at most e = (d + 4) 2^-24 max_j sum |q k_j| / sqrt(d) each
(taken four times for bf16: tensor cores keep sums a little shorter than
fp32); weights and sums of n keys add (n + 64) 2^-24.  So out is off by at
most A (2 e + (n + 64) 2^-24), with bf16 also by 2^-8 A for the rounded weights
and 2^-8 |out| for the result; lse by e + (n + 64) 2^-24 + 2^-22 |lse|."""
import math
import random

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from long_context_decode_gb300 import mac  # noqa: E402

D, PAGE = 128, 16
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_decode_gb300 import build as b
    b.build()
    mac.load()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


def pages_of(n):
    return -(-n // PAGE)


def near(got, want, tol):
    got = got.double()
    assert torch.isfinite(got).all()
    bad = (got - want).abs() > tol
    assert not bad.any(), ((got - want).abs()[bad].max().item(), int(bad.sum()))


class Sources:
    """mem[b] states of each source and new[s] rows of each of its `group` slots."""

    def __init__(self, mem, new, group, Hq, Hkv, dt=BF16, paged=True, seed=0, pad=0, fill=float("nan"), scale=1.0, room=0):
        assert len(new) == len(mem) * group
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.mem, self.new, self.group, self.Hq, self.Hkv, self.dt = mem, new, group, Hq, Hkv, dt
        B, self.T = len(mem), sum(new) + pad
        self.start = np.concatenate([[0], np.cumsum(new)]).tolist()
        width = pages_of(max(mem + [1])) + 1 + pages_of(room)
        cap = width * PAGE
        self.q = (torch.randn(max(self.T, 1), Hq, D, generator=g, device=DEV) * scale).to(dt)
        if pad:
            self.q[sum(new):] = fill
        self.kd, self.vd = (torch.randn(B, Hkv, cap, D, generator=g, device=DEV).to(dt) for _ in range(2))
        self.kd[0, :, 0] *= 6  # a heavy key
        self.table = None
        if paged:
            held = [pages_of(n) for n in mem]
            n_pages = sum(held) + 3
            ids = torch.randperm(n_pages, generator=g, device=DEV)
            self.table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
            self.k = torch.full((n_pages, Hkv, PAGE, D), fill, device=DEV, dtype=dt)
            self.v = self.k.clone()
            at = 0
            for b, (h, n) in enumerate(zip(held, mem)):
                mine = ids[at:at + h]
                self.table[b, :h] = mine.int()
                at += h
                for x, dense in ((self.k, self.kd), (self.v, self.vd)):
                    rows = torch.full((Hkv, h * PAGE, D), fill, device=DEV, dtype=dt)
                    rows[:, :n] = dense[b, :, :n]
                    x[mine] = rows.view(Hkv, h, PAGE, D).transpose(0, 1)
        else:
            self.k, self.v = self.kd.clone(), self.vd.clone()
            for b, n in enumerate(mem):
                self.k[b, :, n:] = fill
                self.v[b, :, n:] = fill
        self.kv = mac.kv_view(self.k, self.v, self.table)
        self.cfg = mac.config(B, Hq, Hkv, dtype=mac.MAC_BF16 if dt == BF16 else mac.MAC_F32, page_size=PAGE if paged else 0, max_context=cap)
        self.q_start, self.mem_len = ints(self.start), ints(mem)
        self.ws = torch.zeros(mac.mac_chunk_workspace_size(self.cfg, max(self.T, 1)), dtype=torch.uint8, device=DEV)
        self.out = torch.full((max(self.T, 1), Hq, D), 7.0, device=DEV, dtype=dt)
        self.lse = torch.full((max(self.T, 1), Hq), 7.0, device=DEV)

    def run(self, stream=None, lse=True):
        mac.mac_cross_attention(self.cfg, self.ws, self.q, self.q_start, self.group, self.mem_len, self.T, self.kv, self.out,
                                self.lse if lse else None, stream)

    def status(self):
        return mac.mac_last_status(self.cfg, self.ws)

    def rows(self, b):
        return self.start[b * self.group], self.start[(b + 1) * self.group]

    def check(self, drop=None, skip=()):
        """Compare with 64 bits; drop[b]: 0-based positions that are left out; skip: sources not looked at."""
        G, bf = self.Hq // self.Hkv, self.dt == BF16
        for b, m in enumerate(self.mem):
            r0, r1 = self.rows(b)
            if b in skip:
                continue
            for lo in range(r0, r1, 512):
                rows = slice(lo, min(r1, lo + 512))
                keep = [x for x in range(m) if not (drop and x in drop.get(b, ()))]
                if not keep:
                    assert (self.out[rows] == 0).all() and (self.lse[rows] == -math.inf).all()
                    continue
                k, v = (x[b, :, keep].double().repeat_interleave(G, 0) for x in (self.kd, self.vd))
                q = self.q[rows].double().transpose(0, 1)
                x = q @ k.transpose(1, 2) / math.sqrt(D)
                big = (q.abs() @ k.abs().transpose(1, 2)).amax(-1) / math.sqrt(D)
                lse = torch.logsumexp(x, -1)
                w = torch.exp(x - lse[..., None])
                want, A = (w @ v).transpose(0, 1), (w @ v.abs()).transpose(0, 1)
                e = (D + 4) * 2.0 ** -24 * big * (4 if bf else 1)
                rest = (m + 64) * 2.0 ** -24
                tol = A * (2 * e + rest).t()[..., None]
                if bf:
                    tol = tol + 2.0 ** -8 * (A + want.abs())
                near(self.out[rows], want, tol)
                near(self.lse[rows].t(), lse, e + rest + 2.0 ** -22 * lse.abs())
        end = self.start[-1]
        assert (self.out[end:] == 7).all() and (self.lse[end:] == 7).all()  # rows behind the last source


SHAPES = [  # states of each source, slots of a source, rows of each slot
    ([1], 1, [1]), ([2], 1, [3]), ([15], 4, [1] * 4), ([16], 1, [1]), ([17], 2, [1, 1]), ([63], 1, [2]), ([64], 1, [17]), ([65], 5, [1] * 5),
    ([127], 1, [1]), ([128], 1, [64]), ([129], 3, [1, 0, 2]), ([500], 1, [129]), ([1000], 4, [1] * 4), ([4097], 1, [1]), ([300], 2, [300, 1]),
    ([40, 0, 700, 16, 1], 2, [1, 1, 2, 0, 3, 70, 0, 0, 1, 0]), ([0], 1, [5]), ([0, 0], 4, [1] * 8), ([33] * 9, 3, [1] * 27),
    ([5, 260], 16, [1] * 32),
]


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (2, 2), (2, 1), (16, 2)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_cross(shape, Hq, Hkv, dt, paged):
    # rows of the cache beyond the lengths, and queries of rows that belong to nobody, are NaN
    mem, group, new = SHAPES[shape]
    c = Sources(mem, new, group, Hq, Hkv, dt, paged, seed=shape, pad=shape % 3)
    c.run()
    assert c.status() == 0
    c.check()


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (8, 1), (4, 4)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_cross_in_a_large_cache(shape, Hq, Hkv, dt, paged):
    # what fits in the cache, not the lengths, says which kernels run
    mem, group, new = SHAPES[shape]
    c = Sources(mem, new, group, Hq, Hkv, dt, paged, seed=shape, pad=shape % 3, room=(1 << 18) // len(mem))
    c.run()
    assert c.status() == 0
    c.check()


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,mem,group,new", [
    (32, 8, [128] * 4, 1, [16] * 4), (32, 8, [100], 1, [75]), (32, 8, [128], 1, [77]), (8, 1, [2000], 1, [9]), (8, 2, [8100], 4, [1, 2, 9, 4]),
    (8, 2, [500, 0, 37], 2, [3, 40, 0, 1, 7, 0]), (4, 4, [1], 1, [600]), (4, 4, [1, 1], 1, [300, 308]), (1, 1, [3, 800, 90], 1, [0, 2400, 1]),
    (2, 2, [1700, 30], 8, [5] * 16), (8, 4, [129, 640, 17], 5, [1] * 15),
])
def test_cross_of_more_rows_than_a_block(Hq, Hkv, mem, group, new, dt, paged):
    c = Sources(mem, new, group, Hq, Hkv, dt, paged, seed=len(new), pad=3)
    c.run()
    assert c.status() == 0
    c.check()


@pytest.mark.parametrize("dt,Hq,Hkv,mem,group,new,paged", [
    (BF16, 32, 8, [1500, 400, 999] * 5, 4, [1] * 60, False),       # a decode step of beams
    (BF16, 32, 8, [3000, 70, 9000], 1, [1500, 2049, 17], True),    # many rows
    (BF16, 32, 4, [20000], 1, [1], True),                          # one row over every CTA
    (BF16, 4, 4, [70001, 70], 1, [1, 1], False),
    (BF16, 1, 1, [64], 1, [4096], False),
    (BF16, 8, 2, [30000], 2, [32, 33], True),
    (BF16, 1, 1, [40000], 1, [3], False),
    (F32, 32, 8, [1500, 400, 999] * 2, 4, [1] * 24, False),
    (F32, 8, 2, [3000, 10], 1, [500, 700], True),
    (F32, 32, 4, [20000], 1, [1], True),
    (F32, 1, 1, [40000], 1, [3], False),
])
def test_cross_over_many_ctas(dt, Hq, Hkv, mem, group, new, paged):
    c = Sources(mem, new, group, Hq, Hkv, dt, paged, seed=1, pad=2)
    c.run()
    assert c.status() == 0
    c.check()


@pytest.mark.parametrize("seed", range(24))
def test_cross_drawn(seed):
    rng = random.Random(seed)
    Hq, Hkv = rng.choice([(32, 8), (32, 4), (8, 8), (8, 1), (4, 2), (1, 1)])
    group, B = rng.choice([1, 1, 2, 4, 7]), rng.choice([1, 2, 5, 12])
    top = rng.choice([20, 300, 3000])
    mem = [rng.choice([0, rng.randint(1, 17), rng.randint(1, top)]) for _ in range(B)]
    most = rng.choice([1, 1, 5, 80])
    new = [rng.randint(0, most) for _ in range(B * group)]
    if not any(new):
        new[-1] = 1
    c = Sources(mem, new, group, Hq, Hkv, rng.choice([BF16, F32]), rng.random() < 0.5, seed, rng.choice([0, 5]))
    c.run(lse=True)
    assert c.status() == 0
    c.check()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("new", [1, 90])
def test_cross_large_scores_and_no_lse(dt, new):
    c = Sources([700], [new], 1, 8, 2, dt, seed=5, scale=30.0)
    c.run(lse=False)
    assert c.status() == 0 and (c.lse == 7).all()
    c.run()
    c.check()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("new", [1, 40])
def test_cross_leaves_out_bad_pages(dt, new):
    c = Sources([100, 40, 16], [new] * 3, 1, 8, 2, dt, seed=2)
    c.table[0, 2], c.table[0, 6] = -1, c.k.shape[0]
    c.table[2, 0] = 1 << 30  # nothing is left of source 2
    c.run()
    assert c.status() == mac.MAC_DEV_BAD_PAGE
    c.check(drop={0: [*range(32, 48), *range(96, 100)], 2: range(16)})


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("paged", [True, False])
def test_cross_bad_lengths_and_rows(dt, paged):
    c = Sources([50, 60, 70, 80], [2, 3, 1, 2], 1, 8, 2, dt, paged, seed=3)
    c.mem_len.copy_(ints([50, -1, 1 << 20, 80]))
    c.run()
    assert c.status() == mac.MAC_DEV_BAD_SEQ_LEN
    for b in (1, 2):
        r0, r1 = c.rows(b)
        assert (c.out[r0:r1] == 0).all() and (c.lse[r0:r1] == -math.inf).all()
    c.check(skip=(1, 2))
    c.out.fill_(7)
    c.lse.fill_(7)
    c.mem_len.copy_(ints(c.mem))
    c.q_start.copy_(ints([0, 2, 5, 6, 99]))  # the last source's rows end behind the batch
    c.run()
    assert c.status() == mac.MAC_DEV_BAD_SEQ_LEN
    assert (c.out[6:] == 7).all()
    c.check(skip=(3,))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_cross_ignores_the_slots_between(dt):
    # q_start's entries between a source's first and last are not looked at
    c = Sources([50, 60], [1, 1, 1, 2, 1, 1], 3, 8, 2, dt, seed=3)
    c.q_start.copy_(ints([0, -5, 1 << 30, 3, 77, -1, 7]))
    c.run()
    assert c.status() == 0
    c.check()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("new", [1, 50])
def test_cross_infinite_and_nan_rows_stay_in_their_row(dt, new):
    c = Sources([90], [new + 2], 1, 8, 2, dt, seed=4)
    clean = c.q.clone()
    c.q[0], c.q[1, 3] = math.inf, math.nan
    c.run()
    rest = c.out[2:].clone(), c.lse[2:].clone()
    assert torch.isnan(c.out[0]).all() and torch.isnan(c.out[1, 3]).all() and torch.isfinite(c.out[1, :3]).all()
    c.q.copy_(clean)
    c.run()
    c.check()
    assert torch.equal(c.out[2:], rest[0]) and torch.equal(c.lse[2:], rest[1])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("new", [1, 60])
def test_cross_on_streams_and_in_graphs(dt, new):
    """A captured call serves other lengths and rows; two graphs with a workspace each run side by side."""
    calls = [Sources([200, 0, 900], [new] * 6, 2, 8, 2, dt, seed=s, pad=4) for s in (1, 2)]
    streams, graphs = [torch.cuda.Stream() for _ in calls], []
    torch.cuda.synchronize()
    for c, s in zip(calls, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run(torch.cuda.current_stream())
        graphs.append(g)
    for mem, rows in (([200, 0, 900], [new] * 6), ([17, 800, 0], [0, new, new, new, 1, 0])):
        for c in calls:
            c.mem, c.new, c.start = mem, rows, np.concatenate([[0], np.cumsum(rows)]).tolist()
            if c.table is not None:  # all pages of the pool, in another order for every source's needs
                ids = torch.randperm(c.k.shape[0], device=DEV)
                held = [pages_of(m) for m in mem]
                assert sum(held) <= len(ids)
                at = 0
                for b, h in enumerate(held):
                    c.table[b, :h] = ids[at:at + h].int()
                    at += h
                    for x, dense in ((c.k, c.kd), (c.v, c.vd)):
                        full = torch.full((c.Hkv, h * PAGE, D), float("nan"), device=DEV, dtype=dt)
                        full[:, :mem[b]] = dense[b, :, :mem[b]]
                        x[ids[at - h:at]] = full.view(c.Hkv, h, PAGE, D).transpose(0, 1)
            c.q = c.q.nan_to_num_(1.0)
            c.mem_len.copy_(ints(mem))
            c.q_start.copy_(ints(c.start))
            c.out.fill_(7)
            c.lse.fill_(7)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for c in calls:
            assert c.status() == 0
            c.check()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_cross_is_the_same_every_time(dt):
    # several pieces per unit, joined in an order of their own
    c = Sources([5000, 3000, 9000], [1] * 12, 4, 8, 2, dt, seed=6)
    c.run()
    first = c.out.clone(), c.lse.clone()
    for _ in range(20):
        c.run()
        assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])
    c.check()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_chunk_and_cross_share_a_workspace(dt):
    # one stream, one workspace: rows of a chunk over its own keys, then over a memory
    c = Sources([333, 40], [9, 70], 1, 8, 2, dt, paged=False, seed=8)
    k, v = torch.randn_like(c.k), torch.randn_like(c.v)
    k, v = k.nan_to_num_(), v.nan_to_num_()
    own_out, own_lse = torch.zeros_like(c.out), torch.zeros_like(c.lse)
    ref_out, ref_lse = torch.zeros_like(c.out), torch.zeros_like(c.lse)
    kv = mac.kv_view(k, v)
    ws = torch.zeros_like(c.ws)
    mac.mac_chunk_attention(c.cfg, ws, c.q, c.q_start, ints([9, 70]), c.T, kv, ref_out, ref_lse)
    mac.mac_chunk_attention(c.cfg, c.ws, c.q, c.q_start, ints([9, 70]), c.T, kv, own_out, own_lse)
    c.run()
    assert c.status() == 0 and torch.equal(own_out, ref_out) and torch.equal(own_lse, ref_lse)
    c.check()


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_cross_spans_without_a_tile(dt, paged):
    # equal spans of the cost axis: the last CTA's may hold no key tile, and it must not look for queries
    for keys in range(1300, 2700, 100):
        c = Sources([0, keys], [0, 0, 0, 1], 2, 8, 8, dt, paged, seed=keys)
        c.run()
        assert c.status() == 0
        c.check()


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("new", [3, 150])
def test_cross_caches_beyond_32_bit_offsets(new, dt, paged):
    # the last source's keys and values lie past element 2^32
    Hkv, mem = 2, [70, 333]
    c = Sources(mem, [new, new], 1, 8, Hkv, dt, paged, seed=12)
    if paged:
        far = (1 << 32) // (Hkv * PAGE * D) + 7
        big = [torch.empty(far + 40, Hkv, PAGE, D, device=DEV, dtype=dt) for _ in range(2)]
        for x, small in zip(big, (c.k, c.v)):
            x[far:far + small.shape[0]] = small
        c.table[c.table >= 0] += far
    else:
        cap = (1 << 32) // (3 * D) + 64
        big = [torch.empty(2, Hkv, cap, D, device=DEV, dtype=dt) for _ in range(2)]
        for x, small in zip(big, (c.k, c.v)):
            x[:, :, :small.shape[2]] = small
            x[:, :, small.shape[2]:small.shape[2] + 256] = float("nan")
        assert big[0][1, 1].storage_offset() > 1 << 32
        c.cfg = mac.config(2, 8, Hkv, dtype=c.cfg.dtype, max_context=cap)
        c.ws = torch.zeros(mac.mac_chunk_workspace_size(c.cfg, c.T), dtype=torch.uint8, device=DEV)
    c.kv = mac.kv_view(*big, c.table)
    c.run()
    assert c.status() == 0
    c.check()


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_cross_wait_runs_out(dt, paged):
    # many rows: the kernels that wait for copies and products.  A key stage that is never filled is reported and left
    c = Sources([3000, 1500], [90, 90], 1, 8, 2, dt, paged, seed=9)
    mac.mac_test_wait_budget(1 << 16, 1)
    c.run()
    torch.cuda.synchronize()
    assert c.status() & mac.MAC_DEV_WAIT_TIMEOUT
    c.ws = torch.zeros_like(c.ws)
    c.run()
    assert c.status() == 0
    c.check()
    # few rows: nothing waits for another role, so no budget runs out
    c = Sources([3000, 1500], [1, 1], 1, 8, 2, dt, paged, seed=9)
    mac.mac_test_wait_budget(1, 0)
    c.run()
    assert c.status() == 0
    c.check()
