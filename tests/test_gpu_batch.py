"""GPU tests of the calls on a batch of new tokens (mac_build_tables,
mac_write_kv, mac_chunk_attention) against plain implementations: whole
numbers in Python, the rest in 64 bits.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value.
  rotation: the angle's fraction of a turn is exact and rounded once to fp32
    (2^-24 of at most pi), sine and cosine are good to 2 ulp, the two
    products and their sum round once each: below (|a| + |b|) 2^-21.
  attention: with x the scores, P the normalised probabilities and
    A = sum P |v|: scores are fp32 sums of d products, off by at most
    e = (d + 4) 2^-24 max_j sum |q k_j| / sqrt(d) each; the weights and
    sums of n keys add (n + 64) 2^-24; so out is off by at most
    A (2 e + (n + 64) 2^-24), and with bf16 also by 2^-8 A for the rounded
    probabilities and 2^-8 |out| for the result; lse by
    e + (n + 64) 2^-24 + 2^-22 |lse|.  Tensor cores keep sums of products a
    little shorter than fp32: e is taken four times for bf16."""
import ctypes
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


def workspace(cfg, T):
    return torch.zeros(mac.mac_chunk_workspace_size(cfg, T), dtype=torch.uint8, device=DEV)


def pages_of(n):
    return -(-n // PAGE)


# ---------------------------------------------------------------------------
# page tables
# ---------------------------------------------------------------------------

def ref_tables(length, new, flags, T, limit, table=None, free=None, n_free=0, capacity=0):
    """The call's definition, request by request.  Returns its outputs and status bits."""
    B, st = len(length), 0
    base, ok = [], []
    for b in range(B):
        good = 0 <= length[b] <= limit
        if flags and flags[b] and good:
            if table is not None:
                for x in range(pages_of(length[b])):
                    free[n_free] = table[b][x]
                    n_free += 1
            base.append(0)
        else:
            base.append(length[b])
        ok.append(good and new[b] >= 0 and base[b] + new[b] <= limit)
        if not ok[b]:
            st |= mac.MAC_DEV_BAD_SEQ_LEN
    avail, asked_pages, asked_rows = n_free, 0, 0
    q_start, pos, slot, len_out = [0], [], [], []
    for b in range(B):
        n = new[b] if ok[b] else 0
        need = pages_of(base[b] + n) - pages_of(base[b]) if table is not None and n else 0
        asked_pages += need
        asked_rows += n
        if n and (asked_rows > T or (need and asked_pages > avail)):
            st |= mac.MAC_DEV_NO_ROOM
            n = need = 0
        if n and table is not None:
            for x in range(pages_of(base[b]), pages_of(base[b]) + need):
                n_free -= 1
                table[b][x] = free[n_free]
        for i in range(n):
            p = base[b] + i
            pos.append(p + 1)
            slot.append(b * capacity + p if table is None else table[b][p // PAGE] * PAGE + p % PAGE)
        q_start.append(q_start[-1] + n)
        len_out.append(base[b] + n)
    pos += [0] * (T - len(pos))
    slot += [-1] * (T - len(slot))
    return len_out, q_start, pos, slot, n_free, st


def make_pool(length, width, spare, seed):
    rng = random.Random(seed)
    held = [pages_of(max(0, min(n, width * PAGE))) for n in length]
    n_pages = sum(held) + spare
    ids = list(range(n_pages))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    free = ids[at:] + [-7] * at
    return table, free, len(ids) - at, n_pages


TABLE_CASES = [
    # B, lengths up to, new up to, resets one in, spare pages, extra rows
    (1, 0, 1, 0, 1, 0),
    (1, 15, 2, 0, 3, 3),
    (3, 40, 33, 0, 40, 0),
    (16, 500, 1, 0, 40, 0),
    (16, 500, 100, 3, 200, 17),
    (40, 200, 90, 2, 300, 5),
    (128, 700, 200, 5, 4000, 100),
    (300, 60, 5, 4, 900, 1),
    (300, 100, 40, 4, 2000, 1),
    (16, 500, 300, 0, 60, 0),   # the pool runs out on the way
    (16, 500, 300, 3, 60, -700),  # so do the rows
]


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("case", range(len(TABLE_CASES)))
def test_tables(case, paged):
    B, hi, new_hi, resets, spare, extra = TABLE_CASES[case]
    rng = random.Random(case)
    length = [rng.randint(0, hi) for _ in range(B)]
    new = [rng.choice([0, 1, rng.randint(0, new_hi)]) if B > 1 else new_hi for _ in range(B)]
    flags = [int(resets and rng.randrange(resets) == 0) for _ in range(B)]
    T = max(1, sum(new) + extra)
    width = pages_of(hi + new_hi) + 1
    check_tables(length, new, flags, T, width, spare, paged, limit=width * PAGE, seed=case)


def check_tables(length, new, flags, T, width, spare, paged, limit, seed, in_place=False):
    B = len(length)
    table, free, n_free, n_pages = make_pool(length, width, spare, seed)
    cfg = mac.config(B, 1, 1, page_size=PAGE if paged else 0, max_context=limit)
    ws = workspace(cfg, T)
    d_table, d_free, d_nf = ints(table), ints(free), ints([n_free])
    d_nf_out = d_nf if in_place else ints([-1])
    d_len, d_new = ints(length), ints(new)
    d_len_out = d_len if in_place else ints([-1] * B)
    q_start, pos, slot = ints([-9] * (B + 1)), ints([-9] * T), ints([-9] * T, torch.int64)
    view = mac.pages_view(d_table, d_free, d_nf, d_nf_out) if paged else mac.pages_view(capacity=width * PAGE)
    mac.mac_build_tables(cfg, ws, view, ints(flags) if any(flags) else None, d_len, d_new, T, d_len_out, q_start, pos, slot)
    want = ref_tables(length, new, flags, T, min(limit, width * PAGE), *((table, free, n_free) if paged else (None, None, 0)),
                      capacity=width * PAGE)
    assert q_start.tolist() == want[1]
    assert d_len_out.tolist() == want[0]
    assert pos.tolist() == want[2]
    assert slot.tolist() == want[3]
    if paged:
        assert d_nf_out.tolist() == [want[4]]
        assert d_table.tolist() == table
        assert d_free.tolist() == free
    assert mac.mac_last_status(cfg, ws) == want[5]
    return want


def test_tables_in_place_and_over_the_limit():
    length, new = [5, 100, 3, 0, 31], [12, 1, -1, 4, 33]
    want = check_tables(length, new, [0, 1, 0, 0, 0], 60, 8, 10, True, limit=63, seed=3, in_place=True)
    assert want[5] == mac.MAC_DEV_BAD_SEQ_LEN  # 100 > 63 (its reset too), -1 new, 31 + 33 > 63
    check_tables([16, 32, 1], [1, 0, 15], [1, 1, 0], 16, 4, 0, True, limit=64, seed=4, in_place=True)


def test_tables_flag_pages_outside_the_cache():
    cfg = mac.config(2, 1, 1, page_size=PAGE, max_context=64)
    ws = workspace(cfg, 8)
    table, free = ints([[99, -1], [0, -1]]), ints([1, 77, -3])
    out = [ints([0, 0]), ints([0] * 3), ints([0] * 8), ints([0] * 8, torch.int64)]
    n_out = ints([0])
    # request 0 goes on on page 99 of 3; request 1 takes the pages 77 (no such page) and -3 from the top
    mac.mac_build_tables(cfg, ws, mac.pages_view(table, free, ints([3]), n_out), None, ints([3, 14]), ints([2, 4]), 8, *out)
    assert mac.mac_last_status(cfg, ws) == mac.MAC_DEV_BAD_PAGE
    assert out[3].tolist() == [-1, -1, 14, 15, -1, -1, -1, -1]
    assert out[1].tolist() == [0, 2, 6] and n_out.tolist() == [2]
    assert table.tolist() == [[99, -1], [0, -1]]
    # a count beyond the stack, and more pages given back than the pool has
    mac.mac_build_tables(cfg, ws, mac.pages_view(table, free, ints([9]), n_out), ints([0, 1]), ints([0, 16]), ints([0, 0]), 8, *out)
    assert mac.mac_last_status(cfg, ws) == mac.MAC_DEV_BAD_PAGE
    assert n_out.tolist() == [3] and free.tolist() == [1, 77, -3] and out[0].tolist() == [0, 0]


# ---------------------------------------------------------------------------
# cache writes
# ---------------------------------------------------------------------------

def ref_rotate(x, pos, mode, base=10000.0):
    """(R(pos) x, |a| + |b| per element) in 64 bits."""
    x = x.double()
    if mode == mac.MAC_ROPE_NONE:
        return x, torch.zeros_like(x)
    w = base ** (-torch.arange(0, D, 2, dtype=torch.float64, device=x.device) / D)
    ang = (pos.double() - 1)[:, None, None] * w
    ia = torch.arange(D // 2, device=x.device) if mode == mac.MAC_ROPE_HALF else torch.arange(0, D, 2, device=x.device)
    ib = ia + D // 2 if mode == mac.MAC_ROPE_HALF else ia + 1
    a, b = x[..., ia], x[..., ib]
    y, z = torch.empty_like(x), torch.empty_like(x)
    y[..., ia], y[..., ib] = a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()
    z[..., ia] = z[..., ib] = a.abs() + b.abs()
    return y, z


def half(dt):
    return torch.finfo(dt).eps / 2


def near(got, want, tol):
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float((got.double() - want).abs().max()), float(tol.max()))


@pytest.mark.parametrize("mode", [mac.MAC_ROPE_HALF, mac.MAC_ROPE_INTERLEAVED, mac.MAC_ROPE_NONE])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("T,Hq,Hkv,paged,fused,with_q", [
    (1, 1, 1, False, False, True), (5, 8, 2, True, True, True), (33, 32, 8, True, False, True),
    (700, 16, 2, False, True, True), (643, 8, 8, True, True, False), (1001, 4, 1, True, False, True)])
def test_write(T, Hq, Hkv, paged, fused, with_q, dt, mode):
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    B, cap = 3, pages_of(T) * PAGE
    n_pages = pages_of(T) + 5
    cfg = mac.config(B, Hq, Hkv, dtype=mac.MAC_BF16 if dt == BF16 else mac.MAC_F32, page_size=PAGE if paged else 0,
                     rope_mode=mode, max_context=1 << 30)
    shape = (n_pages, Hkv, PAGE, D) if paged else (B, Hkv, cap, D)
    kc, vc = (torch.randn(shape, generator=g, device=DEV).to(dt) for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    unit = PAGE if paged else cap
    slot = torch.randperm(shape[0] * unit, generator=g, device=DEV)[:T]
    slot[T // 2] = -1                       # a row that belongs to nobody
    pos = torch.randint(1, 1 << 30, (T,), generator=g, device=DEV, dtype=torch.int32)
    pos[: min(T, 3)] = ints([1, 2, 131072])[: min(T, 3)]
    if fused:
        row = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).to(dt)
        q, k, v = row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:]
    else:
        q, k, v = (torch.randn(T, h, D, generator=g, device=DEV).to(dt) for h in (Hq, Hkv, Hkv))
    q_out = torch.full((T, Hq, D), 7.0, device=DEV, dtype=dt)
    ws = workspace(cfg, T)
    kv = mac.kv_view(kc, vc, ints([[0]])) if paged else mac.kv_view(kc, vc)
    mac.mac_write_kv(cfg, ws, q if with_q else None, k, v, pos, slot, T, kv, q_out if with_q else None)
    assert mac.mac_last_status(cfg, ws) == 0
    live = slot >= 0
    yk, zk = ref_rotate(k, pos, mode)
    want_k, tol_k, want_v = k0.double(), torch.zeros_like(k0.double()), v0.clone()
    s = slot[live]
    want_k[s // unit, :, s % unit] = yk[live]
    rounding = 0.0 if mode == mac.MAC_ROPE_NONE else half(dt)
    tol_k[s // unit, :, s % unit] = (rounding * yk.abs() + 2.0 ** -21 * zk)[live]
    want_v[s // unit, :, s % unit] = v[live]
    near(kc, want_k, tol_k)
    assert torch.equal(vc, want_v)
    if with_q:
        yq, zq = ref_rotate(q, pos, mode)
        near(q_out[live], yq[live], (rounding * yq.abs() + 2.0 ** -21 * zq)[live])
    assert (q_out[~live] == 7).all() and (with_q or (q_out == 7).all())


# bf16 rows past 2048 go two to a CTA; the last CTA of an odd number has one
@pytest.mark.parametrize("mode", [mac.MAC_ROPE_HALF, mac.MAC_ROPE_INTERLEAVED, mac.MAC_ROPE_NONE])
@pytest.mark.parametrize("T,Hq,Hkv,paged,fused,with_q", [
    (2048, 8, 2, True, True, True), (2049, 8, 2, True, False, True), (2501, 12, 3, False, True, True), (4000, 1, 1, True, False, False)])
def test_write_many_rows(T, Hq, Hkv, paged, fused, with_q, mode):
    test_write(T, Hq, Hkv, paged, fused, with_q, BF16, mode)


def test_write_in_place_and_rows_refused_on_the_device():
    cfg = mac.config(1, 8, 2, page_size=PAGE, max_context=4096)
    T = 6
    q, k, v = (torch.randn(T, h, D, device=DEV).to(BF16) for h in (8, 2, 2))
    kc, vc = torch.zeros(2, 2, PAGE, D, device=DEV, dtype=BF16), torch.zeros(2, 2, PAGE, D, device=DEV, dtype=BF16)
    pos, slot = ints([5, 0, 7, 8, -3, 9]), ints([3, 4, 32, 31, 6, 1 << 40], torch.int64)
    ws = workspace(cfg, T)
    out = q.clone()
    ref = torch.zeros_like(q)
    mac.mac_write_kv(cfg, ws, out, k, v, pos, slot, T, mac.kv_view(kc, vc, ints([[0]])), out)
    assert mac.mac_last_status(cfg, ws) == mac.MAC_DEV_BAD_PAGE | mac.MAC_DEV_BAD_SEQ_LEN
    y, z = ref_rotate(q, pos, mac.MAC_ROPE_HALF)
    live = torch.tensor([True, False, False, True, False, False], device=DEV)
    near(out[live], y[live], (2.0 ** -8 * y.abs() + 2.0 ** -21 * z)[live])
    assert torch.equal(out[~live], q[~live])
    written = torch.zeros(2, PAGE, dtype=torch.bool, device=DEV)
    written[0, 3] = written[1, 15] = True
    assert torch.equal((kc != 0).any(-1).any(1), written) and torch.equal((vc != 0).any(-1).any(1), written)
    assert torch.equal(vc[1, :, 15], v[3]) and ref.sum() == 0


# ---------------------------------------------------------------------------
# chunk attention
# ---------------------------------------------------------------------------

class Batch:
    """A cache with `ctx[b] + new[b]` tokens per request and the new tokens' queries."""

    def __init__(self, ctx, new, Hq, Hkv, dt=BF16, paged=True, seed=0, pad=0, fill=float("nan"), scale=1.0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.ctx, self.new, self.Hq, self.Hkv, self.dt, self.paged = ctx, new, Hq, Hkv, dt, paged
        B, total = len(ctx), [c + n for c, n in zip(ctx, new)]
        self.T = sum(new) + pad
        width = pages_of(max(total + [1])) + 1
        self.cap = width * PAGE
        self.start = np.concatenate([[0], np.cumsum(new)]).tolist()
        self.q = (torch.randn(max(self.T, 1), Hq, D, generator=g, device=DEV) * scale).to(dt)
        if pad:
            self.q[sum(new):] = fill
        kk, vv = (torch.randn(B, Hkv, self.cap, D, generator=g, device=DEV).to(dt) for _ in range(2))
        if B:
            kk[0, :, 0] *= 6  # a heavy key
        self.kd, self.vd = kk, vv
        if paged:
            held = [pages_of(n) for n in total]
            n_pages = sum(held) + 3
            ids = torch.randperm(n_pages, generator=g, device=DEV)
            self.table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
            self.k = torch.full((n_pages, Hkv, PAGE, D), fill, device=DEV, dtype=dt)
            self.v = self.k.clone()
            at = 0
            for b, (h, n) in enumerate(zip(held, total)):
                mine = ids[at:at + h]
                self.table[b, :h] = mine.int()
                at += h
                for x, dense in ((self.k, kk), (self.v, vv)):
                    rows = torch.full((Hkv, h * PAGE, D), fill, device=DEV, dtype=dt)
                    rows[:, :n] = dense[b, :, :n]
                    x[mine] = rows.view(Hkv, h, PAGE, D).transpose(0, 1)
            self.kv = mac.kv_view(self.k, self.v, self.table)
        else:
            self.k, self.v = kk.clone(), vv.clone()
            for b, n in enumerate(total):
                self.k[b, :, n:] = fill
                self.v[b, :, n:] = fill
            self.kv = mac.kv_view(self.k, self.v)
        self.cfg = mac.config(B, Hq, Hkv, dtype=mac.MAC_BF16 if dt == BF16 else mac.MAC_F32, page_size=PAGE if paged else 0,
                              max_context=self.cap)
        self.q_start, self.seq_len = ints(self.start), ints(total)
        self.ws = workspace(self.cfg, max(self.T, 1))
        self.out = torch.full((max(self.T, 1), Hq, D), 7.0, device=DEV, dtype=dt)
        self.lse = torch.full((max(self.T, 1), Hq), 7.0, device=DEV)

    def run(self, stream=None, lse=True):
        mac.mac_chunk_attention(self.cfg, self.ws, self.q, self.q_start, self.seq_len, self.T, self.kv, self.out,
                                self.lse if lse else None, stream)

    def status(self):
        return mac.mac_last_status(self.cfg, self.ws)

    def check(self, drop=None):
        """Compare with 64 bits; drop[b]: 0-based positions that are left out."""
        G = self.Hq // self.Hkv
        for b, (c, n) in enumerate(zip(self.ctx, self.new)):
            for lo in range(0, n, 512):
                hi = min(n, lo + 512)
                rows = slice(self.start[b] + lo, self.start[b] + hi)
                seen = c + hi
                k, v = (x[b, :, :seen].double().repeat_interleave(G, 0) for x in (self.kd, self.vd))
                q = self.q[rows].double().transpose(0, 1)
                late = torch.arange(seen, device=DEV)[None] > torch.arange(c + lo, c + hi, device=DEV)[:, None]
                if drop and drop.get(b):
                    late = late.clone()
                    late[:, [x for x in drop[b] if x < seen]] = True
                x = (q @ k.transpose(1, 2) / math.sqrt(D)).masked_fill(late, -math.inf)
                big = (q.abs() @ k.abs().transpose(1, 2)).amax(-1) / math.sqrt(D)
                lse = torch.logsumexp(x, -1)
                w = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
                want, A = (w @ v).transpose(0, 1), (w @ v.abs()).transpose(0, 1)
                bf = self.dt == BF16
                e = (D + 4) * 2.0 ** -24 * big * (4 if bf else 1)
                rest = (seen + 64) * 2.0 ** -24
                tol = A * (2 * e + rest).t()[..., None]
                if bf:
                    tol = tol + 2.0 ** -8 * (A + want.abs())
                near(self.out[rows], want, tol)
                got = self.lse[rows].double().t()
                assert torch.equal(got == -math.inf, lse == -math.inf)
                fine = lse > -math.inf
                near(got[fine], lse[fine], (e + rest + 2.0 ** -22 * lse.abs())[fine])
        end = self.start[-1]
        assert (self.out[end:] == 7).all() and (self.lse[end:] == 7).all()  # rows behind the last sequence


LENGTHS = [
    ([0], [1]), ([0], [2]), ([15], [1]), ([16], [1]), ([127], [1]), ([128], [1]), ([0], [128]), ([0], [129]), ([1], [127]),
    ([63], [65]), ([100], [7]), ([0], [300]), ([1000], [33]), ([2047], [257]), ([5000], [1]),
    ([0, 31, 500, 7, 1200], [1, 0, 64, 3, 130]), ([0, 0, 0], [0, 1, 0]), ([300] * 8, [1] * 8),
]


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (2, 2), (2, 1), (16, 2)])
@pytest.mark.parametrize("lengths", range(len(LENGTHS)))
def test_chunk(lengths, Hq, Hkv, dt, paged):
    # rows of the cache beyond the lengths, and queries of rows that belong to nobody, are NaN
    ctx, new = LENGTHS[lengths]
    b = Batch(ctx, new, Hq, Hkv, dt, paged, seed=lengths, pad=lengths % 3)
    b.run()
    assert b.status() == 0
    b.check()


@pytest.mark.parametrize("dt,Hq,Hkv,ctx,new,paged", [
    (BF16, 32, 8, [3000, 0, 9000], [1500, 2049, 17], True),      # many units, whole and cut
    (BF16, 32, 4, [20000], [1], True),                           # one row over every CTA
    (BF16, 4, 4, [131071, 70], [1, 1], False),
    (BF16, 1, 1, [0], [4096], False),
    (BF16, 8, 2, [30000], [64], True),                           # whole row tiles in many pieces
    (BF16, 1, 1, [40000], [3], False),                           # more pieces than a warp has lanes
    (F32, 8, 2, [3000, 10], [500, 700], True),
    (F32, 8, 2, [9000], [40], True),
    (F32, 1, 1, [20000], [2], False),
    (F32, 1, 1, [4096], [64], False)])
def test_chunk_over_many_ctas(dt, Hq, Hkv, ctx, new, paged):
    b = Batch(ctx, new, Hq, Hkv, dt, paged, seed=5)
    b.run()
    assert b.status() == 0
    b.check()
    first = b.out.clone(), b.lse.clone()
    for _ in range(3):  # the order of the sums does not depend on timing
        b.out.fill_(7)
        b.lse.fill_(7)
        b.run()
        assert torch.equal(b.out, first[0]) and torch.equal(b.lse, first[1])
    b.run(lse=False)
    assert torch.equal(b.out, first[0])


@pytest.mark.parametrize("dt", [BF16, F32])
def test_chunk_several_pieces_per_cta_many_times(dt):
    # the products run ahead into a CTA's next piece while the last one's rows are written
    b = Batch([2000, 700] * 8, [1, 40] * 8, 32, 8, dt, True, seed=12)
    b.run()
    b.check()
    ref = b.out.clone()
    for _ in range(60):
        b.run()
    assert b.status() == 0 and torch.equal(b.out, ref)


@pytest.mark.parametrize("seed", range(16))
def test_chunk_drawn(seed):
    rng = random.Random(seed)
    Hq, Hkv = rng.choice([(8, 8), (8, 4), (8, 2), (16, 2), (1, 1), (24, 3)])
    B = rng.randint(1, 9)
    hi, n = rng.choice([10, 200, 3000, 9000]), rng.choice([1, 4, 70, 600])
    new = [rng.choice([0, 1, rng.randint(0, n)]) for _ in range(B)]
    new[0] = max(new[0], 1)
    b = Batch([rng.randint(0, hi) for _ in range(B)], new, Hq, Hkv, rng.choice([BF16, F32]), rng.random() < 0.5,
              seed=seed, pad=rng.randint(0, 3))
    b.run()
    assert b.status() == 0
    b.check()


# 129 to 256 rows per request and head: one unit or two of half the rows, by the number of SMs
@pytest.mark.parametrize("Hq,Hkv,new", [
    (4, 1, [33] * (torch.cuda.get_device_properties(0).multi_processor_count // 2 if torch.cuda.is_available() else 1)),
    (4, 1, [33] * (torch.cuda.get_device_properties(0).multi_processor_count // 2 + 1 if torch.cuda.is_available() else 1)),
    (8, 2, [64, 32, 65, 0, 33, 63]), (2, 2, [129, 256, 257, 1]), (16, 2, [17, 32, 33])])
def test_chunk_units_of_half_the_rows(Hq, Hkv, new):
    b = Batch([(i * 97) % 500 for i in range(len(new))], new, Hq, Hkv, BF16, True, seed=6, pad=2)
    b.run()
    assert b.status() == 0
    b.check()


# a CTA for every unit; units of many tiles, alike (taken whole) and very unlike (cut)
@pytest.mark.parametrize("dt,Hq,Hkv,ctx,new", [
    (BF16, 32, 8, [1200] * 12, [60] * 12), (BF16, 32, 8, [3000, 10, 0, 700], [60, 64, 1, 65]), (BF16, 8, 8, [2500] * 16, [1] * 16),
    (F32, 4, 2, [700] * 16, [60] * 16), (F32, 8, 2, [2000, 5, 64, 300], [20, 32, 1, 33])])
def test_chunk_a_cta_for_each_unit(dt, Hq, Hkv, ctx, new):
    b = Batch(ctx, new, Hq, Hkv, dt, True, seed=8, pad=1)
    b.run()
    assert b.status() == 0
    b.check()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_chunk_many_requests(dt):
    rng = random.Random(1)
    B = 256
    b = Batch([rng.randint(0, 90) for _ in range(B)], [rng.choice([0, 1, 1, 5, 40]) for _ in range(B)], 4, 2, dt, True, seed=2, pad=3)
    b.run()
    assert b.status() == 0
    b.check()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_chunk_large_scores(dt):
    # scores of a few hundred: the running maximum has to move, nothing overflows
    b = Batch([700, 64], [130, 64], 8, 2, dt, True, seed=3, scale=30.0)
    b.run()
    assert b.status() == 0
    b.check()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_chunk_leaves_out_bad_pages(dt):
    b = Batch([40, 16, 500], [30, 3, 40], 8, 2, dt, True, seed=4)
    b.table[0, 0] = -1            # request 0: tokens 0..15; row by row it still has others
    b.table[0, 4] = 1 << 20       # tokens 64..69, its last page
    b.table[1, :2] = -5           # request 1 has nothing left
    b.table[2, 7:20] = 9999
    b.run()
    assert b.status() == mac.MAC_DEV_BAD_PAGE
    drop = {0: list(range(16)) + list(range(64, 70)), 1: list(range(19)), 2: list(range(112, 320))}
    b.check(drop)
    rows = slice(b.start[1], b.start[2])
    assert (b.out[rows] == 0).all() and (b.lse[rows] == -math.inf).all()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_chunk_bad_lengths(dt):
    b = Batch([40, 16, 50, 5], [30, 3, 40, 2], 8, 2, dt, True, seed=4)
    good = b.seq_len.clone()
    b.seq_len[1] = 2                      # below its three new tokens
    b.seq_len[2] = b.cap + 1              # beyond the table
    b.run()
    assert b.status() == mac.MAC_DEV_BAD_SEQ_LEN
    rows = slice(b.start[1], b.start[3])
    assert (b.out[rows] == 0).all() and (b.lse[rows] == -math.inf).all()
    assert b.status() == 0
    kept = [0, 3]
    for i in kept:
        assert (b.lse[b.start[i]:b.start[i + 1]] > -math.inf).all()
    b.seq_len.copy_(good)
    b.out.fill_(7)
    b.lse.fill_(7)
    b.q_start.copy_(ints([0, 30, 33, 1000, 75]))  # requests 2 and 3 point outside the batch
    b.run()
    assert b.status() == mac.MAC_DEV_BAD_SEQ_LEN
    assert (b.out[33:] == 7).all() and (b.lse[:33] > -math.inf).all()


@pytest.mark.parametrize("dt,ctx,T,B", [(BF16, 1128, 1024, 12), (F32, 280, 280, 16)])
def test_chunk_requests_that_claim_the_same_rows(dt, ctx, T, B):
    # a q_start that goes back is reported; a request whose rows nobody else claims is right all the same,
    # also where the lengths need more units than n_tokens rows in order could
    b = Batch([ctx] + [0] * (B - 1), [24] + [0] * (B - 1), 8, 8, dt, False, seed=13, pad=T)
    b.cfg.max_context = ctx + 24
    b.run()
    assert b.status() == 0
    b.check()
    b.q_start.copy_(ints([0] + [24, 24 + T] * (B // 2)))
    b.seq_len.copy_(ints([ctx + 24] + [T] * (B - 1)))
    for x in (b.k, b.v):  # the other requests' tokens
        x[1:] = 0
    b.out.fill_(7)
    b.lse.fill_(7)
    b.run()
    assert b.status() == mac.MAC_DEV_BAD_SEQ_LEN
    b.out[24:] = 7
    b.lse[24:] = 7
    b.check()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_chunk_infinite_and_nan_rows_stay_in_their_row(dt):
    b = Batch([100], [70], 8, 2, dt, True, seed=6)
    b.run()
    ref = b.out.clone()
    b.q[13, 3] = float("nan")
    b.q[14, 5, 0] = float("inf")
    b.run()
    keep = torch.ones(70, 8, dtype=torch.bool, device=DEV)
    keep[13, 3] = keep[14, 5] = False
    assert torch.equal(b.out[keep], ref[keep])
    assert b.out[13, 3].isnan().all() and not ref.isnan().any()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_chunk_infinite_and_nan_keys_not_yet_attended(dt):
    # a key that later rows of the same chunk attend may be anything for the rows before it
    b = Batch([100], [70], 8, 2, dt, False, seed=6)
    b.run()
    ref = b.out.clone()
    for bad in (float("nan"), float("inf"), float("-inf")):
        b.k[0, :, 140] = bad  # position 141: rows 40 and on
        b.run()
        assert torch.equal(b.out[:40], ref[:40])


def test_chunk_an_infinite_key_weighs_nothing_or_all():
    # scores of -inf leave a key out; those of +inf make the row NaN, as inf - inf does
    b = Batch([40], [1], 2, 1, BF16, False, seed=7)
    b.q.zero_()
    b.q[0, 0, 5], b.q[0, 1, 5] = 1.0, -1.0
    b.k[0, 0, 17] = 0
    b.k[0, 0, 17, 5] = float("-inf")
    b.run()
    x = (b.kd[0, 0, :41, 5].double() / math.sqrt(D)).where(torch.arange(41, device=DEV) != 17, -math.inf)
    w = torch.softmax(x, 0)
    want, A = w @ b.vd[0, 0, :41].double(), w @ b.vd[0, 0, :41].double().abs()
    near(b.out[0, 0], want, 2.0 ** -8 * (A + want.abs()) + 2.0 ** -14 * A)
    assert b.out[0, 1].isnan().all()


@pytest.mark.parametrize("new", [1, 200])
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("use", [0, 1])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_chunk_wait_runs_out(dt, use, paged, new):
    # key stage use `use` is never filled: the wait for it gives up after 2^16 cycles, the launch reports
    # it and returns, and one on a fresh workspace is clean and right
    b = Batch([3000, 1500], [new, new], 8, 2, dt, paged, seed=9)
    mac.mac_test_wait_budget(1 << 16, use)
    b.run()
    torch.cuda.synchronize()
    assert b.status() & mac.MAC_DEV_WAIT_TIMEOUT
    b.ws = workspace(b.cfg, b.T)
    b.run()
    assert b.status() == 0
    b.check()


@pytest.mark.parametrize("dt,Hq,Hkv,ctx,new", [
    (BF16, 8, 2, [80001] * 8, [30] * 8),     # one warp waits for a piece's last value tile, to clear its end
    (F32, 4, 4, [1500] * 250, [2] * 250)])   # and for room for the next pieces, several ahead
def test_chunk_pieces_longer_than_any_wait(dt, Hq, Hkv, ctx, new):
    # no copy or product takes 2^16 cycles, but a piece of 60 tiles (bf16) or 24 (fp32) does: nothing has run out
    b = Batch(ctx, new, Hq, Hkv, dt, False, seed=11)
    mac.mac_test_wait_budget(1 << 16, -1)
    b.run()
    assert b.status() == 0
    b.check()


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("use", [-1, 0, 2])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_chunk_gives_up_at_once_with_work_in_flight(dt, use, paged):
    # a budget of one cycle: every wait that is not over already gives up while copies and products that were
    # issued are in flight.  The launch returns when those have ended, so the launches right behind it, on
    # workspaces of their own, find shared memory and TMEM free and are right.
    b = Batch([3000, 700, 90], [200, 1, 64], 8, 2, dt, paged, seed=10)
    b.run()
    assert b.status() == 0
    b.check()
    ref, bad = b.out.clone(), workspace(b.cfg, b.T)
    good = b.ws
    for _ in range(10):
        b.ws = bad
        bad.zero_()
        mac.mac_test_wait_budget(1, use)
        b.run()
        b.ws = good
        b.run()
        assert torch.equal(b.out, ref) and b.status() == 0
        if use >= 0:
            assert mac.mac_last_status(b.cfg, bad) & mac.MAC_DEV_WAIT_TIMEOUT


def test_chunk_output_on_any_16_byte_boundary():
    b = Batch([50], [70], 8, 2, BF16, True, seed=6)
    b.run()
    ref = b.out.clone()
    raw = torch.zeros(b.out.numel() + 64, device=DEV, dtype=BF16)
    for off in (8, 24):  # rows start at odd multiples of 16 bytes
        b.out = raw[off:off + ref.numel()].view(ref.shape)
        b.run()
        assert torch.equal(ref, b.out)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [BF16, F32])
def test_streams_and_graphs(dt):
    # captured on another stream, replayed with new lengths and inputs in the same buffers
    a, c = Batch([300, 40], [20, 31], 8, 2, dt, True, seed=1), Batch([10, 600], [50, 1], 8, 2, dt, True, seed=2)
    T = 51
    s = torch.cuda.Stream()
    q, q_start, seq = a.q.clone(), a.q_start.clone(), a.seq_len.clone()
    kk, vv = torch.zeros(64, 2, PAGE, D, device=DEV, dtype=dt), torch.zeros(64, 2, PAGE, D, device=DEV, dtype=dt)
    table = torch.full((2, 64), -1, dtype=torch.int32, device=DEV)
    cfg = mac.config(2, 8, 2, dtype=a.cfg.dtype, page_size=PAGE, max_context=1024)
    ws, out, lse = workspace(cfg, T), torch.zeros_like(a.out), torch.zeros_like(a.lse)
    kv = mac.kv_view(kk, vv, table)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mac.mac_chunk_attention(cfg, ws, q, q_start, seq, T, kv, out, lse, torch.cuda.current_stream())
    for x in (a, c, a):
        x.run()
        q.copy_(x.q)
        q_start.copy_(x.q_start)
        seq.copy_(x.seq_len)
        kk[:x.k.shape[0]] = x.k
        vv[:x.v.shape[0]] = x.v
        table.fill_(-1)
        table[:, :x.table.shape[1]] = x.table
        g.replay()
        torch.cuda.synchronize()
        # the pool's size is part of the captured call; pages beyond x's are not in its table
        assert torch.equal(out, x.out) and torch.equal(lse, x.lse)
    with torch.cuda.stream(s):
        a.out.fill_(7)
        a.run(s)
    s.synchronize()
    a.check()


@pytest.mark.parametrize("dt,paged", [(BF16, True), (BF16, False), (F32, True)])
def test_prompts_in_chunks_then_decode(dt, paged):
    """Prompts of two requests enter in chunks beside a third that already decodes; one request's
    slot is then reset and takes a new prompt; decode steps follow on the cache the calls built.
    Everything is compared with attention in 64 bits over the rotated keys of the whole history."""
    Hq, Hkv, B, room = 8, 2, 3, 512
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    n_pages = 3 * room // PAGE
    cfg = mac.config(B, Hq, Hkv, ring_k=32, band_r=16, dtype=mac.MAC_BF16 if dt == BF16 else mac.MAC_F32,
                     page_size=PAGE if paged else 0, max_context=room)
    shape = (n_pages, Hkv, PAGE, D) if paged else (B, Hkv, room, D)
    kc, vc = (torch.full(shape, float("nan"), device=DEV, dtype=dt) for _ in range(2))
    table = torch.full((B, room // PAGE), -1, dtype=torch.int32, device=DEV)
    free, n_free = torch.randperm(n_pages, generator=g, device=DEV).int(), ints([n_pages])
    pages = mac.pages_view(table, free, n_free) if paged else mac.pages_view(capacity=room)
    kv = mac.kv_view(kc, vc, table) if paged else mac.kv_view(kc, vc)
    length = ints([0] * B)
    T = 160
    ws = workspace(cfg, T)
    hist = [[torch.zeros(0, Hkv, D, device=DEV, dtype=dt)] * 2 for _ in range(B)]
    flags = ints([0] * B)
    layer = mac.MacLayer(cfg, device=DEV)
    mac.mac_init_rings(cfg, layer.ring, layer.scratch, None, None, 0, None)
    steps = [([100, 0, 20], []), ([33, 127, 0], []), ([1, 1, 140], []), ([90, 1, 1], [0]), ([1, 1, 1], []), ([1, 1, 1], [])]
    for new, reset in steps:
        for r in reset:
            flags[r] = 1
            hist[r] = [torch.zeros(0, Hkv, D, device=DEV, dtype=dt)] * 2
        q, k, v = (torch.randn(T, h, D, generator=g, device=DEV).to(dt) for h in (Hq, Hkv, Hkv))
        q_start, pos, slot = ints([0] * (B + 1)), ints([0] * T), ints([0] * T, torch.int64)
        q_rot, out, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(T, Hq, device=DEV)
        mac.mac_build_tables(cfg, ws, pages, flags, length, ints(new), T, length, q_start, pos, slot)
        mac.mac_reset_requests(cfg, layer.ring, flags)
        mac.mac_write_kv(cfg, ws, q, k, v, pos, slot, T, kv, q_rot)
        mac.mac_chunk_attention(cfg, ws, q_rot, q_start, length, T, kv, out, lse)
        start = np.concatenate([[0], np.cumsum(new)]).tolist()
        assert q_start.tolist() == start and flags.tolist() == [0] * B
        if new == [1] * B:  # the decode step rotates its own queries and attends the same cache
            o2 = torch.zeros(B, Hq, D, device=DEV)
            mp = ints([[0] * Hq] * B)
            mac.mac_decode_step(cfg, layer.ring, layer.scratch, q[:B].contiguous(), length, kv, o2, mp)
        for b in range(B):
            rows = slice(start[b], start[b + 1])
            hist[b] = [torch.cat([hist[b][0], k[rows]]), torch.cat([hist[b][1], v[rows]])]
            n, tot = new[b], hist[b][0].shape[0]
            assert length.tolist()[b] == tot
            if not n:
                continue
            p = torch.arange(1, tot + 1, device=DEV)
            kr = ref_rotate(hist[b][0], p, mac.MAC_ROPE_HALF)[0].to(dt).double().repeat_interleave(4, 1)
            vr = hist[b][1].double().repeat_interleave(4, 1)
            qr = ref_rotate(q[rows], p[tot - n:], mac.MAC_ROPE_HALF)[0].to(dt).double()
            x = torch.einsum("qhd,khd->hqk", qr, kr) / math.sqrt(D)
            late = p[None] > p[tot - n:, None]
            w = torch.softmax(x.masked_fill(late, -math.inf), -1)
            want, A = torch.einsum("hqk,khd->qhd", w, vr), torch.einsum("hqk,khd->qhd", w, vr.abs())
            # bf16: a key or query element whose rotation lies next to a rounding border may round the other
            # way, moving a score by up to 2^-8 |q k|: ten such elements of size 3 move it by 0.03
            tol = (2.0 ** -8 * (2 * A + want.abs()) + 0.06 * A) if dt == BF16 else 1e-4 * A
            near(out[rows], want, tol)
            if new == [1] * B and (mp[b] < 0).all():
                near(o2[b], want[0], tol[0])
    assert mac.mac_last_status(cfg, ws) == 0 and mac.mac_last_status(cfg, layer.scratch) == 0
    if paged:
        held = sum(pages_of(n) for n in length.tolist())
        assert n_free.tolist() == [n_pages - held]
    layer.release()


@pytest.mark.parametrize("how", ["eager", "graph"])
@pytest.mark.parametrize("dt,Hq,Hkv,paged", [(BF16, 8, 2, True), (BF16, 8, 2, False), (BF16, 16, 2, True), (F32, 4, 4, True)])
def test_keys_and_values_then_decode_steps_of_several_layers(dt, Hq, Hkv, paged, how):
    """A decode step of a model: pages and slots once, then per layer the new token's key and value (no query: the
    step rotates its own) and the step, one behind the other with nothing in between.  It has to leave what the same
    calls leave with the device idle before each."""
    B, layers, steps, room = 5, 4, 14, 512
    g = torch.Generator(device=DEV)
    g.manual_seed(12)
    n_pages = B * room // PAGE
    cfg = mac.config(B, Hq, Hkv, ring_k=32, band_r=16, dtype=mac.MAC_BF16 if dt == BF16 else mac.MAC_F32,
                     page_size=PAGE if paged else 0, max_context=room)
    shape = (n_pages, Hkv, PAGE, D) if paged else (B, Hkv, room, D)
    start = [300, 17, 0, 255, 495]
    cache = [torch.randn(shape, generator=g, device=DEV).to(dt) for _ in range(2 * layers)]
    base = torch.randn(layers, B, Hq, D, generator=g, device=DEV)
    ids = torch.randperm(n_pages, generator=g, device=DEV).int()

    class Model:
        def __init__(self):
            self.cache = [x.clone() for x in cache]
            self.table = torch.full((B, room // PAGE), -1, dtype=torch.int32, device=DEV)
            self.n_free, self.free, at = ints([0]), ids.clone(), n_pages
            for b, n in enumerate(start):
                at -= pages_of(n)
                self.table[b, :pages_of(n)] = ids[at:at + pages_of(n)]
            self.n_free.fill_(at)
            self.pages = mac.pages_view(self.table, self.free, self.n_free) if paged else mac.pages_view(capacity=room)
            self.length, self.new = ints(start), ints([1] * B)
            self.q_start, self.pos, self.slot = ints([0] * (B + 1)), ints([0] * B), ints([0] * B, torch.int64)
            self.ws = workspace(cfg, B)
            self.layers = [mac.MacLayer(cfg, device=DEV) for _ in range(layers)]
            self.q = [torch.zeros(B, Hq, D, device=DEV, dtype=dt) for _ in range(layers)]
            self.kv = [torch.zeros(B, 2 * Hkv, D, device=DEV, dtype=dt) for _ in range(layers)]
            self.out = [torch.zeros(B, Hq, D, device=DEV) for _ in range(layers)]
            self.match = [ints([[0] * Hq] * B) for _ in range(layers)]
            for x in self.layers:
                mac.mac_init_rings(cfg, x.ring, x.scratch, None, None, 0, None)

        def inputs(self, step):
            g = torch.Generator(device=DEV)
            g.manual_seed(1000 + step)
            for i in range(layers):
                noise = torch.randn(B, Hq, D, generator=g, device=DEV)
                self.q[i].copy_(base[i] + (0.02 if step % 3 else 1.0) * noise)
                self.kv[i].copy_(torch.randn(B, 2 * Hkv, D, generator=g, device=DEV))

        def step(self, stream, wait=lambda: None):
            mac.mac_build_tables(cfg, self.ws, self.pages, None, self.length, self.new, B, self.length, self.q_start, self.pos,
                                 self.slot, stream)
            for i, x in enumerate(self.layers):
                view = mac.kv_view(*self.cache[2 * i:2 * i + 2], self.table if paged else None)
                wait()
                mac.mac_write_kv(cfg, self.ws, None, self.kv[i][:, :Hkv], self.kv[i][:, Hkv:], self.pos, self.slot, B, view, None,
                                 stream)
                wait()
                mac.mac_decode_step(cfg, x.ring, x.scratch, self.q[i], self.length, view, self.out[i], self.match[i], stream)
                wait()

    apart, close = Model(), Model()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    if how == "graph":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            close.step(torch.cuda.current_stream())
    hits = 0
    for step in range(steps):
        apart.inputs(step)
        close.inputs(step)
        torch.cuda.synchronize()
        apart.step(s, torch.cuda.synchronize)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay() if how == "graph" else close.step(s)
        torch.cuda.synchronize()
        assert close.length.tolist() == [n + step + 1 for n in start] and torch.equal(close.slot, apart.slot)
        for i in range(layers):
            assert torch.equal(close.match[i], apart.match[i])
            assert torch.equal(close.out[i], apart.out[i])
            hits += int((close.match[i] >= 0).sum())
    assert hits > 0
    for a, c in zip(apart.cache, close.cache):
        assert torch.equal(a, c)
    for m in (apart, close):
        assert mac.mac_last_status(cfg, m.ws) == 0
        for x in m.layers:
            assert mac.mac_last_status(cfg, x.scratch) == 0
            x.release()


# ---------------------------------------------------------------------------
# many requests: more than a CTA has threads, and as many as a table call takes
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("B", [385, 513, 1024])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("G", [1, 4])
def test_chunk_more_requests_than_threads(dt, B, G):
    # the plan's last trip holds the long requests, or the only ones; empty ones and single tokens before them
    for sparse in (False, True):
        ctx, new = [0 if sparse else b % 7 for b in range(B)], [0 if sparse else int(b % 3 == 0) for b in range(B)]
        ctx[B - 1], new[B - 1] = 900, 70
        if B > 513:
            ctx[520:523], new[520:523] = [400, 0, 5], [1, 130, 0]
        b = Batch(ctx, new, G, 1, dt, True, seed=B, pad=1)
        b.run()
        assert b.status() == 0
        b.check()


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("B,rows", [(1023, 1000), (1024, 1024), (1023, 1025), (1024, 3000)])
def test_tables_of_as_many_requests_as_there_may_be(B, rows, paged):
    rng = random.Random(B + rows)
    length = [rng.randint(0, 70) for _ in range(B)]
    new = [rng.choice([0, 1, rows // B * 2]) for _ in range(B)]
    while sum(new) > rows - 3:
        new[rng.randrange(B)] = 0
    new[B - 1] = rows - 3 - sum(new[:-1]) if paged else new[B - 1]  # the last request takes what is left, but three rows
    flags = [int(rng.randrange(4) == 0) for _ in range(B)]
    width = pages_of(70 + max(new)) + 1
    assert check_tables(length, new, flags, rows, width, 6000, paged, limit=width * PAGE, seed=B)[5] == 0


def test_write_leaves_skipped_rows_and_other_slots_alone():
    # every third row is skipped: by a negative slot, one beyond the cache or a position below 1, in CTAs of one and
    # of two rows.  What they would have written, and every slot that no row names, keeps what it held.
    for T in (50, 2100):
        cfg = mac.config(1, 4, 2, page_size=PAGE, max_context=4096)
        n_pages = pages_of(T) + 2
        q, k, v = (torch.randn(T, h, D, device=DEV).to(BF16) for h in (4, 2, 2))
        kc, vc = (torch.randn(n_pages, 2, PAGE, D, device=DEV).to(BF16) for _ in range(2))
        k0, v0, t = kc.clone(), vc.clone(), torch.arange(T, device=DEV)
        slot, pos = torch.randperm(n_pages * PAGE, device=DEV)[:T], (t % 900 + 1).int()
        named = slot.clone()
        slot[t % 9 == 2], slot[t % 9 == 5] = -1, n_pages * PAGE
        pos[t % 9 == 8] = 0
        live = t % 3 != 2
        out, ws = torch.full_like(q, 7.0), workspace(cfg, T)
        mac.mac_write_kv(cfg, ws, q, k, v, pos, slot, T, mac.kv_view(kc, vc, ints([[0]])), out)
        assert mac.mac_last_status(cfg, ws) == mac.MAC_DEV_BAD_PAGE | mac.MAC_DEV_BAD_SEQ_LEN
        assert (out[~live] == 7).all() and (out[live] != 7).any(-1).all()
        kept = torch.ones(n_pages * PAGE, dtype=torch.bool, device=DEV)
        kept[named[live]] = False
        rows = lambda x: x.transpose(1, 2).flatten(0, 1)  # noqa: E731
        assert torch.equal(rows(kc)[kept], rows(k0)[kept]) and torch.equal(rows(vc)[kept], rows(v0)[kept])
        assert torch.equal(rows(vc)[named[live]], v[live])


def test_chunk_fp32_rows_that_attend_an_infinite_key_are_nan_and_no_others():
    # an infinity has no sum of three finite parts: whatever the score, the row says so
    for bad in (float("inf"), -float("inf")):
        b = Batch([100], [70], 8, 2, F32, True, seed=6)
        b.run()
        ref = b.out.clone()
        b.k[b.table[0, 140 // PAGE].long(), 1, 140 % PAGE, 5] = bad  # position 141 of KV head 1: rows 40 and on of heads 4 to 7
        b.run()
        assert b.out[40:, 4:].isnan().all()
        assert torch.equal(b.out[:40], ref[:40]) and torch.equal(b.out[:, :4], ref[:, :4])


# ---------------------------------------------------------------------------
# large offsets, calls at once
# ---------------------------------------------------------------------------

def attend(q, k, v, first):
    """Rows q [n, H, D] at positions first, first + 1, .. (0-based) over k, v [Hkv, seen, D], in 64 bits: out, A = sum P |v|."""
    G = q.shape[1] // k.shape[0]
    q, k, v = q.double().transpose(0, 1), k.double().repeat_interleave(G, 0), v.double().repeat_interleave(G, 0)
    late = torch.arange(k.shape[1], device=DEV)[None] > torch.arange(first, first + q.shape[1], device=DEV)[:, None]
    w = torch.softmax((q @ k.transpose(1, 2) / math.sqrt(D)).masked_fill(late, -math.inf), -1)
    return (w @ v).transpose(0, 1), (w @ v.abs()).transpose(0, 1)


def attention_tol(want, A, dt):
    # up to 4200 normal keys: sum |q k| <= 120, e = (D + 4) 2^-24 120 / sqrt(D) = 2^-13.5 (four times that in bf16), and
    # (n + 64) 2^-24 = 2^-12: 2 e + that is below 2^-10 and 2^-11
    return (2.0 ** -10 * A + 2.0 ** -8 * (A + want.abs())) if dt == BF16 else 2.0 ** -11 * A


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_caches_beyond_32_bit_offsets(dt, paged):
    # keys and values of the last request and of page ids at the pool's end lie past element 2^32
    Hq, Hkv, B, n, ctx = 8, 4, 2, 40, 300
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    total, held = ctx + n, pages_of(ctx + n)
    cap = (1 << 32) // (B * Hkv * D) // PAGE * PAGE + 40000 * PAGE
    n_pages = (1 << 32) // (Hkv * PAGE * D) + 3 * held
    shape = (n_pages, Hkv, PAGE, D) if paged else (B, Hkv, cap, D)
    kc, vc = (torch.empty(shape, device=DEV, dtype=dt) for _ in range(2))
    cfg = mac.config(B, Hq, Hkv, dtype=mac.MAC_BF16 if dt == BF16 else mac.MAC_F32, page_size=PAGE if paged else 0,
                     rope_mode=mac.MAC_ROPE_NONE, max_context=cap if not paged else 4096)
    table = ints([list(range(held)), list(range(n_pages - 1, n_pages - 1 - held, -1))]) if paged else None
    pos = torch.arange(total, device=DEV)
    slot = torch.cat([(table[b, pos // PAGE].long() * PAGE + pos % PAGE) if paged else b * cap + pos for b in range(B)])
    assert kc.numel() > 1 << 32
    T = B * total
    q, k, v = (torch.randn(T, h, D, generator=g, device=DEV).to(dt) for h in (Hq, Hkv, Hkv))
    ws = workspace(cfg, T)
    kv = mac.kv_view(kc, vc, table) if paged else mac.kv_view(kc, vc)
    mac.mac_write_kv(cfg, ws, None, k, v, pos.repeat(B).int() + 1, slot, T, kv, None)
    for b in range(B):
        for x, new in ((kc, k), (vc, v)):
            rows = x[table[b, pos // PAGE].long(), :, pos % PAGE] if paged else x[b, :, :total].transpose(0, 1)
            assert torch.equal(rows, new[b * total:(b + 1) * total])
    qn = torch.cat([q[(b + 1) * total - n:(b + 1) * total] for b in range(B)])
    out, lse = torch.zeros_like(qn), torch.zeros(B * n, Hq, device=DEV)
    mac.mac_chunk_attention(cfg, ws, qn, ints([0, n, 2 * n]), ints([total] * B), B * n, kv, out, lse)
    assert mac.mac_last_status(cfg, ws) == 0
    for b in range(B):
        want, A = attend(qn[b * n:(b + 1) * n], *(x[b * total:(b + 1) * total].transpose(0, 1) for x in (k, v)), ctx)
        near(out[b * n:(b + 1) * n], want, attention_tol(want, A, dt))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_rows_beyond_32_bit_offsets(dt):
    # queries, outputs and a fused projection's rows past element 2^31
    B, Hq, Hkv, n = 64, 64, 16, 4200
    T = B * n
    assert T * Hq * D > 1 << 31
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    cfg = mac.config(B, Hq, Hkv, dtype=mac.MAC_BF16 if dt == BF16 else mac.MAC_F32, page_size=PAGE, rope_mode=mac.MAC_ROPE_NONE,
                     max_context=n + PAGE)
    fused = torch.empty(T, Hq + 2 * Hkv, D, device=DEV, dtype=dt).normal_(generator=g)
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    n_pages = B * pages_of(n)
    kc, vc = (torch.empty(n_pages, Hkv, PAGE, D, device=DEV, dtype=dt) for _ in range(2))
    table = torch.zeros(B, pages_of(n) + 1, dtype=torch.int32, device=DEV)
    free, n_free = torch.randperm(n_pages, generator=g, device=DEV).int(), ints([n_pages])
    length, q_start, pos, slot = ints([0] * B), ints([0] * (B + 1)), ints([0] * T), ints([0] * T, torch.int64)
    ws, kv = workspace(cfg, T), mac.kv_view(kc, vc, table)
    rows, out = (torch.empty(T, Hq, D, device=DEV, dtype=dt) for _ in range(2))
    lse = torch.zeros(T, Hq, device=DEV)
    mac.mac_build_tables(cfg, ws, mac.pages_view(table, free, n_free), None, length, ints([n] * B), T, length, q_start, pos, slot)
    mac.mac_write_kv(cfg, ws, q, k, v, pos, slot, T, kv, rows)
    mac.mac_chunk_attention(cfg, ws, rows, q_start, length, T, kv, out, lse)
    assert mac.mac_last_status(cfg, ws) == 0 and n_free.tolist() == [0]
    for lo in range(0, T, 1 << 15):
        assert torch.equal(rows[lo:lo + (1 << 15)], q[lo:lo + (1 << 15)])
    for b, at in ((0, 0), (31, 17), (B - 2, 4100), (B - 1, n - 40)):
        r = slice(b * n + at, b * n + at + 40)
        want, A = attend(q[r], *(x[b * n:b * n + at + 40].transpose(0, 1) for x in (k, v)), at)
        near(out[r], want, attention_tol(want, A, dt))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_two_captured_batches_at_once(dt):
    """Two programs, each its own stream, workspace, cache and graph of the three calls (rows past those of a single
    CTA of tables), replayed side by side: each leaves what it leaves alone."""
    Hq, Hkv, B, T, room = 8, 2, 6, 1300, 1024
    cfg = mac.config(B, Hq, Hkv, dtype=mac.MAC_BF16 if dt == BF16 else mac.MAC_F32, page_size=PAGE, max_context=room)
    rng = random.Random(7)

    class Program:
        def __init__(self, seed):
            g = torch.Generator(device=DEV)
            g.manual_seed(seed)
            n_pages = B * room // PAGE
            self.cache = [torch.zeros(n_pages, Hkv, PAGE, D, device=DEV, dtype=dt) for _ in range(2)]
            self.table = torch.full((B, room // PAGE), -1, dtype=torch.int32, device=DEV)
            self.free, self.n_free = torch.randperm(n_pages, generator=g, device=DEV).int(), ints([n_pages])
            self.first = self.free.clone()
            self.length, self.new, self.q_start = ints([0] * B), ints([0] * B), ints([0] * (B + 1))
            self.pos, self.slot = ints([0] * T), ints([0] * T, torch.int64)
            self.q, self.k, self.v = (torch.randn(T, h, D, generator=g, device=DEV).to(dt) for h in (Hq, Hkv, Hkv))
            self.rows, self.out, self.lse = torch.zeros_like(self.q), torch.zeros_like(self.q), torch.zeros(T, Hq, device=DEV)
            self.ws, self.stream = workspace(cfg, T), torch.cuda.Stream()
            self.pages, self.kv = mac.pages_view(self.table, self.free, self.n_free), mac.kv_view(*self.cache, self.table)
            torch.cuda.synchronize()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=self.stream):
                s = torch.cuda.current_stream()
                mac.mac_build_tables(cfg, self.ws, self.pages, None, self.length, self.new, T, self.length, self.q_start, self.pos,
                                     self.slot, s)
                mac.mac_write_kv(cfg, self.ws, self.q, self.k, self.v, self.pos, self.slot, T, self.kv, self.rows, s)
                mac.mac_chunk_attention(cfg, self.ws, self.rows, self.q_start, self.length, T, self.kv, self.out, self.lse, s)

        def start(self, new):
            self.new.copy_(ints(new))
            self.length.zero_()
            self.free.copy_(self.first)
            self.n_free.fill_(self.free.numel())
            self.out.zero_()
            torch.cuda.synchronize()

        def replay(self):
            with torch.cuda.stream(self.stream):
                self.graph.replay()  # the batch's tokens
                self.graph.replay()  # and as many more behind them

    both = Program(1), Program(2)
    for _ in range(5):
        lengths = [[rng.choice([0, 1, rng.randint(2, 210)]) for _ in range(B)] for _ in both]
        alone = []
        for p, new in zip(both, lengths):
            p.start(new)
            p.replay()
            torch.cuda.synchronize()
            alone.append([x.clone() for x in (p.out, p.lse, p.slot, p.length, *p.cache)])
        for p, new in zip(both, lengths):
            p.start(new)
        for p in both:
            p.replay()
        torch.cuda.synchronize()
        for p, new, ref in zip(both, lengths, alone):
            assert p.length.tolist() == [2 * n for n in new]
            assert all(torch.equal(x, y) for x, y in zip((p.out, p.lse, p.slot, p.length, *p.cache), ref))
            assert mac.mac_last_status(cfg, p.ws) == 0
