"""GPU tests of beam search's calls (mac_beam_select, mac_reorder_tables,
mac_reorder_state) against plain implementations: whole numbers have to be
equal, copies too.

Tolerance of the scores: a beam's sum of exponentials is known to 2^-17 of
itself before its logarithm (its pieces are fp32 sums), and the score is
rounded to fp32 once: 2^-17 + 2^-24 |s|.  The choice itself is that of 64 bits,
so it has to be equal."""
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


def config(S, Hq=1, Hkv=1, **kw):
    return mac.config(S, Hq, Hkv, **kw)


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------

def ref_select(logits, scores, done, n, n_out, end, placed):
    """The call's definition, group by group, in 64 bits: score, parent, token, done."""
    S, V = logits.shape
    x, c = logits.double().cpu().numpy(), scores.double().cpu().numpy()
    rows = []
    for g in range(S // n):
        pool = []
        for j in range(n):
            b = g * n + j
            if not math.isfinite(c[b]):
                continue
            if done is not None and done[b]:
                pool.append((-c[b], j, end))
                continue
            m = x[b].max()
            if not m > -math.inf or np.isnan(x[b]).any() or m == math.inf:
                continue
            s = c[b] + ((x[b] - m) - np.log(np.exp(x[b] - m).sum()))
            for v in np.argsort(-s, kind="stable")[:n_out]:
                if s[v] > -math.inf:
                    pool.append((-s[v], j, int(v)))
        best = [(-s, j, v, int(v == end or (done is not None and bool(done[g * n + j])))) for s, j, v in sorted(pool)[:n_out]]
        best += [(-math.inf, -1, -1, 1)] * (n_out - len(best))
        if placed:
            put, later = [None] * n, []
            for r in best:
                if r[1] >= 0 and put[r[1]] is None:
                    put[r[1]] = r
                else:
                    later.append(r)
            best = [later.pop(0) if r is None else r for r in put]
        rows.append(best)
    return rows


class Selection:
    def __init__(self, S, n, V, n_out, dt=BF16, gap=0, placed=False, seed=0, offset=0, scale=2.0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        store = torch.full((S * (V + gap) + offset,), float("nan"), device=DEV, dtype=dt)
        self.logits = store[offset:].view(S, V + gap)[:, :V]
        self.logits.copy_(torch.randn(S, V, generator=g, device=DEV) * scale)
        self.scores = -5 * torch.rand(S, generator=g, device=DEV)
        self.S, self.n, self.V, self.n_out, self.placed, self.done, self.end = S, n, V, n_out, placed, None, -1
        self.cfg = config(S)
        self.ws = torch.zeros(mac.mac_beam_workspace_size(self.cfg, n, V, n_out), dtype=torch.uint8, device=DEV)
        self.out = torch.full((S // n, n_out), 7.0, device=DEV)
        self.parent, self.token, self.over = (torch.full((S // n, n_out), 7, dtype=torch.int32, device=DEV) for _ in range(3))

    def run(self, stream=None):
        mac.mac_beam_select(self.cfg, self.ws, self.n, self.logits, self.scores, self.done, self.end, self.n_out, self.placed, self.out,
                            self.parent, self.token, self.over, stream)

    def status(self):
        return mac.mac_last_status(self.cfg, self.ws)

    def check(self):
        done = None if self.done is None else self.done.tolist()
        want = ref_select(self.logits, self.scores, done, self.n, self.n_out, self.end, self.placed)
        for i, got in ((1, self.parent), (2, self.token), (3, self.over)):
            assert got.tolist() == [[r[i] for r in row] for row in want], i
        s = torch.tensor([[r[0] for r in row] for row in want], dtype=torch.float64, device=DEV)
        fine = s > -math.inf
        assert torch.equal(self.out == -math.inf, ~fine)
        assert ((self.out.double() - s)[fine].abs() <= (2.0 ** -17 + 2.0 ** -24 * s.abs())[fine]).all()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("groups,n,V,n_out,gap,offset", [
    (1, 1, 1, 1, 0, 0), (2, 1, 3, 1, 0, 1), (1, 4, 5, 4, 2, 3), (3, 2, 8, 4, 0, 0), (2, 4, 100, 32, 1, 5), (1, 16, 1000, 16, 0, 0),
    (5, 4, 2047, 8, 1, 0), (2, 3, 2049, 3, 0, 1), (16, 4, 8192, 4, 0, 0), (1, 4, 32000, 4, 0, 0), (2, 8, 50001, 16, 7, 0),
    (3, 5, 50257, 10, 0, 0), (40, 4, 20000, 8, 3, 2), (1, 1, 128000, 32, 0, 0), (60, 16, 300, 32, 5, 1), (1, 2, 1 << 20, 4, 0, 0),
    (1, 16, 1 << 20, 32, 1, 0),
])
def test_select(groups, n, V, n_out, gap, offset, dt):
    for placed in (False, True) if n == n_out else (False,):
        s = Selection(groups * n, n, V, n_out, dt, gap, placed, seed=V, offset=offset)
        s.run()
        assert s.status() == 0
        s.check()


@pytest.mark.parametrize("seed", range(20))
def test_select_drawn(seed):
    rng = random.Random(seed)
    n = rng.choice([1, 2, 3, 4, 5, 8, 16])
    V, placed = rng.choice([rng.randint(1, 40), rng.randint(40, 3000), rng.randint(3000, 70000)]), rng.random() < 0.4
    groups = rng.randint(1, 12)
    s = Selection(groups * n, n, V, n if placed else rng.randint(1, 32), rng.choice([BF16, F32]), rng.randint(0, 9), placed, seed,
                  rng.randint(0, 8), rng.choice([0.1, 2.0, 30.0]))
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if rng.random() < 0.5:  # part of the vocabulary is ruled out
        s.logits.masked_fill_(torch.rand(s.logits.shape, generator=g, device=DEV) < rng.choice([0.3, 0.999]), -math.inf)
    if rng.random() < 0.5:
        s.end = rng.randrange(V)
        s.done = (torch.rand(s.S, generator=g, device=DEV) < 0.3).int()
    if rng.random() < 0.5:
        s.scores[torch.rand(s.S, generator=g, device=DEV) < 0.3] = -math.inf
    s.run()
    assert s.status() == 0
    s.check()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("V", [7, 3000, 40000])
def test_select_ties_go_to_the_lowest(dt, V):
    # one value everywhere (more of it than is ranked at once), two zeros, beams that are the same
    for fill in (0.0, -3.5):
        s = Selection(8, 4, V, 6, dt)
        s.logits.fill_(fill)
        s.scores.fill_(-1.0)
        s.run()
        assert s.status() == 0
        for j in range(2):
            flat = [(0, v) for v in range(V)] + [(1, v) for v in range(V)]
            assert list(zip(s.parent[j].tolist(), s.token[j].tolist())) == flat[:6]
    s = Selection(4, 4, V, 5, dt, scale=0.0)
    s.logits[:, V // 2:] = -0.0
    s.logits[1:] = -math.inf
    s.run()
    assert s.parent[0].tolist() == [0] * 5 and s.token[0].tolist() == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("dt", [BF16, F32])
def test_select_more_ties_than_are_ranked_at_once(dt):
    # every piece of every beam offers 32 candidates of the same score, and the scores of beams are the same or differ
    n, V = 16, 70001
    s = Selection(2 * n, n, V, 32, dt)
    s.logits.fill_(1.5)
    s.scores.fill_(-2.0)
    s.scores[n:] = -2.0 - torch.arange(n, device=DEV).flip(0) * 2.0 ** -21
    s.run()
    assert s.status() == 0
    assert s.parent.tolist() == [[0] * 32, [n - 1] * 32] and s.token.tolist() == [list(range(32))] * 2
    s.logits[5, 60000:60010] = 1.5078125  # a few above the rest
    s.run()
    assert s.parent[0].tolist() == [5] * 10 + [0] * 22 and s.token[0].tolist() == list(range(60000, 60010)) + list(range(22))


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("V", [50, 9000, 33333])
def test_select_orders_scores_that_fp32_sums_cannot_tell_apart(dt, V):
    # beams whose best tokens' scores lie within 2^-22 of one another, of other logits and of the same
    for seed in range(4):
        s = Selection(12, 4, V, 8, dt, seed=seed)
        x = s.logits.double()
        lse, top = torch.logsumexp(x, -1), x.amax(-1)
        s.scores = (-4 + lse - top).float()
        s.run()
        assert s.status() == 0
        s.check()
    s = Selection(12, 4, V, 8, dt, gap=1)
    s.logits.copy_(s.logits[:1].clone().expand(12, V))
    s.scores = -1 - 2.0 ** -22 * torch.tensor([3, 0, 2, 1] * 3, device=DEV)
    s.run()
    s.check()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_select_first_step_finished_and_empty_groups(dt):
    s = Selection(16, 4, 3001, 4, dt, gap=2, placed=True)
    s.scores.view(4, 4)[0, 1:] = -math.inf  # a group before its first token: one beam counts
    s.scores.view(4, 4)[1] = -math.inf      # nothing to choose from
    s.end, s.done = 17, ints([0] * 8 + [1, 1, 1, 1] + [0, 1, 0, 1])
    s.logits.view(4, 4, -1)[2] = math.nan   # logits of beams that have none are not looked at
    s.logits.view(4, 4, -1)[0, 1:] = math.nan
    s.run()
    assert s.status() == 0
    s.check()
    s.n_out, s.placed = 9, False
    s.ws = torch.zeros(mac.mac_beam_workspace_size(s.cfg, 4, 3001, 9), dtype=torch.uint8, device=DEV)
    s.out, (s.parent, s.token, s.over) = torch.zeros(4, 9, device=DEV), (torch.zeros(4, 9, dtype=torch.int32, device=DEV) for _ in range(3))
    s.run()
    assert s.status() == 0
    s.check()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_select_leaves_out_beams_with_nan_or_infinite_logits(dt, bad):
    s = Selection(8, 4, 5000, 4, dt)
    s.logits[2, 4321] = bad
    s.logits[7] = -math.inf  # no tokens, no error
    s.run()
    assert s.status() == mac.MAC_DEV_NONFINITE_LOGIT
    s.check()
    s.logits[2, 4321] = 0
    s.scores[1], s.scores[6] = math.nan, math.inf
    s.run()
    assert s.status() == mac.MAC_DEV_NONFINITE_LOGIT
    s.check()


def test_select_large_values():
    s = Selection(4, 4, 3000, 8, F32)
    s.logits *= 1e36
    s.run()
    assert s.status() == 0
    s.check()
    s.logits[:, 5] = torch.finfo(F32).max
    s.logits[:, 6:] = torch.finfo(F32).min
    s.run()
    s.check()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_select_rows_beyond_32_bit_offsets(dt):
    S, V, stride = 70, 900, 32_000_001
    store = torch.empty(S * stride, device=DEV, dtype=dt)
    assert store.numel() > 1 << 31
    s = Selection(S, 2, V, 4, dt)
    rows = store.view(S, stride)[:, :V]
    rows.copy_(s.logits)
    s.logits = rows
    s.run()
    assert s.status() == 0
    s.check()


def test_select_in_place_on_a_stream_and_in_a_graph():
    s = Selection(12, 4, 20000, 4, BF16)
    s.end, s.done = 3, ints([0, 0, 1] * 4)
    first = s.scores.clone(), s.done.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s.run(side)
    side.synchronize()
    s.check()
    keep = [x.clone() for x in (s.out, s.parent, s.token, s.over)]
    s.out, s.over = s.scores, s.done  # the next step's inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        s.run(torch.cuda.current_stream())
    for _ in range(3):
        s.scores.copy_(first[0])
        s.done.copy_(first[1])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((s.out.view(3, 4), s.parent, s.token, s.over.view(3, 4)), keep):
            assert torch.equal(x, y)


def test_select_calls_of_different_sizes_share_a_workspace():
    # groups, vocabularies and candidates differ from call to call; what a call counts is left as it was found
    S = 24
    calls = [Selection(S, n, V, n_out, dt, seed=V + n, placed=n == n_out) for n, V, n_out, dt in [
        (4, 32000, 4, BF16), (1, 300, 32, F32), (12, 50001, 16, F32), (2, 7, 2, BF16), (3, 128000, 1, BF16), (8, 2048, 8, F32)]]
    ws = max((c.ws for c in calls), key=len)
    for c in calls:
        c.ws = ws
    calls[2].scores[:12] = -math.inf  # a group without a beam to look at
    for _ in range(3):
        for c in calls:
            c.out.fill_(7)
            c.parent.fill_(7)
            c.run()
    assert calls[0].status() == 0
    for c in calls:
        c.check()


# ---------------------------------------------------------------------------
# tables
# ---------------------------------------------------------------------------

def ref_reorder(parent, length, shared, n, limit, paged, table=None, free=None, n_free=0, n_pages=0):
    """The call's definition, slot by slot: lengths, shared, moves, table, stack, its count, status."""
    S = len(length)
    status = 0
    up = []
    for s in range(S):
        base = s // n * n
        if any(not 0 <= x <= limit for x in length[base:base + n]):
            status |= mac.MAC_DEV_BAD_SEQ_LEN
            up.append(s)
        elif parent[s] == -1:
            up.append(None)
        elif not 0 <= parent[s] < n:
            status |= mac.MAC_DEV_BAD_PARENT
            up.append(s)
        else:
            up.append(base + parent[s])
    bad = [any(not 0 <= x <= limit for x in length[s // n * n:s // n * n + n]) for s in range(S)]
    new = [0 if u is None else length[u] for u in up]
    moves = [[-1, 0, 0, 0, -1, -1, 0, 0] for _ in range(S)]
    for s, u in enumerate(up):
        if u is not None and u != s:
            moves[s][:4] = [u, shared[s][u % n] + 1, max(length[s], length[u]), length[u]]
    gone = set()
    if paged:
        table, free = [list(r) for r in table], list(free)
        before = [table[s][:pages_of(length[s])] if not bad[s] else [] for s in range(S)]
        after = [[] if u is None else before[u] for u in up]
        for g in range(S // n):  # pages that nobody holds any more
            slots = range(g * n, g * n + n)
            kept = {p for s in slots for p in after[s]}
            for c in range(max((len(before[s]) for s in slots), default=0)):
                for s in slots:
                    if c < len(before[s]) and 0 <= before[s][c] < n_pages and before[s][c] not in kept:
                        kept.add(before[s][c])
                        free[n_free] = before[s][c]
                        n_free += 1
        for s in range(S):
            if not bad[s]:
                table[s][:len(after[s])] = after[s]
        for s, u in enumerate(up):
            if u is None or bad[s] or new[s] % PAGE == 0:
                continue
            keeper = u if up[u] == u else up.index(u)
            if keeper == s:
                continue
            if n_free == 0:
                status |= mac.MAC_DEV_NO_ROOM
                gone.add(s)
                new[s] = 0
                moves[s] = [-1, 0, 0, 0, -1, -1, 0, 0]
                continue
            n_free -= 1
            c = new[s] // PAGE
            moves[s][4:7] = [after[s][c], free[n_free], new[s] % PAGE]
            table[s][c] = free[n_free]
    out = [[0] * n for _ in range(S)]
    for s in range(S):
        for j in range(n):
            o = s // n * n + j
            if up[s] is None or up[o] is None or s in gone or o in gone:
                continue
            out[s][j] = new[s] if o == s else max(new[s] - 1, 0) if up[s] == up[o] else shared[up[s]][up[o] % n]
    return new, out, moves, table, free, n_free, status


class Histories:
    """Slots whose state evolves through reorderings and new tokens, beside the call's definition."""

    def __init__(self, groups, n, width, paged, seed, n_pages=None):
        self.rng = random.Random(seed)
        self.S, self.n, self.paged, self.width = groups * n, n, paged, width
        self.cfg = config(self.S, page_size=PAGE if paged else 0, max_context=width * PAGE - 3)
        self.limit = width * PAGE - 3
        self.n_pages = n_pages or self.S * width
        self.length, self.shared = [0] * self.S, [[0] * n for _ in range(self.S)]
        self.table = [[-1] * width for _ in range(self.S)]
        self.free = list(range(self.n_pages))
        self.rng.shuffle(self.free)
        self.n_free = self.n_pages
        self.ws = torch.zeros(mac.mac_chunk_workspace_size(self.cfg, 1), dtype=torch.uint8, device=DEV)

    def grow(self, most, slots=None):
        """New tokens, as mac_build_tables would bring them."""
        for s in range(self.S):
            if slots is not None and s not in slots:
                continue
            k = min(self.rng.randint(0, most), self.limit - self.length[s])
            for c in range(pages_of(self.length[s]), pages_of(self.length[s] + k)) if self.paged else ():
                self.n_free -= 1
                self.table[s][c] = self.free[self.n_free]
            self.length[s] += k

    def reorder(self, parent, in_place=True, status=0):
        S, n = self.S, self.n
        want = ref_reorder(parent, self.length, self.shared, n, self.limit, self.paged, self.table, self.free, self.n_free, self.n_pages)
        length, shared = ints(self.length), ints(self.shared)
        moves = torch.full((S, 8), 99, dtype=torch.int32, device=DEV)
        pages = None
        if self.paged:
            table, free, n_free = ints(self.table), ints(self.free), ints([self.n_free])
            n_out = n_free if in_place else ints([-1])
            pages = mac.pages_view(table, free, n_free, n_out)
        len_out, shared_out = (length, shared) if in_place else (torch.zeros_like(length), torch.zeros_like(shared))
        mac.mac_reorder_tables(self.cfg, self.ws, pages, n, ints(parent), length, len_out, shared, shared_out, moves)
        assert mac.mac_last_status(self.cfg, self.ws) == want[6] == status
        assert len_out.tolist() == want[0]
        assert shared_out.tolist() == want[1]
        assert moves.tolist() == want[2]
        if self.paged:
            assert n_out.tolist() == [want[5]]
            assert free.tolist() == want[4]
            assert table.tolist() == want[3]
        self.length, self.shared = want[0], want[1]
        if self.paged:
            self.table, self.free, self.n_free = want[3], want[4], want[5]
            self.sound()
        return want[2]

    def sound(self):
        """Every page is held by one group or free, and nothing that will be written is shared."""
        held = {}
        for s in range(self.S):
            for c in range(pages_of(self.length[s])):
                held.setdefault(self.table[s][c], set()).add((s, c))
        for p, where in held.items():
            assert len({s // self.n for s, _ in where}) == 1 and len({c for _, c in where}) == 1
            if len(where) > 1:
                assert all((c + 1) * PAGE <= self.length[s] for s, c in where)
        spare = self.free[:self.n_free]
        assert len(set(spare)) == len(spare) and not set(spare) & set(held) and len(spare) + len(held) == self.n_pages


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("groups,n,width", [(1, 2, 8), (3, 4, 20), (2, 5, 6), (16, 4, 40), (4, 16, 12), (7, 8, 700), (5, 1, 9), (128, 8, 9), (1024, 1, 5), (64, 16, 6)])
def test_reorder_tables(groups, n, width, paged):
    h = Histories(groups, n, width, paged, groups)
    h.grow(width * 9, {g * n for g in range(groups)})  # prompts in the first slot of every group
    h.reorder([0] * (groups * n))
    for step in range(12 if groups * n * width < 5000 else 5):
        h.grow(1 if step % 3 else 20)
        how = h.rng.random()
        parent = [h.rng.randrange(n) for _ in range(h.S)]
        if how < 0.2:
            parent = [s % n for s in range(h.S)]  # nothing changes
        elif how < 0.4:
            parent = [(s + 1) % n for s in range(h.S)]  # all change places
        elif how < 0.6:
            parent = [-1 if h.rng.random() < 0.3 else p for p in parent]
        h.reorder(parent, in_place=step % 2 == 0)
    h.reorder([-1] * h.S)
    assert h.length == [0] * h.S and (not paged or h.n_free == h.n_pages)
    h.grow(30)
    h.reorder([h.rng.randrange(n) for _ in range(h.S)])


def test_reorder_tables_of_different_lengths():
    h = Histories(6, 4, 30, True, 3)
    h.grow(200, {0, 4, 8, 12, 16, 20})
    h.reorder([0] * 24)
    for _ in range(10):
        h.grow(3, {s for s in range(24) if h.rng.random() < 0.6})
        h.reorder([h.rng.randrange(4) for _ in range(24)])


@pytest.mark.parametrize("n", [2, 4, 8])
def test_reorder_tables_bad_parents_and_lengths(n):
    h = Histories(4, n, 10, True, 1)
    h.grow(90)
    parent = [h.rng.randrange(n) for _ in range(h.S)]
    parent[1], parent[n] = n, -2
    h.reorder(parent, status=mac.MAC_DEV_BAD_PARENT)
    for bad in (-1, h.limit + 1, 1 << 30):
        keep = h.length[2 * n]
        h.length[2 * n] = bad
        length = list(h.length)
        want = ref_reorder([0] * h.S, h.length, h.shared, n, h.limit, True, h.table, h.free, h.n_free, h.n_pages)
        table, free, n_free, out, shared = ints(h.table), ints(h.free), ints([h.n_free]), ints(length), ints(h.shared)
        moves = torch.zeros(h.S, 8, dtype=torch.int32, device=DEV)
        mac.mac_reorder_tables(h.cfg, h.ws, mac.pages_view(table, free, n_free), n, ints([0] * h.S), out, out, shared, shared, moves)
        assert mac.mac_last_status(h.cfg, h.ws) == mac.MAC_DEV_BAD_SEQ_LEN == want[6]
        assert out.tolist() == want[0] and moves.tolist() == want[2] and table.tolist() == want[3] and free.tolist() == want[4]
        assert out.tolist()[2 * n:3 * n] == length[2 * n:3 * n] and table.tolist()[2 * n:3 * n] == h.table[2 * n:3 * n]
        h.length[2 * n] = keep


def test_reorder_tables_without_room():
    # more histories part than there are pages
    h = Histories(3, 4, 10, True, 2, n_pages=14)
    for s, k in ((0, 37), (4, 50), (8, 48)):
        h.grow(0)
        for c in range(pages_of(k)):
            h.n_free -= 1
            h.table[s][c] = h.free[h.n_free]
        h.length[s] = k
    assert h.n_free == 4
    h.reorder([0] * 12, status=mac.MAC_DEV_NO_ROOM)
    assert h.length == [37] * 4 + [50, 50, 0, 0] + [48] * 4 and h.n_free == 0
    h.reorder([-1] * 12)


def test_reorder_tables_flag_pages_outside_the_cache():
    h = Histories(2, 4, 10, True, 2)
    h.grow(0)
    for s, k in ((0, 37), (4, 50)):
        for c in range(pages_of(k)):
            h.n_free -= 1
            h.table[s][c] = h.free[h.n_free]
        h.length[s] = k
    h.table[0][1], h.table[4][3] = h.n_pages, -1
    table, free, n_free, length, shared = ints(h.table), ints(h.free), ints([h.n_free]), ints(h.length), ints(h.shared)
    moves = torch.zeros(8, 8, dtype=torch.int32, device=DEV)
    mac.mac_reorder_tables(h.cfg, h.ws, mac.pages_view(table, free, n_free), 4, ints([0, 0, 0, 0, 0, -1, 0, 0]), length, length, shared, shared, moves)
    assert mac.mac_last_status(h.cfg, h.ws) == mac.MAC_DEV_BAD_PAGE
    assert length.tolist() == [37] * 4 + [50, 0, 50, 50]
    k, v = (torch.randn(h.n_pages, 1, PAGE, D, device=DEV).to(BF16) for _ in range(2))
    before = k.clone()
    assert moves[6:, 4].tolist() == [-1, -1]
    mac.mac_reorder_state(h.cfg, h.ws, None, 4, moves, mac.kv_view(k, v, n_pages=h.n_pages))
    assert mac.mac_last_status(h.cfg, h.ws) == mac.MAC_DEV_BAD_PAGE
    for s in (1, 2, 3):
        to = table[s, 2].item()
        assert torch.equal(k[to, :, :5], before[h.table[0][2], :, :5]) and torch.equal(k[to, :, 5:], before[to, :, 5:])
    # a stack count outside the pool
    length, shared = ints(h.length), ints(h.shared)
    mac.mac_reorder_tables(h.cfg, h.ws, mac.pages_view(table, free, ints([h.n_pages + 5]), n_free), 4, ints([-1] * 8), length, length, shared, shared,
                           moves)
    assert mac.mac_last_status(h.cfg, h.ws) & mac.MAC_DEV_BAD_PAGE
    assert length.tolist() == [0] * 8 and n_free.tolist() == [h.n_pages]


# ---------------------------------------------------------------------------
# state
# ---------------------------------------------------------------------------

class Layer:
    """A layer's rings and contiguous cache of histories, and a copy that every move copies whole."""

    def __init__(self, S, Hq, Hkv, K, cap, dt, seed):
        self.cfg = mac.config(S, Hq, Hkv, ring_k=K, max_context=cap, dtype=mac.MAC_BF16 if dt == BF16 else mac.MAC_F32)
        self.layer = mac.MacLayer(self.cfg)
        self.ring = {x: self.layer.ring_view(x) for x in ("pos", "q", "o", "lse")}
        self.k, self.v = (torch.zeros(S, Hkv, cap, D, device=DEV, dtype=dt) for _ in range(2))
        self.whole = [x.clone() for x in (*self.ring.values(), self.k, self.v)]
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)
        self.K, self.S = K, S

    def append(self, slot, pos):
        """Position pos (1-based) of a slot, in both copies."""
        at = pos % self.K
        for i, (mine, x) in enumerate(zip((*self.ring.values(), self.k, self.v), self.whole)):
            to = (slot, at) if i == 0 else (slot, slice(None), at if i < 4 else pos - 1)
            new = pos if i == 0 else torch.randn(x[to].shape, generator=self.g, device=DEV).to(x.dtype)
            x[to] = new
            mine[to] = new

    def move(self, up):
        """The whole copy takes its parents' state (None: keeps)."""
        for x in self.whole:
            old = x.clone()
            for s, u in enumerate(up):
                if u is not None and u != s:
                    x[s] = old[u]

    def same(self, lengths):
        for mine, x in zip(self.ring.values(), self.whole):
            assert torch.equal(mine, x)
        for mine, x in zip((self.k, self.v), self.whole[4:]):
            for s, n in enumerate(lengths):
                assert torch.equal(mine[s, :, :n], x[s, :, :n])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("groups,n,Hq,Hkv,K", [(2, 4, 8, 2, 32), (1, 2, 1, 1, 7), (3, 5, 4, 4, 50), (1, 16, 8, 1, 64), (2, 8, 2, 1, 16), (20, 2, 8, 4, 24)])
def test_reorder_state(groups, n, Hq, Hkv, K, dt):
    """After every step a slot holds what a copy of its parent's whole state would hold."""
    cap = 96
    h = Histories(groups, n, cap // PAGE, False, seed=n)
    x = Layer(h.S, Hq, Hkv, K, cap, dt, seed=K)
    kv = mac.kv_view(x.k, x.v)

    def grow(most, slots):
        before = list(h.length)
        h.grow(most, slots)
        for s in range(h.S):
            for p in range(before[s] + 1, h.length[s] + 1):
                x.append(s, p)

    def reorder(parent):
        base = [s // n * n for s in range(h.S)]
        moves = h.reorder(parent)
        x.move([None if p < 0 else base[s] + p for s, p in enumerate(parent)])
        mac.mac_reorder_state(x.cfg, h.ws, x.layer.ring, n, ints(moves), kv)
        assert mac.mac_last_status(x.cfg, h.ws) == 0
        x.same(h.length)

    grow(40, {g * n for g in range(groups)})
    reorder([0] * h.S)
    for step in range(9):
        grow(1 if step % 3 else 6, None if step % 2 else {s for s in range(h.S) if h.rng.random() < 0.7})
        reorder([(s + 1) % n for s in range(h.S)] if step == 4 else [h.rng.randrange(n) for _ in range(h.S)])
    x.layer.release()


@pytest.mark.parametrize("paged", [True, False])
def test_reorder_tables_and_state_with_common_positions_that_cannot_be(paged):
    """Whatever the caller's array of common positions holds, lengths and parted pages are right and nothing else is touched."""
    h = Histories(3, 4, 12, paged, 4)
    h.grow(150)
    x = Layer(h.S, 4, 2, 40, 12 * PAGE, BF16, 1)
    for seed in range(6):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        shared = torch.randint(-(1 << 31), (1 << 31) - 1, (h.S, 4), generator=g, device=DEV).int()
        if seed % 2:
            shared = torch.randint(-3, 200, (h.S, 4), generator=g, device=DEV).int()
        parent = [h.rng.randrange(-1, 4) for _ in range(h.S)]
        table, free, n_free = ints(h.table), ints(h.free), ints([h.n_free])
        length, moves = ints(h.length), torch.zeros(h.S, 8, dtype=torch.int32, device=DEV)
        mac.mac_reorder_tables(h.cfg, h.ws, mac.pages_view(table, free, n_free) if paged else None, 4, ints(parent), length, length, shared,
                               torch.zeros_like(shared), moves)
        want = [0 if p < 0 else h.length[s // 4 * 4 + p] for s, p in enumerate(parent)]
        assert length.tolist() == want
        assert mac.mac_last_status(h.cfg, h.ws) == 0
        for s, m in enumerate(moves.tolist()):
            assert m[0] == (-1 if parent[s] < 0 or parent[s] == s % 4 else s // 4 * 4 + parent[s])
            if m[0] >= 0:
                assert 1 <= m[1] <= min(h.length[s], want[s]) + 1 and m[2] == max(h.length[s], want[s]) and m[3] == want[s]
            assert not paged or (0 <= n_free.item() <= h.n_pages)
        mac.mac_reorder_state(x.cfg, h.ws, x.layer.ring, 4, moves, mac.kv_view(x.k, x.v))
        assert mac.mac_last_status(h.cfg, h.ws) == 0
    x.layer.release()


@pytest.mark.parametrize("paged", [True, False])
def test_reorder_state_of_rings_or_cache_alone(paged):
    S, n, cap = 6, 3, 64
    x = Layer(S, 2, 1, 16, cap, BF16, 2)
    for s in range(S):
        for p in range(1, 40):
            x.append(s, p)
    cfg = mac.config(S, 2, 1, ring_k=16, page_size=PAGE if paged else 0, max_context=cap)
    ws = torch.zeros(mac.mac_chunk_workspace_size(cfg, 1), dtype=torch.uint8, device=DEV)
    pool = [torch.randn(S * 4, 1, PAGE, D, device=DEV).to(BF16) for _ in range(2)]
    cache = pool if paged else [x.k, x.v]
    moves = ints([[2, 30, 39, 39, 3, 9, 7, 0], [0, 31, 39, 39, -1, -1, 0, 0], [-1, 0, 0, 0, -1, -1, 0, 0]] + [[-1, 0, 0, 0, -1, -1, 0, 0]] * 3)
    rings, keep = [r.clone() for r in x.ring.values()], [c.clone() for c in cache]
    mac.mac_reorder_state(cfg, ws, x.layer.ring, n, moves, None)
    assert all(torch.equal(a, b) for a, b in zip(cache, keep))
    at = [p % 16 for p in range(30, 40)]
    for r, old in zip(x.ring.values(), rings):
        if r.dim() == 2:
            assert torch.equal(r[0, at], old[2, at]) and torch.equal(r[1, at[1:]], old[0, at[1:]]) and torch.equal(r[1, at[0]], old[1, at[0]])
        else:
            assert torch.equal(r[0, :, at], old[2, :, at]) and torch.equal(r[1, :, at[1:]], old[0, :, at[1:]])
            assert torch.equal(r[1, :, at[0]], old[1, :, at[0]])
        assert torch.equal(r[2:], old[2:])
    rings = [r.clone() for r in x.ring.values()]
    mac.mac_reorder_state(cfg, ws, None, n, moves, mac.kv_view(*cache, n_pages=S * 4))
    assert all(torch.equal(a, b) for a, b in zip(x.ring.values(), rings))
    for c, old in zip(cache, keep):
        if paged:
            assert torch.equal(c[9, :, :7], old[3, :, :7])
            c[9] = old[9]
            assert torch.equal(c, old)
        else:
            assert torch.equal(c[0, :, 29:39], old[2, :, 29:39]) and torch.equal(c[1, :, 30:39], old[0, :, 30:39])
            assert torch.equal(c[:, :, :29], old[:, :, :29]) and torch.equal(c[2:], old[2:]) and torch.equal(c[:, :, 39:], old[:, :, 39:])
    assert mac.mac_last_status(cfg, ws) == 0


def test_reorder_state_refuses_moves_outside():
    S, n, cap = 8, 4, 64
    x = Layer(S, 2, 1, 16, cap, BF16, 1)
    for s in range(S):
        for p in range(1, 5 + s):
            x.append(s, p)
    ws = torch.zeros(mac.mac_chunk_workspace_size(x.cfg, 1), dtype=torch.uint8, device=DEV)
    moves = torch.tensor([[-1, 0, 0, 0, -1, -1, 0, 0]] * S, dtype=torch.int32)
    for bad, bit in (([4, 1, 5, 5, -1, -1, 0, 0], mac.MAC_DEV_BAD_PARENT), ([-7, 1, 5, 5, -1, -1, 0, 0], mac.MAC_DEV_BAD_PARENT),
                     ([99, 1, 5, 5, -1, -1, 0, 0], mac.MAC_DEV_BAD_PARENT), ([1, 0, 5, 5, -1, -1, 0, 0], mac.MAC_DEV_BAD_SEQ_LEN),
                     ([1, 1, 5, cap + 1, -1, -1, 0, 0], mac.MAC_DEV_BAD_SEQ_LEN), ([1, 1, -5, 5, -1, -1, 0, 0], mac.MAC_DEV_BAD_SEQ_LEN)):
        m = moves.clone()
        m[0] = torch.tensor(bad, dtype=torch.int32)
        mac.mac_reorder_state(x.cfg, ws, x.layer.ring, n, m.to(DEV), mac.kv_view(x.k, x.v))
        assert mac.mac_last_status(x.cfg, ws) == bit
        x.same([cap] * S)
    paged = mac.config(S, 2, 1, ring_k=16, page_size=PAGE, max_context=cap)
    k, v = (torch.randn(20, 1, PAGE, D, device=DEV).to(BF16) for _ in range(2))
    keep = k.clone(), v.clone()
    for page in ([-1, 3, 4], [3, 20, 4], [20, 3, 4], [3, -1, 4], [3, 4, 17]):
        m = moves.clone()
        m[0] = torch.tensor([1, 1, 5, 5, *page, 0], dtype=torch.int32)
        mac.mac_reorder_state(paged, ws, None, n, m.to(DEV), mac.kv_view(k, v, n_pages=20))
        assert mac.mac_last_status(paged, ws) == mac.MAC_DEV_BAD_PAGE
        assert torch.equal(k, keep[0]) and torch.equal(v, keep[1])


@pytest.mark.parametrize("dt", [BF16, F32])
def test_reorder_state_beyond_32_bit_offsets(dt):
    # the last slots' rings and cache rows lie past element 2^31
    S, n, Hq, Hkv, K = 8, 4, 32, 8, (1 << 16) + 64
    cap = (1 << 32) // (S * Hkv * D) + 64
    cfg = mac.config(S, Hq, Hkv, ring_k=K, max_context=cap, dtype=mac.MAC_BF16 if dt == BF16 else mac.MAC_F32)
    L = mac.mac_ring_layout_of(cfg)
    assert S * Hq * K * D > 1 << 31
    ring = torch.empty(L.total, dtype=torch.uint8, device=DEV)
    q = ring[L.q:L.q + S * Hq * K * D * (2 if dt == BF16 else 4)].view(dt).view(S, Hq, K, D)
    o = ring[L.o:L.o + S * Hq * K * D * 4].view(F32).view(S, Hq, K, D)
    pos = ring[L.pos:L.pos + S * K * 4].view(torch.int32).view(S, K)
    k = torch.empty(S, Hkv, cap, D, device=DEV, dtype=dt)
    ws = torch.zeros(mac.mac_chunk_workspace_size(cfg, 1), dtype=torch.uint8, device=DEV)
    first, last = cap - 5, cap
    for x in (q, o):
        x[4:, :, [p % K for p in range(first, last + 1)]] = torch.randn(4, Hq, 6, D, device=DEV).to(x.dtype)
    pos[4:] = 5
    k[4:, :, first - 1:] = torch.randn(4, Hkv, 6, D, device=DEV).to(dt)
    at = [p % K for p in range(first, last + 1)]
    want = [x[[7, 7, 7, 7]][:, :, at].clone() for x in (q, o)] + [k[[7, 7, 7, 7]][:, :, first - 1:].clone()]
    moves = [[-1, 0, 0, 0, -1, -1, 0, 0]] * 4 + [[7, first, last, last, -1, -1, 0, 0]] * 3 + [[-1, 0, 0, 0, -1, -1, 0, 0]]
    mac.mac_reorder_state(cfg, ws, ring, n, ints(moves), mac.kv_view(k, k))
    assert mac.mac_last_status(cfg, ws) == 0
    for x, y in zip((q[4:, :, at], o[4:, :, at], k[4:, :, first - 1:]), want):
        assert torch.equal(x, y)


# ---------------------------------------------------------------------------
# all of it: beams that decode
# ---------------------------------------------------------------------------

class Beams:
    """A decoder's beams: every step brings a token per slot, decodes it over the slot's history and the source's
    states, and reorders by the selection.  `shared` False: slots share nothing, everything is copied whole."""

    def __init__(self, shared, groups, n, Hq, Hkv, dt, paged, layers, aux=False):
        self.shared, self.G, self.n, self.S, self.paged, self.layers = shared, groups, n, groups * n, paged, layers
        S, cap, self.K = self.S, 160, 24
        kind = mac.MAC_BF16 if dt == BF16 else mac.MAC_F32
        self.cfg = mac.config(S, Hq, Hkv, ring_k=self.K, band_r=8, page_size=PAGE if paged else 0, max_context=cap, dtype=kind)
        self.mem_cfg = mac.config(groups, Hq, Hkv, rope_mode=mac.MAC_ROPE_NONE, max_context=64, dtype=kind)
        self.aux = torch.cuda.Stream() if aux else None
        self.Hq, self.Hkv, self.dt, self.V = Hq, Hkv, dt, 700
        g = torch.Generator(device=DEV)
        g.manual_seed(5)
        n_pages = S * (cap // PAGE) if paged else 0
        shape = (n_pages, Hkv, PAGE, D) if paged else (S, Hkv, cap, D)
        self.cache = [[torch.zeros(shape, device=DEV, dtype=dt) for _ in range(2)] for _ in range(layers)]
        if paged:
            self.table = torch.full((S, cap // PAGE), -1, dtype=torch.int32, device=DEV)
            self.free, self.n_free = torch.arange(n_pages, device=DEV).int(), ints([n_pages])
            self.pages = mac.pages_view(self.table, self.free, self.n_free)
        else:
            self.table, self.pages = None, mac.pages_view(capacity=cap)
        self.kv = [mac.kv_view(*c, self.table) for c in self.cache]
        scratch = torch.zeros(mac.mac_workspace_size(self.cfg)[1], dtype=torch.uint8, device=DEV)
        self.rings = [mac.MacLayer(self.cfg, scratch) for _ in range(layers)]
        self.scratch = scratch
        self.ws = torch.zeros(mac.mac_chunk_workspace_size(self.cfg, S * 40), dtype=torch.uint8, device=DEV)
        self.length, self.common = ints([0] * S), torch.zeros(S, n, dtype=torch.int32, device=DEV)
        self.moves = torch.zeros(S, 8, dtype=torch.int32, device=DEV)
        self.q_start = ints([0] * (S + 1))
        self.pos, self.slot = ints([0] * S * 40), ints([0] * S * 40, torch.int64)
        # weights stand for the model: a token's (and its layer's) query, key and value; the logits of an output
        self.emb = [torch.randn(self.V, Hq + 2 * Hkv, D, generator=g, device=DEV).to(dt) for _ in range(layers)]
        self.head = torch.randn(Hq * D, self.V, generator=g, device=DEV) * 0.2
        self.mem = [torch.randn(groups, Hkv, 64, D, generator=g, device=DEV).to(dt) for _ in range(2)]
        self.mem_kv, self.mem_len = mac.kv_view(*self.mem), ints([33 + 7 * i for i in range(groups)])
        self.mem_ws = torch.zeros(mac.mac_chunk_workspace_size(self.mem_cfg, S), dtype=torch.uint8, device=DEV)
        self.sel_ws = torch.zeros(mac.mac_beam_workspace_size(self.cfg, n, self.V, n), dtype=torch.uint8, device=DEV)
        self.scores = torch.zeros(S, device=DEV)
        self.parent, self.token = ints([0] * S), ints([0] * S)
        self.out, self.hits = torch.zeros(S, Hq, D, device=DEV), 0
        self.cross, self.logits = torch.zeros(S, Hq, D, device=DEV, dtype=dt), torch.zeros(S, self.V, device=DEV)
        self.matched = torch.zeros(S, Hq, dtype=torch.int32, device=DEV)
        self.one = ints([1] * S)

    def prompt(self, tokens):
        """Prompts into slot 0 of each group (all slots where nothing is shared); the rings start empty."""
        new = [0] * self.S
        for g, t in enumerate(tokens):
            for j in range(self.n if not self.shared else 1):
                new[g * self.n + j] = len(t)
        ids = torch.cat([torch.tensor(t) for g, t in enumerate(tokens) for _ in range(self.n if not self.shared else 1)]).to(DEV)
        T = sum(new)
        mac.mac_build_tables(self.cfg, self.ws, self.pages, None, self.length, ints(new), T, self.length, self.q_start, self.pos, self.slot)
        for i in range(self.layers):
            x = self.emb[i][ids]
            mac.mac_write_kv(self.cfg, self.ws, None, x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:], self.pos, self.slot, T,
                             self.kv[i], None)
            mac.mac_init_rings(self.cfg, self.rings[i].ring, self.scratch, None, None, 0, None)
        self.take([0] * self.S)
        self.token.copy_(torch.arange(self.S, device=DEV).int() * 3 + 1)

    def take(self, parent):
        """Slots go on from their parents."""
        up = torch.as_tensor(parent, device=DEV).int().view(-1)
        if self.shared:
            mac.mac_reorder_tables(self.cfg, self.ws, self.pages, self.n, up, self.length, self.length, self.common, self.common, self.moves)
            for i in range(self.layers):
                mac.mac_reorder_state(self.cfg, self.ws, self.rings[i].ring, self.n, self.moves, self.kv[i])
            return
        src = up.long() + torch.arange(self.S, device=DEV) // self.n * self.n
        self.length.copy_(self.length[src])
        for i in range(self.layers):
            if self.aux:
                mac.mac_join_aux(self.rings[i].ring)
            for part in ("pos", "q", "o", "lse"):
                x = self.rings[i].ring_view(part)
                x.copy_(x[src])
            for c in self.cache[i]:
                if self.paged:
                    ids = self.table.long()
                    for s in range(self.S):
                        if src[s] != s:
                            k = pages_of(int(self.length[s]))
                            assert (ids[s, :k] >= 0).all()
                    whole = c[ids.clamp(min=0)][src]
                    c[ids[ids >= 0]] = whole[ids >= 0]
                else:
                    c.copy_(c[src])

    def step(self):
        S = self.S
        mac.mac_build_tables(self.cfg, self.ws, self.pages, None, self.length, self.one, S, self.length, self.q_start, self.pos, self.slot)
        ids = self.token.long()
        for i in range(self.layers):
            x = self.emb[i][ids]
            q, k, v = x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hkv], x[:, self.Hq + self.Hkv:]
            mac.mac_write_kv(self.cfg, self.ws, None, k, v, self.pos, self.slot, S, self.kv[i], None)
            mac.mac_decode_step(self.cfg, self.rings[i].ring, self.scratch, q.contiguous(), self.length, self.kv[i], self.out, self.matched,
                                torch.cuda.current_stream(), self.aux)
            self.hits += (self.matched >= 0).int().sum()
        rows = (self.out + self.emb[0][ids][:, :self.Hq].float()).to(self.dt)
        mac.mac_cross_attention(self.mem_cfg, self.mem_ws, rows, self.q_start, self.n, self.mem_len, S, self.mem_kv, self.cross)
        torch.mm(self.cross.float().view(S, -1) + self.out.view(S, -1), self.head, out=self.logits)
        mac.mac_beam_select(self.cfg, self.sel_ws, self.n, self.logits, self.scores, None, -1, self.n, self.n % 2, self.scores, self.parent, self.token)
        self.take(self.parent)

    def status(self):
        return [mac.mac_last_status(c, w) for c, w in ((self.cfg, self.ws), (self.cfg, self.scratch), (self.mem_cfg, self.mem_ws),
                                                       (self.cfg, self.sel_ws))]


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("groups,n,Hq,Hkv,aux", [(3, 4, 8, 2, False), (2, 5, 8, 1, True), (1, 3, 4, 4, True)])
def test_beams_decode_as_if_everything_were_copied(groups, n, Hq, Hkv, aux, dt, paged):
    """Shared pages and moved state against slots of their own that are copied whole: the same outputs, bit by bit,
    tokens and scores, over steps that cross pages and fill the rings."""
    rng = random.Random(groups)
    tokens = [[rng.randrange(700) for _ in range(rng.randint(14, 40))] for _ in range(groups)]
    both = [Beams(shared, groups, n, Hq, Hkv, dt, paged, 2, aux) for shared in (True, False)]
    for b in both:
        b.scores.copy_(torch.arange(n).neg().float().repeat(groups))
        b.prompt(tokens)
    for step in range(40):
        for b in both:
            b.step()
        x, y = both
        assert torch.equal(x.length, y.length) and torch.equal(x.parent, y.parent) and torch.equal(x.token, y.token)
        assert torch.equal(x.out, y.out) and torch.equal(x.cross, y.cross) and torch.equal(x.scores, y.scores)
        for i in range(2):
            for b in both:
                if aux:
                    mac.mac_join_aux(b.rings[i].ring)
            torch.cuda.synchronize()
            for part in ("pos", "q", "o", "lse"):
                assert torch.equal(x.rings[i].ring_view(part), y.rings[i].ring_view(part)), (step, i, part)
    for b in both:
        assert b.status() == [0, 0, 0, 0]
    assert int(both[0].hits) == int(both[1].hits) > 0  # summaries are reused across reorderings
    if paged:  # histories have pages in common: fewer are held
        assert both[0].n_free.item() > both[1].n_free.item()
    for b in both:
        for r in b.rings:
            r.release()


def captured_step(b, side):
    """A graph of one step; the library's calls take the stream of the capture."""
    graph = torch.cuda.CUDAGraph()
    names = ("mac_build_tables", "mac_write_kv", "mac_cross_attention", "mac_beam_select", "mac_reorder_tables", "mac_reorder_state")
    keep = {x: getattr(mac, x) for x in names}
    for x in names:
        setattr(mac, x, lambda *a, f=keep[x]: f(*a, stream=torch.cuda.current_stream()))
    try:
        with torch.cuda.graph(graph, stream=side):
            b.step()
    finally:
        for x in names:
            setattr(mac, x, keep[x])
    return graph


def ready_beams(groups, n, dt, paged, seed):
    rng = random.Random(seed)
    b = Beams(True, groups, n, 8, 2, dt, paged, 2)
    b.hits = torch.zeros((), dtype=torch.int32, device=DEV)
    b.scores.copy_(torch.arange(n, device=DEV).neg().float().repeat(groups))
    b.prompt([[rng.randrange(700) for _ in range(20 + 9 * g)] for g in range(groups)])
    b.step()
    torch.cuda.synchronize()
    return b


def test_beams_decode_in_a_captured_graph():
    """One graph of a whole step, replayed, against the calls one by one."""
    plain, graphed = (ready_beams(3, 4, BF16, True, 9) for _ in range(2))
    graph = captured_step(graphed, torch.cuda.Stream())
    for _ in range(25):
        plain.step()
        graph.replay()
        torch.cuda.synchronize()
        for x in ("length", "parent", "token", "out", "cross", "scores", "table"):
            assert torch.equal(getattr(plain, x), getattr(graphed, x)), x
    assert plain.status() == graphed.status() == [0, 0, 0, 0]


@pytest.mark.parametrize("paged", [True, False])
def test_two_programs_of_beams_at_once(paged):
    """Two programs, each its own stream, workspaces, cache and graph, replayed side by side: each leaves what it leaves alone."""
    shapes = ((3, 4, BF16), (2, 5, F32))
    alone = []
    for groups, n, dt in shapes:
        b = ready_beams(groups, n, dt, paged, n)
        for _ in range(20):
            b.step()
        torch.cuda.synchronize()
        alone.append(b)
    both = [ready_beams(groups, n, dt, paged, n) for groups, n, dt in shapes]
    sides = [torch.cuda.Stream() for _ in both]
    graphs = [captured_step(b, side) for b, side in zip(both, sides)]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, side in zip(graphs, sides):
            with torch.cuda.stream(side):
                g.replay()
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        for name in ("length", "parent", "token", "out", "cross", "scores", "common"):
            assert torch.equal(getattr(x, name), getattr(y, name)), name
        for i in range(2):
            for part in ("pos", "q", "o", "lse"):
                assert torch.equal(x.rings[i].ring_view(part), y.rings[i].ring_view(part))
        assert y.status() == [0, 0, 0, 0]
