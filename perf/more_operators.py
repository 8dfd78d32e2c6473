"""The operators of beam search and of decoders with an encoder: what is measured, and their plain forms.

A step of beam search over a decoder that also attends an encoder's states makes four kinds of calls.
`cross` attends the new tokens of all beams of a source over the keys and values of that source's
encoder states; `select` picks the next beams from the logits of all beams of a group over the whole
vocabulary; `tables` gives every slot its new parent's history: cache pages, lengths, and which
positions its state has to be moved for; `state` moves that state within a layer: the rings of queries
and summaries, the keys and values of a cache without pages, the last page of one with pages.

`own` False computes each operator with elementary torch operations in 32 bits (64 for the scores that
the selection orders by); `own` True calls this repository's library.
"""
import math
import random

import torch

own = False

PAGE = 16
DIM = 128
MOVE = 8  # numbers of a slot's move: slot copied from, first and last position, its length, page copied from and to, rows of it, 0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(op, name=None, **kw):
    c = {"op": op, "groups": 1, "beams": 4, "lens": 1}
    if op == "cross":
        c.update(heads=32, kv_heads=8, dtype="bf16", paged=False, mem_lo=1, mem_hi=1, new_lo=1, new_hi=1, pad=0, empty=0)
    if op == "select":
        c.update(vocab=32000, gap=0, dtype="bf16", out=4, placed=True, done=0)
    if op == "tables":
        c.update(heads=32, kv_heads=8, paged=True, len_lo=1, len_hi=1, apart=8, ragged=0, fork=False, released=0)
    if op == "state":
        c.update(heads=32, kv_heads=8, dtype="bf16", paged=True, ring=512, len_lo=1, len_hi=1, apart=8, fork=False)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # the shortest call: one token over the states of a few words
        _case("cross", "cross-one", beams=1, heads=8, kv_heads=2, mem_lo=57, mem_hi=57),
        # a decode step of beams over sources of ordinary lengths
        _case("cross", "cross-beams", groups=16, mem_lo=400, mem_hi=1500, lens=2),
        # a decode step over long documents, their states in pages
        _case("cross", "cross-long", groups=4, beams=5, paged=True, mem_lo=8192, mem_hi=32768, lens=3),
        # given answers of odd lengths scored against their documents
        _case("cross", "cross-rows", groups=8, beams=1, paged=True, mem_lo=1000, mem_hi=4096, new_lo=100, new_hi=512, lens=4, pad=3),
        # a decode step of beams in single precision
        _case("cross", "cross-f32", groups=4, dtype="f32", mem_lo=300, mem_hi=1500, lens=5),
        # one source's beams
        _case("select", "select-one"),
        # a serving batch over a large vocabulary
        _case("select", "select-batch", groups=16, vocab=128000, lens=7),
        # wide beams over single-precision logits of an odd vocabulary, twice as many candidates as beams, some beams finished
        _case("select", "select-wide", groups=32, beams=8, vocab=50001, gap=7, dtype="f32", out=16, placed=False, done=5, lens=8),
        # one step of a serving batch: beams change slots, recent pages are given back, last pages parted
        _case("tables", "tables-step", groups=16, len_lo=1000, len_hi=8192, lens=9),
        # beams opened on prompts that one slot of each group has read
        _case("tables", "tables-fork", groups=16, beams=8, len_lo=1, len_hi=32768, fork=True, lens=10),
        # one layer's state in such a step
        _case("state", "state-step", groups=8, len_lo=500, len_hi=2048, apart=12, lens=11),
        # one layer's whole state when beams are opened, single precision without pages
        _case("state", "state-fork", groups=2, heads=8, kv_heads=2, dtype="f32", paged=False, ring=1024, len_lo=300, len_hi=2048,
              fork=True, lens=12),
    ]


def _log_int(rng, lo, hi):
    """Whole number of [lo, hi], spread over the logarithm."""
    lo1, hi1 = math.log(lo + 1), math.log(hi + 1)
    return max(lo, min(hi, int(math.exp(lo1 + (hi1 - lo1) * rng.random())) - 1 + rng.randint(0, 1)))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross", "select", "select", "tables", "state"])
    lens = rng.randrange(1 << 20)
    heads, kv_heads = rng.choice([(32, 8), (32, 4), (8, 2), (8, 4), (4, 4), (1, 1)])
    if op == "cross":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        groups, beams = _log_int(rng, 1, 16), rng.choice([1, 1, 2, 4, 5])
        new_hi = rng.choice([1, 1, _log_int(rng, 2, 512)])
        mem_hi = _log_int(rng, 1, 32768)
        case = _case(op, groups=groups, beams=beams, heads=heads, kv_heads=kv_heads, dtype=dtype, paged=rng.random() < 0.5,
                     mem_lo=max(1, mem_hi // rng.choice([1, 4, 50])), mem_hi=mem_hi, new_lo=0 if new_hi > 1 else 1, new_hi=new_hi, lens=lens,
                     pad=rng.choice([0, rng.randint(1, 20)]), empty=rng.choice([0, 0, 6]))
        while work(case)["bytes"] > 300e6 or work(case)["flops"] > (5e9 if dtype == "f32" else 80e9):
            case.update(groups=max(1, case["groups"] // 2), new_hi=max(1, case["new_hi"] * 2 // 3), mem_hi=case["mem_hi"] * 4 // 5,
                        mem_lo=max(1, case["mem_lo"] * 4 // 5))
        return case
    if op == "select":
        beams, vocab = rng.choice([1, 2, 3, 4, 5, 8, 16]), _log_int(rng, 100, 128000)
        groups = _log_int(rng, 1, max(1, min(32, (1 << 23) // (beams * vocab))))
        placed = rng.random() < 0.5
        return _case(op, groups=groups, beams=beams, vocab=vocab, gap=rng.choice([0, rng.randint(1, 9)]), dtype=rng.choice(["bf16", "f32"]),
                     out=beams if placed else rng.randint(1, 2 * beams), placed=placed, done=rng.choice([0, 3]), lens=lens)
    beams = rng.choice([2, 3, 4, 5, 8, 16])
    if op == "tables":
        return _case(op, groups=_log_int(rng, 1, 128 // beams), beams=beams, heads=8, kv_heads=2, paged=rng.random() < 0.8, len_lo=1,
                     len_hi=_log_int(rng, 16, 32768), apart=_log_int(rng, 1, 500), ragged=rng.choice([0, 0, 5]), fork=rng.random() < 0.3,
                     released=rng.choice([0, 4]), lens=lens)
    ring = rng.choice([128, 512, 1000, 1024])
    groups = _log_int(rng, 1, max(1, 512 * 512 // (beams * ring * max(1, heads // 16))) // 8 + 1)
    return _case(op, groups=min(groups, 32 // beams), beams=beams, heads=heads, kv_heads=kv_heads, dtype=rng.choice(["bf16", "bf16", "f32"]),
                 paged=rng.random() < 0.5, ring=ring, len_lo=1, len_hi=_log_int(rng, 16, 4096), apart=_log_int(rng, 1, 200),
                 fork=rng.random() < 0.3, lens=lens)


def _pages_of(n):
    return -(-n // PAGE)


def _es(case):
    return 4 if case["dtype"] == "f32" else 2


def _cross_lengths(case):
    """Encoder states of every source, and new tokens of every slot (a source's `beams` slots lie next to one another)."""
    rng = random.Random(case["lens"])
    mem = [rng.randint(case["mem_lo"], case["mem_hi"]) for _ in range(case["groups"])]
    if case["empty"]:  # sources without states
        mem = [0 if rng.randrange(case["empty"]) == 0 else n for n in mem]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["groups"] * case["beams"])]
    if not any(new):
        new[0] = 1
    return mem, new


def _history(case, chosen):
    """Per slot: length; the position after which it parts from the slot before it; its new parent within the group (-1: given up).

    `chosen`: parents that survive keep their slots, as after a selection that places them.  The others come as
    they may from one in order of score.
    """
    rng = random.Random(case["lens"])
    length, parts, parent = [], [], []
    n = case["beams"]
    for _ in range(case["groups"]):
        top = rng.randint(case["len_lo"], case["len_hi"])
        if case["fork"]:  # slot 0 has read the prompt, the others hold nothing
            length += [top] + [0] * (n - 1)
            parts += [0] * n
            parent += [0] * n
            continue
        low = top - 1 if case.get("ragged", 0) == 0 else max(1, top - case["ragged"]) - 1
        length += [top if case.get("ragged", 0) == 0 else rng.randint(low + 1, top) for _ in range(n)]
        parts += [0] + [rng.randint(max(0, low - case["apart"]), low) for _ in range(n - 1)]
        if case.get("released", 0) and rng.randrange(case["released"]) == 0:
            parent += [-1] * n
            continue
        up = [rng.randrange(n) for _ in range(n)]
        parent += [i if i in up else p for i, p in enumerate(up)] if chosen else up
    return length, parts, parent


def _shared(case, parts):
    """[slots, beams]: leading positions that a slot has in common with each of its group."""
    n = case["beams"]
    out = []
    for g in range(case["groups"]):
        d = parts[g * n:(g + 1) * n]
        out += [[0 if i == j else min(d[min(i, j) + 1:max(i, j) + 1]) for j in range(n)] for i in range(n)]
    return out


def work(case):
    n, S = case["beams"], case["groups"] * case["beams"]
    if case["op"] == "cross":
        mem, new = _cross_lengths(case)
        H, G = case["heads"], case["kv_heads"]
        rows = [sum(new[g * n:(g + 1) * n]) for g in range(case["groups"])]
        seen = sum(m for m, r in zip(mem, rows) if r)
        table = 4 * sum(_pages_of(m) for m, r in zip(mem, rows) if r) if case["paged"] else 0
        return {"bytes": 2 * seen * G * DIM * _es(case) + sum(rows) * H * (2 * DIM * _es(case) + 4) + table + 4 * (S + 1 + case["groups"]),
                "flops": 4 * DIM * H * sum(m * r for m, r in zip(mem, rows))}
    if case["op"] == "select":
        return {"bytes": S * case["vocab"] * _es(case) + 8 * S + 16 * case["groups"] * case["out"], "flops": 3 * S * case["vocab"]}
    length, parts, parent = _history(case, case["op"] == "state")
    shared = _shared(case, parts)
    total = 0
    for i, p in enumerate(parent):
        base = i // n * n
        if case["op"] == "tables":
            total += 4 * (3 + 2 * n + MOVE)
            if p != i - base and case["paged"]:  # the pages that change
                low = shared[i][p] // PAGE if p >= 0 else 0
                total += 4 * max(0, _pages_of(length[i]) - low) + (8 * max(0, _pages_of(length[base + p]) - low) if p >= 0 else 0)
            continue
        total += 4 * MOVE
        if p == i - base:
            continue
        low, last, its = shared[i][p], max(length[i], length[base + p]), length[base + p]
        total += 2 * min(last - low, case["ring"]) * (case["heads"] * (DIM * (_es(case) + 4) + 4) + 4)
        rows = its % PAGE if case["paged"] else max(0, its - low)
        total += 4 * rows * case["kv_heads"] * DIM * _es(case)
    return {"bytes": total, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).cuda()


def _prepare_cross(s, case, normal, gen):
    mem, new = _cross_lengths(case)
    H, G, n = case["heads"], case["kv_heads"], case["beams"]
    start = [0]
    for k in new:
        start.append(start[-1] + k)
    T = s["T"] = start[-1] + case["pad"]
    room = s["room"] = PAGE * (_pages_of(max(mem)) + 2)
    s["most"] = (max(start[(g + 1) * n] - start[g * n] for g in range(case["groups"])), max(1, max(mem)))  # what a padded batch is made for
    if case["paged"]:
        held = [_pages_of(m) for m in mem]
        width = room // PAGE
        n_pages = sum(held) + width
        ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        at = torch.cumsum(_ints([0] + held[:-1], torch.int64), 0)[:, None] + torch.arange(width, device="cuda")[None]
        s["table"] = torch.where(torch.arange(width, device="cuda")[None] < _ints(held, torch.int64)[:, None], ids[at.clamp(max=n_pages - 1)],
                                 torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous()
        s["k"], s["v"] = normal(n_pages, G, PAGE, DIM), normal(n_pages, G, PAGE, DIM)
    else:
        s["table"] = None
        s["k"], s["v"] = normal(case["groups"], G, room, DIM), normal(case["groups"], G, room, DIM)
    flat = s["k"].view(-1, DIM)  # a few heavy keys: sharp and flat rows both occur
    pick = torch.randint(0, flat.shape[0], (max(1, flat.shape[0] // 4096),), generator=gen, device="cuda")
    flat[pick] *= 4
    s["q"] = normal(T, H, DIM)
    s["q_start"], s["mem_len"] = _ints(start), _ints(mem)
    s["out"] = torch.zeros(T, H, DIM, dtype=s["q"].dtype, device="cuda")
    s["lse"] = torch.zeros(T, H, dtype=torch.float32, device="cuda")


def _prepare_select(s, case, normal, gen):
    S, V = case["groups"] * case["beams"], case["vocab"]
    x = normal(S, V + case["gap"])
    x *= 2.5
    peaks = torch.randint(0, V, (S, 1 + min(10, V // 10)), generator=gen, device="cuda")  # a few likely tokens
    x.scatter_(1, peaks, x.gather(1, peaks) + 6)
    s["logits"] = x[:, :V]
    s["scores"] = -8 * torch.rand(S, generator=gen, device="cuda")
    s["end"] = V // 3
    s["done"] = None
    if case["done"]:
        rng = random.Random(case["lens"])
        s["done"] = _ints([int(rng.randrange(case["done"]) == 0) for _ in range(S)])
        s["scores"] -= 10 * s["done"]  # finished ones compete with the others' next tokens
    rows = (case["groups"], case["out"])
    s["scores_out"] = torch.zeros(rows, device="cuda")
    s["parent"], s["token"], s["done_out"] = (torch.zeros(rows, dtype=torch.int32, device="cuda") for _ in range(3))


def _page_tables(case, length, parts, room, gen):
    """Pages of histories that part: a slot has the pages of the slot before it up to where they part.  -1 where nothing is held."""
    n, width = case["beams"], room // PAGE
    S = len(length)
    col = torch.arange(width, device="cuda")
    held = (_ints(length, torch.int64) + PAGE - 1) // PAGE
    same = _ints([p // PAGE for p in parts], torch.int64)
    source = torch.arange(S, device="cuda")[:, None].expand(S, width).clone()  # the slot whose page it is
    for j in range(1, n):
        source[j::n] = torch.where(col[None] < same[j::n, None], source[j - 1::n], source[j::n])
    ids = torch.randperm(S * width, generator=gen, device="cuda").to(torch.int32)
    return torch.where(col[None] < held[:, None], ids[source * width + col], torch.full((), -1, dtype=torch.int32, device="cuda")).contiguous(), ids


def _prepare_tables(s, case, normal, gen):
    length, parts, parent = _history(case, False)
    room = s["room"] = PAGE * (_pages_of(max(length)) + 2)
    S = len(length)
    s["parent"], s["len"] = _ints(parent), _ints(length)
    s["shared"] = _ints(_shared(case, parts))
    s["len_out"], s["shared_out"] = torch.zeros_like(s["len"]), torch.zeros_like(s["shared"])
    s["moves"] = torch.zeros(S, MOVE, dtype=torch.int32, device="cuda")
    if case["paged"]:
        s["table"], ids = _page_tables(case, length, parts, room, gen)
        used = torch.zeros(ids.shape[0], dtype=torch.bool, device="cuda")
        used[s["table"][s["table"] >= 0].long()] = True
        left = ids[~used[ids.long()]]
        s["free"] = torch.zeros_like(ids)
        s["free"][:left.shape[0]] = left
        s["n_free"], s["n_free_out"] = _ints([left.shape[0]]), _ints([0])


def _ring_parts(case):
    """Where the parts of a layer's rings lie in their workspace: bytes, shapes and types; and its size."""
    S, H, K, es = case["groups"] * case["beams"], case["heads"], case["ring"], _es(case)
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    at, parts = 0, {}
    for name, shape, dt in (("pos", (S, K), torch.int32), ("q", (S, H, K, DIM), torch.float32 if es == 4 else torch.bfloat16),
                            ("o", (S, H, K, DIM), torch.float32), ("lse", (S, H, K), torch.float32)):
        size = math.prod(shape) * dt.itemsize
        parts[name] = (at, size, shape, dt)
        at = up(at + size)
    for size in (S * H * DIM * es, S * H * DIM * 4, S * H * 4, 16 + 16 * S * H):  # a step's own
        at = up(at + size)
    return parts, at


def _prepare_state(s, case, normal, gen):
    length, parts, parent = _history(case, True)
    n, G, S, K = case["beams"], case["kv_heads"], len(length), case["ring"]
    room = s["room"] = PAGE * (_pages_of(max(length)) + 2)
    layout, total = _ring_parts(case)
    s["ring"] = torch.zeros(total, dtype=torch.uint8, device="cuda")
    view = {name: s["ring"][at:at + size].view(dt).view(shape) for name, (at, size, shape, dt) in layout.items()}
    for name in ("q", "o", "lse"):
        view[name].normal_(generator=gen)
    last = _ints(length)[:, None]
    c = torch.arange(K, dtype=torch.int32, device="cuda")[None]
    view["pos"].copy_((last - (last - c) % K).clamp(min=0))  # the newest position of every ring slot
    s["view"] = view
    shared = _shared(case, parts)
    moves, table = [], None
    if case["paged"]:
        table, ids = _page_tables(case, length, parts, room, gen)
        used = torch.zeros(ids.shape[0], dtype=torch.bool, device="cuda")
        used[table[table >= 0].long()] = True
        spare = ids[~used[ids.long()]].tolist()
        table = table.tolist()
        s["k"], s["v"] = normal(S * (room // PAGE), G, PAGE, DIM), normal(S * (room // PAGE), G, PAGE, DIM)
    else:
        s["k"], s["v"] = normal(S, G, room, DIM), normal(S, G, room, DIM)
    for i, p in enumerate(parent):
        src = i // n * n + p
        if src == i:
            moves.append([-1, 0, 0, 0, -1, -1, 0, 0])
            continue
        rows = length[src] % PAGE if case["paged"] else 0
        moves.append([src, shared[i][p] + 1, max(length[i], length[src]), length[src], table[src][length[src] // PAGE] if rows else -1,
                      spare.pop() if rows else -1, rows, 0])
    s["moves"] = _ints(moves)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16

    def normal(*shape):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(generator=gen)

    s = {"case": case}
    {"cross": _prepare_cross, "select": _prepare_select, "tables": _prepare_tables, "state": _prepare_state}[case["op"]](s, case, normal, gen)
    if own:
        from long_context_decode_gb300 import mac
        batch = case["groups"] * (1 if case["op"] == "cross" else case["beams"])
        s["cfg"] = mac.config(batch, case.get("heads", 8), case.get("kv_heads", 2), dtype=mac.MAC_F32 if case.get("dtype") == "f32" else mac.MAC_BF16,
                              ring_k=case.get("ring", 1024), page_size=PAGE if case.get("paged") else 0, max_context=s.get("room", 1))
        if case["op"] == "select":
            size = mac.mac_beam_workspace_size(s["cfg"], case["beams"], case["vocab"], case["out"])
        else:
            size = mac.mac_chunk_workspace_size(s["cfg"], s.get("T", 1))
        s["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
        if case["op"] == "cross":
            s["kv"] = mac.kv_view(s["k"], s["v"], s["table"])
        if case["op"] == "state":
            s["kv"] = mac.kv_view(s["k"], s["v"], n_pages=s["k"].shape[0])  # moves name pages themselves: no page table
    return s


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    from long_context_decode_gb300 import mac
    case, cfg, ws, stream = s["case"], s["cfg"], s["ws"], torch.cuda.current_stream()
    if case["op"] == "cross":
        mac.mac_cross_attention(cfg, ws, s["q"], s["q_start"], case["beams"], s["mem_len"], s["T"], s["kv"], s["out"], s["lse"], stream)
        return [s["out"], s["lse"]]
    if case["op"] == "select":
        mac.mac_beam_select(cfg, ws, case["beams"], s["logits"], s["scores"], s["done"], s["end"], case["out"], case["placed"], s["scores_out"],
                            s["parent"], s["token"], s["done_out"], stream)
        return [s["scores_out"], s["parent"], s["token"], s["done_out"]]
    if case["op"] == "tables":
        if not case["paged"]:
            mac.mac_reorder_tables(cfg, ws, None, case["beams"], s["parent"], s["len"], s["len_out"], s["shared"], s["shared_out"], s["moves"], stream)
            return [s["len_out"], s["shared_out"], s["moves"]]
        table, free = s["table"].clone(), s["free"].clone()  # both change: this pass works on its own
        mac.mac_reorder_tables(cfg, ws, mac.pages_view(table, free, s["n_free"], s["n_free_out"]), case["beams"], s["parent"], s["len"], s["len_out"],
                               s["shared"], s["shared_out"], s["moves"], stream)
        return [s["len_out"], s["shared_out"], s["moves"], table, free, s["n_free_out"]]
    mac.mac_reorder_state(cfg, ws, s["ring"], case["beams"], s["moves"], s["kv"], stream)
    return [s["view"]["pos"], s["view"]["q"], s["view"]["o"], s["view"]["lse"], s["k"], s["v"]]


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _cross(s):
    """All sources at once, padded to the most rows and the longest source."""
    case = s["case"]
    B, H, G, n = case["groups"], case["heads"], case["kv_heads"], case["beams"]
    rows, keys = s["most"]
    first = s["q_start"][::n].long()
    row = torch.arange(rows, device="cuda")
    at = first[:-1, None] + row
    live = at < first[1:, None]
    at = at.clamp(max=s["T"] - 1)
    q = s["q"][at].float().view(B, rows, G, H // G, DIM).permute(0, 2, 3, 1, 4).reshape(B, G, -1, DIM)
    if s["table"] is None:
        k, v = s["k"][:, :, :keys].float(), s["v"][:, :, :keys].float()
    else:
        ids = s["table"][:, :_pages_of(keys)].long().clamp(min=0)
        k, v = (x[ids].transpose(1, 2).flatten(2, 3)[:, :, :keys].float() for x in (s["k"], s["v"]))
    late = torch.arange(keys, device="cuda") >= s["mem_len"][:, None]
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(DIM)
    x.masked_fill_(late[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(m).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / z.clamp(min=1e-30)
    lse = torch.where(z > 0, m + torch.log(z), float("-inf"))
    to = at[live]
    s["out"][to] = o.view(B, G, H // G, rows, DIM).permute(0, 3, 1, 2, 4).reshape(B, rows, H, DIM)[live].to(s["out"].dtype)
    s["lse"][to] = lse.view(B, G, H // G, rows).permute(0, 3, 1, 2).reshape(B, rows, H)[live]
    return [s["out"], s["lse"]]


def _place(parent, rows):
    """Where each of a group's candidates, best first, goes so that a parent's best child is in the parent's slot; the others fill up in order."""
    n = parent.shape[1]
    order = torch.arange(n, device=parent.device)
    earlier = (parent[:, :, None] == parent[:, None, :]) & (order[None, :, None] > order[None, None, :])
    best = ~earlier.any(-1) & (parent >= 0)
    taken = ((parent[:, :, None] == order) & best[:, :, None]).any(1)
    free = torch.sort(taken.int(), dim=1, stable=True).indices
    at = torch.where(best, parent, free.gather(1, torch.where(best, 0, torch.cumsum(~best, 1) - 1)))
    return [torch.zeros_like(x).scatter_(1, at, x) for x in rows]


def _select(s):
    case = s["case"]
    B, n, V = case["groups"], case["beams"], case["vocab"]
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    score = x - (m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))) + s["scores"].double()[:, None]
    if s["done"] is not None:  # a finished beam goes on as it is
        done = s["done"][:, None] != 0
        score = torch.where(done, torch.where(torch.arange(V, device="cuda") == s["end"], s["scores"].double()[:, None], float("-inf")), score)
    best, at = torch.sort(score.view(B, n * V), dim=1, descending=True, stable=True)
    best, at = best[:, :case["out"]], at[:, :case["out"]]
    none = best == float("-inf")
    parent = torch.where(none, -1, at // V)
    token = torch.where(none, -1, at % V)
    over = none | (token == s["end"])
    if s["done"] is not None:
        over |= s["done"].view(B, n).gather(1, parent.clamp(min=0)) != 0
    got = [best.float(), parent.int(), token.int(), over.int()]
    return _place(parent, got) if case["placed"] else got


def _tables(s):
    case = s["case"]
    B, n = case["groups"], case["beams"]
    S = B * n
    slot = torch.arange(n, device="cuda")
    base = n * torch.arange(B, device="cuda")[:, None]
    parent = s["parent"].view(B, n).long()
    kept = parent >= 0
    up = parent.clamp(min=0)
    old = s["len"].view(B, n).long()
    new = torch.where(kept, old.gather(1, up), 0)
    s["len_out"].copy_(new.view(S))
    common = s["shared"].view(B, n, n).long()
    pairs = common.gather(1, up[:, :, None].expand(B, n, n)).gather(2, up[:, None, :].expand(B, n, n))
    pairs = torch.where(up[:, :, None] == up[:, None, :], (new[:, :, None] - 1).clamp(min=0), pairs)
    pairs = torch.where(slot[:, None] == slot, new[:, :, None], torch.where(kept[:, :, None] & kept[:, None, :], pairs, 0))
    s["shared_out"].copy_(pairs.view(S, n))
    moved = kept & (up != slot)
    first = common.gather(2, up[:, :, None])[..., 0] + 1
    # whoever keeps a history's last page: its own slot if that goes on, else the first of its children
    child = (parent[:, :, None] == slot) & kept[:, :, None]
    keeper = torch.where((parent == slot), slot, child.int().argmax(1))
    rows = new % PAGE if case["paged"] else torch.zeros_like(new)
    parted = kept & (rows > 0) & (keeper.gather(1, up) != slot)
    move = torch.zeros(B, n, MOVE, dtype=torch.long, device="cuda")
    move[..., 0] = torch.where(moved, base + up, -1)
    move[..., 1] = torch.where(moved, first, 0)
    move[..., 2] = torch.where(moved, torch.maximum(old, new), 0)
    move[..., 3] = torch.where(moved, new, 0)
    move[..., 4:6] = -1
    if not case["paged"]:
        s["moves"].copy_(move.view(S, MOVE))
        return [s["len_out"], s["shared_out"], s["moves"]]
    table, free = s["table"].clone(), s["free"].clone()
    W = table.shape[1]
    col = torch.arange(W, device="cuda")
    ids = torch.where(col < ((old + PAGE - 1) // PAGE)[..., None], table.view(B, n, W), -1)
    got = torch.where((col < ((new + PAGE - 1) // PAGE)[..., None]) & kept[..., None], ids.gather(1, up[..., None].expand(B, n, W)), -1)
    # pages that no slot of the group holds any more, each once, in order of group, page and slot
    seen = (ids[:, :, None] == got[:, None]).any(2)
    again = ((ids[:, :, None] == ids[:, None]) & (slot[:, None, None] > slot[None, :, None])).any(2)
    back = (ids >= 0) & ~seen & ~again
    b, c, j = torch.nonzero(back.permute(0, 2, 1), as_tuple=True)
    n_free = s["n_free"].long()
    free[n_free + torch.arange(b.shape[0], device="cuda")] = ids[b, j, c]
    n_free = n_free + b.shape[0]
    # a page of its own for every history that parts within a page
    place = torch.cumsum(parted.view(S), 0).view(B, n) - 1
    fresh = free[(n_free - 1 - place).clamp(min=0)].view(B, n)
    at = (new // PAGE).clamp(max=W - 1)
    whose = got.gather(2, at[..., None])[..., 0]
    got = torch.where((col == at[..., None]) & parted[..., None], fresh[..., None], got)
    move[..., 4] = torch.where(parted, whose.long(), -1)
    move[..., 5] = torch.where(parted, fresh.long(), -1)
    move[..., 6] = torch.where(parted, rows, 0)
    table.copy_(torch.where(got >= 0, got, table.view(B, n, W)).view(S, W))  # what lies behind a slot's pages stays
    s["n_free_out"].copy_(n_free - parted.sum())
    s["moves"].copy_(move.view(S, MOVE))
    return [s["len_out"], s["shared_out"], s["moves"], table, free, s["n_free_out"]]


def _state(s):
    case, view = s["case"], s["view"]
    src, first, last, length, page, to, rows = (s["moves"][:, i].long() for i in range(7))
    c = torch.arange(case["ring"], device="cuda")
    newest = last[:, None] - (last[:, None] - c) % case["ring"]  # the newest position of a ring slot
    i, at = torch.nonzero((src >= 0)[:, None] & (newest >= first[:, None].clamp(min=1)), as_tuple=True)
    view["pos"][i, at] = view["pos"][src[i], at]
    view["q"][i, :, at] = view["q"][src[i], :, at]
    view["o"][i, :, at] = view["o"][src[i], :, at]
    view["lse"][i, :, at] = view["lse"][src[i], :, at]
    if case["paged"]:
        i, at = torch.nonzero(torch.arange(PAGE, device="cuda") < rows[:, None], as_tuple=True)
        s["k"][to[i], :, at] = s["k"][page[i], :, at]
        s["v"][to[i], :, at] = s["v"][page[i], :, at]
    else:
        p = torch.arange(s["k"].shape[2], device="cuda")
        i, at = torch.nonzero((src >= 0)[:, None] & (p >= first[:, None] - 1) & (p < length[:, None]), as_tuple=True)
        s["k"][i, :, at] = s["k"][src[i], :, at]
        s["v"][i, :, at] = s["v"][src[i], :, at]
    return [view["pos"], view["q"], view["o"], view["lse"], s["k"], s["v"]]


def run(state):
    if own:
        return _run_own(state)
    return {"cross": _cross, "select": _select, "tables": _tables, "state": _state}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def _exact_cross(case, s):
    mem, new = _cross_lengths(case)
    H, G, n = case["heads"], case["kv_heads"], case["beams"]
    out, lse = s["out"].double(), s["lse"].double()
    row = 0
    for g, m in enumerate(mem):
        r = sum(new[g * n:(g + 1) * n])
        if m == 0:
            out[row:row + r], lse[row:row + r] = 0, float("-inf")
        else:
            t = torch.arange(m, device="cuda")
            if s["table"] is None:
                k, v = s["k"][g, :, :m], s["v"][g, :, :m]
            else:
                page = s["table"][g][t // PAGE].long()
                k, v = s["k"][page, :, t % PAGE].transpose(0, 1), s["v"][page, :, t % PAGE].transpose(0, 1)
            k, v = k.double(), v.double()
            for h in range(H):
                x = s["q"][row:row + r, h].double() @ k[h * G // H].t() * DIM ** -0.5
                l = torch.logsumexp(x, -1)
                out[row:row + r, h] = torch.exp(x - l[:, None]) @ v[h * G // H]
                lse[row:row + r, h] = l
        row += r
    return [out, lse]


def _exact_select(case, s):
    n, V, out = case["beams"], case["vocab"], case["out"]
    rows = []
    for g in range(case["groups"]):
        pool = []  # (score, beam, token) of the best of every beam
        for j in range(n):
            b = g * n + j
            so_far = float(s["scores"][b])
            if s["done"] is not None and int(s["done"][b]):
                pool.append((-so_far, j, s["end"], 1))
                continue
            p = torch.log_softmax(s["logits"][b].double(), -1)
            line = torch.topk(p, min(V, out)).values[-1]
            near = torch.nonzero(p >= line)[:, 0].tolist()
            pool += [(-(so_far + float(p[v])), j, v, int(v == s["end"])) for v in near]
        best = sorted(pool)[:out]
        best += [(float("inf"), -1, -1, 1)] * (out - len(best))
        if case["placed"]:
            rest = [None] * n
            for c in list(best):
                if c[1] >= 0 and rest[c[1]] is None:
                    rest[c[1]] = c
                    best.remove(c)
            best = [best.pop(0) if c is None else c for c in rest]
        rows.append([(-c[0], c[1], c[2], c[3]) for c in best])
    scores = torch.tensor([[c[0] for c in r] for r in rows], dtype=torch.float64).cuda()
    return [scores] + [_ints([[c[i] for c in r] for r in rows]) for i in (1, 2, 3)]


def exact(case, seed):
    if case["op"] in ("tables", "state"):
        return None  # whole numbers and copies: equality says it all
    if case["op"] == "cross":
        mem, new = _cross_lengths(case)
        if case["heads"] * sum(new) * max(mem) > 1 << 33:
            return None  # over about 20 seconds in 64 bits
        return _exact_cross(case, prepare(case, seed))
    return _exact_select(case, prepare(case, seed))
