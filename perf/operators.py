"""The operators that bring a batch of new tokens into the cache and attend them: what is measured, and their plain forms.

A serving step with new tokens is three calls.  `tables` gives every request the cache pages that its
new tokens need and lays the tokens out as packed rows with their positions and cache slots; `write`
rotates the rows' queries and keys and writes keys and values to their slots; `chunk` attends the rows
causally over the cache.  A decode step (one new token per request) runs the same calls.

`own` False computes each operator with elementary torch operations in 32 bits (64 for the rotation
angles); `own` True calls this repository's library.
"""
import math
import random

import torch

own = False

PAGE = 16
DIM = 128
ROPE_BASE = 10000.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(op, name=None, **kw):
    c = {"op": op, "batch": 1, "heads": 32, "kv_heads": 8, "dtype": "bf16", "paged": True,
         "ctx_lo": 0, "ctx_hi": 0, "new_lo": 1, "new_hi": 1, "lens": 1, "pad": 0}
    if op == "tables":
        c["resets"] = 0
    if op == "write":
        c.update(rope="half", fused=True)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of a serving batch: every request grows by one token, one in 16 needs a page
        _case("tables", "tables-decode", batch=16, ctx_lo=8192, ctx_hi=131072),
        # a step that admits prompts of odd lengths into reused slots, some requests idle
        _case("tables", "tables-prompts", batch=128, ctx_lo=1, ctx_hi=8192, new_lo=0, new_hi=2047, lens=2, pad=77, resets=4),
        # a decode step's keys and values, one token per request
        _case("write", "write-decode", batch=16, ctx_lo=8192, ctx_hi=131072, lens=3),
        # a step's budget of prompt tokens over several requests, projected as one fused q/k/v row
        _case("write", "write-prompts", batch=16, ctx_lo=0, ctx_hi=32768, new_lo=200, new_hi=1024, lens=4),
        # a single-precision cache without pages, interleaved rotation, ragged lengths
        _case("write", "write-f32", batch=4, ctx_lo=1, ctx_hi=4096, new_lo=257, new_hi=1021, lens=5, dtype="f32",
              paged=False, heads=32, kv_heads=4, rope="interleaved", fused=False, pad=3),
        # the shortest call: a few tokens after a short context
        _case("chunk", "chunk-short", ctx_lo=100, ctx_hi=100, new_lo=7, new_hi=7),
        # single tokens over long contexts, the cache contiguous
        _case("chunk", "chunk-decode-128k", batch=4, ctx_lo=131071, ctx_hi=131071, paged=False),
        # one chunk of a long prompt
        _case("chunk", "chunk-2k-at-32k", ctx_lo=30720, ctx_hi=30720, new_lo=2048, new_hi=2048),
        # a serving step: short and long chunks and idle slots together
        _case("chunk", "chunk-mixed", batch=16, ctx_lo=8192, ctx_hi=32768, new_lo=0, new_hi=512, lens=8, pad=5),
        # a whole prompt in one call
        _case("chunk", "chunk-prompt-16k", new_lo=16384, new_hi=16384, paged=False),
        # eight query heads per key head, odd lengths
        _case("chunk", "chunk-gqa8", batch=3, kv_heads=4, ctx_lo=1000, ctx_hi=30001, new_lo=99, new_hi=1501, lens=9),
        # single precision
        _case("chunk", "chunk-f32", batch=2, heads=8, kv_heads=2, dtype="f32", paged=False, ctx_lo=1000, ctx_hi=4096,
              new_lo=33, new_hi=300, lens=10),
    ]


def _log_int(rng, lo, hi):
    """Whole number of [lo, hi], spread over the logarithm."""
    lo1, hi1 = math.log(lo + 1), math.log(hi + 1)
    return max(lo, min(hi, int(math.exp(lo1 + (hi1 - lo1) * rng.random())) - 1 + rng.randint(0, 1)))


def draw(rng):
    op = rng.choice(["tables", "write", "chunk", "chunk"])
    lens = rng.randrange(1 << 20)
    heads, kv_heads = rng.choice([(32, 8), (32, 4), (8, 2), (8, 4), (4, 4), (1, 1)])
    paged = rng.random() < 0.6
    if op == "tables":
        batch = _log_int(rng, 1, 128)
        new = rng.choice([1, min(_log_int(rng, 2, 2047), (1 << 17) // batch)])
        return _case(op, batch=batch, heads=32, kv_heads=8, paged=rng.random() < 0.8, ctx_lo=1, ctx_hi=_log_int(rng, 16, 65536),
                     new_lo=rng.choice([0, 1]), new_hi=new, lens=lens, pad=rng.choice([0, rng.randint(1, 100)]), resets=rng.choice([0, 3, 8]))
    if op == "write":
        batch = _log_int(rng, 1, 16)
        return _case(op, batch=batch, heads=heads, kv_heads=kv_heads, dtype=rng.choice(["bf16", "bf16", "f32"]), paged=paged,
                     ctx_lo=0, ctx_hi=_log_int(rng, 1, 32768), new_lo=1, new_hi=min(_log_int(rng, 1, 1024), 9000 // batch), lens=lens,
                     pad=rng.choice([0, rng.randint(1, 50)]), rope=rng.choice(["half", "half", "interleaved", "none"]), fused=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    batch = _log_int(rng, 1, 16)
    if dtype == "f32":
        return _case(op, batch=min(batch, 4), heads=min(heads, 8), kv_heads=min(kv_heads, 2), dtype=dtype, paged=paged, ctx_lo=0,
                     ctx_hi=_log_int(rng, 1, 8192), new_lo=0, new_hi=_log_int(rng, 1, 512), lens=lens, pad=rng.choice([0, 9]))
    if rng.random() < 0.3:  # single tokens
        return _case(op, batch=batch, heads=heads, kv_heads=kv_heads, paged=paged, ctx_lo=1,
                     ctx_hi=min(_log_int(rng, 64, 131071), (1 << 19) // batch), lens=lens)
    ctx_hi = _log_int(rng, 1, 65536)
    new_hi = _log_int(rng, 1, 4096)
    while batch * new_hi * (ctx_hi + new_hi // 2) > (1 << 27):
        batch, new_hi = max(1, batch // 2), new_hi * 2 // 3
    return _case(op, batch=batch, heads=heads, kv_heads=kv_heads, paged=paged, ctx_lo=0, ctx_hi=ctx_hi, new_lo=0,
                 new_hi=new_hi, lens=lens, pad=rng.choice([0, rng.randint(1, 40)]))


def _lengths(case):
    """Tokens in the cache and new tokens of every request; where new_lo is 0 one request in eight brings none."""
    rng = random.Random(case["lens"])
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [rng.randint(max(1, case["new_lo"]), case["new_hi"]) for _ in range(case["batch"])]
    if case["new_lo"] == 0:
        new = [0 if rng.random() < 0.125 else n for n in new]
    if not any(new):
        new[0] = 1
    return ctx, new


def _resets(case):
    """Which requests' slots start over: one in `resets`."""
    rng = random.Random(case["lens"] + 1)
    return [case["resets"] > 0 and rng.randrange(case["resets"]) == 0 for _ in range(case["batch"])]


def _pages_of(n):
    return -(-n // PAGE)


def _capacity(case):
    """Tokens that a request's slot holds: whole pages, a few to spare."""
    ctx, new = _lengths(case)
    return PAGE * (_pages_of(max(c + n for c, n in zip(ctx, new))) + 2)


def _es(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    ctx, new = _lengths(case)
    rows, B = sum(new), case["batch"]
    H, G = case["heads"], case["kv_heads"]
    if case["op"] == "tables":
        gone = _resets(case)
        pages = pushed = 0
        for c, n, r in zip(ctx, new, gone):
            c0 = 0 if r else c
            pages += _pages_of(c0 + n) - _pages_of(c0)
            pushed += _pages_of(c) if r else 0
        if not case["paged"]:
            pages = pushed = 0
        return {"bytes": 16 * B + 4 + 12 * (rows + case["pad"]) + 8 * pages + 8 * pushed, "flops": 0}
    if case["op"] == "write":
        pairs = rows * (H + G) * DIM // 2
        return {"bytes": 2 * rows * (H + 2 * G) * DIM * _es(case) + 12 * (rows + case["pad"]),
                "flops": 0 if case["rope"] == "none" else 6 * pairs}
    seen = sum(c + n for c, n in zip(ctx, new) if n)
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    table = 4 * sum(_pages_of(c + n) for c, n in zip(ctx, new) if n) if case["paged"] else 0
    return {"bytes": 2 * seen * G * DIM * _es(case) + 2 * rows * H * DIM * _es(case) + 4 * rows * H + table + 8 * B,
            "flops": 4 * DIM * H * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).cuda()


def _table_and_stack(case, ctx, room, gen):
    """Shuffled pages: the requests' tables [B, room / PAGE] (-1 where nothing is held) and the stack of free ids."""
    held = [_pages_of(n) for n in ctx]
    width = room // PAGE
    n_pages = sum(held) + sum(width - h for h in held) // 2 + case["batch"] * 2 + width
    ids = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.cumsum(_ints([0] + held[:-1], torch.int64), 0)[:, None] + torch.arange(width, device="cuda")[None]
    table = torch.where(torch.arange(width, device="cuda")[None] < _ints(held, torch.int64)[:, None],
                        ids[at.clamp(max=n_pages - 1)], torch.full((), -1, dtype=torch.int32, device="cuda"))
    free = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    n_free = n_pages - sum(held)
    free[:n_free] = ids[sum(held):]
    return table.contiguous(), free, n_free, n_pages


def prepare(case, seed):
    ctx, new = _lengths(case)
    B, H, G = case["batch"], case["heads"], case["kv_heads"]
    rows = sum(new)
    T = rows + case["pad"]
    room = _capacity(case)
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.empty(shape, dtype=dt, device="cuda").normal_(generator=gen)

    s = {"case": case, "T": T, "room": room}
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    if case["op"] == "tables":
        s["len"], s["new"] = _ints(ctx), _ints(new)
        s["flags"] = _ints([int(r) for r in _resets(case)]) if case["resets"] else None
        s["len_out"], s["q_start"] = _ints([0] * B), _ints([0] * (B + 1))
        s["pos"] = torch.zeros(T, dtype=torch.int32, device="cuda")
        s["slot"] = torch.zeros(T, dtype=torch.int64, device="cuda")
        if case["paged"]:
            s["table"], s["free"], n_free, s["n_pages"] = _table_and_stack(case, ctx, room, gen)
            s["n_free"], s["n_free_out"] = _ints([n_free]), _ints([0])
    else:
        total = [c + n for c, n in zip(ctx, new)]
        if case["paged"]:
            s["table"], _, _, n_pages = _table_and_stack(case, total, room, gen)
            s["k"], s["v"] = normal(n_pages, G, PAGE, DIM), normal(n_pages, G, PAGE, DIM)
        else:
            s["table"] = None
            s["k"], s["v"] = normal(B, G, room, DIM), normal(B, G, room, DIM)
        if case["op"] == "write":
            b = torch.repeat_interleave(torch.arange(B, device="cuda"), _ints(new, torch.int64))
            p = torch.arange(rows, device="cuda") - _ints(start[:-1], torch.int64)[b] + _ints(ctx, torch.int64)[b]
            slot = s["table"][b, p // PAGE].long() * PAGE + p % PAGE if case["paged"] else b * room + p
            s["pos"] = torch.cat([(p + 1).int(), torch.zeros(case["pad"], dtype=torch.int32, device="cuda")])
            s["slot"] = torch.cat([slot, torch.full((case["pad"],), -1, dtype=torch.int64, device="cuda")])
            if case["fused"]:  # one projection's output, the three parts views of its rows
                qkv = normal(T, H + 2 * G, DIM)
                s["q"], s["k_new"], s["v_new"] = qkv[:, :H], qkv[:, H:H + G], qkv[:, H + G:]
            else:
                s["q"], s["k_new"], s["v_new"] = normal(T, H, DIM), normal(T, G, DIM), normal(T, G, DIM)
            s["q_out"] = torch.zeros(T, H, DIM, dtype=dt, device="cuda")
        else:
            # a few heavy keys in every head: sharp and flat rows both occur
            flat = s["k"].view(-1, DIM)
            pick = torch.randint(0, flat.shape[0], (max(1, flat.shape[0] // 8192),), generator=gen, device="cuda")
            flat[pick] *= 4
            s["q"] = normal(T, H, DIM)
            s["q_start"], s["len"] = _ints(start), _ints(total)
            s["out"] = torch.zeros(T, H, DIM, dtype=dt, device="cuda")
            s["lse"] = torch.zeros(T, H, dtype=torch.float32, device="cuda")
    if own:
        from long_context_decode_gb300 import mac
        s["cfg"] = mac.config(B, H, G, dtype=mac.MAC_F32 if case["dtype"] == "f32" else mac.MAC_BF16, rope_base=ROPE_BASE,
                              rope_mode={"half": mac.MAC_ROPE_HALF, "interleaved": mac.MAC_ROPE_INTERLEAVED,
                                         "none": mac.MAC_ROPE_NONE}[case.get("rope", "half")],
                              page_size=PAGE if case["paged"] else 0, max_context=room)
        s["ws"] = torch.zeros(mac.mac_chunk_workspace_size(s["cfg"], T), dtype=torch.uint8, device="cuda")
        if case["op"] != "tables":
            s["kv"] = mac.kv_view(s["k"], s["v"], s["table"])
    return s


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _run_own(s):
    from long_context_decode_gb300 import mac
    case, cfg, ws, stream = s["case"], s["cfg"], s["ws"], torch.cuda.current_stream()
    if case["op"] == "tables":
        table, free = s.get("table"), s.get("free")
        if not case["paged"]:
            pages = mac.pages_view(capacity=s["room"])
        else:
            if case["resets"]:  # a reset changes the table and the stack: this pass works on its own
                table, free = table.clone(), free.clone()
            pages = mac.pages_view(table, free, s["n_free"], s["n_free_out"])
        mac.mac_build_tables(cfg, ws, pages, s["flags"], s["len"], s["new"], s["T"], s["len_out"], s["q_start"], s["pos"],
                             s["slot"], stream)
        got = [s["len_out"], s["q_start"], s["pos"], s["slot"]]
        return got + [table, free, s["n_free_out"]] if case["paged"] else got
    if case["op"] == "write":
        mac.mac_write_kv(cfg, ws, s["q"], s["k_new"], s["v_new"], s["pos"], s["slot"], s["T"], s["kv"], s["q_out"], stream)
        return [s["q_out"], s["k"], s["v"]]
    mac.mac_chunk_attention(cfg, ws, s["q"], s["q_start"], s["len"], s["T"], s["kv"], s["out"], s["lse"], stream)
    return [s["out"], s["lse"]]


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _tables(s):
    case, T, dev = s["case"], s["T"], "cuda"
    B, room = case["batch"], s["room"]
    length, new = s["len"].long(), s["new"].long()
    request = torch.arange(B, device=dev)
    base = length if s["flags"] is None else torch.where(s["flags"] != 0, torch.zeros_like(length), length)
    end = torch.cumsum(new, 0)
    s["len_out"].copy_(base + new)
    s["q_start"][1:] = end
    s["q_start"][0] = 0
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(end, t, right=True)
    live = b < B
    b = b.clamp(max=B - 1)
    p = t - (end - new)[b] + base[b]
    s["pos"].copy_(torch.where(live, p + 1, torch.zeros_like(p)))
    if not case["paged"]:
        s["slot"].copy_(torch.where(live, b * room + p, torch.full_like(p, -1)))
        return [s["len_out"], s["q_start"], s["pos"], s["slot"]]
    table, free, n_free = s["table"], s["free"], s["n_free"].long()
    width = table.shape[1]
    col = torch.arange(width, device=dev)[None]
    if s["flags"] is not None:
        table, free = table.clone(), free.clone()
        held = torch.where(s["flags"] != 0, (length + PAGE - 1) // PAGE, torch.zeros_like(length))
        first = torch.cumsum(held, 0) - held
        row, c = torch.nonzero(col < held[:, None], as_tuple=True)
        free[n_free + first[row] + c] = table[row, c]
        n_free = n_free + held.sum()
    have = (base + PAGE - 1) // PAGE
    want = (base + new + PAGE - 1) // PAGE
    first = torch.cumsum(want - have, 0) - (want - have)
    row, c = torch.nonzero((col >= have[:, None]) & (col < want[:, None]), as_tuple=True)
    table[row, c] = free[n_free - 1 - (first[row] + c - have[row])]
    s["n_free_out"].copy_(n_free - (want - have).sum())
    slot = table[b, (p // PAGE).clamp(0, width - 1)].long() * PAGE + p % PAGE
    s["slot"].copy_(torch.where(live, slot, torch.full_like(slot, -1)))
    return [s["len_out"], s["q_start"], s["pos"], s["slot"], table, free, s["n_free_out"]]


def _rotate(x, pos, mode):
    """R(pos) x in 32 bits, the angles in 64."""
    x = x.float()
    if mode == "none":
        return x
    w = ROPE_BASE ** (-torch.arange(0, DIM, 2, dtype=torch.float64, device=x.device) / DIM)
    angle = (pos.double() - 1)[:, None, None] * w
    c, sn = torch.cos(angle).float(), torch.sin(angle).float()
    if mode == "half":
        a, b = x[..., :DIM // 2], x[..., DIM // 2:]
        return torch.cat([a * c - b * sn, b * c + a * sn], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)


def _write(s):
    case = s["case"]
    n = s["T"] - case["pad"]
    pos, slot, dt = s["pos"][:n], s["slot"][:n], s["q"].dtype
    s["q_out"][:n] = _rotate(s["q"][:n], pos, case["rope"]).to(dt)
    unit = PAGE if case["paged"] else s["room"]
    s["k"][slot // unit, :, slot % unit] = _rotate(s["k_new"][:n], pos, case["rope"]).to(dt)
    s["v"][slot // unit, :, slot % unit] = s["v_new"][:n]
    return [s["q_out"], s["k"], s["v"]]


def _history(s, b, n):
    """Keys and values of request b's first n tokens, [kv_heads, n, DIM]."""
    if s["table"] is None:
        return s["k"][b, :, :n], s["v"][b, :, :n]
    ids = s["table"][b, :_pages_of(n)].long()
    k, v = (x[ids].transpose(0, 1).flatten(1, 2)[:, :n] for x in (s["k"], s["v"]))
    return k, v


def _chunk(s):
    case = s["case"]
    ctx, new = _lengths(case)
    H, G = case["heads"], case["kv_heads"]
    row = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        if not n:
            continue
        k, v = _history(s, b, c + n)
        late = torch.arange(c + n, device="cuda")[None] > torch.arange(c, c + n, device="cuda")[:, None]
        q = s["q"][row:row + n].view(n, G, H // G, DIM)
        for g in range(G):  # a key head at a time keeps the scores within memory
            x = torch.matmul(q[:, g].float(), k[g].float().t()) / math.sqrt(DIM)
            x.masked_fill_(late[:, None], float("-inf"))
            m = x.amax(-1, keepdim=True)
            x = x.sub_(m).exp_()
            z = x.sum(-1, keepdim=True)
            o = torch.matmul(x, v[g].float()) / z
            heads = slice(g * (H // G), (g + 1) * (H // G))
            s["out"][row:row + n, heads] = o.to(s["out"].dtype)
            s["lse"][row:row + n, heads] = (m + torch.log(z))[..., 0]
        row += n
    return [s["out"], s["lse"]]


def run(state):
    if own:
        return _run_own(state)
    return {"tables": _tables, "write": _write, "chunk": _chunk}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers: equality says it all
    s = prepare(case, seed)
    ctx, new = _lengths(case)
    H, G = case["heads"], case["kv_heads"]
    if case["op"] == "write":
        rows = sum(new)
        out = [s["q_out"].double(), s["k"].double(), s["v"].double()]
        turn = torch.arange(DIM // 2, dtype=torch.float64, device="cuda").mul_(-2.0 * math.log(ROPE_BASE) / DIM).exp_()
        z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), (s["pos"][:rows].double() - 1)[:, None] * turn)[:, None]

        def turned(x):
            x = x[:rows].double()
            if case["rope"] == "none":
                return x
            pairs = x.unflatten(-1, (2, DIM // 2)).transpose(-1, -2) if case["rope"] == "half" else x.unflatten(-1, (DIM // 2, 2))
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
            return (y.transpose(-1, -2) if case["rope"] == "half" else y).flatten(-2)

        out[0][:rows] = turned(s["q"])
        for cache, rows_in in ((out[1], turned(s["k_new"])), (out[2], s["v_new"][:rows].double())):
            flat = cache.transpose(1, 2).flatten(0, 1)
            flat[s["slot"][:rows]] = rows_in
            cache.copy_(flat.unflatten(0, (cache.shape[0], cache.shape[2])).transpose(1, 2))
        return out
    if sum(n * (c + n) for c, n in zip(ctx, new)) * H > 1 << 34:
        return None  # over about 20 seconds in 64 bits
    out, lse = s["out"].double(), s["lse"].double()
    row = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        for lo in range(0, n, 256):
            hi = min(n, lo + 256)
            seen = c + hi
            if s["table"] is None:
                k, v = s["k"][b, :, :seen], s["v"][b, :, :seen]
            else:
                at = torch.arange(seen, device="cuda")
                page = s["table"][b][at // PAGE].long()
                k, v = s["k"][page, :, at % PAGE].transpose(0, 1), s["v"][page, :, at % PAGE].transpose(0, 1)
            k, v = k.double().repeat_interleave(H // G, 0), v.double().repeat_interleave(H // G, 0)
            q = s["q"][row + lo:row + hi].double().transpose(0, 1)
            x = torch.einsum("hqd,hkd->hqk", q, k) * DIM ** -0.5
            own_key = torch.arange(c + lo, c + hi, device="cuda")[:, None]
            x = torch.where(torch.arange(seen, device="cuda")[None] <= own_key, x, float("-inf"))
            l = torch.logsumexp(x, -1)
            out[row + lo:row + hi] = torch.einsum("hqk,hkd->hqd", torch.exp(x - l[..., None]), v).transpose(0, 1)
            lse[row + lo:row + hi] = l.t()
        row += n
    return [out, lse]
