"""GPU tests of slots that begin anew while other beams decode on: a group given up and opened on another prompt,
slots set back by reset flags, slots emptied for want of a page.  As everywhere, slots that share pages and move what
differs are compared, bit by bit, with slots of their own that are copied whole."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from long_context_decode_gb300 import mac  # noqa: E402
from test_gpu_beam import BF16, DEV, F32, Beams, ints, pages_of  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_decode_gb300 import build as b
    b.build()
    mac.load()


def begin(b, slots, tokens, how):
    """`slots` (of one group) begin anew: as a group's beams on one prompt, or (one slot) by itself."""
    flags = torch.zeros(b.S, dtype=torch.int32, device=DEV)
    flags[slots] = 1
    group, reset = slots[0] // b.n, flags
    stay = torch.arange(b.S, device=DEV) % b.n
    if b.shared and how == "parent":  # given back by a reordering
        up = stay.clone()
        up[slots] = -1
        b.take(up)
        assert (b.length[slots] == 0).all()
        reset = None
    elif b.shared:  # by flags: what the slots have in common with the others is the caller's to clear
        b.common[slots] = 0
        for s in slots:
            b.common[group * b.n:(group + 1) * b.n, s % b.n] = 0
    one = how == "one slot"
    new = [0] * b.S
    for s in slots if one or not b.shared else slots[:1]:
        new[s] = len(tokens)
    T = sum(new)
    ids = torch.tensor(tokens * (T // len(tokens)), device=DEV)
    mac.mac_build_tables(b.cfg, b.ws, b.pages, reset, b.length, ints(new), T, b.length, b.q_start, b.pos, b.slot)
    for i in range(b.layers):
        x = b.emb[i][ids]
        mac.mac_write_kv(b.cfg, b.ws, None, x[:, b.Hq:b.Hq + b.Hkv], x[:, b.Hq + b.Hkv:], b.pos, b.slot, T, b.kv[i], None)
        mac.mac_reset_requests(b.cfg, b.rings[i].ring, flags.clone())
    if not one:
        up = stay.clone()
        up[slots] = 0
        b.take(up)
        b.scores[slots] = -torch.arange(b.n, device=DEV).float()
    else:
        b.scores[slots] = b.scores[group * b.n:(group + 1) * b.n].max()  # it counts among the others
    b.token[slots] = torch.arange(len(slots), device=DEV).int() * 5 + 2


def same(x, y, aux):
    for name in ("length", "parent", "token", "out", "cross", "scores"):
        assert torch.equal(getattr(x, name), getattr(y, name)), name
    for b in (x, y):
        for r in b.rings:
            if aux:
                mac.mac_join_aux(r.ring)
    torch.cuda.synchronize()
    for i in range(x.layers):
        pos = [b.rings[i].ring_view("pos") for b in (x, y)]
        assert torch.equal(*pos)
        for part in ("q", "o", "lse"):  # (an emptied entry may hold anything)
            u, v = (b.rings[i].ring_view(part) for b in (x, y))
            held = (pos[0] > 0)[:, None].expand(-1, x.Hq, -1)
            assert torch.equal(u[held], v[held]), part


def both_decode(groups, n, dt, paged, aux, first, steps, how, again, more):
    rng = random.Random(first * 7 + n)
    draw = lambda k: [rng.randrange(700) for _ in range(k)]  # noqa: E731
    prompts, fresh = [draw(first + g) for g in range(groups)], draw(again)
    x, y = (Beams(shared, groups, n, 8, 2, dt, paged, 2, aux) for shared in (True, False))
    for b in (x, y):
        b.scores.copy_(torch.arange(n).neg().float().repeat(groups))
        b.prompt(prompts)
    for _ in range(steps):
        for b in (x, y):
            b.step()
        same(x, y, aux)
    slots = [n + 1] if how == "one slot" else list(range(n, 2 * n))  # of the second group
    for b in (x, y):
        begin(b, slots, fresh, how)
    assert torch.equal(x.length, y.length)
    hits = 0
    for _ in range(more):
        for b in (x, y):
            b.step()
        hits += int((x.matched[n:2 * n] >= 0).sum())
        same(x, y, aux)
    assert x.status() == y.status() == [0, 0, 0, 0]
    assert hits > 0  # the new histories' summaries are found, and only theirs
    if paged:  # nothing has got lost: held pages are on no stack, and all that are not held are
        table, length = x.table.tolist(), x.length.tolist()
        held = {table[s][c] for s in range(x.S) for c in range(pages_of(length[s]))}
        free = x.free[:x.n_free.item()].tolist()
        assert len(set(free)) == len(free) and not held & set(free) and len(held) + len(free) == len(x.free)
    for b in (x, y):
        for r in b.rings:
            r.release()


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("groups,n,aux", [(3, 4, False), (2, 5, True)])
def test_a_group_is_given_up_and_opened_on_another_prompt(groups, n, aux, dt, paged):
    both_decode(groups, n, dt, paged, aux, 18, 20, "parent", 37, 30)


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("how", ["flags", "one slot"])
@pytest.mark.parametrize("again", [4, 30])
def test_slots_without_a_common_page_begin_anew_by_flags(again, how, paged):
    # histories shorter than a page: every slot has its own.  What they have in common is cleared by the caller
    both_decode(2, 4, BF16, paged, False, 6, 5, how, again, 30)


def test_slots_of_a_contiguous_cache_begin_anew_by_flags():
    both_decode(3, 4, F32, False, False, 25, 15, "flags", 39, 25)


def test_slots_that_found_no_page_are_empty_and_begin_anew():
    """A child whose page is missing: length 0, a score that the caller takes out, rings that it resets."""
    b = Beams(True, 1, 4, 8, 2, BF16, True, 1)
    b.scores.copy_(torch.arange(4).neg().float())
    b.n_free.fill_(4)  # two pages for the prompt; three histories part, there are pages for two
    b.prompt([list(range(20))])
    assert mac.mac_last_status(b.cfg, b.ws) == mac.MAC_DEV_NO_ROOM
    assert b.length.tolist() == [20, 20, 20, 0] and b.n_free.item() == 0
    assert b.common[3].tolist() == [0] * 4 and b.common[:, 3].tolist() == [0] * 4
    empty = (b.length == 0).int()
    b.scores.masked_fill_(empty.bool(), -torch.inf)
    mac.mac_reset_requests(b.cfg, b.rings[0].ring, empty)
    logits = torch.randn(4, b.V, device=DEV)
    logits[3] += 100  # the empty slot's count for nothing
    mac.mac_beam_select(b.cfg, b.sel_ws, 4, logits, b.scores, None, -1, 4, 0, b.scores, b.parent, b.token)
    assert 3 not in b.parent.tolist() and torch.isfinite(b.scores).all()
    b.free[:10] = torch.arange(4, 14, device=DEV).int()
    b.n_free.fill_(10)
    b.take(b.parent)
    assert b.length.tolist() == [20] * 4
    for _ in range(4):
        b.step()
    assert b.status() == [0, 0, 0, 0]
    for r in b.rings:
        r.release()
