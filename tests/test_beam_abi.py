"""Beam search and encoder states without a GPU: sizes and refused arguments.
Every call here is turned down before anything is enqueued."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def mac():
    from long_context_decode_gb300 import build as b
    b.build()
    from long_context_decode_gb300 import mac as m
    m.load()
    return m


def R(x):
    return ctypes.byref(x)


def refused(mac, fn, good, changes):
    """Each change of one argument is refused with its code."""
    f = getattr(mac.load(), fn)
    for i, value, code in changes:
        args = list(good)
        args[i] = value
        assert f(*args) == code, (fn, i, value)


def test_cross_attention_refusals(mac):
    INV, UNS = mac.MAC_ERR_INVALID_ARG, mac.MAC_ERR_UNSUPPORTED
    cfg = mac.config(2, 8, 2, max_context=4096)
    kv = mac.mac_kv(256, 256, None, 4096, 0, 0)
    good = [R(cfg), 256, 256, 256, 4, 256, 4, R(kv), 512, 256, None]
    refused(mac, "mac_cross_attention", good, [
        (0, None, INV), (0, R(mac.config(2, 32, 2)), UNS), (1, None, INV), (1, 260, INV), (2, None, INV), (2, 264, INV),
        (3, None, INV), (3, 258, INV), (4, 0, INV), (4, -3, INV), (4, 1 << 24, UNS), (5, None, INV), (5, 258, INV), (6, 0, INV),
        (6, 1 << 25, UNS), (7, None, INV), (7, R(mac.mac_kv(256, None, None, 4096, 0, 0)), INV),
        (7, R(mac.mac_kv(264, 256, None, 4096, 0, 0)), INV), (7, R(mac.mac_kv(256, 256, None, 0, 0, 0)), INV), (8, None, INV),
        (8, 520, INV), (8, 256, INV), (9, 258, INV)])
    paged = [R(mac.config(2, 8, 2, page_size=16))] + good[1:]
    refused(mac, "mac_cross_attention", paged, [(7, R(mac.mac_kv(256, 256, None, 0, 8, 8)), INV),
                                                (7, R(mac.mac_kv(256, 256, 258, 0, 8, 8)), INV),
                                                (7, R(mac.mac_kv(256, 256, 256, 0, 8, 0)), INV)])


def test_cross_attention_binding_refuses_short_and_strided_tensors(mac):
    torch = pytest.importorskip("torch")
    cfg = mac.config(2, 8, 2, max_context=4096)
    kv = mac.mac_kv(256, 256, None, 4096, 0, 0)
    whole = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    strided = torch.zeros(4, 12, 128, dtype=torch.bfloat16)[:, :8]
    for q, out in ((strided, whole), (whole, strided), (whole[:3], whole), (whole, whole[:3])):
        with pytest.raises(mac.MacError, match="mac_cross_attention"):
            mac.mac_cross_attention(cfg, 256, q, 256, 1, 256, 4, kv, out)
    with pytest.raises(mac.MacError, match="lse"):
        mac.mac_cross_attention(cfg, 256, whole, 256, 1, 256, 4, kv, whole.clone(), torch.zeros(8, 4).t())


def test_constants_match_the_header(mac):
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "mac.h")).read()
    for name in ("MAC_MAX_BEAMS", "MAC_MAX_CANDIDATES", "MAC_DEV_BAD_PARENT", "MAC_DEV_NONFINITE_LOGIT"):
        assert int(re.search(rf"#define {name}\s+(\w+)", src).group(1), 0) == getattr(mac, name)


def test_beam_workspace_sizes(mac):
    INV, UNS = mac.MAC_ERR_INVALID_ARG, mac.MAC_ERR_UNSUPPORTED
    cfg = mac.config(8, 8, 2)
    small, big = mac.mac_beam_workspace_size(cfg, 4, 100, 4), mac.mac_beam_workspace_size(cfg, 4, 128000, 32)
    assert 0 < small < big < 1 << 20
    size = ctypes.c_size_t()
    for n, vocab, out, code in ((0, 10, 1, INV), (-1, 10, 1, INV), (3, 10, 1, INV), (16, 10, 1, INV), (17, 10, 1, UNS), (4, 0, 1, INV),
                                (4, (1 << 20) + 1, 1, UNS), (4, 10, 0, INV), (4, 10, 33, UNS)):
        assert mac.load().mac_beam_workspace_size(R(cfg), n, vocab, out, R(size)) == code, (n, vocab, out)
    assert mac.load().mac_beam_workspace_size(R(cfg), 4, 10, 4, None) == INV


def test_beam_select_refusals(mac):
    INV, UNS = mac.MAC_ERR_INVALID_ARG, mac.MAC_ERR_UNSUPPORTED
    cfg = mac.config(8, 8, 2)
    good = [R(cfg), 256, 4, 258, mac.MAC_BF16, 1001, 1000, 256, 256, 5, 4, 1, 512, 256, 256, 512, None]
    refused(mac, "mac_beam_select", good, [
        (0, None, INV), (1, None, INV), (1, 264, INV), (2, 0, INV), (2, 3, INV), (2, 17, UNS), (3, None, INV), (3, 257, INV), (4, 2, INV),
        (4, -1, INV), (4, mac.MAC_F32, INV), (5, 999, INV), (6, 0, INV), (6, 1 << 21, UNS), (7, None, INV), (7, 258, INV), (8, 257, INV),
        (9, -1, INV), (9, 1000, INV), (10, 0, INV), (10, 33, UNS), (10, 8, INV), (12, None, INV), (12, 514, INV), (13, None, INV), (13, 258, INV),
        (14, None, INV), (14, 258, INV), (15, 258, INV)])
    other = list(good)
    other[10], other[11] = 8, 0
    refused(mac, "mac_beam_select", other, [(12, 256, INV), (15, 256, INV)])  # in place, but laid out otherwise


def test_beam_select_binding_refuses_what_it_cannot_take(mac):
    torch = pytest.importorskip("torch")
    cfg = mac.config(8, 8, 2)
    x, s = torch.zeros(8, 50), torch.zeros(8)
    i = torch.zeros(8, dtype=torch.int32)
    for logits in (x.half(), x.t(), x[:7], x[:, ::2], x[0]):
        with pytest.raises(mac.MacError, match="logits"):
            mac.mac_beam_select(cfg, 256, 4, logits, s, None, -1, 4, 0, s, i, i)
    for name, args in (("scores", (s[:7], None, s, i, i, i)), ("done", (s, i[:4], s, i, i, i)), ("scores_out", (s, None, s[::2], i, i, i)),
                       ("parent", (s, None, s, i[:7], i, i)), ("token", (s, None, s, i, i[:1], i)), ("done_out", (s, None, s, i, i, i[:7]))):
        sc, done, so, parent, token, over = args
        with pytest.raises(mac.MacError, match=name):
            mac.mac_beam_select(cfg, 256, 4, x, sc, done, -1, 4, 0, so, parent, token, over)


def test_reorder_refusals(mac):
    INV, UNS = mac.MAC_ERR_INVALID_ARG, mac.MAC_ERR_UNSUPPORTED
    cfg = mac.config(8, 8, 2, page_size=16, max_context=4096)

    def pages(**kw):
        base = dict(page_table=256, free_pages=256, n_free_in=256, n_free_out=256, capacity=0, max_pages=8, n_pages=8)
        base.update(kw)
        return R(mac.mac_pages(*[base[f[0]] for f in mac.mac_pages._fields_]))

    good = [R(cfg), 256, pages(), 4, 256, 256, 256, 256, 256, 256, None]
    refused(mac, "mac_reorder_tables", good, [
        (0, None, INV), (1, None, INV), (1, 264, INV), (2, None, INV), (2, pages(page_table=None), INV), (2, pages(free_pages=258), INV),
        (2, pages(n_free_in=None), INV), (2, pages(n_free_out=None), INV), (2, pages(max_pages=0), INV), (2, pages(n_pages=0), INV),
        (3, 0, INV), (3, 3, INV), (3, 32, UNS), (4, None, INV), (4, 257, INV), (5, None, INV), (6, None, INV), (6, 258, INV), (7, None, INV),
        (8, None, INV), (8, 257, INV), (9, None, INV), (9, 264, INV)])
    flat = [R(mac.config(8, 8, 2, max_context=4096))] + good[1:]
    refused(mac, "mac_reorder_tables", flat, [(2, R(mac.mac_pages(None, None, None, None, 0, 0, 0)), INV)])

    kv = mac.mac_kv(256, 256, None, 0, 0, 8)
    good = [R(cfg), 256, 256, 4, 256, R(kv), None]
    refused(mac, "mac_reorder_state", good, [
        (0, None, INV), (1, None, INV), (1, 260, INV), (2, 264, INV), (3, 0, INV), (3, 5, INV), (3, 20, UNS), (4, None, INV), (4, 264, INV),
        (5, R(mac.mac_kv(None, 256, None, 0, 0, 8)), INV), (5, R(mac.mac_kv(256, 264, None, 0, 0, 8)), INV),
        (5, R(mac.mac_kv(256, 256, None, 0, 0, 0)), INV)])
    assert mac.load().mac_reorder_state(R(cfg), 256, None, 4, 256, None, None) == INV
    flat = [R(mac.config(8, 8, 2, max_context=4096))] + good[1:]
    refused(mac, "mac_reorder_state", flat, [(5, R(mac.mac_kv(256, 256, None, 0, 0, 8)), INV)])


def test_reorder_binding_refuses_short_and_strided_tensors(mac):
    torch = pytest.importorskip("torch")
    cfg = mac.config(8, 8, 2, max_context=4096)
    i, w, m = torch.zeros(8, dtype=torch.int32), torch.zeros(8, 4, dtype=torch.int32), torch.zeros(8, 8, dtype=torch.int32)
    good = dict(parent=i, len_in=i, len_out=i, shared_in=w, shared_out=w, moves=m)
    for name, bad in (("parent", i[:7]), ("len_in", m[:, 0]), ("len_out", i[:4]), ("shared_in", w.t()), ("shared_out", w[:7]), ("moves", m[:7])):
        with pytest.raises(mac.MacError, match=name):
            mac.mac_reorder_tables(cfg, 256, None, 4, **{**good, name: bad})
    with pytest.raises(mac.MacError, match="moves"):
        mac.mac_reorder_state(cfg, 256, 256, 4, m[:7], None)
