"""Batch calls (page tables, cache writes, chunk attention) without a GPU:
workspace sizes, struct layouts and refused arguments.  Every call here is
turned down before anything is enqueued."""
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


def test_struct_and_workspace_sizes(mac):
    assert ctypes.sizeof(mac.mac_pages) == 48
    cfg = mac.config(4, 32, 8, max_context=1 << 20)
    small, big = mac.mac_chunk_workspace_size(cfg, 1), mac.mac_chunk_workspace_size(cfg, 100000)
    assert 0 < small < big <= 300 << 20
    assert big == mac.mac_chunk_workspace_size(cfg, 1 << 20)  # a unit's rows are the most a partial holds
    assert big == mac.mac_chunk_workspace_size(mac.config(4, 32, 8, max_context=64), 100000)
    for n, code in ((0, mac.MAC_ERR_INVALID_ARG), (-5, mac.MAC_ERR_INVALID_ARG), (1 << 30, mac.MAC_ERR_UNSUPPORTED)):
        assert mac.load().mac_chunk_workspace_size(R(cfg), n, R(ctypes.c_size_t())) == code
    assert mac.load().mac_chunk_workspace_size(R(cfg), 5, None) == mac.MAC_ERR_INVALID_ARG
    bad = mac.config(1, 30, 8)
    assert mac.load().mac_chunk_workspace_size(R(bad), 5, R(ctypes.c_size_t())) == mac.MAC_ERR_INVALID_ARG


def refused(mac, fn, good, changes):
    """Each change of one argument is refused with its code."""
    f = getattr(mac.load(), fn)
    for i, value, code in changes:
        args = list(good)
        args[i] = value
        assert f(*args) == code, (fn, i, value)


def test_build_tables_refusals(mac):
    INV, UNS = mac.MAC_ERR_INVALID_ARG, mac.MAC_ERR_UNSUPPORTED
    cfg = mac.config(2, 8, 2, page_size=16, max_context=4096)

    def pages(**kw):
        base = dict(page_table=256, free_pages=256, n_free_in=256, n_free_out=256, capacity=0, max_pages=8, n_pages=8)
        base.update(kw)
        return R(mac.mac_pages(*[base[f[0]] for f in mac.mac_pages._fields_]))

    good = [R(cfg), 256, pages(), None, 256, 256, 4, 256, 256, 256, 256, None]
    refused(mac, "mac_build_tables", good, [
        (0, None, INV), (0, R(mac.config(2, 8, 2, page_size=8)), UNS), (1, None, INV), (1, 264, INV), (2, None, INV),
        (3, 258, INV), (4, None, INV), (4, 257, INV), (5, None, INV), (6, 0, INV), (6, -1, INV), (6, (1 << 24) + 1, UNS),
        (7, None, INV), (8, None, INV), (9, None, INV), (10, None, INV), (10, 260, INV),
        (2, pages(page_table=None), INV), (2, pages(free_pages=None), INV), (2, pages(n_free_in=None), INV),
        (2, pages(n_free_out=None), INV), (2, pages(max_pages=0), INV), (2, pages(n_pages=0), INV),
        (2, pages(page_table=258), INV)])
    flat = [R(mac.config(2, 8, 2, max_context=4096))] + good[1:]
    refused(mac, "mac_build_tables", flat, [(2, R(mac.mac_pages(None, None, None, None, 0, 0, 0)), INV)])


def test_write_kv_refusals(mac):
    INV, UNS = mac.MAC_ERR_INVALID_ARG, mac.MAC_ERR_UNSUPPORTED
    cfg = mac.config(2, 8, 2, max_context=4096)
    kv = mac.mac_kv(256, 256, None, 4096, 0, 0)
    good = [R(cfg), 256, 256, 1024, 256, 256, 256, 256, 256, 256, 4, R(kv), 512, None]
    refused(mac, "mac_write_kv", good, [
        (0, None, INV), (1, None, INV), (2, None, INV), (12, None, INV), (2, 264, INV), (12, 264, INV), (3, 1016, INV),
        (3, 1028, INV), (4, None, INV), (4, 260, INV), (5, 128, INV), (5, 260, INV), (6, None, INV), (7, 255, INV),
        (8, None, INV), (8, 258, INV), (9, None, INV), (9, 260, INV), (10, 0, INV), (10, 1 << 25, UNS), (11, None, INV),
        (11, R(mac.mac_kv(None, 256, None, 4096, 0, 0)), INV), (11, R(mac.mac_kv(256, 264, None, 4096, 0, 0)), INV),
        (11, R(mac.mac_kv(256, 256, None, 0, 0, 0)), INV)])
    strided_in_place = list(good)
    strided_in_place[2], strided_in_place[3], strided_in_place[12] = 512, 1536, 512
    assert mac.load().mac_write_kv(*strided_in_place) == INV
    paged = [R(mac.config(2, 8, 2, page_size=16))] + good[1:]
    refused(mac, "mac_write_kv", paged, [(11, R(mac.mac_kv(256, 256, None, 0, 8, 0)), INV)])


def test_write_kv_refuses_rows_whose_heads_are_apart(mac):
    torch = pytest.importorskip("torch")
    cfg = mac.config(2, 8, 2, max_context=4096)
    kv = mac.mac_kv(256, 256, None, 4096, 0, 0)
    x = torch.zeros(4, 8, 256, dtype=torch.bfloat16)
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(mac.MacError):
        mac.mac_write_kv(cfg, 256, x[..., :128], k, k, 256, 256, 4, kv, 512)


def test_row_stride_of_views(mac):
    torch = pytest.importorskip("torch")
    fused = torch.zeros(5, 12, 128, dtype=torch.bfloat16)
    assert mac._row_stride(fused[:, 8:10], 2, 128) == 12 * 128
    assert mac._row_stride(torch.zeros(5, 2, 128), 2, 128) == 256
    # one row of a cache-like [heads, T, d] tensor: its row stride says nothing
    assert mac._row_stride(torch.zeros(2, 1, 128).transpose(0, 1), 2, 128) == 256
    assert mac._row_stride(4096, 2, 128) == 256


def test_chunk_attention_refusals(mac):
    INV, UNS = mac.MAC_ERR_INVALID_ARG, mac.MAC_ERR_UNSUPPORTED
    cfg = mac.config(2, 8, 2, max_context=4096)
    kv = mac.mac_kv(256, 256, None, 4096, 0, 0)
    good = [R(cfg), 256, 256, 256, 256, 4, R(kv), 512, 256, None]
    refused(mac, "mac_chunk_attention", good, [
        (0, None, INV), (0, R(mac.config(2, 32, 2)), UNS), (1, None, INV), (1, 260, INV), (2, None, INV), (2, 264, INV),
        (3, None, INV), (3, 258, INV), (4, None, INV), (4, 258, INV), (5, 0, INV), (5, 1 << 25, UNS), (6, None, INV),
        (6, R(mac.mac_kv(256, None, None, 4096, 0, 0)), INV), (6, R(mac.mac_kv(264, 256, None, 4096, 0, 0)), INV),
        (6, R(mac.mac_kv(256, 256, None, 0, 0, 0)), INV), (7, None, INV), (7, 520, INV), (7, 256, INV), (8, 258, INV)])
    paged = [R(mac.config(2, 8, 2, page_size=16))] + good[1:]
    refused(mac, "mac_chunk_attention", paged, [(6, R(mac.mac_kv(256, 256, None, 0, 8, 8)), INV),
                                                (6, R(mac.mac_kv(256, 256, 256, 0, 8, 0)), INV)])


def test_a_misaligned_page_table_is_refused(mac):
    # the kernels read it in 4-byte words
    INV = mac.MAC_ERR_INVALID_ARG
    cfg = mac.config(2, 8, 2, page_size=16, max_context=4096)
    kv = R(mac.mac_kv(256, 256, 258, 0, 8, 8))
    L = mac.load()
    assert L.mac_chunk_attention(R(cfg), 256, 256, 256, 256, 4, kv, 512, 256, None) == INV
    assert L.mac_full_attention(R(cfg), 256, 256, 256, kv, 512, None, None) == INV
    assert L.mac_full_attention_noalloc(R(cfg), 256, 256, kv, 512, None, None) == INV
    assert L.mac_decode_step(R(cfg), 256, 256, 256, 256, kv, 512, None, None, None) == INV
    assert L.mac_init_rings(R(cfg), 256, 256, 256, 256, 1, kv, None) == INV


def test_binding_refuses_tensors_that_the_calls_cannot_take(mac):
    # the library sees addresses only: rows apart, or fewer than n_tokens, would be read and written at the wrong places
    torch = pytest.importorskip("torch")
    cfg = mac.config(2, 8, 2, max_context=4096)
    kv = mac.mac_kv(256, 256, None, 4096, 0, 0)
    fused = torch.zeros(4, 12, 128, dtype=torch.bfloat16)
    q, k, v = fused[:, :8], fused[:, 8:10], fused[:, 10:]
    whole = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    for out in (q, whole[:3], whole.transpose(0, 1)):  # q_out: a row's heads and the rows end to end, n_tokens of them
        with pytest.raises(mac.MacError, match="q_out"):
            mac.mac_write_kv(cfg, 256, whole, k, v, 256, 256, 4, kv, out)
    for args in ((whole[:3], k, v), (whole, k[:3], v), (whole, k, v[:3]), (whole, k[:, :1], v), (whole[0], k, v)):
        with pytest.raises(mac.MacError):
            mac.mac_write_kv(cfg, 256, *args, 256, 256, 4, kv, 512)
    for args in ((q, whole), (whole, q), (whole[:3], whole), (whole, whole[:3]), (whole, whole[:, :4])):
        with pytest.raises(mac.MacError, match="mac_chunk_attention"):
            mac.mac_chunk_attention(cfg, 256, args[0], 256, 256, 4, kv, args[1])
    with pytest.raises(mac.MacError, match="lse"):
        mac.mac_chunk_attention(cfg, 256, whole, 256, 256, 4, kv, whole.clone(), torch.zeros(8, 4).t())
