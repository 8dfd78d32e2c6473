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
