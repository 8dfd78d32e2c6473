"""GPU tests of fp32 chunk attention on both sides of its rule on rows per request (few rows on average: a kernel
that asks for keys ahead of queries), evenly and unevenly spread, against 64 bits.

Tolerances: as of fp32 chunk attention.  A score of up to 8 is off by 2^-21 of its terms' sizes in the mean square, by
2^-18 of it at most; a weight by e^that, an output by twice that times A = sum P |v|: 2^-16 A.  lse by 2^-18 |x| + 2^-22
|lse|: 2^-15."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from long_context_decode_gb300 import mac  # noqa: E402

D, PAGE, DEV = 128, 16, "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_decode_gb300 import build as b
    b.build()
    mac.load()


def attend(requests, Hq, Hkv, paged, pad=0):
    """requests: (new tokens, tokens with them)."""
    B, T, G = len(requests), sum(n for n, _ in requests) + pad, Hq // Hkv
    g = torch.Generator(device=DEV)
    g.manual_seed(B + T)
    cap = -(-max(m for _, m in requests) // PAGE) * PAGE
    k, v = (torch.randn(B, Hkv, cap, D, generator=g, device=DEV) for _ in range(2))
    for b, (_, m) in enumerate(requests):  # behind a request's tokens the cache may hold anything
        k[b, :, m:] = v[b, :, m:] = math.nan
    q = torch.randn(T, Hq, D, generator=g, device=DEV)
    start = [0]
    for n, _ in requests:
        start.append(start[-1] + n)
    out, lse = torch.full_like(q, 7), torch.full((T, Hq), 7.0, device=DEV)
    cfg = mac.config(B, Hq, Hkv, dtype=mac.MAC_F32, page_size=PAGE if paged else 0, max_context=cap)
    ws = torch.zeros(mac.mac_chunk_workspace_size(cfg, T), dtype=torch.uint8, device=DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    kv = mac.kv_view(k, v)
    if paged:
        ids = torch.randperm(B * cap // PAGE, generator=g, device=DEV)
        pools = [torch.empty(len(ids), Hkv, PAGE, D, device=DEV) for _ in range(2)]
        for x, pool in zip((k, v), pools):
            pool[ids] = x.view(B, Hkv, cap // PAGE, PAGE, D).transpose(1, 2).reshape(-1, Hkv, PAGE, D)
        table = ids.int().view(B, -1).contiguous()
        kv = mac.kv_view(*pools, table)
    mac.mac_chunk_attention(cfg, ws, q, ints(start), ints([m for _, m in requests]), T, kv, out, lse)
    assert mac.mac_last_status(cfg, ws) == 0
    assert (out[start[-1]:] == 7).all() and (lse[start[-1]:] == 7).all()
    for b, (n, m) in enumerate(requests):
        if n == 0:
            continue
        rows = slice(start[b], start[b + 1])
        kb, vb = (x[b, :, :m].double().repeat_interleave(G, 0) for x in (k, v))
        x = q[rows].double().transpose(0, 1) @ kb.transpose(1, 2) / math.sqrt(D)
        x = x.masked_fill(torch.arange(m, device=DEV)[None] >= torch.arange(m - n + 1, m + 1, device=DEV)[:, None], -math.inf)
        l = torch.logsumexp(x, -1)
        w = torch.exp(x - l[..., None])
        want, A = (w @ vb).transpose(0, 1), (w @ vb.abs()).transpose(0, 1)
        assert ((out[rows].double() - want).abs() <= 2.0 ** -16 * A).all()
        assert ((lse[rows].t().double() - l).abs() <= 2.0 ** -15).all()


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (8, 1), (4, 4)])
@pytest.mark.parametrize("requests", [
    [(1, 1)], [(1, 65)] * 3, [(1, 700), (1, 1), (1, 64), (0, 5), (1, 129)], [(2, 300)] * 5, [(3, 300)] * 5, [(8, 200)] * 4, [(9, 200)] * 4,
    [(0, 9)] * 15 + [(16, 400)],                  # one request's rows alone
    [(0, 9)] * 63 + [(64, 400)], [(64, 64)] + [(0, 9)] * 63, [(1, 90)] * 31 + [(33, 500)], [(1, 90)] * 250, [(130, 200)] + [(1, 77)] * 20,
])
def test_few_and_many_rows(requests, Hq, Hkv, paged):
    attend(requests, Hq, Hkv, paged, pad=len(requests) % 3)


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("new", [1, 2, 3])
def test_units_cut_over_many_ctas(new, paged):
    attend([(new, 9000), (new, 5000)], 8, 2, paged)
