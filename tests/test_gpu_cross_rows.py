"""GPU tests of mac_cross_attention where several sources claim the same rows: which of them a row belongs to is not
specified, but every row that a well-formed source claims is written with the output of one that does."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from long_context_decode_gb300 import mac  # noqa: E402

D = 128
BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_decode_gb300 import build as b
    b.build()
    mac.load()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# capacities at which the host expects no unit to be cut; others where pieces are joined by the last of them, or merged
@pytest.mark.parametrize("dt,Hkv,cap", [(BF16, 1, 384), (F32, 1, 256), (BF16, 1, 2000), (BF16, 8, 384), (F32, 8, 1000), (BF16, 2, 4000)])
@pytest.mark.parametrize("starts", [lambda T: [0, T, 0, T, 0, T, 0], lambda T: [0, T // 2, 0, T, T // 3, T, T], lambda T: [T, 0, T, 5, 9, 0, T]])
def test_rows_of_several_sources(starts, dt, Hkv, cap):
    T = 1400 if Hkv == 1 else 96
    start = starts(T)
    B = len(start) - 1
    g = torch.Generator(device=DEV)
    g.manual_seed(cap)
    mem = [cap - 17 * b for b in range(B)]
    q = torch.randn(T, Hkv, D, generator=g, device=DEV).to(dt)
    k, v = (torch.randn(B, Hkv, cap, D, generator=g, device=DEV).to(dt) for _ in range(2))
    out, lse = torch.full_like(q, 7), torch.full((T, Hkv), 7.0, device=DEV)
    cfg = mac.config(B, Hkv, Hkv, dtype=mac.MAC_BF16 if dt == BF16 else mac.MAC_F32, max_context=cap)
    ws = torch.zeros(mac.mac_chunk_workspace_size(cfg, T), dtype=torch.uint8, device=DEV)
    mac.mac_cross_attention(cfg, ws, q, ints(start), 1, ints(mem), T, mac.kv_view(k, v), out, lse)
    assert mac.mac_last_status(cfg, ws) == mac.MAC_DEV_BAD_SEQ_LEN
    fits = torch.zeros(T, Hkv, D, dtype=torch.bool, device=DEV)
    lse_fits = torch.zeros(T, Hkv, dtype=torch.bool, device=DEV)
    for b in range(B):
        r0, r1 = start[b], start[b + 1]
        if r1 <= r0:
            continue
        x = torch.einsum("thd,hjd->thj", q[r0:r1].double(), k[b, :, :mem[b]].double()) / math.sqrt(D)
        l = torch.logsumexp(x, -1)
        w = torch.exp(x - l[..., None])
        want, A = (torch.einsum("thj,hjd->thd", w, u) for u in (v[b, :, :mem[b]].double(), v[b, :, :mem[b]].double().abs()))
        # scores of size 4 at most in sums of 128 products: 2^-19 with what tensor cores cut off; bf16 also rounds weights and outputs
        tol = A * 2.0 ** -16 + (2.0 ** -8 * (A + want.abs()) if dt == BF16 else 0)
        fits[r0:r1] |= (out[r0:r1].double() - want).abs() <= tol
        lse_fits[r0:r1] |= (lse[r0:r1].double() - l).abs() <= 2.0 ** -16
    claimed = torch.zeros(T, dtype=torch.bool, device=DEV)
    for b in range(B):
        claimed[start[b]:max(start[b], start[b + 1])] = True
    assert fits[claimed].all() and lse_fits[claimed].all()
    assert (out[~claimed] == 7).all()
    # the workspace serves a well-formed call afterwards
    start = [T * b // B for b in range(B + 1)]
    mac.mac_cross_attention(cfg, ws, q, ints(start), 1, ints(mem), T, mac.kv_view(k, v), out, lse)
    again, ws2 = torch.zeros_like(out), torch.zeros_like(ws)
    mac.mac_cross_attention(cfg, ws2, q, ints(start), 1, ints(mem), T, mac.kv_view(k, v), again, lse)
    assert mac.mac_last_status(cfg, ws) == 0 and torch.equal(out, again)
