"""fp32 cross attention of few rows multiplies two tf32 parts of each factor: a = a0 + a1, three of the four
products of two such sums, and adds a key tile's to the output in fp32.  The first tests tell the three products
apart: each fails, on the CPU, for an emulation that leaves one of them out, and holds for the whole; the kernel
then has to pass the same ones.  The others pin the sums over long memories: values of one sign, where what the
tensor cores cut off a sum adds up instead of cancelling.

Tolerances, relative to 64 bits.
  random inputs, as of fp32 chunk attention: outputs 2^-19 in the mean square (a score is off by 2^-21 |x|, |x| about 3
    in the mean square; without a product 2^-14 at least), 2^-17 in a single row; lse below 2^-22 + 2^-21 |lse| in the
    mean square.
  inputs whose upper parts cancel: stated at each.
  long memories of values in [1, 2]: a tile's sum is cut off at most three times by a unit of 2^-23, half of it on
    average: 2^-22.4, always towards zero.  Sums over tiles and of weights round to nearest, in the mean square (at
    131072 keys): a warp's 2048 additions by 2^-20.6, of the eight warps 2^-22.1; a lane's 4096 weights by 2^-20.1, of
    32 lanes 2^-22.6.  What scores are off by meets values that differ by 0.3 and averages over thousands of keys.  So
    the mean error is below 2^-21 and the mean square one below 2^-20, however many keys a CTA walks."""
import math

import pytest

torch = pytest.importorskip("torch")

D, PAGE = 128, 16
THREE = [(1, 0), (0, 1), (0, 0)]  # parts of the first and the second factor


def parts(x):
    """Two tf32 numbers (in 64 bits), rounded to 11 bits with halves away from zero."""
    out, x = [], x.float()
    for _ in range(2):
        cut = ((x.view(torch.int32) + 0x1000) & -0x2000).view(torch.float32)
        out.append(cut.double())
        x = x - cut
    return out


def product(a, b, pairs):
    """a b^T over the last axis from parts, sums in 64 bits, rounded to fp32."""
    a, b = parts(a), parts(b)
    return sum(a[i] @ b[j].transpose(-1, -2) for i, j in pairs).float()


def emulate(q, k, v, scores=THREE, values=THREE):
    """Attention of q's rows [H, n, D] over all keys, the way the kernel multiplies."""
    x = product(q, k, scores).double() / math.sqrt(D)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - m).float()
    z = w.double().sum(-1)
    return (product(w, v.transpose(-1, -2).contiguous(), values).double() / z[..., None]).float(), (m[..., 0] + z.log()).float()


def exact(q, k, v):
    q, k, v = q.double(), k.double(), v.double()
    x = q @ k.transpose(-1, -2) / math.sqrt(D)
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[..., None]) @ v, lse


def kernel(q, k, v):
    from long_context_decode_gb300 import mac
    H, n, seen = q.shape[0], q.shape[1], k.shape[1]
    assert n <= 16  # few rows
    cfg = mac.config(1, H, H, dtype=mac.MAC_F32, max_context=seen)
    dev = "cuda"
    k, v, rows = (x.to(dev).contiguous() for x in (k[None], v[None], q.transpose(0, 1)))
    ws = torch.zeros(mac.mac_chunk_workspace_size(cfg, n), dtype=torch.uint8, device=dev)
    out, lse = torch.zeros(n, H, D, device=dev), torch.zeros(n, H, device=dev)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    mac.mac_cross_attention(cfg, ws, rows, ints([0, n]), 1, ints([seen]), n, mac.kv_view(k, v), out, lse)
    assert mac.mac_last_status(cfg, ws) == 0
    return out.transpose(0, 1).cpu(), lse.t().cpu()


def rms(x):
    return float(x.double().pow(2).mean().sqrt())


class Drawn:
    """Normal inputs, one heavy key per head."""

    def __init__(self, seen, rows, heads):
        g = torch.Generator().manual_seed(seen + rows)
        self.q = torch.randn(heads, rows, D, generator=g)
        self.k, self.v = (torch.randn(heads, seen, D, generator=g) for _ in range(2))
        self.k[:, 0] *= 3

    def holds(self, out, lse):
        want, l = exact(self.q, self.k, self.v)
        err = out.double() - want
        row = err.pow(2).mean(-1).sqrt() / want.pow(2).mean(-1).sqrt()
        return (rms(err) < 2.0 ** -19 * rms(want) and float(row.max()) < 2.0 ** -17
                and rms(lse.double() - l) < 2.0 ** -22 + 2.0 ** -21 * rms(l))


def low(j):
    """j 2^-19, j < 128: the second part of 1 + it, whose first part is 1."""
    return j * 2.0 ** -19


class Scores:
    """Scores from the second part of K (or Q) alone: 2^18 (1 + low) in one column and -2^18 in another, so that a low
    of 2^-12 is worth about 6.  The large terms cancel, each of which may be cut off by 2^(18 - 23) up to three times:
    a score is off by that over sqrt(D), an output by twice that times A = sum P |v|, and by 2^-20 A."""

    def __init__(self, of_k):
        g = torch.Generator().manual_seed(1)
        heads, seen = 6, 150
        cols = [(0, 1), (17, 64), (70, 5), (127, 63), (40, 47), (96, 111)]
        self.q, self.k = torch.zeros(heads, 1, D), torch.zeros(heads, seen, D)
        self.v = torch.randn(heads, seen, D, generator=g)
        for h, (a, b) in enumerate(cols):
            if of_k:
                self.q[h, 0, a], self.q[h, 0, b] = 2.0 ** 18, -2.0 ** 18
                self.k[h, :, a] = 1 + low(torch.randint(0, 128, (seen,), generator=g))
                self.k[h, :, b] = 1
            else:
                self.q[h, 0, a], self.q[h, 0, b] = 1 + low(100 + h), 1
                self.k[h, :, a] = 2.0 ** 18 * torch.randint(-1, 2, (seen,), generator=g)
                self.k[h, :, b] = -self.k[h, :, a]
        self.off = 3 * 2.0 ** (18 - 23) / math.sqrt(D)

    def holds(self, out, lse):
        want, l = exact(self.q, self.k, self.v)
        A = exact(self.q, self.k, self.v.abs())[0]
        return bool(((out.double() - want).abs() <= (2 * self.off + 2.0 ** -20) * A).all()
                    and ((lse.double() - l).abs() <= self.off + 2.0 ** -20).all())


class Values:
    """Outputs from the second part of V alone: equal weights (all scores zero) of 1 + low and -1.  Sums of multiples
    of 2^-19 below 8 are exact; the quotient rounds."""

    def __init__(self):
        g = torch.Generator().manual_seed(10)
        self.q, self.k = torch.zeros(3, 1, D), torch.randn(3, 128, D, generator=g)
        self.v = torch.empty(3, 128, D)
        self.v[:, 0::2] = 1 + low(torch.randint(0, 128, (3, 64, D), generator=g))
        self.v[:, 1::2] = -1

    def holds(self, out, lse):
        want, l = exact(self.q, self.k, self.v)
        return bool(((out.double() - want).abs() <= 2.0 ** -23 * want.abs() + 2.0 ** -26).all()) and rms(lse.double() - l) < 2.0 ** -20


class Weights:
    """Eight keys of weights near one, values of +1 and -1: what is left is from the second part of P.  Weights are
    off by 2^-22, above and below the line of an output of size 1 at most; with the sums' roundings below 2^-20."""

    def __init__(self):
        g = torch.Generator().manual_seed(20)
        self.q = torch.randn(64, 1, D, generator=g)
        self.k = torch.randn(64, 8, D, generator=g) * 2.0 ** -8
        self.v = (torch.randint(0, 2, (64, 8, D), generator=g) * 2 - 1).float()

    def holds(self, out, lse):
        want, l = exact(self.q, self.k, self.v)
        return bool(((out.double() - want).abs() <= 2.0 ** -20).all()) and rms(lse.double() - l) < 2.0 ** -20


CASES = {"7 over 100": lambda: Drawn(100, 7, 4), "16 over 300": lambda: Drawn(300, 16, 4), "3 over 20000": lambda: Drawn(20000, 3, 2),
         "K": lambda: Scores(True), "Q": lambda: Scores(False), "V": Values, "P": Weights}
# the products that a case cannot do without: of scores, of values
NEEDS = {"K": ([(0, 1)], []), "Q": ([(1, 0)], []), "V": ([], [(0, 1)]), "P": ([], [(1, 0)])}


@pytest.mark.parametrize("name", CASES)
def test_the_three_products_are_enough_and_needed(name):
    c = CASES[name]()
    assert c.holds(*emulate(c.q, c.k, c.v))
    scores, values = NEEDS.get(name, (THREE, THREE))
    for out in scores:
        assert not c.holds(*emulate(c.q, c.k, c.v, scores=[x for x in THREE if x != out])), ("scores", out)
    for out in values:
        assert not c.holds(*emulate(c.q, c.k, c.v, values=[x for x in THREE if x != out])), ("values", out)


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_kernel(name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    c = CASES[name]()
    assert c.holds(*kernel(c.q, c.k, c.v))


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("Hq,Hkv,seen", [(8, 8, 4096), (8, 8, 32768), (32, 8, 16384), (1, 1, 131072)])
def test_sums_over_long_memories(Hq, Hkv, seen, sign):
    """So many sources that a CTA walks whole memories; they share their pages, so the cache is small."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_decode_gb300 import mac
    B, G, dev, looked = 1024 // Hkv, Hq // Hkv, "cuda", 64 // Hkv * 4
    g = torch.Generator(device=dev)
    g.manual_seed(seen)
    k = torch.randn(Hkv, seen, D, generator=g, device=dev)
    v = (torch.rand(Hkv, seen, D, generator=g, device=dev) + 1) * sign
    paged = [x.view(Hkv, seen // PAGE, PAGE, D).transpose(0, 1).contiguous() for x in (k, v)]
    table = torch.arange(seen // PAGE, device=dev).int()[None].repeat(B, 1).contiguous()
    q = torch.randn(B, Hq, D, generator=g, device=dev)
    cfg = mac.config(B, Hq, Hkv, dtype=mac.MAC_F32, page_size=PAGE, max_context=seen)
    ws = torch.zeros(mac.mac_chunk_workspace_size(cfg, B), dtype=torch.uint8, device=dev)
    out, lse = torch.zeros(B, Hq, D, device=dev), torch.zeros(B, Hq, device=dev)
    lengths = torch.full((B,), seen, dtype=torch.int32, device=dev)
    mac.mac_cross_attention(cfg, ws, q, torch.arange(B + 1, device=dev).int(), 1, lengths, B, mac.kv_view(*paged, table), out, lse)
    assert mac.mac_last_status(cfg, ws) == 0
    off, lse_off = [], []
    for h in range(Hkv):
        heads = slice(h * G, h * G + G)
        want, l = exact(q[:looked, heads].reshape(-1, D), k[h], v[h])
        off.append((out[:looked, heads].reshape(-1, D).double() - want) / want)
        lse_off.append(lse[:looked, heads].reshape(-1).double() - l)
    off, lse_off = torch.cat(off), torch.cat(lse_off)
    assert abs(float(off.mean())) < 2.0 ** -21 and rms(off) < 2.0 ** -20
    assert rms(lse_off) < 2.0 ** -20 + 2.0 ** -22 * math.log(seen)
