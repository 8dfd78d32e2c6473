"""fp32 chunk attention multiplies bf16 parts: a = a0 + a1 + a2, six of the
nine products of two such sums.  These tests tell the six apart: each fails,
on the CPU, for an emulation that leaves any one of them out, and holds for
the whole; the kernel then has to pass the same ones.

Tolerances, relative to 64 bits, with sums that the tensor cores may cut off
instead of rounding (by a unit of the largest term, 2^-23, per step of depth 16).
  random inputs: a score is off by 2^-21 |x| (eight steps of the largest
    product, cut by half a unit on average), |x| about 3 in the mean square and
    the same in all of a row to first order; a weight by that and 2^-22 (the
    exponential); the products left out are 2^-24 on average, 2^-21 at most.
    Outputs: below 2^-19 in the mean square (without one of the six 2^-18 at
    least), 2^-17 in a single row.  lse: below 2^-22 + 2^-21 |lse| in the mean square.
  inputs whose upper parts cancel: stated at each."""
import math

import pytest

torch = pytest.importorskip("torch")

D = 128
SIX = [(2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)]  # parts of the first and the second factor


def parts(x):
    """Three bf16 numbers (in 64 bits) whose sum is the fp32 number x, each cut off."""
    out, x = [], x.float()
    for _ in range(3):
        cut = (x.view(torch.int32) & -65536).view(torch.float32)
        out.append(cut.double())
        x = x - cut
    assert (x == 0).all()
    return out


def product(a, b, pairs):
    """a b^T over the last axis from parts, sums in 64 bits, rounded to fp32."""
    a, b = parts(a), parts(b)
    return sum(a[i] @ b[j].transpose(-1, -2) for i, j in pairs).float()


def emulate(q, k, v, scores=SIX, values=SIX):
    """Causal attention of the last q.shape[1] positions, [H, n, D], the way the kernel multiplies."""
    n, seen = q.shape[1], k.shape[1]
    late = torch.arange(seen)[None] > torch.arange(seen - n, seen)[:, None]
    x = (product(q, k, scores).double() / math.sqrt(D)).masked_fill(late, -math.inf)
    m = x.amax(-1, keepdim=True)
    w = torch.exp(x - m).float()
    z = w.double().sum(-1)
    return (product(w, v.transpose(-1, -2).contiguous(), values).double() / z[..., None]).float(), (m[..., 0] + z.log()).float()


def exact(q, k, v):
    q, k, v = q.double(), k.double(), v.double()
    n, seen = q.shape[1], k.shape[1]
    late = torch.arange(seen, device=q.device)[None] > torch.arange(seen - n, seen, device=q.device)[:, None]
    x = (q @ k.transpose(-1, -2) / math.sqrt(D)).masked_fill(late, -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[..., None]) @ v, lse


def kernel(q, k, v):
    from long_context_decode_gb300 import mac
    H, n, seen = q.shape[0], q.shape[1], k.shape[1]
    cfg = mac.config(1, H, H, dtype=mac.MAC_F32, max_context=seen)
    dev = "cuda"
    k, v, rows = (x.to(dev).contiguous() for x in (k[None], v[None], q.transpose(0, 1)))
    ws = torch.zeros(mac.mac_chunk_workspace_size(cfg, n), dtype=torch.uint8, device=dev)
    out, lse = torch.zeros(n, H, D, device=dev), torch.zeros(n, H, device=dev)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    mac.mac_chunk_attention(cfg, ws, rows, ints([0, n]), ints([seen]), n, mac.kv_view(k, v), out, lse)
    assert mac.mac_last_status(cfg, ws) == 0
    return out.transpose(0, 1).cpu(), lse.t().cpu()


# ---------------------------------------------------------------------------
# inputs, and what their outputs have to hold
# ---------------------------------------------------------------------------

def rms(x):
    return float(x.double().pow(2).mean().sqrt())


class Drawn:
    """Normal inputs, one heavy key per head."""

    def __init__(self, ctx, new, heads):
        g = torch.Generator().manual_seed(ctx + new)
        self.q = torch.randn(heads, new, D, generator=g)
        self.k, self.v = (torch.randn(heads, ctx + new, D, generator=g) for _ in range(2))
        self.k[:, 0] *= 3

    def holds(self, out, lse):
        want, l = exact(self.q, self.k, self.v)
        err = out.double() - want
        row = err.pow(2).mean(-1).sqrt() / want.pow(2).mean(-1).sqrt()
        return (rms(err) < 2.0 ** -19 * rms(want) and float(row.max()) < 2.0 ** -17
                and rms(lse.double() - l) < 2.0 ** -22 + 2.0 ** -21 * rms(l))


def base(part):
    """A number whose last part but `part` ends above 2^-15 (2^-23): 1, or 1 + 2^-8 with a part 1 of its own."""
    return 1.0 if part == 1 else 1 + 2.0 ** -8


def low_bits(j, part):
    """j 2^-15 (part 1) or j 2^-23 (part 2), j < 128: part `part` of base(part) + it, and nothing of the others."""
    return j * 2.0 ** (-15 if part == 1 else -23)


class Scores:
    """Scores from part `part` of K (or Q) alone: 2^s (base + low) in one column and -2^s base in another, s so
    that a low of 2^-8 (2^-16) is worth about 6.  The large terms cancel within one step or two, each of which
    may cut off 2^(s - 23), and the score's own last bit is as large: off by three of them over sqrt(D), an output
    by twice that times A = sum P |v|, and by 2^-20 A."""

    def __init__(self, part, of_k):
        g = torch.Generator().manual_seed(part)
        heads, seen = 6, 150
        s = 14 if part == 1 else 22
        cols = [(0, 1), (17, 64), (70, 5), (127, 63), (40, 47), (96, 111)]
        self.q, self.k = torch.zeros(heads, 1, D), torch.zeros(heads, seen, D)
        self.v = torch.randn(heads, seen, D, generator=g)
        for h, (a, b) in enumerate(cols):
            if of_k:
                self.q[h, 0, a], self.q[h, 0, b] = 2.0 ** s, -2.0 ** s
                self.k[h, :, a] = base(part) + low_bits(torch.randint(0, 128, (seen,), generator=g), part)
                self.k[h, :, b] = base(part)
            else:
                self.q[h, 0, a], self.q[h, 0, b] = base(part) + low_bits(100 + h, part), base(part)
                self.k[h, :, a] = 2.0 ** s * torch.randint(-1, 2, (seen,), generator=g)
                self.k[h, :, b] = -self.k[h, :, a]
        self.off = 3 * 2.0 ** (s - 23) / math.sqrt(D)

    def holds(self, out, lse):
        want, l = exact(self.q, self.k, self.v)
        A = exact(self.q, self.k, self.v.abs())[0]
        return bool(((out.double() - want).abs() <= (2 * self.off + 2.0 ** -20) * A).all()
                    and ((lse.double() - l).abs() <= self.off + 2.0 ** -20).all())


class Values:
    """Outputs from part `part` of V alone: equal weights (all scores zero) of base + low and -base.  Eight steps
    may cut off 2^-23 (2^-22 for terms above 1) of a sum that is divided by 128; the quotient rounds."""

    def __init__(self, part):
        g = torch.Generator().manual_seed(part + 10)
        self.q, self.k = torch.zeros(3, 1, D), torch.randn(3, 128, D, generator=g)
        self.v = torch.empty(3, 128, D)
        self.v[:, 0::2] = base(part) + low_bits(torch.randint(0, 128, (3, 64, D), generator=g), part)
        self.v[:, 1::2] = -base(part)

    def holds(self, out, lse):
        want, l = exact(self.q, self.k, self.v)
        return bool(((out.double() - want).abs() <= 2.0 ** -23 * want.abs() + 2.0 ** -26).all()) and rms(lse.double() - l) < 2.0 ** -20


class Weights:
    """Eight keys of weights near one, values of +1 and -1: what is left is from parts 1 and 2 of P.  Weights are
    off by 2^-22, above and below the line of an output of size 1 at most; with the sums' roundings below 2^-20."""

    def __init__(self):
        g = torch.Generator().manual_seed(20)
        self.q = torch.randn(64, 1, D, generator=g)
        self.k = torch.randn(64, 8, D, generator=g) * 2.0 ** -8
        self.v = (torch.randint(0, 2, (64, 8, D), generator=g) * 2 - 1).float()

    def holds(self, out, lse):
        want, l = exact(self.q, self.k, self.v)
        return bool(((out.double() - want).abs() <= 2.0 ** -20).all()) and rms(lse.double() - l) < 2.0 ** -20


CASES = {
    "7 after 100": lambda: Drawn(100, 7, 4), "300 from the start": lambda: Drawn(0, 300, 4),
    "40 after 5000": lambda: Drawn(5000, 40, 4), "3 after 20000": lambda: Drawn(20000, 3, 2),
    "K part 1": lambda: Scores(1, True), "K part 2": lambda: Scores(2, True), "Q part 1": lambda: Scores(1, False),
    "Q part 2": lambda: Scores(2, False), "V part 1": lambda: Values(1), "V part 2": lambda: Values(2),
    "P parts": Weights,
}
# the products that a case cannot do without: of scores, of values
NEEDS = {"K part 1": ([(0, 1)], []), "K part 2": ([(0, 2)], []), "Q part 1": ([(1, 0)], []), "Q part 2": ([(2, 0)], []),
         "V part 1": ([], [(0, 1)]), "V part 2": ([], [(0, 2)]), "P parts": ([], [(1, 0), (2, 0)])}


@pytest.mark.parametrize("name", CASES)
def test_the_six_products_are_enough_and_needed(name):
    c = CASES[name]()
    assert c.holds(*emulate(c.q, c.k, c.v))
    scores, values = NEEDS.get(name, (SIX, SIX))
    for out in scores:
        assert not c.holds(*emulate(c.q, c.k, c.v, scores=[x for x in SIX if x != out])), ("scores", out)
    for out in values:
        assert not c.holds(*emulate(c.q, c.k, c.v, values=[x for x in SIX if x != out])), ("values", out)


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_kernel(name):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    c = CASES[name]()
    assert c.holds(*kernel(c.q, c.k, c.v))
