"""Plain float64 forms of the attention of new tokens over a cache and of their store, for the tests."""
import torch

D, BLOCK = 128, 64


def ancestors(parent, n):
    """sees [n, n]: node j is node i or an ancestor of it. parent: a list, -1 for a root; one outside -1 .. i-1
    counts as -1. None: a chain."""
    sees = torch.zeros((n, n), dtype=torch.bool)
    for i in range(n):
        j = i
        while j >= 0:
            sees[i, j] = True
            p = j - 1 if parent is None else parent[j]
            j = p if -1 <= p < j else -1
    return sees


def attend(q, k, v, on):
    """(out, bound): q [R, D], k and v [K, D], on [R, K] in float64 -> softmax(q k / sqrt(d)) v [R, D] (zero where
    a row attends nothing), and how far a kernel's bf16 output may be from it.

    The kernel rounds each probability to bf16 (half a step is 2^-8 of it) before it meets the values, and
    the output once more: 2^-8 (sum p |v| + |out|) with sum p = 1. Its scores are float32 sums of 128 exact
    products, each addition off by 2^-23 at most of the sum so far (tensor cores may cut off instead of rounding), so a
    score is off by eta = 128 * 2^-23 * sum |q k| / sqrt(d) at most and a normalised probability by a factor of
    exp(2 eta); the float32 exponentials (2^-22) and sums over the keys (2^-23 each addition; kept by tile, a few
    hundred additions deep) add less than 2^-13 to that. eta is taken from the inputs.
    """
    if q.shape[0] == 0 or k.shape[0] == 0:
        zero = torch.zeros_like(q)
        return zero, zero + 1e-30
    z = (q @ k.T) / D**0.5
    z = torch.where(on, z, torch.full((), -torch.inf, dtype=torch.float64, device=q.device))
    top = z.amax(dim=1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.where(on, torch.exp(z - top), torch.zeros_like(z))
    s = e.sum(dim=1, keepdim=True)
    p = e / torch.where(s > 0, s, torch.ones_like(s))
    out, mag = p @ v, p @ v.abs()
    size = torch.where(on, q.abs() @ k.abs().T, torch.zeros_like(z)).amax(dim=1, keepdim=True) / D**0.5
    eta = 128 * 2.0**-23 * size
    rel = 2.0**-8 + torch.expm1(2 * eta) + 2.0**-13
    return out, 1.0001 * (rel * mag + 2.0**-8 * (out.abs() + rel * mag)) + 1e-30


def window_mean(keys):
    """keys bf16 [32, ...] -> their exact mean rounded once to bf16. A float64 sum of 32 bf16 values within
    2^40 of one another is exact, and so is the division by 32; the rounding to bf16 goes by way of a float32 rounded
    to odd, which no double rounding follows."""
    x = keys.double().sum(dim=0) / 32
    f = x.float()
    back = f.double()
    # round to odd: towards zero, then the last bit set where that lost something
    bits = f.view(torch.int32)
    away = (back.abs() > x.abs())
    bits = torch.where(away, bits - 1, bits)
    bits = torch.where(back != x, bits | 1, bits)
    return bits.view(torch.float32).to(torch.bfloat16)
