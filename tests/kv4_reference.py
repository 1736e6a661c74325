"""The 4-bit grid, decode attention with block weights and the eviction in 64 bits, in plain
numpy / torch on the CPU, for the tests of the 4-bit cache and of the eviction.

Tolerances (derived, not fitted). Attention: the kernels form every score from exact bf16 products
summed in float32, so a score is off by at most E = 130 * 2^-23 * max_t sum_c |q_c k_tc| / sqrt(d)
(130 additions and the scale, one truncation of 2^-23 each), a weight by a factor exp(2 E) (its own score and the
normaliser) and by the exponential's 2^-21; it is then rounded to fp16 (4-bit cache, 2^-11) or bf16
(bf16 cache, 2^-8) as a tensor-core operand, and the output to bf16 (2^-8 relative). So
  |out - ref| <= 2^-8 |ref| + (w_rounding + 2 E + 2^-20) * sum_t p_t |v_t|      (all terms per channel)
and a block's weight, whose terms are never rounded below float32,
  |mass - ref| <= (2 E + 2^-18) * w + 2^-22 * |mass|
(sums of at most 64 * 16 positive float32 terms in trees of depth below 32).
"""
import numpy as np
import torch

D, GROUP = 128, 32


def grid_values(x, key):
    """x bf16 [..., 128] -> float64 array of the values its 4-bit codes stand for."""
    T = torch.bfloat16 if key else torch.float16
    g = x.detach().cpu().float().reshape(-1, GROUP)
    out = torch.empty(g.shape, dtype=torch.float64)
    lo, hi = g.min(dim=1).values, g.max(dim=1).values
    finite = torch.isfinite(g).all(dim=1)
    s = ((hi - lo) / 15.0).to(T).double()
    z = (lo - (16.0 * s).float()).to(T).double()
    bad = ~finite | ~torch.isfinite(s) | ~torch.isfinite(z)
    s, z = torch.where(bad, torch.zeros_like(s), s), torch.where(bad, torch.full_like(z, float("nan")), z)
    diff = (g.double() - z[:, None]).float()                       # rounded once to float32
    step = torch.where(s > 0, s, torch.ones_like(s)).float()[:, None]
    code = ((diff / step) - 16.0).round().clamp(0, 15).double()
    code = torch.where((s > 0)[:, None], code, torch.zeros_like(code))
    # s (16 + code) is exact in float64, the sum is too: one rounding to T, by way of float32
    # rounded to odd so that it stays one
    out = s[:, None] * (16.0 + code) + z[:, None]
    return to_type(out, T).reshape(x.shape).numpy()


def to_type(x, T):
    """float64 -> T rounded to nearest even, once (through a float32 rounded to odd), as float64."""
    f = x.numpy().astype(np.float32)
    back = f.astype(np.float64)
    up = np.abs(back) > np.abs(x.numpy())
    f = np.where(up, np.nextafter(f, np.float32(0)), f)             # truncated
    inexact = f.astype(np.float64) != x.numpy()
    bits = f.view(np.uint32) | (inexact & np.isfinite(f)).astype(np.uint32)
    return torch.from_numpy(bits.view(np.float32).copy()).to(T).double()


def attention(q, k, v, blocks, T, w_rounding):
    """q [H, 128], k, v [cap, 128] float64; blocks: the attended blocks, in order, or None for all.
    -> (out [H, 128], out tolerance, weight of each listed block, its relative tolerance)."""
    if blocks is None:
        blocks = list(range((T - 1) // 64 + 1))
    tok = [np.arange(64 * j, min(64 * j + 64, T)) for j in blocks]
    H = q.shape[0]
    if not tok:
        return np.zeros((H, D)), np.zeros((H, D)), np.zeros(0), 0.0
    t = np.concatenate(tok)
    kk, vv = k[t], v[t]
    s = q @ kk.T / np.sqrt(D)
    p = np.exp(s - s.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    E = 130 * 2.0 ** -23 * float((np.abs(q) @ np.abs(kk).T).max()) / np.sqrt(D)
    out = p @ vv
    tol = 2.0 ** -8 * np.abs(out) + (w_rounding + 2 * E + 2.0 ** -20) * (p @ np.abs(vv)) + 1e-30
    edges = np.cumsum([0] + [len(x) for x in tok])
    w = np.array([p[:, edges[i]:edges[i + 1]].sum() for i in range(len(tok))])
    return out, tol, w, 2 * E + 2.0 ** -18


def kept_blocks(mass, n, keep, recent):
    """The blocks an eviction keeps of n, ascending."""
    if n <= keep:
        return list(range(n))
    forced = {0} | set(range(n - recent, n))
    rank = lambda j: (0 if np.isnan(mass[j]) else 1, -mass[j] if not np.isnan(mass[j]) else 0.0, j)
    rest = sorted((j for j in range(n) if j not in forced), key=rank)
    return sorted(forced | set(rest[:keep - len(forced)]))
