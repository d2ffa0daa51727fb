"""The definition of the cache attention in 64 bits, and how far a 16-bit result may be from it.

Per output element, with u half a step of the storage type (relative), o the exact output, A = sum_t p_t |v_t| over the
visible entries (p the exact weights), L their number and E = max_t scale * sum_d |q_d k_td|:
  the output's own rounding                       u |o|
  every weight rounded once for its product       u A
  32-bit sums of L products, and of L weights     2 * 2^-23 L A
  32-bit scores: D products and the exponent's
  argument, entering every weight twice
  (numerator and sum)                             2 * 2^-23 (D + 8) E A
  the exponential itself                          2^-20 A
  16-bit floats below 2^-14: weights (relative to a maximum, so their sum is at least 1) and outputs are rounded in
  steps of 2^-24                                  2^-25 (sum_t |v_t| + 1)
"""
import math

import numpy as np
import torch


def bound(u, D, half, o, A, L, E, sumv):
    """Elementwise bound; o, A, sumv [rows][D], L [rows], E [rows]."""
    e = u + 2 * 2.0 ** -23 * L + 2 * 2.0 ** -23 * (D + 8) * E + 2.0 ** -20
    tol = u * o.abs() + e[:, None] * A
    if half:
        tol = tol + 2.0 ** -25 * (sumv + 1)
    return tol * 1.001 + 1e-30


def attend(q, k, v, visible, scale, dtype):
    """q [R][Hq][D], k/v [L][Hkv][D] (any float type), visible [R][L] -> (o, tol) [R][Hq][D] in 64 bits.
    Entries that no row sees are dropped first, whatever they hold."""
    R, Hq, D = q.shape
    keep = visible.any(0)
    k, v, visible = k[keep].double(), v[keep].double(), visible[:, keep]
    q = q.double()
    G = Hq // k.shape[1]
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    u = torch.finfo(dtype).eps / 2
    L = visible.sum(1).double()
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        s = (q[:, h] @ kh.T) * scale
        s = s.masked_fill(~visible, -math.inf)
        p = torch.softmax(s, 1)
        e = ((q[:, h].abs() @ kh.abs().T) * scale).masked_fill(~visible, 0).amax(1)
        o = p @ vh
        out[:, h] = o
        tol[:, h] = bound(u, D, dtype == torch.float16, o, p @ vh.abs(), L, e,
                          visible.double() @ vh.abs())
    return out, tol


def tree_visible(n, parent):
    """[N][n + N]: the cache of n entries, then the nodes' own paths (parent None: a chain is passed as one)."""
    N = len(parent)
    own = torch.zeros(N, N, dtype=torch.bool)
    for i in range(N):
        at = i
        while at >= 0:
            own[i, at] = True
            at = int(parent[at])
    return torch.cat([torch.ones(N, n, dtype=torch.bool), own], 1)


def ring_positions(p, S, W):
    """The positions a cache of p committed entries holds that the next token may see."""
    return sorted(set(range(min(S, p))) | set(range(max(0, p - W), p)))


def slot(t, S, W):
    return t if t < S else S + (t - S) % W


def window_visible(at, t, S, W):
    at, t = torch.as_tensor(at)[:, None], torch.as_tensor(t)[None, :]
    return (t <= at) & ((t > at - W) | (t < S))


def random_parents(N, rng, kind="random"):
    if kind == "chain":
        return [-1] + list(range(N - 1))
    if kind == "star":
        return [-1] + [0] * (N - 1)
    return [-1] + [int(rng.integers(max(0, n - 6), n)) for n in range(1, N)]


def check(got, want, tol, what=""):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)  # NaN counts as off
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        worst = float((off / tol).nan_to_num(math.inf).max())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got "
                             f"{float(got[i])}, want {float(want[i])}, may be {float(tol[i])} off; "
                             f"worst {worst:.3g} of the bound")


def tensor(rng, shape, dtype, scale=1.0, device="cuda"):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(device).to(dtype)
