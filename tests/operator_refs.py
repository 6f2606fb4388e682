"""Plain implementations in 64 bits of the operators around a verify step: the
definitions, request by request, and the error that each operator's roundings
allow.  They share no code with the CUDA path."""
import math

import numpy as np
import torch


# ---------------------------------------------------------------------------
# Verification from probabilities
# ---------------------------------------------------------------------------
def probs_request(p, q, drafts, u, u_last):
    """(accepted, token) of one request.  p [n + 1, V], q [n, V] or None (each draft
    certain), float64 of the stored values; u and u_last float32 values."""
    n = len(drafts)
    for i in range(n):
        x = int(drafts[i])
        qx = 1.0 if q is None else q[i][x]
        # both factors hold 24 bits: the product is exact
        if qx == 0.0 or float(u[i]) * qx < p[i][x]:
            continue
        w = p[i].copy()
        if q is None:
            w[x] = 0.0  # max(0, p - 1)
        else:
            w = np.maximum(w - q[i], 0.0)
        if not w.any():
            w = p[i]
        return i, draw(w, u_last)
    return n, draw(p[n], u_last)


def draw(w, u):
    """Smallest j whose prefix sum exceeds u times the total (V - 1 if none does), and
    whether a rounding of the sums could move it: the distance of u from the
    boundaries, over the total."""
    c = np.cumsum(w.astype(np.longdouble))
    goal = np.longdouble(u) * c[-1]
    j = int(np.searchsorted(c, goal, side="right"))
    return min(j, len(w) - 1)


# ---------------------------------------------------------------------------
# Append with rotation
# ---------------------------------------------------------------------------
def rotate(x, pos, inv_freq, interleaved, scale=1.0):
    """x [n, heads, D] float64, pos [n]: the first 2 len(inv_freq) values turned."""
    half = inv_freq.numel()
    ang = pos.double()[:, None] * inv_freq.double()[None, :]
    c, s = (ang.cos() * scale)[:, None, :], (ang.sin() * scale)[:, None, :]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return y


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def attend(q, k, v, seen, scale):
    """q [n, H, D], k, v [L, Hk, D], seen [n, L] bool, float64.  Returns o, lse, the
    largest |error| that the kernel's roundings allow for o (per element) and for lse,
    for weights rounded with unit roundoff u: see tolerance()."""
    n, H, D = q.shape
    r = H // k.shape[1]
    o = torch.zeros_like(q)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    spread = torch.zeros_like(q)   # sum of weights times |v|
    size = torch.zeros((n, H), dtype=torch.float64, device=q.device)
    for h in range(H):
        kh, vh = k[:, h // r], v[:, h // r]
        s = (q[:, h] @ kh.T) * scale
        s = torch.where(seen, s, -math.inf)
        m = s.amax(-1, keepdim=True) if s.shape[1] else torch.full((n, 1), -math.inf, device=q.device)
        some = torch.isfinite(m[:, 0])
        w = torch.exp(s - torch.where(some[:, None], m, 0.0))
        w = torch.where(seen, w, 0.0)
        den = w.sum(-1, keepdim=True)
        safe = torch.where(den > 0, den, 1.0)
        o[:, h] = (w @ vh) / safe
        spread[:, h] = (w @ vh.abs()) / safe
        lse[:, h] = torch.where(some, m[:, 0] + torch.log(safe[:, 0]), torch.full_like(m[:, 0], -math.inf))
        if s.shape[1]:
            size[:, h] = torch.where(seen, (q[:, h].abs() @ kh.abs().T) * scale, 0.0).amax(-1)
    return o, lse, spread, size


def tolerance(o, lse, spread, size, keys, D, vmax, dtype):
    """Allowed errors of o and lse.

    A score is a sum of D products in 32 bits, each addition off by at most 2^-24 of
    the sum of magnitudes: |ds| <= (D + 2) 2^-24 size (two more roundings for the
    scale).  ex2.approx is good to 2^-22, the running sum of `keys` weights to
    keys 2^-24 at worst (in parts of a quarter of a tile, then a tile, so far less:
    counted as 2^-18).  A weight is therefore off by d = |ds| + 2^-17 relative, and
    the rounding to the cache's type adds u = eps / 2.  fp16 weights below 2^-14 are
    off by 2^-25 each, and the largest weight is at least 1.  The output itself is
    rounded once more."""
    u = torch.finfo(dtype).eps / 2
    d = (D + 2) * 2.0 ** -24 * size + 2.0 ** -17
    tol = (u + 2 * d[..., None]) * 1.01 * spread + u * 1.01 * o.abs() + 1e-30
    if dtype == torch.float16:
        tol = tol + keys * 2.0 ** -25 * vmax + 2.0 ** -25
    return tol, d + 2.0 ** -22 * (1.0 + lse.abs())
