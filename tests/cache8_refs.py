"""Plain implementations, in 64 bits or whole numbers, of the operators on a cache of e4m3
codes and on a cache's pages.  They share no code with the CUDA path."""
import math

import torch

# every finite e4m3 magnitude, by its code: 4 exponent bits (bias 7), 3 of mantissa
MAGNITUDES = torch.tensor([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                           for e in range(16) for m in range(8)][:127], dtype=torch.float64)


def values(codes):
    """What codes (uint8) stand for: float64, NaN for 0x7f and 0xff."""
    table = torch.cat([MAGNITUDES, torch.tensor([math.nan], dtype=torch.float64)]).to(codes.device)
    x = table[(codes & 0x7f).long()]
    return torch.where(codes >= 128, -x, x)


def nearest(x):
    """x (float64) rounded to the nearest e4m3 value, ties to the even code, beyond 448 to 448."""
    mag = MAGNITUDES.to(x.device)
    a = x.abs().clamp_max(448.0)
    hi = torch.searchsorted(mag, a.contiguous()).clamp_max(126)
    lo = (hi - 1).clamp_min(0)
    up, down = mag[hi] - a, a - mag[lo]
    take = torch.where(up < down, hi, torch.where(up > down, lo, torch.where(hi % 2 == 0, hi, lo)))
    take = torch.where(mag[hi] == a, hi, take)
    return torch.where(torch.isnan(x), x, mag[take] * torch.where(x < 0, -1.0, 1.0))


def scale_of(most):
    """The smallest power of two s in [2^-32, 2^56] with 448 s >= most (float64)."""
    e = torch.ceil(torch.log2((most / 448.0).clamp(2.0 ** -200, 2.0 ** 200)))
    # (log2 of a power of two may be off by its last bit)
    exact = torch.tensor([2.0 ** i for i in range(-210, 211)], dtype=torch.float64, device=most.device)
    power = lambda x: exact[x.long() + 210]  # noqa: E731
    e = torch.where(448.0 * power(e - 1) >= most, e - 1, e)
    e = torch.where(448.0 * power(e) < most, e + 1, e)
    return power(e.clamp(-32, 56))


def longest(x, rot, interleaved, rope_scale=1.0):
    """[.., H]: the largest magnitude of a value, or of a turning pair (NaN left out)."""
    y = torch.nan_to_num(x, nan=0.0, posinf=math.inf, neginf=-math.inf)
    parts = [y[..., rot:].abs()]
    if rot:
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :rot // 2], y[..., rot // 2:rot])
        parts.append(torch.hypot(a, b) * rope_scale)
    return torch.cat(parts, -1).amax(-1)


class Pages:
    """The page table of a cache, row by row and reference by reference."""

    def __init__(self, table, kv_len, held, ref, free, page):
        self.table, self.kv, self.held = [list(r) for r in table], list(kv_len), list(held)
        self.ref, self.free, self.page = list(ref), list(free), page

    def step(self, tokens, parents=None):
        """Returns whether the takes fit, and the copies (source, destination, tokens)."""
        B, ps = len(self.table), self.page
        parents = list(range(B)) if parents is None else parents
        old = [r[:h] for r, h in zip(self.table, self.held)]
        kv = [0 if p < 0 else self.kv[p] for p in parents]
        n = [0 if p < 0 else t for p, t in zip(parents, tokens)]
        live = [-(-k // ps) for k in kv]
        rows = [[] if p < 0 else old[p][:x] for p, x in zip(parents, live)]
        for row in rows:
            for p in row:
                self.ref[p] += 1
        for row in old:
            for p in row:
                self.ref[p] -= 1
        gone = []
        for b, row in enumerate(old):
            for j, p in enumerate(row):
                if self.ref[p] == 0 and p not in gone and not (parents[b] == b and j < live[b]):
                    gone.append(p)
        self.free += gone
        writes = {b: rows[b][k // ps] for b, k in enumerate(kv) if n[b] > 0 and k % ps}
        own = {}
        for b, p in writes.items():
            if self.ref[p] > 1:
                mine = [x for x, q in writes.items() if q == p]
                if not (len(mine) == self.ref[p] and b == min(mine)):
                    own[b] = p
        takes = sum(-(-(k + x) // ps) - y for k, x, y in zip(kv, n, live)) + len(own)
        fits = takes <= len(self.free)
        copies = []
        if fits:
            for b in range(B):
                if b in own:
                    p = self.free.pop()
                    self.ref[p] = 1
                    self.ref[own[b]] -= 1
                    rows[b][kv[b] // ps] = p
                    copies.append((own[b], p, kv[b] % ps))
                while len(rows[b]) < -(-(kv[b] + n[b]) // ps):
                    p = self.free.pop()
                    self.ref[p] = 1
                    rows[b].append(p)
        for b, row in enumerate(rows):
            self.table[b][:len(row)] = row
            for j in range(len(row), self.held[b]):
                self.table[b][j] = -1
            self.held[b], self.kv[b] = len(row), kv[b]
        return fits, copies

    def compact(self):
        """Returns the remap and the moves (source, destination)."""
        N = len(self.ref)
        n = sum(r > 0 for r in self.ref)
        holes = [p for p in range(n) if self.ref[p] <= 0]
        moves = list(zip([p for p in range(n, N) if self.ref[p] > 0], holes))
        remap = [p if self.ref[p] > 0 else -1 for p in range(N)]
        for a, b in moves:
            remap[a] = b
            self.ref[b], self.ref[a] = self.ref[a], 0
        for row, h in zip(self.table, self.held):
            row[:h] = [remap[p] for p in row[:h]]
        self.free = list(range(N - 1, n - 1, -1))
        return remap, moves
