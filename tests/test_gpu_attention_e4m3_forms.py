"""Attention over a cache of e4m3 codes: the forms of the call beside the plain one, with the
weights' rounding as fp16."""
import math

import pytest
import torch

from cache8_refs import values
from operator_refs import attend
from speculative_decoding_verification_62_gb300 import binding
import test_gpu_attention_e4m3
from test_gpu_attention_e4m3 import DT, S, Batch, ints, tolerance

pytestmark = pytest.mark.gpu


def tight(q, k, o, lse, spread, size, weight, scale, lv, dtype):
    """tolerance() with a weight off by 2^-11 of itself, as fp16 rounds it: the sum of its three
    8-bit floats is that fp16 (the first two are rounded to the nearest, so that what is left
    after them has three bits)."""
    tol, tl = tolerance(q, k, o, lse, spread, size, weight, scale, lv, dtype)
    return tol - (2.0 ** -9 * 1.13 - 2.0 ** -11) * 1.01 * spread, tl


def check(w, out, lse, mask=None, scale=None, only=None):
    """Batch.check with tight()."""
    with pytest.MonkeyPatch.context() as m:
        m.setattr(test_gpu_attention_e4m3, "tolerance", tight)
        return w.check(out, lse, mask, scale, only)


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_weights_are_good_to_fp16(seed):
    """Two keys, the first with values of 0: an output is the second's weight over the sum."""
    w = Batch([1] * 64, [0] * 64, 8, 1, 16, 16, 1, "f16", seed=seed)
    for b in range(64):
        w.bytes[1][w.cache.page_table[b, 0].long(), 0] = 0
        w.v[b][0] = 0.0
    out, lse = w.run()
    scale = w.D ** -0.5
    most = 0.0
    for b in range(64):
        q = w.q[b:b + 1].double()
        seen = torch.ones((1, 2), dtype=torch.bool, device="cuda")
        o, l, spread, size = attend(q, w.k[b], w.v[b], seen, scale)
        weight = 2 * 448.0 * float(w.scales[1][~torch.isnan(w.scales[1])].max())
        tol, _ = tight(q, w.k[b], o, l, spread, size, weight, scale, w.lv, w.dtype)
        most = max(most, float(((out[b:b + 1].double() - o).abs() / tol).max()))
    assert most <= 1.0, most


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale, total", [(1974.0, 47129), (2321.0, 40083), (1917.0, 51067), (-1.0, 0)])
def test_scores_far_from_zero(scale, total, dtype):
    """One key whose score is below 2^27, with values scaled by 2^8.  The logarithm of its weight
    is rounded to a multiple of 8 or 16, and with its values' scale again.  A maximum that came out too small
    leaves a weight of 2^19 (1974, 47129), which is none in fp16; one that came out too large leaves one near
    2^-16, which has no bits in e5m2."""
    if total == 0:  # random keys of scores of that size, several rows and tiles
        w = Batch([300, 77], [3, 1], 4, 2, 64, 16, 16, dtype, spread=0, seed=8)
        scale = 2.0 ** 26 / float(max((w.q.double().abs().amax() * k.abs().sum(-1)).max() for k in w.k))
    else:
        w = Batch([0], [0], 1, 1, 128, 16, 1, dtype, seed=3)
        p = int(w.cache.page_table[0, 0])
        codes = torch.zeros(128)
        steps, rest = values(torch.arange(0x7f, dtype=torch.uint8)), total
        for d in range(128):  # the largest code that fits, each time
            codes[d] = steps[steps <= rest].max()
            rest -= int(codes[d])
        codes = codes.to(torch.float8_e4m3fn).cuda()
        assert float(codes.double().sum()) == total
        w.bytes[0][p, 0, 0] = codes.view(torch.uint8)
        w.scales[0][p, 0, 0], was = 1.0, float(w.scales[1][p, 0, 0])
        w.scales[1][p, 0, 0] = 2.0 ** 8
        w.k[0][0, 0], w.v[0] = codes.double(), w.v[0] * (2.0 ** 8 / was)
        w.q.fill_(1.0)
    out, lse = w.run(scale=scale)
    row = 0
    for b, (n, x) in enumerate(zip(w.lens, w.gam)):
        rows = slice(row, row + x + 1)
        row += x + 1
        seen = torch.arange(n + x + 1, device="cuda")[None, :] <= n + torch.arange(x + 1, device="cuda")[:, None]
        o, l, spread, size = attend(w.q[rows].double(), w.k[b], w.v[b], seen, scale)
        assert torch.isfinite(out[rows]).all() and float(l.max()) < 2.0 ** 27
        # the logarithm of the sum is rounded as the score is
        assert not ((lse[rows].double() - l).abs() > 2.0 ** -21 * l.abs()).any()
        # Where one score stands out by more than all scores' own rounding ((3 D + 3) 2^-24 of the
        # magnitudes, twice, and 45 for weights of 2^-64), that key's value is the output: its weight is off by
        # 2^-11, and by 2^-14 of itself as the largest.
        k = w.k[b].repeat_interleave(w.Hq // w.Hk, 1)
        s = torch.einsum("thd,lhd->thl", w.q[rows].double(), k) * scale
        s = torch.where(seen[:, None], s, -math.inf).sort(-1)[0]
        gap = s[..., -1] - s[..., -2] if n + x > 0 else torch.full_like(s[..., 0], math.inf)
        alone = gap > 2 * (3 * w.D + 3) * 2.0 ** -24 * size + 45
        assert float(alone.double().mean()) > 0.5
        u = torch.finfo(w.dtype).eps / 2
        err = (out[rows].double() - o).abs()
        assert not ((err > (u + 2.0 ** -11 + 2.0 ** -14) * 1.01 * o.abs() + 2.0 ** -25) & alone[..., None]).any()


@pytest.mark.parametrize("power, scale_power", [(115, -116), (122, -122), (100, -102), (-90, 92), (-93, 95)])
def test_queries_of_any_size(power, scale_power):
    """bf16 queries of 2^power whose scores are ordinary by the scale."""
    w = Batch([300, 77, 5], [3, 1, 0], 4, 2, 64, 16, 16, "bf16", seed=9)
    w.q.mul_(2.0 ** power)
    out, lse = w.run(scale=2.0 ** scale_power)
    check(w, out, lse, scale=2.0 ** scale_power)


def test_keys_of_zeros_under_huge_queries():
    """Whatever the queries and the scale, keys of zeros score 0: the values' mean."""
    w = Batch([40], [0], 2, 1, 64, 16, 16, "bf16", spread=0)
    w.bytes[0].zero_()
    w.k[0].zero_()
    w.q.fill_(2.0 ** 127)
    out, lse = w.run(scale=2.0 ** 20)
    check(w, out, lse, scale=2.0 ** 20)
