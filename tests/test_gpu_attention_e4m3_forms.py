"""Attention over a cache of e4m3 codes: the forms of the call beside the plain one, with the
weights' rounding as fp16."""
import math
import time

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


def words(mask):
    return mask.long() & 0xffffffff


def random_words(n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-2 ** 31, 2 ** 31 - 1, (n,), generator=g, dtype=torch.int64).int().cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("prefix", [0, 130])
def test_draft_masks(prefix, dtype):
    """Tree drafts: words with holes, words that name later rows, empty words."""
    w = Batch([0, 100, 128, 250, 96], [7, 31, 5, 9, 31], 8, 2, 128, 16, 8, dtype, prefix)
    mask = random_words(w.T, 4)
    mask[1] = 0
    mask[20] = 0
    out, lse = w.run(mask=mask)
    check(w, out, lse, mask=words(mask))
    if prefix == 0:  # no token before, an empty word: nothing is seen
        assert (out[1] == 0).all() and torch.isinf(lse[1]).all() and (lse[1] < 0).all()
    # the causal words give what no mask gives
    pos = torch.cat([torch.arange(x + 1) for x in w.gam])
    causal = ((torch.ones(w.T, dtype=torch.int64) << (pos + 1)) - 1)
    causal = torch.where(causal >= 2 ** 31, causal - 2 ** 32, causal).int().cuda()
    out, lse = w.run(mask=causal)
    check(w, out, lse)
    # words of nothing but what lies behind the step
    mask = torch.full((w.T,), -2 ** 31, dtype=torch.int32, device="cuda")
    out, lse = w.run(mask=mask)
    check(w, out, lse, mask=torch.cat([torch.full((x + 1,), 2 ** 31 if x == 31 else 0) for x in w.gam]).cuda())


@pytest.mark.parametrize("Hq, D, dtype", [(96, 64, "bf16"), (20, 128, "bf16"), (7, 128, "f16"), (1, 16, "bf16")])
def test_draft_masks_over_row_blocks(Hq, D, dtype):
    """Steps of 32 rows in blocks of 1, 4, 7 and all: a word of a first block may name a row of the last."""
    w = Batch([0, 100, 63, 64], [31, 31, 30, 5], Hq, 1, D, 16, 16, dtype)
    mask = random_words(w.T, 8)
    out, lse = w.run(mask=mask)
    check(w, out, lse, mask=words(mask))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("block", [1, 32])
def test_scales_that_are_no_powers_of_two(block, dtype):
    w = Batch([700, 3, 260], [5, 7, 0], 14, 2, 128, 32, block, dtype, 75, powers=False, spread=6)
    out, lse = w.run()
    check(w, out, lse)


@pytest.mark.parametrize("power", [-23, -20, 40, 67])
def test_keys_scales_at_their_ends(power):
    """The keys' scales, 2^-9 to 2^-3 before, and the queries against them."""
    w = Batch([300, 77], [3, 1], 8, 2, 64, 16, 16, "bf16", 40)
    ends = 2.0 ** power
    w.scales[0].mul_(ends)
    for k in (*w.k, w.pk):
        k.mul_(ends)
    w.q.div_(ends)
    s = w.scales[0][~torch.isnan(w.scales[0])]
    assert 2.0 ** -32 <= float(s.min()) and float(s.max()) <= 2.0 ** 64
    out, lse = w.run()
    check(w, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_values_scales_from_end_to_end(dtype):
    """Values' scales of 2^-32 in some requests, 2^64 (fp16: 2^3) in others, and side by side."""
    w = Batch([300, 77, 130], [3, 1, 2], 8, 2, 64, 16, 16, dtype)
    top = 2.0 ** 64 if dtype == "bf16" else 2.0 ** 3
    for b, ends in enumerate([(2.0 ** -32,), (top,), (2.0 ** -32, 1.0, top)]):
        n = w.v[b].shape[0]
        for i in range(-(-n // 16)):
            s, page = ends[i % len(ends)], int(w.cache.page_table[b, i])
            rows = slice(16 * i, min(n, 16 * i + 16))
            w.v[b][rows] *= s / w.scales[1][page, 0].double()[:, None]
            w.scales[1][page, 0] = s
    w.lv = 64.0
    out, lse = w.run()
    # (a row's own largest scale counts for its weights' smallest step)
    for b, most in enumerate([2.0 ** -32, top, top]):
        known = w.scales[1].clone()
        w.scales[1].fill_(most)
        check(w, out, lse, only=[b])
        w.scales[1].copy_(known)


@pytest.mark.parametrize("bad", [math.nan, 0.0, -1.0, math.inf, 2.0 ** -33, 2.0 ** 65])
@pytest.mark.parametrize("kind", [0, 1])
def test_scales_that_are_none_count_as_1(kind, bad):
    w = Batch([300, 77], [3, 1], 4, 2, 64, 16, 16, "bf16", 20)
    page = int(w.cache.page_table[0, 3])
    x = (w.k, w.v)[kind][0]
    x[48:64, 1] /= w.scales[kind][page, 0, 1].double()
    w.scales[kind][page, 0, 1] = bad
    w.q.mul_(0.01)
    out, lse = w.run(status=S["BAD_SCALE"])
    w.scales[kind][page, 0, 1] = 1.0
    check(w, out, lse)


def test_strided_queries_scale_and_large_scores():
    w = Batch([50, 600], [3, 1], 8, 2, 64, 16, 16, "bf16", 0)
    wide = torch.randn((w.T, 14, 64), device="cuda").to(w.dtype)
    w.q = wide[:, 3:11]
    out, lse = w.run(scale=2.0)
    check(w, out, lse, scale=2.0)
    w.q = wide.transpose(0, 1).contiguous().transpose(0, 1)[:, 3:11]  # heads before rows
    out, lse = w.run(scale=2.0)
    check(w, out, lse, scale=2.0)
    w.q = (wide * 20.0)[:, 3:11]  # nearly one-hot weights, scores of hundreds
    out, lse = w.run()
    check(w, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("up", [1.0, -1.0])
def test_rising_and_falling_scores(up, dtype):
    """The keys' scales grow along the sequence: the maximum moves in every tile, or never again."""
    w = Batch([1500, 900], [2, 6], 4, 1, 128, 16, 1, dtype, 700, spread=0)
    w.q.fill_(up)
    c = w.cache
    for k, ids in ((w.pk, w.prefix_table), (w.k[0], c.page_table[0]), (w.k[1], c.page_table[1])):
        t = torch.arange(k.shape[0], device="cuda")
        s = (2.0 ** -6 * (1.0 + t.float() / 40.0))[:, None]
        codes = (k / 2.0 ** -6).abs() * 0.25  # (exact)
        at = ids.long()[t // 16], t % 16
        w.scales[0][at] = s
        w.bytes[0][at] = codes.float().to(torch.float8_e4m3fn).view(torch.uint8)
        k.copy_(values(w.bytes[0][at]) * s.double()[..., None])
    out, lse = w.run()
    check(w, out, lse)


def test_nan_and_infinite_queries_stay_in_their_rows():
    for bad in (math.nan, math.inf, -math.inf):
        w = Batch([60, 200], [2, 1], 4, 2, 64, 16, 16, "f16", 30)
        good, l0 = w.run()
        keep = torch.ones((w.T, 4), dtype=torch.bool, device="cuda")
        keep[1, 2] = False
        w.q[1, 2, 5] = bad
        out, lse = w.run()
        assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2])
        assert torch.equal(out[keep], good[keep]) and torch.equal(lse[keep], l0[keep])


def test_nan_codes_of_seen_and_unseen_tokens():
    # (codes and scales behind the last token are NaN in every test)
    w = Batch([200, 150], [3, 2], 4, 2, 64, 16, 16, "bf16")
    good, l0 = w.run()
    page, at = int(w.cache.page_table[0, 5]), 7
    w.bytes[0][page, at, 1, 3] = 0x7f  # a key of head 1: scores of its query heads are NaN
    out, lse = w.run()
    assert torch.isnan(out[:4, 2:]).all() and torch.isnan(lse[:4, 2:]).all()
    assert torch.equal(out[:4, :2], good[:4, :2]) and torch.equal(out[4:], good[4:])
    w.bytes[0][page, at, 1, 3] = 0
    w.k[0][5 * 16 + 7, 1, 3] = 0.0
    w.bytes[1][page, at, 0, 9] = 0xff  # a value of head 0: that column of the output
    out, lse = w.run()
    assert torch.isnan(out[:4, :2, 9]).all()
    out[:4, :2, 9] = good[:4, :2, 9]
    check(w, out, lse)


def test_bad_requests_and_pages():
    w = Batch([60, 200, 90], [2, 1, 3], 4, 2, 64, 16, 16, "bf16", 0)
    w.cache.kv_len[1] = 10 ** 6
    out, lse = w.run(status=S["BAD_LENGTH"])
    check(w, out, lse, only=[0, 2])
    assert (out[3:5] == 77.0).all() and (lse[3:5] == 77.0).all()
    w = Batch([60, 200, 90], [2, 1, 3], 4, 2, 64, 16, 16, "bf16", 40)
    cu = w.cu.clone()
    w.cu[1] = 50
    out, lse = w.run(status=S["BAD_GAMMA"])
    check(w, out, lse, only=[2])
    assert (out[:5] == 77.0).all()
    w.cu.copy_(cu)
    # a page outside the pool: zeros, with scales of 1
    for bad in (10 ** 6, -1, int(w.bytes[0].shape[0])):
        w.cache.page_table[0, 1] = bad
        w.k[0][16:32] = w.v[0][16:32] = 0.0
        out, lse = w.run(status=S["BAD_PAGE"])
        w.lv = max(w.lv, 1.0)
        check(w, out, lse)


def test_rows_named_again_and_again_are_left_out():
    """Entries 0, n, 0, n, ..: every other request is consistent by itself, together their keys pass
    any list (1000 requests of 313 blocks of 224000 tiles)."""
    B, n, page, width = 2000, 20000, 4096, 7000
    pools = [torch.zeros((1, page, 1, 16), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.ones((1, page // 128, 1), device="cuda") for _ in range(2)]
    kw = dict(k_scales=scales[0], v_scales=scales[1])
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), page * width - n - 1, dtype=torch.int32, device="cuda")
    cache = binding.PagedCache(*pools, table, lens, **kw)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = n
    q = torch.zeros((n + B, 1, 16), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((n + B, 1), 7.0, device="cuda")
    ws = binding.make_attention_e4m3_workspace(n + B, 1, 16)
    binding.spec_verify_attention_e4m3(q, cache, cu, n, out, ws, lse=lse)
    assert binding.spec_verify_status(ws) == S["BAD_GAMMA"]
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())
    # the workspace serves the next call
    few = binding.PagedCache(*pools, table[:1], lens[:1] * 0, **kw)
    one = torch.empty((1, 1, 16), dtype=torch.bfloat16, device="cuda")
    binding.spec_verify_attention_e4m3(q[:1], few, cu[::2][:2].contiguous(), 0, one, ws)
    assert not one.any() and binding.spec_verify_status(ws) == 0


# A part's sum is exact, up to 2^36: its logarithm is off by a step, 2^-18, and by 2^-20 less the maximum.
# The join adds up to 76 parts a warp (2^-25 each), takes a logarithm (2^-20), adds the maximum (2^-20) and
# multiplies by ln 2 (2^-20): ln 2 (2^-18 + 3 2^-20) + 76 2^-25 + 2^-20 < 34 2^-22
LOG_OF_MANY = 34 * 2.0 ** -22


def test_the_longest_request():
    """2^31 - 4097 keys, all in one page: every score 0, every value 0.5.  A CTA's sums of weights (7
    million of 2^13) and of values stay below 2^24 steps: exact."""
    most, page = 2 ** 31 - 4097, 4096
    k = torch.zeros((1, page, 1, 16), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.full((1, page, 1, 16), 0.5, device="cuda").to(torch.float8_e4m3fn)
    s = torch.ones((1, page // 64, 1), device="cuda")
    table = torch.zeros((1, 2 ** 31 // page), dtype=torch.int32, device="cuda")
    lens = torch.tensor([most - 1], dtype=torch.int32, device="cuda")
    cache = binding.PagedCache(k, v, table, lens, k_scales=s, v_scales=s.clone())
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.ones((1, 1, 16), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((1, 1), 7.0, device="cuda")
    ws = binding.make_attention_e4m3_workspace(1, 1, 16)
    binding.spec_verify_attention_e4m3(q, cache, cu, 0, out, ws, lse=lse)
    assert binding.spec_verify_status(ws) == 0
    assert bool((out == 0.5).all())
    assert abs(float(lse) - math.log(most)) < LOG_OF_MANY
    out.fill_(7.0)
    lens.add_(1)  # one more is refused
    binding.spec_verify_attention_e4m3(q, cache, cu, 0, out, ws, lse=lse)
    assert binding.spec_verify_status(ws) == S["BAD_LENGTH"]
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D, group", [(64, 2), (128, 1)])
@pytest.mark.parametrize("sink", [0, 40001, 65535])
@pytest.mark.parametrize("shared", [False, True])
def test_one_large_weight_before_many_small_ones(shared, sink, D, group, dtype):
    """A key 18 above all others: each of the others weighs 2^-26 of it, all together 0.1 percent.
    As fp16 and in steps of 2^-16 beside a largest of 2^13 they are off by 2^-30 of it each."""
    dt, page, L = DT[dtype], 64, 65536
    g = torch.Generator(device="cuda").manual_seed(5)
    shape = (L // page, page, 1, D)
    k = (torch.randn(shape, generator=g, device="cuda") * 25.0).to(torch.float8_e4m3fn)
    v = ((torch.randn(shape, generator=g, device="cuda") + 1.0) * 64.0).clamp(-448, 448).to(torch.float8_e4m3fn)
    ks, vs = torch.full((L // page, page, 1), 2.0 ** -9, device="cuda"), torch.full((L // page, page, 1), 2.0 ** -6, device="cuda")
    k.view(torch.uint8)[..., 0] = 0
    at = sink // page, sink % page
    one = torch.zeros(D, device="cuda")
    one[0] = 144.0
    k.view(torch.uint8)[at[0], at[1], 0] = one.to(torch.float8_e4m3fn).view(torch.uint8)
    ks[at] = 1.0
    v.view(torch.uint8)[at[0], at[1], 0] = torch.full((D,), 16.0, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    B = 160 * (64 // group) if shared else 400
    pages = torch.arange(L // page, dtype=torch.int32, device="cuda")
    kw = dict(k_scales=ks, v_scales=vs)
    if shared:  # a request has one key of its own: the first of the last page
        table = torch.full((B, 1), L // page - 1, dtype=torch.int32, device="cuda")
        cache = binding.PagedCache(k, v, table, torch.zeros(B, dtype=torch.int32, device="cuda"), **kw)
    else:
        cache = binding.PagedCache(k, v, pages.expand(B, -1).contiguous(),
                                   torch.full((B,), L - 1, dtype=torch.int32, device="cuda"), **kw)
    q = torch.zeros((B, group, D), dtype=dt, device="cuda")
    q[..., 0] = 1.0
    q[..., 1] = torch.rand((B, group), generator=g, device="cuda").to(dt)
    out, lse = torch.empty_like(q), torch.empty((B, group), device="cuda")
    ws = binding.make_attention_e4m3_workspace(B, group, D)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    binding.spec_verify_attention(q, cache, cu, 0, out, ws, lse=lse, prefix_table=pages if shared else None,
                                  prefix_len=L if shared else 0, scale=0.125)
    assert binding.spec_verify_status(ws) == 0
    rows = torch.tensor([0, 1, B // 2, B - 1], device="cuda")
    kk = (values(k.view(torch.uint8)) * ks.double()[..., None]).view(L, 1, D)
    vv = (values(v.view(torch.uint8)) * vs.double()[..., None]).view(L, 1, D)
    if shared:
        kk, vv = torch.cat([kk, kk[L - page:L - page + 1]]), torch.cat([vv, vv[L - page:L - page + 1]])
    seen = torch.ones((4, kk.shape[0]), dtype=torch.bool, device="cuda")
    o, l, spread, size = attend(q[rows].double(), kk, vv, seen, 0.125)
    # one scale for all values: the largest weight is the row's, over its sum at most 1
    tol, tl = tight(q[rows].double(), kk, o, l, spread, size, kk.shape[0] * float(vv.abs().max()), 0.125, 6.0, dt)
    err = (out[rows].double() - o).abs()
    assert not (err > tol).any() and not torch.isnan(err).any(), float((err / tol).max())
    assert not ((lse[rows].double() - l).abs() > tl).any()


PROMPTS = {
    # lens, gamma, Hq, Hk, D, page, block, dtype, prefix: row blocks of 64 (fp16: 48) / group tokens each
    "blocks_of_16": ([0, 70], [2499, 3], 4, 1, 64, 64, 64, "bf16", 0),
    "blocks_of_6": ([1000, 3, 0], [1500, 0, 777], 8, 1, 64, 32, 16, "f16", 0),
    "blocks_of_21": ([129, 5], [2600, 900], 3, 1, 64, 64, 32, "bf16", 0),
    "blocks_of_5": ([0, 31, 500], [1234, 1700, 2], 10, 2, 128, 64, 16, "f16", 0),
    "blocks_of_9_and_a_prefix": ([0, 64, 63], [700, 1300, 5], 7, 1, 64, 16, 16, "bf16", 300),
    "blocks_of_less_than_1": ([40, 0], [130, 70], 96, 1, 64, 16, 2, "bf16", 0),
    "blocks_of_48": ([1, 2], [6001, 1], 1, 1, 64, 64, 64, "f16", 0),
    "few_rows_of_a_long_request": ([9000], [40], 8, 1, 64, 64, 64, "f16", 0),  # joined by a CTA a row
    "twelve_blocks_of_a_long_request": ([20011], [90], 8, 1, 128, 16, 16, "bf16", 0),
    "blocks_of_two_requests": ([7000, 12000], [50, 8], 18, 1, 64, 32, 32, "bf16", 100),
}


@pytest.mark.parametrize("name", list(PROMPTS))
def test_prompts_of_many_row_blocks(name):
    lens, gam, Hq, Hk, D, page, block, dt, prefix = PROMPTS[name]
    w = Batch(lens, gam, Hq, Hk, D, page, block, dt, prefix)
    out, lse = w.run()
    check(w, out, lse)
    again, lse2 = w.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_long_lists():
    """160 blocks of requests behind 6.5 million shared tokens, 27648 tokens each: a list of
    10 million tiles.  All keys stand in one page, every score is 0 and every value 0.5; the log
    of the sum of weights counts the keys that the join found."""
    page, B, own, prefix = 4096, 160 * 64, 432 * 64, 51136 * 128
    k = torch.zeros((1, page, 1, 16), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.full((1, page, 1, 16), 0.5, device="cuda").to(torch.float8_e4m3fn)
    s = torch.ones((1, page // 64, 1), device="cuda")
    cache = binding.PagedCache(k, v, torch.zeros((B, -(-own // page)), dtype=torch.int32, device="cuda"),
                               torch.full((B,), own - 1, dtype=torch.int32, device="cuda"), k_scales=s, v_scales=s.clone())
    q = torch.zeros((B, 1, 16), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((B, 1), 7.0, device="cuda")
    ws = binding.make_attention_e4m3_workspace(B, 1, 16)
    binding.spec_verify_attention_e4m3(q, cache, torch.zeros(B + 1, dtype=torch.int32, device="cuda"), 0, out, ws, lse=lse,
                                       prefix_table=torch.zeros(prefix // page, dtype=torch.int32, device="cuda"),
                                       prefix_len=prefix)
    assert binding.spec_verify_status(ws) == 0
    assert bool((out == 0.5).all())
    assert float((lse.double() - math.log(prefix + own)).abs().max()) < LOG_OF_MANY


def test_two_workspaces_two_streams_and_graphs():
    a = Batch([3000, 20, 500], [3, 0, 2], 8, 2, 128, 16, 16, "bf16", 300, seed=2)
    b = Batch([40, 2000], [1, 5], 6, 6, 64, 32, 8, "f16", 0, seed=3)
    ra, rb = a.run(), b.run()
    wa, wb = (binding.make_attention_e4m3_workspace(x.T, x.Hq, x.D) for x in (a, b))
    oa, ob = torch.empty_like(ra[0]), torch.empty_like(rb[0])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.run(ws=wa, out=oa, lse=False, status=None)
        with torch.cuda.stream(s2):
            b.run(ws=wb, out=ob, lse=False, status=None)
    torch.cuda.synchronize()
    assert torch.equal(oa, ra[0]) and torch.equal(ob, rb[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.run(ws=wa, out=oa, lse=False, status=None)
    oa.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, ra[0])
    # the captured call follows the lengths on the device
    a.cache.kv_len.copy_(ints([129, 7, 0]))
    a.lens = [129, 7, 0]
    a.k = [k[:n + x + 1] for k, n, x in zip(a.k, a.lens, a.gam)]
    a.v = [v[:n + x + 1] for v, n, x in zip(a.v, a.lens, a.gam)]
    graph.replay()
    torch.cuda.synchronize()
    check(a, oa, None)


def test_a_dirty_workspace_and_a_larger_one():
    w = Batch([3000, 20], [3, 0], 8, 2, 128, 16, 16, "bf16", 100)
    ref, _ = w.run()
    ws = torch.full((binding.make_attention_e4m3_workspace(w.T + 50, 8, 128).numel(),), 255, dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    out, _ = w.run(ws=ws)
    assert torch.equal(ref, out)


def test_an_empty_batch():
    w = Batch([5], [0], 2, 1, 64, 16, 16, "bf16", 0)
    empty = binding.PagedCache(w.cache.k_pages, w.cache.v_pages, w.cache.page_table[:0], w.cache.kv_len[:0],
                               k_scales=w.scales[0], v_scales=w.scales[1])
    ws = binding.make_attention_e4m3_workspace(1, 2, 64)
    out = torch.full((0, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.spec_verify_attention_e4m3(w.q[:0], empty, w.cu[:1], 0, out, ws)
    assert binding.spec_verify_status(ws) == 0


def test_refused_tensors():
    w = Batch([50, 60], [3, 1], 8, 2, 64, 16, 16, "bf16", 40)
    ws = binding.make_attention_e4m3_workspace(w.T, 8, 64)
    out = torch.empty((w.T, 8, 64), dtype=w.dtype, device="cuda")
    call = binding.spec_verify_attention_e4m3
    for q, o in ((w.q.float(), out), (w.q.half(), out), (w.q, out.half())):
        with pytest.raises((TypeError, ValueError)):
            call(q, w.cache, w.cu, 3, o, ws)
    with pytest.raises(TypeError):
        call(w.q, w.cache, w.cu, 3, out, ws, draft_mask=torch.zeros(w.T, device="cuda"))
    for kw in (dict(prefix_len=40), dict(prefix_table=w.prefix_table[:1], prefix_len=40),
               dict(lse=torch.zeros((w.T, 4), device="cuda")), dict(draft_mask=torch.zeros(3, dtype=torch.int32).cuda())):
        with pytest.raises(ValueError):
            call(w.q, w.cache, w.cu, 3, out, ws, **kw)
    for kw, code in ((dict(scale=0.0), -1), (dict(max_drafts=-1), -1), (dict(workspace=ws[:512]), -4)):
        a = dict(max_drafts=3, workspace=ws)
        a.update({k: v for k, v in kw.items() if k in a})
        with pytest.raises(binding.SpecVerifyError) as e:
            call(w.q, w.cache, w.cu, a["max_drafts"], out, a["workspace"], scale=kw.get("scale"))
        assert e.value.code == code
    with pytest.raises(binding.SpecVerifyError):  # the smaller workspace of the 16-bit call
        call(w.q, w.cache, w.cu, 3, out, ws[:-256])
    with pytest.raises(binding.SpecVerifyError):  # heads of a query read 16 bytes at a time
        call(torch.zeros((w.T, 8, 68), dtype=w.dtype, device="cuda")[..., :64], w.cache, w.cu, 3, out, ws)
    wide = binding.PagedCache(*(torch.zeros((2, 16, 2, 64), dtype=w.dtype, device="cuda") for _ in range(2)),
                              w.cache.page_table, w.cache.kv_len)
    with pytest.raises(TypeError):  # a cache of 16 bits
        call(w.q, wide, w.cu, 3, out, ws)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_the_wait_limit_ends_a_call_with_its_status(dtype):
    """With a limit of 1 ns a wait for a copy from memory runs out: the call ends with the status bit,
    and the next call is right."""
    w = Batch([4000, 300, 9], [3, 0, 2], 8, 2, 128, 16, 16, dtype, 700)
    ref, _ = w.run()
    ws = binding.make_attention_e4m3_workspace(w.T, w.Hq, w.D)
    for _ in range(3):
        prev = binding.spec_verify_set_wait_limit(1)
        try:
            t0 = time.perf_counter()
            w.run(ws=ws, status=None)
            bits = binding.spec_verify_status(ws)
            assert time.perf_counter() - t0 < 20.0
        finally:
            binding.spec_verify_set_wait_limit(prev)
        assert binding.status_names(bits) == ["TIMEOUT"]
        out, _ = w.run(ws=ws)
        assert torch.equal(out, ref)
