"""Attention over the paged cache against the definition in 64 bits, within the error
that its roundings allow; everything in the pools that no row sees holds NaN."""
import math

import pytest
import torch

from operator_refs import attend, tolerance
from speculative_decoding_verification_62_gb300 import binding

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


class Batch:
    def __init__(self, lens, gam, Hq, Hk, D, page, dtype, prefix=0, layout="nhd", seed=1, scale_q=1.5,
                 spare=2, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        gc = torch.Generator().manual_seed(seed)
        self.lens, self.gam, self.Hq, self.Hk, self.D, self.page, self.prefix = lens, gam, Hq, Hk, D, page, prefix
        self.dtype = DT[dtype]
        B = len(lens)
        need = [-(-(n + x + 1) // page) for n, x in zip(lens, gam)]
        pre = -(-prefix // page)
        total = sum(need) + pre + spare
        perm = torch.randperm(total, generator=gc).int()
        table = torch.full((B, max(need) + 1), -9, dtype=torch.int32)
        shape = (total, page, Hk, D) if layout == "nhd" else (total, Hk, page, D)
        kp = torch.full(shape, math.nan, dtype=self.dtype, device=device)
        vp = torch.full(shape, math.nan, dtype=self.dtype, device=device)
        if layout == "hnd":
            kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
        at = pre
        self.k, self.v = [], []

        def fill(ids, n):
            k = torch.randn((n, Hk, D), generator=g, device=device).to(self.dtype)
            v = (torch.randn((n, Hk, D), generator=g, device=device) + 0.25).to(self.dtype)
            t = torch.arange(n, device=device)
            kp[ids.long().to(device)[t // page], t % page] = k
            vp[ids.long().to(device)[t // page], t % page] = v
            return k.double(), v.double()
        self.prefix_table = perm[:pre].to(device)
        self.pk, self.pv = fill(perm[:pre], prefix) if prefix else (None, None)
        for b in range(B):
            ids = perm[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = ids
            k, v = fill(ids, lens[b] + gam[b] + 1)
            self.k.append(k)
            self.v.append(v)
        self.T = sum(gam) + B
        self.q = (torch.randn((self.T, Hq, D), generator=g, device=device) * scale_q).to(self.dtype)
        self.cu = torch.tensor([0] + torch.tensor(gam).cumsum(0).tolist(), dtype=torch.int32, device=device)
        self.cache = binding.PagedCache(kp, vp, table.to(device), torch.tensor(lens, dtype=torch.int32, device=device))

    def run(self, mask=None, lse=True, scale=None, ws=None, out=None, q=None, status=0):
        if ws is None:
            ws = binding.make_attention_workspace(self.T, self.Hq, self.D)
        if out is None:
            out = torch.full((self.T, self.Hq, self.D), 77.0, dtype=self.dtype, device="cuda")
        l = torch.full((self.T, self.Hq), 77.0, device="cuda") if lse else None
        binding.spec_verify_attention(self.q if q is None else q, self.cache, self.cu, max(self.gam), out, ws,
                                      prefix_table=self.prefix_table, prefix_len=self.prefix, scale=scale,
                                      draft_mask=mask, lse=l)
        if status is not None:
            assert binding.spec_verify_status(ws) == status
        return out, l

    def check(self, out, lse, mask=None, scale=None, only=None):
        scale = self.D ** -0.5 if scale is None else scale
        row = 0
        worst = 0.0
        for b, (n, x) in enumerate(zip(self.lens, self.gam)):
            rows = slice(row, row + x + 1)
            row += x + 1
            if only is not None and b not in only:
                continue
            k, v = self.k[b], self.v[b]
            i, j = torch.arange(x + 1, device="cuda")[:, None], torch.arange(n + x + 1, device="cuda")[None, :]
            if mask is None:
                seen = j <= n + i
            else:
                word = mask[rows].long()[:, None]
                seen = (j < n) | (((word >> (j - n).clamp_min(0)) & 1) == 1)
            if self.prefix:
                k, v = torch.cat([self.pk, k]), torch.cat([self.pv, v])
                seen = torch.cat([torch.ones((x + 1, self.prefix), dtype=torch.bool, device="cuda"), seen], 1)
            o, l, spread, size = attend(self.q[rows].double(), k, v, seen, scale)
            tol, tl = tolerance(o, l, spread, size, k.shape[0], self.D, float(v.abs().max()), self.dtype)
            err = (out[rows].double() - o).abs()
            assert not (err > tol).any() and not torch.isnan(err).any(), (
                b, int((~(err <= tol)).sum()), float((err / tol).max()))
            worst = max(worst, float((err / tol).max()))
            if lse is not None:
                g = lse[rows].double()
                empty = torch.isinf(l)
                assert torch.equal(g[empty], l[empty])
                assert not ((g - l).abs()[~empty] > tl[~empty]).any()
        return worst


CASES = {
    # lens, gamma, Hq, Hk, D, page, dtype, prefix, layout
    "one_token": ([0], [0], 1, 1, 64, 16, "bf16", 0, "nhd"),
    "one_tile": ([100], [3], 8, 2, 128, 16, "bf16", 0, "nhd"),
    "tile_borders": ([127, 128, 124, 255, 0, 1], [0, 0, 3, 1, 5, 7], 4, 1, 128, 32, "bf16", 0, "nhd"),
    "mha_f16": ([30, 500, 77], [2, 0, 4], 6, 6, 64, 16, "f16", 0, "hnd"),
    "odd_dim_80": ([300, 11], [4, 1], 10, 2, 80, 64, "f16", 0, "nhd"),
    "dim_8": ([300, 11], [4, 1], 4, 2, 8, 64, "bf16", 0, "nhd"),
    "dim_40_group_3": ([130, 400], [6, 2], 9, 3, 40, 32, "bf16", 0, "hnd"),
    "group_7": ([700, 3, 260], [5, 7, 0], 14, 2, 128, 128, "bf16", 0, "nhd"),
    "group_128": ([200, 40], [1, 3], 128, 1, 64, 16, "bf16", 0, "nhd"),
    "group_96": ([200, 40], [1, 3], 96, 1, 128, 16, "f16", 0, "nhd"),
    "big_pages": ([1000, 20, 300], [3, 3, 3], 8, 2, 128, 512, "bf16", 0, "hnd"),
    "split_long": ([20000], [3], 8, 1, 128, 64, "bf16", 0, "nhd"),
    "split_long_f16_64": ([9001, 17], [7, 2], 16, 2, 64, 16, "f16", 0, "nhd"),
    "many": ([(37 * b) % 400 for b in range(330)], [b % 4 for b in range(330)], 4, 2, 64, 16, "bf16", 0, "nhd"),
    "more_requests_than_threads": ([(53 * b) % 300 for b in range(900)], [b % 3 for b in range(900)], 2, 1, 64, 32,
                                   "f16", 0, "nhd"),
    "more_requests_and_a_prefix": ([(53 * b) % 90 for b in range(401)], [b % 5 for b in range(401)], 8, 2, 128, 16,
                                   "bf16", 200, "nhd"),
    "long_among_short": ([30, 9000, 5, 0, 77], [1, 2, 0, 3, 4], 4, 4, 128, 64, "f16", 0, "nhd"),
    "prompt": ([0, 64], [399, 150], 4, 2, 128, 16, "bf16", 0, "nhd"),
    "prompt_group_3": ([5], [600], 3, 1, 64, 32, "f16", 0, "nhd"),
    "prefix_1": ([40, 0, 9], [2, 3, 0], 8, 2, 128, 16, "bf16", 1, "nhd"),
    "prefix_small_batch": ([40, 0, 9], [2, 3, 0], 8, 2, 128, 16, "bf16", 300, "nhd"),
    "prefix_two_blocks": ([b * 9 for b in range(40)], [b % 6 for b in range(40)], 8, 1, 128, 16, "bf16", 1000, "hnd"),
    "prefix_three_blocks_f16": ([b * 3 for b in range(70)], [3] * 70, 4, 2, 64, 32, "f16", 2051, "nhd"),
    "prefix_many_heads": ([b * 30 for b in range(30)], [4] * 30, 32, 8, 128, 64, "bf16", 4096, "nhd"),
    "prefix_group_5": ([b * 30 for b in range(30)], [b % 5 for b in range(30)], 20, 4, 96, 128, "bf16", 1500, "nhd"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_definition(name):
    lens, gam, Hq, Hk, D, page, dt, prefix, layout = CASES[name]
    w = Batch(lens, gam, Hq, Hk, D, page, dt, prefix, layout)
    out, lse = w.run()
    worst = w.check(out, lse)
    print(name, "worst error over tolerance", worst)
    again, lse2 = w.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # bit for bit


@pytest.mark.parametrize("prefix", [0, 130])
def test_draft_masks(prefix):
    """Tree drafts: words with holes, words that name later rows, empty words."""
    w = Batch([0, 100, 128, 250], [7, 31, 5, 9], 8, 2, 128, 16, "bf16", prefix)
    g = torch.Generator().manual_seed(4)
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (w.T,), generator=g, dtype=torch.int64).int().cuda()
    mask[1] = 0
    mask[20] = 0
    words = mask.long() & 0xffffffff
    out, lse = w.run(mask=mask)
    w.check(out, lse, mask=words)
    if prefix == 0:  # no token before, an empty word: nothing is seen
        assert (out[1] == 0).all() and torch.isinf(lse[1]).all() and (lse[1] < 0).all()
    # the causal words give what no mask gives
    pos = torch.cat([torch.arange(x + 1) for x in w.gam])
    causal = ((torch.ones(w.T, dtype=torch.int64) << (pos + 1)) - 1)
    causal = torch.where(causal >= 2 ** 31, causal - 2 ** 32, causal).int().cuda()
    a, la = w.run(mask=causal)
    b, lb = w.run()
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_strided_queries_scale_and_large_scores():
    w = Batch([50, 600], [3, 1], 8, 2, 64, 16, "bf16", 0)
    wide = torch.randn((w.T, 14, 64), device="cuda").to(w.dtype)
    q = wide[:, 3:11]
    w.q = q
    out, lse = w.run(scale=2.0)
    w.check(out, lse, scale=2.0)
    w.q = q * 20.0  # nearly one-hot weights, scores of hundreds
    out, lse = w.run()
    w.check(out, lse)


def test_rising_scores_move_the_maximum():
    """Keys whose scores grow along the sequence: the running maximum moves in every tile."""
    w = Batch([1500, 900], [2, 6], 4, 1, 128, 16, "bf16", 700, scale_q=1.0)
    page, c = w.page, w.cache
    up = torch.ones(128, device="cuda")
    w.q = (up * 1.0).expand(w.T, 4, 128).contiguous().to(w.dtype)

    def raise_(k, ids):
        t = torch.arange(k.shape[0], device="cuda")
        k += (t.double() / 40.0)[:, None, None]
        k.copy_(k.to(w.dtype).double())
        c.k_pages[ids.long()[t // page], t % page] = k.to(w.dtype)
    raise_(w.pk, w.prefix_table)
    for b in range(2):
        raise_(w.k[b], c.page_table[b])
    out, lse = w.run()
    w.check(out, lse)


def test_infinite_scores_and_nan_stay_in_their_rows():
    w = Batch([60, 200], [2, 1], 4, 2, 64, 16, "f16", 0)
    w.q[1, 2] = math.nan
    out, lse = w.run()
    assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2])
    keep = torch.ones((w.T, 4), dtype=torch.bool)
    keep[1, 2] = False
    assert not torch.isnan(out[keep.cuda()]).any()
    w.q[1, 2] = 0.0
    out, lse = w.run()
    w.check(out, lse)
    # a key of -inf times a positive query: weight 0
    w = Batch([60], [2], 1, 1, 64, 16, "bf16", 0)
    w.q.abs_()
    ids = w.cache.page_table[0].long()
    w.cache.k_pages[ids[0], 5] = -math.inf
    w.k[0][5] = -1e30
    out, lse = w.run()
    w.k[0][5] = -1e3
    w.check(out, lse)


def test_bad_requests_are_left_out():
    S = {n: b for b, n in binding.STATUS_BITS.items()}
    w = Batch([60, 200, 90], [2, 1, 3], 4, 2, 64, 16, "bf16", 0)
    w.cache.kv_len[1] = 10 ** 6
    out, lse = w.run(status=S["BAD_LENGTH"])
    w.check(out, lse, only=[0, 2])
    assert (out[3:5] == 77.0).all() and (lse[3:5] == 77.0).all()
    w = Batch([60, 200, 90], [2, 1, 3], 4, 2, 64, 16, "bf16", 40)
    cu = w.cu.clone()
    w.cu[1] = 50
    out, lse = w.run(status=S["BAD_GAMMA"])
    w.check(out, lse, only=[2])
    assert (out[:5] == 77.0).all()
    w.cu.copy_(cu)
    w.cache.page_table[0, 1] = 10 ** 6
    out, lse = w.run(status=S["BAD_PAGE"])
    w.check(out, lse, only=[1, 2])


def test_rows_named_again_and_again_are_left_out():
    # entries 0, n, 0, n, ..: every other request is consistent by itself, together their
    # keys pass any list (1000 requests of 157 blocks of half a million tiles)
    B, n, page, width = 2000, 20000, 4096, 7000
    pools = [torch.zeros((1, page, 1, 8), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.zeros((B, width), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), page * width - n - 1, dtype=torch.int32, device="cuda")
    cache = binding.PagedCache(*pools, table, lens)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = n
    q = torch.zeros((n + B, 1, 8), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((n + B, 1), 7.0, device="cuda")
    ws = binding.make_attention_workspace(n + B, 1, 8)
    binding.spec_verify_attention(q, cache, cu, n, out, ws, lse=lse)
    assert binding.spec_verify_status(ws) == 1
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())
    # the workspace serves the next call
    few = binding.PagedCache(*pools, table[:1], lens[:1] * 0)
    one = torch.empty((1, 1, 8), dtype=torch.bfloat16, device="cuda")
    binding.spec_verify_attention(q[:1], few, cu[::2][:2].contiguous(), 0, one, ws)
    assert not one.any()


def test_the_longest_request():
    # 2^31 - 4097 keys, all in one page: every score 0, every value 0.5.  A stream's sum of
    # weights (7 million) and of values stays below 2^24 half units: exact.
    most, page = 2 ** 31 - 4097, 4096
    k = torch.zeros((1, page, 1, 8), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 0.5)
    table = torch.zeros((1, 2 ** 31 // page), dtype=torch.int32, device="cuda")
    lens = torch.tensor([most - 1], dtype=torch.int32, device="cuda")
    cache = binding.PagedCache(k, v, table, lens)
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.ones((1, 1, 8), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((1, 1), 7.0, device="cuda")
    ws = binding.make_attention_workspace(1, 1, 8)
    binding.spec_verify_attention(q, cache, cu, 0, out, ws, lse=lse)
    assert binding.spec_verify_status(ws) == 0
    assert bool((out == 0.5).all())
    assert abs(float(lse) - math.log(most)) < 22 * 2.0 ** -22  # the join's and logarithm's roundings
    out.fill_(7.0)
    lens.add_(1)  # one more is refused
    binding.spec_verify_attention(q, cache, cu, 0, out, ws, lse=lse)
    assert binding.spec_verify_status(ws) == 512
    assert bool((out == 7.0).all())


def test_two_workspaces_two_streams_and_graphs():
    a = Batch([3000, 20, 500], [3, 0, 2], 8, 2, 128, 16, "bf16", 300, seed=2)
    b = Batch([40, 2000], [1, 5], 6, 6, 64, 32, "f16", 0, seed=3)
    ra, rb = a.run(), b.run()
    wa, wb = (binding.make_attention_workspace(x.T, x.Hq, x.D) for x in (a, b))
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
    a.cache.kv_len.copy_(torch.tensor([129, 7, 0]))
    a.lens = [129, 7, 0]
    a.k = [k[:n + x + 1] for k, n, x in zip(a.k, a.lens, a.gam)]
    a.v = [v[:n + x + 1] for v, n, x in zip(a.v, a.lens, a.gam)]
    graph.replay()
    torch.cuda.synchronize()
    a.check(oa, None)


def test_a_dirty_workspace_and_a_larger_one():
    w = Batch([3000, 20], [3, 0], 8, 2, 128, 16, "bf16", 100)
    ref, _ = w.run()
    ws = torch.full((binding.make_attention_workspace(w.T + 50, 8, 128).numel(),), 255, dtype=torch.uint8, device="cuda")
    ws[:4] = 0
    out, _ = w.run(ws=ws)
    assert torch.equal(ref, out)


def test_an_empty_batch_and_no_prefix_pages():
    w = Batch([5], [0], 2, 1, 64, 16, "bf16", 0)
    empty = binding.PagedCache(w.cache.k_pages, w.cache.v_pages, w.cache.page_table[:0],
                               w.cache.kv_len[:0])
    ws = binding.make_attention_workspace(1, 2, 64)
    out = torch.full((0, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.spec_verify_attention(w.q[:0], empty, w.cu[:1], 0, out, ws)
    assert binding.spec_verify_status(ws) == 0


def test_refused_tensors():
    w = Batch([50, 60], [3, 1], 8, 2, 64, 16, "bf16", 40)
    ws = binding.make_attention_workspace(w.T, 8, 64)
    out = torch.empty((w.T, 8, 64), dtype=w.dtype, device="cuda")
    call = binding.spec_verify_attention
    with pytest.raises(TypeError):
        call(w.q.half(), w.cache, w.cu, 3, out, ws)
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
    with pytest.raises(binding.SpecVerifyError):  # heads of a query read 16 bytes at a time
        call(torch.zeros((w.T, 8, 68), dtype=w.dtype, device="cuda")[..., :64], w.cache, w.cu, 3, out, ws)


def test_a_wait_that_runs_out_ends_the_call():
    """With a limit of 1 ns a wait for a copy runs out: the call returns with the status
    bit (or, where every copy was already there, complete), nothing hangs, and the next
    call is right."""
    import time
    w = Batch([4000, 300, 9], [3, 0, 2], 8, 2, 128, 16, "bf16", 700)
    ref, _ = w.run()
    ws = binding.make_attention_workspace(w.T, w.Hq, w.D)
    prev = binding.spec_verify_set_wait_limit(1)
    try:
        t0 = time.perf_counter()
        w.run(ws=ws, status=None)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 20.0
        bits = binding.spec_verify_status(ws)
        assert set(binding.status_names(bits)) <= {"TIMEOUT"}
        print("status", binding.status_names(bits))
    finally:
        binding.spec_verify_set_wait_limit(prev)
    out, _ = w.run(ws=ws)
    assert torch.equal(out, ref)


def test_the_wait_limit_ends_a_call_with_its_status():
    """With a limit of 1 ns the first wait for a copy from memory runs out in every CTA:
    the call ends with the status bit, and the next call is right."""
    import time
    w = Batch([4000, 300, 9], [3, 0, 2], 8, 2, 128, 16, "bf16", 700)
    ref, _ = w.run()
    ws = binding.make_attention_workspace(w.T, w.Hq, w.D)
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


def sink_tolerance(o, lse, spread, size, keys, D, vmax, dtype):
    """tolerance() without its term for narrow fp16 weights, and that term as the kernel's
    shift leaves it: the largest weight of a part is 2^7 at least, so a weight below the
    normal numbers, off by 2^-25, is off by 2^-32 of it."""
    _, tl = tolerance(o, lse, spread, size, keys, D, vmax, dtype)
    u, d = torch.finfo(dtype).eps / 2, tl - 2.0 ** -22 * (1.0 + lse.abs())
    tol = (u + 2 * d[..., None]) * 1.01 * spread + u * 1.01 * o.abs() + 1e-30
    if dtype == torch.float16:
        tol = tol + keys * 2.0 ** -32 * vmax + 2.0 ** -25
    return tol, tl


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D, group", [(64, 2), (128, 1)])
@pytest.mark.parametrize("sink", [0, 40001, 65535])
@pytest.mark.parametrize("shared", [False, True])
def test_one_large_weight_before_many_small_ones(shared, sink, D, group, dtype):
    """A key 17.5 above all others: each of the others weighs 2^-25 of it, all together 0.16
    percent.  So many units that every one lies in one or two shares: 400 requests that
    read the same pages, or 160 pairs of row blocks over a prefix."""
    dt, page, L = DT[dtype], 64, 65536
    g = torch.Generator(device="cuda").manual_seed(5)
    k = (torch.randn((L // page, page, 1, D), generator=g, device="cuda") * 0.05).to(dt)
    v = (torch.randn((L // page, page, 1, D), generator=g, device="cuda") + 1.0).to(dt)
    k[..., 0] = 0.0
    at = sink // page, sink % page
    k[at], v[at] = 0.0, 0.25
    k[at][0, 0] = 17.5 * D ** 0.5
    B = 160 * 2 * (128 // group) if shared else 400
    pages = torch.arange(L // page, dtype=torch.int32, device="cuda")
    if shared:  # a request has one key of its own: the first of the last page
        table = torch.full((B, 1), L // page - 1, dtype=torch.int32, device="cuda")
        cache = binding.PagedCache(k, v, table, torch.zeros(B, dtype=torch.int32, device="cuda"))
    else:
        cache = binding.PagedCache(k, v, pages.expand(B, -1).contiguous(),
                                   torch.full((B,), L - 1, dtype=torch.int32, device="cuda"))
    q = torch.zeros((B, group, D), dtype=dt, device="cuda")
    q[..., 0] = 1.0
    q[..., 1] = torch.rand((B, group), generator=g, device="cuda").to(dt)
    out, lse = torch.empty_like(q), torch.empty((B, group), device="cuda")
    ws = binding.make_attention_workspace(B, group, D)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    binding.spec_verify_attention(q, cache, cu, 0, out, ws, lse=lse, prefix_table=pages if shared else None,
                                  prefix_len=L if shared else 0)
    assert binding.spec_verify_status(ws) == 0
    rows = torch.tensor([0, 1, B // 2, B - 1], device="cuda")
    kk, vv = k.double().view(L, 1, D), v.double().view(L, 1, D)
    if shared:
        kk, vv = torch.cat([kk, kk[L - page:L - page + 1]]), torch.cat([vv, vv[L - page:L - page + 1]])
    seen = torch.ones((4, kk.shape[0]), dtype=torch.bool, device="cuda")
    o, l, spread, size = attend(q[rows].double(), kk, vv, seen, D ** -0.5)
    tol, tl = sink_tolerance(o, l, spread, size, kk.shape[0], D, float(vv.abs().max()), dt)
    err = (out[rows].double() - o).abs()
    assert not (err > tol).any() and not torch.isnan(err).any(), float((err / tol).max())
    assert not ((lse[rows].double() - l).abs() > tl).any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("power", [16, 20, 24, 27])
def test_scores_whose_own_rounding_is_large(power, dtype):
    """Scores up to 2^power, rising along the keys in steps of 2^(power - 9) for three keys
    each, whose scores differ by 0 or 1.  2^27 is what the call allows: the running maximum
    (times log2 e, below 2^28) then has steps of 16 at most, and rounded up by less than one
    step it leaves the largest weight, 2^7 less that, above 2^-9 and off by 2^-16 of itself at
    most; with steps of 32 it would be lost in fp16.  The products are exact in 24 bits and the scale a power of two, so that the
    weights of the keys around the largest score are good to their rounding all the same."""
    w = Batch([1000, 700], [2, 1], 4, 2, 64, 16, dtype, 0, seed=power)
    g = torch.Generator(device="cuda").manual_seed(power)
    scale = 2.0 ** (power - 16)
    for b in range(2):
        n = w.k[b].shape[0]
        t = torch.arange(n, device="cuda")
        w.k[b].zero_()
        w.k[b][:, :, 0] = 128.0 + (t // 3 % 64)[:, None]
        w.k[b][:, :, 1] = 8.0 * (t // 192)[:, None]
        if power <= 24:  # a 2^-8 is the last bit of the products
            w.k[b][:, :, 2] = torch.randint(0, 2, (n, 2), generator=g, device="cuda").double() / scale
        w.cache.k_pages[w.cache.page_table[b].long()[t // 16], t % 16] = w.k[b].to(w.dtype)
    w.q.zero_()
    w.q[:, :, 0], w.q[:, :, 1], w.q[:, :, 2] = 128.0, 1024.0, 1.0
    out, lse = w.run(scale=scale)
    u, row = torch.finfo(w.dtype).eps / 2, 0
    for b, (n, x) in enumerate(zip(w.lens, w.gam)):
        rows = slice(row, row + x + 1)
        row += x + 1
        seen = torch.arange(n + x + 1, device="cuda")[None, :] <= n + torch.arange(x + 1, device="cuda")[:, None]
        o, l, spread, _ = attend(w.q[rows].double(), w.k[b], w.v[b], seen, scale)
        assert 2.0 ** (power - 1) < float(l.min()) and float(l.max()) < 2.0 ** power
        # scores that differ by 1 are off by 2^-22 of that, weights by 2^-17 as in
        # tolerance(); what lies a step of 128 scale or more below has no weight
        tol = (u + 2.0 ** -16 + (2.0 ** -15 if dtype == "f16" and power == 27 else 0)) * 1.01 * spread
        tol = tol + u * 1.01 * o.abs() + 2.0 ** -25
        assert not ((out[rows].double() - o).abs() > tol).any() and torch.isfinite(out[rows]).all()
        assert not ((lse[rows].double() - l).abs() > 2.0 ** -21 * l.abs()).any()


def test_long_lists_at_a_border_of_their_shares():
    """380 blocks of requests behind 6.5 million shared tokens, 27648 tokens each: lists of
    9.7 and 21.1 million tiles, whose share of the CTAs lies within a rounding of 32 bits of
    98.5 of 152.  All keys stand in one page, every score is 0 and every value 0.5; the log
    of the sum of weights counts the keys that the join found."""
    page, B, own, prefix = 4096, 380 * 128, 432 * 64, 51136 * 128
    k = torch.zeros((1, page, 1, 8), dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, 0.5)
    cache = binding.PagedCache(k, v, torch.zeros((B, -(-own // page)), dtype=torch.int32, device="cuda"),
                               torch.full((B,), own - 1, dtype=torch.int32, device="cuda"))
    q = torch.zeros((B, 1, 8), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((B, 1), 7.0, device="cuda")
    ws = binding.make_attention_workspace(B, 1, 8)
    binding.spec_verify_attention(q, cache, torch.zeros(B + 1, dtype=torch.int32, device="cuda"), 0, out, ws, lse=lse,
                                  prefix_table=torch.zeros(prefix // page, dtype=torch.int32, device="cuda"),
                                  prefix_len=prefix)
    assert binding.spec_verify_status(ws) == 0
    assert bool((out == 0.5).all())
    assert float((lse.double() - math.log(prefix + own)).abs().max()) < 20 * 2.0 ** -22


PROMPTS = {
    # lens, gamma, Hq, Hk, D, page, dtype, prefix: row blocks of 128 / group tokens each
    "blocks_of_32": ([0, 70], [2499, 3], 4, 1, 64, 64, "bf16", 0),
    "blocks_of_16": ([1000, 3, 0], [1500, 0, 777], 8, 1, 64, 32, "f16", 0),
    "blocks_of_42": ([129, 5], [2600, 900], 3, 1, 64, 64, "bf16", 0),
    "blocks_of_25": ([0, 31, 500], [1234, 1700, 2], 10, 2, 128, 64, "f16", 0),
    "blocks_of_18_and_a_prefix": ([0, 64, 63], [700, 1300, 5], 7, 1, 64, 16, "bf16", 300),
    "blocks_of_1": ([40, 0], [130, 70], 96, 1, 64, 16, "bf16", 0),
    "blocks_of_128": ([1, 2], [6001, 1], 1, 1, 64, 64, "f16", 0),
    "few_rows_of_a_long_request": ([9000], [40], 8, 1, 64, 64, "f16", 0),  # joined by a CTA a row
    "six_blocks_of_a_long_request": ([20011], [90], 8, 1, 128, 16, "bf16", 0),
    "nine_blocks_of_two_requests": ([7000, 12000], [50, 8], 18, 1, 64, 32, "bf16", 100),
}


@pytest.mark.parametrize("name", list(PROMPTS))
def test_prompts_of_many_row_blocks(name):
    lens, gam, Hq, Hk, D, page, dt, prefix = PROMPTS[name]
    w = Batch(lens, gam, Hq, Hk, D, page, dt, prefix)
    out, lse = w.run()
    w.check(out, lse)
    again, lse2 = w.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("Hq, D", [(96, 64), (20, 128)])
def test_draft_masks_over_row_blocks(Hq, D):
    """Steps of 32 rows in blocks of 1 and of 6: a word of a first block may name a row of the last."""
    w = Batch([0, 100, 63, 64], [31, 31, 30, 5], Hq, 1, D, 16, "bf16")
    g = torch.Generator().manual_seed(8)
    mask = torch.randint(-2 ** 31, 2 ** 31 - 1, (w.T,), generator=g, dtype=torch.int64).int().cuda()
    out, lse = w.run(mask=mask)
    w.check(out, lse, mask=mask.long() & 0xffffffff)
