"""The pages of a cache against a model in plain Python: every whole number and every byte."""
import random

import pytest
import torch

from cache8_refs import Pages
from speculative_decoding_verification_62_gb300 import binding

pytestmark = pytest.mark.gpu
S = {n: b for b, n in binding.STATUS_BITS.items()}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pool:
    """A cache whose pages hold random bytes, and its model."""

    def __init__(self, B, width, pages, page=16, heads=2, D=16, kind="bf16", layout="nhd", block=16, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        es = 1 if kind == "e4m3" else 2
        shape = (pages, page, heads, D * es) if layout != "hnd" else (pages, heads, page, D * es)
        if layout == "wide":  # a token's heads lie in wider rows
            shape = (pages, page, heads + 3, D * es)
        self.raw = [torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        dt = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}[kind]
        pools = [r.view(dt) for r in self.raw]
        if layout == "hnd":
            pools = [p.transpose(1, 2) for p in pools]
        if layout == "wide":
            pools = [p[:, :, 1:heads + 1] for p in pools]
        self.bytes = [r.transpose(1, 2) if layout == "hnd" else r[:, :, 1:heads + 1] if layout == "wide" else r
                      for r in self.raw]
        self.scales = []
        if kind == "e4m3":
            self.scales = [torch.rand((pages, page // block, heads), generator=g, device="cuda") + 0.5 for _ in range(2)]
        self.block, self.page = block, page
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.cache = binding.PagedCache(*pools, table, ints([0] * B),
                                        **(dict(k_scales=self.scales[0], v_scales=self.scales[1]) if self.scales else {}))
        self.pool = binding.PagePool(self.cache)
        self.model = Pages(table.tolist(), [0] * B, [0] * B, [0] * pages, range(pages - 1, -1, -1), page)

    def everything(self):
        return [*self.raw, *self.scales]

    def set_len(self, kv):
        self.cache.kv_len.copy_(ints(kv))
        self.model.kv = list(kv)

    def same(self):
        m, p, c = self.model, self.pool, self.cache
        assert c.page_table.tolist() == m.table and c.kv_len.tolist() == m.kv
        assert p.held.tolist() == m.held and p.ref.tolist() == m.ref
        assert int(p.free_count) == len(m.free) and p.free_pages[:len(m.free)].tolist() == m.free
        # (the workspace is zero again behind the status word, up to the rows' scratch)
        n = -(-4 * p.ref.numel() // 256) * 256
        assert not p.workspace[256:256 + 3 * n].any()

    def step(self, tokens, parents=None, status=0):
        want = [x.clone() for x in self.everything()]
        binding.spec_verify_pages_step(self.cache, self.pool, ints(tokens), None if parents is None else ints(parents))
        fits, copies = self.model.step(tokens, parents)
        assert binding.spec_verify_status(self.pool.workspace) == status | (0 if fits else S["NO_PAGES"])
        self.same()
        got = [x.clone() for x in self.everything()]
        for x, y in zip(self.everything(), want):
            x.copy_(y)
        for src, dst, n in copies:
            for x in self.bytes:
                x[dst, :n] = x[src, :n]
            for x in self.scales:
                x[dst, :-(-n // self.block)] = x[src, :-(-n // self.block)]
        for x, y in zip(got, self.everything()):
            assert torch.equal(x, y)
        return fits, copies

    def compact(self):
        want = [x.clone() for x in self.everything()]
        remap = torch.full((len(self.model.ref),), -7, dtype=torch.int32, device="cuda")
        binding.spec_verify_pages_compact(self.cache, self.pool, remap)
        model, moves = self.model.compact()
        assert binding.spec_verify_status(self.pool.workspace) == 0
        assert remap.tolist() == model
        self.same()
        got = [x.clone() for x in self.everything()]
        for x, y in zip(self.everything(), want):
            x.copy_(y)
        for src, dst in moves:
            for x in [*self.bytes, *self.scales]:
                x[dst] = x[src]
        for x, y in zip(got, self.everything()):
            assert torch.equal(x, y)
        return moves


def test_one_row_takes_and_gives_back():
    w = Pool(1, 4, 6)
    assert w.step([5]) == (True, [])
    w.step([5])                      # the same page again
    w.set_len([5])
    w.step([12])                     # 17 tokens: a second page
    assert w.pool.held.tolist() == [2]
    w.step([11])                     # 16: given back
    w.set_len([16])
    w.step([0])
    w.step([48])                     # the whole table
    w.step([0], [-1])                # ends
    assert int(w.pool.free_count) == 6
    w.step([0])


def test_a_fork_shares_and_copies():
    w = Pool(3, 4, 12, kind="e4m3", block=4)
    w.step([21, 0, 0])
    w.set_len([21, 0, 0])
    fits, copies = w.step([1, 1, 1], [0, 0, 0])
    assert [c[2] for c in copies] == [5, 5] and w.pool.ref.tolist().count(3) == 1
    # one ends, one that only reads holds the partly filled page too
    w.set_len([22, 22, 22])
    w.step([2, 0, 0], [1, 1, -1])
    w.step([2, 2, 0], [0, 0, 0])


@pytest.mark.parametrize("kind, layout, page, heads, D, block", [
    ("bf16", "nhd", 16, 2, 16, 16), ("f16", "hnd", 32, 3, 8, 16), ("e4m3", "nhd", 32, 2, 48, 8),
    ("e4m3", "hnd", 16, 1, 128, 16), ("bf16", "wide", 16, 2, 40, 16), ("e4m3", "wide", 64, 3, 16, 1)])
@pytest.mark.parametrize("B, width, pages", [(1, 3, 5), (7, 6, 40), (33, 5, 90), (70, 70, 900)])
def test_random_steps(B, width, pages, kind, layout, page, heads, D, block):
    rng = random.Random(B * 7 + page + D)
    w = Pool(B, width, pages, page, heads, D, kind, layout, block)
    some_fail = 0
    for turn in range(12):
        most = [width * page - k for k in w.model.kv]
        parents = None
        if turn % 3 != 0:
            parents = [rng.choice([b, b, rng.randrange(B), rng.randrange(B), -1]) for b in range(B)]
            most = [width * page if p < 0 else width * page - w.model.kv[p] for p in parents]
        tokens = [rng.randint(0, min(m, rng.choice([0, 1, 3, 2 * page]))) for m in most]
        fits, _ = w.step(tokens, parents)
        some_fail += not fits
        if fits:  # what the step appended, all or in part
            w.set_len([k + rng.randint(0, t) if p >= 0 else 0
                       for k, t, p in zip(w.model.kv, tokens, parents or range(B))])
        if turn % 4 == 3:
            w.compact()
    w.compact()


def test_no_pages_takes_none():
    w = Pool(4, 4, 6)
    w.step([16, 16, 5, 0])
    w.set_len([16, 16, 5, 0])
    assert w.step([1, 1, 30, 16])[0] is False
    assert w.pool.held.tolist() == [1, 1, 1, 0] and int(w.pool.free_count) == 3
    # a shared page that cannot be copied stays shared
    assert w.step([1, 1, 30, 30], [0, 1, 2, 2])[0] is False
    assert w.step([1, 1, 1, 0], [0, 1, 2, -1])[0] is True


def test_parents_in_a_ring_and_all_of_one():
    B = 40
    w = Pool(B, 3, 300)
    w.step([20 + b % 7 for b in range(B)])
    w.set_len([20 + b % 7 for b in range(B)])
    w.step([3] * B, [(b + 1) % B for b in range(B)])
    w.step([3] * B, [17] * B)
    w.step([3] * B, [-1] * B)
    assert int(w.pool.free_count) == 300


def test_bad_entries():
    w = Pool(3, 4, 20)
    w.step([20, 20, 20])
    w.set_len([20, 20, 20])
    # a parent that is no row: the row continues itself
    w.model.step([1, 1, 1], [0, 1, 2])
    binding.spec_verify_pages_step(w.cache, w.pool, ints([1, 1, 1]), ints([5, -2, 2]))
    assert binding.spec_verify_status(w.pool.workspace) == S["BAD_ROW"]
    w.same()
    # tokens below 0 or past the table count as 0
    w.model.step([0, 0, 1])
    binding.spec_verify_pages_step(w.cache, w.pool, ints([-4, 100, 1]))
    assert binding.spec_verify_status(w.pool.workspace) == S["BAD_LENGTH"]
    w.same()
    # a length past the pages held counts as those
    w.cache.kv_len.copy_(ints([20, 10 ** 9, -3]))
    w.model.kv = [20, 32, 0]
    w.model.step([1, 1, 1])
    binding.spec_verify_pages_step(w.cache, w.pool, ints([1, 1, 1]))
    assert binding.spec_verify_status(w.pool.workspace) == S["BAD_LENGTH"]
    w.same()
    # entries outside the pool are neither counted nor copied
    w.cache.page_table[1, 0] = 1000
    binding.spec_verify_pages_step(w.cache, w.pool, ints([1, 1, 1]), ints([1, 1, 1]))
    assert binding.spec_verify_status(w.pool.workspace) == S["BAD_PAGE"]
    remap = torch.empty(20, dtype=torch.int32, device="cuda")
    binding.spec_verify_pages_compact(w.cache, w.pool, remap)
    assert binding.spec_verify_status(w.pool.workspace) == S["BAD_PAGE"]


def test_a_large_pool_compacts():
    """More pages than a cluster has threads, in every state."""
    N = 30011
    raw = torch.arange(N, dtype=torch.int32, device="cuda").view(N, 1, 1, 1).expand(N, 16, 1, 4).contiguous()
    pools = [raw.view(torch.bfloat16), (raw + 1).view(torch.bfloat16)]
    table = torch.full((9, 4000), -1, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(3)
    held = [0, 1, 4000, 17, 3999, 2, 2500, 3000, 1000]
    order = torch.randperm(N, generator=g).int()
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n].cuda()
        at += n
    cache = binding.PagedCache(*pools, table, ints([16 * n for n in held]))
    prefix = order[at:at + 33].cuda()
    pool = binding.PagePool.of_table(cache, ints(held), prefix)
    used = at + 33
    assert int(pool.free_count) == N - used
    before = table.clone()
    want = [pools[0].view(torch.int32)[:, 0, 0, 0].clone(), pools[1].view(torch.int32)[:, 0, 0, 0].clone()]
    remap = torch.empty(N, dtype=torch.int32, device="cuda")
    binding.spec_verify_pages_compact(cache, pool, remap)
    assert binding.spec_verify_status(pool.workspace) == 0
    live = remap >= 0
    assert int(live.sum()) == used and remap[live].sort()[0].tolist() == list(range(used))
    assert bool((remap[:used][live[:used]] == torch.arange(used, device="cuda")[live[:used]]).all())
    for x, y in zip(pools, want):
        now = x.view(torch.int32)
        assert torch.equal(now[remap[live].long(), 3, 0, 1], y[live])
    for b, n in enumerate(held):
        assert torch.equal(table[b, :n], remap[before[b, :n].long()])
    assert (remap[prefix.long()] >= 0).all() and bool((pool.ref[:used] == 1).all()) and not pool.ref[used:].any()
    assert pool.free_pages[:N - used].tolist() == list(range(N - 1, used - 1, -1))
    # nothing moves twice
    binding.spec_verify_pages_compact(cache, pool, remap)
    assert torch.equal(remap[:used], torch.arange(used, dtype=torch.int32, device="cuda"))


def test_many_rows():
    """More rows than the cluster has warps, and than one sum takes at once."""
    B = 2500
    rng = random.Random(5)
    w = Pool(B, 3, 6000, heads=1, D=8)
    w.step([rng.randint(0, 33) for _ in range(B)])
    w.set_len([rng.randint(0, h * 16) for h in w.model.held])
    w.step([rng.randint(0, 3) if k < 45 else 0 for k in w.model.kv])
    parents = [rng.choice([b, b, b, rng.randrange(B), -1]) for b in range(B)]
    w.step([0 if p < 0 or w.model.kv[p] > 44 else 2 for p in parents], parents)
    w.compact()


def test_streams_graphs_and_a_second_pool():
    a, b = Pool(9, 6, 80, seed=1), Pool(20, 4, 90, page=32, kind="e4m3", seed=2)
    ref_a, ref_b = Pool(9, 6, 80, seed=1), Pool(20, 4, 90, page=32, kind="e4m3", seed=2)
    ta, tb = ints([20] * 9), ints([40] * 20)
    pa, pb = ints([0] * 9), ints([3, -1] * 10)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        binding.spec_verify_pages_step(a.cache, a.pool, ta)
        a.cache.kv_len.add_(ta)
    binding.spec_verify_pages_step(b.cache, b.pool, tb)
    b.cache.kv_len.add_(tb)
    torch.cuda.synchronize()
    graphs = []
    remap = torch.empty(80, dtype=torch.int32, device="cuda")
    for x, t, p in ((a, ta, pa), (b, tb, pb)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            binding.spec_verify_pages_step(x.cache, x.pool, t, p)
            if x is a:
                binding.spec_verify_pages_compact(a.cache, a.pool, remap)
        graphs.append(graph)
    for x, t, p in ((ref_a, [20] * 9, [0] * 9), (ref_b, [40] * 20, [3, -1] * 10)):
        x.step(t)
        x.set_len(t)
        for _ in range(3):
            x.step(t, p)
            if x is ref_a:
                x.compact()
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for x, y in ((a, ref_a), (b, ref_b)):
        x.model = y.model
        x.same()
        for u, v in zip(x.everything(), y.everything()):
            assert torch.equal(u, v)


def test_refused_tensors():
    w = Pool(3, 4, 20)
    good = ints([1, 1, 1])
    for tokens, parents in ((ints([1, 1]), None), (good, ints([0, 1])), (good[::2], None), (good.long(), None),
                            (good.cpu(), None), (good, good.float())):
        with pytest.raises((ValueError, TypeError)):
            binding.spec_verify_pages_step(w.cache, w.pool, tokens, parents)
    with pytest.raises(ValueError):
        binding.spec_verify_pages_compact(w.cache, w.pool, ints([0] * 19))
    with pytest.raises(AttributeError):
        w.pool.held = good
    with pytest.raises(ValueError):
        binding.PagePool(w.cache, held=ints([0, 0]))
    with pytest.raises(ValueError):
        binding.PagePool.of_table(w.cache, ints([1, 0, 0]))  # an entry of -1
    empty = binding.PagedCache(w.cache.k_pages, w.cache.v_pages, w.cache.page_table[:0], w.cache.kv_len[:0])
    binding.spec_verify_pages_step(empty, binding.PagePool(empty), ints([]))
