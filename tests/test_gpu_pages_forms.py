"""The pages of a cache: calls that the tests of the operators themselves do not make."""
import random

import pytest
import torch

from speculative_decoding_verification_62_gb300 import binding
from test_gpu_pages import S, Pool, ints

pytestmark = pytest.mark.gpu


def test_a_pool_serves_caches_of_its_size_alone():
    w = Pool(8, 10, 100)
    remap = torch.empty(100, dtype=torch.int32, device="cuda")
    c = w.cache
    others = [binding.PagedCache(c.k_pages, c.v_pages, *t) for t in (
        (ints([[-1]] * 64), ints([0] * 64)), (c.page_table[:7], c.kv_len[:7]),
        (c.page_table[:, :9].contiguous(), c.kv_len))]
    others.append(binding.PagedCache(c.k_pages[:99], c.v_pages[:99], c.page_table, c.kv_len))
    for other in others:
        with pytest.raises(ValueError):
            binding.spec_verify_pages_step(other, w.pool, ints([1] * other.batch))
        with pytest.raises(ValueError):
            binding.spec_verify_pages_compact(other, w.pool, remap[:other.sizes[1]])
    with pytest.raises(ValueError):
        binding.PagePool(c, held=ints([0] * 8), ref=ints([0] * 100))
    # another cache of the size over the same tensors
    again = binding.PagedCache(c.k_pages, c.v_pages, c.page_table, c.kv_len)
    binding.spec_verify_pages_step(again, w.pool, ints([17] * 8))
    assert binding.spec_verify_status(w.pool.workspace) == 0 and w.pool.held.tolist() == [2] * 8


class Reused(Pool):
    """A pool whose workspace is someone else's: what it held before is no matter."""

    def share(self, ws):
        self.pool.workspace = ws
        return self

    def same(self):
        ws, self.pool.workspace = self.pool.workspace, torch.zeros_like(self.pool.workspace)
        super().same()
        self.pool.workspace = ws


def test_one_workspace_for_pools_of_other_sizes():
    shapes = [(7, 6, 40), (70, 70, 900), (33, 5, 90), (20, 12, 2000)]
    pools = [Reused(b, width, n, seed=n) for b, width, n in shapes]
    size = max(p.pool.workspace.numel() for p in pools)
    ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    ws[:4] = 0
    rng = random.Random(11)
    for turn in range(6):
        for w in pools:
            w.share(ws)
            B, room = len(w.model.kv), len(w.model.table[0]) * w.page
            parents = [rng.choice([b, b, rng.randrange(B), -1]) for b in range(B)] if turn else list(range(B))
            most = [0 if p < 0 else room - w.model.kv[p] for p in parents]
            tokens = [rng.randint(0, min(m, 40)) for m in most]
            if w.step(tokens, parents)[0]:
                w.set_len([k + rng.randint(0, t) if p >= 0 else 0 for k, t, p in zip(w.model.kv, tokens, parents)])
            if turn % 3 == 2:
                w.compact()


@pytest.mark.parametrize("bad", [1000, 20, -1, -2 ** 31])
@pytest.mark.parametrize("own_parents", [False, True])
def test_bad_entries_of_rows_that_continue_themselves(own_parents, bad):
    w = Pool(3, 4, 20)
    parents = ints([0, 1, 2]) if own_parents else None
    w.step([20, 20, 20])
    w.set_len([20, 20, 20])
    w.cache.page_table[1, 1] = w.model.table[1][1] = bad
    bytes_ = [x.clone() for x in w.everything()]
    # the page that row 1 writes to behind 4 tokens
    binding.spec_verify_pages_step(w.cache, w.pool, ints([1, 13, 1]), parents)
    assert binding.spec_verify_status(w.pool.workspace) == S["BAD_PAGE"]
    w.model.table[1][2] = w.model.free.pop()  # (its third page is taken all the same)
    w.model.ref[w.model.table[1][2]] = 1
    w.model.held = [2, 3, 2]
    w.same()
    # given back: it counts for no page
    w.set_len([20, 7, 20])
    binding.spec_verify_pages_step(w.cache, w.pool, ints([1, 1, 1]), parents)
    assert binding.spec_verify_status(w.pool.workspace) == S["BAD_PAGE"]
    w.model.free.append(w.model.table[1][2])
    w.model.ref[w.model.table[1][2]] = 0
    w.model.table[1][1:3] = [-1, -1]
    w.model.held = [2, 1, 2]
    w.same()
    w.step([1, 1, 1])
    for x, y in zip(w.everything(), bytes_):
        assert torch.equal(x, y)


def test_bad_entries_that_forks_take_up():
    """A parent's entry outside the pool: status, and tables and counts as without that page."""
    w = Pool(3, 4, 20)
    w.step([20, 20, 20])
    w.set_len([20, 20, 20])
    table, ref, free = [list(r) for r in w.model.table], list(w.model.ref), list(w.model.free)
    w.cache.page_table[1, 0] = 1000
    binding.spec_verify_pages_step(w.cache, w.pool, ints([0, 0, 0]), ints([1, 1, 1]))
    assert binding.spec_verify_status(w.pool.workspace) == S["BAD_PAGE"]
    shared = table[1][1]
    gone = [table[0][0], table[0][1], table[2][0], table[2][1]]
    for p in gone:
        ref[p] = 0
    ref[shared] = 3
    w.model.table = [[1000, shared, -1, -1] for _ in range(3)]
    w.model.ref, w.model.free = ref, free + gone
    w.same()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_prefix_moves_without_rows(kind):
    w = Pool(2, 3, 30, kind=kind)
    c = w.cache
    more = dict(k_scales=w.scales[0], v_scales=w.scales[1]) if w.scales else {}
    empty = binding.PagedCache(c.k_pages, c.v_pages, c.page_table[:0], c.kv_len[:0], **more)
    prefix = ints([20, 3, 29, 0, 11])
    pool = binding.PagePool.of_table(empty, ints([]), prefix)
    before = [x.clone() for x in w.everything()]
    remap = torch.full((30,), -7, dtype=torch.int32, device="cuda")
    binding.spec_verify_pages_compact(empty, pool, remap)
    assert binding.spec_verify_status(pool.workspace) == 0
    assert remap.tolist() == [{0: 0, 3: 3, 11: 1, 20: 2, 29: 4}.get(p, -1) for p in range(30)]
    assert pool.ref.tolist() == [1] * 5 + [0] * 25 and int(pool.free_count) == 25
    assert pool.free_pages[:25].tolist() == list(range(29, 4, -1))
    for now, was in zip(w.everything(), before):
        assert torch.equal(now[remap[prefix.long()].long()], was[prefix.long()])
    # a step of no rows does nothing
    binding.spec_verify_pages_step(empty, pool, ints([]))
    assert int(pool.free_count) == 25


@pytest.mark.parametrize("B, pages", [(31, 2048), (32, 2049), (33, 2500), (64, 600)])
def test_around_the_borders_of_the_forms(B, pages):
    """One CTA or a cluster: 32 rows and one more, 2048 pages and one more."""
    rng = random.Random(B)
    w = Pool(B, 8, pages, heads=1, D=8)
    w.step([rng.randint(0, 100) for _ in range(B)])
    w.set_len([rng.randint(0, h * 16) for h in w.model.held])
    for turn in range(3):
        parents = [rng.choice([b, b, rng.randrange(B), -1]) for b in range(B)]
        tokens = [0 if p < 0 else rng.randint(0, 128 - w.model.kv[p]) for p in parents]
        w.step(tokens, parents)
        w.compact()
