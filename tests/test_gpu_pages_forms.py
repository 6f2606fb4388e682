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
