"""The pages of a cache: calls that the tests of the operators themselves do not make."""
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
