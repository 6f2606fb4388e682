"""A page pool and the cache that it is used with have one size (on the host, no GPU)."""
from types import SimpleNamespace

import pytest

from speculative_decoding_verification_62_gb300 import binding


def test_a_pool_of_another_size_is_refused():
    """The kernels take the sizes from the cache and write the pool's tensors."""
    mine = (0, 1000, 8, 64)
    pool = SimpleNamespace(sizes=mine)
    for other in ((0, 1000, 64, 8), (0, 1001, 8, 64), (0, 999, 8, 64), (0, 1000, 9, 64), (0, 1000, 8, 63),
                  (1, 1000, 8, 64)):
        cache = SimpleNamespace(sizes=other)
        with pytest.raises(ValueError):
            binding.spec_verify_pages_step(cache, pool, None)
        with pytest.raises(ValueError):
            binding.spec_verify_pages_compact(cache, pool, None)


@pytest.mark.parametrize("given", [("held",), ("held", "ref"), ("free_pages",), ("held", "ref", "free_pages")])
def test_a_pools_tensors_go_together(given):
    with pytest.raises(ValueError):
        binding.PagePool(SimpleNamespace(sizes=(0, 10, 2, 4)), **{n: object() for n in given})
