"""Attention over a cache of e4m3 codes: the forms of the call beside the plain one, with the
weights' rounding as fp16."""
import math

import pytest
import torch

from operator_refs import attend
from speculative_decoding_verification_62_gb300 import binding
from test_gpu_attention_e4m3 import DT, S, Batch, ints, tolerance

pytestmark = pytest.mark.gpu


def tight(q, k, o, lse, spread, size, weight, scale, lv, dtype):
    """tolerance() with a weight off by 2^-11 of itself, as fp16 rounds it: the sum of its three
    8-bit floats is that fp16 (the first two are rounded to the nearest, so that what is left
    after them has three bits)."""
    tol, tl = tolerance(q, k, o, lse, spread, size, weight, scale, lv, dtype)
    return tol - (2.0 ** -9 * 1.13 - 2.0 ** -11) * 1.01 * spread, tl


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
