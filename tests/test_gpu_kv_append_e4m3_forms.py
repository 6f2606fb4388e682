"""The append into a cache of e4m3 codes: calls at the ends of its arguments."""
import pytest
import torch

from speculative_decoding_verification_62_gb300 import binding, rope
from test_gpu_kv_append_e4m3 import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 20])
@pytest.mark.parametrize("size, rope_scale", [(2.0 ** 70, 2.0 ** -20), (2.0 ** 100, 2.0 ** -90), (2.0 ** -60, 2.0 ** 66),
                                              (2.0 ** -90, 1.5 * 2.0 ** 100), (2.0 ** 63, 1.25), (2.0 ** -30, 3.0)])
def test_a_rotations_factor_against_the_values(size, rope_scale, rot, interleaved):
    """The largest magnitude of the turned pair is ordinary, or at the scales' ends, while the squares of the
    values, or of the factor, leave 32 bits."""
    w = Step([9, 40, 0], [5, 20, 3], 4, 2, 64, 32, 16, "bf16", size=size)
    freq = rope.frequencies(rot)
    w.check(w.run(freq, rope_scale=rope_scale, interleaved=interleaved), freq, interleaved, rope_scale=rope_scale)


@pytest.mark.parametrize("rows", [607, 608, 2047, 2048, 6143, 6144])
@pytest.mark.parametrize("D, rot, inter, Hk", [(128, 128, False, 4), (64, 32, True, 9), (48, 20, False, 5)])
def test_around_the_borders_of_the_forms_with_many_heads(rows, D, rot, inter, Hk):
    lens, gam = [5] * 25 + [70] + [31] * 25, [3] * 25 + [rows - 201] + [3] * 25
    w = Step(lens, gam, 2 * Hk, Hk, D, 32, 16, "bf16", seed=9)
    freq = rope.frequencies(rot, 10000.0)
    w.check(w.run(freq, interleaved=inter), freq, inter)
