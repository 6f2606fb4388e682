"""A call whose launch fails returns its error and leaves nothing behind: the next call is
judged by its own launch."""
import ctypes

import pytest
import torch

from speculative_decoding_verification_62_gb300 import binding, rope

pytestmark = pytest.mark.gpu


class InvalidCapture:
    """A stream whose capture has been invalidated on the host: every launch into it is
    refused, nothing runs."""

    def __enter__(self):
        torch.cuda.synchronize()
        cu = self.cu = ctypes.CDLL("libcuda.so.1")
        self.stream = ctypes.c_void_p()
        assert cu.cuStreamCreate(ctypes.byref(self.stream), 1) == 0
        assert cu.cuStreamBeginCapture_v2(self.stream, 2) == 0
        assert cu.cuStreamQuery(self.stream) != 0  # not allowed in a capture: ends its validity
        self.cuda_stream = self.stream.value
        return self

    def __exit__(self, *exc):
        graph = ctypes.c_void_p()
        assert self.cu.cuStreamEndCapture(self.stream, ctypes.byref(graph)) != 0
        assert self.cu.cuStreamDestroy_v2(self.stream) == 0


def verify(schedule, stream=None):
    """A small verify call.  The persistent grid asks for the launch's error."""
    v = binding.Verifier(2, 2, 300)
    z = torch.zeros
    prev = binding.spec_verify_set_schedule(schedule)
    try:
        v.sample(z((2, 3, 300), device="cuda"), z((2, 2, 300), device="cuda"),
                 z((2, 2), dtype=torch.int32, device="cuda"), torch.full((2,), 2, dtype=torch.int32, device="cuda"),
                 torch.full((2, 3), 0.5, device="cuda"), torch.ones(2, device="cuda"), stream=stream)
    finally:
        binding.spec_verify_set_schedule(prev)
    assert v.num_accepted.tolist() == [2, 2] and v.out_tokens[:, 2].tolist() == [150, 150]


def verify_clusters(stream=None):
    verify(binding.SCHEDULE_STREAM, stream)


def verify_auto(stream=None):
    verify(binding.SCHEDULE_AUTO, stream)


def status(stream=None):
    assert binding.spec_verify_status(torch.zeros(256, dtype=torch.uint8, device="cuda"), stream) == 0


def probs(stream=None):
    v = binding.Verifier(2, 1, 64)
    p = torch.full((2, 2, 64), 1 / 64, device="cuda")
    v.sample_probs(p, None, torch.zeros((2, 1), dtype=torch.int32, device="cuda"),
                   torch.ones(2, dtype=torch.int32, device="cuda"), torch.zeros((2, 2), device="cuda"), stream=stream)


def cache():
    pools = [torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    return binding.PagedCache(*pools, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                              torch.zeros(1, dtype=torch.int32, device="cuda"))


def append(stream=None):
    x = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    binding.spec_verify_kv_append(x, x.clone(), x.clone(), cache(), torch.zeros(2, dtype=torch.int32, device="cuda"), 0,
                                  rope.fixed_point(rope.frequencies(64)).cuda(), torch.empty_like(x),
                                  torch.zeros(256, dtype=torch.uint8, device="cuda"), stream=stream)


def attention(stream=None):
    x = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    binding.spec_verify_attention(x, cache(), torch.zeros(2, dtype=torch.int32, device="cuda"), 0, torch.empty_like(x),
                                  binding.make_attention_workspace(1, 1, 64), stream=stream)


@pytest.mark.parametrize("call", [probs, append, attention, verify_clusters, verify_auto, status])
def test_a_refused_launch_is_not_held_against_the_next_call(call):
    verify(binding.SCHEDULE_PERSISTENT)
    call()
    with InvalidCapture() as s:
        with pytest.raises(binding.SpecVerifyError) as e:
            call(s)
        assert e.value.code == -5
    verify(binding.SCHEDULE_PERSISTENT)
    call()
    torch.cuda.synchronize()

