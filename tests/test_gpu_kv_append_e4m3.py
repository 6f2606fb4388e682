"""The append into a cache of e4m3 codes against the definition in 64 bits: scales exactly, codes
up to the rounding of the rotation in 32 bits; every element of the pools that the
step does not own stays as it was."""
import math

import pytest
import torch

from cache8_refs import longest, nearest, scale_of, values
from operator_refs import rotate
from speculative_decoding_verification_62_gb300 import binding, rope

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
S = {n: b for b, n in binding.STATUS_BITS.items()}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Step:
    """Requests with older tokens in a cache of random codes and scales, and a step's rows."""

    def __init__(self, lens, gam, Hq, Hk, D, page, block, dtype, layout="nhd", seed=3, fused=True, size=1.0,
                 far=False, pad=0, shift=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        gc = torch.Generator().manual_seed(seed)
        self.lens, self.gam, self.page, self.block, self.dtype = lens, gam, page, block, DT[dtype]
        B, T = len(lens), sum(gam) + len(gam) + pad
        skip = [n // page if far else 0 for n in lens]  # far: only the pages of the step exist
        need = [-(-(n + x + 1) // page) - k for n, x, k in zip(lens, gam, skip)]
        total = sum(need) + 2
        perm = torch.randperm(total, generator=gc).int()
        self.table = torch.full((B, max(a + k for a, k in zip(need, skip))), -5, dtype=torch.int32)
        at = 0
        for b, (n, k) in enumerate(zip(need, skip)):
            self.table[b, k:k + n] = perm[at:at + n]
            at += n
        shape = (total, page, Hk, D) if layout == "nhd" else (total, Hk, page, D)
        raw = [torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        self.bytes = [r.transpose(1, 2) if layout == "hnd" else r for r in raw]
        self.scales = [torch.exp2(torch.randint(-9, -4, (total, page // block, Hk), generator=g, device="cuda").float())
                       for _ in range(2)]
        self.cache = binding.PagedCache(*(b.view(torch.float8_e4m3fn) for b in self.bytes), self.table.cuda(),
                                        ints(lens), k_scales=self.scales[0], v_scales=self.scales[1])
        qkv = (torch.randn((T, Hq + 2 * Hk, D + shift), generator=g, device="cuda") * size).to(self.dtype)[..., shift:]
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.cu = ints([0] + torch.tensor(gam).cumsum(0).tolist())
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run(self, freq, q_out=None, status=0, G=None, **more):
        if q_out is None:
            q_out = torch.full(self.q.shape, 9.0, dtype=self.dtype, device="cuda")
        self.before = [x.clone() for x in (*self.bytes, *self.scales)]
        fixed = None if freq is None else rope.fixed_point(freq).cuda()
        binding.spec_verify_kv_append_e4m3(self.q, self.k, self.v, self.cache, self.cu, max(self.gam) if G is None else G,
                                           fixed, q_out, self.ws, **more)
        if status is not None:
            assert binding.spec_verify_status(self.ws) == status
        return q_out

    def check(self, q_out, freq, interleaved=False, rope_scale=1.0, positions=None, position_offset=0, only=None):
        """A turned value in 32 bits: two products and a sum of factors good to 2^-22 (the angle to
        2^-24 turns): off by 2^-19 of the pair's larger value at most."""
        f = torch.zeros(0, dtype=torch.float64) if freq is None else freq
        f = f.cuda()
        rot, u = 2 * f.numel(), torch.finfo(self.dtype).eps / 2
        touched = [torch.zeros_like(x, dtype=torch.bool) for x in (*self.bytes, *self.scales)]
        row, page, bt = 0, self.page, self.block
        for b, (n, x) in enumerate(zip(self.lens, self.gam)):
            rows = slice(row, row + x + 1)
            row += x + 1
            if only is not None and b not in only:
                continue
            slots = torch.arange(n, n + x + 1)
            pos = (slots + position_offset if positions is None else positions[rows].long().cpu()).cuda()
            ids = self.table[b].long()
            if q_out is not None:
                want = rotate(self.q[rows].double(), pos, f, interleaved, rope_scale)
                tol = u * want.abs() * 1.001 + 2.0 ** -19 * rope_scale * self.q[rows].double().abs().amax() + 2.0 ** -25
                assert not ((q_out[rows].double() - want).abs() > tol).any()
            for kind in range(2):
                x64 = (self.k, self.v)[kind][rows].double()
                turned = rotate(x64, pos, f, interleaved, rope_scale) if kind == 0 else x64
                err = 2.0 ** -19 * rope_scale * torch.nan_to_num(x64, 0, 0, 0).abs().amax() if kind == 0 and rot else 0.0
                most = longest(x64, rot if kind == 0 else 0, interleaved, rope_scale)
                pool, scales = self.bytes[kind], self.scales[kind]
                was_pool, was_scales = self.before[kind], self.before[2 + kind]
                for first in range(n // bt * bt, n + x + 1, bt):
                    p, at = int(ids[first // page]), first % page
                    mine = (slots >= first) & (slots < first + bt)
                    s = scale_of(most[mine.cuda()].amax(0))
                    old = max(0, n - first)
                    if old:
                        was = was_scales[p, at // bt].double()
                        s = torch.maximum(s, was)
                        want = nearest(values(was_pool[p, at:at + old]) * (was / s)[None, :, None])
                        got = values(pool[p, at:at + old])
                        same = was == s
                        assert torch.equal(torch.nan_to_num(got, 1000.0), torch.nan_to_num(want, 1000.0))
                        assert torch.equal(pool[p, at:at + old][:, same], was_pool[p, at:at + old][:, same])
                        touched[kind][p, at:at + old] = True
                    assert torch.equal(scales[p, at // bt].double(), s), (b, first, kind)
                    touched[2 + kind][p, at // bt] = True
                    k = slots[mine] % page
                    got = values(pool[p][k.cuda()])
                    y = turned[mine.cuda()] / s[None, :, None]
                    near = nearest(y)
                    assert torch.equal(torch.isnan(got), torch.isnan(y))
                    far = (got - y.clamp(-448, 448)).abs() > (near - y.clamp(-448, 448)).abs() + 2 * err / s[None, :, None]
                    assert not (far & ~torch.isnan(y)).any(), (b, first, kind, int(far.sum()))
                    touched[kind][p, k.cuda()] = True
        for now, was, t in zip((*self.bytes, *self.scales), self.before, touched):
            assert torch.equal(now[~t], was[~t])


CASES = [
    # lens, gamma, Hq, Hk, D, rot, page, block, dtype, interleaved, layout
    ([0], [0], 1, 1, 16, 16, 16, 16, "bf16", False, "nhd"),
    ([15, 16, 0, 31], [0, 3, 7, 1], 8, 2, 128, 128, 16, 16, "bf16", False, "nhd"),
    ([100, 5, 63], [5, 0, 2], 6, 3, 64, 64, 64, 32, "f16", True, "hnd"),
    ([7, 1000], [1, 40], 4, 4, 96, 48, 32, 8, "bf16", False, "hnd"),
    ([7, 1000], [1, 4], 5, 1, 80, 40, 32, 32, "f16", False, "nhd"),   # pairs in ones
    ([3, 9], [4, 2], 4, 2, 48, 20, 16, 1, "bf16", True, "nhd"),
    ([3, 9], [40, 20], 4, 2, 128, 2, 16, 2, "bf16", False, "nhd"),
    ([3, 9], [40, 20], 4, 2, 128, 0, 16, 4, "f16", False, "nhd"),
    ([0, 0], [300, 77], 12, 4, 128, 64, 128, 128, "bf16", True, "nhd"),
    ([130, 70], [300, 77], 2, 3, 112, 96, 128, 64, "bf16", False, "hnd"),
    ([50] * 300, [7] * 300, 4, 1, 64, 64, 256, 16, "bf16", False, "nhd"),
    ([3, 30, 77] * 60, [0, 30, 100] * 60, 3, 9, 32, 32, 64, 16, "f16", False, "nhd"),
]


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_against_the_definition(case, fused):
    lens, gam, Hq, Hk, D, rot, page, block, dt, inter, layout = case
    w = Step(lens, gam, Hq, Hk, D, page, block, dt, layout, fused=fused)
    freq = rope.frequencies(rot, 10000.0) if rot else None
    w.check(w.run(freq, interleaved=inter), freq, inter)


@pytest.mark.parametrize("rows", [607, 608, 1216, 1217, 2047, 2048, 19457])
@pytest.mark.parametrize("D, rot, inter", [(128, 128, False), (64, 32, True), (48, 20, False)])
def test_around_the_borders_of_the_forms(rows, D, rot, inter):
    # one long request among short ones, so that the last rows' requests differ
    lens, gam = [5] * 25 + [70] + [31] * 25, [3] * 25 + [rows - 201] + [3] * 25
    w = Step(lens, gam, 3, 2, D, 32, 16, "bf16", seed=9)
    freq = rope.frequencies(rot, 10000.0)
    w.check(w.run(freq, interleaved=inter), freq, inter)


def test_far_positions_offsets_and_scaled_rotation():
    freq = rope.frequencies(64, 500000.0)
    w = Step([(1 << 20) - 1, 131071], [20, 2], 4, 2, 64, 4096, 64, "bf16", far=True)
    w.check(w.run(freq, position_offset=77777, rope_scale=1.25), freq, rope_scale=1.25, position_offset=77777)
    w = Step([9, 40], [5, 2], 4, 2, 64, 32, 16, "f16")
    pos = ints([9, 10, 10, 11, 11, 12, 40, 41, 41])
    w.check(w.run(freq, positions=pos), freq, positions=pos)


def test_no_queries_and_queries_in_place():
    freq = rope.frequencies(64)
    w = Step([9, 40], [5, 20], 4, 2, 64, 32, 16, "bf16")
    ref = w.run(freq)
    w.check(ref, freq)
    w = Step([9, 40], [5, 20], 4, 2, 64, 32, 16, "bf16")
    q = w.q
    w.q = None
    w.before = [x.clone() for x in (*w.bytes, *w.scales)]
    binding.spec_verify_kv_append_e4m3(None, w.k, w.v, w.cache, w.cu, 20, rope.fixed_point(freq).cuda(), None, w.ws)
    w.check(None, freq)
    w = Step([9, 40], [5, 20], 4, 2, 64, 32, 16, "bf16")
    w.run(freq, q_out=w.q)
    assert torch.equal(w.q, ref) and q.shape == ref.shape


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_scales_at_their_borders(dt):
    """Largest values at 448 2^e and one step above, zeros, and blocks whose scale does or
    does not grow."""
    w = Step([8] * 6, [2] * 6, 1, 2, 64, 16, 16, dt)
    step = torch.finfo(w.dtype).eps
    for b, most in enumerate([448.0, 448.0 * (1 + 4 * step), 448.0 * 2.0 ** -8, 0.0, 7.0 * (1 - step), 3.5]):
        rows = slice(3 * b, 3 * b + 3)
        for x in (w.k, w.v):
            x[rows] = (x[rows].float() / 1000.0).clamp(-1, 1) * min(1.0, most)
            x[rows.start + 1, :, 17] = -most
    w.check(w.run(None), None)
    # a block of zeros alone, and one that no longer grows
    w = Step([16, 16], [3, 3], 1, 2, 64, 16, 16, dt)
    w.k[:4] = 0.0
    w.check(w.run(None), None)
    assert bool((w.scales[0][int(w.table[0, 1]), 0] == 2.0 ** -32).all())
    again = [x.clone() for x in (*w.bytes, *w.scales)]
    w.run(None)  # (the same rows again: the same bytes)
    for x, y in zip((*w.bytes, *w.scales), again):
        assert torch.equal(x, y)


def test_tiny_huge_infinite_and_nan_values():
    w = Step([16, 16, 16, 5], [3, 3, 3, 3], 1, 1, 64, 16, 16, "bf16")
    for x in (w.k, w.v):
        x[0:4] *= 2.0 ** -45                  # below the smallest scale's steps
        x[4:8] *= 2.0 ** 70                   # beyond 448 2^56
        x[8, 0, 3], x[9, 0, 5] = math.nan, math.inf
        x[12, 0, 7] = -math.inf
    w.check(w.run(None), None)
    for s in w.scales:
        p = w.table[:, 1].long()
        assert float(s[p[0], 0]) == 2.0 ** -32 and float(s[p[1], 0]) == 2.0 ** 56 and float(s[p[2], 0]) == 2.0 ** 56


def test_bad_entries():
    freq = rope.frequencies(64)

    def fresh(**kw):
        return Step([9, 40, 20], [5, 20, 3], 4, 2, 64, 32, 16, "bf16", **kw)
    # older tokens with a scale that is none: their codes stay, the scale is the new rows'
    for bad in (math.nan, 0.0, -1.0, math.inf, 2.0 ** -33, 2.0 ** 65):
        w = fresh()
        p = int(w.table[0, 0])
        w.scales[0][p, 0] = bad
        w.run(freq, status=S["BAD_SCALE"])
        most = longest(w.k[:6].double(), 64, False).amax(0)
        assert torch.equal(w.scales[0][p, 0].double(), scale_of(most))
        assert torch.equal(w.bytes[0][p, :9], w.before[0][p, :9])
    # a request past its page table, a page outside the pool, a length below 0
    w = fresh()
    w.cache.kv_len[1] = 10 ** 6
    out = w.run(freq, status=S["BAD_LENGTH"])
    w.check(out, freq, only=[0, 2])
    w = fresh()
    w.cache.page_table[1, 1] = 10 ** 6
    w.lens[1] = 40
    out = w.run(freq, status=S["BAD_PAGE"])
    w.check(out, freq, only=[0, 2])
    w = fresh()
    w.cache.kv_len[0] = -4
    out = w.run(freq, status=S["BAD_LENGTH"])
    w.check(out, freq, only=[1, 2])
    # inconsistent lengths
    w = fresh()
    w.cu[1] = 50
    out = w.run(freq, status=S["BAD_GAMMA"])
    assert bool((out[:6] == 9.0).all())
    # rows behind the last request's are no error and stay
    w = fresh(pad=5)
    out = w.run(freq)
    w.check(out, freq)
    assert bool((out[-5:] == 9.0).all())


def test_a_request_that_ends_in_its_table():
    """The rows that fit are stored, the others set the status; blocks are as if they were not."""
    freq = rope.frequencies(64)
    w = Step([9], [40], 4, 2, 64, 16, 16, "bf16")
    narrow = binding.PagedCache(w.cache.k_pages, w.cache.v_pages, w.cache.page_table[:, :2].contiguous(),
                                w.cache.kv_len, k_scales=w.scales[0], v_scales=w.scales[1])
    full, w.cache = w.cache, narrow
    out = w.run(freq, status=S["BAD_LENGTH"])
    rows = 32 - 9
    w.gam, w.q, w.k, w.v = [rows - 1], w.q[:rows], w.k[:rows], w.v[:rows]
    w.check(out[:rows], freq)


def test_steps_rolled_back_and_overwritten():
    """Four steps of one request in 16-token blocks, with rejected rows in between."""
    freq = rope.frequencies(64)
    w = Step([14], [7], 4, 2, 64, 64, 16, "bf16", size=0.01)
    for turn, (n, size) in enumerate([(14, 1.0), (17, 50.0), (18, 0.1), (26, 300.0)]):
        w.lens = [n]
        w.cache.kv_len.fill_(n)
        g = torch.Generator(device="cuda").manual_seed(turn)
        for x in (w.q, w.k, w.v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda") * size)
        w.check(w.run(freq), freq)


def test_streams_and_graphs():
    freq = rope.frequencies(64)
    w, ref = (Step([9, 40], [5, 20], 4, 2, 64, 32, 16, "bf16") for _ in range(2))
    fixed = rope.fixed_point(freq).cuda()
    want = ref.run(freq)
    out = torch.zeros_like(want)
    start = [x.clone() for x in (*w.bytes, *w.scales)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.spec_verify_kv_append_e4m3(w.q, w.k, w.v, w.cache, w.cu, 20, fixed, out, w.ws)
    side = torch.cuda.Stream()
    for x, y in zip((*w.bytes, *w.scales), start):
        x.copy_(y)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    for x, y in zip((*w.bytes, *w.scales), (*ref.bytes, *ref.scales)):
        assert torch.equal(x, y)
    # the 16-bit call's name takes the cache too
    for x, y in zip((*w.bytes, *w.scales), start):
        x.copy_(y)
    binding.spec_verify_kv_append(w.q, w.k, w.v, w.cache, w.cu, 20, fixed, out, w.ws, stream=torch.cuda.current_stream())
    for x, y in zip((*w.bytes, *w.scales), (*ref.bytes, *ref.scales)):
        assert torch.equal(x, y)


def test_refused_tensors():
    w = Step([9, 40], [5, 20], 4, 2, 64, 32, 16, "bf16")
    freq = rope.fixed_point(rope.frequencies(64)).cuda()
    out = torch.empty(w.q.shape, dtype=w.dtype, device="cuda")
    call = binding.spec_verify_kv_append_e4m3
    with pytest.raises(TypeError):
        call(w.q, w.k.half(), w.v, w.cache, w.cu, 20, freq, out, w.ws)
    with pytest.raises(TypeError):
        call(w.q, w.k.float(), w.v.float(), w.cache, w.cu, 20, freq, out, w.ws)
    with pytest.raises(ValueError):
        call(w.q, w.k[:, :1], w.v[:, :1], w.cache, w.cu, 20, freq, out, w.ws)
    pools = [torch.zeros((4, 32, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    wide = binding.PagedCache(*pools, w.cache.page_table, w.cache.kv_len)
    with pytest.raises(TypeError):  # a cache of 16 bits
        call(w.q, w.k, w.v, wide, w.cu, 20, freq, out, w.ws)
    eight = [p.to(torch.float8_e4m3fn) for p in pools]
    s = torch.ones((4, 2, 2), device="cuda")
    for pk, more, error in ((eight, {}, ValueError), (pools, dict(k_scales=s, v_scales=s), TypeError),
                            (eight, dict(k_scales=s), TypeError), (eight, dict(k_scales=s[:3], v_scales=s), ValueError),
                            (eight, dict(k_scales=s.half(), v_scales=s.half()), TypeError),
                            (eight, dict(k_scales=torch.ones((4, 3, 2), device="cuda"), v_scales=s), ValueError),
                            (eight, dict(k_scales=s, v_scales=torch.ones((4, 1, 2), device="cuda")), ValueError)):
        with pytest.raises(error):
            binding.PagedCache(*pk, w.cache.page_table, w.cache.kv_len, **more)
    # head_dim must be a multiple of 16, a block at most 128 tokens
    for page, D, per in ((32, 24, 2), (256, 32, 1)):
        p8 = [torch.zeros((2, page, 1, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
        s = torch.ones((2, per, 1), device="cuda")
        with pytest.raises(ValueError):
            binding.PagedCache(*p8, w.cache.page_table, w.cache.kv_len, k_scales=s, v_scales=s)
