"""The paged append with rotation against the definition in 64 bits; every element of
the pools that the step does not own stays as it was."""
import pytest
import torch

from operator_refs import rotate
from speculative_decoding_verification_62_gb300 import binding, rope

pytestmark = pytest.mark.gpu


def setup(lens, gam, Hq, Hk, D, page, dtype, seed, layout="nhd", fused=True, spare=2):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [-(-(n + x + 1) // page) for n, x in zip(lens, gam)]
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g).int()
    table = torch.full((B, max(need) if need else 0), -5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    shape = (total, page, Hk, D) if layout == "nhd" else (total, Hk, page, D)
    k_pages = torch.randn(shape, generator=g).to(dtype).cuda()
    v_pages = torch.randn(shape, generator=g).to(dtype).cuda()
    if layout == "hnd":
        k_pages, v_pages = k_pages.transpose(1, 2), v_pages.transpose(1, 2)
    T = sum(gam) + B
    qkv = torch.randn((T, Hq + 2 * Hk, D), generator=g).to(dtype).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cu = torch.tensor([0] + torch.tensor(gam).cumsum(0).tolist(), dtype=torch.int32).cuda()
    cache = binding.PagedCache(k_pages, v_pages, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    return q, k, v, cu, cache, table


def expect(q, k, v, cu, cache, table, lens, gam, freq, inter, offset=0, scale=1.0, positions=None):
    """q_out, pools as float64 and the tolerance of a rotated value: two products and a
    sum in 32 bits, of factors good to 2^-22 (the angle to 2^-24 turns), and one rounding."""
    page = cache.page_size
    kp, vp, qo = cache.k_pages.double(), cache.v_pages.double(), q.double().clone()
    row = 0
    for b, (n, x) in enumerate(zip(lens, gam)):
        sl = torch.arange(n, n + x + 1)
        rows = slice(row, row + x + 1)
        pos = (sl + offset if positions is None else positions[rows]).cuda()
        ids = table[b].long()[sl // page].cuda()
        f = freq.cuda() if freq is not None else torch.zeros(0, dtype=torch.float64, device="cuda")
        qo[rows] = rotate(q[rows].double(), pos, f, inter, scale)
        kp[ids, (sl % page).cuda()] = rotate(k[rows].double(), pos, f, inter, scale)
        vp[ids, (sl % page).cuda()] = v[rows].double()
        row += x + 1
    return qo, kp, vp


def check(got, want, x_max, dtype, scale=1.0):
    u = torch.finfo(dtype).eps / 2
    tol = u * want.abs() * 1.001 + 4 * 2.0 ** -21 * x_max * scale + (2.0 ** -25 if dtype == torch.float16 else 0)
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() - tol).max()))


CASES = [
    # lens, gamma, Hq, Hk, D, rot, page, dtype, interleaved, layout
    ([0], [0], 1, 1, 8, 8, 16, "bf16", False, "nhd"),
    ([15, 16, 0, 31], [0, 3, 7, 1], 8, 2, 128, 128, 16, "bf16", False, "nhd"),
    ([100, 5, 63], [5, 0, 2], 6, 3, 64, 64, 64, "f16", True, "hnd"),
    ([7, 1000], [1, 4], 4, 4, 96, 48, 32, "bf16", False, "hnd"),
    ([7, 1000], [1, 4], 5, 1, 80, 40, 32, "f16", False, "nhd"),
    ([3, 9], [4, 2], 4, 2, 72, 20, 16, "bf16", True, "nhd"),
    ([3, 9], [4, 2], 4, 2, 128, 2, 16, "bf16", False, "nhd"),
    ([0, 0], [300, 77], 12, 4, 128, 64, 128, "bf16", True, "nhd"),
    ([50] * 300, [7] * 300, 4, 1, 64, 64, 256, "bf16", False, "nhd"),
    ([1 << 20, 131071], [2, 2], 8, 8, 128, 128, 4096, "bf16", False, "nhd"),
]


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_against_the_definition(case, fused):
    lens, gam, Hq, Hk, D, rot, page, dt, inter, layout = case
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16}[dt]
    if max(lens) > 100000:  # only the pages of the step exist
        table_w = max(lens) // page + 2
        q, k, v, cu, cache, _ = setup([n % page for n in lens], gam, Hq, Hk, D, page, dtype, 3, layout, fused)
        small = cache.page_table.cpu()
        table = torch.full((len(lens), table_w), -5, dtype=torch.int32)
        for b, n in enumerate(lens):
            w = min(small.shape[1], table_w - n // page)
            table[b, n // page:n // page + w] = small[b, :w]
        cache = binding.PagedCache(cache.k_pages, cache.v_pages, table.cuda(),
                                   torch.tensor(lens, dtype=torch.int32).cuda())
    else:
        q, k, v, cu, cache, table = setup(lens, gam, Hq, Hk, D, page, dtype, 3, layout, fused)
    freq = rope.frequencies(rot, 10000.0)
    want = expect(q, k, v, cu, cache, table, lens, gam, freq, inter)
    q_out = torch.full(q.shape, 9.0, dtype=dtype, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    binding.spec_verify_kv_append(q, k, v, cache, cu, max(gam), rope.fixed_point(freq).cuda(), q_out, ws,
                                  interleaved=inter)
    assert binding.spec_verify_status(ws) == 0
    check(q_out, want[0], float(q.abs().max()), dtype)
    check(cache.k_pages, want[1], float(k.abs().max()), dtype)
    assert torch.equal(cache.v_pages.double(), want[2])


@pytest.mark.parametrize("rows", [608, 609, 1217, 2047, 2048, 2049])
@pytest.mark.parametrize("D, rot, inter", [(128, 128, False), (64, 32, True), (72, 20, False)])
def test_around_the_borders_of_the_forms(rows, D, rot, inter):
    # one long request among short ones, so that the last rows' requests differ
    lens, gam = [5] * 25 + [70] + [31] * 25, [3] * 25 + [rows - 201] + [3] * 25
    q, k, v, cu, cache, table = setup(lens, gam, 5, 1, D, 32, torch.bfloat16, 9)
    assert q.shape[0] == rows
    freq = rope.frequencies(rot, 10000.0)
    want = expect(q, k, v, cu, cache, table, lens, gam, freq, inter)
    q_out = torch.full(q.shape, 9.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    binding.spec_verify_kv_append(q, k, v, cache, cu, max(gam), rope.fixed_point(freq).cuda(), q_out, ws,
                                  interleaved=inter)
    assert binding.spec_verify_status(ws) == 0
    check(q_out, want[0], float(q.abs().max()), torch.bfloat16)
    check(cache.k_pages, want[1], float(k.abs().max()), torch.bfloat16)
    assert torch.equal(cache.v_pages.double(), want[2])


@pytest.mark.parametrize("inter", [False, True])
def test_unaligned_inputs_take_the_pair_path(inter):
    """q and k views that start 2 bytes off a 16-byte boundary."""
    lens, gam, Hq, Hk, D, page, dtype = [5, 30], [2, 3], 4, 2, 64, 16, torch.bfloat16
    q, k, v, cu, cache, table = setup(lens, gam, Hq, Hk, D, page, dtype, 4)
    T = q.shape[0]

    def off(x, by):
        flat = torch.empty(x.numel() + by, dtype=dtype, device="cuda")
        y = flat[by:].view(x.shape)
        y.copy_(x)
        return y
    q, k, v = off(q, 1), off(k, 3), off(v, 1)
    freq = rope.frequencies(48)
    want = expect(q, k, v, cu, cache, table, lens, gam, freq, inter)
    q_out = torch.empty((T, Hq, D), dtype=dtype, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    binding.spec_verify_kv_append(q, k, v, cache, cu, 3, rope.fixed_point(freq).cuda(), q_out, ws, interleaved=inter)
    check(q_out, want[0], float(q.abs().max()), dtype)
    check(cache.k_pages, want[1], float(k.abs().max()), dtype)
    assert torch.equal(cache.v_pages.double(), want[2])


def test_positions_offset_scale_in_place_and_no_rotation():
    lens, gam, dtype = [20, 3], [3, 5], torch.bfloat16
    q, k, v, cu, cache, table = setup(lens, gam, 4, 2, 64, 16, dtype, 5)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    freq = rope.frequencies(64, scaling="by_parts", factor=4.0, trained_len=2048)
    fx = rope.fixed_point(freq).cuda()
    scale = rope.by_parts_scale(4.0)
    pos = torch.tensor([23, 24, 24, 25, 5, 6, 7, 7, 8, 9], dtype=torch.int32)
    want = expect(q, k, v, cu, cache, table, lens, gam, freq, False, scale=scale, positions=pos)
    mine = q.contiguous().clone()
    binding.spec_verify_kv_append(mine, k, v, cache, cu, 5, fx, mine, ws, rope_scale=scale, positions=pos.cuda())
    check(mine, want[0], float(q.abs().max()), dtype, scale)
    check(cache.k_pages, want[1], float(k.abs().max()), dtype, scale)
    want = expect(q, k, v, cu, cache, table, lens, gam, freq, True, offset=777)
    binding.spec_verify_kv_append(None, k, v, cache, cu, 5, fx, None, ws, interleaved=True, position_offset=777)
    check(cache.k_pages, want[1], float(k.abs().max()), dtype)
    want = expect(q, k, v, cu, cache, table, lens, gam, None, False)
    out = torch.empty_like(mine)
    binding.spec_verify_kv_append(q, k, v, cache, cu, 5, None, out, ws)
    assert torch.equal(out, q) and torch.equal(cache.k_pages.double(), want[1])
    assert binding.spec_verify_status(ws) == 0


def test_bad_pages_lengths_and_prefixes_write_nothing_else():
    S = {n: b for b, n in binding.STATUS_BITS.items()}
    lens, gam, dtype = [20, 3, 40], [3, 5, 1], torch.bfloat16
    freq = rope.frequencies(64)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def go(change, status, kept):
        q, k, v, cu, cache, table = setup(lens, gam, 4, 2, 64, 16, dtype, 6)
        before = cache.k_pages.clone(), cache.v_pages.clone()
        want = expect(q, k, v, cu, cache, table, lens, gam, freq, False)
        change(cache, cu)
        out = torch.full((q.shape[0], 4, 64), 9.0, dtype=dtype, device="cuda")
        binding.spec_verify_kv_append(q, k, v, cache, cu, 5, rope.fixed_point(freq).cuda(), out, ws)
        assert binding.spec_verify_status(ws) == status
        for b in range(3):
            ids = table[b][table[b] >= 0].long().cuda()
            if b in kept:
                check(cache.k_pages[ids], want[1][ids], float(k.abs().max()), dtype)
            else:
                assert torch.equal(cache.k_pages[ids], before[0][ids])
                assert torch.equal(cache.v_pages[ids], before[1][ids])
        return out

    def bad_page(cache, cu):
        cache.page_table[1, 0] = 10 ** 6
        cache.page_table[0, 1] = -1
    out = go(bad_page, S["BAD_PAGE"], [2])
    assert not (out == 9.0).all(-1).any()  # queries are rotated all the same

    def bad_len(cache, cu):
        cache.kv_len[0] = -4
        cache.kv_len[2] = 10 ** 6
    go(bad_len, S["BAD_LENGTH"], [1])

    def bad_cu(cache, cu):
        cu[1] = 100
    go(bad_cu, S["BAD_GAMMA"], [2])


def test_graph_replay_at_another_length():
    lens, gam, dtype = [20, 3], [3, 5], torch.float16
    q, k, v, cu, cache, table = setup([60, 60], gam, 4, 2, 64, 16, dtype, 8)
    cache.kv_len.copy_(torch.tensor(lens))
    freq = rope.frequencies(64)
    fx = rope.fixed_point(freq).cuda()
    out = torch.empty((q.shape[0], 4, 64), dtype=dtype, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    binding.spec_verify_kv_append(q, k, v, cache, cu, 5, fx, out, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.spec_verify_kv_append(q, k, v, cache, cu, 5, fx, out, ws)
    cache.commit(torch.tensor([2, 0], dtype=torch.int32, device="cuda"))
    lens = [23, 4]
    assert cache.kv_len.tolist() == lens
    want = expect(q, k, v, cu, cache, table, lens, gam, freq, False)
    graph.replay()
    torch.cuda.synchronize()
    check(out, want[0], float(q.abs().max()), dtype)
    check(cache.k_pages, want[1], float(k.abs().max()), dtype)


def test_refused_tensors():
    lens, gam, dtype = [20, 3], [3, 5], torch.bfloat16
    q, k, v, cu, cache, _ = setup(lens, gam, 4, 2, 64, 16, dtype, 9)
    fx = rope.fixed_point(rope.frequencies(64)).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = torch.empty((10, 4, 64), dtype=dtype, device="cuda")
    call = binding.spec_verify_kv_append
    for args in ((q.half(), k, v, cache, cu, 5, fx, out, ws), (q, k, v, cache, cu.long(), 5, fx, out, ws),
                 (q, k, v, cache, cu, 5, fx.int(), out, ws), (q, k.cpu(), v, cache, cu, 5, fx, out, ws)):
        with pytest.raises(TypeError):
            call(*args)
    for args in ((q, k[:, :1], v, cache, cu, 5, fx, out, ws), (q, k, v, cache, cu, 5, fx, None, ws),
                 (q, k, v, cache, cu, 5, fx, out[:1].expand(10, 4, 64), ws), (q, k, v, cache, cu[:2], 5, fx, out, ws),
                 (q[:1], k[:1], v[:1], cache, cu, 5, fx, out[:1], ws)):
        with pytest.raises(ValueError):
            call(*args)
    with pytest.raises(binding.SpecVerifyError):
        call(q, k, v, cache, cu, -1, fx, out, ws)
    pool = torch.zeros((4, 16, 2, 64), dtype=dtype, device="cuda")
    table, n = torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in ((pool[:, :15], pool[:, :15], table, n), (pool, pool[:2], table, n), (pool, pool, table[:1], n),
                (pool, pool, table.long(), n), (pool[:1].expand(4, 16, 2, 64), pool, table, n),
                (pool[..., :60], pool[..., :60], table, n)):
        with pytest.raises((ValueError, TypeError)):
            binding.PagedCache(*bad)
    with pytest.raises(TypeError):
        binding.PagedCache(pool.float(), pool.float(), table, n)


@pytest.mark.parametrize("lens, gam", [([20, 3], [3, 5]), ([17], [0])])
def test_queries_turned_in_place_beside_their_keys_and_values(lens, gam):
    """q, k, v and q_out are slices of one projection's rows."""
    freq = rope.frequencies(64)
    fx, ws = rope.fixed_point(freq).cuda(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    for place in ("q", "beside", "heads"):
        q, k, v, cu, cache, table = setup(lens, gam, 4, 2, 64, 16, torch.bfloat16, 12)
        T = q.shape[0]
        wide = torch.cat([q, k, v, torch.full_like(q, 9.0)], 1)
        if place == "heads":  # stored [head, row, value]
            wide = wide.transpose(0, 1).contiguous().transpose(0, 1)
        before = wide.clone()
        q, k, v = wide[:, :4], wide[:, 4:6], wide[:, 6:8]
        out = q if place == "q" else wide[:, 8:]
        want = expect(before[:, :4], before[:, 4:6], before[:, 6:8], cu, cache, table, lens, gam, freq, False)
        binding.spec_verify_kv_append(q, k, v, cache, cu, max(gam), fx, out, ws)
        check(out, want[0], float(q.abs().max()), torch.bfloat16)
        check(cache.k_pages, want[1], float(k.abs().max()), torch.bfloat16)
        assert torch.equal(cache.v_pages.double(), want[2])
        keep = slice(4, 8) if place == "q" else slice(0, 8)
        assert torch.equal(wide[:, keep], before[:, keep]) and binding.spec_verify_status(ws) == 0
        # a slice that reaches into the keys, or the queries one head on
        for bad in ([wide[:, 2:6], wide[:, 5:9], wide[:, 1:5]] if T > 1 else [wide[:, 2:6], wide[:, 1:5]]):
            with pytest.raises(binding.SpecVerifyError) as e:
                binding.spec_verify_kv_append(q, k, v, cache, cu, max(gam), fx, bad, ws)
            assert e.value.code == -3
        twice = torch.zeros((T + 3) * 64, dtype=torch.bfloat16, device="cuda").as_strided((T, 4, 64), (64, 64, 1))
        if T > 1:
            with pytest.raises(ValueError):
                binding.spec_verify_kv_append(q, k, v, cache, cu, max(gam), fx, twice, ws)
