"""Attention over a cache of e4m3 codes against the definition in 64 bits, within the error that
its roundings allow; codes and scales that no row sees are NaN."""
import math

import pytest
import torch

from cache8_refs import values
from operator_refs import attend
from speculative_decoding_verification_62_gb300 import binding

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
S = {n: b for b, n in binding.STATUS_BITS.items()}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def tolerance(q, k, o, lse, spread, size, weight, scale, lv, dtype):
    """Allowed errors of o and lse.

    A score is a sum of up to 3 D products of 8-bit floats in 32 bits, each addition off by at
    most 2^-24 of the sum of magnitudes, and three more roundings (the keys' scale, the row's
    factor, the maximum): |ds| <= (3 D + 3) 2^-24 size.  A query enters with an error of
    2^-21 of its row's largest: 2^-21 max|q| sum|k| scale more.  The logarithm of the
    values' scale (lv at most) is good to 2^-23 of itself and added with the score: 2^-22 lv.
    ex2.approx is good to 2^-22, running sums to 2^-18: d = |ds| + 2^-17 relative in all.
    A weight is then rounded as fp16 and by 2^-9 of itself (2^-9 1.13), or by 2^-30 of its row's
    largest: `weight` is the sum of the values' magnitudes times that largest, over the
    row's sum.  The output is rounded once more."""
    u, D = torch.finfo(dtype).eps / 2, q.shape[-1]
    r = q.shape[1] // k.shape[1]
    rows = k.abs().sum(-1).amax(0) if k.shape[0] else torch.zeros(k.shape[1], dtype=q.dtype, device=q.device)
    dq = 2.0 ** -21 * q.abs().amax(-1) * rows.repeat_interleave(r)[None, :] * scale
    d = (3 * D + 3) * 2.0 ** -24 * size + dq + 2.0 ** -22 * lv + 2.0 ** -17
    tol = (2.0 ** -9 * 1.13 + 2 * d[..., None]) * 1.01 * spread + 2.0 ** -30 * weight + u * 1.01 * o.abs() + 1e-30
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    return tol, d + 2.0 ** -22 * (1.0 + lse.abs())


class Batch:
    def __init__(self, lens, gam, Hq, Hk, D, page, block, dtype, prefix=0, layout="nhd", seed=1, scale_q=1.5,
                 spread=3, powers=True, spare=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        gc = torch.Generator().manual_seed(seed)
        self.lens, self.gam, self.Hq, self.Hk, self.D, self.page, self.prefix = lens, gam, Hq, Hk, D, page, prefix
        self.dtype, self.block = DT[dtype], block
        B = len(lens)
        need = [-(-(n + x + 1) // page) for n, x in zip(lens, gam)]
        pre = -(-prefix // page)
        total = sum(need) + pre + spare
        perm = torch.randperm(total, generator=gc).int()
        table = torch.full((B, max(need) + 1), -9, dtype=torch.int32)
        shape = (total, page, Hk, D) if layout == "nhd" else (total, Hk, page, D)
        pools = [torch.full(shape, 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2)]
        if layout == "hnd":
            pools = [p.transpose(1, 2) for p in pools]
        self.bytes = pools
        self.scales = [torch.full((total, page // block, Hk), math.nan, device="cuda") for _ in range(2)]
        self.lv = 0.0

        def fill(ids, n):
            """n tokens: codes of normal values near the middle of e4m3's range, scales from block to block."""
            out = []
            t = torch.arange(n, device="cuda")
            where = ids.long().cuda()[t // page]
            for kind in range(2):
                codes = ((torch.randn((n, Hk, D), generator=g, device="cuda") + 0.25 * kind) * 64.0).clamp(-448, 448)
                codes = codes.to(torch.float8_e4m3fn).view(torch.uint8)
                blocks = -(-n // block)
                s = torch.exp2(torch.randint(-spread, spread + 1, (blocks, Hk), generator=g, device="cuda").float() - 6.0)
                if not powers:
                    s = s * (1.0 + torch.rand(s.shape, generator=g, device="cuda"))
                self.lv = max(self.lv, float(s.log2().abs().max()))
                pools[kind][where, t % page] = codes
                first = torch.arange(blocks, device="cuda") * block
                self.scales[kind][ids.long().cuda()[first // page], first % page // block] = s
                out.append(values(codes) * s.double()[t // block][..., None])
            return out
        self.prefix_table = perm[:pre].cuda()
        self.pk, self.pv = fill(perm[:pre], prefix) if prefix else (None, None)
        at, self.k, self.v = pre, [], []
        for b in range(B):
            ids = perm[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = ids
            k, v = fill(ids, lens[b] + gam[b] + 1)
            self.k.append(k)
            self.v.append(v)
        self.T = sum(gam) + B
        self.q = (torch.randn((self.T, Hq, D), generator=g, device="cuda") * scale_q).to(self.dtype)
        self.cu = ints([0] + torch.tensor(gam).cumsum(0).tolist())
        self.cache = binding.PagedCache(*(p.view(torch.float8_e4m3fn) for p in pools), table.cuda(), ints(lens),
                                        k_scales=self.scales[0], v_scales=self.scales[1])

    def run(self, mask=None, lse=True, scale=None, ws=None, out=None, status=0):
        if ws is None:
            ws = binding.make_attention_e4m3_workspace(self.T, self.Hq, self.D)
        if out is None:
            out = torch.full((self.T, self.Hq, self.D), 77.0, dtype=self.dtype, device="cuda")
        l = torch.full((self.T, self.Hq), 77.0, device="cuda") if lse else None
        binding.spec_verify_attention_e4m3(self.q, self.cache, self.cu, max(self.gam), out, ws,
                                           prefix_table=self.prefix_table, prefix_len=self.prefix, scale=scale,
                                           draft_mask=mask, lse=l)
        if status is not None:
            assert binding.spec_verify_status(ws) == status
        return out, l

    def check(self, out, lse, mask=None, scale=None, only=None):
        scale = self.D ** -0.5 if scale is None else scale
        row, worst = 0, 0.0
        for b, (n, x) in enumerate(zip(self.lens, self.gam)):
            rows = slice(row, row + x + 1)
            row += x + 1
            if only is not None and b not in only:
                continue
            k, v = self.k[b], self.v[b]
            i, j = torch.arange(x + 1, device="cuda")[:, None], torch.arange(n + x + 1, device="cuda")[None, :]
            if mask is None:
                seen = j <= n + i
            else:
                word = mask[rows].long()[:, None]
                seen = (j < n) | (((word >> (j - n).clamp_min(0)) & 1) == 1)
            if self.prefix:
                k, v = torch.cat([self.pk, k]), torch.cat([self.pv, v])
                seen = torch.cat([torch.ones((x + 1, self.prefix), dtype=torch.bool, device="cuda"), seen], 1)
            q = self.q[rows].double()
            o, l, spread, size = attend(q, k, v, seen, scale)
            # each weight is off by 2^-30 of the row's largest weight times scale: over all keys at most
            # keys 2^-30 448 max(w vs) / sum(w), with w <= sum(w)
            weight = k.shape[0] * 448.0 * float(max(s[~torch.isnan(s)].max() for s in self.scales[1:]))
            tol, tl = tolerance(q, k, o, l, spread, size, weight, scale, self.lv, self.dtype)
            err = (out[rows].double() - o).abs()
            assert not (err > tol).any() and not torch.isnan(err).any(), (
                b, int((~(err <= tol)).sum()), float((err / tol).max()))
            worst = max(worst, float((err / tol).max()))
            if lse is not None:
                g = lse[rows].double()
                empty = torch.isinf(l)
                assert torch.equal(g[empty], l[empty])
                assert not ((g - l).abs()[~empty] > tl[~empty]).any()
        return worst


CASES = {
    # lens, gamma, Hq, Hk, D, page, block, dtype, prefix, layout
    "one_token": ([0], [0], 1, 1, 64, 16, 16, "bf16", 0, "nhd"),
    "one_tile": ([100], [3], 8, 2, 128, 16, 16, "bf16", 0, "nhd"),
    "one_tile_f16": ([100], [3], 8, 2, 128, 16, 16, "f16", 0, "nhd"),
    "two_tiles_32_columns": ([200], [3], 8, 1, 128, 32, 16, "bf16", 0, "nhd"),
    "two_tiles_64_columns": ([200], [7], 8, 1, 128, 32, 16, "bf16", 0, "nhd"),
    "two_tiles_48_columns_f16": ([200], [5], 8, 1, 128, 32, 16, "f16", 0, "nhd"),
    "tile_borders": ([127, 128, 124, 255, 0, 1, 96, 95], [0, 0, 3, 1, 5, 7, 0, 0], 4, 1, 128, 32, 1, "bf16", 0, "nhd"),
    "mha_f16": ([30, 500, 77], [2, 0, 4], 6, 6, 64, 16, 16, "f16", 0, "hnd"),
    "odd_dim_80": ([300, 11], [4, 1], 10, 2, 80, 64, 32, "f16", 0, "nhd"),
    "dim_16": ([300, 11], [4, 1], 4, 2, 16, 64, 2, "bf16", 0, "nhd"),
    "dim_48_group_3": ([130, 400], [6, 2], 9, 3, 48, 32, 4, "bf16", 0, "hnd"),
    "group_7": ([700, 3, 260], [5, 7, 0], 14, 2, 128, 128, 128, "bf16", 0, "nhd"),
    "group_128": ([200, 40], [1, 3], 128, 1, 64, 16, 16, "bf16", 0, "nhd"),
    "group_200": ([200, 40], [1, 3], 200, 1, 112, 16, 8, "f16", 0, "nhd"),
    "big_pages": ([1000, 20, 300], [3, 3, 3], 8, 2, 128, 512, 64, "bf16", 0, "hnd"),
    "split_long": ([40000], [3], 8, 1, 128, 64, 64, "bf16", 0, "nhd"),
    "split_long_f16_64": ([19001, 17], [7, 2], 16, 2, 64, 16, 16, "f16", 0, "nhd"),
    "many": ([(37 * b) % 400 for b in range(330)], [b % 4 for b in range(330)], 4, 2, 64, 16, 16, "bf16", 0, "nhd"),
    "more_requests_than_threads": ([(53 * b) % 300 for b in range(700)], [b % 3 for b in range(700)], 2, 1, 64, 32, 32,
                                   "f16", 0, "nhd"),
    "more_requests_and_a_prefix": ([(53 * b) % 90 for b in range(401)], [b % 5 for b in range(401)], 8, 2, 128, 16, 16,
                                   "bf16", 200, "nhd"),
    "long_among_short": ([30, 9000, 5, 0, 77], [1, 2, 0, 3, 4], 4, 4, 128, 64, 16, "f16", 0, "nhd"),
    "prompt": ([0, 64], [399, 150], 4, 2, 128, 16, 16, "bf16", 0, "nhd"),
    "prompt_group_3": ([5], [600], 3, 1, 64, 32, 32, "f16", 0, "nhd"),
    "prefix_1": ([40, 0, 9], [2, 3, 0], 8, 2, 128, 16, 16, "bf16", 1, "nhd"),
    "prefix_small_batch": ([40, 0, 9], [2, 3, 0], 8, 2, 128, 16, 16, "bf16", 300, "nhd"),
    "prefix_blocks": ([b * 9 for b in range(40)], [b % 6 for b in range(40)], 8, 1, 128, 16, 16, "bf16", 1000, "hnd"),
    "prefix_f16": ([b * 3 for b in range(70)], [3] * 70, 4, 2, 64, 32, 16, "f16", 2051, "nhd"),
    "prefix_many_heads": ([b * 30 for b in range(30)], [4] * 30, 32, 8, 128, 64, 64, "bf16", 4096, "nhd"),
    "prefix_group_5": ([b * 30 for b in range(30)], [b % 5 for b in range(30)], 20, 4, 96, 128, 32, "bf16", 1500, "nhd"),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_definition(name):
    lens, gam, Hq, Hk, D, page, block, dt, prefix, layout = CASES[name]
    w = Batch(lens, gam, Hq, Hk, D, page, block, dt, prefix, layout)
    out, lse = w.run()
    worst = w.check(out, lse)
    print(name, "worst error over tolerance", worst)
    again, lse2 = w.run()
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # bit for bit
