"""The operators together over a cache in 8 bits whose pages a pool deals out: the page table of a
step (with forks), append, attention over the shared prefix and the cache, verification
from probabilities, rollback by length, compaction."""
import numpy as np
import pytest
import torch

from cache8_refs import values
from operator_refs import attend, probs_request, rotate
from speculative_decoding_verification_62_gb300 import binding, rope
from test_gpu_attention_e4m3_forms import tight

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Loop:
    """A serving loop of B requests over a one-layer stand-in for the target."""

    def __init__(self, dtype, prefix, block, B=6, seed=17):
        self.g = torch.Generator().manual_seed(seed)
        self.V, self.Hq, self.Hk, self.D, self.page, self.block, self.B, self.G = 211, 8, 2, 64, 16, block, B, 4
        self.dtype, self.prefix = dtype, prefix
        self.eq, self.ek, self.ev = (torch.randn((self.V, h, self.D), generator=self.g).to(dtype).cuda()
                                     for h in (self.Hq, self.Hk, self.Hk))
        self.head = (torch.randn((self.Hq * self.D, self.V), generator=self.g) * 0.2).cuda()
        self.freq = rope.frequencies(self.D)
        self.fx = rope.fixed_point(self.freq).cuda()
        width, pre = 8, -(-prefix // self.page)
        n = B * width + pre + 7
        self.bytes = [torch.full((n, self.page, self.Hk, self.D), 0x7f, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.full((n, self.page // block, self.Hk), float("nan"), device="cuda") for _ in range(2)]
        self.pools = [x.view(torch.float8_e4m3fn) for x in self.bytes]
        self.kw = dict(k_scales=self.scales[0], v_scales=self.scales[1])
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.kv_len = ints([0] * B)
        self.cache = binding.PagedCache(*self.pools, self.table, self.kv_len, **self.kw)
        self.ptab = torch.randperm(n, generator=self.g).int()[:pre].cuda()
        self.pool = binding.PagePool.of_table(self.cache, ints([0] * B), self.ptab)
        self.ws = binding.make_attention_e4m3_workspace(B * (self.G + 1), self.Hq, self.D)
        self.shared = torch.randint(0, self.V, (prefix,), generator=self.g).tolist()
        if prefix:  # the prefix enters as a request of its own
            t = torch.tensor(self.shared).cuda()
            one = binding.PagedCache(*self.pools, self.ptab[None].contiguous(), ints([0]), **self.kw)
            binding.spec_verify_kv_append(None, self.ek[t], self.ev[t], one, ints([0, prefix - 1]), prefix - 1, self.fx,
                                          None, self.ws)
        # prompts of 1 to 21 tokens; the last token stays outside the cache
        self.history = [torch.randint(0, self.V, (4 * b + 2,), generator=self.g).tolist() for b in range(B)]
        first = [len(h) - 1 for h in self.history]
        binding.spec_verify_pages_step(self.cache, self.pool, ints(first))
        t = torch.tensor([x for h in self.history for x in h[:-1]]).cuda()
        cu = ints([0] + [sum(n - 1 for n in first[:b + 1]) for b in range(B)])
        binding.spec_verify_kv_append(None, self.ek[t], self.ev[t], self.cache, cu, max(first) - 1, self.fx, None, self.ws,
                                      position_offset=prefix)
        self.cache.commit(ints([n - 1 for n in first]))

    def clear(self):
        assert binding.spec_verify_status(self.ws) == 0 and binding.spec_verify_status(self.pool.workspace) == 0

    def cached(self, table, n):
        """Keys, values and their scales of the first n tokens of a table, as they are held."""
        t = torch.arange(n, device="cuda")
        at = table.long()[t // self.page], t % self.page
        s = [x[at[0], at[1] // self.block].double() for x in self.scales]
        return *(values(x[at]) * y[..., None] for x, y in zip(self.bytes, s)), *s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("prefix, block", [(0, 16), (75, 4)])
def test_steps_with_forks_against_the_whole_history(prefix, block, dtype):
    w = Loop(dtype, prefix, block)
    g, B, G, V, D = w.g, w.B, w.G, w.V, w.D
    f, total = w.freq.cuda(), 0
    for step, parents in enumerate([None, [0, 0, 2, 2, 4, 2], None, [5, 5, 5, 5, 5, 5], [1, 2, 3, 4, 5, 0], None]):
        if parents is not None:
            w.history = [list(w.history[p]) for p in parents]
        gam = torch.randint(0, G + 1, (B,), generator=g).tolist()
        binding.spec_verify_pages_step(w.cache, w.pool, ints([x + 1 for x in gam]), None if parents is None else ints(parents))
        if step % 2:
            remap = torch.empty_like(w.pool.ref)
            binding.spec_verify_pages_compact(w.cache, w.pool, remap)
            w.ptab.copy_(remap[w.ptab.long()])
        w.clear()
        held = -(-(w.kv_len.long() + ints(gam) + 1) // w.page)
        assert w.pool.held.tolist() == held.tolist()
        assert int(w.pool.ref.sum()) == int(held.sum()) + len(w.ptab)
        assert int((w.pool.ref > 0).sum()) + int(w.pool.free_count) == w.pool.ref.numel()
        drafts = [torch.randint(0, V, (x,), generator=g).tolist() for x in gam]
        cu = ints([0] + list(np.cumsum(gam)))
        tok = torch.tensor([x for b in range(B) for x in [w.history[b][-1]] + drafts[b]]).cuda()
        T = tok.numel()
        q_out = torch.empty((T, w.Hq, D), dtype=dtype, device="cuda")
        out, lse = torch.empty_like(q_out), torch.empty((T, w.Hq), device="cuda")
        binding.spec_verify_kv_append(w.eq[tok], w.ek[tok], w.ev[tok], w.cache, cu, G, w.fx, q_out, w.ws, position_offset=prefix)
        binding.spec_verify_attention(q_out, w.cache, cu, G, out, w.ws, prefix_table=w.ptab if prefix else None,
                                      prefix_len=prefix, lse=lse)
        p = torch.softmax(out.flatten(1).float() @ w.head, -1)
        qd = 0.5 * torch.softmax(torch.randn((T - B, V), generator=g), -1).cuda()
        qd += 0.5 * p[torch.cat([torch.arange(n) + int(cu[b]) + b for b, n in enumerate(gam)]).long().cuda()]
        u = torch.rand((T,), generator=g)
        v = binding.Verifier(B, G, V)
        tokens, acc = v.sample_probs_packed(p, qd, cu, ints([x for d in drafts for x in d]), u.cuda())
        w.clear()
        assert binding.spec_verify_status(v.workspace) == 0
        before = w.kv_len.tolist()
        w.cache.commit(acc)
        tokens, acc = tokens.cpu().numpy(), acc.cpu().numpy()
        row = 0
        for b in range(B):
            n = gam[b] + 1
            rows = slice(row, row + n)
            d0 = row - b
            row += n
            assert before[b] == len(w.history[b]) - 1
            # what the cache holds of the whole history: a code is off by 2^-4 of the value, and each
            # rescaling (to twice the scale at least) by half of e4m3's smallest step, 2^-10 of the new scale
            seq = torch.tensor(w.shared + w.history[b] + drafts[b]).cuda()
            pos = torch.arange(len(seq)).cuda()
            own = w.cached(w.table[b], before[b] + n)
            if prefix:
                own = [torch.cat(x) for x in zip(w.cached(w.ptab, prefix), own)]
            for held_, s, x in ((own[0], own[2], rotate(w.ek[seq].double(), pos, f, False)), (own[1], own[3], w.ev[seq].double())):
                tol = 2.0 ** -4 * 1.01 * x.abs() + 2.0 ** -9 * s[..., None] + 2.0 ** -18 * x.abs().amax()
                assert not ((held_ - x).abs() > tol).any()
            # the attention over what is held
            seen = pos[None, :] <= pos[-n:, None]
            o, l, spread, size = attend(q_out[rows].double(), own[0], own[1], seen, D ** -0.5)
            weight = len(seq) * 448.0 * float(own[3].max())
            tol, tl = tight(q_out[rows].double(), own[0], o, l, spread, size, weight, D ** -0.5,
                            float(own[3].log2().abs().max()), dtype)
            assert not ((out[rows].double() - o).abs() > tol).any()
            assert not ((lse[rows].double() - l).abs() > tl).any()
            # the verification from the same probabilities
            pb, qb = p[rows].double().cpu().numpy(), qd[d0:d0 + n - 1].double().cpu().numpy()
            a, z = probs_request(pb, qb, drafts[b], u[rows].numpy(), float(u[rows][-1]))
            assert acc[b] == a and tokens[b].tolist() == drafts[b][:a] + [z] + [-1] * (G - a)
            w.history[b] += drafts[b][:a] + [z]
            total += a
        assert w.kv_len.tolist() == [len(h) - 1 for h in w.history]
    assert total > 0


def test_a_captured_step_repeats_the_eager_one():
    """Page table, append, attention, verification and commit captured once and replayed, beside
    the same calls on a second loop: every tensor equal after each step."""
    a, b = (Loop(torch.bfloat16, 75, 8) for _ in range(2))
    gam = [4, 0, 2, 1, 3, 0]
    T = sum(gam) + a.B

    def buffers(w):
        w.cu, w.tokens = ints([0] + list(np.cumsum(gam))), ints([x + 1 for x in gam])
        w.q, w.k, w.v = (torch.zeros((T, h, w.D), dtype=w.dtype, device="cuda") for h in (w.Hq, w.Hk, w.Hk))
        w.q_out, w.out = torch.empty_like(w.q), torch.empty_like(w.q)
        w.p, w.u = torch.zeros((T, w.V), device="cuda"), torch.zeros((T,), device="cuda")
        w.tok, w.ver = ints([0] * sum(gam)), binding.Verifier(w.B, w.G, w.V)

    def load(w, seed):
        g = torch.Generator().manual_seed(seed)
        for x in (w.q, w.k, w.v):
            x.copy_(torch.randn(x.shape, generator=g) * 2.0 ** (seed % 3))
        w.p.copy_(torch.softmax(torch.randn(w.p.shape, generator=g) * 4.0, -1))
        w.u.copy_(torch.rand(w.u.shape, generator=g))
        w.tok.copy_(w.p[:sum(gam)].argmax(-1))

    def step(w):
        binding.spec_verify_pages_step(w.cache, w.pool, w.tokens)
        binding.spec_verify_kv_append(w.q, w.k, w.v, w.cache, w.cu, w.G, w.fx, w.q_out, w.ws, position_offset=w.prefix)
        binding.spec_verify_attention(w.q_out, w.cache, w.cu, w.G, w.out, w.ws, prefix_table=w.ptab, prefix_len=w.prefix)
        _, acc = w.ver.sample_probs_packed(w.p, None, w.cu, w.tok, w.u)
        w.cache.commit(acc)

    for w in (a, b):
        buffers(w)
        load(w, 0)
        step(w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for seed in range(1, 9):
        for w in (a, b):
            load(w, seed)
        graph.replay()
        step(b)
        for w in (a, b):
            w.clear()
            assert binding.spec_verify_status(w.ver.workspace) == 0
        for x, y in zip((*a.bytes, a.table, a.kv_len, a.q_out, a.out, a.ver.out_tokens, a.pool.held, a.pool.ref,
                         a.pool.free_pages, a.pool.free_count),
                        (*b.bytes, b.table, b.kv_len, b.q_out, b.out, b.ver.out_tokens, b.pool.held, b.pool.ref,
                         b.pool.free_pages, b.pool.free_count)):
            assert torch.equal(x, y)
        for x, y in zip(a.scales, b.scales):
            assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))
        assert torch.isfinite(a.out).all()
    assert min(a.kv_len.tolist()) > 8
