"""The operators together, as a serving step runs them: append with rotation, attention
over the shared prefix and the paged cache, verification from probabilities, rollback by
length.  A one-layer stand-in for the target is recomputed from each request's whole
token history in 64 bits at every step."""
import numpy as np
import pytest
import torch

from operator_refs import attend, probs_request, rotate, tolerance
from speculative_decoding_verification_62_gb300 import binding, rope

pytestmark = pytest.mark.gpu


def test_a_cache_keeps_its_tensors():
    pools = [torch.zeros((2, 16, 1, 8), dtype=torch.float16, device="cuda") for _ in range(2)]
    table, lens = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((3, 2), (3,)))
    cache = binding.PagedCache(*pools, table, lens)
    # the calls hold the addresses: another tensor takes another PagedCache
    for name, t in (("k_pages", pools[1]), ("v_pages", pools[0]), ("page_table", table + 1), ("kv_len", lens + 1)):
        with pytest.raises(AttributeError):
            setattr(cache, name, t)
    cache.commit(torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"))
    assert cache.kv_len is lens and lens.tolist() == [1, 2, 3]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("prefix", [0, 75])
def test_steps_against_the_whole_history(prefix, dtype):
    g = torch.Generator().manual_seed(17)
    V, Hq, Hk, D, page, B, G, steps = 211, 8, 2, 64, 16, 5, 4, 5
    eq, ek, ev = (torch.randn((V, h, D), generator=g).to(dtype).cuda() for h in (Hq, Hk, Hk))
    head = (torch.randn((Hq * D, V), generator=g) * 0.2).cuda()
    freq = rope.frequencies(D)
    fx = rope.fixed_point(freq).cuda()
    # page table: enough for every step; the prefix has pages of its own
    width = -(-(20 + steps * (G + 1) + 1) // page)
    pre = -(-prefix // page)
    pool = B * width + pre
    perm = torch.randperm(pool, generator=g).int()
    kp = torch.full((pool, page, Hk, D), float("nan"), dtype=dtype, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    cache = binding.PagedCache(kp, vp, perm[pre:].view(B, width).contiguous().cuda(),
                               torch.zeros(B, dtype=torch.int32).cuda())
    ptab = perm[:pre].cuda()
    ws = binding.make_attention_workspace(B * 21 + prefix, Hq, D)
    shared = torch.randint(0, V, (prefix,), generator=g).tolist()
    if prefix:  # the prefix enters as a request of its own
        t = torch.tensor(shared).cuda()
        one = binding.PagedCache(kp, vp, ptab[None].contiguous(), torch.zeros(1, dtype=torch.int32).cuda())
        binding.spec_verify_kv_append(None, ek[t], ev[t], one, torch.tensor([0, prefix - 1], dtype=torch.int32).cuda(),
                                      prefix - 1, fx, None, ws)
    # prompts of 1 to 20 tokens; the last token stays outside the cache
    history = [torch.randint(0, V, (4 * b + 2,), generator=g).tolist() for b in range(B)]
    first = [len(h) - 1 for h in history]
    t = torch.tensor([x for h in history for x in h[:-1]]).cuda()
    cu = torch.tensor([0] + [sum(n - 1 for n in first[:b + 1]) for b in range(B)], dtype=torch.int32).cuda()
    binding.spec_verify_kv_append(None, ek[t], ev[t], cache, cu, max(first) - 1, fx, None, ws, position_offset=prefix)
    cache.commit(torch.tensor([n - 1 for n in first], dtype=torch.int32).cuda())
    total_accepted = 0
    for step in range(steps):
        gam = torch.randint(0, G + 1, (B,), generator=g).tolist()
        q_rows, drafts = [], []
        for b in range(B):
            q = torch.softmax(torch.randn((gam[b], V), generator=g) * 1.5, -1)
            q_rows.append(q)
            drafts.append(torch.multinomial(q, 1, generator=g)[:, 0].tolist() if gam[b] else [])
        cu = torch.tensor(np.concatenate([[0], np.cumsum(gam)]).astype(np.int32)).cuda()
        tok = torch.tensor([x for b in range(B) for x in [history[b][-1]] + drafts[b]]).cuda()
        T = tok.numel()
        q_out = torch.empty((T, Hq, D), dtype=dtype, device="cuda")
        out = torch.empty_like(q_out)
        binding.spec_verify_kv_append(eq[tok], ek[tok], ev[tok], cache, cu, G, fx, q_out, ws, position_offset=prefix)
        binding.spec_verify_attention(q_out, cache, cu, G, out, ws, prefix_table=ptab, prefix_len=prefix)
        # the drafts' distributions lean on the target's, so that some are accepted
        logits = out.flatten(1).float() @ head
        p = torch.softmax(logits, -1)
        qd = torch.cat(q_rows).cuda()
        rows = torch.cat([torch.arange(n) + int(cu[b]) + b for b, n in enumerate(gam)]).long().cuda()
        qd = 0.5 * qd + 0.5 * p[rows]
        u = torch.rand((T,), generator=g)
        v = binding.Verifier(B, G, V)
        dt = torch.tensor([x for d in drafts for x in d], dtype=torch.int32).cuda()
        tokens, acc = v.sample_probs_packed(p, qd, cu, dt, u.cuda())
        assert binding.spec_verify_status(v.workspace) == 0 and binding.spec_verify_status(ws) == 0
        cache.commit(acc)
        tokens, acc = tokens.cpu().numpy(), acc.cpu().numpy()
        row = 0
        for b in range(B):
            n = gam[b] + 1
            rows = slice(row, row + n)
            d0 = row - b
            row += n
            # attention of this step's rows from the whole history
            seq = torch.tensor(shared + history[b] + drafts[b]).cuda()
            pos = torch.arange(len(seq)).cuda()
            f = freq.cuda()
            k = rotate(ek[seq].double(), pos, f, False)
            qq = rotate(eq[seq[-n:]].double(), pos[-n:], f, False)
            seen = pos[None, :] <= pos[-n:, None]
            o, lse, spread, size = attend(qq, k, ev[seq].double(), seen, D ** -0.5)
            # q and k are rounded to the cache's type: a score moves by (2 eps/2) of its
            # magnitudes, a weight by twice that (numerator and sum)
            eps = torch.finfo(dtype).eps
            tol, _ = tolerance(o, lse, spread, size, len(seq), D, float(ev.double().abs().max()), dtype)
            tol = tol + 2 * torch.expm1(1.01 * eps * size)[..., None] * spread
            assert not ((out[rows].double() - o).abs() > tol).any()
            # the verification from the same probabilities
            pb, qb = p[rows].double().cpu().numpy(), qd[d0:d0 + n - 1].double().cpu().numpy()
            a, z = probs_request(pb, qb, drafts[b], u[rows].numpy(), float(u[rows][-1]))
            assert acc[b] == a and tokens[b].tolist() == drafts[b][:a] + [z] + [-1] * (G - a)
            history[b] += drafts[b][:a] + [z]
            total_accepted += a
        assert cache.kv_len.tolist() == [len(h) - 1 for h in history]
    assert total_accepted > 0


@pytest.mark.parametrize("prefix", [0, 75])
def test_a_captured_step_of_fixed_size_leaves_the_rows_behind_it(prefix):
    """The append, the attention and the verification captured once for 24 rows and replayed
    for steps of fewer: the rows behind the last request (NaN) are neither read into others
    nor written, and no call takes them for an error."""
    B, T, G, Hq, Hk, D, V, page = 4, 24, 8, 8, 2, 64, 50, 16
    dtype, g = torch.bfloat16, torch.Generator().manual_seed(3)
    lens = [20, 0, 33, 7]
    need = [-(-(n + G + 1) // page) for n in lens]
    pre = -(-prefix // page)
    perm = torch.randperm(sum(need) + pre, generator=g).int()
    table, at = torch.full((B, max(need)), -1, dtype=torch.int32), pre
    for b, n in enumerate(need):
        table[b, :n], at = perm[at:at + n], at + n
    pools = [torch.randn((len(perm), page, Hk, D), generator=g).to(dtype).cuda() for _ in range(2)]
    cache = binding.PagedCache(*pools, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    prefix_table = perm[:pre].cuda()
    freq = rope.frequencies(D)
    fx = rope.fixed_point(freq).cuda()
    nan = float("nan")
    qkv = torch.full((T, Hq + 2 * Hk, D), nan, dtype=dtype, device="cuda")
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    p = torch.full((T, V), nan, device="cuda")
    tok, u = torch.full((T - B,), -9, dtype=torch.int32, device="cuda"), torch.full((T,), nan, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    ws, ver = binding.make_attention_workspace(T, Hq, D), binding.Verifier(B, G, V)
    q_rot, out, lse = torch.empty_like(q), torch.empty((T, Hq, D), dtype=dtype, device="cuda"), torch.empty((T, Hq), device="cuda")
    q_rot = q_rot.contiguous()

    def step():
        binding.spec_verify_kv_append(q, k, v, cache, cu, G, fx, q_rot, ws, position_offset=prefix)
        binding.spec_verify_attention(q_rot, cache, cu, G, out, ws, prefix_table=prefix_table, prefix_len=prefix, lse=lse)
        ver.sample_probs_packed(p, None, cu, tok, u)

    def load(gam):
        n = sum(gam) + B
        qkv.fill_(nan), p.fill_(nan), tok.fill_(-9), u.fill_(nan)
        qkv[:n] = torch.randn((n, Hq + 2 * Hk, D), generator=g).to(dtype)
        p[:n] = torch.softmax(torch.randn((n, V), generator=g), -1)
        tok[:n - B] = torch.randint(0, V, (n - B,), generator=g, dtype=torch.int32)
        u[:n] = torch.rand((n,), generator=g)
        cu.copy_(torch.tensor([0] + list(np.cumsum(gam)), dtype=torch.int32))
        for x in (q_rot, out, lse):
            x.fill_(7.0)
        return n
    load([5, 5, 5, 5])
    step()  # (modules are loaded before the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for gam in ([0, 0, 0, 0], [5, 5, 5, 5], [2, 0, 3, 1], [0, 0, 0, 8], [8, 1, 0, 0]):
        n = load(gam)
        want = rotate(k[:n].double(), torch.cat([torch.arange(x + 1) + m + prefix for x, m in zip(gam, lens)]).cuda(),
                      freq.cuda(), False)
        graph.replay()
        assert binding.spec_verify_status(ws) == 0 and binding.spec_verify_status(ver.workspace) == 0
        for x in (q_rot, out, lse):
            assert bool((x[n:] == 7.0).all()) and not torch.isnan(x[:n]).any()
        tokens, acc = ver.out_tokens.cpu().numpy(), ver.num_accepted.cpu().numpy()
        row = 0
        for b in range(B):
            m = gam[b] + 1
            rows = slice(row, row + m)
            slots = torch.arange(lens[b] + m).cuda()
            ids = table[b].cuda().long()[slots // page]
            keys, vals = (x[ids, slots % page].double() for x in pools)
            assert (keys[lens[b]:] - want[rows]).abs().max() < 2.0 ** -8 * 1.1 * want.abs().max()
            if prefix:
                s = torch.arange(prefix).cuda()
                keys, vals = (torch.cat([x[prefix_table.long()[s // page], s % page].double(), y])
                              for x, y in zip(pools, (keys, vals)))
            seen = torch.arange(len(keys)).cuda()[None] <= prefix + lens[b] + torch.arange(m).cuda()[:, None]
            o, l, spread, size = attend(q_rot[rows].double(), keys, vals, seen, D ** -0.5)
            tol, _ = tolerance(o, l, spread, size, len(keys), D, float(vals.abs().max()), dtype)
            assert not ((out[rows].double() - o).abs() > tol).any()
            a, z = probs_request(p[rows].double().cpu().numpy(), None, tok[row - b:row - b + gam[b]].tolist(),
                                 u[rows].cpu().numpy(), float(u[rows][-1]))
            assert acc[b] == a and tokens[b, a] == z
            row += m
