"""Operators of an 8-bit paged cache and of a cache's pages, as cases that can be timed and compared.

* ``append``: a verify step's keys and values go into a paged cache that holds 8-bit
  floats (e4m3) with a scale for each block of tokens and key head; the rotary
  position rotation is applied on the way;
* ``attention``: the step's query rows read that cache, behind a prefix that the batch
  may share;
* ``step``: the page table of the next step: rows continue other rows (forks, beams),
  pages that nobody holds are given back, pages for the next tokens are taken, and a
  partly filled page that several rows hold is copied before it is written;
* ``compact``: the pages in use move to the front of the pool.

``run`` computes them with elementary torch operations where ``own`` is false and
calls the framework's entry points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # Single-token step of one request: latency alone.
        dict(name="append_b1", op="append", B=1, G=0, heads=32, kv_heads=8, D=128, rot=128,
             interleaved=False, page=16, block=16, dtype="bf16", past=2000),
        # A verify step of a full batch: up to eight rows a request in blocks that hold
        # older tokens, part of the head rotated, interleaved pairs.
        dict(name="append_b256", op="append", B=256, G=7, heads=32, kv_heads=8, D=128, rot=64,
             interleaved=True, page=64, block=32, dtype="bf16", past=100000),
        # Prompts of up to 2501 tokens entering the cache, odd lengths, D = 96.
        dict(name="append_prompts_f16", op="append", B=12, G=2500, heads=24, kv_heads=6, D=96,
             rot=96, interleaved=False, page=32, block=16, dtype="f16", past=0),
        # Single-token decoding of one short request: the smallest call.
        dict(name="attn_b1_token", op="attention", B=1, G=0, heads=32, kv_heads=8, D=128, page=16,
             block=16, dtype="bf16", prefix=0, own=600),
        # One request with seven drafts over a long context of its own.
        dict(name="attn_b1_long", op="attention", B=1, G=7, heads=64, kv_heads=8, D=128, page=64,
             block=64, dtype="bf16", prefix=0, own=131000),
        # One key head a query head, D = 64, fp16, odd group of requests.
        dict(name="attn_b37_mha_f16", op="attention", B=37, G=4, heads=12, kv_heads=12, D=64,
             page=16, block=16, dtype="f16", prefix=0, own=3000),
        # An ordinary batch behind a system prompt that ends inside a page.
        dict(name="attn_b32_prefix", op="attention", B=32, G=3, heads=32, kv_heads=8, D=128,
             page=32, block=32, dtype="bf16", prefix=2051, own=1000),
        # The largest: a full batch of long contexts.
        dict(name="attn_b256", op="attention", B=256, G=5, heads=32, kv_heads=8, D=128,
             page=64, block=32, dtype="bf16", prefix=0, own=5000),
        # Two beams of four over a short context: the smallest table.
        dict(name="step_b8", op="step", B=8, width=4, G=3, kv_heads=8, D=128, page=16, block=0,
             dtype="bf16", own=900),
        # A full batch, four continuations of each of 64 contexts, 8-bit pages.
        dict(name="step_b256_e4m3", op="step", B=256, width=4, G=7, kv_heads=8, D=128, page=64,
             block=16, dtype="e4m3", own=20000),
        # A small pool after a few requests have left.
        dict(name="compact_p300", op="compact", B=9, kv_heads=2, D=64, page=16, block=0, dtype="f16",
             pages=300, live=0.5),
        # A pool of gigabytes, 60 % in use.
        dict(name="compact_p6000", op="compact", B=64, kv_heads=8, D=128, page=64, block=0,
             dtype="bf16", pages=6000, live=0.6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], {"bytes": 0.0, "flops": 0.0})
        m["bytes"], m["flops"] = max(m["bytes"], w["bytes"]), max(m["flops"], w["flops"])
    op = rng.choice(["append", "attention", "attention", "step", "compact"])
    while True:
        kv, D, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128]), rng.choice([16, 32, 64, 128])
        block = rng.choice([16, 32, 64, 128])
        block = min(block, page)
        if op == "append":
            prompts = rng.random() < 0.3
            c = dict(op=op, B=_log(rng, 1, 16 if prompts else 256), G=_log(rng, 100, 2500) if prompts else rng.randint(0, 8),
                     heads=kv * rng.choice([1, 2, 4, 5, 8]), kv_heads=kv, D=D, rot=rng.choice([D, D, D // 2]),
                     interleaved=rng.random() < 0.5, page=page, block=block,
                     dtype=rng.choice(["bf16", "bf16", "f16"]), past=0 if prompts else _log(rng, 1, 100000))
        elif op == "attention":
            c = dict(op=op, B=_log(rng, 1, 256), G=rng.randint(0, 8), heads=kv * rng.choice([1, 2, 4, 5, 8]),
                     kv_heads=kv, D=rng.choice([64, 80, 96, 128, 128]), page=page, block=block,
                     dtype=rng.choice(["bf16", "bf16", "f16"]), prefix=rng.choice([0, 0, _log(rng, 50, 4000)]),
                     own=_log(rng, 20, 30000))
        elif op == "step":
            dtype = rng.choice(["bf16", "f16", "e4m3"])
            c = dict(op=op, B=_log(rng, 2, 256), width=rng.choice([1, 2, 3, 4, 8]), G=rng.randint(0, 8), kv_heads=kv, D=D,
                     page=page, block=block if dtype == "e4m3" else 0, dtype=dtype, own=_log(rng, 20, 20000))
        else:
            dtype = rng.choice(["bf16", "f16", "e4m3"])
            c = dict(op=op, B=_log(rng, 1, 64), kv_heads=kv, D=D, page=page, block=block if dtype == "e4m3" else 0,
                     dtype=dtype, pages=_log(rng, 100, 6000), live=round(rng.uniform(0.2, 0.9), 2))
        w = work(c)
        # what the plain form holds in between has to fit beside the inputs
        fits = op != "attention" or c["B"] * c["own"] * c["kv_heads"] * c["D"] <= 1.4e9
        if op == "step":
            fits = c["B"] // c["width"] * c["own"] * c["kv_heads"] * c["D"] <= 1.4e9
        if fits and w["bytes"] <= most[op]["bytes"] and w["flops"] <= most[op]["flops"]:
            return c


def _lengths(case):
    """Draft lengths [B] and tokens already cached [B] of a case: spread over the
    range, from the shape alone, so that work() needs no device."""
    B, G = case["B"], case["G"]
    gam = [(5 * b + 3 * (b // 7) + G) % (G + 1) if B > 1 else G for b in range(B)]
    if case["op"] == "append":
        if G >= 100:  # prompts of odd lengths
            gam = [G - 1 - (b * 977) % max(1, G // 2) if B > 1 else G for b in range(B)]
        past = case["past"]
        return gam, [past - (b * 7919) % (past // 2 + 1) if B > 1 else past for b in range(B)]
    n = case["own"]
    return gam, [max(0, n - (b * 2741) % n) if B > 1 else n for b in range(B)]


def _row(case):
    """Bytes of a token's keys or values in the pool."""
    return case["kv_heads"] * case["D"] * (1 if case["dtype"] == "e4m3" else 2)


def _groups(case):
    """Of a step: the row that each row continues (-1: it ends), tokens cached, tokens to come."""
    B, w = case["B"], case["width"]
    gam, past = _lengths(case)
    parents = [b // w * w for b in range(B)]
    if B >= 8:  # one context ends
        parents = [-1 if p == (B // w // 2) * w else p for p in parents]
    return parents, past, [g + 1 for g in gam]


def work(case):
    if case["op"] == "step":
        parents, past, n = _groups(case)
        ps = case["page"]
        copied = entries = 0
        for b, p in enumerate(parents):
            entries += -(-past[b] // ps) + (-(-(past[p] + n[b]) // ps) if p >= 0 else 0)
            if p >= 0 and p != b:
                copied += past[p] % ps
        return {"bytes": 4.0 * copied * _row(case) + 16.0 * entries + 24.0 * case["B"], "flops": 0.0}
    if case["op"] == "compact":
        used = int(case["pages"] * case["live"])
        moved = used * (1.0 - case["live"])  # used pages that lie behind the first `used` places
        return {"bytes": 4.0 * moved * case["page"] * _row(case) + 8.0 * case["pages"] + 8.0 * used, "flops": 0.0}
    gam, past = _lengths(case)
    T = sum(gam) + case["B"]
    Hq, Hk, D = case["heads"], case["kv_heads"], case["D"]
    if case["op"] == "append":
        blocks = sum(-(-(p % case["block"] + g + 1) // case["block"]) for p, g in zip(past, gam))
        return {"bytes": 2.0 * T * (2 * Hq + 2 * Hk) * D + 2.0 * T * Hk * D + 8.0 * blocks * Hk,
                "flops": 3.0 * T * (Hq + Hk) * case["rot"]}
    P = case["prefix"]
    keys = P + sum(n + g + 1 for n, g in zip(past, gam))
    seen = sum((g + 1) * (P + n) + (g + 1) * (g + 2) // 2 for n, g in zip(past, gam))
    return {"bytes": (2.0 * D + 8.0 / case["block"]) * keys * Hk + 4.0 * T * Hq * D, "flops": 4.0 * seen * Hq * D}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _ints(v):
    return torch.tensor(v, dtype=torch.int32).to(DEV)


def _deal(need, prefix, page, g):
    """A page table with every request's pages (and the prefix's) dealt out in a
    random order, and a few pages that nobody uses."""
    pre = -(-prefix // page)
    total = sum(need) + pre
    perm = torch.randperm(total + 3, generator=g, device=DEV).int()
    table = torch.full((len(need), max(max(need), 1)), -1, dtype=torch.int32)
    flat, at = perm.cpu(), pre
    for b, n in enumerate(need):
        table[b, :n] = flat[at:at + n]
        at += n
    return total + 3, table, perm[:pre].contiguous()


def _pool8(n, page, block, heads, D, g, fill):
    """A pool of e4m3 and its scales: of normal values, whose size varies from block to block."""
    scales = torch.full((n, page // block, heads), 2.0 ** -32, device=DEV)
    pool = torch.zeros((n, page, heads, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    if fill:
        size = torch.randint(-1, 2, scales.shape, generator=g, device=DEV).float()
        scales = torch.exp2(size - 7.0)  # 1 / 2, 1 or 2 in units whose largest values are near 448
        step = max(1, (1 << 28) // (page * heads * D))
        for i in range(0, n, step):
            x = torch.randn((min(step, n - i), page, heads, D), generator=g, device=DEV)
            pool[i:i + step].copy_((x * 96.0).clamp(-448.0, 448.0))
    return pool, scales


def _prepare_cache(case, g, fill):
    gam, past = _lengths(case)
    B, Hk, D, ps = case["B"], case["kv_heads"], case["D"], case["page"]
    cu = [0]
    for x in gam:
        cu.append(cu[-1] + x)
    # only the pages that the step touches exist for an append far into a context
    skip = [(p // ps) * ps if case["op"] == "append" else 0 for p in past]
    n, table, prefix = _deal([-(-(p - k + x + 1) // ps) for p, k, x in zip(past, skip, gam)],
                             case.get("prefix", 0), ps, g)
    if case["op"] == "append":
        wide = max(-(-(p + x + 1) // ps) for p, x in zip(past, gam))
        full = torch.full((B, wide), -1, dtype=torch.int32)
        for b in range(B):
            at = skip[b] // ps
            w = min(table.shape[1], wide - at)
            full[b, at:at + w] = table[b, :w]
        table = full
    k, ks = _pool8(n, ps, case["block"], Hk, D, g, fill)
    v, vs = _pool8(n, ps, case["block"], Hk, D, g, fill)
    s = dict(case=case, B=B, T=cu[-1] + B, G=max(gam), gam=gam, past=past, k_pages=k, v_pages=v, k_scales=ks, v_scales=vs,
             table=table.to(DEV), prefix=prefix, kv_len=_ints(past), cu=_ints(cu),
             req=_ints([b for b, x in enumerate(gam) for _ in range(x + 1)]).long(),
             place=_ints([i for x in gam for i in range(x + 1)]).long())
    if own:
        from speculative_decoding_verification_62_gb300 import binding
        s["cache"] = binding.PagedCache(k, v, s["table"], s["kv_len"], k_scales=ks, v_scales=vs)
        s["workspace"] = binding.make_attention_e4m3_workspace(s["T"], case["heads"], D)
    return s


def _prepare_append(case, g):
    s = _prepare_cache(case, g, case["past"] > 0)
    Hq, Hk, D, dt = case["heads"], case["kv_heads"], case["D"], DTYPES[case["dtype"]]
    # one projection's output holds q, k and v side by side: strided views
    qkv = torch.randn((s["T"], Hq + 2 * Hk, D), generator=g, device=DEV, dtype=dt)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    s["q_out"] = torch.empty((s["T"], Hq, D), device=DEV, dtype=dt)
    half = case["rot"] // 2
    s["inv_freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    if own:
        from speculative_decoding_verification_62_gb300 import rope
        s["freq"] = rope.fixed_point(s["inv_freq"]).to(DEV)
    s["inv_freq"] = s["inv_freq"].to(DEV)
    return s


def _prepare_attention(case, g):
    s = _prepare_cache(case, g, True)
    s["q"] = (torch.randn((s["T"], case["heads"], case["D"]), generator=g, device=DEV) * 2.0).to(DTYPES[case["dtype"]])
    s["out"] = torch.empty_like(s["q"])
    return s


def _state(B, wide, pages):
    """The page bookkeeping as views of one buffer, so that a pass can start from the same state."""
    sizes = [B * wide, B, B, pages, pages, 1]
    sizes = [-(-n // 64) * 64 for n in sizes]
    book = torch.zeros(sum(sizes), dtype=torch.int32, device=DEV)
    t, k, h, r, f, c = torch.split(book, sizes)
    return dict(book=book, table=t[:B * wide].view(B, wide), kv_len=k[:B], held=h[:B], ref=r[:pages],
                free_pages=f[:pages], free_count=c[:1])


def _prepare_pool(case, g, n):
    Hk, D, ps = case["kv_heads"], case["D"], case["page"]
    if case["dtype"] == "e4m3":
        k, ks = _pool8(n, ps, case["block"], Hk, D, g, True)
        v, vs = _pool8(n, ps, case["block"], Hk, D, g, True)
        return dict(k_pages=k, v_pages=v, k_scales=ks, v_scales=vs)
    k, v = (torch.empty((n, ps, Hk, D), device=DEV, dtype=DTYPES[case["dtype"]]).normal_(generator=g) for _ in range(2))
    return dict(k_pages=k, v_pages=v, k_scales=None, v_scales=None)


def _own_pool(s):
    if own:
        from speculative_decoding_verification_62_gb300 import binding
        s["cache"] = binding.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["kv_len"], k_scales=s["k_scales"],
                                        v_scales=s["v_scales"])
        s["pool"] = binding.PagePool(s["cache"], s["held"], s["ref"], s["free_pages"], s["free_count"])
    s["start"] = s["book"].clone()
    return s


def _prepare_step(case, g):
    """Rows of one context share the pages in front of their last few, as after an earlier fork."""
    B, w, ps = case["B"], case["width"], case["page"]
    parents, past, n = _groups(case)
    held = [-(-(p + x) // ps) for p, x in zip(past, n)]
    lead = [b // w * w for b in range(B)]
    shared = [max(0, min(past[l] // ps, past[b] // ps) - 1) if b != l else 0 for b, l in enumerate(lead)]
    most = max(max(held), max(-(-(past[l] + x) // ps) for l, x in zip(lead, n)))
    total = sum(h - x for h, x in zip(held, shared))
    pages = total + 3 * B + 5
    s = dict(case=case, B=B, **_state(B, most, pages), **_prepare_pool(case, g, pages))
    order = torch.randperm(pages, generator=g, device=DEV).int().cpu()
    table, ref, at = torch.full((B, most), -1, dtype=torch.int32), torch.zeros(pages, dtype=torch.int32), 0
    for b in range(B):
        table[b, :shared[b]] = table[lead[b], :shared[b]]
        table[b, shared[b]:held[b]] = order[at:at + held[b] - shared[b]]
        at += held[b] - shared[b]
        ref.index_add_(0, table[b, :held[b]].long(), torch.ones(held[b], dtype=torch.int32))
    s["table"].copy_(table)
    s["kv_len"].copy_(torch.tensor(past, dtype=torch.int32))
    s["held"].copy_(torch.tensor(held, dtype=torch.int32))
    s["ref"].copy_(ref)
    s["free_pages"][:pages - at].copy_(order[at:])
    s["free_count"].fill_(pages - at)
    s["parents"], s["tokens"] = _ints(parents), _ints(n)
    return _own_pool(s)


def _prepare_compact(case, g):
    B, pages = case["B"], case["pages"]
    used = max(1, int(pages * case["live"]))
    share = [used // B + (1 if b < used % B else 0) for b in range(B)]
    s = dict(case=case, B=B, **_state(B, max(share) + 1, pages), **_prepare_pool(case, g, pages))
    order = torch.randperm(pages, generator=g, device=DEV).int()
    flat, at = order.cpu(), 0
    table = torch.full(tuple(s["table"].shape), -1, dtype=torch.int32)
    for b in range(B):
        table[b, :share[b]] = flat[at:at + share[b]]
        at += share[b]
    s["table"].copy_(table)
    s["held"].copy_(torch.tensor(share, dtype=torch.int32))
    s["kv_len"].copy_(s["held"] * case["page"])
    s["ref"][order[:used].long()] = 1
    s["free_pages"][:pages - used].copy_(order[used:])
    s["free_count"].fill_(pages - used)
    s["remap"] = torch.empty((pages,), dtype=torch.int32, device=DEV)
    return _own_pool(s)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return {"append": _prepare_append, "attention": _prepare_attention, "step": _prepare_step,
            "compact": _prepare_compact}[case["op"]](case, g)


# ---------------------------------------------------------------------------
# The passes
# ---------------------------------------------------------------------------
def _rotated(x, cos, sin, rot, interleaved):
    """x [T, H, D] with its first `rot` values of a head turned, in 32 bits, unrounded."""
    y = x.float()
    r = y[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, y[..., rot:]], -1)


def _squares(x, rot, interleaved):
    """[T, H]: the largest square of a value, or of a turning pair's length (products of
    16-bit values are exact in 32, so the sum is rounded once)."""
    y = x.float().square()
    if rot == 0:
        return y.amax(-1)
    r = y[..., :rot]
    pairs = r[..., 0::2] + r[..., 1::2] if interleaved else r[..., :rot // 2] + r[..., rot // 2:]
    return torch.cat([pairs, y[..., rot:]], -1).amax(-1)


def _power(need2):
    """The smallest power of two s, from 2^-32 to 2^56, with need2 <= (448 s)^2 = 0.765625 2^18 s^2."""
    m, x = torch.frexp(need2)
    d = x - 18
    e = torch.where(d % 2 == 0, d // 2 + (m > 0.765625), (d + 1) // 2)
    e = torch.where(need2 > 0, e, -32)
    return torch.ldexp(torch.ones_like(need2), e.clamp(-32, 56))


def _plain_put(s, pool, scales, x, need2, pos):
    """Rows x [T, Hk, D] (32 bits) at positions pos [T] into an 8-bit pool."""
    case = s["case"]
    ps, bt, Hk = case["page"], case["block"], case["kv_heads"]
    per = ps // bt
    flat = scales.view(-1, Hk)
    bytes_ = pool.view(torch.uint8)
    page = s["table"][s["req"], pos // ps].long()
    block = page * per + pos % ps // bt
    need = torch.zeros_like(flat)
    need.scatter_reduce_(0, block[:, None].expand(-1, Hk), need2, "amax")
    # the block that holds a request's next token may hold older ones
    n = s["kv_len"].long()
    first = s["table"].gather(1, (n // ps)[:, None])[:, 0].long()
    at = first * per + n % ps // bt
    older = (n % bt > 0)[:, None]
    new = _power(need)
    was = flat[at]
    now = torch.where(older, torch.maximum(was, new[at]), new[at])
    i = torch.arange(bt, device=DEV)
    token = (n % ps // bt * bt)[:, None] + i
    old = pool.view(torch.uint8)[first[:, None], token].view(torch.float8_e4m3fn)
    moved = (old.float() * (was / now)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = (i[None, :] < (n % bt)[:, None])[:, :, None, None]
    bytes_[first[:, None], token] = torch.where(keep, moved, old.view(torch.uint8))
    new[at] = now
    flat[block] = new[block]
    codes = (x / new[block][:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    bytes_[page, pos % ps] = codes.view(torch.uint8)


def _plain_append(s):
    case = s["case"]
    rot, inter = case["rot"], case["interleaved"]
    pos = s["kv_len"].long()[s["req"]] + s["place"]
    ang = pos.double()[:, None] * s["inv_freq"][None, :]
    cos, sin = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    _plain_put(s, s["k_pages"], s["k_scales"], _rotated(s["k"], cos, sin, rot, inter), _squares(s["k"], rot, inter), pos)
    _plain_put(s, s["v_pages"], s["v_scales"], s["v"].float(), _squares(s["v"], 0, inter), pos)
    s["q_out"].copy_(_rotated(s["q"], cos, sin, rot, inter))
    return s["q_out"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]


def _run_append(s):
    if not own:
        return _plain_append(s)
    from speculative_decoding_verification_62_gb300 import binding
    binding.spec_verify_kv_append_e4m3(s["q"], s["k"], s["v"], s["cache"], s["cu"], s["G"], s["freq"], s["q_out"],
                                       s["workspace"], interleaved=s["case"]["interleaved"])
    return s["q_out"], s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]


def _values(s, pool, scales, pages):
    """[.., page, Hk, D] of the pages, in 32 bits."""
    x = pool.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
    return x.mul_(scales[pages].repeat_interleave(s["case"]["block"], -2)[..., None])


def _plain_attention(s):
    case = s["case"]
    B, T, ps, P = s["B"], s["T"], case["page"], case["prefix"]
    Hq, Hk, D = case["heads"], case["kv_heads"], case["D"]
    r = Hq // Hk
    N = s["G"] + 1
    table = s["table"].long().clamp_min(0)
    L = table.shape[1] * ps
    # the requests' own keys, padded to the longest
    k = _values(s, s["k_pages"], s["k_scales"], table).reshape(B, L, Hk, D)
    v = _values(s, s["v_pages"], s["v_scales"], table).reshape(B, L, Hk, D)
    q = torch.zeros((B, N, Hk, r, D), device=DEV)
    q[s["req"], s["place"]] = s["q"].float().view(T, Hk, r, D) * (1.0 / math.sqrt(D))
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hk, N * r, D)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1))
    key = torch.arange(L, device=DEV)
    limit = s["kv_len"].long()[:, None] + torch.arange(N, device=DEV).repeat_interleave(r)[None, :] + 1
    hidden = key[None, None, :] >= limit[:, :, None]
    sc.masked_fill_(hidden[:, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    if P:
        pages = s["prefix"].long()
        pk = _values(s, s["k_pages"], s["k_scales"], pages).reshape(-1, Hk, D)[:P]
        pv = _values(s, s["v_pages"], s["v_scales"], pages).reshape(-1, Hk, D)[:P]
        flat = q.permute(1, 0, 2, 3).reshape(Hk, B * N * r, D)
        pc = torch.matmul(flat, pk.permute(1, 2, 0)).view(Hk, B, N * r, P).transpose(0, 1)
        m = torch.maximum(m, pc.amax(-1, keepdim=True))
        pc = (pc - m).exp()
    sc = (sc - m).exp()
    den = sc.sum(-1, keepdim=True)
    o = torch.matmul(sc, v.permute(0, 2, 1, 3))
    if P:
        den = den + pc.sum(-1, keepdim=True)
        flat = pc.transpose(0, 1).reshape(Hk, B * N * r, P)
        o = o + torch.matmul(flat, pv.transpose(0, 1)).view(Hk, B, N * r, D).transpose(0, 1)
    o = (o / den).view(B, Hk, N, r, D).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D)
    s["out"].copy_(o[s["req"], s["place"]])
    return s["out"]


def _run_attention(s):
    if not own:
        return _plain_attention(s)
    from speculative_decoding_verification_62_gb300 import binding
    binding.spec_verify_attention_e4m3(s["q"], s["cache"], s["cu"], s["G"], s["out"], s["workspace"],
                                       prefix_table=s["prefix"] if s["case"]["prefix"] else None,
                                       prefix_len=s["case"]["prefix"])
    return s["out"]


def _books(s):
    return s["table"], s["kv_len"], s["held"], s["ref"], s["free_pages"], s["free_count"]


def _pools(s):
    return [s[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales") if s[n] is not None]


def _bytes(pool):
    return pool.view(torch.uint8)


def _plain_step(s):
    case, B, ps = s["case"], s["B"], s["case"]["page"]
    old, kv_len, held, ref, free, count = _books(s)
    W = old.shape[1]
    b, j = torch.arange(B, device=DEV), torch.arange(W, device=DEV)
    parents = s["parents"].long()
    ends, a = parents < 0, parents.clamp_min(0)
    kv = torch.where(ends, 0, kv_len.long()[a])
    n = torch.where(ends, 0, s["tokens"].long())
    live, need = (kv + ps - 1) // ps, (kv + n + ps - 1) // ps
    new = old[a].long()
    stays = (a == b) & ~ends
    lives = j[None, :] < live[:, None]
    dropped = (j[None, :] < held[:, None]) & ~(stays[:, None] & lives)
    one = torch.ones((), dtype=torch.int32, device=DEV)
    was = old.long().clamp_min(0)
    ref.index_add_(0, new.clamp_min(0).flatten(), (lives & ~stays[:, None]).flatten() * one)
    ref.index_add_(0, was.flatten(), -(dropped.flatten() * one))
    # pages that nobody holds any more, at the first place that dropped them
    place = torch.arange(B * W, device=DEV)
    first = torch.full((ref.numel(),), B * W, device=DEV)
    first.scatter_reduce_(0, was.flatten(), torch.where(dropped.flatten(), place, B * W), "amin")
    frees = dropped.flatten() & (ref[was.flatten()] == 0) & (first[was.flatten()] == place)
    order = frees.long().cumsum(0) - 1
    c, F = count.long(), frees.sum()
    room = torch.cat([free.long(), torch.zeros(1, dtype=torch.int64, device=DEV)])
    room[torch.where(frees, c + order, free.numel())] = was.flatten()
    # partly filled last pages that several rows hold
    writes = (n > 0) & (kv % ps > 0)
    w = torch.where(writes, new.gather(1, (kv // ps).clamp_max(W - 1)[:, None])[:, 0], 0)
    writers = torch.zeros_like(ref).index_add_(0, w, writes.int())
    lowest = torch.full((ref.numel(),), B, device=DEV).scatter_reduce_(0, w, torch.where(writes, b, B), "amin")
    copies = writes & (ref[w] > 1) & ~((writers[w] == ref[w]) & (lowest[w] == b))
    takes = copies.long() + need - live
    before = takes.cumsum(0) - takes
    fits = takes.sum() <= c + F
    copies, takes, need = copies & fits, takes * fits, torch.where(fits, need, live)
    top = c + F - 1 - before
    mine = (j[None, :] >= live[:, None]) & (j[None, :] < need[:, None])
    index = torch.where(mine, copies.long()[:, None] + j[None, :] - live[:, None], 0)
    got = room[(top[:, None] - index).clamp_min(0)]
    fresh = room[top.clamp_min(0)]
    ref.index_add_(0, w, -copies.int())
    ref.index_add_(0, torch.where(mine, got, 0).flatten(), mine.flatten() * one)
    ref.index_add_(0, torch.where(copies, fresh, 0), copies.int())
    here = copies[:, None] & (j[None, :] == (kv // ps)[:, None])
    table = torch.where(lives, new, torch.where(mine, got, torch.where(j[None, :] < held[:, None], -1, old.long())))
    table = torch.where(here, fresh[:, None], table)
    for pool in (s["k_pages"], s["v_pages"]):
        x = _bytes(pool)
        i = torch.arange(ps, device=DEV)
        moves = copies[:, None] & (i[None, :] < (kv % ps)[:, None])
        r, t = moves.nonzero(as_tuple=True)
        x[fresh[r], t] = x[w[r], t]
    if s["k_scales"] is not None:
        for x in (s["k_scales"], s["v_scales"]):
            i = torch.arange(x.shape[1], device=DEV)
            moves = copies[:, None] & (i[None, :] * case["block"] < (kv % ps)[:, None])
            r, t = moves.nonzero(as_tuple=True)
            x[fresh[r], t] = x[w[r], t]
    old.copy_(table)
    kv_len.copy_(kv)
    held.copy_(need)
    free.copy_(room[:-1])
    count.copy_(c + F - takes.sum())


def _run_step(s):
    # (every pass finds the same tables: without this the second would find the first's)
    s["book"].copy_(s["start"])
    if own:
        from speculative_decoding_verification_62_gb300 import binding
        binding.spec_verify_pages_step(s["cache"], s["pool"], s["tokens"], parents=s["parents"])
    else:
        _plain_step(s)
    return [*_books(s), *_pools(s)]


def _plain_compact(s):
    table, _, held, ref, free, count = _books(s)
    N = ref.numel()
    live = ref > 0
    n = int(live.sum())
    src = live[n:].nonzero()[:, 0] + n
    dst = (~live[:n]).nonzero()[:, 0]
    remap = torch.where(live, torch.arange(N, device=DEV), -1)
    remap[src] = dst
    for pool in _pools(s):
        x = _bytes(pool) if pool.dtype == torch.float8_e4m3fn else pool
        x[dst] = x[src]
    mine = torch.arange(table.shape[1], device=DEV)[None, :] < held[:, None]
    table.copy_(torch.where(mine, remap[table.long().clamp_min(0)], table.long()))
    ref[dst] = ref[src]
    ref[src] = 0
    free[:N - n] = torch.arange(N - 1, n - 1, -1, device=DEV, dtype=torch.int32)
    count.fill_(N - n)
    s["remap"].copy_(remap)


def _run_compact(s):
    # (every pass finds the same scattered pages; where they lay they still are)
    s["book"].copy_(s["start"])
    if own:
        from speculative_decoding_verification_62_gb300 import binding
        binding.spec_verify_pages_compact(s["cache"], s["pool"], s["remap"])
    else:
        _plain_compact(s)
    return [s["remap"], *_books(s), *_pools(s)]


def run(state):
    return {"append": _run_append, "attention": _run_attention, "step": _run_step,
            "compact": _run_compact}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The definitions, in 64 bits, request by request
# ---------------------------------------------------------------------------
def _exact_append(s):
    case = s["case"]
    ps, bt, rot, half = case["page"], case["block"], case["rot"], case["rot"] // 2
    k_pages, v_pages, q_out = s["k_pages"].double(), s["v_pages"].double(), s["q"].double().clone()
    k_scales, v_scales = s["k_scales"].double(), s["v_scales"].double()
    row = 0

    def turned(z, ang):
        turn = torch.polar(torch.ones_like(ang), ang)[:, None, :]
        z = z.double().clone()
        if case["interleaved"]:
            z[..., :rot] = torch.view_as_real(torch.view_as_complex(z[..., :rot].reshape(*z.shape[:2], half, 2).contiguous()) * turn).flatten(-2)
        else:
            y = torch.complex(z[..., :half], z[..., half:rot]) * turn
            z[..., :half], z[..., half:rot] = y.real, y.imag
        return z

    def lengths(z, turns):
        """[rows, Hk]: the longest turning pair, or value."""
        z = z.double()
        if not turns:
            return z.abs().amax(-1)
        pair = z[..., :rot].unflatten(-1, (half, 2)).norm(dim=-1) if case["interleaved"] else torch.hypot(z[..., :half], z[..., half:rot])
        return torch.cat([pair, z[..., rot:].abs()], -1).amax(-1)

    for b, (n, x) in enumerate(zip(s["past"], s["gam"])):
        rows = slice(row, row + x + 1)
        row += x + 1
        pos = torch.arange(n, n + x + 1, device=DEV)
        ang = torch.outer(pos.double(), s["inv_freq"])
        q_out[rows] = turned(s["q"][rows], ang)
        page = s["table"][b].long()
        for pool, scales, z, size in ((k_pages, k_scales, turned(s["k"][rows], ang), lengths(s["k"][rows], True)),
                                      (v_pages, v_scales, s["v"][rows].double(), lengths(s["v"][rows], False))):
            first = n // bt
            blocks = pos // bt - first
            most = torch.zeros((int(blocks[-1]) + 1, case["kv_heads"]), dtype=torch.float64, device=DEV)
            most.scatter_reduce_(0, blocks[:, None].expand(-1, case["kv_heads"]), size, "amax")
            scale = torch.exp2(torch.ceil(torch.log2(most / 448.0)).clamp(-32, 56))
            at = page[(first + torch.arange(len(most), device=DEV)) * bt // ps]
            within = (first + torch.arange(len(most), device=DEV)) * bt % ps // bt
            if n % bt:
                was = scales[at[0], within[0]].clone()
                scale[0] = torch.maximum(scale[0], was)
                tokens = torch.arange(n - n % bt, n, device=DEV) % ps
                pool[at[0], tokens] = pool[at[0], tokens] * (was / scale[0])[None, :, None]
            scales[at, within] = scale
            pool[page[pos // ps], pos % ps] = z / scale[blocks][:, :, None]
    return q_out, k_pages, v_pages, k_scales, v_scales


def _exact_attention(s):
    case = s["case"]
    if work(case)["flops"] > 1e12:
        return None
    ps, bt, P, Hk = case["page"], case["block"], case["prefix"], case["kv_heads"]
    r = case["heads"] // Hk
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    row = 0
    for b, (n, x) in enumerate(zip(s["past"], s["gam"])):
        key = torch.cat([torch.arange(P, device=DEV), torch.arange(n + x + 1, device=DEV)])
        page = torch.cat([s["prefix"].long()[key[:P] // ps], s["table"][b].long()[key[P:] // ps]])
        k, v = (pool.view(torch.uint8)[page, key % ps].view(torch.float8_e4m3fn).double() *
                scales[page, key % ps // bt].double()[..., None]
                for pool, scales in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))
        q = s["q"][row:row + x + 1].double()
        seen = torch.arange(P + n + x + 1, device=DEV)[None, :] <= (P + n + torch.arange(x + 1, device=DEV))[:, None]
        for h in range(case["heads"]):
            z = (q[:, h] @ k[:, h // r].T) / math.sqrt(case["D"])
            o[row:row + x + 1, h] = torch.softmax(torch.where(seen, z, -math.inf), -1) @ v[:, h // r]
        row += x + 1
    return o


def exact(case, seed):
    """(The page operators move data and whole numbers: nothing is computed there.)"""
    if case["op"] in ("step", "compact"):
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention}[case["op"]](s)
