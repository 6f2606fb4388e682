"""The operators around one verify step, as cases that can be timed and compared.

Three operators, in the order a serving step runs them:

* ``append``: the step's keys and values go into a paged cache, with the rotary
  position rotation applied to the keys on the way and to the queries beside it;
* ``attention``: the step's query rows (each request's last token and its drafts)
  read the paged cache, where the batch shares a prefix that is read once for all;
* ``probs``: the drafted tokens are verified against the target's probabilities
  (a sampler's output: filtered and renormalised rows) from given uniforms.

``run`` computes them with elementary torch operations where ``own`` is false and
calls the framework's entry points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One interactive request with four drafts over a 32000-token vocabulary
        # (the benchmark's smallest configuration): latency alone.
        dict(name="probs_b1_f32", op="probs", B=1, G=4, V=32000, dtype="f32", drafts="rows",
             layout="padded", ragged=False),
        # A medium batch over the 152064-token vocabulary, probabilities in fp32.
        dict(name="probs_b64_f32", op="probs", B=64, G=5, V=152064, dtype="f32", drafts="rows",
             layout="padded", ragged=False),
        # The large-batch regime with load-adaptive draft lengths, packed rows.
        dict(name="probs_b512_bf16", op="probs", B=512, G=7, V=128256, dtype="bf16", drafts="rows",
             layout="packed", ragged=True),
        # Drafts looked up in the prompt: no draft distribution, odd vocabulary.
        dict(name="probs_point_b128", op="probs", B=128, G=3, V=50257, dtype="f32", drafts="point",
             layout="packed", ragged=True),
        # Single-token step of one request: latency alone.
        dict(name="append_b1", op="append", B=1, G=0, heads=32, kv_heads=8, D=128, rot=128,
             interleaved=False, page=16, dtype="bf16", past=2000),
        # A verify step of a full batch: up to eight rows a request, part of the
        # head rotated, interleaved pairs.
        dict(name="append_b256", op="append", B=256, G=7, heads=32, kv_heads=8, D=128, rot=64,
             interleaved=True, page=64, dtype="bf16", past=100000),
        # Prompts of up to 2501 tokens entering the cache, odd lengths, D = 96.
        dict(name="append_prompts_f16", op="append", B=12, G=2500, heads=24, kv_heads=6, D=96,
             rot=96, interleaved=False, page=32, dtype="f16", past=0),
        # Single-token decoding of one short request: the smallest call.
        dict(name="attn_b1_token", op="attention", B=1, G=0, heads=32, kv_heads=8, D=128, page=16,
             dtype="bf16", prefix=0, own=600),
        # One request with seven drafts over a long context of its own.
        dict(name="attn_b1_long", op="attention", B=1, G=7, heads=64, kv_heads=8, D=128, page=64,
             dtype="bf16", prefix=0, own=131000),
        # An ordinary batch behind a system prompt that ends inside a page.
        dict(name="attn_b32_prefix", op="attention", B=32, G=3, heads=32, kv_heads=8, D=128,
             page=32, dtype="bf16", prefix=2051, own=1000),
        # One key head a query head, D = 64, fp16, odd group of requests.
        dict(name="attn_b37_mha_f16", op="attention", B=37, G=4, heads=12, kv_heads=12, D=64,
             page=16, dtype="f16", prefix=700, own=3000),
        # The largest: a full batch behind a long shared document.
        dict(name="attn_b256_prefix", op="attention", B=256, G=5, heads=32, kv_heads=8, D=128,
             page=64, dtype="bf16", prefix=8192, own=1800),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], {"bytes": 0.0, "flops": 0.0})
        m["bytes"], m["flops"] = max(m["bytes"], w["bytes"]), max(m["flops"], w["flops"])
    op = rng.choice(["probs", "append", "attention", "attention"])
    while True:
        if op == "probs":
            c = dict(op=op, B=_log(rng, 1, 512), G=rng.randint(0, 7), V=_log(rng, 500, 152064),
                     dtype=rng.choice(["f32", "f32", "bf16"]), drafts=rng.choice(["rows", "rows", "point"]),
                     layout=rng.choice(["padded", "packed"]), ragged=rng.random() < 0.7)
        elif op == "append":
            kv = rng.choice([1, 2, 4, 8])
            D = rng.choice([64, 80, 96, 128])
            prompts = rng.random() < 0.3
            c = dict(op=op, B=_log(rng, 1, 16 if prompts else 256), G=_log(rng, 100, 2500) if prompts else rng.randint(0, 8),
                     heads=kv * rng.choice([1, 2, 4, 5, 8]), kv_heads=kv, D=D, rot=rng.choice([D, D, D // 2]),
                     interleaved=rng.random() < 0.5, page=rng.choice([16, 32, 64, 128]),
                     dtype=rng.choice(["bf16", "bf16", "f16"]), past=0 if prompts else _log(rng, 1, 100000))
        else:
            kv = rng.choice([1, 2, 4, 8])
            c = dict(op=op, B=_log(rng, 1, 256), G=rng.randint(0, 8), heads=kv * rng.choice([1, 2, 4, 5, 8]),
                     kv_heads=kv, D=rng.choice([64, 80, 96, 128, 128]), page=rng.choice([16, 32, 64, 128]),
                     dtype=rng.choice(["bf16", "bf16", "f16"]), prefix=rng.choice([0, _log(rng, 50, 16000)]),
                     own=_log(rng, 20, 20000))
        w = work(c)
        # what the plain form holds in between has to fit beside the inputs
        fits = op != "attention" or c["B"] * c["own"] * c["kv_heads"] * c["D"] <= 6e8
        if fits and w["bytes"] <= most[op]["bytes"] and w["flops"] <= most[op]["flops"]:
            return c


def _lengths(case):
    """Draft lengths [B] and tokens already cached [B] of a case: spread over the
    range, from the shape alone, so that work() needs no device."""
    B, G = case["B"], case["G"]
    ragged = case.get("ragged", True)
    gam = [(5 * b + 3 * (b // 7) + G) % (G + 1) if ragged and B > 1 else G for b in range(B)]
    if case["op"] == "probs":
        if ragged and G > 0 and case["drafts"] == "rows":
            gam = [max(1, g) for g in gam]
        return gam, None
    if case["op"] == "append":
        if G >= 100:  # prompts of odd lengths
            gam = [G - 1 - (b * 977) % max(1, G // 2) if B > 1 else G for b in range(B)]
        past = case["past"]
        return gam, [past - (b * 7919) % (past // 2 + 1) if B > 1 else past for b in range(B)]
    n = case["own"]
    return gam, [max(0, n - (b * 2741) % n) if B > 1 else n for b in range(B)]


def work(case):
    gam, past = _lengths(case)
    B = case["B"]
    T = sum(gam) + B
    if case["op"] == "probs":
        # a row of p a request, and one of q where a draft was rejected (most
        # requests with drafts from a distribution: counted as every second)
        V, es = case["V"], 4 if case["dtype"] == "f32" else 2
        rows = B * (1.5 if case["drafts"] == "rows" and case["G"] > 0 else 1.0)
        return {"bytes": rows * V * es + sum(gam) * (8 + 2 * es) + B * (4 * case["G"] + 16), "flops": 3.0 * rows * V}
    Hq, Hk, D = case["heads"], case["kv_heads"], case["D"]
    if case["op"] == "append":
        return {"bytes": 2.0 * 2 * T * (Hq + 2 * Hk) * D, "flops": 3.0 * T * (Hq + Hk) * case["rot"]}
    P = case["prefix"]
    keys = sum(n + g + 1 for n, g in zip(past, gam))
    seen = sum((g + 1) * (P + n) + (g + 1) * (g + 2) // 2 for n, g in zip(past, gam))
    return {"bytes": 2.0 * (2 * (P + keys) * Hk * D + 2 * T * Hq * D), "flops": 4.0 * seen * Hq * D}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _ints(v):
    return torch.tensor(v, dtype=torch.int32).to(DEV)


def _prepare_probs(case, g):
    B, G, V = case["B"], case["G"], case["V"]
    dt = DTYPES[case["dtype"]]
    gam, _ = _lengths(case)
    packed = case["layout"] == "packed"
    cu = [0]
    for x in gam:
        cu.append(cu[-1] + x)
    rows_t, rows_d = (cu[-1] + B, cu[-1]) if packed else (B * (G + 1), B * G)
    t = torch.empty((rows_t, V), dtype=dt, device=DEV)
    d = torch.empty((rows_d, V), dtype=dt, device=DEV)
    tok = torch.empty((rows_d,), dtype=torch.int32, device=DEV)
    # rows of a temperature softmax with a heavy head, the draft's a noisy copy
    # of the target's; drafts are drawn from the draft rows
    step = max(1, (64 << 20) // V)
    for r in range(0, rows_t, step):
        z = torch.randn((min(step, rows_t - r), V), generator=g, device=DEV) * 3.0
        t[r:r + step] = torch.softmax(z, -1).to(dt)
    for b0 in range(0, rows_d, step):
        n = min(step, rows_d - b0)
        i = torch.arange(b0, b0 + n, device=DEV)
        if packed:
            req = torch.searchsorted(_ints(cu[1:]).long(), i, right=True)
            at = i + req
        else:
            at = i // max(G, 1) * (G + 1) + i % max(G, 1)
        z = torch.log(t[at].float().clamp_min(1e-30))
        z += torch.randn(z.shape, generator=g, device=DEV) * 0.8
        q = torch.softmax(z, -1).to(dt)
        d[b0:b0 + n] = q
        race = q.float() / torch.empty_like(z).exponential_(generator=g)
        tok[b0:b0 + n] = race.argmax(-1).int()
    s = dict(case=case, V=V, G=G, B=B, packed=packed, target=t, draft=d if case["drafts"] == "rows" else None,
             tokens=tok, gamma=_ints(gam), cu=_ints(cu))
    s["uniforms"] = torch.rand((rows_t,), generator=g, device=DEV)
    if not packed:
        s["target"], s["tokens"] = t.view(B, G + 1, V), tok.view(B, G)
        s["uniforms"] = s["uniforms"].view(B, G + 1)
        if s["draft"] is not None:
            s["draft"] = d.view(B, G, V)
    s["out"] = torch.full((B, G + 1), -7, dtype=torch.int32, device=DEV)
    s["accepted"] = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    if own:
        from speculative_decoding_verification_62_gb300 import binding
        s["workspace"] = binding.make_workspace(B, G, V)
    return s


def _pages(case, own_tokens, prefix, g):
    """A page pool with every request's pages (and the prefix's) dealt out in a
    random order, and a few pages that nobody uses."""
    ps = case["page"]
    need = [-(-n // ps) for n in own_tokens]
    pre = -(-prefix // ps)
    total = sum(need) + pre
    perm = torch.randperm(total + 3, generator=g, device=DEV).int()
    table = torch.full((len(need), max(max(need), 1)), -1, dtype=torch.int32)
    flat, at = perm.cpu(), pre
    for b, n in enumerate(need):
        table[b, :n] = flat[at:at + n]
        at += n
    return total + 3, table.to(DEV), perm[:pre].contiguous()


def _prepare_cache(case, g, fill):
    gam, past = _lengths(case)
    B, Hk, D = case["B"], case["kv_heads"], case["D"]
    dt = DTYPES[case["dtype"]]
    cu = [0]
    for x in gam:
        cu.append(cu[-1] + x)
    T = cu[-1] + B
    # only the pages that the step touches exist for an append far into a context
    skip = [(p // case["page"]) * case["page"] if case["op"] == "append" else 0 for p in past]
    n, table, prefix = _pages(case, [p - k + x + 1 for p, k, x in zip(past, skip, gam)], case.get("prefix", 0), g)
    if case["op"] == "append":
        wide = max((p + x + 1 + case["page"] - 1) // case["page"] for p, x in zip(past, gam))
        full = torch.full((B, wide), -1, dtype=torch.int32)
        rows = table.cpu()
        for b in range(B):
            at = skip[b] // case["page"]
            w = min(rows.shape[1], wide - at)
            full[b, at:at + w] = rows[b, :w]
        table = full.to(DEV)
    shape = (n, case["page"], Hk, D)
    if fill:
        k = torch.randn(shape, generator=g, device=DEV, dtype=dt)
        v = torch.randn(shape, generator=g, device=DEV, dtype=dt)
    else:
        k, v = torch.zeros(shape, device=DEV, dtype=dt), torch.zeros(shape, device=DEV, dtype=dt)
    return dict(case=case, B=B, T=T, G=max(gam), gam=gam, past=past, k_pages=k, v_pages=v, table=table,
                prefix=prefix, kv_len=_ints(past), cu=_ints(cu),
                workspace=None, req=_ints([b for b, x in enumerate(gam) for _ in range(x + 1)]).long(),
                place=_ints([i for x in gam for i in range(x + 1)]).long())


def _prepare_append(case, g):
    s = _prepare_cache(case, g, False)
    Hq, Hk, D, dt = case["heads"], case["kv_heads"], case["D"], DTYPES[case["dtype"]]
    # one projection's output holds q, k and v side by side: strided views
    qkv = torch.randn((s["T"], Hq + 2 * Hk, D), generator=g, device=DEV, dtype=dt)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    s["q_out"] = torch.empty((s["T"], Hq, D), device=DEV, dtype=dt)
    half = case["rot"] // 2
    s["inv_freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    if own:
        from speculative_decoding_verification_62_gb300 import binding, rope
        s["freq"] = rope.fixed_point(s["inv_freq"]).to(DEV)
        s["cache"] = binding.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["kv_len"])
        s["workspace"] = binding.make_attention_workspace(s["T"], Hq, D)
    s["inv_freq"] = s["inv_freq"].to(DEV)
    return s


def _prepare_attention(case, g):
    s = _prepare_cache(case, g, True)
    Hq, D, dt = case["heads"], case["D"], DTYPES[case["dtype"]]
    s["q"] = (torch.randn((s["T"], Hq, D), generator=g, device=DEV) * 2.0).to(dt)
    s["out"] = torch.empty_like(s["q"])
    if own:
        from speculative_decoding_verification_62_gb300 import binding
        s["cache"] = binding.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["kv_len"])
        s["workspace"] = binding.make_attention_workspace(s["T"], Hq, D)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return {"probs": _prepare_probs, "append": _prepare_append, "attention": _prepare_attention}[case["op"]](case, g)


# ---------------------------------------------------------------------------
# The passes
# ---------------------------------------------------------------------------
def _rows_of(s):
    """First target and draft row of each request, as int64 [B]."""
    if s["packed"]:
        cu = s["cu"][:-1].long()
        return cu + torch.arange(s["B"], device=DEV), cu
    b = torch.arange(s["B"], device=DEV)
    return b * (s["G"] + 1), b * s["G"]


def _plain_probs(s):
    B, G, V = s["B"], s["G"], s["V"]
    t, tok, u = s["target"].reshape(-1, V), s["tokens"].reshape(-1), s["uniforms"].reshape(-1)
    d = None if s["draft"] is None else s["draft"].reshape(-1, V)
    gam = s["gamma"].long()
    t0, d0 = _rows_of(s)
    i = torch.arange(G, device=DEV)
    valid = i[None, :] < gam[:, None]
    ti, di = torch.where(valid, t0[:, None] + i, 0), torch.where(valid, d0[:, None] + i, 0)
    k = gam.clone()
    x = torch.zeros((B, G), dtype=torch.int64, device=DEV)
    if G > 0 and tok.numel() > 0:
        x = torch.where(valid, tok[di].long(), 0)
        p = t[ti, x].double()
        q = torch.ones_like(p) if d is None else d[di, x].double()
        ok = (q == 0) | (u[ti].double() * q < p)  # products of two 32-bit values: exact
        bad = valid & ~ok
        first = torch.where(bad, i[None, :], G).amin(-1)
        k = torch.minimum(first, gam)
    row = t[t0 + k].double()
    rejected = k < gam
    w = row
    if G > 0 and tok.numel() > 0:
        kr = torch.where(rejected, k, 0)
        if d is None:
            q = torch.zeros_like(row)
            q[torch.arange(B, device=DEV), x.gather(1, kr[:, None].clamp_max(G - 1))[:, 0]] = 1.0
        else:
            q = d[torch.where(rejected, d0 + kr, 0)].double()
        w = torch.where(rejected[:, None], (row - q).clamp_min(0.0), row)
        w = torch.where(w.sum(-1, keepdim=True) > 0, w, row)
    c = w.cumsum(-1)
    last = t0 + gam if s["packed"] else t0 + G
    goal = u[last].double() * c[:, -1]
    z = torch.searchsorted(c, goal[:, None], right=True)[:, 0].clamp_max(V - 1)
    j = torch.arange(G + 1, device=DEV)[None, :]
    drafts = torch.cat([x, torch.zeros((B, 1), dtype=torch.int64, device=DEV)], 1)
    s["out"].copy_(torch.where(j < k[:, None], drafts, torch.where(j == k[:, None], z[:, None], -1)))
    s["accepted"].copy_(k)
    return s["out"], s["accepted"]


def _run_probs(s):
    if not own:
        return _plain_probs(s)
    from speculative_decoding_verification_62_gb300 import binding
    if s["packed"]:
        binding.spec_verify_sample_probs_packed(s["target"], s["draft"], s["cu"], s["tokens"], s["uniforms"],
                                                s["out"], s["accepted"], s["workspace"])
    else:
        binding.spec_verify_sample_probs(s["target"], s["draft"], s["tokens"], s["gamma"], s["uniforms"],
                                         s["out"], s["accepted"], s["workspace"])
    return s["out"], s["accepted"]


def _rotated(x, cos, sin, rot, interleaved):
    """x [T, H, D] with its first `rot` values of a head turned, in 32 bits."""
    y = x.float()
    r = y[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, y[..., rot:]], -1).to(x.dtype)


def _plain_append(s):
    case = s["case"]
    pos = s["kv_len"].long()[s["req"]] + s["place"]
    ang = pos.double()[:, None] * s["inv_freq"][None, :]
    cos, sin = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    page = s["table"][s["req"], pos // case["page"]].long()
    s["k_pages"][page, pos % case["page"]] = _rotated(s["k"], cos, sin, case["rot"], case["interleaved"])
    s["v_pages"][page, pos % case["page"]] = s["v"]
    s["q_out"].copy_(_rotated(s["q"], cos, sin, case["rot"], case["interleaved"]))
    return s["q_out"], s["k_pages"], s["v_pages"]


def _run_append(s):
    if not own:
        return _plain_append(s)
    from speculative_decoding_verification_62_gb300 import binding
    binding.spec_verify_kv_append(s["q"], s["k"], s["v"], s["cache"], s["cu"], s["G"], s["freq"], s["q_out"],
                                  s["workspace"], interleaved=s["case"]["interleaved"])
    return s["q_out"], s["k_pages"], s["v_pages"]


def _plain_attention(s):
    case = s["case"]
    B, T, ps, P = s["B"], s["T"], case["page"], case["prefix"]
    Hq, Hk, D = case["heads"], case["kv_heads"], case["D"]
    r = Hq // Hk
    N = s["G"] + 1
    table = s["table"].long().clamp_min(0)
    L = table.shape[1] * ps
    # the requests' own keys, padded to the longest
    k = s["k_pages"][table].reshape(B, L, Hk, D).float()
    v = s["v_pages"][table].reshape(B, L, Hk, D).float()
    q = torch.zeros((B, N, Hk, r, D), device=DEV)
    q[s["req"], s["place"]] = s["q"].float().view(T, Hk, r, D) * (1.0 / math.sqrt(D))
    q = q.permute(0, 2, 1, 3, 4).reshape(B, Hk, N * r, D)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1))
    key = torch.arange(L, device=DEV)
    limit = s["kv_len"].long()[:, None] + torch.arange(N, device=DEV).repeat_interleave(r)[None, :] + 1
    hidden = key[None, None, :] >= limit[:, :, None]
    sc.masked_fill_(hidden[:, None], -math.inf)
    v.masked_fill_((key[None, :] >= s["kv_len"].long()[:, None] + N)[:, :, None, None], 0.0)
    m = sc.amax(-1, keepdim=True)
    if P:
        pk = s["k_pages"][s["prefix"].long()].reshape(-1, Hk, D)[:P].float()
        pv = s["v_pages"][s["prefix"].long()].reshape(-1, Hk, D)[:P].float()
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
    binding.spec_verify_attention(s["q"], s["cache"], s["cu"], s["G"], s["out"], s["workspace"],
                                  prefix_table=s["prefix"], prefix_len=s["case"]["prefix"])
    return s["out"]


def run(state):
    return {"probs": _run_probs, "append": _run_append, "attention": _run_attention}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The definitions, in 64 bits, request by request
# ---------------------------------------------------------------------------
def _exact_probs(s):
    import numpy as np
    B, G, V = s["B"], s["G"], s["V"]
    t, u, tok = s["target"].reshape(-1, V), s["uniforms"].reshape(-1).cpu().numpy().astype(np.float64), s["tokens"].reshape(-1).cpu().numpy()
    d = None if s["draft"] is None else s["draft"].reshape(-1, V)
    cu, gam = s["cu"].cpu().numpy(), s["gamma"].cpu().numpy()
    out, acc = np.full((B, G + 1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        t0, d0 = (int(cu[b]) + b, int(cu[b])) if s["packed"] else (b * (G + 1), b * G)
        n = int(gam[b])
        w = None
        for i in range(n):
            x = int(tok[d0 + i])
            p = t[t0 + i].double().cpu().numpy()
            q = np.eye(1, V, x)[0] if d is None else d[d0 + i].double().cpu().numpy()
            if q[x] == 0 or u[t0 + i] < p[x] / q[x]:
                out[b, i] = x
                acc[b] += 1
                continue
            w = np.maximum(p - q, 0.0)
            if not w.any():
                w = p
            break
        if w is None:
            w = t[t0 + n].double().cpu().numpy()
        c = np.cumsum(w)
        out[b, acc[b]] = min(V - 1, int(np.searchsorted(c, u[t0 + (n if s["packed"] else G)] * c[-1], side="right")))
    return out, acc


def _exact_append(s):
    case = s["case"]
    ps, rot, half = case["page"], case["rot"], case["rot"] // 2
    k_pages, v_pages, q_out = s["k_pages"].double(), s["v_pages"].double(), s["q"].double().clone()
    row = 0
    for b, (n, x) in enumerate(zip(s["past"], s["gam"])):
        pos = torch.arange(n, n + x + 1, device=DEV)
        ang = torch.outer(pos.double(), s["inv_freq"])
        turn = torch.polar(torch.ones_like(ang), ang)[:, None, :]
        rows = slice(row, row + x + 1)
        row += x + 1
        for src, dst in ((s["q"], q_out), (s["k"], None)):
            z = src[rows].double().clone()
            if case["interleaved"]:
                z[..., :rot] = torch.view_as_real(torch.view_as_complex(z[..., :rot].reshape(*z.shape[:2], half, 2).contiguous()) * turn).flatten(-2)
            else:
                y = torch.complex(z[..., :half], z[..., half:rot]) * turn
                z[..., :half], z[..., half:rot] = y.real, y.imag
            if dst is not None:
                dst[rows] = z
            else:
                at = s["table"][b].long()[pos // ps]
                k_pages[at, pos % ps] = z
                v_pages[at, pos % ps] = s["v"][rows].double()
    return q_out, k_pages, v_pages


def _exact_attention(s):
    case = s["case"]
    if work(case)["flops"] > 4e12:
        return None
    ps, P, Hk = case["page"], case["prefix"], case["kv_heads"]
    r = case["heads"] // Hk
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    row = 0
    for b, (n, x) in enumerate(zip(s["past"], s["gam"])):
        key = torch.cat([torch.arange(P, device=DEV), torch.arange(n + x + 1, device=DEV)])
        page = torch.cat([s["prefix"].long()[key[:P] // ps], s["table"][b].long()[key[P:] // ps]])
        k, v = s["k_pages"][page, key % ps].double(), s["v_pages"][page, key % ps].double()
        q = s["q"][row:row + x + 1].double()
        seen = torch.arange(P + n + x + 1, device=DEV)[None, :] <= (P + n + torch.arange(x + 1, device=DEV))[:, None]
        for h in range(case["heads"]):
            z = (q[:, h] @ k[:, h // r].T) / math.sqrt(case["D"])
            o[row:row + x + 1, h] = torch.softmax(torch.where(seen, z, -math.inf), -1) @ v[:, h // r]
        row += x + 1
    return o


def exact(case, seed):
    s = prepare(case, seed)
    return {"probs": _exact_probs, "append": _exact_append, "attention": _exact_attention}[case["op"]](s)
