"""Verification from given probabilities against the definition in 64 bits: every
decision and every drawn token has to be the same."""
import numpy as np
import pytest
import torch

from operator_refs import probs_request
from speculative_decoding_verification_62_gb300 import binding

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(B, G, V, dtype, seed, gamma=None, filtered=False, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    t = torch.softmax(torch.randn((B, G + 1, V), generator=g) * sharp, -1)
    if filtered:  # a nucleus: most entries exactly 0, the rest renormalised
        keep = torch.rand((B, G + 1, V), generator=g) < 0.1
        keep[..., 0] = True
        t = t * keep
        t = t / t.sum(-1, keepdim=True)
    z = torch.log(t[:, :G].clamp_min(1e-12)) + torch.randn((B, G, V), generator=g) * 0.7
    d = torch.softmax(z, -1)
    t, d = t.to(DT[dtype]), d.to(DT[dtype])
    tok = torch.zeros((B, G), dtype=torch.int32)
    if G:
        noise = torch.empty((B, G, V)).exponential_(generator=g)
        tok = (d.float() / noise).argmax(-1).int()
    if gamma is None:
        gam = torch.full((B,), G, dtype=torch.int32)
    else:
        gam = torch.randint(0, G + 1, (B,), generator=g).int()
    u = torch.rand((B, G + 1), generator=g)
    return t, d, tok, gam, u


def reference(t, d, tok, gam, u):
    B, G1, _ = t.shape
    out, acc = np.full((B, G1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n = int(gam[b])
        q = None if d is None else d[b, :n].double().numpy()
        acc[b], z = probs_request(t[b, :n + 1].double().numpy(), q, tok[b, :n].numpy(),
                                  u[b].numpy(), float(u[b, G1 - 1]))
        out[b, :acc[b]] = tok[b, :acc[b]].numpy()
        out[b, acc[b]] = z
    return out, acc


def run(t, d, tok, gam, u, status=0):
    B, G1, V = t.shape
    v = binding.Verifier(B, G1 - 1, V)
    v.out_tokens.fill_(-7)
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    out, acc = v.sample_probs(c(t), c(d), c(tok), c(gam), c(u))
    assert binding.spec_verify_status(v.workspace) == status
    return out.cpu().numpy(), acc.cpu().numpy()


def pack(t, d, tok, gam, u):
    B, G1, V = t.shape
    n = gam.tolist()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
    tp = torch.cat([t[b, :n[b] + 1] for b in range(B)])
    dp = None if d is None else torch.cat([d[b, :n[b]] for b in range(B)])
    kp = torch.cat([tok[b, :n[b]] for b in range(B)])
    up = torch.cat([torch.cat([u[b, :n[b]], u[b, G1 - 1:]]) for b in range(B)])
    return tp, dp, cu, kp, up


@pytest.mark.parametrize("drafts", ["rows", "point"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,G,V", [(1, 0, 1), (1, 4, 7), (3, 31, 33), (5, 3, 4096), (2, 5, 32000),
                                   (40, 4, 1001), (200, 2, 515), (700, 1, 64)])
def test_against_the_definition(B, G, V, dtype, drafts):
    t, d, tok, gam, u = make(B, G, V, dtype, 100 + B + G + V, gamma="ragged")
    if drafts == "point":
        d = None
    ref, ra = reference(t, d, tok, gam, u)
    out, acc = run(t, d, tok, gam, u)
    assert (acc == ra).all() and (out == ref).all()


@pytest.mark.parametrize("drafts", ["rows", "point"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_equals_padded(dtype, drafts):
    t, d, tok, gam, u = make(60, 5, 2003, dtype, 7, gamma="ragged")
    if drafts == "point":
        d = None
    out, acc = run(t, d, tok, gam, u)
    tp, dp, cu, kp, up = pack(t, d, tok, gam, u)
    v = binding.Verifier(60, 5, 2003)
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    o, a = v.sample_probs_packed(c(tp), c(dp), c(cu), c(kp), c(up))
    assert binding.spec_verify_status(v.workspace) == 0
    assert (o.cpu().numpy() == out).all() and (a.cpu().numpy() == acc).all()


def test_filtered_rows_and_unaligned_views():
    """Rows that are mostly exact zeros, and rows that start off a 16-byte boundary."""
    t, d, tok, gam, u = make(9, 3, 5000, "f32", 11, filtered=True)
    ref, ra = reference(t, d, tok, gam, u)
    out, acc = run(t, d, tok, gam, u)
    assert (acc == ra).all() and (out == ref).all()
    v = binding.Verifier(9, 3, 5000)
    big_t, big_d = torch.empty(t.numel() + 1, device="cuda"), torch.empty(d.numel() + 3, device="cuda")
    tv, dv = big_t[1:].view(t.shape), big_d[3:].view(d.shape)
    tv.copy_(t)
    dv.copy_(d)
    o, a = v.sample_probs(tv, dv, tok.cuda(), gam.cuda(), u.cuda())
    assert (o.cpu().numpy() == ref).all() and (a.cpu().numpy() == ra).all()


def test_exact_boundaries():
    """Probabilities that are powers of two: u on a boundary belongs to the next token,
    one step below it to the token before."""
    w = torch.tensor([0.25, 0.0, 0.125, 0.5, 0.125, 0.0])
    steps = [0.0, 0.25, 0.375, 0.875]
    below = [float(np.nextafter(np.float32(x), np.float32(0))) for x in steps[1:]]
    us = steps + below + [float(np.nextafter(np.float32(1), np.float32(0)))]
    want = [0, 2, 3, 4, 0, 2, 3, 4]
    B = len(us)
    t = w.repeat(B, 1, 1)
    out, acc = run(t, None, torch.zeros((B, 0), dtype=torch.int32), torch.zeros(B, dtype=torch.int32),
                   torch.tensor(us)[:, None])
    assert out[:, 0].tolist() == want and (acc == 0).all()


def test_acceptance_is_strict_and_exact():
    """u q == p refuses, the next smaller u accepts; q = 0 accepts; looked-up drafts
    test u < p."""
    p, q = 0.25, 0.5
    us = [0.5, float(np.nextafter(np.float32(0.5), np.float32(0))), 0.999]
    t = torch.zeros((4, 2, 4))
    d = torch.zeros((4, 1, 4))
    t[:, 0] = torch.tensor([p, 0.75, 0.0, 0.0])
    t[:, 1, 3] = 1.0
    d[:, 0] = torch.tensor([q, 0.0, 0.5, 0.0])
    d[2, 0, 0] = 0.0
    u = torch.full((4, 2), 0.5)
    u[:3, 0] = torch.tensor([us[0], us[1], us[2]])
    u[3, 0] = 0.25
    tok, gam = torch.zeros((4, 1), dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    out, acc = run(t, d, tok, gam, u)
    assert acc.tolist() == [0, 1, 1, 1]
    assert out.tolist() == [[1, -1], [0, 3], [0, 3], [0, 3]]
    out, acc = run(t, None, tok, gam, u)
    assert acc.tolist() == [0, 0, 0, 0]
    u[:, 0] = float(np.nextafter(np.float32(0.25), np.float32(0)))
    out, acc = run(t, None, tok, gam, u)
    assert acc.tolist() == [1, 1, 1, 1]


def test_vanished_residual_draws_from_p():
    """p == q at the refused row (a draft with p(x) = 0 < q(x) cannot be: x has u = 1 - ulp
    and q barely above p): every residual weight is 0 after the rounding of neither."""
    t = torch.tensor([[[0.5, 0.5], [1.0, 0.0]]] * 3)
    d = torch.tensor([[[1.0, 0.5]]] * 3)
    # the residual is max(0, [-.5, 0]) = 0
    u = torch.tensor([[0.75, 0.0], [0.75, 0.49], [0.75, 0.5]])
    tok, gam = torch.zeros((3, 1), dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    out, acc = run(t, d, tok, gam, u)
    assert acc.tolist() == [0, 0, 0] and out[:, 0].tolist() == [0, 0, 1]
    # looked-up draft: all of p on the refused token cannot be refused but by u >= p
    t = torch.tensor([[[0.5, 0.0], [1.0, 0.0]]])
    out, acc = run(t, None, torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32),
                   torch.tensor([[0.9, 0.3]]))
    assert acc.tolist() == [0] and out.tolist() == [[0, -1]]


def test_bad_values_are_flagged_and_stay_inside():
    S = {n: b for b, n in binding.STATUS_BITS.items()}
    t, d, tok, gam, u = make(6, 2, 300, "f32", 5)
    bad = t.clone()
    bad[0, :, 5] = float("nan")
    bad[1, :, 6] = -1.0
    bad[2, :, 7] = 3.0
    out, _ = run(bad, d, tok, gam, u, status=S["BAD_PROB"])
    assert ((out >= -1) & (out < 300)).all()
    zero = t.clone()
    zero[3] = 0.0
    out, acc = run(zero, d, tok, gam, u, status=S["BAD_PROB"])
    assert acc[3] == 0 and out[3, 0] == 299
    run(t, d, torch.full_like(tok, 300), gam, u, status=S["BAD_TOKEN"])
    run(t, d, tok, torch.tensor([0, 1, 2, 3, -1, 2], dtype=torch.int32), u, status=S["BAD_GAMMA"])
    run(t, d, tok, gam, u + 1.0, status=S["BAD_UNIFORM"])
    ones = torch.ones((1, 1, 70000))
    run(ones, None, torch.zeros((1, 0), dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
        torch.tensor([[0.9]]), status=S["BAD_PROB"])


def test_inconsistent_packed_prefix():
    S = {n: b for b, n in binding.STATUS_BITS.items()}
    t, d, tok, gam, u = make(4, 3, 100, "f32", 9)
    tp, dp, cu, kp, up = pack(t, d, tok, gam, u)
    cu = torch.tensor([0, 9, 2, 40, 12], dtype=torch.int32)
    v = binding.Verifier(4, 3, 100)
    o, a = v.sample_probs_packed(tp.cuda(), dp.cuda(), cu.cuda(), kp.cuda(), up.cuda())
    assert binding.spec_verify_status(v.workspace) == S["BAD_GAMMA"]
    assert ((o >= -1) & (o < 100)).all() and (a >= 0).all()


def test_large_vocabulary_many_requests():
    """Two requests an SM and more, one CTA a request; V of the large configurations."""
    t, d, tok, gam, u = make(4, 2, 152064, "bf16", 21, gamma="ragged")
    ref, ra = reference(t, d, tok, gam, u)
    n = 90
    out, acc = run(t.repeat(n, 1, 1), d.repeat(n, 1, 1), tok.repeat(n, 1), gam.repeat(n), u.repeat(n, 1))
    assert (out.reshape(n, 4, 3) == ref).all() and (acc.reshape(n, 4) == ra).all()


def test_no_requests_is_a_noop():
    z = torch.zeros
    ws = binding.make_workspace(1, 2, 50)
    out, acc = z((0, 3), dtype=torch.int32, device="cuda"), z((0,), dtype=torch.int32, device="cuda")
    binding.spec_verify_sample_probs(z((0, 3, 50), device="cuda"), z((0, 2, 50), device="cuda"),
                                     z((0, 2), dtype=torch.int32, device="cuda"), acc.clone(),
                                     z((0, 3), device="cuda"), out, acc, ws)
    assert binding.spec_verify_status(ws) == 0


def test_refused_tensors():
    t, d, tok, gam, u = (x.cuda() for x in make(2, 2, 40, "f32", 1))
    v = binding.Verifier(2, 2, 40)
    for bad in (dict(t=t.half()), dict(d=d.bfloat16()), dict(u=u.double()), dict(tok=tok.long()), dict(u=u.cpu())):
        a = dict(t=t, d=d, tok=tok, gam=gam, u=u)
        a.update(bad)
        with pytest.raises(TypeError):
            v.sample_probs(a["t"], a["d"], a["tok"], a["gam"], a["u"])
    for bad in (dict(t=t[:, :, ::2]), dict(d=d[:, :1]), dict(gam=gam[:1])):
        a = dict(t=t, d=d, tok=tok, gam=gam, u=u)
        a.update(bad)
        with pytest.raises(ValueError):
            v.sample_probs(a["t"], a["d"], a["tok"], a["gam"], a["u"])


def test_side_stream_and_graph():
    t, d, tok, gam, u = (x.cuda() for x in make(20, 3, 3000, "f32", 33, gamma="ragged"))
    v = binding.Verifier(20, 3, 3000)
    ref = [x.clone() for x in v.sample_probs(t, d, tok, gam, u)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w = binding.Verifier(20, 3, 3000)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        w.sample_probs(t, d, tok, gam, u)
    s.synchronize()
    assert torch.equal(w.out_tokens, ref[0]) and torch.equal(w.num_accepted, ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.sample_probs(t, d, tok, gam, u)
    u2 = torch.rand_like(u)
    u.copy_(u2)
    graph.replay()
    torch.cuda.synchronize()
    ref = v.sample_probs(t, d, tok, gam, u2)
    assert torch.equal(w.out_tokens, ref[0]) and torch.equal(w.num_accepted, ref[1])


def test_more_than_the_logits_path_and_the_same_decisions():
    """Softmax rows handed over as probabilities: the decisions agree with the logits
    path wherever its own near ties do not lie (p and q rounded to fp32 first)."""
    g = torch.Generator().manual_seed(3)
    B, G, V = 50, 4, 4000
    zt = torch.randn((B, G + 1, V), generator=g) * 2
    zd = zt[:, :G] + torch.randn((B, G, V), generator=g) * 0.5
    p, q = torch.softmax(zt.double(), -1), torch.softmax(zd.double(), -1)
    tok = (q / torch.empty((B, G, V), dtype=torch.float64).exponential_(generator=g)).argmax(-1).int()
    u = torch.rand((B, G + 1), generator=g)
    gam = torch.full((B,), G, dtype=torch.int32)
    v = binding.Verifier(B, G, V)
    a = [x.clone() for x in v.sample(zt.cuda(), zd.cuda(), tok.cuda(), gam.cuda(), u.cuda(), torch.ones(B).cuda())]
    b = v.sample_probs(p.float().cuda(), q.float().cuda(), tok.cuda(), gam.cuda(), u.cuda())
    ratio = torch.gather(p[:, :G], 2, tok[..., None].long()) / torch.gather(q, 2, tok[..., None].long())
    clear = ((ratio[..., 0] - u[:, :G]).abs() > 1e-5).all(-1).cuda()
    assert clear.sum() >= B - 2
    assert torch.equal(a[1][clear], b[1][clear])
    # a draw differs only where u lies within the fp32 rounding of a boundary
    assert (a[0][clear] != b[0][clear]).any(-1).sum() <= 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_sum_to_little_or_much(dtype):
    """A draw goes by its weights' own total; weights below 2^-47 count as 0 (the rest of
    a weight is added to 1.5 2^-23, whose last bit is 2^-46)."""
    S = {n: b for b, n in binding.STATUS_BITS.items()}
    w = torch.tensor([0.25, 0.0, 0.125, 0.5, 0.125, 0.0], dtype=DT[dtype])
    us = [0.0, 0.24, 0.25, 0.374, 0.375, 0.874, 0.875, 0.999]
    want = [0, 0, 2, 2, 3, 3, 4, 4]
    tok, gam = torch.zeros((8, 0), dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    for power in (-43, -20, 1):  # (2^-43 of 0.125 is one step)
        out, _ = run((w * 2.0 ** power).repeat(8, 1, 1), None, tok, gam, torch.tensor(us)[:, None])
        assert out[:, 0].tolist() == want
    # many entries of 1: their sum is exact
    out, _ = run(torch.ones((8, 1, 60000), dtype=DT[dtype]), None, tok, gam, torch.tensor(us)[:, None])
    assert out[:, 0].tolist() == [int(np.floor(np.float32(u).astype(np.float64) * 60000)) for u in us]
    out, _ = run((w * 2.0 ** -60).repeat(8, 1, 1), None, tok, gam, torch.tensor(us)[:, None], status=S["BAD_PROB"])
    assert (out[:, 0] == 5).all()
