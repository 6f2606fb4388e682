"""Arguments that the new operators refuse on the host, before any launch (CPU only), and
the host logic beside them."""
import ctypes
import math

import pytest
import torch

from speculative_decoding_verification_62_gb300 import binding, rope


def ptr(addr=0x100000):
    return ctypes.c_void_p(addr)


def probs(packed=False, **over):
    lib = binding.load_library()
    a = dict(t=ptr(), d=ptr(), dtype=0, B=2, G=3, V=64, cu=ptr(), total=4, tok=ptr(), gamma=ptr(),
             u=ptr(), out=ptr(), acc=ptr(), ws=ptr(), ws_bytes=1 << 30)
    a.update(over)
    if packed:
        return lib.spec_verify_sample_probs_packed(
            a["t"], a["d"], a["dtype"], a["B"], a["G"], a["V"], a["cu"], a["total"], a["tok"], a["u"],
            a["out"], a["acc"], a["ws"], a["ws_bytes"], None)
    return lib.spec_verify_sample_probs(a["t"], a["d"], a["dtype"], a["B"], a["G"], a["V"], a["tok"],
                                        a["gamma"], a["u"], a["out"], a["acc"], a["ws"],
                                        a["ws_bytes"], None)


@pytest.mark.parametrize("packed", [False, True])
def test_probs_refusals(packed):
    for bad in (dict(B=-1), dict(G=-1), dict(G=32), dict(V=0), dict(V=(1 << 24) + 1), dict(dtype=2)):
        assert probs(packed, **bad) == -1, bad
    for name in ("t", "u", "out", "acc", "ws", "tok", "cu" if packed else "gamma"):
        assert probs(packed, **{name: None}) == -2, name
    assert probs(packed, ws_bytes=100) == -4
    for name, at in (("t", 0x100002), ("d", 0x100002), ("u", 0x100002), ("out", 0x100001),
                     ("tok", 0x100002), ("ws", 0x100010)):
        assert probs(packed, **{name: ptr(at)}) == -3, name
    assert probs(packed, B=0) == 0
    if packed:
        assert probs(True, total=-1) == -1


def cache(**over):
    c = binding._KvCache(0x100000, 0x200000, 1, 10, 16, 2, 64, (ctypes.c_int64 * 3)(2048, 128, 64),
                         (ctypes.c_int64 * 3)(2048, 128, 64), 0x300000, 4, 3, 0x400000)
    for k, v in over.items():
        if k.endswith("strides"):
            v = (ctypes.c_int64 * 3)(*v)
        setattr(c, k, v)
    return c


BAD_CACHES = [dict(dtype=0), dict(dtype=3), dict(num_pages=0), dict(page_size=8), dict(page_size=24),
              dict(page_size=8192), dict(kv_heads=0), dict(head_dim=0), dict(head_dim=60),
              dict(head_dim=136), dict(k_strides=(2048, 128, 4)), dict(v_strides=(0, 128, 64)),
              dict(k_strides=(2048, -128, 64)), dict(batch=-1), dict(max_pages=-1)]
NULL_CACHES = [dict(k_pages=None), dict(v_pages=None), dict(page_table=None), dict(kv_len=None)]
OFF_CACHES = [dict(k_pages=0x100008), dict(v_pages=0x100002), dict(kv_len=0x400002), dict(page_table=0x300001)]


def append(c=None, **over):
    lib = binding.load_library()
    two = (ctypes.c_int64 * 2)(512, 64)
    a = dict(q=ptr(), qs=two, heads=4, k=ptr(), ks=two, v=ptr(), vs=two, o=ptr(), os=two, cu=ptr(),
             total=5, G=3, freq=ptr(), rot=64, inter=0, scale=1.0, pos=None, off=0, ws=ptr(), ws_bytes=256)
    a.update(over)
    return lib.spec_verify_kv_append(a["q"], a["qs"], a["heads"], a["k"], a["ks"], a["v"], a["vs"], a["o"],
                                     a["os"], ctypes.byref(c or cache()), a["cu"], a["total"], a["G"], a["freq"],
                                     a["rot"], a["inter"], a["scale"], a["pos"], a["off"], a["ws"],
                                     a["ws_bytes"], None)


def test_append_refusals():
    for bad in BAD_CACHES:
        assert append(cache(**bad)) == -1, bad
    for bad in NULL_CACHES:
        assert append(cache(**bad)) == -2, bad
    for bad in OFF_CACHES:
        assert append(cache(**bad)) == -3, bad
    for bad in (dict(total=-1), dict(G=-1), dict(heads=-1), dict(rot=63), dict(rot=66), dict(rot=-2),
                dict(inter=2), dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf), dict(total=2 ** 31 - 2)):
        assert append(**bad) == -1, bad
    for name in ("q", "qs", "k", "ks", "v", "vs", "o", "os", "cu", "freq", "ws"):
        assert append(**{name: None}) == -2, name
    assert append(ws_bytes=2) == -4
    for name, at in (("k", 0x100001), ("freq", 0x100004), ("cu", 0x100002), ("pos", 0x100002), ("ws", 0x100010)):
        assert append(**{name: ptr(at)}) == -3, name
    assert append(cache(batch=0)) == 0


def attention(c=None, **over):
    lib = binding.load_library()
    a = dict(q=ptr(), qs=(ctypes.c_int64 * 2)(256, 64), heads=4, pre=ptr(), plen=20, cu=ptr(), total=5, G=3,
             scale=0.125, mask=None, out=ptr(), lse=None, ws=ptr(), ws_bytes=1 << 40)
    a.update(over)
    return lib.spec_verify_attention(a["q"], a["qs"], a["heads"], ctypes.byref(c or cache()), a["pre"], a["plen"],
                                     a["cu"], a["total"], a["G"], a["scale"], a["mask"], a["out"], a["lse"],
                                     a["ws"], a["ws_bytes"], None)


def test_attention_refusals():
    for bad in BAD_CACHES:
        assert attention(cache(**bad)) == -1, bad
    for bad in NULL_CACHES:
        assert attention(cache(**bad)) == -2, bad
    for bad in OFF_CACHES:
        assert attention(cache(**bad)) == -3, bad
    for bad in (dict(total=-1), dict(G=-1), dict(heads=0), dict(heads=5), dict(heads=258), dict(plen=-1),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
                dict(mask=ptr(), G=32), dict(qs=(ctypes.c_int64 * 2)(256, 4)), dict(qs=(ctypes.c_int64 * 2)(0, 64))):
        assert attention(**bad) == -1, bad
    for name in ("q", "qs", "pre", "cu", "out", "ws"):
        assert attention(**{name: None}) == -2, name
    for name, at in (("q", 0x100008), ("out", 0x100008), ("lse", 0x100002), ("mask", 0x100002), ("pre", 0x100002),
                     ("ws", 0x100010)):
        assert attention(**{name: ptr(at)}) == -3, name
    need = binding.load_library().spec_verify_attention_workspace_size(8, 4, 64)
    assert attention(ws_bytes=need - 1) == -4
    assert attention(cache(batch=0)) == 0


def test_attention_refuses_prefixes_whose_places_pass_32_bits():
    # the most goes on to the next check
    for plen in (2 ** 31 - 4096, 2 ** 31 - 1):
        assert attention(plen=plen) == -1
    assert attention(plen=2 ** 31 - 4097, ws_bytes=0) == -4


def test_attention_refuses_an_output_within_the_queries():
    # 8 rows of 4 heads of 64, 256 a row: 4096 bytes of q and of out; wider q rows reach further
    for out in (0x100000, 0x100ff0, 0xff010):
        assert attention(out=ptr(out)) == -3, hex(out)
    assert attention(out=ptr(0x101000), qs=(ctypes.c_int64 * 2)(512, 64)) == -3


def test_attention_workspace_size():
    size = binding.load_library().spec_verify_attention_workspace_size
    assert size(1, 1, 8) > 0 and size(8, 4, 64) % 256 == 0
    assert size(1000, 32, 128) > size(10, 32, 128) > size(10, 32, 64)
    for bad in ((-1, 4, 64), (1, 0, 64), (1, 4, 60), (1, 4, 136), (1, 4, 0)):
        assert size(*bad) == 0


def test_binding_refuses_cpu_tensors_and_shapes():
    z = torch.zeros
    with pytest.raises(TypeError):
        binding.PagedCache(z(4, 16, 2, 64).bfloat16(), z(4, 16, 2, 64).bfloat16(), z(1, 4).int(), z(1).int())
    with pytest.raises(TypeError):
        binding.spec_verify_sample_probs(z(1, 2, 8), z(1, 1, 8), z(1, 1).int(), z(1).int(), z(1, 2), z(1, 2).int(),
                                         z(1).int(), z(256).byte())


# ---------------------------------------------------------------------------
# Rotary frequencies
# ---------------------------------------------------------------------------
def test_fixed_point_holds_the_exact_turns():
    """f 2^64 / (2 pi), rounded: checked against pi to 50 digits."""
    from decimal import Decimal, getcontext
    getcontext().prec = 80
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    f = torch.cat([rope.frequencies(128, 500000.0), torch.tensor([0.0, 7.5, -1.25, 1e-12, 1e6], dtype=torch.float64)])
    for x, t in zip(f.tolist(), rope.fixed_point(f).tolist()):
        want = Decimal(x) / two_pi * 2 ** 64
        diff = (Decimal(t) - want) % (1 << 64)
        assert min(diff, (1 << 64) - diff) <= Decimal("0.5") + Decimal("1e-9")


def test_frequencies():
    f = rope.frequencies(8, 10000.0)
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-14)
    assert torch.allclose(rope.frequencies(8, scaling="linear", factor=4.0), f / 4, rtol=1e-14)
    n = rope.frequencies(8, scaling="ntk", factor=4.0)
    assert n[0] == 1.0 and math.isclose(n[-1], f[-1] / 4, rel_tol=1e-12)
    b = rope.frequencies(128, scaling="by_parts", factor=8.0, trained_len=4096)
    full = rope.frequencies(128)
    turns = full * 4096 / (2 * math.pi)
    assert torch.equal(b[turns > 40], full[turns > 40])
    assert torch.allclose(b[turns < 0.8], full[turns < 0.8] / 8, rtol=1e-14)
    assert bool((b <= full).all()) and bool((b >= full / 8).all()) and bool((b.diff() < 0).all())
    assert math.isclose(rope.by_parts_scale(8.0), 0.1 * math.log(8.0) + 1.0) and rope.by_parts_scale(1.0) == 1.0
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, factor=0.5), dict(rot_dim=8, base=1.0),
                dict(rot_dim=8, scaling="other"), dict(rot_dim=2, scaling="ntk"),
                dict(rot_dim=8, scaling="by_parts", trained_len=0)):
        with pytest.raises(ValueError):
            rope.frequencies(**bad)
    for bad in (torch.tensor([math.inf]), torch.ones(2, 2)):
        with pytest.raises(ValueError):
            rope.fixed_point(bad)


@pytest.mark.parametrize("rot, base, factor, trained", [(128, 10000.0, 4.0, 131072), (64, 10000.0, 8.0, 131072),
                                                         (128, 500000.0, 16.0, 1 << 23), (64, 10000.0, 8.0, 1 << 30),
                                                         (128, 10000.0, 4.0, 4096), (32, 10000.0, 2.0, 40)])
def test_by_parts_where_every_pair_turns_often(rot, base, factor, trained):
    """Beyond trained_len = 2 pi base beta_slow the ramp ends behind the last pair: a pair
    that turns more than beta_slow times is never divided by the whole factor."""
    f0, f = rope.frequencies(rot, base), rope.frequencies(rot, base, "by_parts", factor, trained)
    turns = f0 * trained / (2 * math.pi)
    part = (1 - f / f0) / (1 - 1 / factor)  # the ramp: 0 stays, 1 takes the whole factor
    assert bool((part[turns >= 32.0].abs() < 1e-12).all())
    assert bool((part[turns > 1.0] < 1 - 1e-6).all())
    assert bool(((part[turns <= 1.0] - 1).abs() < 1e-12).all())
    # linear between the pairs (whole numbers) that turn at least 32 times and at most once
    per_pair = math.log(base) * 2 / rot
    lo = max(0, math.floor(math.log(trained / (2 * math.pi * 32.0)) / per_pair))
    hi = math.ceil(math.log(trained / (2 * math.pi)) / per_pair)
    for i in range(rot // 2):
        assert math.isclose(part[i], min(max((i - lo) / (hi - lo), 0.0), 1.0), rel_tol=1e-9, abs_tol=1e-9)


def test_append_refuses_a_q_out_within_its_inputs():
    """8 rows of 4 heads of 64 (k and v: 2 heads); all of these calls end on the host."""
    def two(*s):
        return (ctypes.c_int64 * 2)(*s)
    # rows of 8 heads: q, k, v at 0, 512 and 768 bytes
    fused = dict(q=ptr(0x100000), qs=two(512, 64), k=ptr(0x100200), ks=two(512, 64), v=ptr(0x100300), vs=two(512, 64))
    far = dict(q=ptr(0x500000), qs=two(256, 64), k=ptr(0x600000), ks=two(128, 64), v=ptr(0x700000), vs=two(128, 64))
    # q_out on itself: row 0's head 1 is row 1's head 0; heads or rows closer than a head
    for s in (two(64, 64), two(192, 64), two(256, 32), two(32, 256), two(0, 64), two(256, 0), two(64, 448),
              two(-64, 64), two(-192, 64)):
        assert append(**far, o=ptr(0x800000), os=s) == -1, tuple(s)
    # within q, shifted or with other strides
    for base, at, s in ((fused, 0x100002, two(512, 64)), (fused, 0x100080, two(512, 64)), (fused, 0x100000, two(256, 64)),
                        (far, 0x500080, two(256, 64)), (far, 0x500000, two(512, 64)), (far, 0x4ff800, two(256, 64)),
                        (far, 0x500e00, two(-256, 64)), (far, 0x500000, two(64, 512))):
        assert append(**base, o=ptr(at), os=s) == -3, (hex(at), tuple(s))
    # within k or v: a window of the rows that reaches into theirs (also around the row's end)
    for at in (0x100100, 0x100180, 0x100200, 0x100280, 0x100300, 0x100380):
        assert append(**fused, o=ptr(at), os=two(512, 64)) == -3, hex(at)
    for at in (0x600000, 0x6003f0, 0x5ffe02, 0x700000):
        assert append(**far, o=ptr(at), os=two(256, 64)) == -3, hex(at)
