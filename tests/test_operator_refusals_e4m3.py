"""Arguments that the operators of an 8-bit cache and of a cache's pages refuse on the host,
before any launch (CPU only: every call here ends with an error, or without rows)."""
import ctypes
import math

import pytest

from speculative_decoding_verification_62_gb300 import binding

two = ctypes.c_int64 * 2
three = ctypes.c_int64 * 3


def ptr(addr=0x100000):
    return ctypes.c_void_p(addr)


def cache(**over):
    c = binding._KvCache(0x100000, 0x200000, binding.SV_E4M3, 10, 16, 2, 64, three(2048, 128, 64), three(2048, 128, 64),
                         0x300000, 4, 3, 0x400000)
    for k, v in over.items():
        setattr(c, k, three(*v) if k.endswith("strides") else v)
    return c


def scales(k=0x500000, v=0x600000, block=16):
    return binding._KvScales(k, v, block)


def ref(x):
    return None if x is None else ctypes.byref(x)


BAD_CACHES = [dict(dtype=0), dict(dtype=1), dict(dtype=2), dict(dtype=4), dict(num_pages=0), dict(page_size=8),
              dict(page_size=24), dict(page_size=8192), dict(kv_heads=0), dict(head_dim=0), dict(head_dim=56),
              dict(head_dim=144), dict(k_strides=(2048, 128, 8)), dict(v_strides=(0, 128, 64)),
              dict(k_strides=(2048, -128, 64)), dict(v_strides=(2040, 128, 64)), dict(batch=-1), dict(max_pages=-1)]
NULL_CACHES = [dict(k_pages=None), dict(v_pages=None), dict(page_table=None), dict(kv_len=None)]
OFF_CACHES = [dict(k_pages=0x100008), dict(v_pages=0x100002), dict(kv_len=0x400002), dict(page_table=0x300001)]
BAD_SCALES = [(dict(block=0), -1), (dict(block=3), -1), (dict(block=32), -1), (dict(block=256), -1), (dict(block=-16), -1),
              (dict(k=None), -2), (dict(v=None), -2), (dict(k=0x500002), -3), (dict(v=0x600001), -3)]


def append(c=None, s=None, **over):
    a = dict(q=ptr(0x1000000), qs=two(512, 64), heads=4, k=ptr(0x2000000), ks=two(512, 64), v=ptr(0x3000000),
             vs=two(512, 64), dtype=1, o=ptr(0x4000000), os=two(512, 64), cu=ptr(), total=5, G=3, freq=ptr(), rot=64,
             inter=0, scale=1.0, pos=None, off=0, ws=ptr(), ws_bytes=256)
    a.update(over)
    return binding.load_library().spec_verify_kv_append_e4m3(
        a["q"], a["qs"], a["heads"], a["k"], a["ks"], a["v"], a["vs"], a["dtype"], a["o"], a["os"], ref(c or cache()),
        ref(s or scales()), a["cu"], a["total"], a["G"], a["freq"], a["rot"], a["inter"], a["scale"], a["pos"], a["off"],
        a["ws"], a["ws_bytes"], None)


def attention(c=None, s=None, **over):
    a = dict(q=ptr(0x1000000), qs=two(256, 64), heads=4, dtype=1, pre=ptr(), plen=20, cu=ptr(), total=5, G=3, scale=0.125,
             mask=None, out=ptr(0x4000000), lse=None, ws=ptr(), ws_bytes=1 << 40)
    a.update(over)
    return binding.load_library().spec_verify_attention_e4m3(
        a["q"], a["qs"], a["heads"], a["dtype"], ref(c or cache()), ref(s or scales()), a["pre"], a["plen"], a["cu"],
        a["total"], a["G"], a["scale"], a["mask"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)


def pool(**over):
    p = binding._PagePool(0x700000, 0x800000, 0x900000, 0xa00000)
    for k, v in over.items():
        setattr(p, k, v)
    return p


def step(c=None, s=None, p=None, **over):
    a = dict(parents=ptr(), tokens=ptr(), ws=ptr(), ws_bytes=1 << 30)
    a.update(over)
    return binding.load_library().spec_verify_pages_step(ref(c or cache()), ref(s or scales()), ref(p or pool()),
                                                         a["parents"], a["tokens"], a["ws"], a["ws_bytes"], None)


def compact(c=None, s=None, p=None, **over):
    a = dict(remap=ptr(), ws=ptr(), ws_bytes=1 << 30)
    a.update(over)
    return binding.load_library().spec_verify_pages_compact(ref(c or cache()), ref(s or scales()), ref(p or pool()),
                                                            a["remap"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("call", [append, attention, step, compact])
def test_bad_caches_and_scales(call):
    for bad in BAD_CACHES:
        if call in (step, compact) and bad.get("dtype") in (1, 2):
            continue  # (caches of 16 bits are theirs too)
        assert call(cache(**bad)) == -1, bad
    for bad in NULL_CACHES:
        assert call(cache(**bad)) == -2, bad
    for bad in OFF_CACHES:
        assert call(cache(**bad)) == -3, bad
    for bad, code in BAD_SCALES:
        assert call(None, scales(**bad)) == code, bad


def test_append_refusals():
    for bad in (dict(dtype=0), dict(dtype=3), dict(total=-1), dict(G=-1), dict(heads=-1), dict(rot=63), dict(rot=66),
                dict(rot=-2), dict(inter=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
                dict(total=2 ** 31 - 2), dict(total=2 ** 31 - 1000), dict(total=2 ** 31 - 4099)):
        assert append(**bad) == -1, bad
    assert append(total=2 ** 31 - 4100, ws_bytes=2) == -4  # (the most goes on to the next check)
    for name in ("q", "qs", "k", "ks", "v", "vs", "o", "os", "cu", "freq", "ws"):
        assert append(**{name: None}) == -2, name
    lib = binding.load_library()
    assert lib.spec_verify_kv_append_e4m3(*[None] * 2, 0, *[None] * 4, 1, *[None] * 3, ref(scales()), None, 0, 0, None, 0, 0,
                                          1.0, None, 0, None, 0, None) == -2
    assert append(ws_bytes=2) == -4
    for name, at in (("q", 0x1000001), ("k", 0x2000001), ("v", 0x3000001), ("o", 0x4000001), ("freq", 0x100004),
                     ("cu", 0x100002), ("pos", 0x100002), ("ws", 0x100010)):
        assert append(**{name: ptr(at)}) == -3, name
    # q_out on itself, within q but not q, within k or v
    for s in (two(64, 64), two(192, 64), two(512, 32), two(0, 64)):
        assert append(os=s) == -1, tuple(s)
    for at in (0x1000002, 0x1000080, 0x2000000, 0x2000080, 0x3000000):
        assert append(o=ptr(at)) == -3, hex(at)
    assert append(o=ptr(0x1000000), os=two(256, 64)) == -3
    assert append(cache(batch=0)) == 0


def test_attention_refusals():
    for bad in (dict(dtype=0), dict(dtype=3), dict(total=-1), dict(G=-1), dict(heads=0), dict(heads=5), dict(heads=65538),
                dict(plen=-1), dict(plen=2 ** 31 - 4096), dict(plen=2 ** 31 - 1), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=math.nan), dict(scale=math.inf), dict(scale=3e38), dict(mask=ptr(), G=32), dict(qs=two(256, 4)),
                dict(qs=two(0, 64)), dict(total=2 ** 30, heads=8)):
        assert attention(**bad) == -1, bad
    for name in ("q", "qs", "pre", "cu", "out", "ws"):
        assert attention(**{name: None}) == -2, name
    for name, at in (("q", 0x1000008), ("out", 0x4000008), ("lse", 0x100002), ("mask", 0x100002), ("pre", 0x100002),
                     ("cu", 0x100002), ("ws", 0x100010)):
        assert attention(**{name: ptr(at)}) == -3, name
    # 8 rows of 4 heads of 64: 4096 bytes of q and of out; wider q rows reach further
    for out in (0x1000000, 0x1000ff0, 0xfff010):
        assert attention(out=ptr(out)) == -3, hex(out)
    assert attention(out=ptr(0x1001000), qs=two(512, 64)) == -3
    size = binding.load_library().spec_verify_attention_e4m3_workspace_size
    assert attention(ws_bytes=size(8, 4, 64) - 1) == -4
    assert attention(cache(batch=0)) == 0
    assert size(1, 1, 16) > 0 and size(8, 4, 64) % 256 == 0
    for bad in ((-1, 4, 64), (1, 0, 64), (1, 65536, 64), (1, 4, 56), (1, 4, 144), (1, 4, 0)):
        assert size(*bad) == 0


def test_page_refusals():
    lib = binding.load_library()
    size = lib.spec_verify_pages_workspace_size
    for call in (step, compact):
        assert call(cache(dtype=3), None, pool(ref=None)) == -2
        for name in ("held", "ref", "free_pages", "free_count"):
            assert call(None, None, pool(**{name: None})) == -2, name
            assert call(None, None, pool(**{name: 0x700002})) == -3, name
        assert call(cache(max_pages=0)) == -1
        assert call(cache(max_pages=2 ** 30, batch=3)) == -1
        assert call(cache(max_pages=2 ** 20, page_size=4096)) == -1
        assert call(ws=None) == -2 and call(ws=ptr(0x100010)) == -3
        assert call(ws_bytes=size(10, 3, 4) - 1) == -4
    assert step(tokens=None) == -2 and step(tokens=ptr(0x100002)) == -3 and step(parents=ptr(0x100002)) == -3
    assert compact(remap=None) == -2 and compact(remap=ptr(0x100002)) == -3
    assert lib.spec_verify_pages_step(None, ref(scales()), ref(pool()), None, ptr(), ptr(), 1 << 30, None) == -2
    assert lib.spec_verify_pages_step(ref(cache()), None, ref(pool()), None, ptr(), ptr(), 1 << 30, None) == -2
    assert lib.spec_verify_pages_step(ref(cache()), ref(scales()), None, None, ptr(), ptr(), 1 << 30, None) == -2
    assert step(cache(batch=0)) == 0
    # a compaction of no rows reads the pools all the same
    for bad in (dict(k_pages=None), dict(v_pages=None)):
        assert compact(cache(batch=0, **bad)) == -2
    assert compact(cache(batch=0, k_pages=0x100008)) == -3
    assert compact(cache(batch=0), scales(k=None)) == -2 and compact(cache(batch=0), scales(v=0x600002)) == -3
    assert compact(cache(batch=0), None, pool(ref=None)) == -2
    for bad in ((0, 3, 4), (10, -1, 4), (10, 3, 0), (10, 2 ** 30, 4)):
        assert size(*bad) == 0
    assert size(10, 3, 4) > 0 and size(10, 0, 4) > 0 and size(1000, 3, 4) > size(10, 3, 4)
