"""Host-side refusals of the prefill, shared-prefix, accumulate and eviction calls (no device needed)."""

import ctypes

import pytest
import torch

from token_sparse_decode_b200 import binding as B
from token_sparse_decode_b200.build import build

INVALID, UNSUP, ALIGN, WS = 1, 2, 3, 4
HUGE = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build()
    return B.lib()


def kv(**kw):
    c = B.KVCache()
    c.k, c.v, c.offsets = 0x10_0000_0000, 0x20_0000_0000, 0x30000
    c.batch, c.n_kv_heads, c.head_dim, c.max_len = 2, 8, 128, 1000
    c.total_tokens, c.stride_tok, c.stride_head = 2000, 8 * 128, 128
    for a, b in kw.items():
        setattr(c, a, b)
    return c


def u8(*vals):
    a = (ctypes.c_uint8 * len(vals))(*vals)
    return a


def ref(c):
    return None if c is None else ctypes.byref(c)


BAD_CACHES = [(dict(head_dim=96), UNSUP), (dict(k=0x10_0000_0008), ALIGN), (dict(stride_tok=8 * 128 + 4), ALIGN),
              (dict(n_kv_heads=0), INVALID), (dict(total_tokens=1 << 31), INVALID), (dict(ring_sink=4, ring_window=60), INVALID),
              (dict(batch=70000), UNSUP), (dict(offsets=None), INVALID)]


def prefill(lib, c, **kw):
    a = dict(q=0x40000, hq=32, qo=0x50000, total=10, roles=u8(*([1, 2] * 4)), sink=4, window=60, scale=0.1, out=0x60000,
             ws=0x70000, n=HUGE)
    a.update(kw)
    r = None if a["roles"] is None else ctypes.cast(a["roles"], ctypes.c_void_p)
    return lib.aoh_stream_prefill(a["q"], a["hq"], ref(c), a["qo"], a["total"], r, a["sink"], a["window"], a["scale"],
                                  a["out"], a["ws"], a["n"], None)


def test_prefill_refusals(lib):
    for bad, st in BAD_CACHES:
        assert prefill(lib, kv(**bad)) == st, bad
    assert prefill(lib, None) == INVALID
    assert prefill(lib, kv(), hq=30) == INVALID
    assert prefill(lib, kv(n_kv_heads=1), hq=33, roles=u8(1)) == UNSUP
    assert prefill(lib, kv(), roles=None) == INVALID
    assert prefill(lib, kv(), roles=u8(0, 1, 2, 3, 1, 1, 1, 1)) == INVALID
    for bad in (dict(sink=-1), dict(window=-1), dict(total=-1), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(q=None), dict(qo=None), dict(out=None)):
        assert prefill(lib, kv(), **bad) == INVALID, bad
    assert prefill(lib, kv(), q=0x40008) == ALIGN
    assert prefill(lib, kv(), out=0x60008) == ALIGN
    assert prefill(lib, kv(batch=0)) == 0 and prefill(lib, kv(), total=0) == 0


def prefix(lib, p, c, **kw):
    a = dict(q=0x40000, hq=32, ss=0x50000, scale=0.1, out=0x60000, ws=0x70000, n=HUGE)
    a.update(kw)
    return lib.aoh_prefix_decode(a["q"], a["hq"], ref(p), a["ss"], ref(c), a["scale"], a["out"], a["ws"], a["n"], None)


def test_prefix_refusals(lib):
    for bad, st in BAD_CACHES:
        assert prefix(lib, kv(**bad), kv()) == st, bad
        assert prefix(lib, kv(), kv(**bad)) == st, bad
    assert prefix(lib, None, kv()) == INVALID and prefix(lib, kv(), None) == INVALID
    assert prefix(lib, kv(batch=0), kv()) == INVALID                 # no prefix
    assert prefix(lib, kv(batch=2), kv(), ss=None) == INVALID        # which sequence continues which?
    assert prefix(lib, kv(n_kv_heads=4), kv()) == INVALID
    assert prefix(lib, kv(head_dim=64), kv()) == INVALID
    slots = u8(0, 1, 2, 3, 4, 5, 6, 255)
    assert prefix(lib, kv(), kv(head_slot=ctypes.cast(slots, ctypes.c_void_p).value)) == INVALID
    for bad in (dict(scale=float("nan")), dict(q=None), dict(out=None)):
        assert prefix(lib, kv(), kv(), **bad) == INVALID, bad
    assert prefix(lib, kv(), kv(), q=0x40008) == ALIGN and prefix(lib, kv(), kv(), out=0x60004) == ALIGN
    assert prefix(lib, kv(), kv(batch=0)) == 0


def accum(lib, c, **kw):
    a = dict(q=0x40000, hq=32, scale=0.1, decay=1.0, mi=None, mo=0x50000, out=0x60000, ws=0x70000, n=HUGE)
    a.update(kw)
    return lib.aoh_accum_decode(a["q"], a["hq"], ref(c), a["scale"], a["decay"], a["mi"], a["mo"], a["out"], a["ws"],
                                a["n"], None)


def test_accum_refusals(lib):
    for bad, st in BAD_CACHES:
        assert accum(lib, kv(**bad)) == st, bad
    for bad in (dict(scale=float("nan")), dict(decay=float("inf")), dict(q=None), dict(mo=None), dict(out=None)):
        assert accum(lib, kv(), **bad) == INVALID, bad
    assert accum(lib, kv(), out=0x60004) == ALIGN
    need = lib.aoh_accum_decode_workspace_size(ref(kv()), 32)
    assert need >= 8 * 2000 * 4 * 4 and need % 256 == 0
    assert accum(lib, kv(), n=need - 1) == WS and accum(lib, kv(), ws=None) == WS and accum(lib, kv(), ws=0x70010) == WS
    assert lib.aoh_accum_decode_workspace_size(ref(kv(head_dim=96)), 32) == 0
    assert accum(lib, kv(batch=0)) == 0


def evict(lib, s, d, **kw):
    a = dict(mass=0x40000, budget=64, sink=4, recent=16, dl=0x50000, dm=None, idx=0x60000, count=0x68000, ws=0x70000, n=HUGE)
    a.update(kw)
    return lib.aoh_cache_evict(ref(s), a["mass"], a["budget"], a["sink"], a["recent"], ref(d), a["dl"], a["dm"], a["idx"],
                               a["count"], a["ws"], a["n"], None)


def other(**kw):
    return kv(**{"k": 0x50_0000_0000, "v": 0x60_0000_0000, **kw})


def test_evict_refusals(lib):
    for bad, st in BAD_CACHES:
        assert evict(lib, kv(**bad), other()) == st, bad
        b = dict(bad)
        if "k" in b:
            b["k"] = 0x50_0000_0008
        d = other()
        for n, val in b.items():
            setattr(d, n, val)
        assert evict(lib, kv(), d) == st, bad
    assert evict(lib, None, other()) == INVALID and evict(lib, kv(), None) == INVALID
    assert evict(lib, kv(), other(batch=1)) == INVALID and evict(lib, kv(), other(head_dim=64)) == INVALID
    for bad in (dict(budget=0), dict(sink=-1), dict(recent=-1), dict(sink=40, recent=25), dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1),
                dict(mass=None), dict(dl=None), dict(idx=None), dict(count=None)):
        assert evict(lib, kv(), other(), **bad) == INVALID, bad
    assert evict(lib, kv(), kv()) == INVALID                                   # the same memory
    assert evict(lib, kv(), other(v=0x10_0000_0000 + 2 * 1024 * 1999)) == INVALID  # dst V begins inside src K
    assert evict(lib, kv(), other(), dm=0x40000 + 4 * 8 * 2000 - 4) == INVALID  # the masses overlap
    need = lib.aoh_cache_evict_workspace_size(ref(kv()))
    assert need > 0 and evict(lib, kv(), other(), n=need - 1) == WS and evict(lib, kv(), other(), ws=None) == WS
    assert evict(lib, kv(batch=0), other(batch=0)) == 0
    assert evict(lib, kv(max_len=5_000_000), other()) == UNSUP


def test_append_at_refusals(lib):
    def call(c, positions=0x58000, lengths=0x50000):
        return lib.aoh_kv_append_at(None, 0, 0x40000, 0x48000, 1e4, ref(c), None, 0, lengths, positions, None, None)

    assert call(None) == INVALID and call(kv(), positions=None) == INVALID and call(kv(), lengths=None) == INVALID
    assert call(kv(ring_sink=1, ring_window=4)) == INVALID
    assert call(kv(batch=0), positions=None) == 0


def test_binding_checks_tensors():
    c = kv()
    bf, f = torch.zeros((2, 32, 128), dtype=torch.bfloat16), torch.zeros((2, 32, 128))
    ws = torch.zeros(16, dtype=torch.uint8)
    for call in (lambda: B.stream_prefill(f, c, None, [1] * 8, 0, 0, 0.1, bf, ws),
                 lambda: B.prefix_decode(bf[:, :, :64], c, None, c, 0.1, f, ws),
                 lambda: B.accum_decode(bf[:1], c, 0.1, 1.0, None, f, f, ws),
                 lambda: B.cache_evict(c, f, 4, 0, 0, c, None, None, None, None, ws)):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_ints_that_would_be_cut():
    for name in ("sink", "window"):
        with pytest.raises(ValueError):
            B._int32("x", **{name: 2 ** 32})
    B._int32("x", sink=2 ** 31 - 1, window=-2 ** 31)


def test_prefill_workspace_is_monotone(lib):
    r = ctypes.cast(u8(*([1, 2] * 4)), ctypes.c_void_p)
    c = kv(max_len=100000, total_tokens=200000)
    sizes = [lib.aoh_stream_prefill_workspace_size(ref(c), 32, n, r, 4, 5000) for n in (1, 2, 50, 300, 1000, 9000, 100000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert prefill(lib, c, total=1, n=sizes[0] // 4) == WS
    assert lib.aoh_stream_prefill_workspace_size(ref(kv(head_dim=96)), 32, 1, r, 4, 5000) == 0
