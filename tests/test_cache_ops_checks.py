"""More host-side checks of the cache operators (no device needed)."""

import re
from pathlib import Path

import numpy as np
import pytest
import torch

from test_cache_ops_refusals import INVALID, WS, accum, evict, kv, lib, other, prefill, prefix  # noqa: F401 (lib: fixture)
from token_sparse_decode_b200 import binding as B
from token_sparse_decode_b200.step import EvictDecodeStep


def empty(**kw):
    return kv(**{"k": None, "v": None, "total_tokens": 0, "max_len": 0, **kw})


def test_a_cache_without_rows_needs_no_address(lib):
    # the arguments pass: the missing workspace is what is refused
    assert accum(lib, empty(), mo=None, ws=None) == WS
    assert prefix(lib, kv(), empty(), ws=None) == WS and prefix(lib, empty(), kv(), ws=None) == WS
    assert evict(lib, empty(), other(), mass=None, ws=None) == WS and evict(lib, kv(), empty(), ws=None) == WS
    assert lib.aoh_accum_decode_workspace_size(empty(), 32) > 0
    # with rows it does
    for gone in ("k", "v"):
        bad = kv(**{gone: None})
        assert accum(lib, bad) == INVALID and prefill(lib, bad) == INVALID
        assert prefix(lib, bad, kv()) == INVALID and prefix(lib, kv(), bad) == INVALID
        assert evict(lib, bad, other()) == INVALID and evict(lib, kv(), other(**{gone: None})) == INVALID


def test_accumulated_weights_overlap_wholly_or_not_at_all(lib):
    n = 4 * 8 * 2000  # bytes
    for mi in (0x100000 - n + 4, 0x100000 - 4, 0x100000 + 4, 0x100000 + n - 4):
        assert accum(lib, kv(), mi=mi, mo=0x100000) == INVALID, hex(mi)
    for mi in (None, 0x100000 - n, 0x100000, 0x100000 + n):  # the workspace is what is refused
        assert accum(lib, kv(), mi=mi, mo=0x100000, ws=None) == WS, mi


@pytest.mark.parametrize("budget,sink,recent", [(64, 40, 25), (0, 0, 0), (64, -1, 4), (64, 4, -1)])
def test_bounded_decode_refuses_a_budget_that_eviction_would_refuse(budget, sink, recent):
    with pytest.raises(ValueError):
        EvictDecodeStep(2, 8, 2, 64, 1e4, budget, 8, sink, recent, 0.1)


def test_the_cubic_of_the_tile_softmax_against_exp2():
    """2^f on [-1/2, 1/2] with the kernel's constants, in fp32 as the kernel adds it up, against exp2: within 2^-13.2
    (the fit's 2^-13.3 and three roundings of 2^-24)."""
    src = (Path(__file__).parent.parent / "token_sparse_decode_b200" / "csrc" / "tile_attend.cuh").read_text()
    c1, c2, c3 = (np.float32(re.search(rf"kEx2C{i} = ([0-9.]+)f", src).group(1)) for i in (1, 2, 3))
    f = np.linspace(-0.5, 0.5, 200_001, dtype=np.float32)
    r = c3
    for c in (c2, c1, np.float32(1)):
        r = (np.float64(r) * f + c).astype(np.float32)  # one rounding, as an fma
    err = np.abs(r.astype(np.float64) / np.exp2(f.astype(np.float64)) - 1)
    assert err.max() <= 2.0 ** -13.2 and err[f == 0] == 0


class OnDevice:
    """What make_kv looks at of a CUDA tensor."""

    is_cuda = True

    def __init__(self, dev, dtype, *shape):
        self.dev, self.dtype, self.shape = dev, dtype, shape

    def get_device(self):
        return self.dev

    def stride(self, i=None):
        s = (self.shape[1] * self.shape[2], self.shape[2], 1)
        return s if i is None else s[i]

    def numel(self):
        return int(np.prod(self.shape))

    def data_ptr(self):
        return 0x10000


@pytest.mark.parametrize("wrong", [None, "v", "offsets", "lengths", "k_dom"])
def test_a_cache_is_on_one_device(wrong):
    at = {n: int(n == wrong) for n in ("v", "offsets", "lengths", "k_dom")}
    bf, i32 = torch.bfloat16, torch.int32
    k_dom = OnDevice(at["k_dom"], bf, 2, 10, 16)
    k_dom.is_contiguous = lambda: True
    args = (OnDevice(0, bf, 10, 2, 64), OnDevice(at["v"], bf, 10, 2, 64), OnDevice(at["offsets"], i32, 3), 5, 10, k_dom,
            OnDevice(at["lengths"], i32, 2))
    if wrong is None:
        assert B.make_kv(*args).device == 0
    else:
        with pytest.raises(ValueError, match=wrong):
            B.make_kv(*args)


def test_append_at_checks_the_chunk_table(monkeypatch):
    monkeypatch.setattr(B, "_device", lambda *caches: -1)  # where CPU tensors are
    c = kv()
    row = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    for idom, n_dom in ((torch.zeros((8, 4), dtype=torch.int64), 4), (torch.zeros((8, 3), dtype=torch.int32), 4),
                        (torch.zeros((8, 4), dtype=torch.int32), 2 ** 32 + 4)):
        with pytest.raises(ValueError, match="idom|n_dom"):
            B.kv_append_at(None, row, row, 1e4, c, idom, n_dom, n, n.clone(), None)
