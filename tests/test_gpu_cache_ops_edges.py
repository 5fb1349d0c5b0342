"""The cache operators where their arguments share memory, their numbers are extreme or their
workspaces are used again: each against the definition, in float64 or exactly."""

import pytest
import torch

from gpu_helpers import check_device, launches_of
from test_gpu_cache_ops import (DENSE, STREAM, Cache, check_evict, check_prefill, check_prefix, draw_mass, i32, queries,
                                run_evict, run_prefill, run_prefix)
from token_sparse_decode_b200 import binding as B

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------------- eviction

def test_evict_with_one_lengths_array_for_both_caches():
    # far more copy blocks than run at once: those that start late must keep what the first ones keep
    c = Cache(301, [2500 + 11 * b for b in range(64)], 4, 64)
    budget, sink, recent = 1000, 4, 100
    mass = draw_mass(302, 4, c.T, "plain")
    dst = Cache(303, [0] * 64, 4, 64, room=budget)
    dst.max_len = budget
    lengths = i32(c.lens)  # the source's, and written as the destination's
    src = B.make_kv(c.k, c.v, c.offsets, c.max_len, c.T, lengths=lengths)
    dst.k.fill_(5.0)
    dst.v.fill_(6.0)
    res = dict(dst=dst, idx=torch.full((64, 4, budget), -7, dtype=torch.int32, device="cuda"),
               count=torch.full((64, 4), -7, dtype=torch.int32, device="cuda"),
               mass=torch.full((4, dst.T), 7.0, device="cuda"), lengths=lengths)
    ws = B.workspace(B.cache_evict_workspace_size(src), "cuda")
    B.cache_evict(src, mass.cuda(), budget, sink, recent, dst.kv(), lengths, res["mass"], res["idx"], res["count"], ws)
    torch.cuda.synchronize()
    check_device()
    check_evict(c, mass, budget, sink, recent, res)


def test_evict_of_very_long_rows_on_a_workspace_that_served_another_cache():
    # more than 262144 positions: scores and histograms in the workspace, at places that depend on the cache
    kinds, ws = ("special", "ties", "plain"), None
    for i, (lens, hkv) in enumerate((([300_000], 2), ([270_000, 9], 1), ([290_000], 1))):
        c = Cache(311 + i, lens, hkv, 64)
        mass, dst = draw_mass(315 + i, hkv, c.T, kinds[i]), Cache(318, [0] * len(lens), hkv, 64, room=4000)
        dst.max_len = 4000
        dst.k.fill_(5.0)
        dst.v.fill_(6.0)
        need = B.cache_evict_workspace_size(c.kv())
        if ws is None:
            ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        assert need <= ws.numel()
        res = dict(dst=dst, idx=torch.full((len(lens), hkv, 4000), -7, dtype=torch.int32, device="cuda"),
                   count=torch.full((len(lens), hkv), -7, dtype=torch.int32, device="cuda"),
                   mass=torch.full((hkv, dst.T), 7.0, device="cuda"), lengths=i32([-7] * len(lens)))
        got = launches_of(lambda: B.cache_evict(c.kv(), mass.cuda(), 4000, 4, 500, dst.kv(), res["lengths"], res["mass"],
                                                res["idx"], res["count"], ws))
        check_device()
        assert got["evict_key_kernel"] == got["select_hist_kernel"] == got["select_write_kernel"] == 1
        check_evict(c, mass, 4000, 4, 500, res)


@pytest.mark.parametrize("L", [200, 140_000, 270_000])  # the cluster select, and the two selects of longer rows
def test_evict_takes_an_infinite_weight_before_the_largest_finite_one(L):
    c = Cache(321, [L], 1, 64)
    mass = torch.full((1, L), torch.finfo(torch.float32).max)
    mass[0, 100:110] = float("inf")
    mass[0, 150:160] = -float("inf")
    for budget, sink, recent in ((13, 2, 1), (13, 0, 0), (12, 6, 6)):
        res = run_evict(c, mass, budget, sink, recent, budget)
        check_device()
        check_evict(c, mass, budget, sink, recent, res)


def test_evict_clears_the_weights_of_a_region_too_small():
    # what is appended to the empty sequence later must not add to weights of tokens that are gone
    c = Cache(331, [10, 100, 20], 2, 64)
    mass = draw_mass(332, 2, c.T, "plain")
    res = run_evict(c, mass, 50, 1, 1, 30)
    st, detail = B.device_check()
    assert st == 6 and detail == [4, 1, 50, 30] and res["lengths"].tolist() == [10, 0, 20]
    off = res["dst"].off
    assert bool((res["mass"][:, off[1]:off[2]] == 0).all())
    for b in (0, 2):
        n = c.lens[b]
        assert torch.equal(res["mass"][:, off[b]:off[b] + n].cpu(), mass[:, c.off[b]:c.off[b] + n])
        assert bool((res["mass"][:, off[b] + n:off[b + 1]] == 0).all())


# ----------------------------------------------------------------------------------- caches without rows

def no_rows(batch, hkv, d):
    """A cache whose tensors have no elements (and so no address)."""
    k = torch.empty((0, hkv, d), dtype=torch.bfloat16, device="cuda")
    return B.make_kv(k, torch.empty_like(k), i32([0] * (batch + 1)), 0, 0)


@pytest.mark.parametrize("nb", [3, 70])  # the dense pass alone, and tiles
def test_prefix_decode_when_one_side_has_no_rows(nb):
    full, zero = Cache(341, [700], 2, 128), Cache(342, [0] * nb, 2, 128)
    q = queries(343, nb, 8, 128)
    out = torch.full(q.shape, 7.0, device="cuda")
    own, prefix = no_rows(nb, 2, 128), no_rows(1, 2, 128)
    B.prefix_decode(q.cuda(), full.kv(), None, own, 0.1, out,
                    B.workspace(B.prefix_decode_workspace_size(full.kv(), own, 8), "cuda"))
    check_device()
    check_prefix(full, zero, q, None, 0.1, out.cpu(), seqs=(0, 1, nb - 1))
    c, nothing = Cache(344, [b % 5 for b in range(nb)], 2, 128), Cache(345, [0], 2, 128)
    B.prefix_decode(q.cuda(), prefix, None, c.kv(), 0.1, out,
                    B.workspace(B.prefix_decode_workspace_size(prefix, c.kv(), 8), "cuda"))
    check_device()
    check_prefix(nothing, c, q, None, 0.1, out.cpu(), seqs=(0, 1, nb - 1))
    out.fill_(7.0)
    B.prefix_decode(q.cuda(), prefix, None, own, 0.1, out, B.workspace(B.prefix_decode_workspace_size(prefix, own, 8), "cuda"))
    check_device()
    assert bool((out == 0).all())


def test_the_other_calls_on_a_cache_without_rows():
    kv, q = no_rows(3, 2, 64), queries(351, 3, 4, 64).cuda()
    out, mass = torch.full((3, 4, 64), 7.0, device="cuda"), torch.zeros((2, 0), device="cuda")
    B.accum_decode(q, kv, 0.1, 0.9, mass, mass, out, B.workspace(B.accum_decode_workspace_size(kv, 4), "cuda"))
    assert bool((out == 0).all())
    pout = torch.full_like(q, 7.0)
    B.stream_prefill(q, kv, i32([0, 1, 1, 3]), [DENSE, STREAM], 1, 1, 0.1, pout,
                     B.workspace(B.stream_prefill_workspace_size(kv, 4, 3, [DENSE, STREAM], 1, 1), "cuda"))
    assert bool((pout == 0).all())
    idx, count = torch.zeros((3, 2, 5), dtype=torch.int32, device="cuda"), torch.full((3, 2), 7, dtype=torch.int32, device="cuda")
    lengths, ws = i32([7, 7, 7]), B.workspace(B.cache_evict_workspace_size(kv), "cuda")
    B.cache_evict(kv, mass, 5, 1, 1, no_rows(3, 2, 64), lengths, mass.clone(), idx, count, ws)
    assert lengths.tolist() == [0, 0, 0] and bool((count == 0).all()) and bool((idx == -1).all())
    check_device()
    src = Cache(352, [4, 0, 9], 2, 64)  # rows to keep, and no room
    B.cache_evict(src.kv(), torch.rand((2, src.T), device="cuda"), 5, 1, 1, no_rows(3, 2, 64), lengths, None, idx, count,
                  B.workspace(B.cache_evict_workspace_size(src.kv()), "cuda"))
    st, detail = B.device_check()
    assert st == 6 and detail[0] == 4 and lengths.tolist() == [0, 0, 0]


# ----------------------------------------------------------------------------------- large values

def heavy_late(c, u, gain, values):
    """Two tokens of every sequence, in its middle and near its end, whose logits with the query u stand `gain` and
    1.5 gain above the others'; values scaled by `values`."""
    for b, n in enumerate(c.lens):
        o = c.off[b]
        c.kh[o:o + n] = (c.kh[o:o + n].float() * 0.05).bfloat16()
        for at, f in ((n // 2, 1.0), (n - 1 - n // 9, 1.5)):
            c.kh[o + at] = (u * (f * gain / float(u @ u))).bfloat16()
    c.vh.mul_(values)
    c.k.copy_(c.kh)
    c.v.copy_(c.vh)


@pytest.mark.parametrize("gain", [3.0, 20.0, 27.0])  # 4, 29 and 39 (then 58) powers of two above a row's first tokens
def test_values_near_the_largest_when_maxima_grow(gain):
    u = torch.randn(64, generator=torch.Generator().manual_seed(361))
    big = 2.0 ** 100
    c = Cache(362, [900, 300], 2, 64)
    heavy_late(c, u, gain, big)
    new = [260, 300]
    q = (u + 0.02 * queries(363, sum(new), 4, 64).float()).bfloat16()
    out = run_prefill(c, q, new, [DENSE, STREAM], 4, 200, 1.0)
    assert bool(out[:, :2].isfinite().all())
    check_prefill(c, q, new, [DENSE, STREAM], 4, 200, 1.0, out, rows=(0, 100, 150, 259, 290))
    p, own = Cache(364, [1500], 2, 64), Cache(365, [(5 * b) % 40 for b in range(70)], 2, 64)
    heavy_late(p, u, gain, big)
    own.vh.mul_(big)
    own.v.copy_(own.vh)
    q = (u + 0.02 * queries(366, 70, 4, 64).float()).bfloat16()
    out = run_prefix(p, own, q, None, 1.0)  # tiles and the dense pass
    check_prefix(p, own, q, None, 1.0, out, seqs=(0, 1, 7, 69))
