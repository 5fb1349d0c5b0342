"""The cache operators where their arguments share memory, their numbers are extreme or their
workspaces are used again: each against the definition, in float64 or exactly."""

import pytest
import torch

from gpu_helpers import check_device, launches_of
from test_gpu_cache_ops import (DENSE, STREAM, Cache, check_evict, check_prefill, check_prefix, draw_mass, grow,
                                i32, offs, queries, run_evict, run_prefill, run_prefix)
from token_sparse_decode_b200 import binding as B
from token_sparse_decode_b200.step import EvictDecodeStep, PrefillStep

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


# ----------------------------------------------------------------------------------- long rows

def long_rows(L, sink=0, window=None):
    """(mean of out / reference - 1, launches) of 640 query rows at the end of L positions, 4 heads on each of 8 KV heads:
    as many CTAs as do not split a row for the SMs' sake.  The keys are small, so that every token weighs about
    1 / L, and the values lie between 1 and 2, at another level in each of the 512 columns."""
    g = torch.Generator(device="cuda").manual_seed(371)
    hkv, d, n = 8, 64, 640
    k, v = (torch.empty((L, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    level = torch.linspace(1, 1.75, hkv * d, device="cuda").view(hkv, d)
    for h in range(hkv):
        k[:, h] = (torch.randn((L, d), generator=g, device="cuda") * 0.05).bfloat16()
        v[:, h] = (torch.rand((L, d), generator=g, device="cuda") * 0.25 + level[h]).bfloat16()
    q = torch.randn((n, 4 * hkv, d), generator=g, device="cuda").bfloat16()
    step = PrefillStep(k, v, i32([0, L]), L, L, 4 * hkv, [DENSE if window is None else STREAM] * hkv, sink, window or 0, 0.1, n)
    out = torch.zeros_like(q)
    got = launches_of(lambda: step(q, i32([0, n]), out))
    check_device()
    rows = torch.tensor([0, 1, 300, 635, 639], device="cuda")
    p, t = (L - n + rows).repeat_interleave(4)[:, None], torch.arange(L, device="cuda")
    hidden = t > p if window is None else (t > p) | ((t >= sink) & (t <= p - window))
    rel = []
    for h in range(hkv):
        x = 0.1 * (q[rows, 4 * h:4 * h + 4].double().reshape(-1, d) @ k[:, h].double().T)  # [rows * 4, L]
        ref = torch.softmax(x.masked_fill(hidden, -float("inf")), 1) @ v[:, h].double()
        rel.append(out[rows, 4 * h:4 * h + 4].double().reshape(-1, d) / ref - 1)
    rel = torch.stack(rel)
    assert float(rel.abs().max()) <= 2 * 2.0 ** -8  # the rounding of the output and of its weights, a half step each
    return float(rel.mean()), got


@pytest.mark.parametrize("L,sink,window", [(100_000, 0, None), (300_000, 0, None), (300_000, 128, 280_000), (1_000_000, 0, None)])
def test_prefill_of_long_rows_does_not_drift(L, sink, window):
    """The product with V drops the bits below the accumulator's last, always towards zero: less than 2^-23 of it per
    16 tokens, on 131072 tokens at most.  Weights and outputs are rounded to nearest: a column's outputs are
    nearly the same and share their rounding, at most 2^-8 and 2^-8 / sqrt(3) in the mean square, so that the mean
    over 512 columns stays within 4 x 1.0e-4 (four standard deviations).  A quarter of the weights come from a
    cubic within 1e-4, in the row's sum as well."""
    drift, got = long_rows(L, sink, window)
    assert got == {"tile_attend_kernel": 1}
    assert -(min(L, 131072) / 16 * 2.0 ** -23 + 5e-4) <= drift <= 5e-4, drift


@pytest.mark.parametrize("rows,launches", [(360, {"tile_attend_kernel": 1, "tile_merge_kernel": 1}), (600, {"tile_attend_kernel": 1})])
def test_prefill_of_long_rows_whose_maxima_grow(rows, launches):
    # two CTAs of more than 131072 tokens per row, or one of all; beside them short rows and one that sees nothing
    c = Cache(381, [300_000, 40, 0, 3000], 1, 64, room=3)
    grow(c)
    new = [5, 40, 2, rows]
    q = queries(382, sum(new) + 2, 32, 64)
    kv = c.kv()
    ws = B.workspace(B.stream_prefill_workspace_size(kv, 32, q.shape[0], [DENSE], 0, 0), "cuda").fill_(255)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    assert launches_of(lambda: B.stream_prefill(q.cuda(), kv, i32(offs(new)), [DENSE], 0, 0, 0.4, out, ws)) == launches
    check_device()
    check_prefill(c, q, new, [DENSE], 0, 0, 0.4, out.cpu(), rows=(0, 39, 150))


def test_prefill_of_short_rows_in_a_cache_that_may_hold_long_ones():
    c = Cache(383, [40, 2500, 1], 1, 64)
    new = [40, 700, 1]
    q = queries(384, sum(new) + 3, 32, 64)
    kv = c.kv()
    kv.max_len = 1 << 20
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    ws = B.workspace(B.stream_prefill_workspace_size(kv, 32, q.shape[0], [DENSE], 0, 0), "cuda").fill_(255)
    assert launches_of(lambda: B.stream_prefill(q.cuda(), kv, i32(offs(new)), [DENSE], 0, 0, 0.1, out, ws)) == {
        "tile_attend_kernel": 1}
    check_device()
    check_prefill(c, q, new, [DENSE], 0, 0, 0.1, out.cpu(), rows=(0, 39, 300, 699))
    again = torch.full_like(out, 7.0)
    kv.max_len = c.max_len  # no room for partials asked for, and none used
    B.stream_prefill(q.cuda(), kv, i32(offs(new)), [DENSE], 0, 0, 0.1, again, ws)
    assert torch.equal(out, again)


# ----------------------------------------------------------------------------------- bounded cache

def test_bounded_decode_captured_over_a_whole_cycle():
    """Two equal steps, one eager, one captured from a full buffer over 2 * slack calls and replayed."""
    slack, nb, hq, hkv, d = 3, 2, 4, 2, 64
    steps = [EvictDecodeStep(nb, hq, hkv, d, 1e4, 12, slack, 2, 4, 0.125, 0.9) for _ in range(2)]
    new = [tuple(queries(400 + 3 * i + k, nb, h, d).cuda() for k, h in enumerate((hq, hkv, hkv))) for i in range(30)]
    it = 0
    while not (steps[0].held == steps[0].cap and steps[0].cur == 0 and it > slack):
        for s in steps:
            s(*new[it])
        it += 1
    eager, captured = steps
    static = [tuple(torch.zeros_like(x) for x in new[0]) for _ in range(2 * slack)]
    outs = [torch.zeros_like(captured.out) for _ in range(2 * slack)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        for x, o in zip(static, outs):
            o.copy_(captured(*x))
    assert captured.held == captured.cap and captured.cur == 0
    for _ in range(2):
        for i, x in enumerate(static):
            for a, b in zip(x, new[it + i]):
                a.copy_(b)
        graph.replay()
        for i in range(2 * slack):
            assert torch.equal(eager(*new[it + i]), outs[i])
        it += 2 * slack
        assert torch.equal(eager.positions, captured.positions) and torch.equal(eager.mass, captured.mass)
        assert torch.equal(eager.k[eager.cur], captured.k[captured.cur])
    check_device()
