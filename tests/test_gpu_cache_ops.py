"""Role prefill, shared-prefix decode, accumulated-weight decode and eviction against their
formulas in float64.

Tolerances follow from the arithmetic, per output row: with u = 2^-24, A = sum_t w_t |v_t| and
X = scale * max_t sum_c |q_c k_c|,
  * a logit is an fp32 dot of d exact products: off by at most gamma_{d+8} X, and twice that in a
    weight's exponent difference (a weight is a ratio of two exponentials);
  * exp2 and the scaling of its argument: 2^-21 relative;
  * fp32 sums over L tokens: gamma_{L+64};
  * weights enter the product with V as bf16 (half a step: 2^-8 relative) in the prefill, and as
    hi + lo bf16 parts (2^-16) in the decode calls; bf16 outputs are rounded once (2^-8).
Slots that no row may see hold NaN, and what a call must not write holds a sentinel.
"""

import math

import pytest
import torch

from gpu_helpers import check_device, launches_of
from token_sparse_decode_b200 import binding as B
from token_sparse_decode_b200.step import (AccumDecodeStep, EvictDecodeStep, EvictStep, PrefillStep, PrefixDecodeStep)

pytestmark = pytest.mark.gpu

DENSE, STREAM, SPARSE = B.ROLE_DENSE, B.ROLE_STREAM, B.ROLE_SPARSE
U = 2.0 ** -24


def gamma(n):
    return n * U / (1 - n * U)


def offs(lengths):
    o = [0]
    for n in lengths:
        o.append(o[-1] + n)
    return o


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Cache:
    """A ragged cache with spare room per sequence, NaN in every slot past a length."""

    def __init__(self, seed, lens, hkv, d, room=0, layout="plain", slots=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.d = lens, hkv, d
        self.off = offs([n + room for n in lens])
        T, ns = max(self.off[-1], 1), hkv if slots is None else max([s for s in slots if s != B.NO_SLOT], default=0) + 1
        self.slots = list(range(hkv)) if slots is None else slots
        k = torch.randn((T, ns, d), generator=g)
        v = torch.randn((T, ns, d), generator=g)
        self.kh, self.vh = k.bfloat16(), v.bfloat16()
        for b, n in enumerate(lens):
            if n:
                self.kh[self.off[b]] *= 3  # one heavy token per sequence
            self.kh[self.off[b] + n:self.off[b + 1]] = math.nan
            self.vh[self.off[b] + n:self.off[b + 1]] = math.nan
        if layout == "interleaved":  # K and V rows of a token and head side by side, with a gap
            buf = torch.full((T, ns, 2 * d + 16), math.nan, dtype=torch.bfloat16, device="cuda")
            self.k, self.v = buf[:, :, :d], buf[:, :, d:2 * d]
            self.k.copy_(self.kh)
            self.v.copy_(self.vh)
        elif layout == "head_major":
            self.k = self.kh.transpose(0, 1).contiguous().cuda().transpose(0, 1)
            self.v = self.vh.transpose(0, 1).contiguous().cuda().transpose(0, 1)
        else:
            self.k, self.v = self.kh.cuda(), self.vh.cuda()
        self.offsets, self.lengths = i32(self.off), i32(lens)
        self.T, self.max_len = self.off[-1], max(lens, default=0)

    def kv(self, with_lengths=True):
        return B.make_kv(self.k, self.v, self.offsets, self.max_len, self.T, lengths=self.lengths if with_lengths else None,
                         head_slot=self.slots, n_kv_heads=self.hkv)

    def rows(self, b, g):
        s = slice(self.off[b], self.off[b] + self.lens[b])
        return self.kh[s, self.slots[g]].double(), self.vh[s, self.slots[g]].double()


def attend(q, k, v, seen, scale):
    """(out, weights, A, X) in float64 of one query row over k, v; seen: bool [L]."""
    d = q.shape[0]
    if k.shape[0] == 0 or not bool(seen.any()):
        return torch.zeros(d, dtype=torch.float64), torch.zeros(k.shape[0], dtype=torch.float64), torch.zeros(d), 0.0
    x = scale * (k @ q)
    x[~seen] = -math.inf
    w = torch.softmax(x, 0)
    return w @ v, w, w @ v.abs(), abs(scale) * float((k.abs() @ q.abs())[seen].max())


def weight_rel(d, L, X):
    return 2 * gamma(d + 8) * X + 2.0 ** -21 + gamma(L + 64)


def queries(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


# ----------------------------------------------------------------------------------- prefill

def run_prefill(c, q, new, roles, sink, window, scale, with_lengths=True):
    total = q.shape[0]
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    kv = c.kv(with_lengths)
    ws = B.workspace(B.stream_prefill_workspace_size(kv, q.shape[1], total, roles, sink, window), "cuda")
    qd, qo = q.cuda(), i32(offs(new))
    B.stream_prefill(qd, kv, qo, roles, sink, window, scale, out, ws)
    torch.cuda.synchronize()
    check_device()
    again = torch.full_like(out, 7.0)
    B.stream_prefill(qd, kv, qo, roles, sink, window, scale, again, ws)
    assert torch.equal(out, again)  # the same bits on the same inputs
    return out.cpu()


def check_prefill(c, q, new, roles, sink, window, scale, out, rows=None):
    hkv, G, d = c.hkv, q.shape[1] // c.hkv, c.d
    qoff = offs(new)
    if qoff[-1] < q.shape[0]:
        assert bool((out[qoff[-1]:] == 7.0).all())  # rows behind the last sequence
    for b, n in enumerate(new):
        L = c.lens[b]
        pick = range(n) if rows is None else sorted({i for i in rows if i < n} | {n - 1} - {-1})
        for g in range(hkv):
            if roles[g] == SPARSE or c.slots[g] == B.NO_SLOT:
                assert bool((out[qoff[b]:qoff[b + 1], g * G:(g + 1) * G] == 7.0).all())
                continue
            k, v = c.rows(b, g)
            t = torch.arange(L)
            for i in pick:
                p = L - n + i
                seen = t <= p
                if roles[g] == STREAM:
                    seen &= (t < sink) | (t > p - window)
                for h in range(g * G, (g + 1) * G):
                    ref, _, A, X = attend(q[qoff[b] + i, h].double(), k, v, seen, scale)
                    tol = A * (2 * 2.0 ** -8 * (1 + 2.0 ** -7) + weight_rel(d, L, X)) + 1e-30
                    err = (out[qoff[b] + i, h].double() - ref).abs()
                    assert bool((err <= tol).all()), (b, g, i, h, float((err / tol).max()))


@pytest.mark.parametrize("hkv,G,d", [(4, 1, 64), (2, 4, 128), (1, 7, 128), (2, 5, 64), (1, 32, 128)])
@pytest.mark.parametrize("new,ctx", [((1, 1, 1), (0, 5, 300)), ((5, 0, 33), (0, 7, 100)), ((130, 64), (127, 1)), ((300,), (0,))])
def test_prefill_matches_the_formula(hkv, G, d, new, ctx):
    c = Cache(11, [a + b for a, b in zip(new, ctx)], hkv, d, room=3)
    q = queries(12, sum(new) + 2, hkv * G, d)
    roles = [DENSE if g % 2 == 0 else STREAM for g in range(hkv)]
    scale = 1 / math.sqrt(d)
    out = run_prefill(c, q, new, roles, 4, 60, scale)
    check_prefill(c, q, new, roles, 4, 60, scale, out, rows=(0, 1, 17, 63, 64, 127, 128, 200))


@pytest.mark.parametrize("sink,window", [(0, 0), (0, 1), (1, 0), (4, 60), (0, 128), (128, 129), (130, 5), (1000, 1),
                                         (0, 10 ** 9), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_prefill_windows_and_rows_that_see_nothing(sink, window):
    c = Cache(21, [413, 130, 9], 2, 64)
    new = [270, 129, 9]
    q = queries(22, sum(new), 4, 64)
    out = run_prefill(c, q, new, [STREAM, DENSE], sink, window, 0.125)
    check_prefill(c, q, new, [STREAM, DENSE], sink, window, 0.125, out, rows=(0, 1, 5, 127, 128, 129, 255, 256))
    if sink == 0 and window == 0:
        assert bool((out[:, :2] == 0).all())


def test_prefill_more_queries_than_positions():
    # n_b > L_b: the first rows stand before position 0 and see nothing
    c = Cache(31, [0, 3, 200], 1, 128, room=8)
    new = [2, 6, 201]
    q = queries(32, sum(new), 2, 128)
    out = run_prefill(c, q, new, [DENSE], 0, 0, 0.09)
    check_prefill(c, q, new, [DENSE], 0, 0, 0.09, out)
    assert bool((out[:5] == 0).all()) and bool((out[8] == 0).all())


@pytest.mark.parametrize("layout", ["interleaved", "head_major"])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_layouts_slots_and_roles(layout, d):
    c = Cache(41, [150, 257], 4, d, room=5, layout=layout, slots=[2, B.NO_SLOT, 0, 1])
    new = [150, 40]
    q = queries(42, sum(new), 8, d)
    roles = [STREAM, DENSE, SPARSE, DENSE]
    out = run_prefill(c, q, new, roles, 3, 31, 0.1)
    check_prefill(c, q, new, roles, 3, 31, 0.1, out, rows=(0, 39, 128))


@pytest.mark.parametrize("scale", [0.0, -0.11, 3.0])
def test_prefill_scales(scale):
    c = Cache(51, [200], 1, 64)
    q = queries(52, 200, 3, 64)
    out = run_prefill(c, q, [200], [DENSE], 0, 0, scale)
    check_prefill(c, q, [200], [DENSE], 0, 0, scale, out, rows=(0, 7, 130))


def test_prefill_single_token_equals_stream_decode():
    c = Cache(61, [1, 700, 129], 2, 128, room=1)
    q = queries(62, 3, 8, 128)
    roles, scale = [DENSE, STREAM], 0.09
    out = run_prefill(c, q, [1, 1, 1], roles, 4, 100, scale)
    ref = torch.zeros((3, 8, 128), device="cuda")
    kv = c.kv()
    B.stream_decode(q.cuda(), kv, roles, 4, 100, scale, ref,
                    B.workspace(B.stream_decode_workspace_size(kv, 8, roles, 4, 100), "cuda"))
    torch.cuda.synchronize()
    check_device()
    # both within their tolerances of the exact value; the bf16 one dominates (|out| <= max |v| = A's bound)
    A = float(c.vh[torch.isfinite(c.vh)].abs().max())
    assert float((out.float() - ref.cpu()).abs().max()) <= A * (2.1 * 2.0 ** -8 + 2.0 ** -12)


def test_prefill_in_chunks_equals_the_whole_prompt():
    # a prompt attended in chunks: row for row the tolerance of either side
    c = Cache(71, [513], 2, 128)
    q = queries(72, 513, 4, 128)
    roles = [DENSE, STREAM]
    for n0 in (1, 128, 400):
        part = Cache(71, [513], 2, 128)
        part.lens, part.lengths = [n0], i32([n0])
        out = run_prefill(part, q[:n0], [n0], roles, 4, 77, 0.1)
        check_prefill(part, q[:n0], [n0], roles, 4, 77, 0.1, out, rows=(0, 5, 127))
    out = run_prefill(c, q[400:], [113], roles, 4, 77, 0.1)
    check_prefill(c, q[400:], [113], roles, 4, 77, 0.1, out, rows=(0, 5, 80))


@pytest.mark.parametrize("hkv,G,d", [(2, 4, 128), (1, 7, 64)])
def test_prefill_few_rows_on_a_long_cache(hkv, G, d):
    # few rows: the key range is split over CTAs and joined by a second launch
    new, ctx = [1, 3, 0, 2], [5000, 9000, 40, 0]
    c = Cache(75, [a + b for a, b in zip(new, ctx)], hkv, d, room=1)
    q = queries(76, sum(new) + 1, hkv * G, d)
    for roles, sink, window in (([DENSE] * hkv, 0, 0), ([STREAM] * hkv, 700, 3001)):
        got = {}
        got.update(launches_of(lambda: got.setdefault("out", run_prefill(c, q, new, roles, sink, window, 0.11))))
        assert got["tile_attend_kernel"] == got["tile_merge_kernel"] == 2
        check_prefill(c, q, new, roles, sink, window, 0.11, got["out"])


def test_prefill_step_serves_fewer_rows_than_it_was_built_for():
    c = Cache(86, [9000, 300], 2, 128)
    step = PrefillStep(c.k, c.v, c.offsets, c.max_len, c.T, 8, [DENSE, STREAM], 4, 3000, 0.1, 9300)
    for new in ([1, 1], [3, 40], [700, 300]):
        q = queries(87, sum(new), 8, 128)
        out = step(q.cuda(), i32(offs(new)))
        torch.cuda.synchronize()
        check_device()
        check_prefill(c, q, new, [DENSE, STREAM], 4, 3000, 0.1, out.cpu(), rows=(0, 39, 299))


def test_prefill_workspace_covers_every_smaller_call():
    c = Cache(88, [40000, 9, 9000], 4, 64)
    kv = c.kv()
    for roles, sink, window in (([DENSE] * 4, 0, 0), ([STREAM] * 4, 4, 5000), ([SPARSE] * 3 + [STREAM], 1, 2000)):
        sizes = [B.stream_prefill_workspace_size(kv, 12, n, roles, sink, window) for n in range(1, 4000, 13)]
        assert sizes == sorted(sizes)


def grow(c):
    """Keys that outgrow everything before them, late in every sequence (the reference value has to move)."""
    for b, n in enumerate(c.lens):
        for at, f in ((n // 2, 8.0), (n - n // 5, 30.0)):
            if n > 8:
                c.kh[c.off[b] + at] = (c.kh[c.off[b] + at].float() * f).bfloat16()
    c.k.copy_(c.kh)


def test_prefill_maxima_that_grow_along_the_row():
    c = Cache(77, [700], 2, 128)
    grow(c)
    q = queries(78, 300, 8, 128)
    out = run_prefill(c, q, [300], [DENSE, STREAM], 4, 333, 1.5)
    check_prefill(c, q, [300], [DENSE, STREAM], 4, 333, 1.5, out, rows=(0, 100, 200, 299))


def test_prefill_many_sequences():
    new = [(3 * b) % 4 for b in range(1100)]
    c = Cache(79, [n + (7 * b) % 5 for b, n in enumerate(new)], 1, 64, room=1)
    q = queries(80, sum(new), 2, 64)
    out = run_prefill(c, q, new, [STREAM], 1, 2, 0.2)
    check_prefill(c, q, new, [STREAM], 1, 2, 0.2, out)


def test_prefill_offsets_past_the_rows_are_recorded():
    c = Cache(83, [20], 1, 64)
    q = queries(84, 3, 2, 64).cuda()
    big = torch.full((9, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    kv = c.kv()
    B.stream_prefill(q, kv, i32([0, 5]), [DENSE], 0, 0, 0.1, big[:3],
                     B.workspace(B.stream_prefill_workspace_size(kv, 2, 3, [DENSE], 0, 0), "cuda"))
    st, detail = B.device_check()
    assert st == 6 and detail[0] == 1
    assert bool((big[3:] == 7.0).all())
    for i in range(3):  # the rows that exist stand at L - 5 + i
        k, v = c.rows(0, 0)
        ref = attend(q[i, 0].cpu().double(), k, v, torch.arange(20) <= 15 + i, 0.1)[0]
        assert float((big[i, 0].cpu().double() - ref).abs().max()) <= 2 * 2.0 ** -8 * float(v.abs().max()) + 1e-3


# ----------------------------------------------------------------------------------- shared prefix

def run_prefix(p, c, q, start, scale):
    out = torch.full(q.shape, 7.0, device="cuda")
    pk, kv = p.kv(), c.kv()
    ws = B.workspace(B.prefix_decode_workspace_size(pk, kv, q.shape[1]), "cuda")
    qd, ss = q.cuda(), None if start is None else i32(start)
    B.prefix_decode(qd, pk, ss, kv, scale, out, ws)
    torch.cuda.synchronize()
    check_device()
    again = torch.full_like(out, 7.0)
    B.prefix_decode(qd, pk, ss, kv, scale, again, ws)
    assert torch.equal(out, again)
    return out.cpu()


def check_prefix(p, c, q, start, scale, out, seqs=None):
    G, d = q.shape[1] // c.hkv, c.d
    for b in range(len(c.lens)) if seqs is None else seqs:
        i = 0 if start is None else next(j for j in range(len(start) - 1) if start[j] <= b < start[j + 1])
        for g in range(c.hkv):
            if c.slots[g] == B.NO_SLOT:
                assert bool((out[b, g * G:(g + 1) * G] == 7.0).all())
                continue
            (pk, pv), (k, v) = p.rows(i, g), c.rows(b, g)
            k, v = torch.cat([pk, k]), torch.cat([pv, v])
            L = k.shape[0]
            for h in range(g * G, (g + 1) * G):
                ref, _, A, X = attend(q[b, h].double(), k, v, torch.ones(L, dtype=torch.bool), scale)
                tol = A * (2.0 ** -16 + weight_rel(d, L, X)) + 1e-30
                err = (out[b, h].double() - ref).abs()
                assert bool((err <= tol).all()), (b, h, float((err / tol).max()))


@pytest.mark.parametrize("hkv,G,d", [(4, 1, 64), (2, 4, 128), (1, 7, 128), (2, 5, 64), (1, 32, 128), (1, 17, 64)])
@pytest.mark.parametrize("plen,lens", [(1, (0, 1)), (127, (3, 0, 40)), (128, (5,)), (1000, (200, 1, 0, 33, 64, 65, 17))])
def test_prefix_matches_the_formula(hkv, G, d, plen, lens):
    p, c = Cache(81, [plen], hkv, d, room=2), Cache(82, list(lens), hkv, d, room=1)
    q = queries(83, len(lens), hkv * G, d)
    out = run_prefix(p, c, q, None, 1 / math.sqrt(d))
    check_prefix(p, c, q, None, 1 / math.sqrt(d), out)


@pytest.mark.parametrize("start", [(0, 3, 3, 70), (0, 0, 69, 70), (0, 40, 41, 70)])
def test_prefix_groups(start):
    # three prefixes, one of them empty of sequences or of tokens
    p = Cache(91, [300, 0, 515], 2, 128, room=1)
    c = Cache(92, [(7 * b) % 90 for b in range(70)], 2, 128)
    q = queries(93, 70, 8, 128)
    out = run_prefix(p, c, q, start, 0.088)
    check_prefix(p, c, q, start, 0.088, out, seqs=(0, 1, 2, 3, 13, 39, 40, 41, 68, 69))


def test_prefix_nothing_to_see_layouts_and_slots():
    p = Cache(101, [0], 3, 64, slots=[1, B.NO_SLOT, 0])
    c = Cache(102, [0, 9], 3, 64, room=1, layout="interleaved", slots=[0, B.NO_SLOT, 1])
    q = queries(103, 2, 6, 64)
    out = run_prefix(p, c, q, None, 0.1)
    check_prefix(p, c, q, None, 0.1, out)
    assert bool((out[0, :2] == 0).all()) and bool((out[0, 4:] == 0).all())
    p = Cache(104, [333], 3, 64, layout="head_major", slots=[1, B.NO_SLOT, 0])
    out = run_prefix(p, c, q, None, -0.1)
    check_prefix(p, c, q, None, -0.1, out)


def test_prefix_sequence_outside_every_range_is_recorded():
    p, c = Cache(111, [50], 1, 64), Cache(112, [4, 5], 1, 64)
    q = queries(113, 2, 2, 64)
    out = torch.zeros(q.shape, device="cuda")
    ws = B.workspace(B.prefix_decode_workspace_size(p.kv(), c.kv(), 2), "cuda")
    B.prefix_decode(q.cuda(), p.kv(), i32([0, 1]), c.kv(), 0.1, out, ws)
    st, detail = B.device_check()
    assert st == 6 and detail[0] == 1
    check_prefix(p, c, q, None, 0.1, out.cpu(), seqs=(0,))
    ref = attend(q[1, 0].double(), *c.rows(1, 0), torch.ones(5, dtype=torch.bool), 0.1)[0]
    assert float((out[1, 0].cpu().double() - ref).abs().max()) < 1e-3  # its own tokens only
    B.prefix_decode(q.cuda(), p.kv(), i32([0, 2]), c.kv(), 0.1, out, ws)
    check_device()
    check_prefix(p, c, q, None, 0.1, out.cpu())


@pytest.mark.parametrize("G,nb", [(8, 5), (7, 40), (1, 129), (32, 2)])
def test_prefix_long_rows_and_growing_maxima(G, nb):
    # rows past the 512 tokens that an accumulator gathers, several splits, maxima that grow along them
    p, c = Cache(115, [5003], 1, 128), Cache(116, [(31 * b) % 150 for b in range(nb)], 1, 128, room=1)
    q = queries(117, nb, G, 128)
    out = run_prefix(p, c, q, None, 0.09)
    check_prefix(p, c, q, None, 0.09, out, seqs=(0, 1, nb // 2, nb - 1))
    grow(p)
    grow(c)
    out = run_prefix(p, c, q, None, 1.1)
    check_prefix(p, c, q, None, 1.1, out, seqs=(0, 1, nb // 2, nb - 1))


def test_prefix_many_sequences():
    nb = 1100
    p, c = Cache(118, [130, 5, 700], 1, 64), Cache(119, [(7 * b) % 4 for b in range(nb)], 1, 64, room=1)
    q = queries(120, nb, 2, 64)
    start = (0, 3, 600, nb)
    out = run_prefix(p, c, q, start, 0.13)
    check_prefix(p, c, q, start, 0.13, out, seqs=(0, 2, 3, 599, 600, 900, nb - 1))


@pytest.mark.parametrize("start", [(0, 2, 2, 6), (0, 0, 5, 6), (0, 6, 6, 6)])
def test_prefix_groups_of_few_rows(start):
    p = Cache(94, [300, 0, 129], 2, 64, room=1)
    c = Cache(95, [0, 70, 1, 64, 200, 3], 2, 64)
    q = queries(96, 6, 10, 64)
    out = run_prefix(p, c, q, start, 0.12)
    check_prefix(p, c, q, start, 0.12, out)


# ----------------------------------------------------------------------------------- accumulated weights

def check_accum(c, q, scale, decay, mass_in, out, mass_out):
    G, d = q.shape[1] // c.hkv, c.d
    for g in range(c.hkv):
        if c.slots[g] == B.NO_SLOT:
            assert bool((mass_out[g] == 7.0).all()) and bool((out[:, g * G:(g + 1) * G] == 7.0).all())
            continue
        for b, L in enumerate(c.lens):
            k, v = c.rows(b, g)
            add, rel = torch.zeros(L, dtype=torch.float64), 0.0
            for h in range(g * G, (g + 1) * G):
                ref, w, A, X = attend(q[b, h].double(), k, v, torch.ones(L, dtype=torch.bool), scale)
                r = weight_rel(d, L, X)
                err = (out[b, h].double() - ref).abs()
                assert bool((err <= A * (2.0 ** -16 + r) + 1e-30).all()), (b, h)
                add, rel = add + w, max(rel, r)
            s = slice(c.off[b], c.off[b] + L)
            old = torch.zeros(L, dtype=torch.float64) if mass_in is None else decay * mass_in[g, s].double()
            tol = add * (rel + gamma(G + 2)) + 4 * U * (old.abs() + add) + 1e-36
            err = (mass_out[g, s].double() - old - add).abs()
            assert bool((err <= tol).all()), (b, g, float((err / tol).max()))
            assert bool((mass_out[g, c.off[b] + L:c.off[b + 1]] == 7.0).all())  # past the length: untouched


@pytest.mark.parametrize("hkv,G,d", [(4, 1, 64), (2, 4, 128), (1, 7, 128), (2, 12, 64), (1, 32, 128), (1, 17, 64)])
@pytest.mark.parametrize("lens", [(1, 0, 2), (63, 64, 65), (1500, 3, 300), (5000,)])
def test_accum_matches_the_formula(hkv, G, d, lens):
    c = Cache(121, list(lens), hkv, d, room=2)
    q = queries(122, len(lens), hkv * G, d)
    mass = torch.rand((hkv, c.T), generator=torch.Generator().manual_seed(123))
    kv = c.kv()
    ws = B.workspace(B.accum_decode_workspace_size(kv, hkv * G), "cuda")
    for decay, mi in ((1.0, mass), (0.9, mass), (1.0, None)):
        out = torch.full(q.shape, 7.0, device="cuda")
        mo = torch.full_like(mass, 7.0, device="cuda")
        B.accum_decode(q.cuda(), kv, 0.1, decay, None if mi is None else mi.cuda(), mo, out, ws)
        torch.cuda.synchronize()
        check_device()
        check_accum(c, q, 0.1, decay, mi, out.cpu(), mo.cpu())
    inplace = mass.cuda()
    B.accum_decode(q.cuda(), kv, 0.1, 0.9, inplace, inplace, out, ws)
    other = torch.empty_like(inplace)
    B.accum_decode(q.cuda(), kv, 0.1, 0.9, mass.cuda(), other, out, ws)
    for b, L in enumerate(lens):
        assert torch.equal(inplace[:, c.off[b]:c.off[b] + L], other[:, c.off[b]:c.off[b] + L])


@pytest.mark.parametrize("nb", [300, 1100])
def test_accum_many_sequences(nb):
    c = Cache(124, [(13 * b) % 90 if b % 3 else 0 for b in range(nb)], 1, 64, room=1)
    q = queries(125, nb, 3, 64)
    mass = torch.rand((1, c.T), generator=torch.Generator().manual_seed(126))
    kv = c.kv()
    out, mo = torch.full(q.shape, 7.0, device="cuda"), torch.full((1, c.T), 7.0, device="cuda")
    B.accum_decode(q.cuda(), kv, 0.2, 0.5, mass.cuda(), mo, out, B.workspace(B.accum_decode_workspace_size(kv, 3), "cuda"))
    torch.cuda.synchronize()
    check_device()
    check_accum(c, q, 0.2, 0.5, mass, out.cpu(), mo.cpu())


def test_accum_long_ragged_rows():
    # rows cut over many CTAs, with ring rounds to spare, and rows that share a CTA
    c = Cache(127, [20001, 3, 64, 9000, 0, 777, 12345], 2, 128, room=1)
    grow(c)
    q = queries(128, 7, 14, 128)
    kv = c.kv()
    ws = B.workspace(B.accum_decode_workspace_size(kv, 14), "cuda")
    out, mo = torch.full(q.shape, 7.0, device="cuda"), torch.full((2, c.T), 7.0, device="cuda")
    B.accum_decode(q.cuda(), kv, 0.3, 1.0, None, mo, out, ws)
    again = torch.full_like(mo, 7.0)
    B.accum_decode(q.cuda(), kv, 0.3, 1.0, None, again, torch.empty_like(out), ws)
    torch.cuda.synchronize()
    check_device()
    assert torch.equal(mo, again)
    check_accum(c, q, 0.3, 1.0, None, out.cpu(), mo.cpu())


def test_accum_layouts_and_slots():
    c = Cache(131, [400, 77], 3, 128, room=1, layout="interleaved", slots=[1, B.NO_SLOT, 0])
    q = queries(132, 2, 12, 128)
    kv = c.kv()
    out, mo = torch.full(q.shape, 7.0, device="cuda"), torch.full((3, c.T), 7.0, device="cuda")
    B.accum_decode(q.cuda(), kv, -0.1, 1.0, None, mo, out, B.workspace(B.accum_decode_workspace_size(kv, 12), "cuda"))
    torch.cuda.synchronize()
    check_device()
    check_accum(c, q, -0.1, 1.0, None, out.cpu(), mo.cpu())


# ----------------------------------------------------------------------------------- eviction

def kept_positions(mass, L, budget, sink, recent):
    """The definition: protected positions first, then by weight, the lower position among equals."""
    def key(p):
        m = float(mass[p])
        held = p < sink or p >= L - recent
        return (0 if held else 1, 0.0 if held else (math.inf if math.isnan(m) else -m), p)

    return sorted(sorted(range(L), key=key)[:min(budget, L)])


def run_evict(c, mass, budget, sink, recent, dst_cap, dst_layout="plain", dst_slots=None):
    dst = Cache(141, [0] * len(c.lens), c.hkv, c.d, room=dst_cap, layout=dst_layout, slots=dst_slots or c.slots)
    dst.k.fill_(5.0)
    dst.v.fill_(6.0)
    dst.max_len = dst_cap
    src, dkv = c.kv(), dst.kv()
    ws = B.workspace(B.cache_evict_workspace_size(src), "cuda")
    nb = len(c.lens)
    res = dict(dst=dst, idx=torch.full((nb, c.hkv, budget), -7, dtype=torch.int32, device="cuda"),
               count=torch.full((nb, c.hkv), -7, dtype=torch.int32, device="cuda"),
               mass=torch.full((c.hkv, dst.T), 7.0, device="cuda"),
               lengths=torch.full((nb,), -7, dtype=torch.int32, device="cuda"))
    for _ in range(2):  # the workspace serves call after call
        B.cache_evict(src, mass.cuda(), budget, sink, recent, dkv, res["lengths"], res["mass"], res["idx"],
                      res["count"], ws)
    torch.cuda.synchronize()
    return res


def check_evict(c, mass, budget, sink, recent, res):
    dst = res["dst"]
    dk, dv, dm, idx, count = (x.cpu() for x in (dst.k, dst.v, res["mass"], res["idx"], res["count"]))
    assert res["lengths"].tolist() == [min(budget, n) for n in c.lens]
    for b, L in enumerate(c.lens):
        n, o = min(budget, L), dst.off[b]
        for g in range(c.hkv):
            if c.slots[g] == B.NO_SLOT:
                assert bool((dm[g] == 7.0).all())
                continue
            keep = kept_positions(mass[g, c.off[b]:c.off[b] + L], L, budget, sink, recent)
            assert idx[b, g].tolist() == keep + [-1] * (budget - n) and int(count[b, g]) == n
            s, ds = c.slots[g], dst.slots[g]
            src = torch.tensor([c.off[b] + p for p in keep], dtype=torch.int64)
            assert torch.equal(dk[o:o + n, ds], c.kh[src, s]) and torch.equal(dv[o:o + n, ds], c.vh[src, s])
            want = mass[g, src]
            assert torch.equal(dm[g, o:o + n].nan_to_num(-1.0), want.nan_to_num(-1.0))
            assert bool((dm[g, o + n:dst.off[b + 1]] == 0).all())
            assert bool((dk[o + n:dst.off[b + 1], ds] == 5.0).all()) and bool((dv[o + n:dst.off[b + 1], ds] == 6.0).all())


def draw_mass(seed, hkv, T, kind):
    g = torch.Generator().manual_seed(seed)
    m = torch.rand((hkv, max(T, 1)), generator=g)
    if kind == "ties":
        m = (m * 4).floor()
    if kind == "zeros":
        m.zero_()
    if kind == "special":
        m[m < 0.2] = math.nan
        m[(m > 0.2) & (m < 0.3)] = math.inf
        m[(m > 0.3) & (m < 0.4)] = -math.inf
        m[(m > 0.4) & (m < 0.5)] = -0.0
    return m[:, :T]


@pytest.mark.parametrize("kind", ["plain", "ties", "zeros", "special"])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 4, 16), (65, 0, 65), (200, 200, 0),
                                                (300, 4, 0), (1000, 128, 256)])
def test_evict_keeps_what_the_definition_keeps(kind, budget, sink, recent):
    c = Cache(151, [0, 1, 63, 64, 65, 700], 3, 64, room=2)
    mass = draw_mass(152, 3, c.T, kind)
    res = run_evict(c, mass, budget, sink, recent, min(budget, 700) + 3)
    check_device()
    check_evict(c, mass, budget, sink, recent, res)


@pytest.mark.parametrize("d", [64, 128])
def test_evict_layouts_slots_and_long_rows(d):
    c = Cache(161, [3001, 20000], 3, d, room=1, layout="interleaved", slots=[2, B.NO_SLOT, 0])
    mass = draw_mass(162, 3, c.T, "plain")
    res = run_evict(c, mass, 2048, 4, 512, 2050, dst_layout="head_major", dst_slots=[0, B.NO_SLOT, 1])
    check_device()
    check_evict(c, mass, 2048, 4, 512, res)


def test_evict_rows_too_long_for_a_cluster():
    # more than 131072 positions: the scores go through memory
    c = Cache(165, [140000, 50], 1, 64)
    mass = draw_mass(166, 1, c.T, "ties")
    res = []
    got = launches_of(lambda: res.append(run_evict(c, mass, 3000, 4, 100, 3000)))
    check_device()
    assert got["evict_key_kernel"] == 2 and got["evict_copy_kernel"] == 2
    check_evict(c, mass, 3000, 4, 100, res[0])


def test_evict_records_a_region_too_small():
    c = Cache(171, [10, 100, 20], 2, 64)
    mass = draw_mass(172, 2, c.T, "plain")
    res = run_evict(c, mass, 50, 1, 1, 30)  # sequence 1 keeps 50 rows, its region holds 30
    st, detail = B.device_check()
    assert st == 6 and detail[0] == 4 and detail[1] == 1
    assert res["lengths"].tolist() == [10, 0, 20]
    dst = res["dst"]
    assert bool((dst.k[dst.off[1]:dst.off[2]] == 5.0).all()) and bool((dst.v[dst.off[1]:dst.off[2]] == 6.0).all())
    assert torch.equal(dst.k[:10].cpu(), c.kh[:10])


# ----------------------------------------------------------------------------------- together

def test_nothing_held_anywhere():
    c, p = Cache(175, [0, 0], 2, 128, room=4), Cache(176, [0], 2, 128, room=1)
    d = Cache(177, [0, 0], 2, 128, room=4)
    q = queries(178, 2, 4, 128).cuda()
    kv = c.kv()
    out, mo = torch.full((2, 4, 128), 7.0, device="cuda"), torch.full((2, c.T), 7.0, device="cuda")
    B.accum_decode(q, kv, 0.1, 1.0, None, mo, out, B.workspace(B.accum_decode_workspace_size(kv, 4), "cuda"))
    assert bool((out == 0).all()) and bool((mo == 7.0).all())
    out.fill_(7.0)
    B.prefix_decode(q, p.kv(), None, kv, 0.1, out, B.workspace(B.prefix_decode_workspace_size(p.kv(), kv, 4), "cuda"))
    assert bool((out == 0).all())
    pout = torch.full_like(q, 7.0)
    B.stream_prefill(q, kv, i32([0, 1, 2]), [DENSE, STREAM], 1, 1, 0.1, pout,
                     B.workspace(B.stream_prefill_workspace_size(kv, 4, 2, [DENSE, STREAM], 1, 1), "cuda"))
    assert bool((pout == 0).all())
    idx, count = torch.zeros((2, 2, 3), dtype=torch.int32, device="cuda"), i32([[7, 7], [7, 7]])
    lengths = i32([7, 7])
    B.cache_evict(kv, mo, 3, 1, 1, d.kv(), lengths, None, idx, count, B.workspace(B.cache_evict_workspace_size(kv), "cuda"))
    assert lengths.tolist() == [0, 0] and bool((count == 0).all()) and bool((idx == -1).all())
    check_device()


def test_append_at_leaves_a_refused_sequence_alone():
    off = [0, 4, 8, 12]
    k, v = torch.zeros((12, 1, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((12, 1, 64), dtype=torch.bfloat16, device="cuda")
    lengths, positions = i32([3, 4, 2]), i32([30, 9, -1])
    kv = B.make_kv(k, v, i32(off), 4, 12, lengths=lengths)
    kn, vn = queries(188, 3, 1, 64).cuda(), queries(189, 3, 1, 64).cuda()
    B.kv_append_at(None, kn, vn, 1e4, kv, None, 0, lengths, positions, None)
    st, detail = B.device_check()
    assert st == 6 and detail[0] == 4
    assert lengths.tolist() == [4, 4, 2] and positions.tolist() == [31, 9, -1]
    assert torch.equal(v[3], vn[0]) and bool((v[4:] == 0).all()) and bool((k[4:] == 0).all())
    want = rope64(kn[0, 0].cpu(), 30, 1e4)
    assert float((k[3, 0].cpu().double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max())


def test_calls_on_two_streams_at_once():
    """Steps with workspaces of their own, on two streams at the same time: the results of one after the other."""
    c = [Cache(210 + i, [4000, 3000, 17], 2, 128) for i in range(2)]
    q = [queries(212 + i, 3, 8, 128).cuda() for i in range(2)]
    own = [Cache(214 + i, [20 * b for b in range(12)], 2, 128) for i in range(2)]
    qp = [queries(216 + i, 12, 8, 128).cuda() for i in range(2)]
    steps = []
    for i in range(2):
        acc = AccumDecodeStep(c[i].k, c[i].v, c[i].offsets, c[i].max_len, c[i].T, 8, 0.1)
        pre = PrefillStep(c[i].k, c[i].v, c[i].offsets, c[i].max_len, c[i].T, 8, [DENSE, STREAM], 4, 900, 0.1, 3)
        pfx = PrefixDecodeStep(c[i].k, c[i].v, c[i].offsets[:2], 4000, 4000, own[i].k, own[i].v, own[i].offsets, 240,
                               own[i].T, 8, 0.1)
        steps.append((acc, pre, pfx, torch.zeros((2, c[i].T), device="cuda"), torch.zeros_like(q[i]), i32([0, 1, 2, 3])))

    def run(i):
        acc, pre, pfx, mass, out, qo = steps[i]
        acc(q[i], None, mass)
        pre(q[i], qo, out)
        pfx(qp[i])
        return [acc.out, mass, out, pfx.out]

    alone = [[x.clone() for x in run(i)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                run(i)
    torch.cuda.synchronize()
    check_device()
    for i in range(2):
        acc, pre, pfx, mass, out, qo = steps[i]
        for a, b in zip(alone[i], [acc.out, mass, out, pfx.out]):
            assert torch.equal(a, b)


def test_steps_launch_the_kernels():
    c = Cache(181, [700, 300], 2, 128)
    q = queries(182, 2, 8, 128).cuda()
    pre = PrefillStep(c.k, c.v, c.offsets, c.max_len, c.T, 8, [DENSE, STREAM], 4, 100, 0.1, 2)
    got = launches_of(lambda: pre(q, i32([0, 1, 2])))
    assert got.pop("tile_attend_kernel") == 1
    acc = AccumDecodeStep(c.k, c.v, c.offsets, c.max_len, c.T, 8, 0.1)
    assert launches_of(lambda: acc(q, torch.zeros((2, c.T), device="cuda"))) == {"dense_pass_kernel": 1,
                                                                                  "accum_merge_kernel": 1}
    d = Cache(183, [128, 128], 2, 128)
    ev = EvictStep(c.k, c.v, c.offsets, c.max_len, c.T, d.k, d.v, d.offsets, 128, d.T, 128, 4, 16)
    got = launches_of(lambda: ev(torch.rand((2, c.T), device="cuda"), None, d.lengths))
    assert got == {"select_cluster_kernel": 1, "evict_copy_kernel": 1}
    pfx = PrefixDecodeStep(c.k, c.v, c.offsets[:2], 700, 700, d.k, d.v, d.offsets, 128, d.T, 8, 0.1)
    assert launches_of(lambda: pfx(q)) == {"dense_pass_kernel": 1, "tile_merge_kernel": 1}  # few rows: one pass
    many = Cache(185, [30] * 9, 2, 128)
    pfx = PrefixDecodeStep(c.k, c.v, c.offsets[:2], 700, 700, many.k, many.v, many.offsets, 30, many.T, 8, 0.1)
    assert launches_of(lambda: pfx(queries(186, 9, 8, 128).cuda())) == {
        "tile_attend_kernel": 1, "dense_pass_kernel": 1, "tile_merge_kernel": 1}
    check_device()
    with pytest.raises(ValueError):
        pre(queries(184, 3, 8, 128).cuda(), i32([0, 1, 3]))


def rope64(x, pos, theta):
    d = x.shape[-1]
    a = pos * theta ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    u, v = x[..., :d // 2].double(), x[..., d // 2:].double()
    return torch.cat([a.cos() * u - a.sin() * v, a.sin() * u + a.cos() * v], -1)


def test_bounded_decode_follows_the_definition():
    """Prompt prefill, eviction of the prompt to the budget, then decode steps that append, accumulate and
    evict: after every step the cache, the mass and the outputs against a float64 model that takes the
    library's kept positions (they depend on rounded weights), checked to be the heaviest of its mass."""
    Bn, hkv, G, d, theta = 2, 2, 4, 64, 1e4
    budget, slack, sink, recent, scale, decay = 40, 6, 2, 8, 0.125, 0.95
    prompt = Cache(191, [100, 57], hkv, d, room=1)
    q = queries(192, 157, hkv * G, d)
    pre = PrefillStep(prompt.k, prompt.v, prompt.offsets, prompt.max_len, prompt.T, hkv * G, [DENSE] * hkv, 0, 0, scale, 157,
                      lengths=prompt.lengths)
    pre_out = pre(q.cuda(), i32([0, 100, 157]))
    torch.cuda.synchronize()
    check_prefill(prompt, q, [100, 57], [DENSE] * hkv, 0, 0, scale, pre_out.cpu(), rows=(0, 56))
    # weights of the prompt's last token start the mass
    mass0 = torch.zeros((hkv, prompt.T), device="cuda")
    acc = AccumDecodeStep(prompt.k, prompt.v, prompt.offsets, prompt.max_len, prompt.T, hkv * G, scale, lengths=prompt.lengths)
    acc(q[[99, 156]].cuda(), None, mass0)
    step = EvictDecodeStep(Bn, hkv * G, hkv, d, theta, budget, slack, sink, recent, scale, decay)
    step.load(prompt.kv(), mass0, prompt.lengths)
    torch.cuda.synchronize()
    check_device()
    model = {}
    for b in range(Bn):
        for g in range(hkv):
            m = mass0[g, prompt.off[b]:prompt.off[b] + prompt.lens[b]].cpu()
            keep = kept_positions(m, prompt.lens[b], budget, sink, recent)
            k, v = prompt.rows(b, g)
            model[b, g] = [k[keep], v[keep], m.double()[keep]]
    gen = torch.Generator().manual_seed(193)
    for it in range(3 * slack + 2):
        if step.held == step.cap:
            before = step.mass.cpu()
            step.evict()
            torch.cuda.synchronize()
            for (b, g), row in model.items():
                n = row[0].shape[0]
                m = before[g, b * step.cap:b * step.cap + n]
                keep = step.idx[b, g].tolist()
                assert keep == kept_positions(m, n, budget, sink, recent)
                model[b, g] = [x[keep] for x in row]
        qn, kn, vn = (torch.randn((Bn, h, d), generator=gen).bfloat16() for h in (hkv * G, hkv, hkv))
        out = step(qn.cuda(), kn.cuda(), vn.cuda())
        torch.cuda.synchronize()
        check_device()
        for b in range(Bn):
            pos = prompt.lens[b] + it
            assert int(step.positions[b]) == pos + 1
            for g in range(hkv):
                row = model[b, g]
                got_k = step.k[step.cur][b * step.cap + row[0].shape[0], g].cpu()
                kr = rope64(kn[b, g], pos, theta)
                assert float((got_k.double() - kr).abs().max()) <= 2.0 ** -8 * float(kr.abs().max())
                row[0] = torch.cat([row[0], got_k.double()[None]])
                row[1] = torch.cat([row[1], vn[b, g].double()[None]])
                row[2] = torch.cat([row[2], torch.zeros(1, dtype=torch.float64)]) * decay
                n = row[0].shape[0]
                assert int(step.lengths[step.cur][b]) == n
                assert torch.equal(step.k[step.cur][b * step.cap:b * step.cap + n, g].cpu().double(), row[0])
                for h in range(g * G, (g + 1) * G):
                    qr = step.q_rot[b, h].cpu().double()
                    assert float((qr - rope64(qn[b, h], pos, theta)).abs().max()) <= 2.0 ** -8 * float(qr.abs().max() + 1e-3)
                    ref, w, A, X = attend(qr, row[0], row[1], torch.ones(n, dtype=torch.bool), scale)
                    assert bool(((out[b, h].cpu().double() - ref).abs() <= A * (2.0 ** -16 + weight_rel(d, n, X))).all())
                    row[2] = row[2] + w
                got_m = step.mass[g, b * step.cap:b * step.cap + n].cpu().double()
                assert bool(((got_m - row[2]).abs() <= 1e-4 * (row[2] + 1e-6)).all())
    assert step.held <= step.cap


def test_calls_captured_in_a_graph_replay_on_changed_data():
    c = Cache(201, [900, 130], 2, 128)
    d = Cache(202, [64, 64], 2, 128)
    q = queries(203, 2, 8, 128).cuda()
    mass, mo = torch.zeros((2, c.T), device="cuda"), torch.zeros((2, c.T), device="cuda")
    pre = PrefillStep(c.k, c.v, c.offsets, c.max_len, c.T, 8, [DENSE, STREAM], 4, 100, 0.1, 2)
    acc = AccumDecodeStep(c.k, c.v, c.offsets, c.max_len, c.T, 8, 0.1)
    ev = EvictStep(c.k, c.v, c.offsets, c.max_len, c.T, d.k, d.v, d.offsets, 64, d.T, 64, 4, 16)
    pfx = PrefixDecodeStep(c.k, c.v, c.offsets, c.max_len, c.T, d.k, d.v, d.offsets, 64, d.T, 8, 0.1, seq_start=i32([0, 1, 2]))
    qo, pre_out = i32([0, 1, 2]), torch.zeros_like(q)

    def everything():
        pre(q, qo, pre_out)
        acc(q, mass, mo)
        ev(mo, None, d.lengths)
        pfx(q)
        return [x.clone() for x in (pre_out, acc.out, mo, ev.idx, d.k, pfx.out)]

    everything()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        everything()
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            captured = everything()
    torch.cuda.synchronize()
    for seed in (1, 2):
        q.copy_(queries(seed, 2, 8, 128))
        mass.copy_(torch.rand(mass.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in captured]
        for a, b in zip(got, everything()):
            assert torch.equal(a, b)
    check_device()


def test_offsets_past_32_bits():
    # a cache whose rows lie more than 2^32 bytes (and 2^31 elements) apart: 2.4 M tokens x 8 heads x 128
    T, hkv, d = 2_400_000, 8, 128
    k = torch.zeros((T, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(5)
    n = 300
    k[-n:] = torch.randn((n, hkv, d), generator=g, device="cuda").bfloat16()
    v[-n:] = torch.randn((n, hkv, d), generator=g, device="cuda").bfloat16()
    offsets = i32([0, T - n, T])
    lengths = i32([0, n])
    small = Cache(0, [0, n], hkv, d)
    small.kh, small.vh = k[-n:].cpu(), v[-n:].cpu()
    q = queries(6, 2, 16, d)
    kv = B.make_kv(k, v, offsets, n, T, lengths=lengths)
    out, mo = torch.zeros((2, 16, d), device="cuda"), torch.zeros((hkv, T), device="cuda")
    B.accum_decode(q.cuda(), kv, 0.1, 1.0, None, mo, out, B.workspace(B.accum_decode_workspace_size(kv, 16), "cuda"))
    small.off = [0, 0, n]
    check_accum(small, q, 0.1, 1.0, None, out.cpu(), mo[:, -n:].cpu())
    pout = torch.full((2, 16, d), 7.0, dtype=torch.bfloat16, device="cuda")
    roles = [DENSE, STREAM] * 4
    B.stream_prefill(q.cuda(), kv, i32([0, 0, 2]), roles, 2, 50, 0.1, pout,
                     B.workspace(B.stream_prefill_workspace_size(kv, 16, 2, roles, 2, 50), "cuda"))
    check_prefill(small, q, [0, 2], roles, 2, 50, 0.1, pout.cpu())
    B.prefix_decode(q.cuda(), kv, i32([0, 0, 2]), small.kv(), 0.1, out,
                    B.workspace(B.prefix_decode_workspace_size(kv, small.kv(), 16), "cuda"))
    torch.cuda.synchronize()
    check_device()
