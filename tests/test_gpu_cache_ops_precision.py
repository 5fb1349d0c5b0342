"""What the cache operators with fp32 outputs keep of their precision, and where they read and write
in very large caches.

The errors here are 2-norms of the difference over 2-norms of the result, against float64 on unit-normal
data at scale 1 / sqrt(d).  Both bounds follow from the kernels' roundings and lie below what the
loss of any one mechanism would give:
  * accumulated weights: exp2 within 2^-22, logits of 8 products of 16 columns whose sums drop bits (about 4 of
    2^-24 of a logit around 1), each 16 tokens' product from zero and added in fp32, rounded to nearest: 3 to 4e-7.
    Bound 1e-6.  Two bf16 terms of a weight instead of three leave 2^-17 (rms 4.4e-6), sums gathered by the
    tensor cores 3e-6 after 900 tokens.
  * shared prefixes through tiles: the same, and 3 x 16 products per segment of 256 tokens, each dropping half
    of an accumulator's last bit on average (0.72 x 2^-24 of it, and O half as large as at the end): 1.03e-6, with
    the above 1.1e-6.  Bound 1.3e-6.  Segments of 512 tokens give 1.7e-6, two terms 4.7e-6, no segments 9e-6 after
    3600 tokens.
"""

import math

import pytest
import torch

from gpu_helpers import check_device, launches_of
from test_gpu_cache_ops import Cache, attend, check_prefix, i32, queries, weight_rel
from token_sparse_decode_b200 import binding as B
from token_sparse_decode_b200.step import AccumDecodeStep, EvictStep, PrefixDecodeStep

pytestmark = pytest.mark.gpu


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def softmax64(q, k, v, scale):
    """(out, weights) in float64 of queries [n, d] over keys [L, d]."""
    w = torch.softmax(scale * (q.double() @ k.double().T), 1)
    return w @ v.double(), w


def off_by(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("d,G,lens", [(128, 4, [9000, 700, 40000]), (64, 1, [20000]), (128, 17, [30000, 5])])
def test_accumulated_weights_keep_fp32(d, G, lens):
    hkv, T = 2, sum(lens)
    k, v, q = normal(501, T, hkv, d), normal(502, T, hkv, d), normal(503, len(lens), hkv * G, d)
    off = [sum(lens[:i]) for i in range(len(lens) + 1)]
    step = AccumDecodeStep(k, v, i32(off), max(lens), T, hkv * G, 1 / math.sqrt(d))
    mass = torch.zeros((hkv, T), device="cuda")
    out = step(q, None, mass)
    check_device()
    for b, (o, n) in enumerate(zip(off, lens)):
        for g in range(hkv):
            ref, w = softmax64(q[b, g * G:(g + 1) * G], k[o:o + n, g], v[o:o + n, g], 1 / math.sqrt(d))
            assert off_by(out[b, g * G:(g + 1) * G], ref) <= 1e-6
            assert off_by(mass[g, o:o + n], w.sum(0)) <= 1e-6


@pytest.mark.parametrize("d,G,plens,nb", [(128, 4, [8000], 70), (64, 1, [20000], 200), (128, 7, [3600, 12000], 90)])
def test_shared_prefixes_keep_fp32(d, G, plens, nb):
    hkv, P = 2, sum(plens)
    own = [(37 * b) % 300 for b in range(nb)]
    pk, pv, k, v = normal(511, P, hkv, d), normal(512, P, hkv, d), normal(513, sum(own), hkv, d), normal(514, sum(own), hkv, d)
    q = normal(515, nb, hkv * G, d)
    poff, off = [sum(plens[:i]) for i in range(len(plens) + 1)], [sum(own[:i]) for i in range(nb + 1)]
    start = [0, nb] if len(plens) == 1 else [0, nb // 2, nb]
    step = PrefixDecodeStep(pk, pv, i32(poff), max(plens), P, k, v, i32(off), max(own), sum(own), hkv * G, 1 / math.sqrt(d),
                            seq_start=i32(start))
    res = []
    assert launches_of(lambda: res.append(step(q))).get("tile_attend_kernel") == 1
    check_device()
    ref = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for b in range(nb):
        i = 0 if b < start[1] else 1
        for g in range(hkv):
            kk = torch.cat([pk[poff[i]:poff[i + 1], g], k[off[b]:off[b + 1], g]])
            vv = torch.cat([pv[poff[i]:poff[i + 1], g], v[off[b]:off[b + 1], g]])
            ref[b, g * G:(g + 1) * G] = softmax64(q[b, g * G:(g + 1) * G], kk, vv, 1 / math.sqrt(d))[0]
    assert off_by(res[0], ref) <= 3e-6


@pytest.mark.parametrize("d,hkv,G,P,nb,own", [(128, 8, 4, 600, 64, 100), (128, 2, 4, 1765, 64, 100), (64, 1, 5, 1765, 33, 50),
                                              (128, 2, 7, 8192, 40, 700), (64, 2, 4, 30000, 40, 0)])
def test_shared_prefixes_of_every_length_keep_fp32(d, hkv, G, P, nb, own):
    lens = [(37 * b) % (own + 1) for b in range(nb)]
    off, T = [sum(lens[:i]) for i in range(nb + 1)], sum(lens)
    pk, pv, k, v = normal(541, P, hkv, d), normal(542, P, hkv, d), normal(543, T, hkv, d), normal(544, T, hkv, d)
    q = normal(545, nb, hkv * G, d)
    step = PrefixDecodeStep(pk, pv, i32([0, P]), P, P, k, v, i32(off), max(lens), T, hkv * G, 1 / math.sqrt(d))
    out = step(q)
    check_device()
    ref = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for b in range(nb):
        for g in range(hkv):
            kk, vv = torch.cat([pk[:, g], k[off[b]:off[b + 1], g]]), torch.cat([pv[:, g], v[off[b]:off[b + 1], g]])
            ref[b, g * G:(g + 1) * G] = softmax64(q[b, g * G:(g + 1) * G], kk, vv, 1 / math.sqrt(d))[0]
    assert off_by(out, ref) <= 1.3e-6


# ----------------------------------------------------------------------------------- very large caches

@pytest.fixture(scope="module")
def far():
    """2.4 M tokens x 8 heads x 128: the last 300 rows, an own sequence, lie more than 2^32 bytes and 2^31 elements in."""
    T, hkv, d, n = 2_400_000, 8, 128, 300
    k = torch.zeros((T, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[-n:], v[-n:] = normal(521, n, hkv, d), normal(522, n, hkv, d)
    near = Cache(0, [0, n], hkv, d)
    near.kh, near.vh, near.off = k[-n:].cpu(), v[-n:].cpu(), [0, 0, n]
    near.k, near.v, near.offsets = k[-n:].clone(), v[-n:].clone(), i32([0, 0, n])
    yield k, v, i32([0, T - n, T]), i32([0, n]), near
    del k, v


@pytest.mark.parametrize("nb", [2, 70])  # one dense pass, and tiles
def test_shared_prefix_past_32_bits(far, nb):
    k, v, offsets, lengths, near = far
    kv = B.make_kv(k, v, offsets, 300, k.shape[0], lengths=lengths)
    own = Cache(523, [(3 * b) % 20 for b in range(nb)], 8, 128)
    q = queries(524, nb, 16, 128)
    out = torch.full(q.shape, 7.0, device="cuda")
    for start in ([0, 0, nb], [0, 1, nb]):  # behind the far prefix; the first one behind the empty one
        B.prefix_decode(q.cuda(), kv, i32(start), own.kv(), 0.1, out,
                        B.workspace(B.prefix_decode_workspace_size(kv, own.kv(), 16), "cuda"))
        check_device()
        check_prefix(near, own, q, start, 0.1, out.cpu(), seqs=(0, 1, nb - 1))
    # and the own tokens of the far sequence
    p = Cache(525, [100], 8, 128)
    q = queries(526, 2, 16, 128)
    out = torch.full(q.shape, 7.0, device="cuda")
    B.prefix_decode(q.cuda(), p.kv(), None, kv, 0.1, out, B.workspace(B.prefix_decode_workspace_size(p.kv(), kv, 16), "cuda"))
    check_device()
    check_prefix(p, near, q, None, 0.1, out.cpu())


def test_evict_past_32_bits(far):
    k, v, offsets, lengths, near = far
    T, n = k.shape[0], 300
    mass = torch.zeros((8, T), device="cuda")
    mass[:, -n:] = torch.rand((8, n), generator=torch.Generator(device="cuda").manual_seed(527), device="cuda")
    dk, dv = torch.zeros((64, 8, 128), dtype=torch.bfloat16, device="cuda"), torch.zeros((64, 8, 128), dtype=torch.bfloat16, device="cuda")
    dl, dm = i32([7, 7]), torch.full((8, 64), 7.0, device="cuda")
    idx, count = EvictStep(k, v, offsets, n, T, dk, dv, i32([0, 0, 64]), 64, 64, 50, 4, 8, lengths=lengths)(mass, dm, dl)
    check_device()
    assert dl.tolist() == [0, 50] and count[0].tolist() == [0] * 8 and count[1].tolist() == [50] * 8
    for g in range(8):
        m = mass[g, -n:].clone()
        m[:4] = m[-8:] = math.inf
        keep = torch.topk(m, 50).indices.sort().values
        assert torch.equal(idx[1, g].long(), keep)
        assert torch.equal(dk[:50, g], k[T - n + keep, g]) and torch.equal(dv[:50, g], v[T - n + keep, g])
        assert torch.equal(dm[g, :50], mass[g, T - n + keep]) and bool((dm[g, 50:] == 0).all())
    # into a far region
    back = torch.zeros_like(k)
    step = EvictStep(near.k, near.v, near.offsets, n, n, back, torch.zeros_like(back), offsets, n, T, 50, 4, 8)
    idx, count = step(mass[:, -n:].contiguous(), None, dl)
    check_device()
    assert dl.tolist() == [0, 50] and int((back != 0).any(2).any(1).sum()) == 50
    for g in range(8):
        assert torch.equal(back[T - n:T - n + 50, g], near.k[idx[1, g].long(), g])


def test_append_at_past_32_bits(far):
    k, v, offsets, lengths, near = far
    kv = B.make_kv(k, v, i32([0, k.shape[0] - 200, k.shape[0]]), 300, k.shape[0])
    kn, vn = normal(528, 2, 8, 128), normal(529, 2, 8, 128)
    at, pos = i32([1, 199]), i32([0, 0])  # position 0: no rotation
    old = k[-1].clone(), v[-1].clone(), k[1].clone(), v[1].clone()
    B.kv_append_at(None, kn, vn, 1e4, kv, None, 0, at, pos, None)
    check_device()
    assert torch.equal(k[-1], kn[1]) and torch.equal(v[-1], vn[1]) and torch.equal(v[1], vn[0])
    assert at.tolist() == [2, 200] and pos.tolist() == [1, 1]
    k[-1], v[-1], k[1], v[1] = old


@pytest.mark.parametrize("nb", [3, 60])  # the dense pass alone, and tiles
def test_a_sequence_outside_every_range_attends_to_its_own_tokens(nb):
    p, c = Cache(531, [500, 30], 2, 64), Cache(532, [4 + b % 40 for b in range(nb)], 2, 64)
    q = queries(533, nb, 8, 64)
    out = torch.full(q.shape, 7.0, device="cuda")
    ws = B.workspace(B.prefix_decode_workspace_size(p.kv(), c.kv(), 8), "cuda")
    start = [1, nb - 2, nb - 1]  # the first and the last one have no prefix
    B.prefix_decode(q.cuda(), p.kv(), i32(start), c.kv(), 0.1, out, ws)
    st, detail = B.device_check()
    assert st == 6 and detail[0] == 1
    check_prefix(p, c, q, start, 0.1, out.cpu(), seqs=range(1, nb - 1))
    for b in (0, nb - 1):
        for h in range(8):
            ref, _, A, X = attend(q[b, h].double(), *c.rows(b, h // 4), torch.ones(c.lens[b], dtype=torch.bool), 0.1)
            tol = A * (2.0 ** -22 + weight_rel(64, c.lens[b], X))  # three bf16 terms of a weight keep 24 bits
            assert bool(((out[b, h].cpu().double() - ref).abs() <= tol).all())
