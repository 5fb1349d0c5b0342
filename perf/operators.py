"""Cases of the cache-side attention operators: role prefill, shared-prefix decode, decode that
accumulates attention weight, and eviction by that weight.

Each operator has a plain form in elementary torch operations (``own`` false) and the calls a
user makes of the framework's kernels (``own`` true).  Shapes:

  q          bf16 [rows, Hq, d]; q head h reads KV head h // (Hq // Hkv)
  k, v       bf16 [T, Hkv, d], sequence b at tokens offsets[b] .. offsets[b + 1] - 1
  mass       fp32 [Hkv, T], accumulated attention weight per KV head and token
"""

import math
import random

import torch

own = False

DENSE, STREAM = 1, 2  # head roles: the whole past, or a few first tokens and a window


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a chat turn of a small model: a few new tokens per sequence over a short cache (latency)
        dict(name="prefill_turn_d64", op="prefill", batch=4, hq=4, hkv=4, d=64, n_lo=1, n_hi=33, c_lo=100, c_hi=512,
             dense=2, sink=4, window=60, pad=3, lseed=1),
        # ragged prompts of a serving batch, 7 query heads per KV head, one retrieval head of four
        dict(name="prefill_ragged_g7", op="prefill", batch=5, hq=28, hkv=4, d=128, n_lo=301, n_hi=2500, c_lo=0, c_hi=37,
             dense=1, sink=128, window=1000, pad=0, lseed=2),
        # one long prompt, 2 of 8 KV groups retrieval heads, the others sink 128 + window 4096
        dict(name="prefill_prompt_8k", op="prefill", batch=1, hq=32, hkv=8, d=128, n_lo=8192, n_hi=8192, c_lo=0, c_hi=0,
             dense=2, sink=128, window=4096, pad=0, lseed=3),
        # a chunk of a chunked prompt: 1000 new tokens on a cache of 32K, every head a retrieval head
        dict(name="prefill_chunk_32k", op="prefill", batch=1, hq=32, hkv=8, d=128, n_lo=1000, n_hi=1000, c_lo=31768,
             c_hi=31768, dense=8, sink=0, window=0, pad=0, lseed=4),
        # a few samples of one short prompt on a small model (latency)
        dict(name="prefix_small_d64", op="prefix", batch=4, hq=4, hkv=4, d=64, p_lo=512, p_hi=512, np=1, s_lo=1, s_hi=40,
             lseed=5),
        # a serving batch behind one system prompt of 8K
        dict(name="prefix_serving_8k", op="prefix", batch=64, hq=32, hkv=8, d=128, p_lo=8192, p_hi=8192, np=1, s_lo=16,
             s_hi=700, lseed=6),
        # two long shared documents, 7 query heads per KV head, ragged answers
        dict(name="prefix_documents_32k", op="prefix", batch=96, hq=28, hkv=4, d=128, p_lo=20011, p_hi=32768, np=2,
             s_lo=0, s_hi=2000, lseed=7),
        # decode with accumulated weights: a small model's step (latency), a serving batch at its budget
        # plus slack, one long context
        dict(name="accum_small_d64", op="accum", batch=1, hq=4, hkv=4, d=64, l_lo=512, l_hi=512, decay=1.0, lseed=8),
        dict(name="accum_serving_b48", op="accum", batch=48, hq=28, hkv=4, d=128, l_lo=1, l_hi=8000, decay=0.98, lseed=9),
        dict(name="accum_long_128k", op="accum", batch=1, hq=32, hkv=8, d=128, l_lo=131072, l_hi=131072, decay=1.0,
             lseed=10),
        # eviction of a serving batch to 2048 rows per head; of long prompts to an eighth
        dict(name="evict_serving_b32", op="evict", batch=32, hq=32, hkv=8, d=128, l_lo=700, l_hi=4500, budget=2048, sink=4,
             recent=256, lseed=11),
        dict(name="evict_long_64k", op="evict", batch=2, hq=32, hkv=8, d=128, l_lo=60001, l_hi=65536, budget=8192, sink=128,
             recent=4096, lseed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["prefill", "prefix", "accum", "evict"])
    hkv, g, d = rng.choice([(1, 5, 64), (2, 8, 128), (4, 1, 64), (4, 7, 128), (8, 4, 128), (8, 1, 128), (8, 4, 64), (3, 2, 64)])
    c = dict(op=op, hq=hkv * g, hkv=hkv, d=d, lseed=rng.randrange(1 << 30))
    if op == "prefill":
        b = _log(rng, 1, 12)
        n = _log(rng, 1, 4000)
        ctx = rng.choice([0, _log(rng, 1, 16000)])
        # no more score entries than the largest listed case
        while b * c["hq"] * n * (n + ctx) > 9e8:
            n, ctx, b = max(1, n * 3 // 4), ctx * 3 // 4, max(1, b - 1)
        c.update(batch=b, n_lo=max(1, n // 4), n_hi=n, c_lo=ctx // 3, c_hi=ctx, dense=rng.randint(0, hkv),
                 sink=rng.choice([0, 1, 4, 128]), window=_log(rng, 1, 5000), pad=rng.randint(0, 5))
    elif op == "prefix":
        b, p = _log(rng, 1, 96), _log(rng, 17, 32768)
        while b * c["hq"] * p > 96 * 28 * 25000:
            b, p = max(1, b * 7 // 8), p * 7 // 8
        c.update(batch=b, p_lo=max(1, p // 2), p_hi=p, np=rng.randint(1, min(b, 3)), s_lo=0, s_hi=_log(rng, 1, 2000))
    elif op == "accum":
        b, l = _log(rng, 1, 48), _log(rng, 30, 131072)
        while b * l * hkv * d > 131072 * 1024:
            b, l = max(1, b * 3 // 4), l * 7 // 8
        c.update(batch=b, l_lo=max(1, l // 10), l_hi=l, decay=rng.choice([1.0, 0.9, 0.99]))
    else:
        b, l = _log(rng, 1, 32), _log(rng, 30, 65536)
        while b * l * hkv * d > 131072 * 480:
            b, l = max(1, b * 3 // 4), l * 7 // 8
        budget = max(8, int(l * rng.uniform(0.05, 0.9)))
        sink = rng.choice([0, 1, 4])
        c.update(batch=b, l_lo=max(1, l // 4), l_hi=l, budget=budget, sink=sink, recent=rng.randint(0, (budget - sink) // 2))
    return c


def _lengths(case, key, count, salt=0):
    r = random.Random(case["lseed"] * 7 + salt)
    lo, hi = case[key + "_lo"], case[key + "_hi"]
    return [r.randint(lo, hi) for _ in range(count)]


def _offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _roles(case):
    return [DENSE if g < case["dense"] else STREAM for g in range(case["hkv"])]


def _prefixes(case):
    """Prefix lengths and the first sequence of each prefix (sequences in prefix order)."""
    r = random.Random(case["lseed"] * 7 + 3)
    cut = sorted(r.sample(range(1, case["batch"]), case["np"] - 1)) if case["np"] > 1 else []
    return _lengths(case, "p", case["np"], 4), [0] + cut + [case["batch"]]


# ------------------------------------------------------------------------------------ inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _cache(gen, lengths, hkv, d, u):
    """Keys and values of ragged sequences: unit normal, the first tokens and one token in 64 leaning
    towards the heads' common query direction (attention sinks and salient tokens)."""
    T = sum(lengths)
    k, v = _normal(gen, T, hkv, d), _normal(gen, T, hkv, d)
    lean = (torch.rand((T, hkv, 1), generator=gen, device="cuda") < 1 / 64).float() * 3
    start = torch.tensor([o for o, n in zip(_offsets(lengths), lengths) if n], device="cuda", dtype=torch.int64)
    lean[start] = 6.0
    return (k + lean * u).bfloat16(), v.bfloat16()


def _queries(gen, rows, hq, hkv, d, u):
    return (_normal(gen, rows, hq, d) + u.repeat_interleave(hq // hkv, 0)).bfloat16()


def _plan(lengths):
    """Places of ragged rows in a padded [B, max] layout: token of every place (0 behind a sequence),
    its validity, and (sequence, place) of every token."""
    n = torch.tensor(lengths, device="cuda")
    first = torch.tensor(_offsets(lengths)[:-1], device="cuda")
    t = torch.arange(max(max(lengths), 1), device="cuda")
    ok = t < n[:, None]
    return dict(n=n, t=t, ok=ok, at=torch.where(ok, t + first[:, None], 0), of=ok.nonzero(as_tuple=True))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d, op = case["hq"], case["hkv"], case["d"], case["op"]
    u = _normal(gen, hkv, d)
    u = u / u.norm(dim=-1, keepdim=True)
    s = dict(case=case, scale=1.0 / math.sqrt(d))

    def offsets(lengths):
        return torch.tensor(_offsets(lengths), dtype=torch.int32, device="cuda")

    if op == "prefill":
        new, ctx = _lengths(case, "n", case["batch"], 1), _lengths(case, "c", case["batch"], 2)
        lens = [a + b for a, b in zip(new, ctx)]
        s["new"], s["lens"] = new, lens
        s["k"], s["v"] = _cache(gen, lens, hkv, d, u)
        s["q"] = _queries(gen, sum(new) + case["pad"], hq, hkv, d, u)
        s["offsets"], s["q_offsets"] = offsets(lens), offsets(new)
        s["out"] = torch.zeros_like(s["q"])
    elif op == "prefix":
        plens, start = _prefixes(case)
        lens = _lengths(case, "s", case["batch"], 1)
        s["plens"], s["start"], s["lens"] = plens, start, lens
        s["pk"], s["pv"] = _cache(gen, plens, hkv, d, u)
        s["k"], s["v"] = _cache(gen, lens, hkv, d, u)
        s["q"] = _queries(gen, case["batch"], hq, hkv, d, u)
        s["p_offsets"], s["offsets"] = offsets(plens), offsets(lens)
        s["seq_start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    else:
        lens = _lengths(case, "l", case["batch"], 1)
        s["lens"] = lens
        s["k"], s["v"] = _cache(gen, lens, hkv, d, u)
        s["offsets"] = offsets(lens)
        # weights so far: heavy-tailed, a tenth of the tokens exactly zero (nothing attended to them)
        m = torch.rand((hkv, sum(lens)), generator=gen, device="cuda")
        zero = torch.rand((hkv, sum(lens)), generator=gen, device="cuda") < 0.1
        s["mass"] = torch.where(zero, 0.0, 0.01 / (m + 1e-3))
        if op == "accum":
            s["q"] = _queries(gen, case["batch"], hq, hkv, d, u)
            s["mass_out"] = torch.zeros_like(s["mass"])
        else:
            kept = [min(n, case["budget"]) for n in lens]
            s["kept"] = kept
            s["dk"] = torch.zeros((sum(kept), hkv, d), dtype=torch.bfloat16, device="cuda")
            s["dv"], s["d_offsets"] = torch.zeros_like(s["dk"]), offsets(kept)
            s["d_mass"] = torch.zeros((hkv, sum(kept)), device="cuda")
            s["d_lengths"] = torch.zeros(case["batch"], dtype=torch.int32, device="cuda")
    # where the ragged rows stand: the index plan that a program keeps beside its batch
    s["plan"] = _plan(s["lens"])
    if op == "evict":
        s["kept_of"] = _plan(s["kept"])["of"]
    if op == "prefill":
        s["q_plan"] = _plan(s["new"])
    if op == "prefix":
        def of(ns):
            return torch.tensor([i for i, n in enumerate(ns) for _ in range(n)], device="cuda")
        s["p_of_token"], s["p_of_seq"] = of(plens), of([b - a for a, b in zip(start, start[1:])])
    if own:  # the step object a serving program keeps: cache descriptors and workspace
        s["step"] = _step(s)
    return s


# ------------------------------------------------------------------------------------ the framework

def _step(s):
    from token_sparse_decode_b200 import step

    c = s["case"]
    op, lens = c["op"], s["lens"]
    if op == "prefill":
        return step.PrefillStep(s["k"], s["v"], s["offsets"], max(lens), sum(lens), c["hq"], _roles(c), c["sink"], c["window"],
                                s["scale"], s["q"].shape[0])
    if op == "prefix":
        return step.PrefixDecodeStep(s["pk"], s["pv"], s["p_offsets"], max(s["plens"]), sum(s["plens"]), s["k"], s["v"],
                                     s["offsets"], max(lens), sum(lens), c["hq"], s["scale"], seq_start=s["seq_start"])
    if op == "accum":
        return step.AccumDecodeStep(s["k"], s["v"], s["offsets"], max(lens), sum(lens), c["hq"], s["scale"], decay=c["decay"])
    return step.EvictStep(s["k"], s["v"], s["offsets"], max(lens), sum(lens), s["dk"], s["dv"], s["d_offsets"],
                          max(s["kept"]), sum(s["kept"]), c["budget"], c["sink"], c["recent"])


# ------------------------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        if op == "prefill":
            return s["step"](s["q"], s["q_offsets"], s["out"])
        if op == "prefix":
            return s["step"](s["q"])
        if op == "accum":
            return [s["step"](s["q"], s["mass"], s["mass_out"]), s["mass_out"]]
        idx, count = s["step"](s["mass"], s["d_mass"], s["d_lengths"])
        return [s["dk"], s["dv"], s["d_mass"], s["d_lengths"], idx, count]
    return {"prefill": _prefill, "prefix": _prefix, "accum": _accum, "evict": _evict}[op](s)


def _softmax(x):
    """Softmax of the last axis in fp32; a row of nothing but -inf gives zeros."""
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    t = e.sum(-1, keepdim=True)
    return e / torch.where(t == 0, 1.0, t)


def _prefill(s):
    c = s["case"]
    B, hkv, d = c["batch"], c["hkv"], c["d"]
    g = c["hq"] // hkv
    plan, qplan = s["plan"], s["q_plan"]
    at, ok, t, qat = plan["at"], plan["ok"], plan["t"], qplan["at"]
    pos = (plan["n"] - qplan["n"])[:, None] + qplan["t"]  # [B, n]
    past = (t <= pos[:, :, None]) & ok[:, None, :]  # [B, n, L]
    window = past & ((t < c["sink"]) | (t > pos[:, :, None] - c["window"]))
    seen = torch.stack([past if r == DENSE else window for r in _roles(c)], 1)  # [B, Hkv, n, L]
    q = s["q"].float()[qat].view(B, -1, hkv, g, d).permute(0, 2, 3, 1, 4)  # [B, Hkv, g, n, d]
    k, v = (x.float()[at].permute(0, 2, 3, 1) for x in (s["k"], s["v"]))  # [B, Hkv, d, L]
    x = torch.matmul(q.reshape(B, hkv, -1, d), k).view(B, hkv, g, *seen.shape[2:]) * s["scale"]
    x.masked_fill_(~seen[:, :, None], -math.inf)
    o = torch.matmul(_softmax(x).view(B, hkv, -1, at.shape[1]), v.transpose(2, 3))
    o = o.view(B, hkv, g, -1, d).permute(0, 3, 1, 2, 4).reshape(B, -1, c["hq"], d)
    of = qplan["of"]
    s["out"][:of[0].shape[0]] = o[of].bfloat16()
    return s["out"]


def _prefix(s):
    c = s["case"]
    B, hkv, d = c["batch"], c["hkv"], c["d"]
    q = s["q"].float().view(B, hkv, -1, d)
    at, ok = s["plan"]["at"], s["plan"]["ok"]
    if s["k"].shape[0]:
        k, v = s["k"].float()[at], s["v"].float()[at]  # [B, L, Hkv, d]
    else:
        k = v = torch.zeros((B, at.shape[1], hkv, d), device="cuda")
    own_x = torch.einsum("bhgd,blhd->bhgl", q, k).masked_fill_(~ok[:, None, None, :], -math.inf)
    pk, pv = s["pk"].float(), s["pv"].float()
    x = torch.einsum("bhgd,lhd->bhgl", q, pk)
    x.masked_fill_((s["p_of_token"] != s["p_of_seq"][:, None])[:, None, None, :], -math.inf)
    w = _softmax(torch.cat([x, own_x], -1) * s["scale"])
    o = torch.einsum("bhgl,lhd->bhgd", w[..., :pk.shape[0]], pv) + torch.einsum("bhgl,blhd->bhgd", w[..., pk.shape[0]:], v)
    return o.reshape(B, c["hq"], d)


def _accum(s):
    c = s["case"]
    B, hkv, d = c["batch"], c["hkv"], c["d"]
    q = s["q"].float().view(B, hkv, -1, d)
    at, ok = s["plan"]["at"], s["plan"]["ok"]
    k, v = s["k"].float()[at], s["v"].float()[at]
    x = torch.einsum("bhgd,blhd->bhgl", q, k) * s["scale"]
    w = _softmax(x.masked_fill_(~ok[:, None, None, :], -math.inf))
    o = torch.einsum("bhgl,blhd->bhgd", w, v)
    seq, place = s["plan"]["of"]
    add = w.sum(2)[seq, :, place].t()  # [Hkv, T]
    return [o.reshape(B, c["hq"], d), c["decay"] * s["mass"] + add]


def _evict(s):
    c = s["case"]
    hkv, budget = c["hkv"], c["budget"]
    at, ok, L, t = (s["plan"][key] for key in ("at", "ok", "n", "t"))
    held = ok & ((t < c["sink"]) | (t >= L[:, None] - c["recent"]))
    x = s["mass"][:, at].permute(1, 0, 2).masked_fill(held[:, None], math.inf).masked_fill(~ok[:, None], -math.inf)
    order = torch.sort(x, dim=-1, descending=True, stable=True)[1][..., :budget]  # equal weights: the lower place
    if order.shape[-1] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]), value=at.shape[1])
    count = torch.clamp(L, max=budget)
    keep = torch.arange(budget, device="cuda") < count[:, None]
    big = torch.iinfo(torch.int64).max
    idx = torch.where(keep[:, None], order, big).sort(-1)[0]  # [B, Hkv, budget], ascending
    seq, place = s["kept_of"]
    src = idx[seq, :, place] + s["offsets"][seq, None]  # [kept, Hkv]
    head = torch.arange(hkv, device="cuda")
    s["dk"].copy_(s["k"][src, head])
    s["dv"].copy_(s["v"][src, head])
    return [s["dk"], s["dv"], s["mass"][head, src].t().contiguous(), count.int(),
            torch.where(keep[:, None], idx, -1).int(), count[:, None].expand(-1, hkv).int().contiguous()]


# ------------------------------------------------------------------------------------ work and definition

def _seen_pairs(case):
    """(query, token) pairs that are visible, summed over KV heads, and the KV rows that any query sees."""
    new, ctx = _lengths(case, "n", case["batch"], 1), _lengths(case, "c", case["batch"], 2)
    pairs = rows = 0
    for n, p0 in zip(new, ctx):
        dense = n * p0 + n * (n + 1) // 2
        stream = 0
        for p in range(p0, p0 + n):
            first = min(case["sink"], p + 1)
            stream += first + p + 1 - max(first, p + 1 - case["window"])
        first = min(case["sink"], p0 + n)
        pairs += case["dense"] * dense + (case["hkv"] - case["dense"]) * stream
        rows += case["dense"] * (p0 + n) + (case["hkv"] - case["dense"]) * (
            first + p0 + n - max(first, p0 + 1 - case["window"]) if case["window"] else first)
    return pairs, rows, sum(new)


def work(case):
    hq, hkv, d, B = case["hq"], case["hkv"], case["d"], case["batch"]
    g = hq // hkv
    if case["op"] == "prefill":
        pairs, rows, n = _seen_pairs(case)
        return {"bytes": 4 * d * rows + 4 * n * hq * d, "flops": 4 * d * g * pairs}
    if case["op"] == "prefix":
        plens, start = _prefixes(case)
        lens = _lengths(case, "s", B, 1)
        pairs = sum(lens) + sum(p * (b - a) for p, a, b in zip(plens, start, start[1:]))
        return {"bytes": 4 * d * hkv * (sum(plens) + sum(lens)) + 6 * B * hq * d, "flops": 4 * d * hq * pairs}
    lens = _lengths(case, "l", B, 1)
    if case["op"] == "accum":
        return {"bytes": (4 * d + 8) * hkv * sum(lens) + 6 * B * hq * d, "flops": 4 * d * hq * sum(lens)}
    kept = sum(min(n, case["budget"]) for n in lens)
    return {"bytes": hkv * (4 * sum(lens) + (8 * d + 4) * kept + 4 * B * case["budget"]), "flops": 2 * hkv * sum(lens)}


def _attend64(q, k, v, seen, scale):
    """float64 weights and outputs of queries [r, d] over rows [l, d]; seen [r, l] or None."""
    x = (q @ k.t()) * scale
    if seen is not None:
        x = x.masked_fill(~seen, -math.inf)
    if x.shape[1] == 0:
        return x, torch.zeros_like(q)
    w = torch.softmax(x, -1).nan_to_num(0.0)
    return w, w @ v


def exact(case, seed):
    s = prepare(case, seed)
    c, B, hkv, d = case, case["batch"], case["hkv"], case["d"]
    g, scale = c["hq"] // hkv, 1.0 / math.sqrt(d)
    op, off = c["op"], _offsets(s["lens"])
    if op == "evict":
        dk, dv, dm = s["dk"].double(), s["dv"].double(), s["d_mass"].double()
        doff = _offsets(s["kept"])
        for b in range(B):
            n, o = s["lens"][b], off[b]
            for h in range(hkv):
                m = s["mass"][h, o:o + n].double()
                m[:c["sink"]] = math.inf
                m[max(0, n - c["recent"]):] = math.inf
                # rank of a token: tokens heavier than it, and equal ones before it
                keep = torch.argsort(-m, stable=True)[:c["budget"]].sort()[0]
                dk[doff[b]:doff[b + 1], h] = s["k"][o + keep, h].double()
                dv[doff[b]:doff[b + 1], h] = s["v"][o + keep, h].double()
                dm[h, doff[b]:doff[b + 1]] = s["mass"][h, o + keep].double()
        return [dk, dv, dm, None, None, None]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    if op == "prefill":
        qoff = _offsets(s["new"])
        for b in range(B):
            n, L, o = s["new"][b], s["lens"][b], off[b]
            p = torch.arange(L - n, L, device="cuda")[:, None]
            t = torch.arange(L, device="cuda")[None, :]
            for h in range(c["hq"]):
                seen = t <= p
                if h // g >= c["dense"]:
                    seen = seen & ((t < c["sink"]) | (t >= p + 1 - c["window"]))
                out[qoff[b]:qoff[b + 1], h] = _attend64(s["q"][qoff[b]:qoff[b + 1], h].double(), s["k"][o:o + L, h // g].double(),
                                                        s["v"][o:o + L, h // g].double(), seen, scale)[1]
        return out
    mass = s["mass"].double() * c["decay"] if op == "accum" else None
    for b in range(B):
        rows = slice(off[b], off[b + 1])
        k, v = s["k"][rows], s["v"][rows]
        if op == "prefix":
            i = next(j for j in range(c["np"]) if s["start"][j] <= b < s["start"][j + 1])
            po = _offsets(s["plens"])
            k, v = torch.cat([s["pk"][po[i]:po[i + 1]], k]), torch.cat([s["pv"][po[i]:po[i + 1]], v])
        for h in range(hkv):
            w, o = _attend64(s["q"][b, h * g:(h + 1) * g].double(), k[:, h].double(), v[:, h].double(), None, scale)
            out[b, h * g:(h + 1) * g] = o
            if op == "accum":
                mass[h, rows] += w.sum(0)
    return out if op == "prefix" else [out, mass]
