"""Operators of decoding with a shared prefix and with a cache that evicts: their cases, plain forms and exact values.

  shared   attention of many query tokens over one sequence of a bf16 cache: the prefix that a batch shares,
           read once for all of them; with `joined`, merged with an attention over each query's own tokens
  coded    the same over one sequence of a coded cache: its keys and values are rebuilt once for all queries
  scored   decode attention over a bf16 cache that adds every token's attention weight to its score
  evict    eviction from a bf16 cache: sinks, recent tokens and the highest scores stay within a budget

Every operator has its plain form in torch operations (fp32, rounded once), its call into the library, and its
definition in fp64.
"""
import math

import torch

own = False

DEV = "cuda"
THETA = 1.0e4
LOOPS = 4                                                     # loop steps of the coded cases


# ------------------------------------------------------------------ cases

def _shared(name, n, rows, hkv, hq, d, joined, start=0, seqs=1, seq=0):
    return dict(name=name, op="shared", n=n, rows=rows, hkv=hkv, hq=hq, d=d, joined=joined, start=start, seqs=seqs,
                seq=seq)


def _coded(name, n, rows, hkv, hq, d, c, joined, start=0, seqs=1, seq=0, tc=4, ncb=1, t=1):
    return dict(name=name, op="coded", n=n, rows=rows, hkv=hkv, hq=hq, d=d, c=c, joined=joined, start=start, seqs=seqs,
                seq=seq, tc=tc, ncb=ncb, t=t)


def _scored(name, b, n, hkv, hq, d, joined, ragged):
    return dict(name=name, op="scored", b=b, n=n, hkv=hkv, hq=hq, d=d, joined=joined, ragged=ragged)


def _evict(name, b, n, hkv, d, budget, sink, recent, ragged):
    return dict(name=name, op="evict", b=b, n=n, hkv=hkv, d=d, budget=budget, sink=sink, recent=recent, ragged=ragged)


def listed():
    return [
        # a few requests behind a system prompt of a thousand tokens: latency counts
        _shared("shared 1000 x 3", 1000, 3, 16, 16, 128, False),
        # a full batch behind a few-shot prompt, each with its own answer so far
        _shared("shared 4096 x 32 joined", 4096, 32, 16, 16, 128, True),
        # a long document asked several questions at once: the cache's bytes count
        _shared("shared 32768 x 8 joined", 32768, 8, 16, 16, 128, True),
        # a large batch with grouped heads: 256 query rows per key head, an odd length
        _shared("shared 16347 x 64 gqa joined", 16347, 64, 4, 16, 128, True),
        # one query on the smallest coded shape
        _coded("coded 250 x 1 d64", 250, 1, 1, 1, 64, 4, False),
        # the long document held at half a bit per element
        _coded("coded 32768 x 32 joined", 32768, 32, 16, 16, 128, 4, True),
        # grouped heads at a quarter of a bit, an odd length
        _coded("coded 16379 x 64 gqa joined", 16379, 64, 4, 16, 128, 8, True),
        # one short request
        _scored("scored 1 x 500 d64", 1, 500, 2, 4, 64, False, False),
        # a full batch behind a shared prefix: weights of the joint softmax
        _scored("scored 32 x 4096 joined", 32, 4096, 16, 16, 128, True, False),
        # grouped heads, requests of many lengths
        _scored("scored 16 x 16384 gqa ragged", 16, 16384, 4, 16, 128, False, True),
        # one token too many, in every step of a full batch
        _evict("evict 32 x 2049 to 2048", 32, 2049, 16, 128, 2048, 8, 64, False),
        # the cut after a long prompt
        _evict("evict 2 x 32768 to 4096", 2, 32768, 16, 128, 4096, 8, 64, False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("shared", "coded", "scored", "evict"))
    d = rng.choice((64, 128, 128))
    hkv = rng.choice((1, 2, 4, 8, 16, 40))
    if op in ("shared", "coded"):
        hq = hkv * rng.choice((1, 1, 2, 4, 8))
        rows = _log(rng, 1, 160)
        n = _log(rng, 1, 32768)
        while n * hkv > 32768 * 16 or n * rows * hq > 16347 * 64 * 16 or rows * hq * d > 64 * 40 * 128:
            n, rows = max(1, n * 3 // 4), max(1, rows * 7 // 8)
        start = rng.choice((0, 0, rng.randrange(n)))
        seqs = rng.choice((1, 2, 3))
        seq = rng.randrange(seqs)
        joined = rng.random() < 0.5
        if op == "shared":
            c = _shared("", n, rows, hkv, hq, d, joined, start, seqs, seq)
        else:
            width, tc = rng.choice(((4, 4), (8, 4), (16, 2), (16, 1), (32, 1)))
            per_group = rng.random() < 0.2
            c = _coded("", n, rows, hkv, hq, d, width, joined, start, seqs, seq, tc, d // width if per_group else 1,
                       rng.randrange(LOOPS))
    elif op == "scored":
        hq = hkv * rng.choice((1, 1, 2, 4, 8))
        b, n = _log(rng, 1, 64), _log(rng, 1, 32768)
        while b * n * hkv * d > 16 * 16384 * 4 * 128:
            b, n = max(1, b * 7 // 8), max(1, n * 3 // 4)
        c = _scored("", b, n, hkv, hq, d, rng.random() < 0.5, rng.random() < 0.5)
    else:
        b, n = _log(rng, 1, 64), _log(rng, 200, 32768)
        while b * n * hkv * d > 2 * 32768 * 16 * 128:
            b, n = max(1, b * 7 // 8), max(200, n * 3 // 4)
        budget = rng.choice((max(80, n - rng.randrange(1, 129)), rng.randrange(80, n)))
        recent = rng.choice((0, 16, 64))
        c = _evict("", b, n, hkv, d, budget, rng.choice((0, 4, 8)), recent, rng.random() < 0.5)
    del c["name"]
    return c


def _lens(case):
    """Lengths of the sequences: all n, or spread between nothing and n."""
    b, n = case["b"], case["n"]
    if not case["ragged"]:
        return [n] * b
    return [n if i == 0 else (i * 7919 * n // 10007) % (n + 1) for i in range(b)]


def _nmax(n):
    return (n + 7) // 4 * 4                                   # room behind the last token; a multiple of 4


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _bf16(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _other(g, rows, hq, d, tokens):
    """An attention over other tokens: averages of values, and sums of exponentials of scores near N(0, 1)."""
    out = _randn(g, rows, hq, d) / math.sqrt(tokens)
    lse = math.log(tokens) + 0.5 + 0.1 * _randn(g, rows, hq)
    return out, lse


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=case)
    op, n, d, hkv = case["op"], case["n"], case["d"], case["hkv"]
    nmax = _nmax(n)
    if op in ("shared", "coded"):
        rows, hq, seqs = case["rows"], case["hq"], case["seqs"]
        s["q"] = _bf16(g, rows, hq, d)
        s["starts"] = torch.full((seqs,), case["start"], dtype=torch.int32, device=DEV)
        s["lens"] = torch.full((seqs,), n, dtype=torch.int32, device=DEV)
        s["other"] = _other(g, rows, hq, d, 500) if case["joined"] else None
        if op == "shared":
            s["k"], s["v"] = _bf16(g, seqs, hkv, nmax, d), _bf16(g, seqs, hkv, nmax, d)
        else:
            c, tc, ncb, entries = case["c"], case["tc"], case["ncb"], 256
            nb, words = LOOPS // tc, d // (2 * c)
            s["idx"] = torch.randint(-2 ** 31, 2 ** 31, (1, nb, seqs, hkv, nmax // 4, words, 4), generator=g, device=DEV,
                                     dtype=torch.int32)
            s["codebook"] = _bf16(g, 1, nb, 2, hkv, ncb, entries, c * tc)
            # the slice of every loop step, and the rotation table: cut once when a model is loaded
            cb = s["codebook"].view(1, nb, 2, hkv, ncb, entries, c, tc)
            s["slices"] = cb.permute(0, 1, 7, 2, 3, 5, 4, 6).reshape(1, LOOPS, 2, hkv, entries, ncb * c).contiguous()
            w = THETA ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=DEV) / d)
            a = torch.arange(nmax, dtype=torch.float64, device=DEV)[:, None] * w
            s["rope"] = torch.cat([torch.cos(a), torch.sin(a)], 1).float()
        return s
    b = case["b"]
    s["k"], s["v"] = _bf16(g, b, hkv, nmax, d), _bf16(g, b, hkv, nmax, d)
    s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
    # scores as a run leaves them: a few tokens hold most of the weight, many hold next to nothing, some are equal
    # (each of the last hundred steps has shared out a weight of one)
    s["score"] = torch.exp(2.0 * _randn(g, b, hkv, nmax)) * (torch.rand(b, hkv, nmax, generator=g, device=DEV) < 0.9)
    s["score"] *= 100.0 / (7.0 * n)
    s["score_out"] = torch.zeros_like(s["score"])
    if op == "scored":
        s["q"] = _bf16(g, b, case["hq"], d)
        s["other"] = _other(g, b, case["hq"], d, 2000) if case["joined"] else None
        return s
    # the position that a slot holds: after the sinks a thousand tokens have gone, and some slots, refilled by earlier
    # evictions, lie out of order
    s["next_pos"] = s["lens"] + 1000
    slot = torch.arange(nmax, device=DEV, dtype=torch.int32)
    s["pos"] = torch.where(slot >= 8, slot + 1000, slot).expand(b, hkv, nmax).contiguous()
    some = slice(13, max(13, case["budget"] // 2), 16)
    s["pos"][:, :, some] = s["pos"][:, :, some].roll(3, 2)
    s["pos_out"] = torch.zeros_like(s["pos"])
    s["lens_out"] = torch.zeros_like(s["lens"])
    return s


# ------------------------------------------------------------------ plain forms

def _join(num, m, l, other):
    """out and lse of sum exp(s - m) v = num, sum exp(s - m) = l, with another part's (out, lse) merged in."""
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)
    out = torch.where(l > 0, num / l, 0.0)
    if other is None:
        return out, lse.squeeze(-1)
    oo, ol = other[0], other[1].unsqueeze(-1)
    top = torch.maximum(lse, ol)
    top = torch.where(top == -math.inf, 0.0, top)
    wa, wb = torch.exp(lse - top), torch.exp(ol - top)
    w = wa + wb
    return torch.where(w > 0, (wa * out + wb * oo) / w, 0.0), (torch.where(w > 0, top + torch.log(w), -math.inf)).squeeze(-1)


def _attend_shared(q, k, v, other):
    """q [R][Hq][D], k and v fp32 [Hkv][n][D]: every query attends to every token."""
    rows, hq, d = q.shape
    hkv = k.shape[0]
    qh = q.float().view(rows, hkv, hq // hkv, d).permute(1, 0, 2, 3).reshape(hkv, -1, d)
    s = torch.matmul(qh, k.transpose(1, 2)) * (1.0 / math.sqrt(d))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    back = lambda x: x.view(hkv, rows, hq // hkv, -1).permute(1, 0, 2, 3).reshape(rows, hq, -1)  # noqa: E731
    return _join(back(torch.matmul(p, v)), back(m), back(l), other)


def _rebuild(s, kv, dtype):
    """Keys (kv = 0, rotated) or values (kv = 1) [Hkv][n][D] of the attended tokens, from codes and slices."""
    case = s["case"]
    c, d, ncb, n, start = case["c"], case["d"], case["ncb"], case["n"], case["start"]
    hkv, groups = case["hkv"], d // c
    w = s["idx"][0, case["t"] // case["tc"], case["seq"]].permute(0, 1, 3, 2).reshape(hkv, -1, groups // 2)[:, start:n]
    codes = torch.cat([(w >> (16 * kv)) & 255, (w >> (16 * kv + 8)) & 255], 2).long()      # [Hkv][n][groups]
    table = s["slices"][0, case["t"], kv].to(dtype).view(hkv, 256, ncb, c)
    head = torch.arange(hkv, device=DEV)[:, None, None]
    group = torch.arange(groups, device=DEV) if ncb > 1 else torch.zeros(groups, dtype=torch.long, device=DEV)
    x = table[head, codes, group].reshape(hkv, n - start, d)
    if kv:
        return x
    cos, sin = s["rope"][start:n, :d // 2].to(dtype), s["rope"][start:n, d // 2:].to(dtype)
    a, b = x[..., :d // 2], x[..., d // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_scored(s):
    case, q = s["case"], s["q"]
    b, hq, d = q.shape
    hkv, nmax = case["hkv"], s["k"].shape[2]
    x = torch.matmul(q.float().view(b, hkv, hq // hkv, d), s["k"].float().transpose(2, 3)) * (1.0 / math.sqrt(d))
    there = (torch.arange(nmax, device=DEV) < s["lens"][:, None])[:, None, None]           # [B][1][1][Nmax]
    x = torch.where(there, x, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    num = torch.matmul(p, s["v"].float())
    out, lse = _join(num.reshape(b, hq, d), m.reshape(b, hq, 1), l.reshape(b, hq, 1), s["other"])
    at = lse.view(b, hkv, -1, 1)
    p = torch.where(there, torch.exp(x - torch.where(at == -math.inf, 0.0, at)), 0.0)
    s["score_out"].copy_(torch.where(there[:, 0], s["score"] + p.sum(2), s["score_out"]))
    return dict(out=out, lse=lse, score=s["score_out"])


def _plain_evict(s):
    case, lens = s["case"], s["lens"]
    budget, nmax = case["budget"], s["k"].shape[2]
    slot = torch.arange(nmax, device=DEV)
    valid = slot < lens[:, None, None]
    # scores in the order of whole numbers: minus infinity and NaN lowest, kept positions above all
    bits = (s["score"] + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, -2 ** 31 - bits - 1)
    key = torch.where(torch.isnan(s["score"]), -2 ** 32, key)
    fixed = (s["pos"] < case["sink"]) | (s["pos"] >= s["next_pos"][:, None, None] - case["recent"])
    key = torch.where(valid, torch.where(fixed, 2 ** 32, key), -2 ** 33)
    order = torch.sort(key, dim=2, descending=True, stable=True).indices                   # ties: the lowest slot first
    rank = torch.empty_like(order).scatter_(2, order, slot.expand_as(order))
    kept = (rank < budget) & valid
    # the i-th emptied slot below the budget takes the i-th kept token above it
    hole = ~kept & (slot < budget) & valid
    above = torch.where(kept & (slot >= budget), slot, nmax).sort(2).values
    take = torch.where(hole, above.gather(2, (hole.long().cumsum(2) - 1).clamp(min=0)), slot)
    take = torch.where(take < nmax, take, slot)
    new = torch.clamp(lens, max=budget)
    live = slot < new[:, None, None]
    s["score_out"].copy_(torch.where(live, s["score"].gather(2, take), s["score_out"]))
    s["pos_out"].copy_(torch.where(live, s["pos"].gather(2, take), s["pos_out"]))
    s["lens_out"].copy_(new)
    at = take[:, :, :budget, None].expand(-1, -1, -1, case["d"])
    for x in (s["k"], s["v"]):
        x[:, :, :budget] = x.gather(2, at)
    return dict(k=s["k"], v=s["v"], score=s["score_out"], pos=s["pos_out"], lens=s["lens_out"])


def _plain(s):
    case = s["case"]
    if case["op"] == "shared":
        part = lambda x: x[case["seq"], :, case["start"]:case["n"]].float()  # noqa: E731
        out, lse = _attend_shared(s["q"], part(s["k"]), part(s["v"]), s["other"])
        return dict(out=out, lse=lse)
    if case["op"] == "coded":
        out, lse = _attend_shared(s["q"], _rebuild(s, 0, torch.float32), _rebuild(s, 1, torch.float32), s["other"])
        return dict(out=out, lse=lse)
    return _plain_scored(s) if case["op"] == "scored" else _plain_evict(s)


# ------------------------------------------------------------------ the library's calls

def _own(s):
    import looped_lm_decode_b200 as LQ
    case = s["case"]
    op, n = case["op"], case["n"]
    if op == "coded":
        cache = LQ.Cache(1, LOOPS, case["tc"], case["hkv"], case["hq"], case["d"], case["c"], 256, case["seqs"],
                         _nmax(n), THETA, alloc=False, ncb=case["ncb"])
        cache.idx, cache.codebook, cache.slices, cache.rope = s["idx"], s["codebook"], s["slices"], s["rope"]
        out, lse = LQ.shared_attn(cache, 0, case["t"], case["seq"], s["q"], s["lens"], n, starts=s["starts"],
                                  other=s["other"])
        return dict(out=out, lse=lse)
    cache = LQ.Bf16Cache(s["k"], s["v"], case["hkv"] if op == "evict" else case["hq"])
    if op == "shared":
        out, lse = LQ.bf16_shared_attn(cache, case["seq"], s["q"], s["lens"], n, starts=s["starts"], other=s["other"])
        return dict(out=out, lse=lse)
    if op == "scored":
        out, lse, score = LQ.bf16_decode_attn_scored(cache, s["q"], s["lens"], n, s["score"], score_out=s["score_out"],
                                                     other=s["other"])
        return dict(out=out, lse=lse, score=score)
    score, pos, lens = LQ.bf16_evict(cache, s["score"], s["pos"], s["lens"], s["next_pos"], n, case["budget"],
                                     case["sink"], case["recent"], score_out=s["score_out"], pos_out=s["pos_out"],
                                     lens_out=s["lens_out"])
    return dict(k=s["k"], v=s["v"], score=score, pos=pos, lens=lens)


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------ work and exact values

def work(case):
    op, n, d, hkv = case["op"], case["n"], case["d"], case["hkv"]
    if op in ("shared", "coded"):
        rows, hq, tokens = case["rows"], case["hq"], n - case["start"]
        io = rows * hq * (2 * d + (4 * d + 4) * (2 if case["joined"] else 1))
        if op == "shared":
            cache = tokens * hkv * 4 * d
        else:
            cache = tokens * hkv * 2 * (d // case["c"]) + tokens * 4 * d + hkv * 2 * 256 * case["c"] * case["ncb"] * 2
        return {"bytes": cache + io, "flops": 4 * rows * hq * d * tokens}
    tokens = sum(_lens(case))
    if op == "scored":
        io = case["b"] * case["hq"] * (2 * d + (4 * d + 4) * (2 if case["joined"] else 1))
        return {"bytes": tokens * hkv * (4 * d + 8) + io, "flops": 4 * tokens * case["hq"] * d}
    # scores and positions read and the kept ones written; the rows that move, read and written: about as many as the
    # share of the kept tokens that lies behind the budget
    moved = sum(min(x, case["budget"]) * max(0, x - case["budget"]) / max(1, x) for x in _lens(case))
    kept = sum(min(x, case["budget"]) for x in _lens(case))
    return {"bytes": hkv * (tokens * 8 + kept * 8 + moved * 8 * d), "flops": hkv * tokens}


def _exact_part(q, k, v, other_out, other_lse):
    """One query head in fp64: q [R][D], k and v [n][D]."""
    s = (q @ k.T) / math.sqrt(q.shape[1])
    lse = torch.logsumexp(s, 1)
    out = torch.softmax(s, 1) @ v
    if other_lse is None:
        return out, lse
    both = torch.logaddexp(lse, other_lse)
    return torch.exp(lse - both)[:, None] * out + torch.exp(other_lse - both)[:, None] * other_out, both


def _exact_keys(s, h):
    """Rotated keys and values of one KV head in fp64, from the codebook's own coordinates and fp64 angles."""
    case = s["case"]
    c, d, tc, n = case["c"], case["d"], case["tc"], case["n"]
    groups, half = d // c, d // (2 * c)
    block, m = divmod(case["t"], tc)
    token = torch.arange(case["start"], n, device=DEV)
    word = s["idx"][0, block, case["seq"], h].long() % 2 ** 32                             # [Nmax/4][NP][4]
    parts = []
    for kv in range(2):
        x = torch.empty(len(token), d, dtype=torch.float64, device=DEV)
        for g in range(groups):
            byte = 2 * kv + (g >= half)
            code = (word[token // 4, g % half, token % 4] // 256 ** byte) % 256
            book = s["codebook"][0, block, kv, h, g if case["ncb"] > 1 else 0].double()    # [K][c*tc]
            x[:, g * c:(g + 1) * c] = book[code][:, m::tc]
        parts.append(x)
    f = torch.arange(d // 2, dtype=torch.float64, device=DEV)
    turn = torch.exp(1j * token[:, None].double() * torch.exp(-2 * f / d * math.log(THETA)))
    z = torch.complex(parts[0][:, :d // 2], parts[0][:, d // 2:]) * turn
    return torch.cat([z.real, z.imag], 1), parts[1]


def exact(case, seed):
    s = prepare(case, seed)
    op, hkv = case["op"], case["hkv"]
    if op in ("shared", "coded"):
        group = case["hq"] // hkv
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
        for h in range(hkv):
            if op == "shared":
                k = s["k"][case["seq"], h, case["start"]:case["n"]].double()
                v = s["v"][case["seq"], h, case["start"]:case["n"]].double()
            else:
                k, v = _exact_keys(s, h)
            for j in range(h * group, (h + 1) * group):
                o = (s["other"][0][:, j].double(), s["other"][1][:, j].double()) if case["joined"] else (None, None)
                out[:, j], lse[:, j] = _exact_part(s["q"][:, j].double(), k, v, *o)
        return dict(out=out, lse=lse)
    if op == "scored":
        group = case["hq"] // hkv
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
        score = torch.zeros(s["score"].shape, dtype=torch.float64, device=DEV)
        for i, n in enumerate(_lens(case)):
            k, v = s["k"][i, :, :n].double(), s["v"][i, :, :n].double()
            q = s["q"][i].double().view(hkv, group, -1)
            x = q @ k.transpose(1, 2) / math.sqrt(case["d"])
            alone = torch.logsumexp(x, 2)                                                  # of no token: -inf
            both = alone
            o = torch.softmax(x, 2) @ v
            if case["joined"]:
                there = s["other"][1][i].double().view(hkv, group)
                both = torch.logaddexp(alone, there)
                o = torch.exp(alone - both)[..., None] * o
                o = o + torch.exp(there - both)[..., None] * s["other"][0][i].double().view(hkv, group, -1)
            out[i], lse[i] = o.reshape(-1, case["d"]), both.reshape(-1)
            score[i, :, :n] = s["score"][i, :, :n].double() + torch.exp(x - both[..., None]).sum(1)
        return dict(out=out, lse=lse, score=score)
    # eviction only chooses and copies: whole numbers and values that are moved
    score, pos = s["score"].double().cpu(), s["pos"].cpu()
    k, v = s["k"].double(), s["v"].double()
    score_out, pos_out = torch.zeros_like(score), torch.zeros_like(pos)
    budget = case["budget"]
    for i, n in enumerate(_lens(case)):
        until = int(s["next_pos"][i]) - case["recent"]
        for h in range(hkv):
            p, x = pos[i, h, :n], score[i, h, :n].clone()
            x[(p < case["sink"]) | (p >= until)] = math.inf
            best = torch.argsort(-x, stable=True)[:budget]
            left = torch.ones(n, dtype=torch.bool)
            left[best] = False
            into = torch.nonzero(left[:budget]).view(-1)
            frm = budget + torch.nonzero(~left[budget:]).view(-1) if n > budget else into
            a = torch.arange(min(n, budget))
            a[into] = frm
            score_out[i, h, :len(a)], pos_out[i, h, :len(a)] = score[i, h, a], pos[i, h, a]
            if len(into):
                to, src = into.to(DEV), frm.to(DEV)
                k[i, h, to], v[i, h, to] = k[i, h, src], v[i, h, src]
    return dict(k=k, v=v, score=score_out, pos=pos_out, lens=torch.clamp(s["lens"], max=budget))
