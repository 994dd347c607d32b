"""Cases that time the operators of token-by-token decoding between int8 layers.

The int8 projections and their adapters give the queries, keys and values of
each new token and, at the end, its logits. What lies between are the paged
key-value cache, the attention that reads it and beam search, in the sizes of
the layers that this repository works with (768, 4096 and 12288 features wide)
and in odd ones:

  append    the new tokens' keys and values into their pages
  attend    attention of one new token of each sequence over its pages
  fork      beams follow their parents: pages are shared, copied, freed, allocated
  compact   the pages in use move to the front of the pool
  select    the best continuations over a request's beams and the vocabulary

`own` false: the plain form in elementary torch operations in 32 bits (64 where
scores are compared); true: the library's kernels. Both take what prepare()
gives.
"""

import math
import random

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4}


def listed():
    return [
        # one decoded token of each of 64 requests of the widest layer goes into its page
        dict(name="append decode", op="append", requests=64, new=1, L=2048, kv=96, d=128, page=16, x="f16"),
        # five prompts of uneven lengths fill their pages behind a short system prompt
        dict(name="append prompts", op="append", requests=5, new=4101, L=1100, kv=32, d=128, page=32, x="bf16"),
        # the narrowest layer, one request, little said yet: latency only
        dict(name="attend short", op="attend", requests=1, beams=1, own=0, lo=131, L=131, heads=12, kv=12, d=64, page=16,
             alibi=False, x="f16"),
        # the widest layer's decode batch: 64 requests from a few tokens to a full context
        dict(name="attend batch", op="attend", requests=64, beams=1, own=0, lo=3, L=2048, heads=96, kv=96, d=128, page=16,
             alibi=False, x="f16"),
        # long documents under heads that share keys and values by eight
        dict(name="attend long", op="attend", requests=16, beams=1, own=0, lo=1000, L=32767, heads=64, kv=8, d=128,
             page=64, alibi=False, x="bf16"),
        # beam search: eight requests, four beams each, which share all but their last tokens; linear position biases
        dict(name="attend beams", op="attend", requests=8, beams=4, own=45, lo=700, L=2040, heads=32, kv=32, d=128,
             page=16, alibi=True, x="f16"),
        # a small beam search moves on by one token
        dict(name="fork few", op="fork", requests=4, beams=4, alive=2, own=19, lo=90, L=333, kv=12, d=64, page=16,
             pools=2, spare=40, x="f16"),
        # many beams of many requests over the pools of two layers
        dict(name="fork many", op="fork", requests=64, beams=4, alive=3, own=45, lo=500, L=2040, kv=8, d=128, page=16,
             pools=4, spare=1500, x="bf16"),
        # a pool that few sequences are left in
        dict(name="compact few", op="compact", requests=9, L=300, lo=20, kv=12, d=64, page=16, pools=2, holes=0.7, x="f16"),
        # a large pool in which every other page was freed, two layers
        dict(name="compact pool", op="compact", requests=61, L=2048, lo=900, kv=8, d=128, page=16, pools=4, holes=0.5,
             x="bf16"),
        # one request's four beams over a vocabulary that no vector divides
        dict(name="select one", op="select", requests=1, beams=4, k=4, vocab=50257, T=37, x="f16"),
        # a full batch, eight beams each, twice as many kept as there are beams (some may have ended)
        dict(name="select batch", op="select", requests=64, beams=8, k=16, vocab=50272, T=700, x="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "fork", "compact", "select"])
    x, page, d = rng.choice(["f16", "bf16"]), rng.choice([16, 16, 32, 64, 128]), rng.choice([64, 80, 96, 128, 128, 256])
    if op == "select":
        requests, beams = _log_int(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 8])
        vocab = min(_log_int(rng, 257, 250000), 25_700_000 // (requests * beams))
        return dict(op=op, requests=requests, beams=beams, k=beams * rng.choice([1, 2]), vocab=vocab,
                    T=_log_int(rng, 1, 1000), x=rng.choice(["f16", "bf16", "f32"]))
    if op == "append":
        requests, kv = _log_int(rng, 1, 128), rng.choice([1, 4, 8, 12, 32, 40, 96])
        new = rng.choice([1, 1, _log_int(rng, 2, 4096)])
        new = max(1, min(new, 16_000_000 // (requests * kv * d)))
        return dict(op=op, requests=requests, new=new, L=_log_int(rng, 1, 1024), kv=kv, d=d, page=page, x=x)
    if op == "compact":
        return dict(op=op, requests=_log_int(rng, 1, 61), L=_log_int(rng, 30, 2048), lo=rng.choice([1, 20]), kv=rng.choice([1, 4, 8]),
                    d=rng.choice([64, 128]), page=rng.choice([16, 16, 32]), pools=rng.choice([1, 2, 4]),
                    holes=rng.choice([0.1, 0.5, 0.5, 0.8]), x=x)
    if op == "fork":
        beams, L = rng.choice([2, 3, 4, 5, 8]), _log_int(rng, 20, 2040)
        return dict(op=op, requests=_log_int(rng, 1, 256 // beams), beams=beams, alive=rng.randint(1, beams), own=rng.randint(1, 60),
                    lo=max(1, L // 3), L=L, kv=rng.choice([1, 4, 8]), d=rng.choice([64, 128]), page=rng.choice([16, 16, 32]),
                    pools=rng.choice([1, 2, 4]), spare=300, x=x)
    kv, group = rng.choice([(1, 8), (2, 4), (4, 1), (8, 1), (8, 8), (12, 1), (32, 1), (40, 1), (8, 4), (96, 1), (5, 3), (4, 16)])
    beams = rng.choice([1, 1, 1, 2, 4, 5])
    requests, L = _log_int(rng, 1, 64), _log_int(rng, 1, 32768)
    L = max(1, min(L, 390_000_000 // (requests * beams * kv * d), 2_100_000_000 // (requests * beams * kv * group * d)))
    return dict(op=op, requests=requests, beams=beams, own=rng.randint(1, 100), lo=rng.choice([1, max(1, L // 2), L]), L=L,
                heads=kv * group, kv=kv, d=d, page=page, alibi=rng.random() < 0.3, x=x)


# ------------------------------------------------------------------ the caches that the cases start from

def _lens(case):
    """The requests' lengths: spread evenly from lo to L."""
    n, lo, hi = case["requests"], min(case["lo"], case["L"]), case["L"]
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _split(case, length):
    """(pages that a request's beams share, pages that each has for itself)."""
    pages = -(-length // case["page"])
    shared = max(0, length - case["own"]) // case["page"] if case["beams"] > 1 else 0
    return shared, pages - shared


def _cache(case, rng, spare):
    """(lens, tables, refs) of the beams of all requests, on pages in no order; unused entries are -1."""
    lens, beams = _lens(case), case.get("beams", 1)
    rng.shuffle(lens)
    parts = [_split({"beams": 1, "own": 0, **case}, length) for length in lens]
    need = sum(s + beams * o for s, o in parts)
    ids = rng.sample(range(need + spare), need)
    refs, tables = [0] * (need + spare), []
    width = -(-(case["L"] + 1) // case["page"])
    for shared, mine in parts:
        common = [ids.pop() for _ in range(shared)]
        for _ in range(beams):
            row = common + [ids.pop() for _ in range(mine)]
            for p in row:
                refs[p] += 1
            tables.append(row + [-1] * (width - len(row)))
    return [length for length in lens for _ in range(beams)], tables, refs


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _values(g, shape, dtype):
    """N(0, 1) in `dtype`, made in pieces that need little room beside the result."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for at in range(0, flat.numel(), step):
        n = min(step, flat.numel() - at)
        flat[at:at + n] = torch.randn(n, generator=g, device="cuda").to(dtype)
    return out


def _starts(case):
    """For an append: (first new position, number of new tokens) of each request; prompts' lengths are uneven."""
    n, new = case["requests"], case["new"]
    counts = [new if new == 1 else max(1, new * (2 * i + 1) // (2 * n)) for i in range(n)]
    return [(case["L"] * (i + 1) // n, c) for i, c in enumerate(counts)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    op, dtype, st = case["op"], _TYPES[case["x"]], {"case": case}
    if op == "select":
        rows, V = case["requests"] * case["beams"], case["vocab"]
        # a few likely tokens and a long tail
        logits = torch.randn((rows, V), generator=g, device="cuda") * 2.0 - 4.0
        likely = torch.randint(0, V, (rows, min(V, 40)), generator=g, device="cuda")
        logits.scatter_add_(1, likely, 8.0 * torch.rand(likely.shape, generator=g, device="cuda"))
        st["logits"] = logits.to(dtype)
        st["scores"] = -5.0 - 3.0 * torch.rand((case["requests"], case["beams"]), generator=g, device="cuda")
        st["history"] = torch.randint(0, V, (rows, case["T"]), generator=g, device="cuda", dtype=torch.int32)
        return st
    kv, d, page = case["kv"], case["d"], case["page"]
    if op == "append":
        starts = _starts(case)
        rng.shuffle(starts)
        width = -(-max(a + c for a, c in starts) // page)
        need = [-(-(a + c) // page) for a, c in starts]
        ids = rng.sample(range(sum(need) + 7), sum(need))
        st["tables"] = _ints([[ids.pop() for _ in range(k)] + [-1] * (width - k) for k in need])
        st["seq"] = _ints([i for i, (_, c) in enumerate(starts) for _ in range(c)])
        st["pos"] = _ints([a + t for a, c in starts for t in range(c)])
        st["K_pages"] = _values(g, (sum(need) + 7, kv, page, d), dtype)
        st["V_pages"] = _values(g, (sum(need) + 7, kv, page, d), dtype)
        # the fused projection's rows: queries, keys, values
        st["rows"] = _values(g, (st["seq"].numel(), 3 * kv * d), dtype)
        return st
    if op == "compact":
        lens, tables, refs = _cache(case, rng, 0)
        spare = int(len(refs) * case["holes"] / (1.0 - case["holes"]))
        places = rng.sample(range(len(refs) + spare), len(refs))
        moved = [0] * (len(refs) + spare)
        for p, r in zip(places, refs):
            moved[p] = r
        st["tables"] = _ints([[places[p] if p >= 0 else -1 for p in row] for row in tables])
        st["refs"] = _ints(moved)
        st["pools"] = [_values(g, (len(moved), kv, page, d), dtype) for _ in range(case["pools"])]
        return st
    lens, tables, refs = _cache(case, rng, case.get("spare", 5))
    st["lens"], st["tables"] = _ints(lens), _ints(tables)
    if op == "fork":
        beams = case["beams"]
        parents = []
        for r in range(case["requests"]):    # `alive` of a request's beams go on, the first of them in several
            kept = rng.sample(range(beams), case["alive"])
            parents += sorted(r * beams + kept[k % case["alive"]] for k in range(beams))
        st["refs"], st["parents"] = _ints(refs), _ints(parents)
        st["grow"] = torch.ones(len(parents), dtype=torch.int32, device="cuda")
        st["pools"] = [_values(g, (len(refs), kv, page, d), dtype) for _ in range(case["pools"])]
        return st
    st["K_pages"], st["V_pages"] = (_values(g, (len(refs), kv, page, d), dtype) for _ in range(2))
    # the fused projection's rows, of which the first part are the queries
    st["rows"] = _values(g, (len(lens), (case["heads"] + 2 * kv) * d), dtype)
    st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / case["heads"]) for h in range(case["heads"])],
                                device="cuda") if case["alibi"] else None
    return st


def work(case):
    op, e = case["op"], _BYTES[case["x"]]
    if op == "select":
        n, K, V, k, T = case["requests"], case["beams"], case["vocab"], case["k"], case["T"]
        return {"bytes": n * K * V * e + 4 * n * K + 12 * n * k + 4 * n * k * (2 * T + 1), "flops": 5 * n * K * V}
    kv, d, page = case["kv"], case["d"], case["page"]
    if op == "append":
        s = sum(c for _, c in _starts(case))
        return {"bytes": 4 * s * kv * d * e + 8 * s, "flops": 0}
    parts = [_split({"beams": 1, "own": 0, **case}, length) for length in _lens(case)]
    beams = case.get("beams", 1)
    entries = case["requests"] * beams * -(-(case["L"] + 1) // page)
    pages = sum(s + beams * o for s, o in parts)
    if op == "attend":
        n, heads = case["requests"] * beams, case["heads"]
        tokens = sum(s * page + beams * (length - s * page) for (s, _), length in zip(parts, _lens(case)))
        return {"bytes": 2 * tokens * kv * d * e + 2 * n * heads * d * e + 4 * n * heads + 4 * sum(s + beams * o for s, o in parts),
                "flops": 4 * heads * d * beams * sum(_lens(case))}
    bytes_of_page = case["pools"] * kv * page * d * e
    if op == "fork":
        copies = sum(length % page != 0 for length in _lens(case)) * (beams - case["alive"])
        return {"bytes": 2 * copies * bytes_of_page + 8 * entries + 8 * (pages + case["spare"]), "flops": 0}
    pool = pages + int(pages * case["holes"] / (1.0 - case["holes"]))
    moved = round(pages * (pool - pages) / pool)           # of the pages in use, those in the pool's tail
    return {"bytes": 2 * moved * bytes_of_page + 8 * entries + 12 * pool, "flops": 0}


# ------------------------------------------------------------------ plain forms

def _plain_append(st):
    (P, kv, page, d), rows = st["K_pages"].shape, st["rows"]
    pos = st["pos"].long()
    pages = st["tables"][st["seq"].long(), pos // page].long()
    _, k, v = rows.view(-1, 3, kv, d).unbind(1)
    st["K_pages"][pages, :, pos % page] = k
    st["V_pages"][pages, :, pos % page] = v
    return {"K_pages": st["K_pages"], "V_pages": st["V_pages"]}


def _dense(pages, tables):
    """[n, kv, positions, d] in 32 bits: each sequence's pages in a row."""
    x = pages[tables.long().clamp(min=0)]
    n, M, kv, page, d = x.shape
    return x.transpose(1, 2).float().reshape(n, kv, M * page, d)


def _plain_attend(st):
    case, lens = st["case"], st["lens"]
    n, heads, kv, d = lens.numel(), case["heads"], case["kv"], case["d"]
    q = st["rows"][:, :heads * d].float().reshape(n, kv, heads // kv, d)
    s = (q @ _dense(st["K_pages"], st["tables"]).transpose(2, 3)).reshape(n, heads, -1) / math.sqrt(d)
    at = torch.arange(s.shape[2], device=s.device)
    if st["slopes"] is not None:
        s = s + st["slopes"][None, :, None] * (at - (lens[:, None, None] - 1)).float()
    s = torch.where(at < lens[:, None, None], s, float("-inf"))
    m = s.amax(2, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(2, keepdim=True)
    o = (p / total).reshape(n, kv, heads // kv, -1) @ _dense(st["V_pages"], st["tables"])
    return {"out": o.reshape(n, heads * d).to(st["rows"].dtype), "lse": (m + torch.log(total))[:, :, 0]}


def _plain_fork(st):
    page, tables, lens = st["case"]["page"], st["tables"], st["lens"]
    P, M = st["refs"].numel(), tables.shape[1]
    col = torch.arange(M, device=tables.device)
    used = (lens + page - 1) // page
    kept = torch.zeros_like(lens).index_add_(0, st["parents"].long(), torch.ones_like(st["parents"])) - 1
    held = col < used[:, None]
    refs = st["refs"].clone().index_add_(0, tables[held].long(), kept[:, None].expand(-1, M)[held])
    tables, lens, used = tables[st["parents"].long()], lens[st["parents"].long()], used[st["parents"].long()]
    n = lens.numel()
    j = torch.arange(n, device=lens.device, dtype=torch.int32)
    # a last page that is not full is written next: all that share it but the last one take a copy
    part = (st["grow"] > 0) & (lens % page != 0)
    last = torch.where(part, tables.gather(1, (lens // page).clamp(max=M - 1).long()[:, None])[:, 0], P).long()
    growing = torch.zeros(P + 1, dtype=torch.int32, device=lens.device).index_add_(0, last, torch.ones_like(j))
    keeper = torch.full((P + 1,), -1, dtype=torch.int32, device=lens.device).scatter_reduce_(0, last, j, "amax")
    counted = torch.cat([refs, refs.new_zeros(1)])
    copy = part & ~((keeper[last] == j) & (growing[last] >= counted[last]))
    full = lens + st["grow"]
    want = torch.where(full <= M * page, (full + page - 1) // page - used + copy, 0)
    upto = torch.cumsum(want, 0)
    free = refs <= 0
    n_free = free.sum()
    ok = (full <= M * page) & ((want == 0) | (upto <= n_free))
    copy = copy & ok
    order = torch.argsort((~free).to(torch.int8), stable=True).to(torch.int32)
    base = upto - want
    now = torch.where(ok, full, lens)
    fresh = (base + copy - used)[:, None] + col
    new = torch.where((col >= used[:, None]) & (col < ((now + page - 1) // page)[:, None]),
                      order[fresh.clamp(0, P - 1).long()], torch.where(col < used[:, None], tables, -1))
    at = torch.nonzero(copy)[:, 0]
    source, target = last[at], order[base[at].long()]
    new[at, (lens[at] // page).long()] = target
    taken = torch.where(ok, upto, 0).amax()
    refs = torch.where(torch.zeros_like(refs).scatter_(0, order.long(), torch.arange(P, device=refs.device, dtype=torch.int32)) < taken,
                       torch.ones_like(refs), refs)
    refs.index_add_(0, source, -torch.ones_like(target))
    [p.index_copy_(0, target.long(), p[source]) for p in st["pools"]]
    state = torch.stack([n_free - taken, (upto[-1] - n_free).clamp(min=0), (~ok).sum(), copy.sum()]).to(torch.int32)
    return {"tables": new, "lens": now, "refs": refs, "state": state, "pools": st["pools"]}


def _plain_compact(st):
    refs, tables = st["refs"], st["tables"]
    P = refs.numel()
    at = torch.arange(P, device=refs.device, dtype=torch.int32)
    live = refs > 0
    n = live.sum()
    source = torch.nonzero(live & (at >= n))[:, 0]
    target = torch.nonzero(~live & (at < n))[:, 0]
    moved = torch.where(live, at, -1)
    moved[source] = target.to(torch.int32)
    out = refs.clone()
    out[target] = refs[source]
    out[source] = 0
    new = torch.where(tables >= 0, moved[tables.clamp(min=0).long()], tables)
    [p.index_copy_(0, target, p[source]) for p in st["pools"]]
    return {"tables": new, "refs": out, "moved": moved, "state": torch.stack([n, (live & (at >= n)).sum()]).to(torch.int32),
            "pools": st["pools"]}


def _plain_select(st):
    scores, k = st["scores"], st["case"]["k"]
    n, K = scores.shape
    x = st["logits"].double()
    m = x.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(1, keepdim=True))
    total = (scores.double().reshape(-1, 1) + (x - lse)).reshape(n, -1)
    best, at = torch.sort(total, dim=1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    V = x.shape[1]
    parents = at // V + K * torch.arange(n, device=at.device)[:, None]
    tokens = (at % V).to(torch.int32)
    history = torch.cat([st["history"][parents.reshape(-1)], tokens.reshape(-1, 1)], 1)
    return {"scores": best.float(), "parents": parents.to(torch.int32), "tokens": tokens, "history": history}


def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "fork": _plain_fork, "compact": _plain_compact,
                "select": _plain_select}[op](st)
    import int8_quantized_matmul_amd as i8
    if op == "append":
        w = case["kv"] * case["d"]
        i8.cache_append(st["rows"][:, w:2 * w], st["rows"][:, 2 * w:], st["K_pages"], st["V_pages"], st["tables"], st["pos"],
                        st["seq"])
        return {"K_pages": st["K_pages"], "V_pages": st["V_pages"]}
    if op == "attend":
        out, lse = i8.decode_attention(st["rows"][:, :case["heads"] * case["d"]], st["K_pages"], st["V_pages"], st["tables"],
                                       st["lens"], slopes=st["slopes"], beams=case["beams"])
        return {"out": out, "lse": lse}
    if op == "fork":
        tables, lens, refs, state = i8.cache_fork(st["tables"], st["lens"], st["refs"], case["page"], parents=st["parents"],
                                                  grow=st["grow"], pools=st["pools"])
        return {"tables": tables, "lens": lens, "refs": refs, "state": state, "pools": st["pools"]}
    if op == "compact":
        tables, refs, moved, state = i8.cache_compact(st["tables"], st["refs"], pools=st["pools"])
        return {"tables": tables, "refs": refs, "moved": moved, "state": state, "pools": st["pools"]}
    scores, parents, tokens, history = i8.beam_select(st["logits"], st["scores"], k=case["k"], history=st["history"])
    return {"scores": scores, "parents": parents, "tokens": tokens, "history": history}


# ------------------------------------------------------------------ the definitions

def _exact_attend(st):
    case = st["case"]
    heads, kv, d = case["heads"], case["kv"], case["d"]
    outs, sums = [], []
    for i, (length, row) in enumerate(zip(st["lens"].tolist(), st["tables"])):
        ids = row[:-(-length // case["page"])].long()
        k, v = (p[ids].double().permute(1, 0, 2, 3).reshape(kv, -1, d)[:, :length] for p in (st["K_pages"], st["V_pages"]))
        q = st["rows"][i, :heads * d].double().reshape(kv, -1, d)
        s = torch.bmm(q, k.transpose(1, 2).contiguous()) * d ** -0.5
        if st["slopes"] is not None:
            s += st["slopes"].double().reshape(kv, -1, 1) * torch.arange(1 - length, 1, device=s.device, dtype=torch.float64)
        outs.append(torch.bmm(torch.softmax(s, 2), v).reshape(-1))
        sums.append(torch.logsumexp(s, 2).reshape(-1))
    return {"out": torch.stack(outs), "lse": torch.stack(sums)}


def _exact_fork(st):
    """Sequence after sequence, on lists; the pools' pages are copies of one another."""
    page, lens, tables, refs = st["case"]["page"], st["lens"].tolist(), st["tables"].tolist(), st["refs"].tolist()
    parents, grow, M = st["parents"].tolist(), st["grow"].tolist(), len(tables[0])
    rows = [tables[i][:-(-n // page)] for i, n in enumerate(lens)]
    new = [list(rows[p]) for p in parents]
    size = [lens[p] for p in parents]
    for row in rows:
        for p in row:
            refs[p] -= 1
    for row in new:
        for p in row:
            refs[p] += 1
    after = list(refs)
    free = [p for p, r in enumerate(refs) if r <= 0]
    short = missed = copies = wanted = 0
    writes = [(row[-1] if g > 0 and n % page else None) for row, n, g in zip(new, size, grow)]
    for j, (row, n, g) in enumerate(zip(new, size, grow)):
        p = writes[j]
        later = p is not None and p in writes[j + 1:]
        copy = p is not None and (later or writes.count(p) < refs[p])
        need = -(-(n + g) // page) - len(row) + copy
        if n + g > M * page:
            missed += 1
            continue
        wanted += need
        if need and wanted > len(free):
            missed += 1
            continue
        got = free[wanted - need:wanted]
        for q in got:
            after[q] = 1
        if copy:
            after[p] -= 1
            copies += 1
            row[-1] = got.pop(0)
        row += got
        size[j] = n + g
    short = max(0, wanted - len(free))
    state = [sum(r <= 0 for r in after), short, missed, copies]
    return {"tables": _ints([row + [-1] * (M - len(row)) for row in new]), "lens": _ints(size), "refs": _ints(after),
            "state": _ints(state), "pools": [None] * len(st["pools"])}


def _exact_compact(st):
    refs, tables = st["refs"].tolist(), st["tables"].tolist()
    live = sum(r > 0 for r in refs)
    gaps = [p for p in range(live) if refs[p] <= 0]
    tail = [p for p in range(live, len(refs)) if refs[p] > 0]
    to = {p: p for p in range(live) if refs[p] > 0}
    to.update(zip(tail, gaps))
    out = [0 if p >= live else r for p, r in enumerate(refs)]
    for a, b in zip(tail, gaps):
        out[b] = refs[a]
    return {"tables": _ints([[p if p < 0 else to.get(p, -1) for p in row] for row in tables]), "refs": _ints(out),
            "moved": _ints([to.get(p, -1) for p in range(len(refs))]), "state": _ints([live, len(tail)]),
            "pools": [None] * len(st["pools"])}


def _exact_select(st):
    k, V = st["case"]["k"], st["case"]["vocab"]
    n, K = st["scores"].shape
    best, parents, tokens = [], [], []
    for b in range(n):
        cand = (torch.log_softmax(st["logits"][b * K:(b + 1) * K].double(), 1) + st["scores"][b].double()[:, None]).reshape(-1)
        floor = torch.topk(cand, k).values[-1]
        at = torch.nonzero(cand >= floor)[:, 0]
        ranked = sorted(zip((-cand[at]).tolist(), at.tolist()))[:k]
        best.append([-v for v, _ in ranked])
        parents.append([b * K + i // V for _, i in ranked])
        tokens.append([i % V for _, i in ranked])
    history = [st["history"][p] for row in parents for p in row]
    last = _ints(tokens).reshape(-1, 1)
    return {"scores": torch.tensor(best, dtype=torch.float64, device="cuda"), "parents": _ints(parents), "tokens": _ints(tokens),
            "history": torch.cat([torch.stack(history), last], 1)}


def exact(case, seed):
    if case["op"] == "append":        # copies alone: nothing is computed
        return None
    st = prepare(case, seed)
    return {"attend": _exact_attend, "fork": _exact_fork, "compact": _exact_compact, "select": _exact_select}[case["op"]](st)
