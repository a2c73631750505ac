"""The paged-cache operators as measured: plain torch forms, the framework's calls, and their 64-bit values.

A case's "op" is append, attend or evict.  The lengths of a case's sequences follow from the case alone (so that
`work` knows them); keys, values, queries, scores and the order of the pages come from the seed.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one chat turn just begun: a single sequence of a few hundred tokens; latency counts
        dict(name="attend_one_short", op="attend", dtype="bf16", batch=1, hq=32, hkv=8, d=128, dv=128, page=16,
             longest=300, ragged=False, tokens_first=False, coreset=0, accumulate=False),
        # the KV-cache workload's shape: one long context, 32 query heads over 8 kv heads
        dict(name="attend_kv", op="attend", dtype="bf16", batch=1, hq=32, hkv=8, d=128, dv=128, page=64,
             longest=32768, ragged=False, tokens_first=False, coreset=0, accumulate=False),
        # a serving batch in mid-flight: lengths of 0 to 8191, pages of 16 in token-major order, weights accumulated
        # for the eviction that follows
        dict(name="attend_batch_scored", op="attend", dtype="bf16", batch=32, hq=32, hkv=8, d=128, dv=128, page=16,
             longest=8191, ragged=True, tokens_first=True, coreset=0, accumulate=True),
        # the long workload's heads (no grouping), four sequences; the largest pass
        dict(name="attend_long", op="attend", dtype="bf16", batch=4, hq=8, hkv=8, d=128, dv=128, page=128,
             longest=131072, ragged=False, tokens_first=False, coreset=0, accumulate=False),
        # fp32 inputs, narrow heads, an odd page size
        dict(name="attend_fp32", op="attend", dtype="fp32", batch=8, hq=8, hkv=4, d=64, dv=64, page=24,
             longest=5000, ragged=True, tokens_first=False, coreset=0, accumulate=True),
        # the compressed prompt (r = 1024 of the KV-cache workload) with the exact tail generated since
        dict(name="attend_coreset_tail", op="attend", dtype="bf16", batch=8, hq=32, hkv=8, d=128, dv=128, page=16,
             longest=1500, ragged=True, tokens_first=False, coreset=1024, accumulate=False),
        # one decode step's new rows of a batch
        dict(name="append_step", op="append", dtype="bf16", batch=32, hkv=8, d=128, dv=128, page=16, rows=1,
             longest=4096, ragged=False, tokens_first=False),
        # two prompts written into the cache
        dict(name="append_prompt", op="append", dtype="bf16", batch=2, hkv=8, d=128, dv=128, page=64, rows=32768,
             longest=32768, ragged=True, tokens_first=True),
        # the KV-cache workload's cache cut to its coreset's size
        dict(name="evict_kv", op="evict", dtype="bf16", batch=1, hkv=8, d=128, dv=128, page=64, longest=32768,
             ragged=False, tokens_first=False, keep=1024, sink=4, recent=128),
        # a batch over its budget: ragged lengths, some of them short of it
        dict(name="evict_batch", op="evict", dtype="bf16", batch=32, hkv=8, d=128, dv=128, page=16, longest=8191,
             ragged=True, tokens_first=False, keep=2048, sink=4, recent=64),
        # fp32 heads of the 512-key size
        dict(name="evict_small_fp32", op="evict", dtype="fp32", batch=1, hkv=1, d=64, dv=64, page=16, longest=512,
             ragged=False, tokens_first=True, keep=32, sink=0, recent=8),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    d = rng.choice([64, 64, 128, 128, 128, 72, 96, 256, 16])
    dv = d if rng.random() < 0.8 else rng.choice([64, 128, 40])
    page = rng.choice([16, 16, 32, 64, 128, 1, 7, 24])
    batch = _log_int(rng, 1, 64)
    # bytes of all keys and values of the case: at most 2^30, half of the largest listed pass
    row = hkv * (d + dv) * (4 if dtype == "fp32" else 2)
    longest = _log_int(rng, 1, max(1, min(131072, (1 << 30) // (row * batch))))
    case = dict(op=op, dtype=dtype, batch=batch, hkv=hkv, d=d, dv=dv, page=page, longest=longest,
                ragged=rng.random() < 0.7, tokens_first=rng.random() < 0.5)
    if op == "attend":
        coreset = _log_int(rng, 1, 2048) if rng.random() < 0.3 else 0
        case.update(hq=hkv * group, coreset=coreset, accumulate=rng.random() < 0.5)
    elif op == "append":
        case.update(rows=1 if rng.random() < 0.4 else _log_int(rng, 1, longest))
    else:
        keep = _log_int(rng, 1, longest)
        sink = min(keep, rng.choice([0, 1, 4, 16]))
        case.update(keep=keep, sink=sink, recent=min(keep - sink, rng.choice([0, 8, 33, 128])))
    return case


def _lengths(case):
    """Tokens of each sequence (append: new rows of each sequence): the case's own, the same for every seed."""
    most = case["rows"] if case["op"] == "append" else case["longest"]
    if not case["ragged"]:
        return [most] * case["batch"]
    r = random.Random("%d %d %d" % (case["batch"], most, case["page"]))
    lens = [r.randint(0, most) for _ in range(case["batch"])]
    lens[-1] = most
    return lens


def _group(case):
    return case["hq"] // case["hkv"]


def work(case):
    lens = _lengths(case)
    tokens, B, hkv = sum(lens), case["batch"], case["hkv"]
    size = 4 if case["dtype"] == "fp32" else 2
    row = (case["d"] + case["dv"]) * size
    if case["op"] == "append":
        return {"bytes": tokens * hkv * (2 * row + 4), "flops": 0}
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        scanned = sum(n for n in lens if n > case["keep"])
        return {"bytes": hkv * (4 * scanned + kept * (2 * row + 12)), "flops": 0}
    r = case["coreset"]
    moved = tokens * hkv * (row + (8 if case["accumulate"] else 0))
    moved += B * hkv * r * (case["d"] * size + 4 * (case["dv"] + 1))
    moved += B * case["hq"] * (case["d"] * size + 4 * case["dv"])
    return {"bytes": moved, "flops": 2 * (tokens + B * r) * case["hq"] * (case["d"] + case["dv"])}


def _pages(case, g, n_pages, width):
    """A pool of pages [n_pages, hkv, page, width]; a token-major one as the transposed view of its memory."""
    if case["tokens_first"]:
        shape = (n_pages, case["page"], case["hkv"], width)
        return torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[case["dtype"]]).transpose(1, 2)
    shape = (n_pages, case["hkv"], case["page"], width)
    return torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, hkv, page, dt = case["batch"], case["hkv"], case["page"], DTYPES[case["dtype"]]
    lens = _lengths(case)
    longest = case["longest"] if case["op"] != "append" else case["longest"] + case["rows"]
    max_pages = (longest + page - 1) // page
    n_tables = 2 if case["op"] == "evict" else 1     # an eviction writes into pages of its own
    n_pages = n_tables * B * max_pages + 3
    order = torch.randperm(n_pages, generator=g, device="cuda")[: n_tables * B * max_pages]
    tables = order.to(torch.int32).reshape(n_tables, B, max_pages).contiguous()
    k_pages, v_pages = _pages(case, g, n_pages, case["d"]), _pages(case, g, n_pages, case["dv"])
    s = dict(case=case, k_pages=k_pages, v_pages=v_pages, table=tables[0],
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), scores=None)
    cap = max_pages * page
    if case["op"] == "append":
        s["K"] = torch.randn(B, hkv, case["rows"], case["d"], generator=g, device="cuda", dtype=dt)
        s["V"] = torch.randn(B, hkv, case["rows"], case["dv"], generator=g, device="cuda", dtype=dt)
        s["pos"] = torch.randint(0, case["longest"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["scores"] = torch.rand(B, hkv, cap, generator=g, device="cuda")
    elif case["op"] == "attend":
        # queries wider than the keys: the attention of a trained head is far from uniform
        q = 2.0 * torch.randn(B, case["hq"], case["d"], generator=g, device="cuda")
        s["Q"] = q.to(dt)
        if case["accumulate"]:
            s["scores"] = torch.rand(B, hkv, cap, generator=g, device="cuda")
        if case["coreset"]:
            r = case["coreset"]
            Ks = torch.randn(B, hkv, r, case["d"], generator=g, device="cuda").to(dt)
            w = torch.exp(torch.randn(B, hkv, r, 1, generator=g, device="cuda")) * 16.0
            v = torch.randn(B, hkv, r, case["dv"], generator=g, device="cuda")
            rank = torch.full((B, hkv), r, dtype=torch.int32, device="cuda")
            rank[0, 0] = (r + 1) // 2       # a selection that stopped early
            s["coreset"] = (Ks, torch.cat([w * v, w], dim=-1).contiguous(), rank)
    else:
        # accumulated weights: a few heavy positions, many light ones, equal ones where nothing was accumulated yet
        x = torch.exp(2.0 * torch.randn(B, hkv, cap, generator=g, device="cuda") - 6.0)
        x[..., cap - cap // 8:] = 0.0
        s["scores"] = x
        s["into"] = tables[1]
        s["scores_into"] = torch.zeros_like(x)
    if own:
        from coreset_attention_approximation_b200 import wildcat

        s["cache"] = wildcat.PagedCache(k_pages, v_pages, s["table"], hq=case.get("hq", hkv), scores=s["scores"])
    return s


def _gathered(pages, table):
    """Every sequence's rows in order of position: [B, hkv, max_pages * page, width]."""
    x = pages[table.long()]
    B, m, h, p, w = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, h, m * p, w)


def _attend(s):
    case, lens = s["case"], s["lens"]
    B, hkv, G = case["batch"], case["hkv"], _group(case)
    k = _gathered(s["k_pages"], s["table"]).float()
    v = _gathered(s["v_pages"], s["table"]).float()
    q = s["Q"].float().reshape(B, hkv, G, case["d"])
    valid = torch.arange(k.shape[2], device="cuda")[None, :] < lens[:, None]
    logits = (q @ k.transpose(-1, -2)) / math.sqrt(case["d"])
    logits = logits.masked_fill(~valid[:, None, None, :], float("-inf"))
    v = v.masked_fill(~valid[:, None, :, None], 0.0)
    top = logits.amax(dim=-1, keepdim=True)
    if case["coreset"]:
        Ks, W, rank = s["coreset"]
        extra = (q @ Ks.float().transpose(-1, -2)) / math.sqrt(case["d"])
        used = torch.arange(Ks.shape[2], device="cuda")[None, None, :] < rank[:, :, None]
        extra = extra.masked_fill(~used[:, :, None, :], float("-inf"))
        top = torch.maximum(top, extra.amax(dim=-1, keepdim=True))
    m = top.masked_fill(top == float("-inf"), 0.0)
    p = torch.exp(logits - m)
    num, den = p @ v, p.sum(dim=-1, keepdim=True)
    if case["coreset"]:
        a = torch.exp(extra - m) @ W
        num, den = num + a[..., :-1], den + a[..., -1:]
    empty = top == float("-inf")
    safe = den.masked_fill(empty, 1.0)
    out = (num / safe).reshape(B, hkv * G, case["dv"])
    lse = (m + torch.log(safe)).masked_fill(empty, float("-inf")).reshape(B, hkv * G)
    if case["accumulate"]:
        s["scores"] += (p / safe).sum(dim=2)
    return [out, lse] + ([s["scores"]] if case["accumulate"] else [])


def _append(s):
    case = s["case"]
    j = torch.arange(case["rows"], device="cuda")[None, :]
    b, j = torch.nonzero(j < s["lens"][:, None], as_tuple=True)
    at = s["pos"].long()[b] + j
    page = s["table"].long()[b, at // case["page"]]
    s["k_pages"][page, :, at % case["page"]] = s["K"][b, :, j]
    s["v_pages"][page, :, at % case["page"]] = s["V"][b, :, j]
    s["scores"][b, :, at] = 0.0
    return [s["k_pages"], s["v_pages"], s["scores"]]


def _evict(s):
    case, lens, scores = s["case"], s["lens"].long(), s["scores"]
    keep, page = case["keep"], case["page"]
    B, hkv, cap = scores.shape
    at = torch.arange(cap, device="cuda")[None, :]
    always = (at < case["sink"]) | (at >= lens[:, None] - case["recent"]) | (lens[:, None] <= keep)
    key = scores.masked_fill(torch.isnan(scores), float("-inf"))
    key = key.masked_fill(always[:, None, :], float("inf")).double()
    # a class above the score: 2 always kept, 1 by its score, 0 behind the end
    kind = torch.where(at >= lens[:, None], 0, torch.where(always, 2, 1))[:, None, :].expand(B, hkv, cap)
    first = torch.sort(key, dim=-1, descending=True, stable=True).indices
    second = torch.sort(kind.gather(-1, first), dim=-1, descending=True, stable=True).indices
    best = first.gather(-1, second)[..., : min(keep, cap)]
    new = torch.minimum(lens, torch.full_like(lens, keep))
    slot = torch.arange(best.shape[-1], device="cuda")
    held = (slot[None, :] < new[:, None])[:, None, :].expand(B, hkv, -1)
    order = torch.sort(best.masked_fill(~held, cap), dim=-1).values
    b, h, j = torch.nonzero(held, as_tuple=True)
    src = order[b, h, j]
    table, into = s["table"].long(), s["into"].long()
    was, now = table[b, src // page], into[b, j // page]
    s["k_pages"][now, h, j % page] = s["k_pages"][was, h, src % page]
    s["v_pages"][now, h, j % page] = s["v_pages"][was, h, src % page]
    s["scores_into"][b, h, j] = scores[b, h, src]
    idx = torch.full((B, hkv, keep), -1, dtype=torch.int32, device="cuda")
    idx[..., : order.shape[-1]] = order.masked_fill(~held, -1).to(torch.int32)
    return [idx, new.to(torch.int32), s["k_pages"], s["v_pages"], s["scores_into"]]


def run(s):
    case = s["case"]
    if not own:
        return {"append": _append, "attend": _attend, "evict": _evict}[case["op"]](s)
    cache = s["cache"]
    if case["op"] == "append":
        cache.append(s["K"], s["V"], s["pos"], count=s["lens"])
        return [s["k_pages"], s["v_pages"], s["scores"]]
    if case["op"] == "attend":
        out, lse = cache.attend(s["Q"], s["lens"], coreset=s.get("coreset"), accumulate=case["accumulate"],
                                return_lse=True)
        return [out, lse] + ([s["scores"]] if case["accumulate"] else [])
    res = cache.evict(s["lens"], case["keep"], sink=case["sink"], recent=case["recent"], into=s["into"],
                      scores_into=s["scores_into"])
    return [res["idx"], res["lens"], s["k_pages"], s["v_pages"], s["scores_into"]]


def exact(case, seed):
    """attend in 64 bits, one sequence and kv head at a time; append and evict only move values."""
    if case["op"] != "attend":
        return None
    s = prepare(case, seed)
    B, hkv, G, page = case["batch"], case["hkv"], _group(case), case["page"]
    out = torch.zeros(B, hkv * G, case["dv"], dtype=torch.float64, device="cuda")
    lse = torch.full((B, hkv * G), float("-inf"), dtype=torch.float64, device="cuda")
    scores = s["scores"].double() if case["accumulate"] else None
    beta = 1.0 / math.sqrt(case["d"])
    for b, n in enumerate(_lengths(case)):
        used = s["table"][b, : (n + page - 1) // page].long()
        for h in range(hkv):
            k = s["k_pages"][used, h].reshape(-1, case["d"])[:n].double()
            v = s["v_pages"][used, h].reshape(-1, case["dv"])[:n].double()
            q = s["Q"][b, h * G:(h + 1) * G].double()
            a, c = torch.einsum("gd,nd->gn", q, k) * beta, torch.ones(n, 1, dtype=torch.float64, device="cuda")
            vc = torch.cat([v, c], dim=1)
            if case["coreset"]:
                Ks, W, rank = s["coreset"]
                r = int(rank[b, h])
                a = torch.cat([a, torch.einsum("gd,nd->gn", q, Ks[b, h, :r].double()) * beta], dim=1)
                vc = torch.cat([vc, W[b, h, :r].double()], dim=0)
            if not a.shape[1]:
                continue
            top = a.max(dim=1, keepdim=True).values
            e = torch.exp(a - top)
            o = torch.einsum("gn,nc->gc", e, vc)
            rows = slice(h * G, (h + 1) * G)
            out[b, rows] = o[:, :-1] / o[:, -1:]
            lse[b, rows] = top[:, 0] + torch.log(o[:, -1])
            if scores is not None:
                scores[b, h, :n] += (e[:, :n] / o[:, -1:]).sum(dim=0)
    return [out, lse] + ([scores] if scores is not None else [])
