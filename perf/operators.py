"""Cases of the paged key/value cache operators: a step's block tables and slot
maps from request lengths (`fa2_paged_plan`), new key/value rows written to
their slots (`fa2_paged_append`) and attention of each request's new tokens
over its pages (`fa2_paged_fwd`).

`run` computes an operator in its plain form (elementary torch operations,
32-bit) or, with `own` set, through the framework's public calls.  `exact`
computes the same from the definition in 64 bits, token by token.
"""
import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def listed():
    cases = []
    # One short conversation, one new token: what a single user waits for.
    cases.append(_fwd("decode_b1_short", batch=1, hq=32, hkv=8, d=128, dtype="bf16", page=16, new=(1, 1), ctx=(600, 600)))
    # A server's ordinary decoding step: 32 requests of mixed age, one token each, small pages.
    cases.append(_fwd("decode_b32", batch=32, hq=32, hkv=8, d=128, dtype="bf16", page=16, new=(1, 1), ctx=(1, 8192)))
    # A full server on long contexts: the decoding step that reads gigabytes of cache.
    cases.append(_fwd("decode_b64_long", batch=64, hq=32, hkv=8, d=128, dtype="bf16", page=64, new=(1, 1),
                      ctx=(1000, 32000)))
    # Verification of a few drafted tokens per request on a model with one K/V head per query head.
    cases.append(_fwd("verify_d64_fp16", batch=8, hq=16, hkv=16, d=64, dtype="fp16", page=32, new=(5, 5), ctx=(3, 2043)))
    # One step that mixes a chunk of a long prompt with requests that decode.
    cases.append(_fwd("chunk_mixed", batch=17, hq=32, hkv=8, d=128, dtype="bf16", page=16, new=(1, 1), ctx=(1, 4096),
                      chunk=1000, chunk_ctx=5000))
    # The last chunk of a 16384-token prompt: most of the arithmetic of a long prefill.
    cases.append(_fwd("prefill_chunk", batch=1, hq=32, hkv=8, d=128, dtype="bf16", page=64, new=(2048, 2048),
                      ctx=(14336, 14336)))
    # Sliding window with four sink keys at head dim 256, ragged chunks, large pages.
    cases.append(_fwd("window_d256_fp16", batch=4, hq=8, hkv=4, d=256, dtype="fp16", page=128, new=(3, 700),
                      ctx=(1, 3000), window=1023, prefix=4))
    # Tables and slots of a small decoding step.
    cases.append(_plan("plan_b8", batch=8, page=16, new=(1, 1), ctx=(0, 2000)))
    # Tables and slots of a large mixed step: prompts of new requests and decoding ones, padded to a fixed length.
    cases.append(_plan("plan_b2048", batch=2048, page=16, new=(1, 100), ctx=(0, 4000), pad=1000))
    # New rows of a decoding step.
    cases.append(_append("append_b64", tokens=64, pad=0, hkv=8, d=128, dtype="bf16", page=16, pages=512, fused=False))
    # New rows of a prompt chunk, cut from a fused QKV projection, at one K/V head per query head.
    cases.append(_append("append_fused_fp16", tokens=2047, pad=1, hkv=16, d=64, dtype="fp16", page=32, pages=320,
                         fused=True))
    # New rows of whole prompts.
    cases.append(_append("append_prompts", tokens=32768, pad=0, hkv=8, d=128, dtype="bf16", page=64, pages=640,
                         fused=False))
    return cases


def _fwd(name, batch, hq, hkv, d, dtype, page, new, ctx, chunk=0, chunk_ctx=0, window=-1, prefix=0, lens_seed=1):
    return {"name": name, "op": "fwd", "batch": batch, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "page": page,
            "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1], "chunk": chunk,
            "chunk_ctx": chunk_ctx, "window": window, "prefix": prefix, "lens_seed": lens_seed}


def _plan(name, batch, page, new, ctx, pad=0, lens_seed=1):
    return {"name": name, "op": "plan", "batch": batch, "page": page, "new_lo": new[0], "new_hi": new[1],
            "ctx_lo": ctx[0], "ctx_hi": ctx[1], "chunk": 0, "chunk_ctx": 0, "pad": pad, "lens_seed": lens_seed}


def _append(name, tokens, pad, hkv, d, dtype, page, pages, fused):
    return {"name": name, "op": "append", "tokens": tokens, "pad": pad, "hkv": hkv, "d": d, "dtype": dtype,
            "page": page, "pages": pages, "fused": fused}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: attention, planning or appending, sizes spread over their logarithms."""
    kind = rng.choice(["decode", "decode", "few", "chunk", "chunk", "plan", "append"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    if kind == "plan":
        batch = _log(rng, 1, 2048)
        case = _plan("", batch=batch, page=page, new=(rng.choice([0, 1]), _log(rng, 1, 100)),
                     ctx=(0, _log(rng, 1, 4000)), pad=rng.choice([0, 1, 77]), lens_seed=rng.randrange(1 << 30))
    elif kind == "append":
        hkv, d = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128, 256])
        rows = 40960 * 1024 // (hkv * d)
        tokens = _log(rng, 1, min(32768, rows * 4 // 5))
        case = _append("", tokens=tokens, pad=rng.choice([0, 0, 5]), hkv=hkv, d=d,
                       dtype=rng.choice(["fp16", "bf16"]), page=page,
                       pages=(tokens + tokens // 4 + page - 1) // page + 1, fused=rng.random() < 0.5)
    else:
        hkv, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        while hkv * group > 64:
            hkv //= 2
        d = rng.choice([64, 128, 128, 256])
        batch = _log(rng, 1, 64)
        if kind == "decode":
            new = (1, 1)
        elif kind == "few":
            new = (1, rng.randrange(2, 17))
        else:
            new = (1, _log(rng, 17, 2048))
        ctx = (1, _log(rng, 64, 32000))
        window, prefix = -1, 0
        if rng.random() < 0.3:
            window, prefix = _log(rng, 16, 4096), rng.choice([0, 4, 100])
        case = _fwd("", batch=batch, hq=hkv * group, hkv=hkv, d=d, dtype=rng.choice(["fp16", "bf16"]), page=page,
                    new=new, ctx=ctx, window=window, prefix=prefix, lens_seed=rng.randrange(1 << 30))
        # no more reading or arithmetic than the largest listed cases
        while True:
            w = work(case)
            if w["bytes"] <= 4e9 and w["flops"] <= 5e11 and case["batch"] * case["new_hi"] <= 16384:
                break
            case["batch"] = case["batch"] // 2 if case["batch"] > 1 else 1
            case["new_hi"] = max(case["new_lo"], case["new_hi"] * 2 // 3)
            case["ctx_hi"] = max(case["ctx_lo"], case["ctx_hi"] * 2 // 3)
    del case["name"]
    return case


# ---------------------------------------------------------------- lengths and sizes

def _lengths(case):
    """(context lengths, new tokens) of every request; they belong to the case, not to the seed."""
    r = random.Random(case["lens_seed"])
    n = case["batch"]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
    if case["chunk"]:
        at = n // 2
        ctx[at], new[at] = case["chunk_ctx"], case["chunk"]
    return ctx, new


def _visible(n_q, n_k, window, prefix):
    """(visible pairs, keys some query sees) of one request under a causal band with a prefix."""
    i = np.arange(n_q, dtype=np.int64) + (n_k - n_q)
    lo = np.maximum(i - window, 0) if window >= 0 else np.zeros_like(i)
    pre = min(prefix, n_k)
    pairs = np.maximum(i + 1 - np.maximum(lo, pre), 0).sum() + pre * n_q
    union = max(0, n_k - max(int(lo[0]) if n_q else n_k, pre)) + pre if n_q else 0
    return int(pairs), int(union)


def work(case):
    if case["op"] == "fwd":
        ctx, new = _lengths(case)
        pairs = keys = pages = 0
        for c, n in zip(ctx, new):
            p, u = _visible(n, c + n, case["window"], case["prefix"])
            pairs += p
            keys += u
            pages += -(-u // case["page"])
        rows = sum(new) * case["hq"]
        d = case["d"]
        return {"bytes": keys * case["hkv"] * d * 4 + rows * (d * 4 + 4) + pages * 4 + case["batch"] * 8,
                "flops": 4 * d * pairs * case["hq"]}
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        page = case["page"]
        taken = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))
        partial = sum(1 for c, n in zip(ctx, new) if n and c % page)
        return {"bytes": case["batch"] * 16 + taken * 8 + partial * 4 + (sum(new) + case["pad"]) * 4 + 12,
                "flops": 0}
    rows = case["tokens"] * case["hkv"] * case["d"]
    return {"bytes": 2 * rows * 4 + (case["tokens"] + case["pad"]) * 4, "flops": 0}


# ---------------------------------------------------------------- what a program has in hand

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "fwd":
        return _prepare_fwd(case, g)
    if case["op"] == "plan":
        return _prepare_plan(case, g)
    return _prepare_append(case, g)


def _tables(case, g, lens, pages):
    """Block table [batch, widest] with the given lengths' pages drawn from `pages` in random order, -1 beyond them."""
    page = case["page"]
    need = [-(-n // page) for n in lens]
    widest = max(1, max(need))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    cell = torch.arange(widest, device="cuda")[None, :]
    needs = torch.tensor(need, device="cuda")[:, None]
    first = torch.cumsum(needs, 0) - needs
    table = torch.where(cell < needs, order[(first + cell).clamp_(max=pages - 1)], torch.full_like(order[:1], -1))
    return table.contiguous(), order, sum(need)


def _prepare_fwd(case, g):
    dtype, d, page = _DTYPES[case["dtype"]], case["d"], case["page"]
    ctx, new = _lengths(case)
    lens = [c + n for c, n in zip(ctx, new)]
    pages = sum(-(-n // page) for n in lens) + 3
    table, _, _ = _tables(case, g, lens, pages)
    total = max(1, sum(new))
    return {"case": case, "new": new, "lens": lens, "table": table,
            "cu": torch.tensor(np.concatenate([[0], np.cumsum(new)]), device="cuda", dtype=torch.int32),
            "lens_k": torch.tensor(lens, device="cuda", dtype=torch.int32),
            "q": _normal(g, (total, case["hq"], d), dtype),
            "k": _normal(g, (pages, case["hkv"], page, d), dtype),
            "v": _normal(g, (pages, case["hkv"], page, d), dtype),
            "scale": 1.0 / math.sqrt(d)}


def _prepare_plan(case, g):
    page = case["page"]
    ctx, new = _lengths(case)
    lens = [c + n for c, n in zip(ctx, new)]
    held = [-(-c // page) for c in ctx]
    taken = sum(-(-n // page) for n in lens) - sum(held)
    pages = sum(held) + taken + 17
    table, order, used = _tables(case, g, ctx, pages)
    widest = max(-(-n // page) for n in lens) + 2
    wide = torch.full((case["batch"], widest), -1, device="cuda", dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    free = order[used:].contiguous()   # a stack: its last free_count entries' top is taken first
    return {"case": case, "table": wide, "free": free, "pages": pages, "total": max(1, sum(new) + case["pad"]),
            "tokens": sum(new), "taken": taken,
            "ctx": torch.tensor(ctx, device="cuda", dtype=torch.int32),
            "new": torch.tensor(new, device="cuda", dtype=torch.int32),
            "count": torch.tensor([free.numel()], device="cuda", dtype=torch.int32)}


def _prepare_append(case, g):
    dtype, d, hkv, page = _DTYPES[case["dtype"]], case["d"], case["hkv"], case["page"]
    total = case["tokens"] + case["pad"]
    if case["fused"]:   # [q heads | k heads | v heads] of one projection: strided views
        rows = _normal(g, (total, 3 * hkv, d), dtype)
        k, v = rows[:, hkv:2 * hkv], rows[:, 2 * hkv:]
    else:
        k, v = _normal(g, (total, hkv, d), dtype), _normal(g, (total, hkv, d), dtype)
    slots = torch.full((total,), -1, device="cuda", dtype=torch.int32)
    # runs of one page each, pages in random order, as a table of requests gives them
    order = torch.randperm(case["pages"], generator=g, device="cuda")
    at = torch.arange(case["tokens"], device="cuda")
    slots[:case["tokens"]] = (order[at // page] * page + at % page).to(torch.int32)
    return {"case": case, "k": k, "v": v, "slots": slots, "tokens": case["tokens"],
            "k_cache": _normal(g, (case["pages"], hkv, page, d), dtype),
            "v_cache": _normal(g, (case["pages"], hkv, page, d), dtype)}


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "fwd":
        return _plain_fwd(state)
    if op == "plan":
        return _plain_plan(state)
    return _plain_append(state)


def _own(state, op):
    import exact_tiled_attention_fa2_gb300 as fa2
    case = state["case"]
    if op == "fwd":
        return fa2.fa2_paged_fwd(state["q"], state["k"], state["v"], state["table"], state["cu"], state["lens_k"],
                                 scale=state["scale"], window_left=case["window"], window_right=0,
                                 prefix_len=case["prefix"], max_seqlen_q=max(1, max(state["new"])))
    if op == "plan":
        cu, lens, slots, left = fa2.fa2_paged_plan(state["ctx"], state["new"], state["table"], state["free"],
                                                   state["count"], state["pages"], case["page"], state["total"])
        return cu, lens, slots, left, state["table"]
    fa2.fa2_paged_append(state["k"], state["v"], state["slots"], state["k_cache"], state["v_cache"])
    return state["k_cache"], state["v_cache"]


def _plain_fwd(state):
    case, q = state["case"], state["q"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    group = hq // hkv
    o = torch.empty_like(q)
    lse = torch.empty((hq, q.shape[0]), device=q.device, dtype=torch.float32)
    row = 0
    for b, (n, n_k) in enumerate(zip(state["new"], state["lens"])):
        if n == 0:
            continue
        own_pages = state["table"][b, :-(-n_k // page)].long()
        k = state["k"][own_pages].transpose(0, 1).reshape(hkv, -1, d)[:, :n_k].float()
        v = state["v"][own_pages].transpose(0, 1).reshape(hkv, -1, d)[:, :n_k].float()
        x = q[row:row + n].float().reshape(n, hkv, group, d).permute(1, 2, 0, 3).reshape(hkv, group * n, d)
        s = torch.matmul(x, k.transpose(1, 2)).mul_(state["scale"]).reshape(hkv, group, n, n_k)
        if n > 1 or case["window"] >= 0:
            i = torch.arange(n_k - n, n_k, device=q.device)[:, None]
            j = torch.arange(n_k, device=q.device)[None, :]
            seen = j <= i
            if case["window"] >= 0:
                seen = seen & (j >= i - case["window"])
            if case["prefix"]:
                seen = seen | (j < case["prefix"])
            s.masked_fill_(~seen, float("-inf"))
        m = s.amax(dim=-1, keepdim=True)
        p = s.sub_(m).exp_()
        total = p.sum(dim=-1, keepdim=True)
        y = torch.matmul(p.reshape(hkv, group * n, n_k), v).reshape(hkv, group, n, d) / total
        o[row:row + n] = y.permute(2, 0, 1, 3).reshape(n, hq, d).to(q.dtype)
        lse[:, row:row + n] = (m + total.log()).reshape(hq, n)
        row += n
    return o, lse


def _plain_plan(state):
    page, ctx, new, table = state["case"]["page"], state["ctx"], state["new"], state["table"]
    batch = ctx.numel()
    zero = torch.zeros(1, device=ctx.device, dtype=torch.int32)
    lens = ctx + new
    cu = torch.cat([zero, torch.cumsum(new, 0).to(torch.int32)])
    held = (ctx + page - 1) // page
    fresh = (lens + page - 1) // page - held
    before = torch.cumsum(fresh, 0) - fresh
    request = torch.arange(batch, device=ctx.device)
    # pages taken from the top of the stack, in order of the requests and of each request's pages
    taken = torch.arange(state["taken"], device=ctx.device)
    owner = torch.repeat_interleave(request, fresh, output_size=state["taken"])
    table[owner, held[owner] + taken - before[owner]] = state["free"][state["count"].long() - 1 - taken]
    token = torch.arange(state["tokens"], device=ctx.device)
    owner = torch.repeat_interleave(request, new, output_size=state["tokens"])
    at = ctx[owner] + token - cu[owner]
    slots = torch.full((state["total"],), -1, device=ctx.device, dtype=torch.int32)
    slots[:state["tokens"]] = (table[owner, at // page] * page + at % page).to(torch.int32)
    left = (state["count"] - fresh.sum()).to(torch.int32)
    return cu, lens, slots, left, table


def _plain_append(state):
    page = state["case"]["page"]
    slots = state["slots"][:state["tokens"]].long()
    where, at = slots // page, slots % page
    state["k_cache"][where, :, at] = state["k"][:state["tokens"]]
    state["v_cache"][where, :, at] = state["v"][:state["tokens"]]
    return state["k_cache"], state["v_cache"]


# ---------------------------------------------------------------- from the definition, in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "fwd":
        return _exact_fwd(state)
    if case["op"] == "plan":
        return _exact_plan(state)
    return _exact_append(state)


def _exact_fwd(state):
    case = state["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    group = hq // hkv
    table = state["table"].cpu().numpy()
    total = state["q"].shape[0]
    o = torch.empty((total, hq, d), device="cuda", dtype=torch.float64)
    lse = torch.empty((hq, total), device="cuda", dtype=torch.float64)
    start = 0
    for b, (n, n_k) in enumerate(zip(state["new"], state["lens"])):
        j = np.arange(n_k)
        page_of = torch.from_numpy(table[b, j // page].astype(np.int64)).cuda()
        at = torch.from_numpy(j % page).cuda()
        key = torch.from_numpy(j).cuda()
        for h in range(hkv):
            keys, values = state["k"][page_of, h, at].double(), state["v"][page_of, h, at].double()
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                place = torch.arange(i0, i1, device="cuda") + (n_k - n)
                hidden = key[None, :] > place[:, None]
                if case["window"] >= 0:
                    hidden |= key[None, :] + case["window"] < place[:, None]
                hidden &= key[None, :] >= case["prefix"]
                for m in range(h * group, (h + 1) * group):
                    x = state["q"][start + i0:start + i1, m].double() @ keys.T
                    x = x * state["scale"] + torch.zeros_like(x).masked_fill_(hidden, -math.inf)
                    norm = torch.logsumexp(x, dim=1)
                    o[start + i0:start + i1, m] = torch.exp(x - norm[:, None]) @ values
                    lse[m, start + i0:start + i1] = norm
        start += n
    return o, lse


def _exact_plan(state):
    page = state["case"]["page"]
    ctx, new = state["ctx"].tolist(), state["new"].tolist()
    table, free = state["table"].cpu().numpy().copy(), state["free"].tolist()
    cu, lens, slots = [0], [], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        for pos in range(c, c + n):
            if pos % page == 0:
                table[b, pos // page] = free.pop()
            slots.append(int(table[b, pos // page]) * page + pos % page)
        cu.append(cu[-1] + n)
        lens.append(c + n)
    slots += [-1] * (state["total"] - len(slots))
    whole = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    return whole(cu), whole(lens), whole(slots), whole([len(free)]), torch.from_numpy(table).cuda()


def _exact_append(state):
    page = state["case"]["page"]
    k_cache, v_cache = state["k_cache"].double(), state["v_cache"].double()
    for cache, rows in ((k_cache, state["k"]), (v_cache, state["v"])):
        flat = cache.transpose(1, 2).reshape(-1, cache.shape[1], cache.shape[3])
        keep = state["slots"] >= 0
        flat[state["slots"][keep].long()] = rows[keep].double()
        cache.copy_(flat.reshape(cache.shape[0], page, cache.shape[1], cache.shape[3]).transpose(1, 2))
    return k_cache, v_cache
