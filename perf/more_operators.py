"""Cases of the paged cache in 8 bits and of shared prefixes: key/value rows
quantised as they are written and read back (`fa2_paged_append_fp8`,
`fa2_paged_read_fp8`), attention that reads the 8-bit pages
(`fa2_paged_fwd_fp8`), and attention of requests that share the first pages of
their prompts, which are attended once for all (`fa2_paged_fwd_shared`).

A row of the 8-bit cache (one token of one K/V head) is d e4m3 codes and one
exponent byte u: it stands for code * 2^(u - 127), with the smallest power of
two that brings the row's largest value to 448 or below.

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
# a row's exponents, by the type that it is written from
_EXPONENTS = {torch.float16: (-15, 8), torch.bfloat16: (-60, 60)}


# ---------------------------------------------------------------- cases

def listed():
    cases = []
    # One short conversation on an 8-bit cache, one new token: what a single user waits for.
    cases.append(_fwd("fp8_decode_b1", batch=1, hq=32, hkv=8, d=128, dtype="bf16", page=16, new=(1, 1), ctx=(600, 600)))
    # A server's ordinary decoding step on an 8-bit cache: 32 requests of mixed age, small pages.
    cases.append(_fwd("fp8_decode_b32", batch=32, hq=32, hkv=8, d=128, dtype="bf16", page=16, new=(1, 1), ctx=(1, 8192)))
    # A full server on long contexts, which the halved cache makes room for.
    cases.append(_fwd("fp8_decode_b64_long", batch=64, hq=32, hkv=8, d=128, dtype="bf16", page=64, new=(1, 1),
                      ctx=(1000, 32000)))
    # Verification of a few drafted tokens per request on a model with one K/V head per query head.
    cases.append(_fwd("fp8_verify_d64_fp16", batch=8, hq=16, hkv=16, d=64, dtype="fp16", page=32, new=(5, 5),
                      ctx=(3, 2043)))
    # Ragged short chunks under a sliding window with sink keys at head dim 256, large pages.
    cases.append(_fwd("fp8_window_d256_fp16", batch=4, hq=8, hkv=4, d=256, dtype="fp16", page=128, new=(3, 200),
                      ctx=(1, 3000), window=1023, sinks=4))
    # New rows of a decoding step, quantised as they are written, and read back.
    cases.append(_write("fp8_write_b64", tokens=64, pad=0, hkv=8, d=128, dtype="bf16", page=16, pages=512, fused=False))
    # Rows of a prompt chunk cut from a fused QKV projection, with padding, and read back.
    cases.append(_write("fp8_write_fused_fp16", tokens=2047, pad=1, hkv=16, d=64, dtype="fp16", page=32, pages=320,
                        fused=True))
    # Rows of whole prompts, and read back as the 16-bit rows that a chunk's attention takes.
    cases.append(_write("fp8_write_prompts", tokens=32768, pad=0, hkv=8, d=128, dtype="bf16", page=64, pages=640,
                        fused=False))
    # A decoding step of 64 requests behind one long system prompt.
    cases.append(_shared("shared_decode_b64", batch=64, groups=1, hq=32, hkv=8, d=128, dtype="bf16", page=16,
                         new=(1, 1), shared=(8200, 8200), ctx=(1, 1000)))
    # Two prompts of different lengths, drafted tokens, one K/V head per query head.
    cases.append(_shared("shared_two_d64_fp16", batch=24, groups=2, hq=16, hkv=16, d=64, dtype="fp16", page=32,
                         new=(1, 4), shared=(500, 2500), ctx=(1, 300)))
    # Many samples of one long document: the prefix is nearly all there is.
    cases.append(_shared("shared_samples_b128", batch=128, groups=1, hq=32, hkv=8, d=128, dtype="bf16", page=64,
                         new=(1, 1), shared=(32000, 32000), ctx=(1, 500)))
    # Ragged chunks of user prompts behind one system prompt at head dim 256.
    cases.append(_shared("shared_chunks_d256", batch=6, groups=1, hq=8, hkv=4, d=256, dtype="bf16", page=128,
                         new=(1, 300), shared=(6000, 6000), ctx=(0, 200)))
    return cases


def _fwd(name, batch, hq, hkv, d, dtype, page, new, ctx, window=-1, sinks=0, lens_seed=1):
    return {"name": name, "op": "fwd", "batch": batch, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "page": page,
            "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1], "window": window, "sinks": sinks,
            "lens_seed": lens_seed}


def _write(name, tokens, pad, hkv, d, dtype, page, pages, fused):
    return {"name": name, "op": "write", "tokens": tokens, "pad": pad, "hkv": hkv, "d": d, "dtype": dtype,
            "page": page, "pages": pages, "fused": fused}


def _shared(name, batch, groups, hq, hkv, d, dtype, page, new, shared, ctx, lens_seed=1):
    return {"name": name, "op": "shared", "batch": batch, "groups": groups, "hq": hq, "hkv": hkv, "d": d,
            "dtype": dtype, "page": page, "new_lo": new[0], "new_hi": new[1], "shared_lo": shared[0],
            "shared_hi": shared[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1], "lens_seed": lens_seed}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: attention on 8 bits, writing and reading, shared prefixes; sizes spread over their logarithms."""
    kind = rng.choice(["fwd", "fwd", "fwd", "write", "shared", "shared", "shared"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    d = rng.choice([64, 128, 128, 256])
    dtype = rng.choice(["fp16", "bf16"])
    lens_seed = rng.randrange(1 << 30)
    if kind == "write":
        hkv = rng.choice([1, 2, 3, 4, 8, 16])
        tokens = _log(rng, 1, min(32768, 32768 * 1024 // (hkv * d)))
        case = _write("", tokens=tokens, pad=rng.choice([0, 0, 5]), hkv=hkv, d=d, dtype=dtype, page=page,
                      pages=(tokens + tokens // 4 + page - 1) // page + 1, fused=rng.random() < 0.5)
        del case["name"]
        return case
    hkv, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    while hkv * group > 64:
        hkv //= 2
    new = rng.choice([(1, 1), (1, 1), (1, rng.randrange(2, 17)), (1, _log(rng, 17, 300))])
    if kind == "fwd":
        window, sinks = -1, 0
        if rng.random() < 0.3:
            window, sinks = _log(rng, 16, 4096), rng.choice([0, 4, 100])
        case = _fwd("", batch=_log(rng, 1, 64), hq=hkv * group, hkv=hkv, d=d, dtype=dtype, page=page, new=new,
                    ctx=(1, _log(rng, 64, 32000)), window=window, sinks=sinks, lens_seed=lens_seed)
    else:
        batch = _log(rng, 2, 128)
        top = _log(rng, 64, 32000)
        case = _shared("", batch=batch, groups=rng.randrange(1, min(4, batch // 2) + 1), hq=hkv * group, hkv=hkv, d=d,
                       dtype=dtype, page=page, new=new, shared=(top // 2, top), ctx=(0, _log(rng, 1, 2000)),
                       lens_seed=lens_seed)
    # no more reading or arithmetic than the largest listed cases
    while True:
        w = work(case)
        if w["bytes"] <= 2e9 and w["flops"] <= 7e10 and case["batch"] * case["new_hi"] <= 4096:
            break
        case["batch"] = max(1 if kind == "fwd" else 2, case["batch"] // 2)
        case["new_hi"] = max(case["new_lo"], case["new_hi"] * 2 // 3)
        for n in ("ctx_hi", "shared_hi"):
            if n in case:
                case[n] = max(case[n[:-2] + "lo"], case[n] * 2 // 3)
        if kind == "shared":
            case["groups"] = min(case["groups"], case["batch"] // 2)
            case["shared_lo"] = min(case["shared_lo"], case["shared_hi"] * 3 // 4)
    del case["name"]
    return case


# ---------------------------------------------------------------- lengths and sizes

def _lengths(case):
    """(cached keys before the new tokens, new tokens) of every request; they belong to the case, not to the seed."""
    r = random.Random(case["lens_seed"])
    n = case["batch"]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
    if case["op"] == "shared":
        cuts, shared = _groups(case)
        for g, s in enumerate(shared):
            for b in range(cuts[g], cuts[g + 1]):
                ctx[b] += s
    return ctx, new


def _groups(case):
    """(first request of each group and the number of requests, keys that each group's requests share)."""
    r = random.Random(case["lens_seed"] + 1)
    cuts = [0] + sorted(r.sample(range(1, case["batch"]), case["groups"] - 1)) + [case["batch"]]
    return cuts, [r.randint(case["shared_lo"], case["shared_hi"]) for _ in range(case["groups"])]


def _visible(n_q, n_k, window, sinks):
    """(visible pairs, keys some query sees) of one request under a causal band with sink keys."""
    i = np.arange(n_q, dtype=np.int64) + (n_k - n_q)
    lo = np.maximum(i - window, 0) if window >= 0 else np.zeros_like(i)
    beside = np.minimum(np.minimum(sinks, i + 1), lo)
    pairs = (i + 1 - lo + beside).sum()
    return int(pairs), int(n_k - lo[0] + max(0, min(sinks, int(lo[0]))))


def work(case):
    d = case["d"]
    if case["op"] == "write":
        rows = case["tokens"] * case["hkv"]
        # K and V: 16-bit rows in, codes and exponents out, 16-bit rows out again; slots
        return {"bytes": 2 * rows * (2 * d + (d + 1) + 2 * d) + (case["tokens"] + case["pad"]) * 4, "flops": 0}
    ctx, new = _lengths(case)
    rows = sum(new) * case["hq"]
    window, sinks = case.get("window", -1), case.get("sinks", 0)
    pairs = keys = pages = 0
    for c, n in zip(ctx, new):
        p, u = _visible(n, c + n, window, sinks)
        pairs += p
        keys += u
        pages += -(-u // case["page"])
    if case["op"] == "shared":   # a group's whole shared pages once
        cuts, shared = _groups(case)
        for g, s in enumerate(shared):
            again = cuts[g + 1] - cuts[g] - 1
            keys -= again * (s // case["page"]) * case["page"]
            pages -= again * (s // case["page"])
    per_key = 2 * (d + 1) if case["op"] == "fwd" else 4 * d
    return {"bytes": keys * case["hkv"] * per_key + rows * (d * 4 + 4) + pages * 4 + case["batch"] * 8,
            "flops": 4 * d * pairs * case["hq"]}


# ---------------------------------------------------------------- what a program has in hand

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _rows(g, shape, dtype):
    """Key or value rows, whose sizes differ from token to token and head to head."""
    size = torch.exp(0.3 * torch.randn(shape[:-1], generator=g, device="cuda", dtype=torch.float32))
    return _normal(g, shape, dtype).mul_(size[..., None].to(dtype))


def _quantise(x, dtype):
    """(codes, exponent bytes) of the rows along x's last dimension."""
    low, high = _EXPONENTS[dtype]
    x = x.float().clamp(-240.0 * 2.0 ** high, 240.0 * 2.0 ** high)   # the next code times 2^8 is no fp16 value
    top = x.abs().amax(dim=-1)
    fraction, e = torch.frexp(top)       # top = fraction * 2^e, fraction in [0.5, 1); 448 = 0.875 * 2^9
    e = e - 9 + (fraction > 0.875)
    e = e.clamp(low, high)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    codes = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _values(codes, exps):
    """What codes and exponent bytes stand for, in 32 bits."""
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), exps.int()[..., None] - 127)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "fwd":
        return _prepare_fwd(case, g)
    if case["op"] == "shared":
        return _prepare_shared(case, g)
    return _prepare_write(case, g)


def _ints(x):
    return torch.tensor(np.asarray(x), device="cuda", dtype=torch.int32)


def _tables(case, lens, pages, g, cuts=None, common=None):
    """Block table [batch, widest], pages in random order, -1 beyond each request's; the rows of a group (cuts) begin
    with the same `common` pages."""
    page = case["page"]
    need = np.array([-(-n // page) for n in lens])
    order = torch.randperm(pages, generator=g, device="cuda").cpu().numpy().astype(np.int32)
    table = np.full((len(lens), max(1, need.max())), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        first = 0
        if cuts is not None:
            k = int(np.searchsorted(cuts, b, side="right")) - 1
            if b > cuts[k]:
                first = common[k]
                table[b, :first] = table[cuts[k], :first]
        table[b, first:n] = order[at:at + n - first]
        at += n - first
    return torch.from_numpy(table).cuda(), at


def _prepare_fwd(case, g):
    dtype, d, page = _DTYPES[case["dtype"]], case["d"], case["page"]
    ctx, new = _lengths(case)
    lens = [c + n for c, n in zip(ctx, new)]
    pages = sum(-(-n // page) for n in lens) + 3
    table, _ = _tables(case, lens, pages, g)
    state = {"case": case, "new": new, "lens": lens, "table": table,
             "cu": _ints(np.concatenate([[0], np.cumsum(new)])), "lens_k": _ints(lens),
             "q": _normal(g, (sum(new), case["hq"], d), dtype), "scale": 1.0 / math.sqrt(d)}
    for x in ("k", "v"):
        codes = torch.empty((pages, case["hkv"], page, d), device="cuda", dtype=torch.float8_e4m3fn)
        exps = torch.empty((pages, case["hkv"], page), device="cuda", dtype=torch.uint8)
        step = max(1, (1 << 28) // (case["hkv"] * page * d))
        for p in range(0, pages, step):
            part = codes[p:p + step]
            codes[p:p + step], exps[p:p + step] = _quantise(_rows(g, part.shape, dtype), dtype)
        state[x], state[x + "_exps"] = codes, exps
    return state


def _prepare_shared(case, g):
    dtype, d, page = _DTYPES[case["dtype"]], case["d"], case["page"]
    ctx, new = _lengths(case)
    cuts, shared = _groups(case)
    lens = [c + n for c, n in zip(ctx, new)]
    common = [s // page for s in shared]
    pages = sum(-(-n // page) for n in lens) + 3 - sum(
        (cuts[k + 1] - cuts[k] - 1) * common[k] for k in range(len(shared)))
    table, _ = _tables(case, lens, pages, g, cuts, common)
    return {"case": case, "new": new, "lens": lens, "cuts": cuts, "common": [c * page for c in common], "table": table,
            "cu": _ints(np.concatenate([[0], np.cumsum(new)])), "lens_k": _ints(lens),
            "cu_groups": _ints(cuts), "shared": _ints([c * page for c in common]),
            "q": _normal(g, (sum(new), case["hq"], d), dtype),
            "k": _normal(g, (pages, case["hkv"], page, d), dtype),
            "v": _normal(g, (pages, case["hkv"], page, d), dtype), "scale": 1.0 / math.sqrt(d)}


def _prepare_write(case, g):
    dtype, d, hkv, page = _DTYPES[case["dtype"]], case["d"], case["hkv"], case["page"]
    total = case["tokens"] + case["pad"]
    if case["fused"]:   # [q heads | k heads | v heads] of one projection: strided views
        rows = _rows(g, (total, 3 * hkv, d), dtype)
        k, v = rows[:, hkv:2 * hkv], rows[:, 2 * hkv:]
    else:
        k, v = _rows(g, (total, hkv, d), dtype), _rows(g, (total, hkv, d), dtype)
    slots = torch.full((total,), -1, device="cuda", dtype=torch.int32)
    # runs of one page each, pages in random order, as a table of requests gives them
    order = torch.randperm(case["pages"], generator=g, device="cuda")
    at = torch.arange(case["tokens"], device="cuda")
    slots[:case["tokens"]] = (order[at // page] * page + at % page).to(torch.int32)
    state = {"case": case, "k": k, "v": v, "slots": slots}
    for x in ("k", "v"):
        state[x + "_cache"] = torch.zeros((case["pages"], hkv, page, d), device="cuda", dtype=torch.uint8).view(
            torch.float8_e4m3fn)
        state[x + "_exps"] = torch.full((case["pages"], hkv, page), 127, device="cuda", dtype=torch.uint8)
        state[x + "_back"] = torch.zeros((total, hkv, d), device="cuda", dtype=dtype)
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "fwd":
        return _plain_fwd(state)
    if op == "shared":
        return _plain_shared(state)
    return _plain_write(state)


def _own(state, op):
    import exact_tiled_attention_fa2_gb300 as fa2
    case = state["case"]
    if op == "fwd":
        return fa2.fa2_paged_fwd_fp8(state["q"], state["k"], state["v"], state["k_exps"], state["v_exps"],
                                     state["table"], state["cu"], state["lens_k"], scale=state["scale"],
                                     window_left=case["window"], window_right=0, sink_len=case["sinks"],
                                     max_seqlen_q=max(state["new"]))
    if op == "shared":
        return fa2.fa2_paged_fwd_shared(state["q"], state["k"], state["v"], state["table"], state["cu"],
                                        state["lens_k"], state["cu_groups"], state["shared"], scale=state["scale"],
                                        window_right=0, max_seqlen_q=max(state["new"]))
    cache = state["k_cache"], state["v_cache"], state["k_exps"], state["v_exps"]
    fa2.fa2_paged_append_fp8(state["k"], state["v"], state["slots"], *cache)
    return fa2.fa2_paged_read_fp8(state["slots"], *cache, k=state["k_back"], v=state["v_back"])


def _heads_first(q, hkv):
    """[n, hq, d] as [hkv, group * n, d], the rows of a K/V head's query heads one after another, in 32 bits."""
    n, hq, d = q.shape
    return q.float().reshape(n, hkv, hq // hkv, d).permute(1, 2, 0, 3).reshape(hkv, -1, d)


def _heads_back(x, n):
    """The inverse of _heads_first."""
    hkv, rows, d = x.shape
    return x.reshape(hkv, rows // n, n, d).permute(2, 0, 1, 3).reshape(n, -1, d)


def _attend(x, k, v, scale, hidden=None):
    """(m, l, O) of query rows x [hkv, rows, d] over k, v [hkv, keys, d]; hidden: [queries, keys], repeated over the
    rows."""
    s = torch.matmul(x, k.transpose(1, 2)).mul_(scale)
    if hidden is not None:
        s.view(s.shape[0], -1, *hidden.shape).masked_fill_(hidden, float("-inf"))
    m = s.amax(dim=-1, keepdim=True)
    p = s.sub_(m).exp_()
    return m, p.sum(dim=-1, keepdim=True), torch.matmul(p, v)


def _hidden(n, n_k, window, sinks, device):
    i = torch.arange(n_k - n, n_k, device=device)[:, None]
    j = torch.arange(n_k, device=device)[None, :]
    hidden = j > i
    if window >= 0:
        hidden = hidden | ((j < i - window) & (j >= sinks))
    return hidden


def _keys(cache, pages, n):
    """[heads, n, d] of the keys on these pages, 32-bit."""
    x = cache[pages].transpose(0, 1)
    return x.reshape(x.shape[0], -1, x.shape[-1])[:, :n].float()


def _plain_fwd(state):
    case, q = state["case"], state["q"]
    hkv, page = case["hkv"], case["page"]
    o = torch.empty_like(q)
    lse = torch.empty((case["hq"], q.shape[0]), device=q.device, dtype=torch.float32)
    codes = {x: state[x].view(torch.uint8) for x in ("k", "v")}
    row = 0
    for b, (n, n_k) in enumerate(zip(state["new"], state["lens"])):
        pages = state["table"][b, :-(-n_k // page)].long()
        k, v = (_values(codes[x][pages], state[x + "_exps"][pages]).transpose(0, 1).reshape(hkv, -1, case["d"])[:, :n_k]
                for x in ("k", "v"))
        hidden = None
        if n > 1 or case["window"] >= 0:
            hidden = _hidden(n, n_k, case["window"], case["sinks"], q.device)
        m, total, y = _attend(_heads_first(q[row:row + n], hkv), k, v, state["scale"], hidden)
        o[row:row + n] = _heads_back(y / total, n).to(q.dtype)
        lse[:, row:row + n] = (m + total.log()).reshape(-1, n)
        row += n
    return o, lse


def _plain_shared(state):
    """Every group's shared pages once for all of its query rows, then each request's own keys."""
    case, q, cuts = state["case"], state["q"], state["cuts"]
    hkv, page, scale = case["hkv"], case["page"], state["scale"]
    o = torch.empty_like(q)
    lse = torch.empty((case["hq"], q.shape[0]), device=q.device, dtype=torch.float32)
    first = [0] + np.cumsum(state["new"]).tolist()
    for g, common in enumerate(state["common"]):
        r0, r1 = first[cuts[g]], first[cuts[g + 1]]
        if common:
            pages = state["table"][cuts[g], :common // page].long()
            k, v = _keys(state["k"], pages, common), _keys(state["v"], pages, common)
            m0, l0, y0 = _attend(_heads_first(q[r0:r1], hkv), k, v, scale)
            m0, l0, y0 = (x.reshape(hkv, -1, r1 - r0, x.shape[-1]) for x in (m0, l0, y0))
        for b in range(cuts[g], cuts[g + 1]):
            row, n, n_k = first[b], state["new"][b], state["lens"][b]
            pages = state["table"][b, common // page:-(-n_k // page)].long()
            k, v = _keys(state["k"], pages, n_k - common), _keys(state["v"], pages, n_k - common)
            hidden = _hidden(n, n_k - common, -1, 0, q.device) if n > 1 else None
            m, total, y = _attend(_heads_first(q[row:row + n], hkv), k, v, scale, hidden)
            if common:   # join the two parts
                at = slice(row - r0, row - r0 + n)
                part = [x[:, :, at].reshape(hkv, -1, x.shape[-1]) for x in (m0, l0, y0)]
                top = torch.maximum(m, part[0])
                f, f0 = (m - top).exp(), (part[0] - top).exp()
                m, total, y = top, total * f + part[1] * f0, y * f + part[2] * f0
            o[row:row + n] = _heads_back(y / total, n).to(q.dtype)
            lse[:, row:row + n] = (m + total.log()).reshape(-1, n)
    return o, lse


def _plain_write(state):
    page, tokens = state["case"]["page"], state["case"]["tokens"]
    slots = state["slots"][:tokens].long()
    where, at = slots // page, slots % page
    for x in ("k", "v"):
        rows, codes, exps, back = state[x], state[x + "_cache"].view(torch.uint8), state[x + "_exps"], state[x + "_back"]
        c, e = _quantise(rows[:tokens], rows.dtype)
        codes[where, :, at] = c.view(torch.uint8)
        exps[where, :, at] = e
        back[:tokens] = _values(codes[where, :, at], exps[where, :, at]).to(back.dtype)
    return state["k_back"], state["v_back"]


# ---------------------------------------------------------------- from the definition, in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "write":
        return tuple(_exact_row_values(state, x) for x in ("k", "v"))
    return _exact_attention(state)


def _code_table():
    """The values of the 256 e4m3 codes: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7f and 0xff are NaN."""
    t = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = (f / 8) * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        t[c] = math.nan if e == 15 and f == 7 else -x if c & 128 else x
    return torch.from_numpy(t).cuda()


def _exact_row_values(state, x):
    """Each written row's values on the grid of its codes: steps of an eighth of the value's power of two, from
    2^-9 on, in units of the row's scale; halves to the even multiple."""
    rows = state[x].double()
    tokens = state["case"]["tokens"]
    lowest, highest = (2.0 ** e for e in _EXPONENTS[state[x].dtype])
    rows = rows.clamp(-240 * highest, 240 * highest)
    out = torch.zeros_like(rows)
    rows = rows[:tokens]
    top = rows.abs().amax(-1, keepdim=True)
    scale = torch.ones_like(top)
    for _ in range(150):   # the smallest power of two with top <= 448 * scale
        scale = torch.where((top > 448 * scale) & (scale < highest), scale * 2, scale)
        scale = torch.where((top <= 224 * scale) & (scale > lowest) & (top > 0), scale / 2, scale)
    y = rows / scale
    power = torch.full_like(y, 2.0 ** -6)
    for _ in range(15):
        power = torch.where(y.abs() >= 2 * power, power * 2, power)
    step = power / 8
    out[:tokens] = torch.round(y / step) * step * scale   # round: halves to even
    return out


def _exact_attention(state):
    case = state["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    group, window, sinks = hq // hkv, case.get("window", -1), case.get("sinks", 0)
    table = state["table"].cpu().numpy()
    total = state["q"].shape[0]
    o = torch.empty((total, hq, d), device="cuda", dtype=torch.float64)
    lse = torch.empty((hq, total), device="cuda", dtype=torch.float64)
    codes = _code_table() if case["op"] == "fwd" else None

    def rows(x, page_of, h, at):
        if codes is None:
            return state[x][page_of, h, at].double()
        e = state[x + "_exps"][page_of, h, at].double() - 127
        return codes[state[x].view(torch.uint8)[page_of, h, at].long()] * torch.exp2(e)[:, None]

    start = 0
    for b, (n, n_k) in enumerate(zip(state["new"], state["lens"])):
        j = np.arange(n_k)
        page_of = torch.from_numpy(table[b, j // page].astype(np.int64)).cuda()
        at = torch.from_numpy(j % page).cuda()
        key = torch.from_numpy(j).cuda()
        place = torch.arange(n, device="cuda") + (n_k - n)
        hidden = key[None, :] > place[:, None]
        if window >= 0:
            hidden |= (key[None, :] + window < place[:, None]) & (key[None, :] >= sinks)
        for h in range(hkv):
            keys, values = rows("k", page_of, h, at), rows("v", page_of, h, at)
            for m in range(h * group, (h + 1) * group):
                x = state["q"][start:start + n, m].double() @ keys.T
                x = (x * state["scale"]).masked_fill_(hidden, -math.inf)
                norm = torch.logsumexp(x, dim=1)
                o[start:start + n, m] = torch.exp(x - norm[:, None]) @ values
                lse[m, start:start + n] = norm
        start += n
    return o, lse
