"""Measured cases of the serving operators that stand beside the decode.

* ``decode_attention``: attention of one new token per sequence over a paged or
  contiguous KV cache, optionally through a sliding window with visible first
  tokens, optionally storing the new token's K/V row first.
* ``PagePool``: forking, reserving, trimming and compacting the pages of a paged
  cache.
* ``token_logprobs``: log probabilities of given tokens with entropy, rank and
  top alternatives.

``run`` computes the plain forms (elementary torch operations in 32 bits) or,
with ``own`` set, calls the package.  Head layouts, vocabularies and page sizes
are those of the synthetic decoder shapes (tiny, 1B, 8B, MoE), or generic.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- the cases

def _attn(name, seqs, heads, kv_heads, dim, page, length, *, ragged=False, kv="bf16", io="bf16", window=0,
          sinks=0, append=False):
    c = {"op": "attention", "seqs": seqs, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
         "length": length, "ragged": ragged, "kv": kv, "io": io, "window": window, "sinks": sinks, "append": append}
    return {"name": name, **c} if name else c


def _pages(name, op, layers, kv_heads, dim, page, rows, length, spare, *, kv="bf16", fan="beam", window=0, sinks=0):
    c = {"op": op, "layers": layers, "kv_heads": kv_heads, "dim": dim, "page": page, "rows": rows, "length": length,
         "spare": spare, "kv": kv, "fan": fan, "window": window, "sinks": sinks}
    return {"name": name, **c} if name else c


def _logp(name, rows, vocab, dtype, top_k, *, pad=0, allowed=0):
    c = {"op": "logprobs", "rows": rows, "vocab": vocab, "dtype": dtype, "top_k": top_k, "pad": pad,
         "allowed": allowed}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one user's step of the 1B shape: the smallest call, its new row stored on the way
        _attn("attn_1b_one_user", 1, 32, 8, 64, 128, 1024, append=True),
        # eight users of the 8B shape at ragged lengths up to 8192, fp32 q and output as inside the decode
        _attn("attn_8b_ragged_fp32", 8, 32, 8, 128, 64, 8192, ragged=True, io="fp32"),
        # four documents of 131072 positions in an e4m3 cache: the largest read
        _attn("attn_8b_long_e4m3", 4, 32, 8, 128, 64, 131072, kv="e4m3"),
        # many streaming users behind a 4096-position window with 4 first tokens kept, seven query heads per kv head
        _attn("attn_window_sinks", 64, 28, 4, 128, 16, 20011, ragged=True, window=4096, sinks=4),
        # a beam step of the 1B shape: half of eight rows survive, each forked once
        _pages("fork_beam_1b", "fork", 16, 8, 64, 128, 8, 1061, 24),
        # one 8B prompt fanned out to 32 samples
        _pages("fork_fan_8b", "fork", 32, 8, 128, 64, 32, 1000, 48, fan="fan"),
        # a small e4m3 pool of the MoE shape behind a window: trimmed, then compacted
        _pages("compact_window_moe_e4m3", "compact", 24, 4, 128, 64, 6, 1500, 10, kv="e4m3", window=512, sinks=4),
        # an 8B pool after half of its pages were given back: the largest move
        _pages("compact_8b", "compact", 32, 8, 128, 64, 4, 2090, 130),
        # one token of the 1B vocabulary with its five best alternatives
        _logp("logprobs_1b_one", 1, 32000, "fp32", 5),
        # a decode step of eight sequences of the 8B vocabulary
        _logp("logprobs_8b_step", 8, 128256, "fp32", 20),
        # scoring a prompt of 1024 tokens
        _logp("logprobs_8b_score", 1024, 128256, "fp32", 0),
        # ragged: bf16 logits of an odd vocabulary with padded rows, most of it masked by a grammar
        _logp("logprobs_masked_bf16", 333, 64007, "bf16", 64, pad=9, allowed=20000),
    ]


def _span(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "fork", "compact", "logprobs", "logprobs"])
    if op == "attention":
        heads, kv_heads, dim = rng.choice([(4, 2, 64), (32, 8, 64), (32, 8, 128), (16, 4, 128), (28, 4, 128),
                                           (6, 6, 64), (10, 2, 128), (16, 1, 128)])
        kv = rng.choice(["bf16", "e4m3"])
        seqs = _span(rng, 1, 64)
        room = (1 << 30) // (seqs * kv_heads * dim * 2 * (2 if kv == "bf16" else 1))
        length = _span(rng, 1, min(131072, room))
        window = rng.choice([0, 0, _span(rng, 1, 8192)])
        return _attn(None, seqs, heads, kv_heads, dim, rng.choice([0, 16, 24, 64, 128]), length,
                     ragged=rng.random() < 0.5, kv=kv, io=rng.choice(["bf16", "fp32"]), window=window,
                     sinks=rng.choice([0, 1, 4, 70]) if window else 0, append=length < 2048 and rng.random() < 0.5)
    if op in ("fork", "compact"):
        kv_heads, dim, page = rng.choice([(2, 64, 128), (8, 64, 128), (8, 128, 64), (4, 128, 64), (3, 64, 24)])
        layers, rows = rng.choice([2, 16, 24, 32]), _span(rng, 2, 24)
        kv = rng.choice(["bf16", "e4m3"])
        page_bytes = layers * 2 * kv_heads * dim * page * (2 if kv == "bf16" else 1)
        pages = max(3 * rows, min(4000, (1 << 31) // page_bytes))
        length = _span(rng, 1, max(2, (pages // rows // 2) * page))
        return _pages(None, op, layers, kv_heads, dim, page, rows, length, rows + _span(rng, 1, max(2, pages // 4)),
                      kv=kv, fan=rng.choice(["beam", "fan"]),
                      window=_span(rng, 1, length) if op == "compact" and rng.random() < 0.6 else 0,
                      sinks=rng.choice([0, 4]))
    vocab = rng.choice([4096, 32000, 64000, 128256, _span(rng, 100, 200000)])
    rows = _span(rng, 1, max(2, min(1024, (1 << 27) // vocab)))
    return _logp(None, rows, vocab, rng.choice(["fp32", "bf16"]), min(vocab, rng.choice([0, 1, 5, 20, 64])),
                 pad=rng.choice([0, 0, 3, 8]), allowed=rng.choice([0, 0, max(1, vocab // 3)]))


# ---------------------------------------------------------------- shapes that follow from a case alone

def _lengths(c):
    """Positions of each sequence: all `length`, or spread evenly down from it."""
    n = c["seqs"]
    if not c["ragged"]:
        return [c["length"]] * n
    return [max(1, c["length"] - (c["length"] * b * 7) // (8 * n)) for b in range(n)]


def _visible(c, n):
    if not c["window"] or n <= c["window"]:
        return n
    return min(n, c["window"] + min(c["sinks"], n - c["window"]))


def _row_lengths(c):
    """Positions of each row of a page case (not all multiples of the page)."""
    return [max(1, c["length"] - (r * c["length"]) // (3 * c["rows"])) for r in range(c["rows"])]


def _parents(c):
    if c["fan"] == "fan":
        return [0] * c["rows"]
    return [r // 2 for r in range(c["rows"])]


def _kept(c, n):
    """The page columns of a row of n positions that its window still shows."""
    P = c["page"]
    return [j for j in range(-(-n // P))
            if not c["window"] or (j + 1) * P > n - c["window"] or j * P < c["sinks"]]


def _live_split(c):
    """(pages in the pool, live pages, live pages numbered past them) of a compaction case."""
    lens = _row_lengths(c)
    live = sum(len(_kept(c, n)) for n in lens)
    held = sum(-(-n // c["page"]) for n in lens)
    total = held + c["spare"]
    high = min(total - live, live) * live // total if total else 0
    return total, live, max(min(1, total - live, live), high)


def work(case):
    c = case
    if c["op"] == "attention":
        e = 2 if c["kv"] == "bf16" else 1
        io = 2 if c["io"] == "bf16" else 4
        seen = sum(_visible(c, n) for n in _lengths(c))
        b = seen * c["kv_heads"] * c["dim"] * 2 * e + c["seqs"] * c["heads"] * (c["dim"] * 2 * io + 4)
        if c["append"]:
            b += c["seqs"] * c["kv_heads"] * c["dim"] * 2 * io
        return {"bytes": b, "flops": 4 * seen * c["heads"] * c["dim"]}
    if c["op"] == "logprobs":
        e = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": c["rows"] * (c["vocab"] * e + 16 + 8 * c["top_k"]), "flops": 5 * c["rows"] * c["vocab"]}
    row = c["layers"] * 2 * c["kv_heads"] * c["dim"] * (2 if c["kv"] == "bf16" else 1)   # one position
    lens, P = _row_lengths(c), c["page"]
    cols = -(-(max(lens) + P) // P) + 1
    table = 8 * c["rows"] * cols
    if c["op"] == "fork":
        par = _parents(c)
        extra = sum(lens[p] % P for i, p in enumerate(par) if p in par[:i] or (p != i and par[p] == p))
        return {"bytes": 2 * row * extra + table, "flops": 0}
    total, live, high = _live_split(c)
    return {"bytes": 2 * row * P * high + table + 12 * total, "flops": 0}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 2 + 1)


def _cache(shape, kv, g, std):
    x = torch.empty(shape, dtype=BF16, device=DEV).normal_(0.0, std, generator=g)
    if kv == "bf16":
        return x
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    for i in range(shape[0]):
        out[i] = (x[i].float() / KV_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return out


KV_SCALE = 2.0 ** -5        # 6 standard deviations of the entries sit just under e4m3's largest value
KV_STD = 0.02 * 64          # a projection of a unit-RMS activation of width 4096


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "attention":
        return _prepare_attention(c, g)
    if c["op"] == "logprobs":
        return _prepare_logprobs(c, g)
    return _prepare_pages(c, g)


def _prepare_attention(c, g):
    lens = _lengths(c)
    B, H, KH, D = c["seqs"], c["heads"], c["kv_heads"], c["dim"]
    io = F32 if c["io"] == "fp32" else BF16
    P = c["page"] or c["length"]
    cols = -(-c["length"] // P)
    if c["page"]:
        pages = sum(-(-n // P) for n in lens) + 3
        ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).tolist()
        table, at = [], 0
        for n in lens:
            used = -(-n // P)
            table.append(ids[at:at + used] + [-1] * (cols - used))
            at += used
        table = torch.tensor(table, dtype=torch.int32, device=DEV)
    else:
        pages, table = B, None
    s = {"c": c, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV),
         "k": _cache((pages, KH, P, D), c["kv"], g, KV_STD), "v": _cache((pages, KH, P, D), c["kv"], g, KV_STD),
         "q": (torch.randn(B, H, D, generator=g, device=DEV) * KV_STD).to(io),
         "k_new": None, "v_new": None, "scale": KV_SCALE if c["kv"] == "e4m3" else 1.0}
    if c["append"]:
        s["k_new"] = (torch.randn(B, KH, D, generator=g, device=DEV) * KV_STD).to(io)
        s["v_new"] = (torch.randn(B, KH, D, generator=g, device=DEV) * KV_STD).to(io)
    return s


def _prepare_pages(c, g):
    lens, P = _row_lengths(c), c["page"]
    rows, cols = c["rows"], -(-(max(lens) + P) // P) + 1
    if c["op"] == "fork":
        pages = sum(-(-n // P) for n in lens) + c["spare"]
        ids = torch.randperm(pages, generator=g, device=DEV).tolist()
        gone = []
    else:
        # the pages that stay sit scattered over the pool, `high` of them numbered past their count
        pages, live, high = _live_split(c)
        lo = torch.randperm(live, generator=g, device=DEV).tolist()
        hi = (torch.randperm(pages - live, generator=g, device=DEV) + live).tolist()
        stay = lo[: live - high] + hi[:high]
        order = torch.randperm(live, generator=g, device=DEV).tolist()
        ids = [stay[i] for i in order]
        gone = lo[live - high:] + hi[high:]
    table, refs = [[-1] * cols for _ in range(rows)], [0] * pages
    for r, n in enumerate(lens):
        keep = set(_kept(c, n)) if c["op"] == "compact" else set(range(cols))
        for j in range(-(-n // P)):
            table[r][j] = ids.pop() if j in keep else gone.pop()
            refs[table[r][j]] += 1
    parents = _parents(c)
    shape = (c["layers"], pages, c["kv_heads"], P, c["dim"])
    i32 = dict(dtype=torch.int32, device=DEV)
    after = [lens[p] for p in parents] if c["op"] == "fork" else lens
    return {"c": c, "k": _cache(shape, c["kv"], g, KV_STD), "v": _cache(shape, c["kv"], g, KV_STD),
            "table": torch.tensor(table, **i32), "refs": torch.tensor(refs, **i32), "lens": torch.tensor(lens, **i32),
            "parents": torch.tensor(parents, **i32), "want": torch.tensor([n + 1 for n in after], **i32),
            "status": torch.zeros(1, **i32)}


def _prepare_logprobs(c, g):
    rows, vocab = c["rows"], c["vocab"]
    x = torch.randn(rows, vocab + c["pad"], generator=g, device=DEV) * 2.5
    if c["allowed"]:
        # a grammar leaves about `allowed` tokens, at least the first and the last
        shut = torch.rand(rows, vocab + c["pad"], generator=g, device=DEV) >= c["allowed"] / vocab
        shut[:, 0] = False
        shut[:, vocab - 1] = False
        x = x.masked_fill_(shut, float("-inf"))
    x = x.to(F32 if c["dtype"] == "fp32" else BF16)[:, :vocab]
    # half of the tokens were sampled from the distribution, the others are a text's
    noise = -torch.log(-torch.log(torch.rand(rows, vocab, generator=g, device=DEV).clamp_(1e-20, 1 - 1e-7)))
    tokens = (x.float() + noise).argmax(1)
    text = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    tokens = torch.where(torch.arange(rows, device=DEV) % 2 == 0, tokens, text).to(torch.int32)
    return {"c": c, "logits": x, "tokens": tokens}


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["c"]["op"]
    if op == "attention":
        return _run_attention(state)
    if op == "logprobs":
        return _run_logprobs(state)
    return _run_pages(state)


def _values(t):
    """A cache tensor as the values it stands for."""
    return t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t


def _run_attention(s):
    c = s["c"]
    if own:
        from persistent_decode_b200 import decode_attention
        out, lse = decode_attention(s["q"], s["k"], s["v"], s["lens"], page_table=s["table"], k_new=s["k_new"],
                                    v_new=s["v_new"], window=c["window"], sinks=c["sinks"], k_scale=s["scale"],
                                    v_scale=s["scale"], return_lse=True)
    else:
        out, lse = _plain_attention(s)
    r = {"out": out, "lse": lse}
    if c["append"]:
        r["k"], r["v"] = _values(s["k"]), _values(s["v"])
    return r


def _plain_attention(s):
    c, q, lens = s["c"], s["q"], s["lens"].long()
    B, H, D = q.shape
    KH, P = s["k"].shape[1], s["k"].shape[2]
    table = s["table"].long() if s["table"] is not None else torch.arange(B, device=q.device)[:, None]
    if s["k_new"] is not None:
        at = table.gather(1, ((lens - 1) // P)[:, None])[:, 0]
        for name in ("k", "v"):
            new = s[name + "_new"].float() / s["scale"]
            if s[name].dtype == torch.uint8:
                new = new.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name][at, :, (lens - 1) % P] = new.to(s[name].dtype)
    pos = torch.arange(table.shape[1] * P, device=q.device)
    see = pos < lens[:, None]
    if c["window"]:
        see = see & ((pos >= lens[:, None] - c["window"]) | (pos < c["sinks"]))
    flat = table.clamp(min=0).reshape(-1)

    def rows(t):
        x = _values(t[flat]).float() * s["scale"]
        return x.view(B, table.shape[1], KH, P, D).permute(0, 2, 1, 3, 4).reshape(B, KH, -1, D)

    scores = torch.matmul(q.float().view(B, KH, H // KH, D), rows(s["k"]).transpose(2, 3)) / math.sqrt(D)
    scores = scores.masked_fill(~see[:, None, None], float("-inf"))
    top = scores.amax(3, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(3, keepdim=True)
    out = torch.matmul(p, rows(s["v"])) / total
    lse = (top + torch.log(total)).reshape(B, H)
    return out.reshape(B, H, D).to(q.dtype), lse


def _run_logprobs(s):
    c, x, tok = s["c"], s["logits"], s["tokens"]
    if own:
        from persistent_decode_b200 import token_logprobs
        r = token_logprobs(x, tok, top_k=c["top_k"])
        out = {"logprob": r.logprob, "entropy": r.entropy, "rank": r.rank}
        if c["top_k"]:
            out["top_ids"], out["top_logprobs"] = r.top_ids, r.top_logprobs
        return out
    x = x.float()
    top = x.amax(1, keepdim=True)
    d = x - top
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    norm = top + torch.log(total)
    mine = x.gather(1, tok.long()[:, None])
    before = torch.arange(c["vocab"], device=x.device) < tok[:, None]
    out = {"logprob": (mine - norm)[:, 0],
           "entropy": (torch.log(total) - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / total)[:, 0],
           "rank": ((x > mine) | ((x == mine) & before)).sum(1).to(torch.int32)}
    if c["top_k"]:
        best, ids = torch.sort(x, dim=1, descending=True, stable=True)
        out["top_ids"] = ids[:, :c["top_k"]].to(torch.int32)
        out["top_logprobs"] = best[:, :c["top_k"]] - norm
    return out


def _run_pages(s):
    c = s["c"]
    table, refs, lens = s["table"].clone(), s["refs"].clone(), s["lens"].clone()
    remap = None
    if own:
        from persistent_decode_b200 import PagePool
        pool = PagePool(s["k"], s["v"], table, lens, refs, status=s["status"])
        if c["op"] == "fork":
            pool.fork(s["parents"])
            pool.reserve(s["want"])
        else:
            pool.trim(c["window"], c["sinks"])
            remap = pool.compact()
    elif c["op"] == "fork":
        table, refs, lens = _plain_fork(s["k"], s["v"], table, refs, lens, s["parents"].long())
        table, refs = _plain_reserve(table, refs, lens, s["want"], s["k"].shape[3])
    else:
        table, refs = _plain_trim(table, refs, lens, c["window"], c["sinks"], s["k"].shape[3])
        table, refs, remap = _plain_compact(s["k"], s["v"], table, refs)
    r = {"k": _values(s["k"]), "v": _values(s["v"]), "table": table, "refs": refs, "lens": lens}
    return r if remap is None else {**r, "remap": remap}


def _free_pages(refs, n):
    """The n lowest-numbered pages that nothing refers to."""
    return torch.sort((refs > 0).to(torch.int32), stable=True).indices[:n]


def _counts(table, refs):
    """How often each page stands in the table."""
    n = torch.zeros(refs.shape[0] + 1, dtype=torch.int32, device=refs.device)
    n.index_add_(0, (table + 1).reshape(-1).long(), torch.ones(table.numel(), dtype=torch.int32, device=refs.device))
    return n[1:]


def _plain_fork(k, v, table, refs, lens, parents):
    """Row r becomes row parents[r] (-1: empty).  Full pages are shared; the heir of a
    row (itself, or else its first child) keeps the partly filled page and the reserved
    ones behind it, every other child gets a copy of the filled positions."""
    P, rows, dev = k.shape[3], table.shape[0], table.device
    me = torch.arange(rows, device=dev)
    child = parents[None, :] == me[:, None]                                   # [parent][child]
    first = torch.where(child, me[None, :], rows).amin(1)
    heir = torch.where(child.diagonal(), me, first)
    par = parents.clamp(min=0)
    inherits = (heir[par] == me) & (parents >= 0)
    had = lens[par] * (parents >= 0).to(lens.dtype)
    full = had // P
    col = torch.arange(table.shape[1], device=dev)
    out = torch.where((col < full[:, None]) | inherits[:, None], table[par], -1)
    out = torch.where((parents >= 0)[:, None], out, -1)
    needs = (parents >= 0) & ~inherits & (had % P > 0)
    fresh = _free_pages(refs, rows)[(needs.cumsum(0) - 1).clamp(min=0)]
    at = full.long().clamp(max=table.shape[1] - 1)
    src = table[par, at].long()
    who = torch.nonzero(needs)[:, 0]
    filled = (torch.arange(P, device=dev) < (had % P)[who, None])[None, :, None, :, None]
    for t in (k, v):
        t[:, fresh[who]] = torch.where(filled, t[:, src[who]], t[:, fresh[who]])
    out[who, at[who]] = fresh[who].to(torch.int32)
    return out, refs + _counts(out, refs) - _counts(table, refs), had


def _plain_reserve(table, refs, lens, want, P):
    """Each row gets the pages that want[r] positions need and it lacks, in row order."""
    col = torch.arange(table.shape[1], device=table.device)
    lacks = (table < 0) & (col >= (lens // P)[:, None]) & (col * P < want[:, None])
    nth = lacks.reshape(-1).cumsum(0).reshape(lacks.shape) - 1
    fresh = _free_pages(refs, refs.shape[0]).to(torch.int32)
    out = torch.where(lacks, fresh[nth.clamp(0, refs.shape[0] - 1)], table)
    return out, refs + _counts(out, refs) - _counts(table, refs)


def _plain_trim(table, refs, lens, window, sinks, P):
    """Pages that no later token can see through the window are given back."""
    col = torch.arange(table.shape[1], device=table.device)
    gone = ((col + 1) * P <= lens[:, None] - window) & (col * P >= sinks) & bool(window)
    out = torch.where(gone, -1, table)
    return out, refs + _counts(out, refs) - _counts(table, refs)


def _plain_compact(k, v, table, refs):
    """The k-th free page below the number of live pages takes the k-th live page above it."""
    used = refs > 0
    live = used.sum()
    ids = torch.arange(refs.shape[0], device=refs.device)
    holes = torch.nonzero(~used & (ids < live))[:, 0]
    high = torch.nonzero(used & (ids >= live))[:, 0]
    for t in (k, v):
        t[:, holes] = t[:, high]
    remap = torch.where(used, ids, -1)
    remap[high] = holes
    out_refs = refs.clone()
    out_refs[holes] = refs[high]
    out_refs[high] = 0
    out = torch.where(table >= 0, remap[table.clamp(min=0).long()], -1)
    return out.to(torch.int32), out_refs, remap.to(torch.int32)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "attention":
        return _exact_attention(c, s)
    if c["op"] == "logprobs":
        return _exact_logprobs(c, s)
    return None     # pages move whole: nothing is computed but whole numbers


def _exact_attention(c, s):
    lens, P, g = _lengths(c), s["k"].shape[2], c["heads"] // c["kv_heads"]
    out = torch.zeros(c["seqs"], c["heads"], c["dim"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(c["seqs"], c["heads"], dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        p = torch.arange(n, device=DEV)
        if c["window"]:
            p = p[(p >= n - c["window"]) | (p < c["sinks"])]
        page = s["table"][b][p // P].long() if s["table"] is not None else torch.full_like(p, b)
        for h in range(c["kv_heads"]):
            kv = []
            for name in ("k", "v"):
                x = s[name][page, h, p % P]
                if c["append"]:
                    new = s[name + "_new"][b, h].double() / s["scale"]
                    if x.dtype == torch.uint8:
                        x[-1] = new.clamp(-448, 448).float().to(torch.float8_e4m3fn).view(torch.uint8)
                    else:
                        x[-1] = new.to(x.dtype)
                kv.append((x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x).to(F32).double() * s["scale"])
            for j in range(h * g, h * g + g):
                score = (kv[0] * s["q"][b, j].double()).sum(1) / c["dim"] ** 0.5
                lse[b, j] = torch.logsumexp(score, 0)
                out[b, j] = (torch.exp(score - lse[b, j])[:, None] * kv[1]).sum(0)
    r = {"out": out, "lse": lse}
    return {**r, "k": None, "v": None} if c["append"] else r


def _exact_logprobs(c, s):
    rows, k = c["rows"], c["top_k"]
    logprob = torch.zeros(rows, dtype=torch.float64, device=DEV)
    entropy = torch.zeros_like(logprob)
    best = torch.zeros(rows, k, dtype=torch.float64, device=DEV)
    for r in range(rows):
        lp = torch.log_softmax(s["logits"][r].double(), 0)
        logprob[r] = lp[s["tokens"][r].long()]
        keep = lp[lp > -math.inf]
        entropy[r] = -(keep.exp() * keep).sum()
        if k:
            best[r] = torch.topk(lp, k).values
    out = {"logprob": logprob, "entropy": entropy, "rank": None}
    return {**out, "top_ids": None, "top_logprobs": best} if k else out
