"""Measured cases of the 8-bit paged key/value cache's page bookkeeping, and of the
attention over it with other scores and masks.

Four operators, each in a plain form (elementary torch operations) and, where
``own`` is true, through the library's entry points:

* ``attention``  softmax(x + mask) V over the cached tokens with x = scale q.k,
                 capped (cap tanh(x / cap)), biased by distance (minus a head's slope
                 times the distance), with prefixes that every query of a sequence
                 sees, documents that end a query's sight, a sliding window and
                 first tokens that stay visible.
* ``grow``       a serving step's pages: give back what the last step's guess took
                 and what slid out of the window, take pages for the new tokens.
* ``fork``       release the child sequences, let them share a prefix of their
                 parents' pages, copy the pages that end inside the prefix.
* ``compact``    move the pages in use to the front of the pool.

The cache is K codes int8 [page][kv head][slot][dim], V codes int8
[page][kv head][dim][slot] and fp32 scales [page][kv head][K, V].  The book is
refs int32 [pages], the number of table entries that hold each page, and the block
table int32 [sequence][entry]; the lowest free page is always taken first.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
ALL = (1 << 31) - 1


def _attention(dtype, seqs, new, kv, q_heads, kv_heads, dim, page, ragged=False, window=0, sinks=0, cap=0.0, biased=False,
               prefix=0.0, docs=0):
    return {"op": "attention", "dtype": dtype, "seqs": seqs, "new": new, "kv": kv, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "ragged": ragged, "window": window, "sinks": sinks, "cap": cap,
            "biased": biased, "prefix": prefix, "docs": docs}


def _grow(rows, new, kv, page, pool, window=0, sinks=0):
    return {"op": "grow", "rows": rows, "new": new, "kv": kv, "page": page, "pool": pool, "window": window, "sinks": sinks}


def _fork(parents, children, kv, kv_heads, dim, page, layers):
    return {"op": "fork", "parents": parents, "children": children, "kv": kv, "kv_heads": kv_heads, "dim": dim,
            "page": page, "layers": layers}


def _compact(rows, kv, kv_heads, dim, page, layers, held):
    return {"op": "compact", "rows": rows, "kv": kv, "kv_heads": kv_heads, "dim": dim, "page": page, "layers": layers,
            "held": held}


def listed():
    named = {
        # one user's next token over a short chat, capped scores, wide heads: pure latency
        "capped decode short": _attention("f16", 1, 1, 777, 16, 8, 256, 16, cap=50.0),
        # a full serving batch at ragged lengths, capped scores in a sliding window
        "capped decode 64 sequences": _attention("bf16", 64, 1, 8192, 64, 8, 128, 64, ragged=True, window=4096, sinks=4,
                                                 cap=30.0),
        # one user's next token over a long document, biased by distance, every head with its own keys (a 4096-wide layer)
        "biased decode long": _attention("f16", 1, 1, 32768, 32, 32, 128, 32, biased=True),
        # a whole prompt with capped scores (an 8192-wide layer)
        "capped prompt 8192": _attention("bf16", 1, 8192, 8192, 64, 8, 128, 64, cap=50.0),
        # odd documents packed into one prompt, biased by distance
        "biased packed documents": _attention("f16", 1, 8191, 8191, 32, 8, 128, 64, biased=True, docs=11),
        # prompts whose first three quarters (an image, an instruction) are read in both directions, wide heads
        "prefix prompts": _attention("bf16", 8, 2048, 2500, 16, 4, 256, 32, ragged=True, prefix=0.75, cap=50.0),
        # a step of a serving batch: a page for every sixteenth sequence or so, pages behind the window back
        "grow 256 sequences": _grow(256, 1, 8192, 16, 131072, window=4096, sinks=4),
        # long prompts arriving in an almost full pool of small pages
        "grow long prompts": _grow(16, 32768, 40000, 16, 36001),
        # four samples of each of a few chats, all layers of a small model
        "fork chats": _fork(3, 4, 1001, 4, 64, 16, 6),
        # many requests that begin with one of two long shared prompts
        "fork shared prompts": _fork(2, 64, 16384, 8, 128, 64, 4),
        # a small pool, a few pages to move
        "compact few": _compact(5, 900, 4, 64, 32, 6, 0.8),
        # a big pool half empty after many sequences have ended
        "compact half empty": _compact(64, 4000, 8, 128, 64, 2, 0.5),
    }
    return [{"name": n, **c} for n, c in named.items()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# A drawn case stays below the largest listed ones:
MOST_PAIRS = 64 * 8192 * 8192 * 128 // 2 # products of a query with a cached key
MOST_CODES = 64 * 8 * 3000 * 128         # K codes in the cache
MOST_POOL = 256 << 20                    # K codes of all layers


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "grow", "fork", "compact"])
    page = rng.choice([16, 32, 64, 128])
    if op == "grow":
        window, sinks = (0, 0) if rng.random() < 0.5 else (_log(rng, 64, 8192), rng.choice([0, 4, 100]))
        new, rows = rng.choice([1, _log(rng, 2, 16384)]), _log(rng, 1, 512)
        past = _log(rng, 1, 16384)
        while rows * (new + past) // page > 200000:
            rows = (rows + 1) // 2
        return _grow(rows, new, new + past, page, rows * (-(-(new + past) // page) + 1) + _log(rng, 1, 60000), window, sinks)
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    if op != "attention":
        layers, kv = rng.choice([1, 2, 5, 8]), _log(rng, 20, 16384)
        parents, children, rows, held = _log(rng, 1, 16), _log(rng, 1, 64), _log(rng, 1, 64), rng.uniform(0.2, 0.95)
        seqs = parents if op == "fork" else rows
        while layers * kv_heads * dim * (seqs * (kv + page) + (parents * children * page if op == "fork" else kv)) / \
                (held if op == "compact" else 1.0) > MOST_POOL:
            seqs, children, kv = (seqs + 1) // 2, (children + 1) // 2, kv if seqs > 1 else (kv + 1) // 2
            parents = min(parents, seqs)
        if op == "fork":
            return _fork(seqs, children, kv, kv_heads, dim, page, layers)
        return _compact(seqs, kv, kv_heads, dim, page, layers, held)
    q_heads = kv_heads * rng.choice([1, 3, 4, 7, 8])
    window, sinks, prefix, docs = 0, 0, 0.0, 0
    new = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 4096), _log(rng, 17, 4096)])
    seqs = _log(rng, 1, 64 if new <= 16 else 8)
    past = rng.choice([0, _log(rng, 1, 65536 if new <= 16 else 16384)])
    if rng.random() < 0.4:
        window, sinks = _log(rng, 16, 8192), rng.choice([0, 1, 4, 20])
    if rng.random() < 0.4:
        prefix = rng.uniform(0.1, 1.0)
    if rng.random() < 0.4:
        docs = _log(rng, 2, 40)
    cap, biased = rng.choice([(0.0, True), (30.0, False), (50.0, False), (20.0, True), (0.0, False)])
    while seqs * (new + past) * kv_heads * dim > MOST_CODES or seqs * new * q_heads * (new + past) * dim > MOST_PAIRS:
        seqs, new, past = (seqs + 1) // 2, (new + 1) // 2 if seqs == 1 else new, (past + 1) // 2 if seqs == 1 else past
    return _attention(rng.choice(["f16", "bf16"]), seqs, new, new + past, q_heads, kv_heads, dim, page, rng.random() < 0.6,
                      window, sinks, cap, biased, prefix, docs)


def _spread(n):
    return [(b * 0.6180339887498949 + 0.37) % 1.0 for b in range(n)]


def _lengths(c):
    """(new tokens, cached tokens) of each sequence of an attention: the case's, or spread below them."""
    if not c["ragged"]:
        return [c["new"]] * c["seqs"], [c["kv"]] * c["seqs"]
    new = [max(1, int(c["new"] * (1.0 - 0.75 * u))) for u in _spread(c["seqs"])]
    return new, [n + int((c["kv"] - c["new"]) * ((u * 7.13 + 0.11) % 1.0)) for n, u in zip(new, _spread(c["seqs"]))]


def _borders(c, length):
    """Where the documents of a sequence begin, the first at 0."""
    return [0] + sorted({max(1, int(length * u)) for u in _spread(c["docs"] - 1)} - {length}) if c["docs"] else [0]


def _sights(c):
    """Per sequence (its length, and per new token the sight: position, first of the document, last visible)."""
    out = []
    for n, m in zip(*_lengths(c)):
        borders, k, rows = _borders(c, m), 0, []
        prefix = m - n + int(n * c["prefix"]) if c["prefix"] else 0
        for p in range(m - n, m):
            while k + 1 < len(borders) and borders[k + 1] <= p:
                k += 1
            rows.append((p, borders[k], max(p, prefix - 1)))
        out.append((m, prefix, rows))
    return out


def _fork_lengths(c):
    """(parents' lengths, per child its parent and how much of it the child takes)."""
    kv = [max(1, int(c["kv"] * (1.0 - 0.3 * u))) for u in _spread(c["parents"])]
    lens = [(i // c["children"], 0) for i in range(c["parents"] * c["children"])]
    return kv, [(p, max(1, int(kv[p] * (1.0 if i % 2 else 0.4 + 0.6 * u))))
                for i, ((p, _), u) in enumerate(zip(lens, _spread(len(lens))))]


def _grow_lengths(c):
    """(lengths before the step, lengths after it, what lies before the window) per sequence."""
    after = [max(c["new"], int(c["kv"] * (1.0 - 0.6 * u))) for u in _spread(c["rows"])]
    gone = [max(0, a - c["window"]) if c["window"] else 0 for a in after]
    return [a - c["new"] for a in after], after, gone


def _pages(tokens, page):
    return -(-tokens // page)


def _table(lens, stride, page, pool, g, dev):
    """Pages of the pool dealt out in random order: block table int32 [sequences][stride]."""
    order = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), stride), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, m in enumerate(lens):
        n = _pages(m, page)
        table[b, :n] = order[at:at + n]
        at += n
    return table


def _refs(table, pool):
    """How many entries of the table hold each page."""
    flat = table.flatten().long()
    refs = torch.zeros(pool + 1, dtype=torch.int32, device=table.device)
    refs.index_add_(0, torch.where(flat >= 0, flat, pool), torch.ones_like(flat, dtype=torch.int32))
    return refs[:pool].contiguous()


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    if c["op"] == "attention":
        return _prepare_attention(c, g, dev)
    P = c["page"]
    s = {"case": c}
    if c["op"] == "grow":
        before, after, gone = _grow_lengths(c)
        s["pool"] = c["pool"]
        s["table"] = _table(before, max(_pages(a, P) for a in after), P, c["pool"], g, dev)
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731
        s["rows"], s["before"], s["all"] = ints(list(range(c["rows"]))), ints(before), ints([ALL] * c["rows"])
        s["first"], s["gone"], s["lens"] = ints([c["sinks"]] * c["rows"]), ints(gone), ints(after)
        s["moves"] = torch.zeros(1, 2, dtype=torch.int32, device=dev)
        s["refs"] = _refs(s["table"], s["pool"])
        return s
    if c["op"] == "fork":
        kv, forks = _fork_lengths(c)
        rows, used = kv + [0] * len(forks), sum(_pages(m, P) for m in kv)
        s["pool"] = used + len(forks) + 5
        s["moves"] = torch.zeros(len(forks) + 1, 2, dtype=torch.int32, device=dev)
        s["parents"] = torch.tensor([p for p, _ in forks], dtype=torch.int32, device=dev)
        s["children"] = torch.arange(len(kv), len(rows), dtype=torch.int32, device=dev)
        s["lens"] = torch.tensor([n for _, n in forks], dtype=torch.int32, device=dev)
        s["table"] = _table(rows, _pages(max(kv), P) + 3, P, s["pool"], g, dev)
        s["refs"] = _refs(s["table"], s["pool"])
    else:
        rows = [max(1, int(c["kv"] * (1.0 - 0.5 * u))) for u in _spread(c["rows"])]
        used = sum(_pages(m, P) for m in rows)
        s["pool"] = int(used / c["held"]) + 4
        s["pool"] -= s["pool"] % 4                                            # (the book's two arrays lie in one)
        s["most"] = s["pool"] // 2
        s["moves"] = torch.zeros(s["most"] + 1, 2, dtype=torch.int32, device=dev)
        table = _table(rows, _pages(max(rows), P), P, s["pool"], g, dev)
        s["book"] = torch.cat([_refs(table, s["pool"]), table.flatten()])
        s["now"] = s["book"].clone()
        s["refs"], s["table"] = s["now"][:s["pool"]], s["now"][s["pool"]:].view(table.shape)
    # One page more than the pool has, for nothing to be copied to itself
    N, H, D = s["pool"] + 1, c["kv_heads"], c["dim"]
    s["layers"] = []
    for _ in range(c["layers"]):
        codes = [torch.randint(-127, 128, shape, generator=g, device=dev, dtype=torch.int8) for shape in ((N, H, P, D), (N, H, D, P))]
        s["layers"].append((*codes, torch.rand(N, H, 2, generator=g, device=dev).mul_(0.02).add_(0.005)))
    return s


def _prepare_attention(c, g, dev):
    dt = TYPES[c["dtype"]]
    P, D, Hq, Hk = c["page"], c["dim"], c["q_heads"], c["kv_heads"]
    new, kv = _lengths(c)
    T = sum(new)
    used = sum(_pages(k, P) for k in kv)
    pages = used + 1                      # the pool's last page is not handed out
    table = _table(kv, max(_pages(k, P) for k in kv), P, used, g, dev)
    # Keys and values of earlier steps: normal, a few key dimensions several times larger, codes with a scale for each
    # page and head.  Queries whose scores have to be capped are several times larger too.
    gain = 1.0 + 5.0 * (torch.rand(Hk, D, generator=g, device=dev) < 0.03)
    k = torch.randn(pages, Hk, P, D, generator=g, device=dev).mul_(gain[None, :, None, :])
    scales = torch.empty(pages, Hk, 2, device=dev)
    scales[..., 0] = k.abs().amax(dim=(2, 3)) / 127
    k_codes = k.div_(scales[..., 0, None, None]).round_().to(torch.int8)
    del k
    v = torch.randn(pages, Hk, D, P, generator=g, device=dev)
    scales[..., 1] = v.abs().amax(dim=(2, 3)) / 127
    v_codes = v.div_(scales[..., 1, None, None]).round_().to(torch.int8)
    del v
    sights = _sights(c)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)          # noqa: E731
    return {"case": c, "T": T, "k_codes": k_codes, "v_codes": v_codes, "scales": scales, "table": table,
            "offsets": ints([0] + new).cumsum(0).to(torch.int32), "kv_lens": ints(kv), "max_new": max(new), "max_kv": max(kv),
            "q": torch.randn(T, Hq, D, generator=g, device=dev).mul_(6.0 if c["cap"] else 1.0).to(dt),
            "scale": 1.0 / math.sqrt(D), "y": torch.empty(T, Hq, D, dtype=dt, device=dev),
            "slopes": torch.tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)], device=dev) if c["biased"] else None,
            "prefix": ints([prefix for _, prefix, _ in sights]) if c["prefix"] else None,
            "starts": ints([lo for _, _, rows in sights for _, lo, _ in rows]) if c["docs"] else None}


def run(state):
    s = state
    op = s["case"]["op"]
    if op == "attention":
        return _own_attention(s) if own else _plain_attention(s)
    if op == "compact":
        s["now"].copy_(s["book"])         # the pool as the ended sequences left it
    if own:
        return {"grow": _own_grow, "fork": _own_fork, "compact": _own_compact}[op](s)
    return {"grow": _plain_grow, "fork": _plain_fork, "compact": _plain_compact}[op](s)


# ---------------------------------------------------------------------------
# the library's entry points

def _handles(s):
    """The descriptors and the workspace that a serving program keeps with its caches, book and batch."""
    from quantized_linear_layers_packed_amd import qlin
    c = s["case"]
    s["handles"] = h = {"qlin": qlin}
    if c["op"] != "attention":
        h["book"] = qlin.Kv8Book(s["refs"], s["table"], c["page"])
        if c["op"] != "grow":
            h["caches"] = qlin.Kv8Caches([qlin.Kv8Cache(*layer) for layer in s["layers"]])
        return h
    h["cache"] = cache = qlin.Kv8Cache(s["k_codes"], s["v_codes"], s["scales"])
    h["batch"] = batch = qlin.Kv8Batch(s["offsets"], s["kv_lens"], s["table"], s["T"], s["max_new"], s["max_kv"])
    h["scoring"] = qlin.Kv8Scoring(c["cap"], s["slopes"], s["prefix"], s["starts"])
    h["dtype"] = qlin.QLIN_F16 if c["dtype"] == "f16" else qlin.QLIN_BF16
    need = qlin.qlin_kv8_attention_workspace_bytes(cache, batch, c["q_heads"], c["window"], c["sinks"])
    h["workspace"] = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
    return h


def _own_attention(s):
    h = s.get("handles") or _handles(s)
    c = s["case"]
    h["qlin"].qlin_kv8_attention_scored(h["cache"], h["batch"], s["q"], h["dtype"], c["q_heads"], s["scale"], c["window"],
                                        c["sinks"], h["scoring"], s["y"], h["workspace"])
    return s["y"]


def _book(s):
    return {"table": s["table"], "refs": s["refs"], "moves": s["moves"]}


def _own_grow(s):
    h = s.get("handles") or _handles(s)
    qlin, book = h["qlin"], h["book"]
    qlin.qlin_kv8_free(book, s["rows"], s["before"], s["all"])
    if s["case"]["window"]:
        qlin.qlin_kv8_free(book, s["rows"], s["first"], s["gone"])
    qlin.qlin_kv8_grow(book, s["lens"], s["moves"])
    return _book(s)


def _own_fork(s):
    h = s.get("handles") or _handles(s)
    qlin, book = h["qlin"], h["book"]
    qlin.qlin_kv8_free(book, s["children"])
    qlin.qlin_kv8_fork(book, s["parents"], s["children"], s["lens"], s["moves"])
    qlin.qlin_kv8_copy_pages(h["caches"], h["caches"], s["moves"])
    return {**_book(s), "layers": s["layers"]}


def _own_compact(s):
    h = s.get("handles") or _handles(s)
    qlin = h["qlin"]
    qlin.qlin_kv8_compact(h["book"], s["moves"])
    qlin.qlin_kv8_copy_pages(h["caches"], h["caches"], s["moves"])
    return {**_book(s), "layers": s["layers"]}


# ---------------------------------------------------------------------------
# plain forms

def _plain_attention(s):
    c = s["case"]
    dt = TYPES[c["dtype"]]
    T, P, D, Hq, Hk = s["T"], c["page"], c["dim"], c["q_heads"], c["kv_heads"]
    G, B = Hq // Hk, c["seqs"]
    off, kv = s["offsets"].long(), s["kv_lens"].long()
    n = off[1:] - off[:-1]
    N, L = s["max_new"], s["table"].shape[1] * P
    table = s["table"].long().clamp(min=0)
    k = s["k_codes"][table].float().mul_(s["scales"][table][..., 0, None, None])           # [B][pages][Hk][P][D]
    k = k.transpose(1, 2).reshape(B, Hk, L, D)
    v = s["v_codes"][table].float().mul_(s["scales"][table][..., 1, None, None])           # [B][pages][Hk][D][P]
    v = v.permute(0, 2, 1, 4, 3).reshape(B, Hk, L, D)
    row = torch.arange(N, device=off.device)
    token = (off[:-1, None] + row).clamp(max=T - 1)                                        # [B][N]
    q = s["q"][token].float()                                                              # [B][N][Hq][D]
    q = q.view(B, N, Hk, G, D).transpose(1, 2).reshape(B, Hk, N * G, D)
    w = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(B, Hk, N, G, L)
    at = (kv - n)[:, None, None] + row[None, :, None]                                      # positions [B][N][1]
    j = torch.arange(L, device=off.device)
    if c["cap"]:
        w.div_(c["cap"]).tanh_().mul_(c["cap"])
    if c["biased"]:
        distance = (at - j).abs().float()                                                  # [B][N][L]
        w -= s["slopes"].view(Hk, 1, G, 1) * distance[:, None, :, None]
    seen = j <= at
    if c["prefix"]:
        seen = seen | (j < s["prefix"][:, None, None])
    start = s["starts"][token][:, :, None] if c["docs"] else torch.zeros_like(at)
    if c["window"]:
        seen &= (j > at - c["window"]) | (j < start + c["sinks"])
    seen &= (j >= start) & (j < kv[:, None, None])
    w = w.masked_fill_(~seen[:, None, :, None], -math.inf)
    w = w.sub_(w.amax(dim=-1, keepdim=True)).exp_().view(B, Hk, N * G, L)
    o = torch.matmul(w, v) / w.sum(dim=-1, keepdim=True)
    o = o.view(B, Hk, N, G, D).transpose(1, 2).reshape(B * N, Hq, D)
    tok = torch.arange(T, device=off.device)
    seq = torch.searchsorted(off[1:], tok, right=True)
    return o[seq * N + tok - off[seq]].to(dt)


def _count(refs, pages, by):
    """refs[page] += by for every page of `pages` that is not below 0."""
    flat = pages.flatten().long()
    refs.index_add_(0, flat.clamp(min=0), torch.where(flat >= 0, by, 0).to(torch.int32))


def _plain_free(s, rows, begin, end):
    """Entries of the rows whose tokens all lie in begin .. end-1 go back to the pool."""
    P, table = s["case"]["page"], s["table"]
    first = torch.arange(table.shape[1], device=table.device) * P
    mine = table[rows.long()]
    back = (first >= begin[:, None]) & (first + P <= end[:, None])
    _count(s["refs"], torch.where(back, mine, -1), -1)
    table[rows.long()] = torch.where(back, -1, mine)


def _free_pages(refs):
    """The free pages in ascending order (the others behind them), and how many there are."""
    free = refs == 0
    rank = torch.where(free, free.cumsum(0) - 1, free.sum() + (~free).cumsum(0) - 1)
    order = torch.empty(len(refs), dtype=torch.int32, device=refs.device)
    order[rank] = torch.arange(len(refs), dtype=torch.int32, device=refs.device)
    return order, free.sum()


def _take(s, wanted):
    """Pages for the wanted places (truth values) in their order, -1 elsewhere or if they do not suffice; updates refs and
    the first pair of the moves."""
    order, free = _free_pages(s["refs"])
    flat = wanted.flatten()
    total = flat.sum()
    enough = total <= free
    pages = order[(flat.cumsum(0) - 1).clamp(min=0, max=len(order) - 1)]
    pages = torch.where(flat & enough, pages, -1)
    _count(s["refs"], pages, 1)
    s["moves"][0, 0] = torch.where(enough, total, 0)
    s["moves"][0, 1] = (total - free).clamp(min=0)
    return pages.view(wanted.shape)


def _plain_grow(s):
    c, table = s["case"], s["table"]
    _plain_free(s, s["rows"], s["before"], s["all"])
    if c["window"]:
        _plain_free(s, s["rows"], s["first"], s["gone"])
    entry = torch.arange(table.shape[1], device=table.device)
    want = ((s["lens"] + c["page"] - 1) // c["page"])[:, None]
    last = torch.where((table >= 0) & (entry < want), entry, -1).amax(dim=1, keepdim=True)
    wanted = (entry > last) & (entry < want)
    pages = _take(s, wanted)
    table.copy_(torch.where(pages >= 0, pages, table))
    return _book(s)


def _plain_copy(s, src, dst):
    """Pages src to dst, those below 0 the spare page to itself."""
    src, dst = (torch.where(x >= 0, x, s["pool"]).long() for x in (src, dst))
    for layer in s["layers"]:
        for x in layer:
            x[dst] = x[src]


def _plain_fork(s):
    P, table = s["case"]["page"], s["table"]
    all_of = torch.zeros_like(s["children"])
    _plain_free(s, s["children"], all_of, all_of + ALL)
    entry = torch.arange(table.shape[1], device=table.device)
    theirs = table[s["parents"].long()]
    full = s["lens"] // P
    shared = torch.where(entry < full[:, None], theirs, -1)
    src = theirs.gather(1, full.long()[:, None])[:, 0]
    split = (s["lens"] % P > 0) & (src >= 0)
    dst = _take(s, split)
    src = torch.where(split, src, -1)
    _count(s["refs"], shared, 1)
    table[s["children"].long()] = torch.where(entry == full[:, None], dst[:, None], shared)
    s["moves"][0, 0] = len(src)           # a pair for every child, -1 where nothing is to be copied
    s["moves"][1:, 0], s["moves"][1:, 1] = src, dst
    _plain_copy(s, src, dst)
    return {**_book(s), "layers": s["layers"]}


def _plain_compact(s):
    refs, table, most = s["refs"], s["table"], s["most"]
    N = len(refs)
    page = torch.arange(N, dtype=torch.int32, device=refs.device)
    free = refs == 0
    dst = _free_pages(refs)[0][:most]                                                      # the lowest free ones
    last = N - 1 - _free_pages(free.flip(0).to(torch.int32))[0][:most]                      # the highest used ones
    i = torch.arange(len(dst), device=refs.device)
    moved = (i < free.sum()) & (i < N - free.sum()) & (last > dst)
    src, dst = torch.where(moved, last, -1), torch.where(moved, dst, -1)
    to = torch.cat([page, page.new_full((1,), -1)])                                        # where each page goes; entry -1 stays
    at = torch.where(moved, src, N).long()
    to[at] = torch.where(moved, dst, -1)
    table.copy_(to[table.long()])
    refs.copy_(torch.zeros(N + 1, dtype=torch.int32, device=refs.device).index_add_(
        0, to[:N].long(), refs)[:N])
    s["moves"][0, 0], s["moves"][0, 1] = moved.sum(), 0
    s["moves"][1:, 0], s["moves"][1:, 1] = src, dst
    _plain_copy(s, src, dst)
    return {**_book(s), "layers": s["layers"]}


# ---------------------------------------------------------------------------
# work and 64-bit values

def _page_bytes(c):
    return c["kv_heads"] * (2 * c["page"] * c["dim"] + 8) * c["layers"]


def work(case):
    c = case
    P = c["page"]
    if c["op"] == "grow":
        before, after, gone = _grow_lengths(c)
        entries = sum(_pages(a, P) - _pages(b, P) for a, b in zip(after, before))
        return {"bytes": 4 * (3 * entries + 2 * c["rows"]), "flops": entries}               # a free count found and set, an entry
    if c["op"] == "fork":
        _, forks = _fork_lengths(c)
        entries = sum(_pages(n, P) for _, n in forks)
        splits = sum(n % P > 0 for _, n in forks)
        return {"bytes": 4 * 4 * entries + 8 * splits + 2 * splits * _page_bytes(c), "flops": entries}
    if c["op"] == "compact":
        rows = [max(1, int(c["kv"] * (1.0 - 0.5 * u))) for u in _spread(c["rows"])]
        used = sum(_pages(m, P) for m in rows)
        moved = int(used * (1.0 - c["held"]))                                              # expected of a random order
        pool = int(used / c["held"])
        return {"bytes": 4 * (2 * pool + 2 * used) + 8 * moved + 2 * moved * _page_bytes(c), "flops": pool + used}
    D, Hq, Hk = c["dim"], c["q_heads"], c["kv_heads"]
    pairs = tokens = T = 0
    for m, _, rows in _sights(c):
        edge = [0] * (m + 1)                                                               # where sights begin and end
        for p, lo, hi in rows:
            first = max(lo, p - c["window"] + 1) if c["window"] else lo
            kept = min(c["sinks"], first - lo)
            pairs += hi + 1 - first + kept
            edge[first] += 1
            edge[hi + 1] -= 1
            if kept:
                edge[lo] += 1
                edge[lo + kept] -= 1
        T += len(rows)
        depth = 0
        for e in edge[:-1]:
            depth += e
            tokens += depth > 0
    return {"bytes": 2 * T * Hq * D * 2 + tokens * Hk * 2 * D + (tokens // P + c["seqs"]) * Hk * 8,
            "flops": 4 * D * Hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "grow": _exact_grow, "fork": _exact_fork, "compact": _exact_compact}[case["op"]](s)


def _exact_attention(s):
    """One sequence, one key/value head and up to 1024 queries at a time in fp64."""
    c = s["case"]
    Hq, Hk = c["q_heads"], c["kv_heads"]
    G = Hq // Hk
    y = torch.empty(s["T"], Hq, c["dim"], dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (m, _, rows) in enumerate(_sights(c)):
        pages = s["table"][b, :_pages(m, c["page"])].long()
        key_at = torch.arange(m, device=y.device)
        sight = torch.tensor(rows, device=y.device)
        for h in range(Hk):
            k = (s["k_codes"][pages, h].double() * s["scales"][pages, h, 0].double()[:, None, None]).flatten(0, 1)[:m]
            v = (s["v_codes"][pages, h].double() * s["scales"][pages, h, 1].double()[:, None, None])
            v = v.transpose(1, 2).flatten(0, 1)[:m]
            for i in range(0, len(rows), 1024):
                where, lo, hi = (x[:, None] for x in sight[i:i + 1024].unbind(1))
                n = len(where)
                q = s["q"][at + i:at + i + n, h * G:(h + 1) * G].double()
                hidden = (key_at > hi) | (key_at < lo)
                if c["window"]:
                    hidden |= (where - key_at >= c["window"]) & (key_at - lo >= c["sinks"])
                logits = (q.flatten(0, 1) @ k.T).view(n, G, m) * s["scale"]
                if c["cap"]:
                    logits = c["cap"] * torch.tanh(logits / c["cap"])
                if c["biased"]:
                    slope = s["slopes"][h * G:(h + 1) * G].double()
                    logits = logits - slope[None, :, None] * (where - key_at).abs()[:, None].double()
                weights = torch.softmax(logits.masked_fill(hidden[:, None], -math.inf), dim=-1)
                y[at + i:at + i + n, h * G:(h + 1) * G] = (weights.flatten(0, 1) @ v).view(n, G, -1)
        at += len(rows)
    return y


def _device_book(s, table, moves):
    """The book of a table given as lists, as tensors."""
    refs = [0] * s["pool"]
    for row in table:
        for p in row:
            if p >= 0:
                refs[p] += 1
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=s["table"].device)   # noqa: E731
    return {"table": ints(table), "refs": ints(refs), "moves": ints(moves)}


def _unused(s, table):
    held = {p for row in table for p in row}
    return [p for p in range(s["pool"]) if p not in held]


def _exact_grow(s):
    c, P = s["case"], s["case"]["page"]
    before, after, gone = _grow_lengths(c)
    table = s["table"].tolist()
    for row, g in zip(table, gone):
        for e in range(_pages(c["sinks"], P), g // P):
            row[e] = -1
    unused = _unused(s, table)
    at = 0
    for row, b, a in zip(table, before, after):
        held = [e for e in range(_pages(b, P)) if row[e] >= 0]
        for e in range(held[-1] + 1 if held else 0, _pages(a, P)):
            row[e] = unused[at]
            at += 1
    return _device_book(s, table, [[at, 0]])


def _copied(s, moves):
    layers = []
    for layer in s["layers"]:
        layers.append(tuple(x.clone() for x in layer))
        for src, dst in moves:
            if src >= 0:
                for to, x in zip(layers[-1], layer):
                    to[dst] = x[src]
    return layers


def _exact_fork(s):
    P, table = s["case"]["page"], s["table"].tolist()
    kv, forks = _fork_lengths(s["case"])
    unused, moves = _unused(s, table), []
    for i, (parent, n) in enumerate(forks):
        row = table[parent][:n // P]
        if n % P:
            moves.append([table[parent][n // P], unused.pop(0)])
            row.append(moves[-1][1])
        else:
            moves.append([-1, -1])
        table[len(kv) + i] = row + [-1] * (len(table[0]) - len(row))
    return {**_device_book(s, table, [[len(moves), 0]] + moves), "layers": _copied(s, moves)}


def _exact_compact(s):
    table = s["table"].tolist()
    unused = _unused(s, table)
    used = sorted({p for row in table for p in row if p >= 0}, reverse=True)
    moves = [[src, dst] for src, dst in zip(used, unused) if src > dst][:s["most"]]
    to = dict(moves)
    table = [[to.get(p, p) for p in row] for row in table]
    pad = [[-1, -1]] * (s["most"] - len(moves))
    return {**_device_book(s, table, [[len(moves), 0]] + moves + pad), "layers": _copied(s, moves)}
