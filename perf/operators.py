"""Measured cases of the 8-bit paged key/value cache: appending with the position
rotation, and the attention that reads it.

Two operators, each in a plain form (elementary torch operations in fp32) and,
where ``own`` is true, through the library's entry points:

* ``append``     rotate the new queries and keys, quantize the new keys and values
                 into the pages of their sequences (one scale for each page and
                 head, grown in place), and read the touched pages back in 16 bits
                 (so the outputs are the values that the cache now stands for).
* ``attention``  softmax(scale Q K^T + mask) V over the cached tokens, causal, with
                 an optional sliding window and first tokens that stay visible.

The cache is K codes int8 [page][kv head][slot][dim], V codes int8
[page][kv head][dim][slot] and fp32 scales [page][kv head][K, V]; a batch is
ragged: sequence b owns the new tokens offsets[b] .. offsets[b+1]-1, which are the
last ones of its kv_lens[b] cached tokens, and its pages are block_table[b].
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
BASE = 10000.0          # rotation frequencies BASE^(-2i / rot)


def _case(op, dtype, seqs, new, kv, q_heads, kv_heads, dim, page, ragged=False, window=0, sinks=0, rot=0, style="half"):
    return {"op": op, "dtype": dtype, "seqs": seqs, "new": new, "kv": kv, "q_heads": q_heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "ragged": ragged, "window": window, "sinks": sinks, "rot": rot, "style": style}


def listed():
    named = {
        # one user's next token: pure latency (a 4096-wide layer, 8 key/value heads)
        "append 1 token": _case("append", "f16", 1, 1, 1001, 32, 8, 128, 64, rot=128),
        # a serving batch, one token each at ragged lengths, most into half-filled pages (an 8192-wide layer)
        "append 64 sequences": _case("append", "bf16", 64, 1, 4096, 64, 8, 128, 64, ragged=True, rot=128),
        # ragged prompts behind cached prefixes of odd length, half the dimensions rotated in neighbouring pairs
        "append prompts": _case("append", "f16", 4, 4096, 5003, 64, 8, 128, 32, ragged=True, rot=64, style="pairs"),
        # one user's next token over a short chat, every head with its own keys (a 4096-wide layer)
        "decode short": _case("attention", "f16", 1, 1, 777, 32, 32, 128, 16),
        # one user's next token over a very long document
        "decode long": _case("attention", "bf16", 1, 1, 131072, 64, 8, 128, 64),
        # a full serving batch at ragged lengths
        "decode 64 sequences": _case("attention", "f16", 64, 1, 8192, 64, 8, 128, 64, ragged=True),
        # a 6656-wide layer (52 heads of 128) without shared heads
        "decode 52 heads": _case("attention", "bf16", 16, 1, 2048, 52, 52, 128, 32, ragged=True),
        # five draft tokens to verify, sliding window with first tokens kept, narrow heads
        "verify window sinks": _case("attention", "f16", 32, 5, 32768, 32, 4, 64, 128, ragged=True, window=4096, sinks=4),
        # a whole prompt (an 8192-wide layer)
        "prompt 8192": _case("attention", "f16", 1, 8192, 8192, 64, 8, 128, 64),
        # a chunk of a long prompt over what is cached already
        "chunk of long prompt": _case("attention", "bf16", 1, 512, 32768, 64, 8, 128, 128),
        # ragged prompts under a window, wide heads
        "prompts window sinks": _case("attention", "bf16", 8, 2048, 2500, 16, 4, 256, 32, ragged=True, window=1024, sinks=4),
        # short odd prompts of a small model
        "prompts short": _case("attention", "f16", 3, 333, 401, 12, 4, 64, 16, ragged=True),
    }
    return [{"name": n, **c} for n, c in named.items()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# A drawn case stays below the largest listed ones:
MOST_PAIRS = 64 * 8192 * 8192 * 128 // 2 # products of a query with a cached key
MOST_CODES = 64 * 8 * 3000 * 128         # K codes in the cache
MOST_BYTES = 200 << 20                   # what an append takes in and gives out


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "attention"])
    dtype = rng.choice(["f16", "bf16"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    q_heads = kv_heads * rng.choice([1, 3, 4, 7, 8])
    ragged = rng.random() < 0.6
    window, sinks, rot, style = 0, 0, 0, "half"
    if op == "append":
        new = rng.choice([1, _log(rng, 2, 4096)])
        seqs = _log(rng, 1, 128 if new == 1 else max(1, 16384 // new))
        past = _log(rng, 1, 4096)
        rot, style = rng.choice([dim, dim // 2, 16]), rng.choice(["half", "pairs"])
    else:
        new = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 4096)])
        seqs = _log(rng, 1, 64 if new <= 16 else 8)
        past = _log(rng, 1, 65536 if new <= 16 else 16384)
        if rng.random() < 0.4:
            window, sinks = _log(rng, 16, 8192), rng.choice([0, 1, 4, 20])
    while seqs * (new + past) * kv_heads * dim > MOST_CODES or \
            (seqs * new * (q_heads + kv_heads) * dim * 4 > MOST_BYTES if op == "append"
             else seqs * new * q_heads * (new + past) * dim > MOST_PAIRS):
        seqs, new, past = (seqs + 1) // 2, (new + 1) // 2 if seqs == 1 else new, (past + 1) // 2 if seqs == 1 else past
    return _case(op, dtype, seqs, new, new + past, q_heads, kv_heads, dim, page, ragged, window, sinks, rot, style)


def _lengths(c):
    """(new tokens, cached tokens) of each sequence: the case's, or spread below them."""
    if not c["ragged"]:
        return [c["new"]] * c["seqs"], [c["kv"]] * c["seqs"]
    spread = [(b * 0.6180339887498949 + 0.37) % 1.0 for b in range(c["seqs"])]
    new = [max(1, int(c["new"] * (1.0 - 0.75 * u))) for u in spread]
    return new, [n + int((c["kv"] - c["new"]) * ((u * 7.13 + 0.11) % 1.0)) for n, u in zip(new, spread)]


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = TYPES[c["dtype"]]
    B, P, D, Hq, Hk = c["seqs"], c["page"], c["dim"], c["q_heads"], c["kv_heads"]
    new, kv = _lengths(c)
    T = sum(new)
    table_pages = max(-(-k // P) for k in kv)
    used = sum(-(-k // P) for k in kv)
    pages = used + 1                      # the pool's last page is not handed out
    order = torch.randperm(used, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, table_pages), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(kv):
        n = -(-k // P)
        table[b, :n] = order[at:at + n]
        at += n
    # Cached keys and values of earlier steps: normal, a few key dimensions several times larger, codes with a scale
    # for each page and head.
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
    s = {"case": c, "T": T, "pages": pages, "k_codes": k_codes, "v_codes": v_codes, "scales": scales, "table": table,
         "offsets": torch.tensor([0] + new, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32),
         "kv_lens": torch.tensor(kv, dtype=torch.int32, device=dev), "max_new": max(new), "max_kv": max(kv)}
    if c["op"] == "append":
        qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g, device=dev)          # the fused projection's output
        qkv[:, Hq:Hq + Hk] *= gain
        s["qkv"] = qkv.to(dt)
        pos = torch.arange(max(kv), device=dev, dtype=torch.float64)
        freq = BASE ** (-2.0 * torch.arange(c["rot"] // 2, device=dev, dtype=torch.float64) / c["rot"])
        s["cos"] = (pos[:, None] * freq).cos().float().contiguous()
        s["sin"] = (pos[:, None] * freq).sin().float().contiguous()
        # The read-back covers the touched pages: from the first slot of the page that the first new token falls into.
        back = [n + (k - n) % P for n, k in zip(new, kv)]
        s["back"] = sum(back)
        s["max_back"] = max(back)
        s["back_offsets"] = torch.tensor([0] + back, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
        s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
        s["k_out"] = torch.empty(s["back"], Hk, D, dtype=dt, device=dev)
        s["v_out"] = torch.empty(s["back"], Hk, D, dtype=dt, device=dev)
    else:
        s["q"] = torch.randn(T, Hq, D, generator=g, device=dev).to(dt)
        s["scale"] = 1.0 / math.sqrt(D)
        s["y"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
    return s


def run(state):
    if own:
        return _own_append(state) if state["case"]["op"] == "append" else _own_attention(state)
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_attention(state)


# ---------------------------------------------------------------------------
# the library's entry points

def _handles(s):
    """The descriptors and the workspace that a serving program keeps with its cache and batch."""
    from quantized_linear_layers_packed_amd import qlin
    c = s["case"]
    cache = qlin.Kv8Cache(s["k_codes"], s["v_codes"], s["scales"])
    batch = qlin.Kv8Batch(s["offsets"], s["kv_lens"], s["table"], s["T"], s["max_new"], s["max_kv"])
    s["handles"] = h = {"qlin": qlin, "cache": cache, "batch": batch,
                        "dtype": qlin.QLIN_F16 if c["dtype"] == "f16" else qlin.QLIN_BF16}
    if c["op"] == "append":
        h["back"] = qlin.Kv8Batch(s["back_offsets"], s["kv_lens"], s["table"], s["back"], s["max_back"], s["max_kv"])
        h["style"] = qlin.QLIN_ROPE_HALF if c["style"] == "half" else qlin.QLIN_ROPE_PAIRS
    else:
        need = qlin.qlin_kv8_attention_workspace_bytes(cache, batch, c["q_heads"], c["window"], c["sinks"])
        h["workspace"] = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
    return h


def _own_append(s):
    h = s.get("handles") or _handles(s)
    c, qlin, qkv = s["case"], h["qlin"], s["qkv"]
    Hq, Hk = c["q_heads"], c["kv_heads"]
    qlin.qlin_kv8_append(h["cache"], h["batch"], qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], h["dtype"], Hq,
                         s["cos"], s["sin"], c["rot"], h["style"], s["q_out"])
    qlin.qlin_kv8_gather(h["cache"], h["back"], s["k_out"], s["v_out"], h["dtype"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_attention(s):
    h = s.get("handles") or _handles(s)
    c = s["case"]
    h["qlin"].qlin_kv8_attention(h["cache"], h["batch"], s["q"], h["dtype"], c["q_heads"], s["scale"], c["window"],
                                 c["sinks"], s["y"], h["workspace"])
    return s["y"]


# ---------------------------------------------------------------------------
# plain forms

def _rotate(x, cos, sin, rot, style):
    """x fp32 [T][H][D], cos / sin [T][1][rot/2]: the first rot dimensions rotated in pairs."""
    out = x.clone()
    if style == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2] = a * cos - b * sin
        out[..., rot // 2:rot] = b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2] = a * cos - b * sin
        out[..., 1:rot:2] = b * cos + a * sin
    return out


def _plain_append(s):
    c = s["case"]
    dt = TYPES[c["dtype"]]
    T, P, Hq, Hk = s["T"], c["page"], c["q_heads"], c["kv_heads"]
    off, kv = s["offsets"].long(), s["kv_lens"].long()
    n = off[1:] - off[:-1]
    start = kv - n
    tok = torch.arange(T, device=off.device)
    seq = torch.searchsorted(off[1:], tok, right=True)
    pos = tok - off[seq] + start[seq]
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    x = s["qkv"].float()
    q = _rotate(x[:, :Hq], cos, sin, c["rot"], c["style"])
    k = _rotate(x[:, Hq:Hq + Hk], cos, sin, c["rot"], c["style"])
    v = x[:, Hq + Hk:]
    # the touched pages: the J pages from each sequence's first one, of which those past its end go to the spare page
    J = (s["max_new"] + 2 * P - 2) // P
    index = start[:, None] // P + torch.arange(J, device=off.device)                       # [B][J]
    touched = index * P < kv[:, None]
    page = s["table"].gather(1, index.clamp(max=s["table"].shape[1] - 1)).long()
    page = torch.where(touched, page, s["pages"] - 1)
    at = index[..., None] * P + torch.arange(P, device=off.device)                         # positions [B][J][P]
    is_new = (at >= start[:, None, None]) & (at < kv[:, None, None])
    is_old = at < start[:, None, None]
    src = (off[:-1, None, None] + at - start[:, None, None]).clamp(0, T - 1)
    some_old = (is_old.any(-1) & touched)[..., None]

    def store(fresh, codes, which):
        """fresh [T][H][D] into codes [page][H][P][D]; the touched pages' values [B][J][P][H][D]."""
        x = fresh[src] * is_new[..., None, None]
        s_old = s["scales"][page][..., which]                                              # [B][J][H]
        s_new = torch.maximum(x.abs().amax(dim=(2, 4)) / 127, torch.where(some_old, s_old, 0.0))
        inv = torch.where(s_new > 0, 1.0 / s_new, 0.0)
        codes_new = (x * inv[:, :, None, :, None]).round().clamp(-127, 127)
        old = codes[page].permute(0, 1, 3, 2, 4).float()                                   # [B][J][P][H][D]
        codes_old = (old * (s_old * inv)[:, :, None, :, None]).round().clamp(-127, 127)
        q = torch.where(is_new[..., None, None], codes_new, torch.where(is_old[..., None, None], codes_old, old))
        codes[page] = q.permute(0, 1, 3, 2, 4).to(torch.int8)
        s["scales"][page.reshape(-1), :, which] = s_new.reshape(-1, s_new.shape[-1])
        return q * s_new[:, :, None, :, None]

    ks = store(k, s["k_codes"], 0)
    vs = store(v, s["v_codes"].transpose(2, 3), 1)
    boff = s["back_offsets"].long()
    tok = torch.arange(s["back"], device=off.device)
    seq = torch.searchsorted(boff[1:], tok, right=True)
    where = (seq * J * P) + tok - boff[seq]
    return {"q": q.to(dt), "k": ks.flatten(0, 2)[where].to(dt), "v": vs.flatten(0, 2)[where].to(dt)}


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
    q = s["q"][(off[:-1, None] + row).clamp(max=T - 1)].float()                            # [B][N][Hq][D]
    q = q.view(B, N, Hk, G, D).transpose(1, 2).reshape(B, Hk, N * G, D)
    w = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    at = (kv - n)[:, None, None] + row[None, :, None]                                      # positions [B][N][1]
    j = torch.arange(L, device=off.device)
    seen = j <= at
    if c["window"]:
        seen &= (j > at - c["window"]) | (j < c["sinks"])
    seen = seen[:, None].repeat_interleave(G, dim=2)                                       # [B][1][N G][L]
    w = w.masked_fill_(~seen, -math.inf)
    w = w.sub_(w.amax(dim=-1, keepdim=True)).exp_()
    o = torch.matmul(w, v) / w.sum(dim=-1, keepdim=True)
    o = o.view(B, Hk, N, G, D).transpose(1, 2).reshape(B * N, Hq, D)
    tok = torch.arange(T, device=off.device)
    seq = torch.searchsorted(off[1:], tok, right=True)
    return o[seq * N + tok - off[seq]].to(dt)


# ---------------------------------------------------------------------------
# work and 64-bit values

def _visible(c, n, kv):
    """(visible pairs, cached tokens seen by any query) of one sequence."""
    W, S = c["window"] or kv, c["sinks"]
    hidden = [max(0, p - W + 1) for p in range(kv - n, kv)]                                # tokens before the window
    return sum(p + 1 - lo + min(S, lo) for p, lo in zip(range(kv - n, kv), hidden)), kv - hidden[0] + min(S, hidden[0])


def work(case):
    c = case
    P, D, Hq, Hk = c["page"], c["dim"], c["q_heads"], c["kv_heads"]
    new, kv = _lengths(c)
    T = sum(new)
    if c["op"] == "append":
        old = sum((k - n) % P for n, k in zip(new, kv))                                    # earlier tokens of touched pages
        pages = sum(-(-k // P) - (k - n) // P for n, k in zip(new, kv))
        back = T + old
        size = T * (2 * Hq + 2 * Hk) * D * 2                                               # queries in and out, keys and values in
        size += 2 * (T + old) * Hk * D + pages * Hk * 8                                    # codes written or read, scales
        size += 2 * back * Hk * D * 2                                                      # values out
        return {"bytes": size, "flops": T * (Hq + Hk) * c["rot"] * 3 + T * 2 * Hk * D * 4 + back * 2 * Hk * D}
    pairs = tokens = 0
    for n, k in zip(new, kv):
        p, t = _visible(c, n, k)
        pairs, tokens = pairs + p, tokens + t
    return {"bytes": 2 * T * Hq * D * 2 + tokens * Hk * 2 * D + (tokens // P + c["seqs"]) * Hk * 8,
            "flops": 4 * D * Hq * pairs}


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    return _exact_append(s) if c["op"] == "append" else _exact_attention(s)


def _exact_append(s):
    """Sequence by sequence, page by page in fp64."""
    c = s["case"]
    P, Hq, Hk = c["page"], c["q_heads"], c["kv_heads"]
    new, kv = _lengths(c)
    half = c["rot"] // 2
    table = s["table"].tolist()
    qs, outs, at = [], ([], []), 0
    for b, (n, m) in enumerate(zip(new, kv)):
        x = s["qkv"][at:at + n].double()
        at += n
        first = m - n
        turn = torch.complex(s["cos"][first:m].double(), s["sin"][first:m].double())[:, None]    # e^(i angle)
        qk = x[:, :Hq + Hk].clone()
        if c["style"] == "half":
            z = torch.complex(qk[..., :half].contiguous(), qk[..., half:2 * half].contiguous()) * turn
            qk[..., :half], qk[..., half:2 * half] = z.real, z.imag
        else:
            z = torch.view_as_complex(qk[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * turn
            qk[..., :2 * half] = torch.view_as_real(z).flatten(-2)
        qs.append(qk[:, :Hq])
        for which, fresh in ((0, qk[:, Hq:]), (1, x[:, Hq + Hk:])):
            for i in range(first // P, (m - 1) // P + 1):
                page = table[b][i]
                codes = s["k_codes"][page] if which == 0 else s["v_codes"][page].transpose(1, 2)       # [H][P][D]
                lo, hi = max(first, i * P), min(m, i * P + P)
                values = fresh[lo - first:hi - first].transpose(0, 1)                                  # [H][t][D]
                step = values.abs().amax(dim=(1, 2)) / 127
                if lo > i * P:
                    before = s["scales"][page, :, which].double()
                    step = torch.maximum(step, before)
                    kept = torch.round(codes[:, :lo - i * P].double() * (before / step)[:, None, None])
                    outs[which].append((kept * step[:, None, None]).transpose(0, 1))
                code = torch.round(values / step[:, None, None]).clamp(-127, 127)
                outs[which].append((code * step[:, None, None]).transpose(0, 1))
    return {"q": torch.cat(qs), "k": torch.cat(outs[0]), "v": torch.cat(outs[1])}


def _exact_attention(s):
    """One sequence, one key/value head and up to 2048 queries at a time in fp64."""
    c = s["case"]
    P, D, Hq, Hk = c["page"], c["dim"], c["q_heads"], c["kv_heads"]
    G = Hq // Hk
    new, kv = _lengths(c)
    y = torch.empty(s["T"], Hq, D, dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (n, m) in enumerate(zip(new, kv)):
        pages = s["table"][b, :-(-m // P)].long()
        key_at = torch.arange(m, device=y.device)
        for h in range(Hk):
            k = (s["k_codes"][pages, h].double() * s["scales"][pages, h, 0].double()[:, None, None]).flatten(0, 1)[:m]
            v = (s["v_codes"][pages, h].double() * s["scales"][pages, h, 1].double()[:, None, None])
            v = v.transpose(1, 2).flatten(0, 1)[:m]
            for i in range(0, n, 2048):
                count = min(2048, n - i)
                q = s["q"][at + i:at + i + count, h * G:(h + 1) * G].double()
                where = torch.arange(m - n + i, m - n + i + count, device=y.device)[:, None]
                hidden = key_at > where
                if c["window"]:
                    hidden |= (key_at <= where - c["window"]) & (key_at >= c["sinks"])
                logits = (q.flatten(0, 1) @ k.T).view(count, G, m) * s["scale"]
                weights = torch.softmax(logits.masked_fill(hidden[:, None], -math.inf), dim=-1)
                y[at + i:at + i + count, h * G:(h + 1) * G] = (weights.flatten(0, 1) @ v).view(count, G, D)
        at += n
    return y
