"""Cases of attention with shared key heads over a paged key/value cache, the attention weight that
each cached token has had, and eviction by it.

A server that keeps a bounded number of tokens a sequence runs four operators, each measured by
itself, around the selection that the library has:

* ``chunk``   causal attention of a chunk of new tokens (a prompt's piece, drafted tokens) over the
  cached ones, with the logarithm of each row's sum of exponentials;
* ``weigh``   the attention weight that the last of those tokens give every cached token, summed over
  them and over the query heads of a key head, added to what the token has had;
* ``decode``  attention of one new token a sequence, with the same sums from the same reading;
* ``evict``   the kept tokens of each key head moved to the front of their sequence's blocks (or into
  new blocks where others hold them), with their weights.

``run`` computes a case in plain torch operations; with ``own`` set, through the library.
A case's lengths follow from its numbers alone; a seed changes the values, the placement and the lists.
"""

import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # a serving batch verifies two to six drafted tokens a sequence
        _chunk("chunk of drafted tokens", seqs=64, lo=64, hi=2048, new_lo=2, new_hi=6, heads=32,
               kv_heads=8, dim=128, block=16, dtype="bf16"),
        # pieces of prompts, five query heads to a key head
        _chunk("chunk of prompts", seqs=16, lo=512, hi=2048, new_lo=512, new_hi=512, heads=40,
               kv_heads=8, dim=128, block=16, dtype="bf16"),
        # the last piece of one user's long prompt
        _chunk("chunk of one long context", seqs=1, lo=30011, hi=30011, new_lo=1024, new_hi=1024,
               heads=32, kv_heads=8, dim=128, block=16, dtype="f16"),
        # what the end of one user's prompt attends to
        _weigh("weigh one long context", seqs=1, lo=30011, hi=30011, new_lo=1024, new_hi=1024,
               window=32, heads=32, kv_heads=8, dim=128, block=16, dtype="bf16"),
        # what the ends of a batch of prompts attend to
        _weigh("weigh a batch", seqs=32, lo=2000, hi=16384, new_lo=32, new_hi=512, window=32,
               heads=64, kv_heads=8, dim=128, block=16, dtype="f16"),
        # what all of short prompts attends to, seven query heads to a key head
        _weigh("weigh whole short prompts", seqs=12, lo=200, hi=1500, new_lo=200, new_hi=1500,
               window=0, heads=28, kv_heads=4, dim=64, block=8, dtype="bf16"),
        # one user's next token
        _decode("decode one long context", seqs=1, lo=30011, hi=30011, heads=32, kv_heads=8,
                dim=128, block=16, dtype="bf16"),
        # a batch in which eight query heads share each key head
        _decode("decode a batch, grouped", seqs=64, lo=900, hi=16384, heads=64, kv_heads=8,
                dim=128, block=16, dtype="bf16"),
        # a full batch of short and middling contexts, every head with its own keys
        _decode("decode a batch, every head", seqs=64, lo=1, hi=2048, heads=40, kv_heads=40,
                dim=128, block=16, dtype="f16"),
        # one user's long prompt cut to its budget
        _evict("evict from one long context", seqs=1, lo=30011, hi=30011, keep=4096, kv_heads=8,
               dim=128, block=16, dtype="bf16"),
        # a batch of prompts cut to their budget, the shortest within it
        _evict("evict from a batch", seqs=64, lo=900, hi=16384, keep=1024, kv_heads=8, dim=128,
               block=16, dtype="bf16"),
        # two samples of each prompt, whose blocks both still read: kept tokens go to new ones
        _evict("evict from forked samples", seqs=32, lo=700, hi=3000, keep=512, kv_heads=4, dim=64,
               block=8, dtype="f16", forked=True),
    ]


def _chunk(name, seqs, lo, hi, new_lo, new_hi, heads, kv_heads, dim, block, dtype):
    return {"name": name, "op": "chunk", "seqs": seqs, "lo": lo, "hi": hi, "new_lo": new_lo,
            "new_hi": new_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "block": block,
            "dtype": dtype}


def _weigh(name, seqs, lo, hi, new_lo, new_hi, window, heads, kv_heads, dim, block, dtype):
    return {"name": name, "op": "weigh", "seqs": seqs, "lo": lo, "hi": hi, "new_lo": new_lo,
            "new_hi": new_hi, "window": window, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "block": block, "dtype": dtype}


def _decode(name, seqs, lo, hi, heads, kv_heads, dim, block, dtype):
    return {"name": name, "op": "decode", "seqs": seqs, "lo": lo, "hi": hi, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "block": block, "dtype": dtype}


def _evict(name, seqs, lo, hi, keep, kv_heads, dim, block, dtype, forked=False):
    return {"name": name, "op": "evict", "seqs": seqs, "lo": lo, "hi": hi, "keep": keep,
            "kv_heads": kv_heads, "dim": dim, "block": block, "dtype": dtype, "forked": forked}


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("chunk", "weigh", "decode", "evict"))
    most = [work(c) for c in listed() if c["op"] == op]
    most = {k: max(w[k] for w in most) for k in ("bytes", "flops")}
    while True:
        lo = _log(rng, 1, 20000)
        hi = _log(rng, lo, 32768)
        kv = rng.choice((1, 2, 3, 4, 5, 8, 16, 40))
        group = rng.choice((1, 2, 4, 5, 7, 8, 16)) if kv <= 8 else 1
        c = {"op": op, "seqs": _log(rng, 1, 128), "lo": lo, "hi": hi, "kv_heads": kv,
             "block": rng.choice((8, 16, 32, 64)), "dim": rng.choice((64, 128, 128, 256)),
             "dtype": rng.choice(("f16", "bf16"))}
        if op != "evict":
            c["heads"] = kv * group
        if op in ("chunk", "weigh"):
            c["new_lo"] = _log(rng, 1, lo)
            c["new_hi"] = _log(rng, c["new_lo"], lo) if rng.random() < 0.5 else c["new_lo"]
        if op == "weigh":
            c["window"] = rng.choice((0, 1, 16, 32, 50, 64))
        if op == "evict":
            c["keep"] = _log(rng, 1, 8192)
            c["forked"] = rng.random() < 0.25
            if c["keep"] >= hi:
                continue  # some sequence has to lose tokens
        w = work(c)
        if all(w[k] <= most[k] for k in most) and _cached(c) <= 6e9 and _logits(c) <= 6e9:
            return c


def _cached(c):
    """Bytes of the cache that a case keeps."""
    return sum(-(-n // c["block"]) for n in _lengths(c)) * c["block"] * c["kv_heads"] * c["dim"] * 4


def _logits(c):
    """Bytes of the logits of every row that any sequence might have."""
    if c["op"] == "evict":
        return 0
    rows = max(_counted(c)) if "new_hi" in c else 1
    return 4 * c["seqs"] * c["heads"] * rows * max(_lengths(c))


def _spread(lo, hi, n, step):
    """n whole numbers of [lo, hi]: lo + (hi - lo) times the fractions of i * step."""
    return [lo + round((hi - lo) * ((i * step) % 1.0)) for i in range(n)]


def _lengths(c):
    lens = _spread(c["hi"], c["lo"], c["seqs"], 0.6180339887498949)
    if c.get("forked"):  # the second of two samples has the first one's length
        lens = [lens[i - i % 2] for i in range(c["seqs"])]
    return lens


def _new(c):
    return [min(a, b) for a, b in zip(_spread(c["new_hi"], c["new_lo"], c["seqs"], 0.7548776662466927),
                                      _lengths(c))]


def _counted(c):
    """The new tokens whose rows a pass computes."""
    return [min(m, c["window"]) if c.get("window") else m for m in _new(c)]


def _sinks(c):
    return min(4, c["keep"])


def work(case):
    c, lens, bs = case, _lengths(case), case["block"]
    kv, d, n = c["kv_heads"], c["dim"], c["seqs"]
    tables = sum(4 * -(-x // bs) for x in lens) + 4 * n
    if c["op"] == "evict":
        cut = [x for x in lens if x > c["keep"]]
        moved = len(cut) * (c["keep"] if c["forked"] else c["keep"] - _sinks(c)) * kv
        return {"bytes": moved * (d * 8 + 4) + 4 * sum(cut) * kv
                + 4 * kv * sum(min(x, c["keep"]) for x in lens) + tables, "flops": 0}
    if c["op"] == "decode":
        return {"bytes": sum(lens) * kv * (d * 4 + 8) + 4 * n * c["heads"] * d + tables,
                "flops": 4 * sum(lens) * c["heads"] * d}
    rows = _counted(c)
    # row j of the last m tokens of n sees n - m + j + 1 of them
    seen = sum(m * x - m * (m - 1) // 2 for x, m in zip(lens, rows)) * c["heads"]
    if c["op"] == "chunk":
        return {"bytes": sum(lens) * kv * d * 4 + sum(rows) * c["heads"] * (d * 4 + 4) + tables,
                "flops": 4 * seen * d}
    return {"bytes": sum(lens) * kv * (d * 2 + 8) + sum(rows) * c["heads"] * (d * 2 + 4) + tables,
            "flops": 2 * seen * d}


# ---------------------------------------------------------------------- inputs
def _pages(c, gen, spare=3):
    """Block tables (entries past a sequence's blocks are -1), lengths, number of blocks, and the
    tables that an eviction moves into (None: the same)."""
    lens = _lengths(c)
    nb = torch.tensor([-(-n // c["block"]) for n in lens])
    width, total = int(nb.max()), int(nb.sum())
    fresh = -(-min(c["keep"], max(lens)) // c["block"]) if c.get("forked") else 0
    order = torch.randperm(total + spare + c["seqs"] * fresh, generator=gen).to(torch.int32)
    tables = torch.full((c["seqs"], width), -1, dtype=torch.int32)
    tables[torch.arange(width)[None, :] < nb[:, None]] = order[:total]
    new = None
    if c.get("forked"):
        tables[1::2] = tables[:-1:2][:len(tables[1::2])]
        new = torch.full((c["seqs"], width), -1, dtype=torch.int32)
        new[:, :fresh] = order[total:total + c["seqs"] * fresh].view(-1, fresh)
        whole = torch.tensor(lens) <= c["keep"]
        new[whole] = tables[whole]  # nothing is evicted, nothing moves
        new = new.to(DEVICE)
    return tables.to(DEVICE), torch.tensor(lens, dtype=torch.int32, device=DEVICE), len(order), new


def prepare(case, seed):
    c = case
    gen = torch.Generator().manual_seed(seed)
    dev = torch.Generator(device=DEVICE).manual_seed(seed)
    kv, d, n = c["kv_heads"], c["dim"], c["seqs"]

    def normal(*shape):
        return torch.randn(shape, generator=dev, device=DEVICE, dtype=TYPES[c["dtype"]])

    s = {"op": c["op"], "scale": 1 / math.sqrt(d)}
    s["tables"], s["lens"], blocks, s["new_tables"] = _pages(c, gen)
    s["k_cache"] = normal(blocks, kv, c["block"], d)
    room = s["tables"].shape[1] * c["block"]
    if c["op"] != "chunk":
        # a few tokens have had much of the weight, most of them little
        s["weights"] = torch.rand((n, kv, room), generator=dev, device=DEVICE).pow_(4)
        s["weights"] *= 5 * c.get("heads", kv) / kv / s["lens"][:, None, None]
    if c["op"] != "weigh":
        s["v_cache"] = normal(blocks, kv, c["block"], d)
    if c["op"] == "decode":
        s["q"] = normal(n, c["heads"], d)
        return s
    if c["op"] == "evict":
        s["kept"] = _lists(c, s["weights"], s["lens"])
        return s
    new = torch.tensor(_new(c))
    start = torch.zeros(n + 1, dtype=torch.int32)
    start[1:] = new.cumsum(0)
    s["start"], s["most"] = start.to(DEVICE), int(new.max())
    s["q"] = normal(int(start[-1]), c["heads"], d)
    s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEVICE)
    if c["op"] == "weigh":
        s["window"] = c["window"]
        s["lse"].zero_()
        for i, (length, first, end, rows) in enumerate(zip(_lengths(c), start, start[1:], _counted(c))):
            lot = slice(int(end) - rows, int(end))
            keys = s["k_cache"][s["tables"][i, :-(-length // c["block"])].long()].float().transpose(0, 1)
            logits = _grouped(s["q"][lot].float(), kv) @ keys.flatten(1, 2)[:, :length].transpose(1, 2)
            logits = logits.view(kv, rows, -1, length).mul_(s["scale"])
            past = torch.arange(length, device=DEVICE) > torch.arange(length - rows, length, device=DEVICE)[:, None]
            s["lse"][lot] = logits.masked_fill_(past[:, None], -math.inf).logsumexp(-1).transpose(0, 1).flatten(1)
    return s


def _grouped(q, kv):
    """Rows [T, heads, D] as [key heads, T * heads of each, D]."""
    return q.unflatten(1, (kv, -1)).permute(1, 0, 2, 3).flatten(1, 2)


def _lists(c, weights, lens):
    """Ascending places to keep, then -1: the first, the last and those with the most weight."""
    n, kv, room = weights.shape
    place = torch.arange(room, device=DEVICE)
    length = lens[:, None, None]
    value = weights.masked_fill((place < _sinks(c)) | (place >= length - c["keep"] // 4), math.inf)
    value = value.masked_fill(place >= length, -math.inf)
    keep = min(c["keep"], room)
    best = value.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    best = best.masked_fill(torch.arange(keep, device=DEVICE) >= length, room).sort(-1).values
    kept = torch.full((n, kv, c["keep"]), -1, dtype=torch.int32, device=DEVICE)
    kept[..., :keep] = best.masked_fill(best == room, -1)
    return kept


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        return _own(s)
    return {"chunk": _plain_chunk, "weigh": _plain_weigh, "decode": _plain_decode,
            "evict": _plain_evict}[s["op"]](s)


def _own(s):
    from paged_kv_cache_317_gb300 import binding as pa
    if s["op"] == "chunk":
        out = pa.paged_attn_chunk(s["q"], s["start"], s["most"], s["k_cache"], s["v_cache"], s["tables"],
                                  s["lens"], s["scale"], out_dtype=s["q"].dtype, lse=s["lse"])
        return {"out": out, "lse": s["lse"]}
    if s["op"] == "weigh":
        pa.paged_chunk_weights(s["q"], s["lse"], s["start"], s["most"], s["k_cache"], s["tables"], s["lens"],
                               s["scale"], s["weights"], window=s["window"])
        return s["weights"]
    if s["op"] == "decode":
        out = pa.paged_attn_decode_weights(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                           s["scale"], s["weights"], out_dtype=s["q"].dtype)
        return {"out": out, "weights": s["weights"]}
    pa.kv_cache_evict(s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["kept"], weights=s["weights"],
                      new_tables=s["new_tables"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": s["weights"]}


def _cached_rows(cache, tables):
    """[N, key heads, places, D] in 32 bits."""
    return cache[tables.clamp(min=0).long()].transpose(1, 2).flatten(2, 3).float()


def _rows(s, kv, window):
    """The new tokens by sequence: which row of q each is [N, most], which there are, their queries
    [N, key heads, most, heads of each, D] in 32 bits, and which of the places each sees."""
    start, lens = s["start"].long(), s["lens"].long()
    new = start[1:] - start[:-1]
    used = new.clamp(max=window) if window else new
    most = min(s["most"], window) if window else s["most"]
    j = torch.arange(most, device=DEVICE)
    there = j < used[:, None]
    row = ((start[1:] - used)[:, None] + j).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().unflatten(2, (kv, -1)).transpose(1, 2)
    seen = torch.arange(s["tables"].shape[1] * s["k_cache"].shape[2], device=DEVICE) <= (
        (lens - used)[:, None] + j)[..., None]
    return row, there, q, seen & there[..., None]


def _plain_chunk(s):
    kv = s["k_cache"].shape[1]
    row, there, q, seen = _rows(s, kv, 0)
    most, group = q.shape[2:4]
    logits = q.flatten(2, 3) @ _cached_rows(s["k_cache"], s["tables"]).transpose(2, 3)
    logits = logits.unflatten(2, (most, group)).mul_(s["scale"])
    logits.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-3e38)
    w = logits.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    values = _cached_rows(s["v_cache"], s["tables"])
    values.masked_fill_((torch.arange(values.shape[2], device=DEVICE) >= s["lens"][:, None])[:, None, :, None], 0)
    out = (w.flatten(2, 3) @ values).unflatten(2, (most, group)) / total
    lse = (top + total.log()).squeeze(-1)
    result = torch.empty_like(s["q"])
    result[row[there]] = out.permute(0, 2, 1, 3, 4).flatten(2, 3)[there].to(result.dtype)
    s["lse"][row[there]] = lse.permute(0, 2, 1, 3).flatten(2, 3)[there]
    return {"out": result, "lse": s["lse"]}


def _plain_weigh(s):
    kv = s["k_cache"].shape[1]
    row, there, q, seen = _rows(s, kv, s["window"])
    most, group = q.shape[2:4]
    logits = q.flatten(2, 3) @ _cached_rows(s["k_cache"], s["tables"]).transpose(2, 3)
    lse = s["lse"][row].unflatten(2, (kv, group)).transpose(1, 2).unsqueeze(-1)
    w = logits.unflatten(2, (most, group)).mul_(s["scale"]).sub_(lse)
    w = w.masked_fill_(~seen[:, None, :, None], -math.inf).exp_()
    s["weights"] += w.sum((2, 3))
    return s["weights"]


def _plain_decode(s):
    n, heads, d = s["q"].shape
    kv = s["k_cache"].shape[1]
    keys, values = _cached_rows(s["k_cache"], s["tables"]), _cached_rows(s["v_cache"], s["tables"])
    past = (torch.arange(keys.shape[2], device=DEVICE) >= s["lens"][:, None])[:, None, None]
    logits = s["q"].float().view(n, kv, -1, d) @ keys.transpose(2, 3)
    w = logits.mul_(s["scale"]).masked_fill_(past, -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True)).exp_()
    w /= w.sum(-1, keepdim=True)
    s["weights"] += w.sum(2)
    out = w @ values.masked_fill_(past.transpose(2, 3), 0)
    return {"out": out.view(n, heads, d).to(s["q"].dtype), "weights": s["weights"]}


def _plain_evict(s):
    n, kv, keep = s["kept"].shape
    bs = s["k_cache"].shape[2]
    there = s["kept"] >= 0
    place = s["kept"].clamp(min=0).long()
    new = s["tables"] if s["new_tables"] is None else s["new_tables"]
    block = s["tables"].long().gather(1, (place // bs).flatten(1)).view_as(place)[there]
    at = torch.arange(keep, device=DEVICE).expand_as(place)
    to = new.long().gather(1, (at // bs).clamp(max=new.shape[1] - 1).flatten(1)).view_as(place)[there]
    head = torch.arange(kv, device=DEVICE)[:, None].expand_as(place)[there]
    k, v = (x[block, head, place[there] % bs] for x in (s["k_cache"], s["v_cache"]))
    s["k_cache"][to, head, at[there] % bs], s["v_cache"][to, head, at[there] % bs] = k, v
    w = s["weights"]
    moved = torch.zeros_like(w)
    moved[..., :keep] = (w.gather(2, place) * there)[..., :w.shape[2]]
    held = torch.arange(w.shape[2], device=DEVICE) < s["lens"][:, None, None]
    w.copy_(torch.where(held, moved, w))
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": w}


# ------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"chunk": _exact_chunk, "weigh": _exact_weigh, "decode": _exact_decode,
            "evict": _exact_evict}[s["op"]](s)


def _exact_weights(s, i, q, places, repeat):
    """Logits [heads, rows, length] of a sequence's rows at `places`, -inf where they are not seen."""
    length, bs = int(s["lens"][i]), s["k_cache"].shape[2]
    pages = s["tables"][i, :-(-length // bs)].long()
    keys = s["k_cache"][pages].permute(1, 0, 2, 3).flatten(1, 2)[:, :length].double()
    logits = torch.einsum("rhd,htd->hrt", q.double(), keys.repeat_interleave(repeat, 0)) * s["scale"]
    for r, place in enumerate(places):
        logits[:, r, place + 1:] = -math.inf
    return logits


def _exact_values(s, i, w, repeat):
    length, bs = int(s["lens"][i]), s["v_cache"].shape[2]
    pages = s["tables"][i, :-(-length // bs)].long()
    values = s["v_cache"][pages].permute(1, 0, 2, 3).flatten(1, 2)[:, :length].double()
    return torch.einsum("hrt,htd->rhd", w, values.repeat_interleave(repeat, 0))


def _exact_chunk(s):
    repeat = s["q"].shape[1] // s["k_cache"].shape[1]
    out, lse = s["q"].double(), s["lse"].double()
    start = s["start"].tolist()
    for i, length in enumerate(s["lens"].tolist()):
        for a in range(start[i], start[i + 1], 256):
            b = min(a + 256, start[i + 1])
            first = length - start[i + 1] + a
            logits = _exact_weights(s, i, s["q"][a:b], range(first, first + b - a), repeat)
            lse[a:b] = torch.logsumexp(logits, -1).t()
            out[a:b] = _exact_values(s, i, torch.softmax(logits, -1), repeat)
    return {"out": out, "lse": lse}


def _exact_weigh(s):
    kv = s["k_cache"].shape[1]
    repeat = s["q"].shape[1] // kv
    total = s["weights"].double()
    start = s["start"].tolist()
    for i, length in enumerate(s["lens"].tolist()):
        begin = max(start[i], start[i + 1] - s["window"]) if s["window"] else start[i]
        for a in range(begin, start[i + 1], 256):
            b = min(a + 256, start[i + 1])
            first = length - start[i + 1] + a
            logits = _exact_weights(s, i, s["q"][a:b], range(first, first + b - a), repeat)
            w = torch.exp(logits - s["lse"][a:b].double().t()[..., None])
            total[i, :, :length] += w.sum(1).view(kv, repeat, length).sum(1)
    return total


def _exact_decode(s):
    kv = s["k_cache"].shape[1]
    repeat = s["q"].shape[1] // kv
    out, total = s["q"].double(), s["weights"].double()
    for i, length in enumerate(s["lens"].tolist()):
        w = torch.softmax(_exact_weights(s, i, s["q"][i:i + 1], [length - 1], repeat), -1)
        out[i] = _exact_values(s, i, w, repeat)[0]
        total[i, :, :length] += w.view(kv, repeat, length).sum(1)
    return {"out": out, "weights": total}


def _exact_evict(s):
    bs = s["k_cache"].shape[2]
    out = {k: s[k].clone() for k in ("k_cache", "v_cache", "weights")}  # values move, none is computed
    new = s["tables"] if s["new_tables"] is None else s["new_tables"]
    for i, length in enumerate(s["lens"].tolist()):
        out["weights"][i, :, :length] = 0
        for h in range(s["kept"].shape[1]):
            old = s["kept"][i, h].long()
            old = old[old >= 0]
            at = torch.arange(len(old), device=DEVICE)
            source, to = s["tables"][i].long()[old // bs], new[i].long()[at // bs]
            for k in ("k_cache", "v_cache"):
                out[k][to, h, at % bs] = s[k][source, h, old % bs]
            out["weights"][i, h, at] = s["weights"][i, h, old]
    return {k: v.double() for k, v in out.items()}
