"""Cases of the rotated append and of block-sparse decode over a paged key/value cache.

One decode step of a sparse server is a chain of five operators, each measured by itself:

* ``append``  rotates queries and keys by their positions, writes keys and values into their
  slots and keeps each block's channel-wise key bounds (smallest and largest value) up;
* ``bounds``  computes those bounds anew from cached keys (after a prompt, a load, a rollback);
* ``scores``  the largest logit that any key of a block can have, from the bounds;
* ``select``  the best blocks of every (sequence, key/value head), first and last ones always;
* ``attend``  softmax attention over the tokens of the listed blocks.

``run`` computes a case in plain torch operations; with ``own`` set, through the library.
A case's lengths follow from its numbers alone; a seed changes the values and the placement.
"""

import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- the cases
def listed():
    return [
        # one user's next token: the smallest append there is
        _append("append one token", seqs=1, lo=4000, hi=4000, new_lo=1, new_hi=1, heads=32,
                kv_heads=8, dim=128, rot=128, block=16, dtype="bf16"),
        # the append of a decode step over a full batch, every head with its own keys
        _append("append step of 256 x 40 heads", seqs=256, lo=1, hi=400, new_lo=1, new_hi=1,
                heads=40, kv_heads=40, dim=128, rot=128, block=16, dtype="bf16"),
        # prompts with images, ragged: positions of three axes, half of each head rotated
        _append("append ragged prompts, three axes", seqs=24, lo=700, hi=1500, new_lo=1,
                new_hi=700, heads=32, kv_heads=8, dim=128, rot=64, block=16, dtype="f16",
                axes=3, interleaved=True),
        # a few short sequences after a rollback of drafted tokens
        _bounds("bounds of short sequences", seqs=9, lo=1, hi=333, kv_heads=4, dim=64, block=8,
                dtype="f16"),
        # prompts that came into the cache from elsewhere
        _bounds("bounds of long prompts", seqs=32, lo=500, hi=16384, kv_heads=8, dim=128,
                block=16, dtype="bf16"),
        # one user's long context
        _scores("scores of one long context", seqs=1, lo=30011, hi=30011, heads=32, kv_heads=8,
                dim=128, block=16, dtype="bf16"),
        # a batch of long contexts, ragged
        _scores("scores of a batch", seqs=48, lo=2000, hi=32768, heads=64, kv_heads=8, dim=128,
                block=16, dtype="f16"),
        # the lists of one user's long context
        _select("select of one long context", seqs=1, lo=30011, hi=30011, kv_heads=8, block=16,
                keep=128, sink=1, recent=4),
        # the lists of a batch of long contexts, every head its own
        _select("select of a batch", seqs=32, lo=2000, hi=131072, kv_heads=40, block=16,
                keep=256, sink=1, recent=8),
        # one user's token over 64 blocks of a long context
        _attend("attend one long context", seqs=1, lo=30011, hi=30011, heads=32, kv_heads=8,
                dim=128, block=16, keep=64, dtype="bf16"),
        # a batch in which eight query heads share each key head
        _attend("attend a batch, grouped", seqs=64, lo=900, hi=16384, heads=64, kv_heads=8,
                dim=128, block=16, keep=128, dtype="bf16"),
        # long contexts, every head its own keys and lists
        _attend("attend a batch, every head", seqs=32, lo=16384, hi=16384, heads=40,
                kv_heads=40, dim=128, block=16, keep=64, dtype="f16"),
    ]


def _append(name, seqs, lo, hi, new_lo, new_hi, heads, kv_heads, dim, rot, block, dtype, axes=1,
            interleaved=False):
    return {"name": name, "op": "append", "seqs": seqs, "lo": lo, "hi": hi, "new_lo": new_lo,
            "new_hi": new_hi, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "block": block, "dtype": dtype, "axes": axes, "interleaved": interleaved}


def _bounds(name, seqs, lo, hi, kv_heads, dim, block, dtype):
    return {"name": name, "op": "bounds", "seqs": seqs, "lo": lo, "hi": hi,
            "kv_heads": kv_heads, "dim": dim, "block": block, "dtype": dtype}


def _scores(name, seqs, lo, hi, heads, kv_heads, dim, block, dtype):
    return {"name": name, "op": "scores", "seqs": seqs, "lo": lo, "hi": hi, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "block": block, "dtype": dtype}


def _select(name, seqs, lo, hi, kv_heads, block, keep, sink, recent):
    return {"name": name, "op": "select", "seqs": seqs, "lo": lo, "hi": hi,
            "kv_heads": kv_heads, "block": block, "keep": keep, "sink": sink, "recent": recent}


def _attend(name, seqs, lo, hi, heads, kv_heads, dim, block, keep, dtype):
    return {"name": name, "op": "attend", "seqs": seqs, "lo": lo, "hi": hi, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "block": block, "keep": keep, "dtype": dtype}


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("append", "bounds", "scores", "select", "attend"))
    most = max(work(c)["bytes"] for c in listed() if c["op"] == op)
    while True:
        lo = _log(rng, 1, 20000)
        hi = _log(rng, lo, 32768)
        kv = rng.choice((1, 2, 3, 4, 5, 8, 16, 32, 40))
        group = rng.choice((1, 1, 2, 4, 5, 7, 8, 16)) if kv <= 8 else 1
        c = {"op": op, "seqs": _log(rng, 1, 256), "lo": lo, "hi": hi, "kv_heads": kv,
             "block": rng.choice((8, 16, 32, 64))}
        if op in ("append", "scores", "attend"):
            c["heads"] = kv * group
        if op != "select":
            c["dim"] = rng.choice((64, 128, 128, 256))
            c["dtype"] = rng.choice(("f16", "bf16"))
        if op == "append":
            c["axes"] = rng.choice((1, 1, 2, 3))
            c["interleaved"] = rng.random() < 0.5
            c["rot"] = rng.choice((c["dim"], c["dim"] // 2, 32))
            c["new_lo"] = _log(rng, 1, lo) if rng.random() < 0.5 else 1
            c["new_hi"] = _log(rng, c["new_lo"], lo) if rng.random() < 0.5 else c["new_lo"]
        if op in ("select", "attend"):
            c["keep"] = _log(rng, 1, 512)
        if op == "select":
            c["lo"], c["hi"] = lo * 4, hi * 4
            c["sink"] = rng.randint(0, min(4, max(0, c["keep"] - 2)))
            c["recent"] = rng.randint(0, min(8, max(0, c["keep"] - c["sink"] - 2)))
            if c["keep"] < 2 or -(-c["hi"] // c["block"]) < c["keep"] + 64:
                continue  # some sequence has to have blocks to choose from
        if work(c)["bytes"] <= most and _cached(c) <= (2e9 if op == "append" else 14e9):
            return c


def _cached(c):
    """Bytes of the cache that a case keeps."""
    return sum(-(-n // c["block"]) for n in _lengths(c)) * c["block"] * c["kv_heads"] * c.get("dim", 0) * 4


def _spread(lo, hi, n, step):
    """n whole numbers of [lo, hi]: lo + (hi - lo) times the fractions of i * step."""
    return [lo + round((hi - lo) * ((i * step) % 1.0)) for i in range(n)]


def _lengths(c):
    return _spread(c["hi"], c["lo"], c["seqs"], 0.6180339887498949)


def _new(c):
    return [min(a, b) for a, b in zip(_spread(c["new_hi"], c["new_lo"], c["seqs"], 0.7548776662466927),
                                      _lengths(c))]


def work(case):
    c, lens, bs = case, _lengths(case), case["block"]
    nb = [-(-n // bs) for n in lens]
    blocks, kv = sum(nb), c["kv_heads"]
    tables = 4 * blocks + 4 * c["seqs"]
    if c["op"] == "append":
        new, d = _new(c), c["dim"]
        tokens = sum(new)
        fresh = sum(-(-n // bs) - -(-(n - m) // bs) for n, m in zip(lens, new))
        merged = sum((n - m) % bs > 0 for n, m in zip(lens, new))
        rows = min(tokens, max(lens)) if c["axes"] == 1 else tokens
        size = (tokens * (2 * c["heads"] + 4 * kv) * d * 2 + rows * c["rot"] * 4
                + (fresh * 2 + merged * 4) * kv * d * 2
                + 4 * (fresh + merged + 2 * c["seqs"]) + (4 * c["axes"] * tokens if c["axes"] > 1 else 0))
        return {"bytes": size, "flops": 3 * tokens * (c["heads"] + kv) * c["rot"]}
    if c["op"] == "bounds":
        return {"bytes": (sum(lens) * 2 + blocks * 4) * kv * c["dim"] + tables,
                "flops": 2 * sum(lens) * kv * c["dim"]}
    if c["op"] == "scores":
        return {"bytes": blocks * kv * c["dim"] * 4 + c["seqs"] * (c["heads"] * c["dim"] * 2 + kv * max(nb) * 4)
                + tables, "flops": 4 * blocks * c["heads"] * c["dim"]}
    if c["op"] == "select":
        return {"bytes": 4 * kv * (blocks + c["seqs"] * c["keep"]) + 4 * c["seqs"], "flops": blocks * kv}
    listed_blocks = sum(min(n, c["keep"]) for n in nb)
    # the last block is taken as listed in proportion: its empty rows are not read
    tokens = sum(n if b <= c["keep"] else c["keep"] * n / b for n, b in zip(lens, nb))
    return {"bytes": int(tokens * kv * c["dim"] * 4 + 2 * c["seqs"] * c["heads"] * c["dim"] * 2
                         + 4 * c["seqs"] * kv * c["keep"] + 4 * listed_blocks),
            "flops": 4 * tokens * c["heads"] * c["dim"]}


# ---------------------------------------------------------------------- inputs
def _pages(c, gen, spare=3):
    """Block tables (entries past a sequence's blocks are -1), lengths, number of blocks."""
    lens = _lengths(c)
    nb = torch.tensor([-(-n // c["block"]) for n in lens])
    width, total = int(nb.max()), int(nb.sum())
    order = torch.randperm(total + spare, generator=gen)[:total].to(torch.int32)
    tables = torch.full((c["seqs"], width), -1, dtype=torch.int32)
    tables[torch.arange(width)[None, :] < nb[:, None]] = order
    return tables.to(DEVICE), torch.tensor(lens, dtype=torch.int32, device=DEVICE), total + spare


def prepare(case, seed):
    c = case
    gen = torch.Generator().manual_seed(seed)
    dev = torch.Generator(device=DEVICE).manual_seed(seed)
    s = {"op": c["op"], "block": c["block"]}

    def normal(*shape):
        return torch.randn(shape, generator=dev, device=DEVICE, dtype=TYPES[c["dtype"]])

    kv, d, n = c["kv_heads"], c.get("dim"), c["seqs"]
    s["tables"], s["lens"], blocks = _pages(c, gen)
    if "heads" in c:
        s["scale"] = 1 / math.sqrt(d)
    if c["op"] == "append":
        new = torch.tensor(_new(c))
        start = torch.zeros(n + 1, dtype=torch.int32)
        start[1:] = new.cumsum(0)
        tokens = int(start[-1])
        s["start"], s["most"] = start.to(DEVICE), int(new.max())
        # one projection gives queries, keys and values side by side
        fused = normal(tokens, (c["heads"] + 2 * kv) * d)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in
                                  fused.split([c["heads"] * d, kv * d, kv * d], dim=1))
        s["k_cache"], s["v_cache"] = normal(blocks, kv, c["block"], d), normal(blocks, kv, c["block"], d)
        s["k_min"], s["k_max"] = s["k_cache"].amin(2), s["k_cache"].amax(2)
        reach = max(_lengths(c))
        rates = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEVICE) / c["rot"])
        angles = torch.arange(reach, dtype=torch.float64, device=DEVICE)[:, None] * rates
        s["cos_sin"] = torch.cat([angles.cos(), angles.sin()], 1).float()
        s["interleaved"], s["positions"], s["pair_axis"] = c["interleaved"], None, None
        if c["axes"] > 1:
            s["positions"] = torch.randint(0, reach, (c["axes"], tokens), generator=gen).to(torch.int32).to(DEVICE)
            # the axes take turns over the pairs, in runs of four
            s["pair_axis"] = [j // 4 % c["axes"] for j in range(c["rot"] // 2)]
        return s
    if c["op"] == "bounds":
        s["k_cache"] = normal(blocks, kv, c["block"], d)
        s["k_min"], s["k_max"] = normal(blocks, kv, d), normal(blocks, kv, d)
        return s
    if c["op"] == "scores":
        a, b = normal(blocks, kv, d), normal(blocks, kv, d)
        # sixteen normal values lie between about -1.8 and 1.8
        s["k_min"], s["k_max"] = torch.minimum(a, b) - 1, torch.maximum(a, b) + 1
        s["q"] = normal(n, c["heads"], d)
        return s
    if c["op"] == "select":
        width = s["tables"].shape[1]
        # scores of which some are equal, as those of repeated text are
        s["scores"] = (torch.randn((n, kv, width), generator=dev, device=DEVICE) * 512).round() / 64
        s["scores"].masked_fill_(torch.arange(width, device=DEVICE) * c["block"] >= s["lens"][:, None, None],
                                 -math.inf)
        s["keep"], s["sink"], s["recent"] = c["keep"], c["sink"], c["recent"]
        return s
    s["q"] = normal(n, c["heads"], d)
    s["k_cache"], s["v_cache"] = normal(blocks, kv, c["block"], d), normal(blocks, kv, c["block"], d)
    width = s["tables"].shape[1]
    keep = min(c["keep"], width)
    held = torch.arange(width, device=DEVICE) * c["block"] < s["lens"][:, None, None]
    rank = torch.rand((n, kv, width), generator=dev, device=DEVICE).masked_fill_(~held, 2.0)
    rank, at = rank.sort(-1)
    at = at[..., :keep].masked_fill(rank[..., :keep] > 1, width).sort(-1).values
    s["selected"] = torch.full((n, kv, c["keep"]), -1, dtype=torch.int32, device=DEVICE)
    s["selected"][..., :keep] = at.masked_fill(at == width, -1)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        return _own(s)
    return {"append": _plain_append, "bounds": _plain_bounds, "scores": _plain_scores,
            "select": _plain_select, "attend": _plain_attend}[s["op"]](s)


def _own(s):
    from paged_kv_cache_317_gb300 import binding as pa
    if s["op"] == "append":
        q = pa.kv_cache_append_rope(s["q"], s["k"], s["v"], s["start"], s["most"], s["k_cache"],
                                    s["v_cache"], s["tables"], s["lens"], s["cos_sin"],
                                    interleaved=s["interleaved"], positions=s["positions"],
                                    pair_axis=s["pair_axis"], k_min=s["k_min"], k_max=s["k_max"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_min": s["k_min"],
                "k_max": s["k_max"]}
    if s["op"] == "bounds":
        pa.kv_block_bounds(s["k_cache"], s["tables"], s["lens"], s["k_min"], s["k_max"])
        return {"k_min": s["k_min"], "k_max": s["k_max"]}
    if s["op"] == "scores":
        return pa.paged_block_scores(s["q"], s["k_min"], s["k_max"], s["tables"], s["lens"], s["scale"],
                                     s["block"])
    if s["op"] == "select":
        return pa.paged_block_select(s["scores"], s["lens"], s["block"], s["keep"], sink_blocks=s["sink"],
                                     recent_blocks=s["recent"])
    return pa.paged_attn_sparse(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["selected"],
                                s["scale"], out_dtype=s["q"].dtype)


def _turn(x, cos, sin, interleaved):
    """x [T, heads, D] in 32 bits, its first dims rotated by cos and sin [T, 1, pairs]."""
    rot = 2 * cos.shape[-1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, w], -1).flatten(-2) if interleaved else torch.cat([u, w], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_append(s):
    lens, start, bs = s["lens"].long(), s["start"].long(), s["block"]
    tokens = s["q"].shape[0]
    t = torch.arange(tokens, device=DEVICE)
    seq = torch.searchsorted(start, t, right=True) - 1
    place = lens[seq] - start[seq + 1] + t
    pairs = s["cos_sin"].shape[1] // 2
    if s["positions"] is None:
        rows = s["cos_sin"][place]
        cos, sin = rows[:, None, :pairs], rows[:, None, pairs:]
    else:
        axis = torch.tensor(s["pair_axis"], device=DEVICE)
        at = s["positions"].long()[axis].t()
        pair = torch.arange(pairs, device=DEVICE)
        cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, pair + pairs][:, None]
    q = _turn(s["q"].float(), cos, sin, s["interleaved"]).to(s["q"].dtype)
    k = _turn(s["k"].float(), cos, sin, s["interleaved"]).to(s["k"].dtype)
    block, row = s["tables"][seq, place // bs].long(), place % bs
    s["k_cache"][block, :, row] = k
    s["v_cache"][block, :, row] = s["v"]
    low, high = s["k_min"].float(), s["k_max"].float()
    begun = block[row == 0]
    low[begun], high[begun] = math.inf, -math.inf
    low.index_reduce_(0, block, k.float(), "amin")
    high.index_reduce_(0, block, k.float(), "amax")
    s["k_min"].copy_(low)
    s["k_max"].copy_(high)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "k_min": s["k_min"], "k_max": s["k_max"]}


def _plain_bounds(s):
    bs, lens = s["block"], s["lens"]
    width = s["tables"].shape[1]
    at = torch.arange(width, device=DEVICE) * bs
    held = at < lens[:, None]
    block = s["tables"][held].long()
    rows = (lens[:, None] - at)[held]
    keys = s["k_cache"][block].float()
    empty = (torch.arange(bs, device=DEVICE) >= rows[:, None])[:, None, :, None]
    s["k_min"][block] = keys.masked_fill(empty, math.inf).amin(2).to(s["k_min"].dtype)
    s["k_max"][block] = keys.masked_fill(empty, -math.inf).amax(2).to(s["k_max"].dtype)
    return {"k_min": s["k_min"], "k_max": s["k_max"]}


def _plain_scores(s):
    n, width = s["tables"].shape
    kv, d = s["k_min"].shape[1:]
    block = s["tables"].clamp(min=0).long()
    q = s["q"].float().reshape(n, kv, -1, d)
    low, high = (x[block].float().permute(0, 2, 3, 1) for x in (s["k_min"], s["k_max"]))
    best = (q.clamp(min=0) @ high + q.clamp(max=0) @ low).amax(2) * s["scale"]
    past = torch.arange(width, device=DEVICE) * s["block"] >= s["lens"][:, None, None]
    return best.masked_fill(past, -math.inf)


def _plain_select(s):
    n, kv, width = s["scores"].shape
    held = ((s["lens"].long() + s["block"] - 1) // s["block"])[:, None, None]
    b = torch.arange(width, device=DEVICE)
    value = s["scores"].masked_fill((b < s["sink"]) | (b >= held - s["recent"]), math.inf)
    # blocks past the last one go behind every other; among equals the lowest first
    order = torch.where(b < held, value, -math.inf).sort(dim=-1, descending=True, stable=True).indices
    keep = min(s["keep"], width)
    best = torch.where(torch.arange(keep, device=DEVICE) < held, order[..., :keep], width)
    best = best.sort(-1).values
    out = torch.full((n, kv, s["keep"]), -1, dtype=torch.int32, device=DEVICE)
    out[..., :keep] = best.masked_fill(best == width, -1)
    return out


def _plain_attend(s):
    n, heads, d = s["q"].shape
    kv, bs = s["k_cache"].shape[1:3]
    chosen = s["selected"].long()
    block = s["tables"].long().gather(1, chosen.clamp(min=0).flatten(1)).view_as(chosen).clamp(min=0)
    head = torch.arange(kv, device=DEVICE)[:, None]
    k, v = (x[block, head].float().flatten(2, 3) for x in (s["k_cache"], s["v_cache"]))
    place = chosen[..., None] * bs + torch.arange(bs, device=DEVICE)
    hidden = ((chosen[..., None] < 0) | (place >= s["lens"][:, None, None, None])).flatten(2)[:, :, None]
    q = s["q"].float().reshape(n, kv, -1, d)
    logits = (q @ k.transpose(2, 3) * s["scale"]).masked_fill_(hidden, -math.inf)
    w = (logits - logits.amax(-1, keepdim=True)).exp_()
    out = w @ v.masked_fill_(hidden.transpose(2, 3), 0) / w.sum(-1, keepdim=True)
    return out.reshape(n, heads, d).to(s["q"].dtype)


# ------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "select":
        return None  # whole numbers
    if case["op"] == "append" and sum(m // case["block"] + 2 for m in _new(case)) > 20000:
        return None
    s = prepare(case, seed)
    return {"append": _exact_append, "bounds": _exact_bounds, "scores": _exact_scores,
            "attend": _exact_attend}[s["op"]](s)


def _exact_append(s):
    lens, start, bs = s["lens"].tolist(), s["start"].tolist(), s["block"]
    pairs = s["cos_sin"].shape[1] // 2
    table = s["cos_sin"].double()
    out = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double(),
           "k_min": s["k_min"].double(), "k_max": s["k_max"].double()}
    q, keys = s["q"].double(), s["k"].double()
    axis = s["pair_axis"] or [0] * pairs
    first = [2 * j if s["interleaved"] else j for j in range(pairs)]
    second = [2 * j + 1 if s["interleaved"] else j + pairs for j in range(pairs)]
    place = torch.cat([torch.arange(n - (b - a), n) for n, a, b in zip(lens, start, start[1:])]).to(DEVICE)
    for x in (q, keys):
        for j in range(pairs):
            p = place if s["positions"] is None else s["positions"][axis[j]].long()
            c, r = table[p, j][:, None], table[p, j + pairs][:, None]
            a, b = x[..., first[j]].clone(), x[..., second[j]].clone()
            x[..., first[j]], x[..., second[j]] = a * c - b * r, a * r + b * c
    out["q"] = q
    for i, (n, a, b) in enumerate(zip(lens, start, start[1:])):
        at = n - (b - a)
        while at < n:
            end = min(n, (at // bs + 1) * bs)
            page = int(s["tables"][i, at // bs])
            lot = slice(a + at - (n - (b - a)), a + end - (n - (b - a)))
            rows = slice(at % bs, at % bs + end - at)
            out["k_cache"][page, :, rows] = keys[lot].transpose(0, 1)
            out["v_cache"][page, :, rows] = s["v"][lot].transpose(0, 1).double()
            low, high = keys[lot].amin(0), keys[lot].amax(0)
            if at % bs:
                low, high = torch.minimum(low, out["k_min"][page]), torch.maximum(high, out["k_max"][page])
            out["k_min"][page], out["k_max"][page] = low, high
            at = end
    return out


def _exact_bounds(s):
    out = {"k_min": s["k_min"].double(), "k_max": s["k_max"].double()}
    bs = s["block"]
    for i, n in enumerate(s["lens"].tolist()):
        pages = s["tables"][i, :-(-n // bs)].long()
        keys = s["k_cache"][pages].double()
        out["k_min"][pages], out["k_max"][pages] = keys.amin(2), keys.amax(2)
        tail = keys[-1, :, :n - (len(pages) - 1) * bs]
        out["k_min"][pages[-1]], out["k_max"][pages[-1]] = tail.amin(1), tail.amax(1)
    return out


def _exact_scores(s):
    n, width = s["tables"].shape
    kv, d = s["k_min"].shape[1:]
    out = torch.full((n, kv, width), -math.inf, dtype=torch.float64, device=DEVICE)
    q = s["q"].double().reshape(n, kv, -1, d)
    for i, length in enumerate(s["lens"].tolist()):
        held = -(-length // s["block"])
        pages = s["tables"][i, :held].long()
        low, high = s["k_min"][pages].double(), s["k_max"][pages].double()
        best = [torch.maximum(q[i, :, g] * low, q[i, :, g] * high).sum(-1) for g in range(q.shape[2])]
        out[i, :, :held] = torch.stack(best).amax(0).t() * s["scale"]
    return out


def _exact_attend(s):
    n, heads, d = s["q"].shape
    kv, bs = s["k_cache"].shape[1:3]
    out = torch.zeros((n, kv, heads // kv, d), dtype=torch.float64, device=DEVICE)
    q = s["q"].double().reshape(n, kv, -1, d)
    head = torch.arange(kv, device=DEVICE)[:, None]
    for i, length in enumerate(s["lens"].tolist()):
        chosen = s["selected"][i].long()
        held = int((chosen >= 0).sum(1).max())
        chosen = chosen[:, :held]
        page = s["tables"][i].long()[chosen]
        token = (chosen[..., None] * bs + torch.arange(bs, device=DEVICE)).reshape(kv, -1)
        k, v = (x[page, head].reshape(kv, -1, d).double() for x in (s["k_cache"], s["v_cache"]))
        logits = torch.einsum("hgd,htd->hgt", q[i], k) * s["scale"]
        logits[(token >= length)[:, None].expand_as(logits)] = -math.inf
        out[i] = torch.einsum("hgt,htd->hgd", torch.softmax(logits, -1), v)
    return out.reshape(n, heads, d)
