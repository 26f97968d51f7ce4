"""Cases and plain forms of two more sets of operators on the 8-bit paged cache:
attention whose scores are capped, biased by distance, or masked by documents and
prefixes, and the pool of pages behind the tables: sharing, reserving (with the
copy of a shared page that is about to be written), freeing and compacting.

A cache holds pages of `page` tokens: int8 codes [n_pages][n_kv][page][d] for K
and for V with one f32 scale per page and kv head; table[s][j] is the page of
tokens j*page .. j*page+page-1 of sequence s (-1: none), len[s] its number of
tokens.  A pool has refs[p] beside that, the number of table entries that name
page p (0: free), for all layers alike.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
WS_BYTES = 96 << 20      # the workspace that a serving program keeps

H8B = (32, 8, 128)       # the 8B-shaped layer of the benchmark: query heads, kv heads, head size
HSMALL = (14, 2, 64)     # hidden 896


def _attn(name, dtype, n_seq, new, len_min, len_max, heads, page, cap=0.0, bias=False, doc=0, prefix=0, window=0, sinks=0,
          ragged=False, idle=False):
    n_q, n_kv, d = heads
    return {"name": name, "op": "attn", "dtype": dtype, "n_seq": n_seq, "new": new, "len_min": len_min, "len_max": len_max,
            "n_q": n_q, "n_kv": n_kv, "d": d, "page": page, "cap": cap, "bias": bias, "doc": doc, "prefix": prefix,
            "window": window, "sinks": sinks, "ragged": ragged, "idle": idle}


def _pool(name, op, layers, heads, page, n_seq, len_min, len_max, blocks, share=1, new=1, part=1.0, spare=0.25):
    """share: sequences of one parent; new: tokens that a sequence asks room for; part: sequences that the pass is about;
    spare: free pages over all pages."""
    return {"name": name, "op": op, "layers": layers, "n_kv": heads[1], "d": heads[2], "page": page, "n_seq": n_seq,
            "len_min": len_min, "len_max": len_max, "blocks": blocks, "share": share, "new": new, "part": part, "spare": spare}


def listed():
    return [
        # one user's decode step with capped scores, q in f32 as the mat-vec writes it
        _attn("cap_step_1x4096", "f32", 1, 1, 4096, 4096, H8B, 64, cap=50.0),
        # a serving batch of mixed contexts, heads biased by distance, small pages, idle slots
        _attn("bias_step_64_ragged", "bf16", 64, 1, 64, 16384, H8B, 16, bias=True, idle=True),
        # decode steps of a sliding-window layer with capped scores
        _attn("cap_step_window", "f16", 32, 1, 1000, 32768, H8B, 32, cap=50.0, window=4096),
        # a prompt chunk behind a long cached prefix, capped scores
        _attn("cap_chunk_2048", "bf16", 1, 2048, 10240, 10240, H8B, 64, cap=30.0),
        # documents packed into long prompts, the first tokens of each seen from all of it
        _attn("documents_4096", "bf16", 2, 4096, 4096, 4096, H8B, 64, doc=700, prefix=100),
        # prompts of odd lengths with a prefix seen whole and biased heads
        _attn("prefix_prompts_ragged", "f16", 4, 2000, 500, 2000, HSMALL, 128, bias=True, prefix=257, ragged=True),
        # a beam search of 4 beams goes on from its best beam: tables shared, the page in progress copied
        _pool("beam_step_4", "fork", 24, HSMALL, 32, 4, 1000, 1000, 64, share=4),
        # 32 prompts sampled 8 times each
        _pool("sample_32x8", "fork", 32, H8B, 32, 256, 500, 2000, 72, share=8),
        # drafted tokens taken back and room for the next ones made in each sequence
        _pool("draft_rollback_16", "turnover", 24, HSMALL, 16, 16, 100, 5000, 512, new=5),
        # a quarter of a large batch is finished and makes room for new prompts
        _pool("turnover_1024", "turnover", 32, H8B, 16, 1024, 200, 16384, 2048, new=3000, part=0.25),
        # a small model's pool gives back its upper half
        _pool("compact_small", "compact", 24, HSMALL, 32, 24, 100, 3000, 128, spare=0.5),
        # a large model's pool gives back a third
        _pool("compact_8b", "compact", 32, H8B, 64, 16, 500, 4000, 128, spare=0.35),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    cases = listed()
    while True:
        if rng.random() < 0.5:
            c = _draw_attn(rng)
            like = [x for x in cases if x["op"] == "attn"]
        else:
            c = _draw_pool(rng)
            like = [x for x in cases if x["op"] != "attn"]
        w = work(c)
        if all(w[k] <= max(work(x)[k] for x in like) for k in w) and _extent(c) <= max(_extent(x) for x in like):
            del c["name"]
            return c


def _extent(c):
    """What the plain form or the inputs hold at once: scores of every sequence, or bytes of the pool."""
    if c["op"] == "attn":
        return c["n_seq"] * c["len_max"] * max(c["new"] * c["n_q"], 2 * c["n_kv"] * c["d"])
    return _pages(c)[1] * c["layers"] * c["n_kv"] * c["page"] * c["d"] if c["op"] != "turnover" else 0


def _draw_attn(rng):
    dtype = rng.choice(["f32", "f16", "bf16"])
    heads = rng.choice([H8B, H8B, HSMALL, (12, 12, 64), (16, 1, 64), (20, 4, 128)])
    new = 1 if rng.random() < 0.5 else _log_int(rng, 2, 128 if dtype == "f32" else 4096)
    len_max = max(new, _log_int(rng, 16, 32768))
    kind = rng.choice(["cap", "bias", "prefix", "doc", "all"])
    windowed = rng.random() < 0.3
    return _attn("", dtype, _log_int(rng, 1, 64), new, rng.randint(max(1, len_max // 64), len_max), len_max, heads,
                 rng.choice([16, 32, 64, 128]), cap=rng.choice([20.0, 30.0, 50.0]) if kind in ("cap", "all") else 0.0,
                 bias=kind in ("bias", "all"), doc=_log_int(rng, 30, 3000) if kind in ("doc", "all") else 0,
                 prefix=_log_int(rng, 1, 600) if kind in ("prefix", "all") or (kind == "doc" and rng.random() < 0.5) else 0,
                 window=_log_int(rng, 16, 8192) if windowed else 0, sinks=rng.randint(0, 70) if windowed else 0,
                 ragged=new > 1 and rng.random() < 0.6, idle=rng.random() < 0.3)


def _draw_pool(rng):
    op = rng.choice(["fork", "turnover", "compact"])
    heads = rng.choice([H8B, HSMALL, (12, 12, 64), (16, 1, 64), (20, 4, 128)])
    page = rng.choice([16, 32, 64, 128])
    share = rng.randint(2, 9) if op == "fork" else 1
    n_seq = _log_int(rng, 1, 256 if op == "fork" else 1024 if op == "turnover" else 64) * share
    len_max = _log_int(rng, 20, 16384 if op == "turnover" else 4000)
    new = _log_int(rng, 1, 3000) if op == "turnover" else rng.choice([1, 1, 4, 40])
    return _pool("", op, rng.randint(1, 32), heads, page, n_seq, rng.randint(max(1, len_max // 32), len_max), len_max,
                 -(-(len_max + new) // page) + rng.randint(0, 9), share=share, new=new,
                 part=rng.choice([1.0, 0.5, 0.25]), spare=rng.uniform(0.1, 0.6))


def _lens(c):
    """Tokens of each sequence: spread over [len_min, len_max], the first the longest."""
    out = []
    for i in range(c["n_seq"]):
        f = 1.0 if i == 0 else (i * 0.6180339887) % 1.0
        n = round(c["len_min"] * (c["len_max"] / c["len_min"]) ** f)
        out.append(0 if c.get("idle") and i % 8 == 5 else n)
    return out


# ---------------------------------------------------------------- attention: rows and what they see

def _news(c):
    """Rows of each sequence (one each in a decode step, idle slots included)."""
    if c["new"] == 1:
        return [1] * c["n_seq"]
    out = []
    for i, n in enumerate(_lens(c)):
        m = c["new"] if i == 0 or not c["ragged"] else 1 + int((c["new"] - 1) * ((i * 0.7548776662) % 1.0))
        out.append(min(n, m))
    return out


def _bounds(c):
    """(position, first token, end of the prefix) of every row: documents of doc/2 .. 2 doc tokens one after the other, or one."""
    rows = []
    for s, (n, m) in enumerate(zip(_lens(c), _news(c))):
        starts, k = [0], s
        while c["doc"] and starts[-1] < n:
            k += 1
            starts.append(starts[-1] + max(1, round(c["doc"] * 4.0 ** ((k * 0.6180339887) % 1.0 - 0.5))))
        at = 0
        for p in range(n - m, n):
            while at + 1 < len(starts) and starts[at + 1] <= p:
                at += 1
            end = starts[at] + c["prefix"]
            rows.append((p, starts[at], min(end, starts[at + 1] if at + 1 < len(starts) else n, n)))
    return rows


def _attn_work(c):
    e, d, pairs, seen = SIZES[c["dtype"]], c["d"], 0, 0
    rows, at = _bounds(c), 0
    for n, m in zip(_lens(c), _news(c)):
        spans = []
        for p, first, end in rows[at:at + m]:
            if p < 0:
                continue
            lo = max(first, p - c["window"] + 1) if c["window"] else first
            parts = [(lo, max(p + 1, end))]
            extra = min(c["sinks"] if c["window"] else 0, lo) - first
            if c["window"] and extra > 0:
                parts.append((first, first + extra))
            if c["window"] and min(end, lo) > max(first, min(c["sinks"], lo)):
                parts.append((max(first, min(c["sinks"], lo)), min(end, lo)))
            pairs += sum(b - a for a, b in parts)
            spans += parts
        at += m
        # tokens that some row of the sequence sees
        reach = 0
        for a, b in sorted(spans):
            seen += max(0, b - max(a, reach))
            reach = max(reach, b)
    return {"bytes": 2 * len(rows) * c["n_q"] * d * e + seen * 2 * c["n_kv"] * d + 8 * c["n_kv"] * (seen // c["page"] + 1),
            "flops": 4 * d * c["n_q"] * pairs}


# ---------------------------------------------------------------- the pool's layout

def _held(c):
    """Blocks that each sequence holds pages for at the start, and tokens it asks room for."""
    page, out = c["page"], []
    for i, n in enumerate(_lens(c)):
        if c["op"] == "fork":
            out.append((-(-n // page) if i % c["share"] == 0 else 0, c["new"]))
        elif c["op"] == "turnover":
            # a drafted sequence holds room for its draft
            out.append((-(-(n + (c["new"] if c["part"] == 1.0 else 0)) // page), c["new"] if _about(c, i) else 0))
        else:
            out.append((-(-n // page), 0))
    return out


def _about(c, i):
    return (i * c["part"]) % 1.0 < c["part"] - 1e-9 if c["part"] < 1.0 else True


def _pages(c):
    """Pages in use at the start, all pages, and how many of those in use lie above what they need."""
    held = _held(c)
    used = sum(h for h, _ in held)
    room = sum(-(-new // c["page"]) + 1 for _, new in held)
    n_pages = max(used + room, round(used / (1.0 - c["spare"]))) + 1
    return used, n_pages, round(used * (n_pages - used) / n_pages)


def _pool_work(c):
    page, lens = c["page"], _lens(c)
    token = 2 * c["n_kv"] * c["d"] * c["layers"]         # bytes of a token in all layers
    scales = 8 * c["n_kv"] * c["layers"]
    used, n_pages, high = _pages(c)
    if c["op"] == "compact":
        return {"bytes": 2 * high * (page * token + scales) + 8 * n_pages + 4 * c["n_seq"] * c["blocks"] + 4 * high, "flops": 0}
    if c["op"] == "fork":
        total = 0
        for i, n in enumerate(lens):
            n = lens[i - i % c["share"]]
            fresh = -(-(n + c["new"]) // page) - n // page
            if i % c["share"]:
                # its row is written, its pages counted, the part of a page that it shares copied
                total += -(-n // page) * (4 + 4 + 8) + (2 * (n % page) * token + 2 * scales if n % page else 0)
            total += fresh * 12
        return {"bytes": total, "flops": 0}
    total = 0
    for i, (held, new) in enumerate(_held(c)):
        if not new:
            continue
        keep = lens[i] if c["part"] == 1.0 else 0
        freed = max(0, held - -(-keep // page))
        fresh = -(-(keep + new) // page) - -(-keep // page)
        total += 16 + freed * 16 + fresh * 12
    return {"bytes": total, "flops": 0}


def work(c):
    return _attn_work(c) if c["op"] == "attn" else _pool_work(c)


# ---------------------------------------------------------------- inputs

def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_attn(c, g) if c["op"] == "attn" else _prepare_pool(c, g)


def _codes(shape, g):
    c8 = torch.empty(shape, dtype=torch.int8, device=g.device)
    flat = c8.view(-1)
    for i in range(0, flat.numel(), 64 << 20):
        part = flat[i:i + (64 << 20)]
        part.copy_((torch.randn(part.shape, generator=g, device=g.device) * 30).round().clamp(-127, 127))
    return c8


def _scales(shape, g):
    return (torch.randn(shape, generator=g, device=g.device) * 0.2).exp() * 0.033


def _rows_of(order, counts, width):
    """A table whose row s names the next counts[s] pages of `order`."""
    counts = torch.tensor(counts, device=order.device)
    at, col = torch.cumsum(counts, 0) - counts, torch.arange(width, device=order.device)
    index = (at[:, None] + col).clamp(max=max(order.numel() - 1, 0))
    return torch.where(col < counts[:, None], order[index], torch.full_like(order[:1], -1)).contiguous()


def _prepare_attn(c, g):
    dev, dt = g.device, DTYPES[c["dtype"]]
    lens, news = _lens(c), _news(c)
    n_q, n_kv, d, page = c["n_q"], c["n_kv"], c["d"], c["page"]
    counts = [-(-n // page) for n in lens]
    used = max(1, sum(counts))
    n_pages = used + 1                   # the last page stays free
    # pages in the scattered order that a pool hands them out
    order = torch.randperm(used, generator=g, device=dev).to(torch.int32)
    rows = sum(news)
    starts = [0]
    for m in news:
        starts.append(starts[-1] + m)
    bounds = _bounds(c)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    # heads' slopes fall geometrically from 1/2 to 2^-8, as they are chosen for distance biases
    slope = 2.0 ** (-8.0 * (torch.arange(n_q, dtype=torch.float64, device=dev) + 1) / n_q)
    return {"case": c, "k": _codes((n_pages, n_kv, page, d), g), "v": _codes((n_pages, n_kv, page, d), g),
            "ks": _scales((n_pages, n_kv), g), "vs": _scales((n_pages, n_kv), g),
            "table": _rows_of(order, counts, max(1, max(counts))), "len": ints(lens),
            # the fused projection's output, [q | k | v] in each row: scores of +-4 and up to some 18, which a cap bends
            "qkv": (torch.randn(rows, (n_q + 2 * n_kv) * d, generator=g, device=dev) * 4.0).to(dt),
            "rows": rows, "row_start": ints(starts), "max_new": max(news),
            "slope": slope.float() if c["bias"] else None, "first": ints([b[1] for b in bounds]) if c["doc"] else None,
            "prefix": ints([b[2] for b in bounds]) if c["prefix"] else None,
            "ws": torch.zeros(WS_BYTES, dtype=torch.uint8, device=dev),
            "out": torch.empty(rows, n_q * d, dtype=dt, device=dev)}


def _prepare_pool(c, g):
    dev, n_seq = g.device, c["n_seq"]
    lens, held = _lens(c), _held(c)
    used, n_pages, high = _pages(c)
    # the pages in use lie scattered over the pool, `high` of them above the first `used`
    low = torch.randperm(used, generator=g, device=dev)[:used - high]
    up = torch.randperm(n_pages - used, generator=g, device=dev)[:high] + used
    order = torch.cat([low, up])[torch.randperm(used, generator=g, device=dev)].to(torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    refs[order.long()] = 1
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    shape = (c["layers"], n_pages, c["n_kv"])
    moves = c["op"] != "turnover"        # a turnover touches no codes
    s = {"case": c, "table": _rows_of(order, [h for h, _ in held], c["blocks"]), "refs": refs,
         "len": ints([n if h else 0 for n, (h, _) in zip(lens, held)]), "new": ints([a for _, a in held]),
         "k": _codes(shape + (c["page"], c["d"]), g) if moves else None,
         "v": _codes(shape + (c["page"], c["d"]), g) if moves else None,
         "ks": _scales(shape, g) if moves else None, "vs": _scales(shape, g) if moves else None,
         "status": torch.zeros(2, dtype=torch.int32, device=dev),
         "ws": torch.zeros(WS_BYTES, dtype=torch.uint8, device=dev)}
    if c["op"] == "fork":
        children = [i for i in range(n_seq) if i % c["share"]]
        s["to"], s["from"] = ints(children), ints([i - i % c["share"] for i in children])
    elif c["op"] == "turnover":
        s["seq"] = ints([i for i in range(n_seq) if _about(c, i)])
        # a drafted sequence keeps its tokens, a finished one none
        s["begin"] = s["len"].clone() if c["part"] == 1.0 else None
    else:
        s["table0"], s["refs0"] = s["table"].clone(), s["refs"].clone()
        s["moved"] = torch.empty(n_pages, dtype=torch.int32, device=dev)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return {"attn": _own_attn, "fork": _own_fork, "turnover": _own_turnover, "compact": _own_compact}[op](s)
    return {"attn": _plain_attn, "fork": _plain_fork, "turnover": _plain_turnover, "compact": _plain_compact}[op](s)


# ---------------------------------------------------------------- the framework's calls

def _own_attn(s):
    import quantized_weight_mat_gb300 as pq
    c = s["case"]
    if "cache" not in s:      # the handles on the program's own buffers, made once
        s["cache"] = pq.pq_kv_cache(s["k"], s["v"], s["ks"], s["vs"], s["table"], s["len"], s["k"].shape[0],
                                    c["n_kv"], c["page"], c["d"], c["n_seq"], s["table"].shape[1])
        s["mod"] = pq.pq_score_mod(cap=c["cap"], slope=s["slope"], first=s["first"], prefix=s["prefix"])
    start = None if c["new"] == 1 else s["row_start"]
    pq.pq_attn_mod(s["cache"], start, s["rows"], c["dtype"], s["qkv"], s["qkv"].shape[1], c["n_q"], c["d"] ** -0.5,
                   c["window"], c["sinks"], s["mod"], s["out"], c["n_q"] * c["d"], s["ws"], WS_BYTES)
    return s["out"]


def _own_pool(s):
    import quantized_weight_mat_gb300 as pq
    c = s["case"]
    if "pool" not in s:
        n_pages = s["refs"].shape[0]
        s["pool"] = pq.pq_kv_pool(s["refs"], s["table"], s["len"], n_pages, c["page"], c["n_seq"], c["blocks"])
        s["layers"] = pq.pq_kv_layers([
            pq.pq_kv_cache(s["k"][i], s["v"][i], s["ks"][i], s["vs"][i], s["table"], s["len"], n_pages, c["n_kv"],
                           c["page"], c["d"], c["n_seq"], c["blocks"])
            for i in range(c["layers"])]) if s["k"] is not None else None
    return pq, s["pool"], s["layers"]


def _own_fork(s):
    pq, pool, layers = _own_pool(s)
    pq.pq_kv_fork(pool, s["to"].numel(), s["from"], s["to"], None, s["ws"], WS_BYTES)
    pq.pq_kv_reserve(pool, layers, s["new"], s["status"], s["ws"], WS_BYTES)
    # codes move as they are, so they are returned as they are
    return s["table"], s["refs"], s["len"], s["status"], s["k"], s["v"], s["ks"], s["vs"]


def _own_turnover(s):
    pq, pool, layers = _own_pool(s)
    pq.pq_kv_free(pool, s["seq"].numel(), s["seq"], s["begin"], None)
    pq.pq_kv_reserve(pool, layers, s["new"], s["status"], s["ws"], WS_BYTES)
    return s["table"], s["refs"], s["len"], s["status"]


def _own_compact(s):
    pq, pool, layers = _own_pool(s)
    # scattered again, since a compacted pool has nothing to move
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    pq.pq_kv_compact(pool, layers, s["moved"], s["status"], s["ws"], WS_BYTES)
    return s["table"], s["refs"], s["moved"], s["status"][:1], s["k"], s["v"], s["ks"], s["vs"]


# ---------------------------------------------------------------- plain forms: attention

def _plain_attn(s):
    c = s["case"]
    n_q, n_kv, d, page, n_seq = c["n_q"], c["n_kv"], c["d"], c["page"], c["n_seq"]
    grp, most, dev = n_q // n_kv, s["max_new"], s["qkv"].device
    pages = s["table"].long()                                   # -1 is the free page, never visible
    width = pages.shape[1] * page

    def dense(codes, scale):
        x = codes[pages].float() * scale[pages][..., None, None]
        return x.transpose(1, 2).reshape(n_seq, n_kv, width, d)

    n = (s["row_start"][1:] - s["row_start"][:-1]).long()
    i = torch.arange(most, device=dev)
    row = (s["row_start"][:-1].long()[:, None] + i).clamp(max=s["rows"] - 1)
    pos = torch.where(i < n[:, None], s["len"].long()[:, None] - n[:, None] + i, torch.full_like(row, -1))
    q = s["qkv"][:, :n_q * d].float()[row].reshape(n_seq, most, n_kv, grp, d)
    q = q.permute(0, 2, 3, 1, 4)                                # [n_seq, n_kv, grp, most, d]
    t = torch.arange(width, device=dev)
    at = pos[..., None]                                         # [n_seq, most, 1]
    see = t <= at
    if c["window"]:
        see = see & ((at - t < c["window"]) | (t < c["sinks"]))
    if s["prefix"] is not None:
        see = see | ((t < s["prefix"].long()[row][..., None]) & (t < s["len"].long()[:, None, None]) & (at >= 0))
    if s["first"] is not None:
        see = see & (t >= s["first"].long()[row][..., None])
    x = torch.matmul(q, dense(s["k"], s["ks"])[:, :, None].transpose(3, 4)) * d ** -0.5
    if c["cap"]:
        x = torch.tanh(x / c["cap"]) * c["cap"]
    if s["slope"] is not None:
        x = x - s["slope"].reshape(n_kv, grp, 1, 1) * (at - t).abs()[:, None, None].float()
    x = torch.where(see[:, None, None], x, torch.full((), -math.inf, device=dev))
    top = x.amax(4, keepdim=True)
    x = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = x.sum(4, keepdim=True)
    y = torch.matmul(x, dense(s["v"], s["vs"])[:, :, None]) / torch.where(total > 0, total, torch.ones_like(total))
    y = y.permute(0, 3, 1, 2, 4).reshape(n_seq * most, n_q * d)
    # back from [sequence][row] to the rows' own order
    seq = torch.repeat_interleave(torch.arange(n_seq, device=dev), n, output_size=s["rows"])
    back = seq * most + torch.arange(s["rows"], device=dev) - s["row_start"].long()[seq]
    return y[back].to(s["qkv"].dtype)


# ---------------------------------------------------------------- plain forms: the pool

def _count(refs, table, by):
    """refs[p] += by for every entry of `table` that names a page."""
    p = table.reshape(-1).long()
    ok = (p >= 0) & (p < refs.shape[0])
    refs.index_add_(0, torch.where(ok, p, torch.zeros_like(p)), ok.to(refs.dtype) * by)


def _fork(s):
    table, size = s["table"], s["case"]["page"]
    frm, to = s["from"].long(), s["to"].long()
    m = s["len"][frm].clamp(min=0)
    col = torch.arange(table.shape[1], device=table.device)
    rows = torch.where(col * size < m[:, None], table[frm], torch.full_like(table[:1], -1))
    _count(s["refs"], rows, 1)
    _count(s["refs"], table[to], -1)
    table[to] = rows
    s["len"][to] = m


def _reserve(s):
    c, table, refs, n = s["case"], s["table"], s["refs"], s["len"].clamp(min=0)
    size, n_seq, width = c["page"], c["n_seq"], s["table"].shape[1]
    n_pages = refs.shape[0]
    first, last = n // size, (n + s["new"] - 1) // size
    wants = s["new"] > 0
    fits = last < width
    col, seq = torch.arange(width, device=table.device), torch.arange(n_seq, device=table.device)
    asked = (col >= first[:, None]) & (col <= last[:, None]) & (wants & fits)[:, None]
    page = table.long()
    there = (page >= 0) & (page < n_pages)
    at = torch.where(there, page, torch.zeros_like(page))
    writes = asked & there
    # of the sequences that write a page, the lowest keeps it if nobody else holds it
    writers = torch.zeros_like(refs).index_add_(0, at.reshape(-1), writes.reshape(-1).to(refs.dtype))
    lowest = torch.full((n_pages,), n_seq, device=table.device).scatter_reduce_(
        0, at.reshape(-1), torch.where(writes, seq[:, None], torch.full_like(page, n_seq)).reshape(-1), "amin")
    shared = writes & (refs[at] > 1)
    shared = shared & ~((writers[at] == refs[at]) & (lowest[at] == seq[:, None]))
    fresh = (asked & ~there) | shared
    free = torch.nonzero(refs <= 0).reshape(-1)
    short = (fresh.sum() - free.numel()).clamp(min=0)
    narrow = (wants & ~fits).sum()
    s["status"].copy_(torch.stack([short, narrow]))
    fresh = fresh & (short == 0) & (narrow == 0)
    where = torch.nonzero(fresh)                               # in order of sequence and block
    new = free[:where.shape[0]]
    r, j = where[:, 0], where[:, 1]
    old, held = at[r, j], there[r, j]
    refs.index_add_(0, old, -held.to(refs.dtype))
    refs[new] = 1
    table[r, j] = new.to(table.dtype)
    if s["k"] is None:
        return
    # tokens that the sequence has in the page go along
    count = torch.where(held, (n[r] - j * size).clamp(0, size), torch.zeros_like(old))
    moves = torch.nonzero(count > 0).reshape(-1)
    src, dst, count = old[moves], new[moves], count[moves]
    slot = (torch.arange(size, device=table.device) < count[:, None])[None, :, None, :, None]
    for codes, scale in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        codes[:, dst] = torch.where(slot, codes[:, src], codes[:, dst])
        scale[:, dst] = scale[:, src]


def _plain_fork(s):
    _fork(s)
    _reserve(s)
    return s["table"], s["refs"], s["len"], s["status"], s["k"], s["v"], s["ks"], s["vs"]


def _plain_turnover(s):
    c, table, seq = s["case"], s["table"], s["seq"].long()
    n = s["len"][seq]
    keep = s["begin"].clamp(min=0) if s["begin"] is not None else torch.zeros_like(n)
    col = torch.arange(table.shape[1], device=table.device)
    out = col * c["page"] >= keep[:, None]
    rows = table[seq]
    _count(s["refs"], torch.where(out, rows, torch.full_like(rows, -1)), -1)
    table[seq] = torch.where(out, torch.full_like(rows, -1), rows)
    s["len"][seq] = torch.minimum(n, keep)
    _reserve(s)
    return s["table"], s["refs"], s["len"], s["status"]


def _plain_compact(s):
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    table, refs = s["table"], s["refs"]
    n_pages = refs.shape[0]
    live = refs > 0
    ids = torch.arange(n_pages, device=refs.device)
    up = ids >= live.sum()
    src, dst = torch.nonzero(live & up).reshape(-1), torch.nonzero(~live & ~up).reshape(-1)
    moved = torch.where(live, ids, torch.full_like(ids, -1))
    moved[src] = dst
    s["moved"].copy_(moved)
    refs[dst] = refs[src]
    refs[src] = 0
    page = table.long()
    there = (page >= 0) & (page < n_pages)
    to = moved[torch.where(there, page, torch.zeros_like(page))]
    table.copy_(torch.where(there & (to >= 0), to, page))
    for x in (s["k"], s["v"], s["ks"], s["vs"]):
        x[:, dst] = x[:, src]
    s["status"][:1].copy_(live.sum())
    return s["table"], s["refs"], s["moved"], s["status"][:1], s["k"], s["v"], s["ks"], s["vs"]


# ---------------------------------------------------------------- 64 bits

def exact(c, seed):
    """Attention in 64 bits, one sequence and query head at a time; pages are moved and counted, nothing is computed there."""
    if c["op"] != "attn":
        return None
    s = prepare(c, seed)
    n_q, n_kv, d, page = c["n_q"], c["n_kv"], c["d"], c["page"]
    lens, starts = s["len"].tolist(), s["row_start"].tolist()
    out = torch.zeros(s["rows"], n_q, d, dtype=torch.float64, device=s["qkv"].device)
    for i, n in enumerate(lens):
        r0, r1 = starts[i], starts[i + 1]
        if n == 0 or r1 == r0:
            continue
        t = torch.arange(n, device=out.device)
        pid = s["table"][i, t // page].long()
        p = t[n - (r1 - r0):, None]
        ahead, far = t > p, torch.zeros(1, dtype=torch.bool, device=out.device)
        if c["window"]:
            far = (t <= p - c["window"]) & (t >= c["sinks"])
        hidden = ahead | far
        if s["prefix"] is not None:
            hidden &= t >= s["prefix"][r0:r1, None]
        if s["first"] is not None:
            hidden |= t < s["first"][r0:r1, None]
        for h in range(n_kv):
            k = s["k"][pid, h, t % page].double() * s["ks"][pid, h].double()[:, None]
            v = s["v"][pid, h, t % page].double() * s["vs"][pid, h].double()[:, None]
            for j in range(h * n_q // n_kv, (h + 1) * n_q // n_kv):
                x = s["qkv"][r0:r1, j * d:(j + 1) * d].double() @ k.T / math.sqrt(d)
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if c["bias"]:
                    x -= s["slope"][j].double() * (p - t).abs()
                x = torch.exp_(x.masked_fill_(hidden, -math.inf).sub_(x.amax(1, keepdim=True)))
                out[r0:r1, j] = (x @ v) / x.sum(1, keepdim=True)
    return out.flatten(1)
