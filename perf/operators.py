"""Cases and plain forms of the 8-bit paged-cache operators: appending keys and
values with the position rotation on the way, reading cached tokens back, and
attention over the cache (causal, optionally with a sliding window and first
tokens that stay visible).

A cache holds pages of `page` tokens: int8 codes [n_pages][n_kv][page][d] for K
and for V with one f32 scale per page and kv head; table[s][j] is the page of
tokens j*page .. j*page+page-1 of sequence s, len[s] its number of tokens, the
rows of this call included: row i of the n_s rows of sequence s is the token at
position len[s] - n_s + i.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
WS_BYTES = 64 << 20      # the attention workspace a serving program keeps


def _case(name, op, dtype, n_seq, new, len_min, len_max, heads, page, rope="half", rot=None, window=0, sinks=0,
          ragged=False, idle=False):
    n_q, n_kv, d = heads
    return {"name": name, "op": op, "dtype": dtype, "n_seq": n_seq, "new": new, "len_min": len_min,
            "len_max": len_max, "n_q": n_q, "n_kv": n_kv, "d": d, "page": page, "rope": rope,
            "rot": d if rot is None else rot, "window": window, "sinks": sinks, "ragged": ragged, "idle": idle}


H8B = (32, 8, 128)       # the 8B-shaped layer of the benchmark
HSMALL = (14, 2, 64)     # hidden 896: 14 query heads, 2 kv heads


def listed():
    return [
        # one user's decode step, q/k/v in f32 as the mat-vec writes them
        _case("append_step_1", "append", "f32", 1, 1, 1000, 1000, H8B, 64),
        # a full serving batch, one token each, some slots idle
        _case("append_step_128", "append", "bf16", 128, 1, 17, 2048, H8B, 16, idle=True),
        # several prompts of odd lengths behind cached prefixes, part of each head rotated
        _case("append_prompts_ragged", "append", "f16", 7, 777, 300, 1500, HSMALL, 32, rope="pair", rot=32, ragged=True),
        # a long prompt from its first token
        _case("append_prompt_8192", "append", "bf16", 1, 8192, 8192, 8192, H8B, 64),
        # one user's decode step at a middling context
        _case("attn_step_1x4096", "attn", "f32", 1, 1, 4096, 4096, H8B, 64),
        # one user with a very long context
        _case("attn_step_1x131072", "attn", "bf16", 1, 1, 131072, 131072, H8B, 64),
        # a serving batch of mixed contexts, small pages, idle slots
        _case("attn_step_64_ragged", "attn", "bf16", 64, 1, 64, 16384, H8B, 16, idle=True),
        # a sliding-window layer with sink tokens
        _case("attn_step_window", "attn", "f16", 32, 1, 1000, 65536, H8B, 32, window=4096, sinks=4),
        # checking five drafted tokens in each sequence
        _case("attn_verify_5", "attn", "f32", 16, 5, 100, 5000, HSMALL, 16),
        # a prompt piece as wide as the mat-vec's widest pass
        _case("attn_piece_32", "attn", "f32", 1, 32, 2500, 2500, H8B, 64),
        # a prompt chunk behind a long cached prefix
        _case("attn_chunk_2048", "attn", "bf16", 1, 2048, 10240, 10240, H8B, 64),
        # prompts of a sliding-window layer, odd lengths
        _case("attn_prompts_window", "attn", "f16", 4, 4096, 1000, 4096, HSMALL, 128, window=1024, sinks=4, ragged=True),
    ]


def _log_int(rng, lo, hi):
    n = min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
    return n + 1 if n == 3 << 10 else n


def draw(rng):
    most = [max(work(c)[k] for c in listed()) for k in ("bytes", "flops")]
    while True:
        op = rng.choice(["append", "attn", "attn"])
        dtype = rng.choice(["f32", "f16", "bf16"])
        heads = rng.choice([H8B, H8B, HSMALL, (12, 12, 64), (16, 1, 64), (20, 4, 128)])
        n_seq = _log_int(rng, 1, 128)
        new = 1 if rng.random() < 0.5 else _log_int(rng, 2, 128 if dtype == "f32" else 4096)
        len_max = max(new, _log_int(rng, 16, 131072 if op == "attn" else 8192))
        len_min = rng.randint(max(1, len_max // 64), len_max)
        windowed = op == "attn" and rng.random() < 0.4
        c = _case("", op, dtype, n_seq, new, len_min, len_max, heads, rng.choice([16, 32, 64, 128]),
                  rope=rng.choice(["half", "pair"]), rot=rng.choice([heads[2], heads[2] // 2]),
                  window=_log_int(rng, 16, 8192) if windowed else 0, sinks=rng.randint(0, 70) if windowed else 0,
                  ragged=new > 1 and rng.random() < 0.6, idle=rng.random() < 0.3)
        del c["name"]
        # the padded plain form keeps every sequence's scores at once
        padded = n_seq * len_max * max(new * heads[0], 2 * heads[1] * heads[2])
        w = work(c)
        if w["bytes"] <= most[0] and w["flops"] <= most[1] and padded <= 6e9 and sum(_lens(c)) <= 700_000:
            return c


def _lens(c):
    """Tokens of each sequence: spread over [len_min, len_max], the first the longest."""
    out = []
    for i in range(c["n_seq"]):
        f = 1.0 if i == 0 else (i * 0.6180339887) % 1.0
        n = round(c["len_min"] * (c["len_max"] / c["len_min"]) ** f)
        out.append(0 if c["idle"] and i % 8 == 5 else n)
    return out


def _news(c):
    """Rows of each sequence (one each in a decode step, idle slots included)."""
    if c["new"] == 1:
        return [1] * c["n_seq"]
    out = []
    for i, n in enumerate(_lens(c)):
        m = c["new"] if i == 0 or not c["ragged"] else 1 + int((c["new"] - 1) * ((i * 0.7548776662) % 1.0))
        out.append(min(n, m))
    return out


def _visible(c, pos):
    """How many tokens the row at this position sees."""
    if pos < 0:
        return 0
    if not c["window"] or pos + 1 <= c["window"]:
        return pos + 1
    return c["window"] + min(c["sinks"], pos + 1 - c["window"])


def work(c):
    e, lens, news = SIZES[c["dtype"]], _lens(c), _news(c)
    n_q, n_kv, d, page = c["n_q"], c["n_kv"], c["d"], c["page"]
    rows = sum(news)
    if c["op"] == "append":
        # q, k, v in; rotated q, codes and scales out; the touched blocks read back as values
        back = sum(n - (n - m) // page * page for n, m in zip(lens, news) if n)
        return {"bytes": rows * d * (2 * n_q * e + 2 * n_kv * e + 2 * n_kv) + back * 2 * n_kv * d * (1 + e),
                "flops": rows * d * (3 * n_q + 7 * n_kv) + back * 2 * n_kv * d}
    pairs, seen = 0, 0
    for n, m in zip(lens, news):
        first = n - m
        if n == 0 or m == 0:
            continue
        pairs += sum(_visible(c, p) for p in range(max(first, 0), n))
        # tokens that some row of the sequence sees
        lo = max(0, first - c["window"] + 1) if c["window"] else 0
        seen += n - lo + min(lo, c["sinks"])
    return {"bytes": 2 * rows * n_q * d * e + seen * 2 * n_kv * d + 8 * n_kv * (seen // page + 1),
            "flops": 4 * d * n_q * pairs}


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    lens, news = _lens(c), _news(c)
    n_q, n_kv, d, page, n_seq = c["n_q"], c["n_kv"], c["d"], c["page"], c["n_seq"]
    width = max(1, -(-max(lens) // page))
    used = sum(-(-n // page) for n in lens)
    n_pages = used + 1

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # pages in the scattered order that a pool hands them out; the last page stays free
    order = torch.randperm(used, generator=g, device=dev).to(torch.int32)
    counts = torch.tensor([-(-n // page) for n in lens], device=dev)
    at = torch.cumsum(counts, 0) - counts
    col = torch.arange(width, device=dev)
    index = (at[:, None] + col).clamp(max=used - 1)
    table = torch.where(col < counts[:, None], order[index], torch.full_like(order[:1], -1)).contiguous()

    def codes():
        c8 = torch.empty(n_pages, n_kv, page, d, dtype=torch.int8, device=dev)
        step = max(1, (64 << 20) // (n_kv * page * d))
        for i in range(0, n_pages, step):
            part = c8[i:i + step]
            part.copy_((normal(*part.shape) * 30).round().clamp(-127, 127))
        return c8

    def scales():
        return (normal(n_pages, n_kv) * 0.2).exp() * 0.033

    rows = sum(news)
    # the fused projection's output, [q | k | v] in each row
    qkv = normal(rows, (n_q + 2 * n_kv) * d).to(dt)
    starts = [0]
    for m in news:
        starts.append(starts[-1] + m)
    back = [n - (n - m) // page * page if n else 0 for n, m in zip(lens, news)]
    bstarts = [0]
    for m in back:
        bstarts.append(bstarts[-1] + m)
    half = c["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
    angle = torch.arange(max(lens) + 1, dtype=torch.float64, device=dev)[:, None] * inv
    s = {"case": c, "k": codes(), "v": codes(), "ks": scales(), "vs": scales(), "table": table,
         "len": torch.tensor(lens, dtype=torch.int32, device=dev), "qkv": qkv, "rows": rows,
         "k_new": qkv[:, n_q * d:], "v_new": qkv[:, (n_q + n_kv) * d:],
         "row_start": torch.tensor(starts, dtype=torch.int32, device=dev),
         "back": bstarts[-1], "back_start": torch.tensor(bstarts, dtype=torch.int32, device=dev),
         "cos": angle.cos().float(), "sin": angle.sin().float(), "max_len": max(lens), "max_new": max(news),
         "ws": torch.zeros(WS_BYTES, dtype=torch.uint8, device=dev),
         "out": torch.empty(rows, n_q * d, dtype=dt, device=dev),
         "k_back": torch.empty(bstarts[-1], n_kv * d, dtype=dt, device=dev),
         "v_back": torch.empty(bstarts[-1], n_kv * d, dtype=dt, device=dev)}
    return s


def run(s):
    c = s["case"]
    if own:
        return _own_append(s) if c["op"] == "append" else _own_attn(s)
    return _plain_append(s) if c["op"] == "append" else _plain_attn(s)


# ---------------------------------------------------------------- the framework's calls

def _own_cache(s):
    import quantized_weight_mat_gb300 as pq
    c = s["case"]
    if "cache" not in s:      # the handle on the program's own buffers, made once
        s["cache"] = pq.pq_kv_cache(s["k"], s["v"], s["ks"], s["vs"], s["table"], s["len"], s["k"].shape[0],
                                    c["n_kv"], c["page"], c["d"], c["n_seq"], s["table"].shape[1])
    return pq, c, s["cache"]


def _own_append(s):
    pq, c, cache = _own_cache(s)
    n_q, n_kv, d, qkv = c["n_q"], c["n_kv"], c["d"], s["qkv"]
    ld = qkv.shape[1]                       # q, k and v are columns of the same rows
    start = None if c["new"] == 1 else s["row_start"]
    pq.pq_kv_append(cache, start, s["rows"], c["dtype"], s["k_new"], ld, s["v_new"], ld, qkv, ld,
                    n_q, s["out"], n_q * d, s["cos"], s["sin"], s["cos"].shape[0], c["rot"], c["rope"])
    pq.pq_kv_gather(cache, s["back_start"], s["back"], c["dtype"], s["k_back"], n_kv * d, s["v_back"], n_kv * d)
    return s["out"], s["k_back"], s["v_back"]


def _own_attn(s):
    pq, c, cache = _own_cache(s)
    start = None if c["new"] == 1 else s["row_start"]
    pq.pq_attn(cache, start, s["rows"], c["dtype"], s["qkv"], s["qkv"].shape[1], c["n_q"], c["d"] ** -0.5,
               c["window"], c["sinks"], s["out"], c["n_q"] * c["d"], s["ws"], WS_BYTES)
    return s["out"]


# ---------------------------------------------------------------- plain forms

def _row_places(s, starts, rows):
    """Sequence and position of each of the rows."""
    n = (starts[1:] - starts[:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=starts.device), n, output_size=rows)
    pos = s["len"].long()[seq] - n[seq] + torch.arange(rows, device=starts.device) - starts.long()[seq]
    return seq, pos


def _rotate(x, cos, sin, rot, rope):
    """x [rows, heads, d] in f32, cos/sin [rows, rot/2]."""
    c, s, h = cos[:, None], sin[:, None], rot // 2
    y = x.clone()
    if rope == "half":
        a, b = x[..., :h], x[..., h:rot]
        y[..., :h], y[..., h:rot] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    return y


def _store(codes, scale, x, seq, pos, page_of, first_page, first_slot, page):
    """Quantizes x [rows, n_kv, d] into the blocks of its rows."""
    n_pages, n_kv = scale.shape
    full = torch.full((), 127.0, device=x.device)
    ok = (pos >= 0)[:, None]
    top = torch.zeros_like(scale).scatter_reduce(0, page_of[:, None].expand(-1, n_kv),
                                                 x.abs().amax(2) * ok, "amax") / full
    top = torch.where(top >= 2.0 ** -126, top, torch.zeros_like(top))
    # the older tokens of a sequence's first block keep the block's scale or are rescaled to the larger one
    old = torch.where((first_slot > 0)[:, None], scale[first_page], torch.zeros_like(scale[first_page]))
    new = torch.maximum(old, top[first_page])
    ratio = torch.where(new > 0, old / new, torch.ones_like(new))
    slot = torch.arange(page, device=x.device)
    before = (slot < first_slot[:, None])[:, None, :, None]
    was = codes[first_page]
    codes[first_page] = torch.where(before, (was * ratio[:, :, None, None]).round().to(torch.int8), was)
    scale[page_of] = torch.where(ok, top[page_of], scale[page_of])
    scale[first_page] = torch.where((first_slot >= 0)[:, None], new, scale[first_page])
    now = scale[page_of][:, :, None]
    inv = torch.where(now > 0, torch.ones_like(now) / now, torch.zeros_like(now))
    head = torch.arange(n_kv, device=x.device)
    put = (x * inv).round().clamp(-127, 127).to(torch.int8)
    at = (page_of[:, None], head, (pos % page)[:, None])
    codes[at] = torch.where(ok[:, :, None], put, codes[at])


def _plain_append(s):
    c = s["case"]
    n_q, n_kv, d, page, dt = c["n_q"], c["n_kv"], c["d"], c["page"], s["qkv"].dtype
    seq, pos = _row_places(s, s["row_start"], s["rows"])
    x = s["qkv"].float().reshape(s["rows"], n_q + 2 * n_kv, d)
    at = pos.clamp(min=0)
    qk = _rotate(x[:, :n_q + n_kv], s["cos"][at], s["sin"][at], c["rot"], c["rope"])
    # sequences without rows that reach the cache are sent to the free page at the end
    table = s["table"].long()
    n = (s["row_start"][1:] - s["row_start"][:-1]).long()
    start = s["len"].long() - n
    active = (n > 0) & (s["len"] > 0)
    first_page = torch.where(active, torch.gather(table, 1, (start.clamp(min=0) // page).clamp(
        max=table.shape[1] - 1)[:, None])[:, 0], torch.full_like(n, -1))
    first_slot = torch.where(active, start.clamp(min=0) % page, torch.full_like(n, -1))
    page_of = torch.where(pos >= 0, table[seq, at // page], torch.full_like(pos, -1)) % s["ks"].shape[0]
    first_page = first_page % s["ks"].shape[0]
    _store(s["k"], s["ks"], qk[:, n_q:], seq, pos, page_of, first_page, first_slot, page)
    _store(s["v"], s["vs"], x[:, n_q + n_kv:], seq, pos, page_of, first_page, first_slot, page)
    # read the touched blocks back
    bseq, bpos = _row_places(s, s["back_start"], s["back"])
    p, head = table[bseq, bpos // page], torch.arange(n_kv, device=x.device)
    where = (p[:, None], head, (bpos % page)[:, None])
    vals = [(codes[where].float() * scale[p][:, :, None]).reshape(s["back"], n_kv * d).to(dt)
            for codes, scale in ((s["k"], s["ks"]), (s["v"], s["vs"]))]
    # a row before the cache's first token is rotated as position 0
    return qk[:, :n_q].reshape(s["rows"], n_q * d).to(dt), vals[0], vals[1]


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
    q = q.permute(0, 2, 1, 3, 4).reshape(n_seq, n_kv, most * grp, d)
    t = torch.arange(width, device=dev)
    see = t <= pos[..., None]
    if c["window"]:
        see = see & ((pos[..., None] - t < c["window"]) | (t < c["sinks"]))
    see = see[:, None, :, None].expand(-1, -1, -1, grp, -1).reshape(n_seq, 1, most * grp, width)
    x = torch.matmul(q, dense(s["k"], s["ks"]).transpose(2, 3)) * d ** -0.5
    x = torch.where(see, x, torch.full((), -math.inf, device=dev))
    top = x.amax(3, keepdim=True)
    x = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = x.sum(3, keepdim=True)
    y = torch.matmul(x, dense(s["v"], s["vs"])) / torch.where(total > 0, total, torch.ones_like(total))
    y = y.reshape(n_seq, n_kv, most, grp, d).permute(0, 2, 1, 3, 4).reshape(n_seq * most, n_q * d)
    # back from [sequence][row] to the rows' own order
    seq = torch.repeat_interleave(torch.arange(n_seq, device=dev), n, output_size=s["rows"])
    back = seq * most + torch.arange(s["rows"], device=dev) - s["row_start"].long()[seq]
    return y[back].to(s["qkv"].dtype)


# ---------------------------------------------------------------- 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    return _exact_append(s) if c["op"] == "append" else _exact_attn(s)


def _exact_append(s):
    c = s["case"]
    n_q, n_kv, d, page = c["n_q"], c["n_kv"], c["d"], c["page"]
    x = s["qkv"].double().view(s["rows"], n_q + 2 * n_kv, d)
    lens, table, starts = s["len"].tolist(), s["table"].tolist(), s["row_start"].tolist()
    h, qs, ks, vs = c["rot"] // 2, [], [], []
    for i, n in enumerate(lens):
        r0, r1 = starts[i], starts[i + 1]
        if r1 == r0:
            continue
        first = n - (r1 - r0)
        p = torch.arange(first, n, device=x.device).clamp(min=0)
        z = torch.complex(s["cos"].double()[p], s["sin"].double()[p])[:, None]
        part = x[r0:r1, :n_q + n_kv, :c["rot"]]
        pair = (part.unflatten(2, (2, h)).transpose(2, 3) if c["rope"] == "half" else part.unflatten(2, (h, 2)))
        turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
        turned = (turned.transpose(2, 3) if c["rope"] == "half" else turned).flatten(2)
        qk = torch.cat([turned, x[r0:r1, :n_q + n_kv, c["rot"]:]], 2)
        qs.append(qk[:, :n_q].flatten(1))
        if n == 0:
            continue
        for new, codes, scale, out in ((qk[:, n_q:], s["k"], s["ks"], ks), (x[r0:r1, n_q + n_kv:], s["v"], s["vs"], vs)):
            for b in range(first // page, -(-n // page)):
                lo, hi = max(first, b * page), min(n, (b + 1) * page)
                fresh, pid = new[lo - first:hi - first], table[i][b]
                keep = lo - b * page
                top = fresh.abs().amax((0, 2)) / 127
                old = scale[pid].double() if keep else torch.zeros_like(top)
                now = torch.maximum(old, top)
                kept = codes[pid, :, :keep].double().transpose(0, 1)
                kept = torch.round(kept * (old / now)[:, None]) if keep else kept
                whole = torch.cat([kept, torch.round(fresh / now[:, None])], 0) * now[:, None]
                out.append(whole.flatten(1))
    return torch.cat(qs), torch.cat(ks), torch.cat(vs)


def _exact_attn(s):
    c = s["case"]
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
        hidden = t > p
        if c["window"]:
            hidden = hidden | ((t <= p - c["window"]) & (t >= c["sinks"]))
        for h in range(n_kv):
            k = s["k"][pid, h, t % page].double() * s["ks"][pid, h].double()[:, None]
            v = s["v"][pid, h, t % page].double() * s["vs"][pid, h].double()[:, None]
            for j in range(h * n_q // n_kv, (h + 1) * n_q // n_kv):
                q = s["qkv"][r0:r1, j * d:(j + 1) * d].double()
                x = (q @ k.T / math.sqrt(d)).masked_fill_(hidden, -math.inf)
                x = torch.exp_(x - x.amax(1, keepdim=True))
                out[r0:r1, j] = (x @ v) / x.sum(1, keepdim=True)
    return out.flatten(1)
