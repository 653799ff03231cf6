"""Cases of the operators around a cache that is held in 8 bits: rotary positions of
q and k, keys and values quantised as they are appended and read back, and
attention of single tokens over such a cache.

``run`` computes a case either in plain torch operations (``own`` false) or
through this framework's calls (``own`` true). The cache's book is one int32
tensor: 4 header words, the length of each sequence slot, the reference count of
each page, and the page table of each slot (-1 where there is no page). Pages are
(layers, pages, page_size, kv_heads, dim), one tensor of 8-bit codes for K and one
for V. A block is 16 tokens of one head; its scale is a power of two, the smallest
under which the block's values are in the codes' range, in a tensor
(layers, pages, page_size / 16, kv_heads). A block that takes further tokens keeps
its scale or gets a larger one, for which the codes it holds are rounded again.
"""
import math
import random

import torch

own = False

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}
STORE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}
BLOCK = 16
LEAST = -126  # exponent of the smallest scale


def listed():
    def rope(name, act, heads, kv, dim, rotary, rows, far, scaling="none", pairs=False, packed=False, inverse=False):
        return {"name": name, "op": "rope", "act": act, "heads": heads, "kv_heads": kv, "dim": dim, "rotary": rotary, "rows": rows,
                "far": far, "scaling": scaling, "pairs": pairs, "packed": packed, "inverse": inverse}

    def write(name, act, store, kv, dim, lens, held, page):
        return {"name": name, "op": "write", "act": act, "store": store, "kv_heads": kv, "dim": dim, "lens": lens, "held": held,
                "page": page}

    def read(name, act, store, kv, dim, lens, page):
        return {"name": name, "op": "read", "act": act, "store": store, "kv_heads": kv, "dim": dim, "lens": lens, "page": page}

    def decode(name, act, store, heads, kv, dim, batch, shared, most, page):
        return {"name": name, "op": "decode", "act": act, "store": store, "heads": heads, "kv_heads": kv, "dim": dim,
                "batch": batch, "shared": shared, "own": most, "page": page}

    return [
        # a decode step of one chat batch: a quarter of each head is rotated; latency
        rope("rope step", "bf16", 24, 4, 256, 64, 64, 300000, "yarn 4"),
        # a prefill step over slices of one q/k/v buffer, neighbouring values paired
        rope("rope packed", "f16", 48, 8, 128, 128, 4097, 9000, "linear 8", True, True),
        # one long document, whole heads
        rope("rope long", "bf16", 24, 4, 256, 256, 16384, 0),
        # one decode step's new keys and values, into blocks that are partly filled
        write("write step", "bf16", "int8", 4, 256, ",".join(["1"] * 64), 900, 16),
        # a prefill step's keys and values, lengths as they come
        write("write prompts", "f16", "e4m3", 4, 256, "700,1,333,2049,64,129,0,820", 0, 64),
        # the next turn of a few long chats
        write("write long", "bf16", "int8", 8, 128, "16000,9000,7001", 1005, 128),
        # one short sequence leaves the cache: latency
        read("read one", "bf16", "e4m3", 4, 256, "300", 32),
        # sequences that are moved out of the cache
        read("read many", "f16", "int8", 4, 256, "8000,12345,16,0,3333,20000,1", 64),
        # a single user: latency
        decode("decode one", "f16", "int8", 24, 4, 256, 1, 0, 1000, 16),
        # a batch of chats behind one system prompt
        decode("decode sixteen", "bf16", "e4m3", 24, 4, 256, 16, 8245, 600, 64),
        # many chats of very different lengths
        decode("decode many", "f16", "e4m3", 24, 4, 256, 64, 0, 8192, 64),
        # one long document in heads of 128
        decode("decode long", "bf16", "int8", 48, 8, 128, 1, 0, 262144, 128),
    ]


LAYOUTS = [(24, 4, 256), (24, 4, 256), (48, 8, 128), (12, 4, 256), (8, 8, 256), (32, 8, 128), (28, 4, 128), (16, 1, 128),
           (16, 16, 128)]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    act, store = rng.choice(["f16", "bf16"]), rng.choice(["int8", "e4m3"])
    heads, kv, dim = rng.choice(LAYOUTS)
    op = rng.choice(["rope", "write", "read", "decode", "decode"])
    if op == "rope":
        rotary = rng.choice([dim, dim, dim // 4, 32, 80, 96])
        most = 16384 * 28 * 256 // ((heads + kv) * dim)
        return {"op": op, "act": act, "heads": heads, "kv_heads": kv, "dim": dim, "rotary": rotary, "rows": log_int(rng, 1, most),
                "far": rng.choice([0, 1]) * log_int(rng, 1, 1 << 22), "scaling": rng.choice(["none", "none", "linear 4", "ntk 8", "yarn 16"]),
                "pairs": rng.random() < 0.5, "packed": rng.random() < 0.5, "inverse": rng.random() < 0.25}
    page = rng.choice([16, 32, 64, 128])
    # a token's keys and values take kv * dim values: no more of them than the largest cases take
    room = min(1.0, 1024 / (kv * dim))
    if op in ("write", "read"):
        if op == "write" and rng.random() < 0.5:
            lens = [1] * log_int(rng, 1, 200)
        else:
            lens = [log_int(rng, 1, int(10000 * room)) for _ in range(rng.choice([1, 2, 3]))]
        c = {"op": op, "act": act, "store": store, "kv_heads": kv, "dim": dim, "lens": ",".join(map(str, lens)), "page": page}
        return c | ({"held": rng.choice([0, 1]) * log_int(rng, 1, 1500)} if op == "write" else {})
    batch = log_int(rng, 1, 64)
    most = log_int(rng, 1, int(room * (8192 if batch > 1 else 200000)))
    shared = rng.choice([0, 0, 1]) * log_int(rng, 1, int(room * 16000)) if batch > 1 else 0
    return {"op": op, "act": act, "store": store, "heads": heads, "kv_heads": kv, "dim": dim, "batch": batch, "shared": shared,
            "own": most, "page": page}


# ---- what a case holds, apart from the values -------------------------------


def ints(text):
    return [int(x) for x in text.split(",")]


def up(a, b):
    return -(-a // b)


def frequencies(case):
    """Radians a position for each pair, and the factor of the rotated values."""
    rotary, base, gain = case["rotary"], 10000.0, 1.0
    kind, _, by = case["scaling"].partition(" ")
    factor = float(by or 1)
    if kind == "ntk":
        base *= factor ** (rotary / (rotary - 2))
    f = [base ** (-2 * i / rotary) for i in range(rotary // 2)]
    if kind == "linear":
        f = [x / factor for x in f]
    if kind == "yarn":
        def at(turns):  # the pair that turns so often over the original 4,096 positions
            return rotary * math.log(4096 / (2 * math.pi * turns)) / (2 * math.log(base))
        low, high = max(math.floor(at(32)), 0), min(math.ceil(at(1)), rotary - 1)
        keep = [1 - min(max((i - low) / max(high - low, 0.001), 0), 1) for i in range(rotary // 2)]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, keep)]
        gain = 0.1 * math.log(factor) + 1
    return f, gain


def own_lens(case):
    """Tokens that each sequence of a decode batch has of its own."""
    n = case["batch"]
    return [case["own"]] if n == 1 else [1 + (i * 7919 + case["own"] - 1) % case["own"] for i in range(n)]


def spread(case, seed, count, total):
    """`count` different page numbers out of `total`."""
    return random.Random("%s %s" % (seed, sorted(case.items()))).sample(range(total), count)


def tables_of(lens, page, width, numbers):
    rows, at = [], 0
    for n in lens:
        k = up(n, page)
        rows.append(numbers[at:at + k] + [-1] * (width - k))
        at += k
    return rows


def book_of(lens, refs, tables):
    flat = [0, 0, 0, 0] + lens + refs + [p for row in tables for p in row]
    return torch.tensor(flat, dtype=torch.int32)


def offsets_of(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def generator(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def normal(shape, act, seed, dev, scale=1.0):
    x = torch.empty(shape, dtype=DTYPE[act], device=dev)
    return x.normal_(0.0, scale, generator=generator(seed, dev))


def keys(shape, act, seed, dev):
    """Values as a cache gets them: a few channels of a head are much larger than the others."""
    x = normal(shape, act, seed, dev)
    x[..., 5::61] *= 8
    return x


def power(e):
    """2^e in 32 bits, for whole numbers e from -126 to 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def least_exponent(largest, store):
    """The smallest e with largest <= TOP * 2^e."""
    m, e = torch.frexp(largest)
    top, bits = (127 / 128, 7) if store == "int8" else (448 / 512, 9)
    e = torch.where(largest > 0, e.int() - bits + (m > top).int(), torch.full_like(e.int(), LEAST))
    return e.clamp(min=LEAST)


def round_to(x, store):
    """Codes of 32-bit values that are in their range, as bytes."""
    return torch.round(x).to(torch.int8) if store == "int8" else x.to(torch.float8_e4m3fn).view(torch.int8)


def worth(codes, store):
    """The codes' values in 32 bits."""
    return codes.float() if store == "int8" else codes.view(torch.float8_e4m3fn).float()


def held_pool(case, pages, seed, dev, fill=None):
    """Pages whose blocks are all quantised: (codes as bytes, scales)."""
    page, kv, dim, store = case["page"], case["kv_heads"], case["dim"], case["store"]
    codes = torch.empty((1, pages, page, kv, dim), dtype=torch.int8, device=dev)
    scales = torch.empty((1, pages, page // BLOCK, kv), dtype=torch.float32, device=dev)
    x = keys((pages, page, kv, dim), case["act"], seed, dev)
    if fill is not None:
        fill(x)
    step = max(1, (1 << 26) // (page * kv * dim))
    for a in range(0, pages, step):
        y = x[a:a + step].float().view(-1, page // BLOCK, BLOCK, kv, dim)
        e = least_exponent(y.abs().amax((2, 4)), store)
        codes[0, a:a + step] = round_to(y * power(-e)[:, :, None, :, None], store).view(-1, page, kv, dim)
        scales[0, a:a + step] = power(e)
    return codes, scales


def prepare(case, seed):
    dev = torch.device("cuda")
    op, act, kv, dim = case["op"], case["act"], case["kv_heads"], case["dim"]
    s = {"case": dict(case)}
    if op == "rope":
        heads, rows, far = case["heads"], case["rows"], case["far"]
        if case["packed"]:
            x = normal((rows, heads + 2 * kv, dim), act, 3 * seed, dev)
            q, k = x[:, :heads], x[:, heads:heads + kv]
        else:
            q, k = normal((rows, heads, dim), act, 3 * seed, dev), normal((rows, kv, dim), act, 3 * seed + 1, dev)
        if far and rows <= 4096:  # a step of many sequences
            at = torch.randint(0, far, (rows,), generator=generator(3 * seed + 2, dev), device=dev)
        else:  # a prompt, behind what is held
            at = far + torch.arange(rows, device=dev)
        f, gain = frequencies(case)
        s |= {"q": q, "k": k, "positions": at.int(), "freqs": torch.tensor(f, dtype=torch.float64, device=dev), "gain": gain,
              "q_out": torch.empty(q.shape, dtype=q.dtype, device=dev), "k_out": torch.empty(k.shape, dtype=k.dtype, device=dev)}
        if own:
            import exl3_trellis_quantized_rot_gb300 as tfx
            kind, _, by = case["scaling"].partition(" ")
            s["rope"] = tfx.Rope(dim, rotary=case["rotary"], interleaved=case["pairs"], scaling=None if kind == "none" else kind,
                                 factor=float(by or 1), original=4096)
        return s
    page = case["page"]
    fill = None
    if op == "decode":
        lens, shared = own_lens(case), case["shared"]
        full = shared // page  # pages that all sequences share; the one in which the prefix ends is each one's own
        mine = [up(shared + n, page) - full for n in lens]
        pages = full + sum(mine) + 7
        numbers = spread(case, seed, full + sum(mine), pages)
        width, at, tables = full + max(mine), full, []
        for k in mine:
            tables.append(numbers[:full] + numbers[at:at + k] + [-1] * (width - full - k))
            at += k
        refs = [0] * pages
        for row in tables:
            for p in row:
                if p >= 0:
                    refs[p] += 1
        held = [shared + n for n in lens]
        if shared % page:  # the copies of the prefix's last page hold the same tokens in every sequence
            last = torch.tensor([row[full] for row in tables], device=dev)

            def fill(x):
                x[last, :shared % page] = x[last[:1], :shared % page].clone()
        s["q"] = normal((case["batch"], case["heads"], dim), act, 3 * seed + 2, dev, 1.5)
        s["seqs"] = torch.tensor(spread(case, seed + 1, len(lens), len(lens)), dtype=torch.int32, device=dev)
    else:
        lens = ints(case["lens"])
        held = [case["held"] if i % 3 else case["held"] // 2 for i in range(len(lens))] if op == "write" else lens
        add = lens if op == "write" else [0] * len(lens)
        used = sum(up(n, page) for n in held)
        pages = sum(up(a + n, page) for a, n in zip(held, add)) + 5
        width = max(up(a + n, page) for a, n in zip(held, add))
        numbers = spread(case, seed, used, pages)
        refs = [0] * pages
        for p in numbers:
            refs[p] = 1
        tables = tables_of(held, page, width, numbers)
        # what is read: sequences whole, or from the block that the first new token joins
        starts = [n // BLOCK * BLOCK for n in held] if op == "write" else [0] * len(lens)
        at = offsets_of([a + n - b for a, n, b in zip(held, add, starts)])
        dtype = DTYPE[act]
        s |= {"seqs": torch.arange(len(lens), dtype=torch.int32, device=dev),
              "starts": torch.tensor(starts, dtype=torch.int32, device=dev),
              "ends": torch.tensor(at, dtype=torch.int32, device=dev), "rows": at[-1],
              "k_out": torch.empty((at[-1], kv, dim), dtype=dtype, device=dev),
              "v_out": torch.empty((at[-1], kv, dim), dtype=dtype, device=dev)}
        if op == "write":
            at = offsets_of(lens)
            s |= {"offsets": torch.tensor(at, dtype=torch.int32, device=dev), "k_new": keys((at[-1], kv, dim), act, 3 * seed + 1, dev),
                  "v_new": keys((at[-1], kv, dim), act, 3 * seed + 2, dev) * 0.5}
    s["k"], s["k_scale"] = held_pool(case, pages, 5 * seed + 3, dev, fill)
    s["v"], s["v_scale"] = held_pool(case, pages, 5 * seed + 4, dev, fill)
    s |= {"book": book_of(held, refs, tables).to(dev), "slots": len(lens), "width": width}
    s["book_before"] = s["book"].clone()
    if own:
        import exl3_trellis_quantized_rot_gb300 as tfx
        store = STORE[case["store"]]
        s["cache"] = tfx.Cache(s["k"].view(store), s["v"].view(store), s["slots"], s["width"], book=s["book"],
                               k_scale=s["k_scale"], v_scale=s["v_scale"], act=DTYPE[act])
        tfx.cache_reserve(s["cache"], max_batch=max(1, len(lens)), heads=case.get("heads", kv))
    return s


# ---- the plain forms --------------------------------------------------------


def views(s):
    """The book's parts: lengths, reference counts, page tables."""
    book, pages, slots, width = s["book"], s["k"].shape[1], s["slots"], s["width"]
    at = 4 + slots + pages
    return book[4:4 + slots], book[4 + slots:at], book[at:at + slots * width].view(slots, width)


def plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["freqs"][None, :]
    cos, sin = (torch.cos(angle) * s["gain"]).float()[:, None, :], (torch.sin(angle) * s["gain"]).float()[:, None, :]
    if c["inverse"]:
        sin = -sin

    def turned(x):
        y = x.float()
        head, rest = y[..., :c["rotary"]], y[..., c["rotary"]:]
        if c["pairs"]:
            a, b = head[..., ::2], head[..., 1::2]
            head = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = head.chunk(2, -1)
            head = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((head, rest), -1).to(x.dtype)

    return {"q": turned(s["q"]), "k": turned(s["k"])}


def plain_read(s):
    c = s["case"]
    _, _, tables = views(s)
    page, store = c["page"], c["store"]
    ends = s["ends"].long()
    row = torch.repeat_interleave(torch.arange(len(s["seqs"]), device=ends.device), ends[1:] - ends[:-1])
    pos = s["starts"].long()[row] + torch.arange(len(row), device=ends.device) - ends[row]
    number = tables[s["seqs"].long()[row], pos // page].long()
    out = {}
    for name in ("k", "v"):
        x = worth(s[name][0, number, pos % page], store) * s[name + "_scale"][0, number, pos % page // BLOCK][..., None]
        out[name] = x.to(DTYPE[c["act"]])
    return out


def plain_write(s):
    c = s["case"]
    lens, refs, tables = views(s)
    page, store, seqs, offsets = c["page"], c["store"], s["seqs"].long(), s["offsets"].long()
    dev = seqs.device
    add = offsets[1:] - offsets[:-1]
    old = lens[seqs].long()
    have = (old + page - 1) // page
    more = (old + add + page - 1) // page - have
    ends = more.cumsum(0)
    fresh = (refs == 0).nonzero()[:, 0][:int(ends[-1])]
    slot = torch.repeat_interleave(torch.arange(len(seqs), device=dev), more)
    col = have[slot] + torch.arange(len(fresh), device=dev) - (ends - more)[slot]
    tables[seqs[slot], col] = fresh.int()
    refs[fresh] = 1
    lens[seqs] = (old + add).int()
    # the blocks that get tokens: of each sequence, from the one its first new token joins
    first = old // BLOCK
    blocks = torch.where(add > 0, (old + add + BLOCK - 1) // BLOCK - first, torch.zeros_like(add))
    i = torch.repeat_interleave(torch.arange(len(seqs), device=dev), blocks)
    b = first[i] + torch.arange(len(i), device=dev) - (blocks.cumsum(0) - blocks)[i]
    pos = b[:, None] * BLOCK + torch.arange(BLOCK, device=dev)[None, :]
    number = tables[seqs[i], b * BLOCK // page].long()
    at, part = pos % page, b * BLOCK % page // BLOCK
    was, new = pos < old[i][:, None], (pos >= old[i][:, None]) & (pos < (old + add)[i][:, None])
    source = torch.where(new, offsets[i][:, None] + pos - old[i][:, None], torch.zeros_like(pos))
    for name in ("k", "v"):
        x = torch.where(new[:, :, None, None], s[name + "_new"].float()[source], torch.zeros((), device=dev))
        e = least_exponent(x.abs().amax((1, 3)), store)
        before = s[name + "_scale"][0, number, part]
        grown = torch.maximum(power(e), torch.where(was[:, :1], before, torch.zeros_like(before)))
        codes = s[name][0, number[:, None], at]
        kept = worth(codes, store) * (before / grown)[:, None, :, None]
        x = torch.where(was[:, :, None, None], kept, x / grown[:, None, :, None])
        s[name + "_scale"][0, number, part] = grown
        s[name][0, number[:, None], at] = torch.where((was | new)[:, :, None, None], round_to(x, store), codes)
    return plain_read(s) | {"book": s["book"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def plain_decode(s):
    lens, _, tables = views(s)
    c, q = s["case"], s["q"].float()
    batch, heads, dim = q.shape
    page, kv, store = c["page"], c["kv_heads"], c["store"]
    shared = c["shared"] // BLOCK * BLOCK  # whole blocks; what follows is read through each sequence's own table
    seqs, dev = s["seqs"].long(), q.device
    q = q.view(batch, kv, heads // kv, dim)

    def rows(name, number, at):
        return worth(s[name][0, number, at], store) * s[name + "_scale"][0, number, at // BLOCK][..., None]

    pos = torch.arange(shared, device=dev)
    number = tables[seqs[0]].long()[pos // page]
    ks, vs = rows("k", number, pos % page), rows("v", number, pos % page)
    pos = shared + torch.arange(c["shared"] - shared + c["own"], device=dev)
    seen = pos[None, :] < lens[seqs].long()[:, None]
    number = tables[seqs].long()[:, (pos // page).clamp(max=s["width"] - 1)].clamp(min=0)
    at = (pos % page)[None, :].expand_as(number)
    ko, vo = rows("k", number, at), rows("v", number, at)
    a = torch.einsum("bhgd,lhd->bhgl", q, ks)
    b = torch.einsum("bhgd,blhd->bhgl", q, ko)
    scores = torch.cat([a, b.masked_fill_(~seen[:, None, None, :], -math.inf)], -1).mul_(1 / math.sqrt(dim))
    e = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    z = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgl,lhd->bhgd", e[..., :shared], vs) + torch.einsum("bhgl,blhd->bhgd", e[..., shared:], vo)
    return (o / z).reshape(batch, heads, dim).to(s["q"].dtype)


PLAIN = {"rope": plain_rope, "write": plain_write, "read": plain_read, "decode": plain_decode}


# ---- one pass ---------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if op == "write":
        s["book"].copy_(s["book_before"])  # the step begins from the same book each time
    if not own:
        return PLAIN[op](s)
    import exl3_trellis_quantized_rot_gb300 as tfx
    if op == "rope":
        q, k = tfx.rope(s["rope"], s["q"], s["k"], s["positions"], out=(s["q_out"], s["k_out"]), inverse=s["case"]["inverse"])
        return {"q": q, "k": k}
    cache = s["cache"]
    if op == "decode":
        return tfx.attn_decode(cache, 0, s["q"], s["seqs"], shared=s["case"]["shared"])
    if op == "write":
        tfx.cache_extend(cache, s["seqs"], s["offsets"])
        tfx.cache_append(cache, 0, s["k_new"], s["v_new"])
    k, v = tfx.cache_read(cache, 0, s["seqs"], s["starts"], s["ends"], s["rows"], out=(s["k_out"], s["v_out"]))
    out = {"k": k, "v": v}
    return out | {"book": s["book"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]} if op == "write" else out


def work(case):
    op, kv, dim = case["op"], case["kv_heads"], case["dim"]
    if op == "rope":
        rows, values = case["rows"], (case["heads"] + kv)
        return {"bytes": 4 * rows * values * dim + 4 * rows, "flops": 3 * rows * values * case["rotary"]}
    token = 2 * kv * dim  # bytes of one token's K and V codes
    if op == "decode":
        lens, heads, batch, shared = own_lens(case), case["heads"], case["batch"], case["shared"]
        tokens = shared + sum(lens)
        return {"bytes": tokens * token + 2 * kv * 4 * up(tokens, BLOCK) + 2 * batch * heads * dim * 2,
                "flops": 4 * dim * heads * (batch * shared + sum(lens))}
    lens = ints(case["lens"])
    if op == "read":
        return {"bytes": 3 * token * sum(lens) + 2 * kv * 4 * sum(up(n, BLOCK) for n in lens), "flops": token * sum(lens)}
    held = [case["held"] if i % 3 else case["held"] // 2 for i in range(len(lens))]
    back = sum(h % BLOCK + n for h, n in zip(held, lens))  # tokens that are read back
    return {"bytes": 3 * token * (sum(lens) + back) + 4 * kv * 4 * sum(up(h % BLOCK + n, BLOCK) for h, n in zip(held, lens)),
            "flops": 3 * token * sum(lens) + token * back}


# ---- in 64 bits, from the definitions ---------------------------------------


def value_of(codes, scale, store):
    """Codes (bytes) and their scales in 64 bits."""
    c = codes.double() if store == "int8" else codes.view(torch.float8_e4m3fn).double()
    return c * scale.double()[..., None]


def power64(e):
    """2^e in 64 bits, exactly, which pow() on the GPU does not promise."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def nearest(y, store):
    """The nearest value that a code has, ties to even."""
    if store == "int8":
        return torch.round(y)
    _, e = torch.frexp(y)
    step = power64((e - 4).clamp(min=-9))  # 3 bits behind the first; subnormals in steps of 2^-9
    return torch.round(y / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        f, gain = frequencies(case)
        angle = s["positions"].double()[:, None] * torch.tensor(f, dtype=torch.float64, device=s["q"].device)
        turn = torch.polar(torch.full_like(angle, gain), -angle if case["inverse"] else angle)[:, None, :]
        out, r = {}, case["rotary"]
        for name in ("q", "k"):
            x = s[name].double()
            z = x[..., :r].unflatten(-1, (r // 2, 2)) if case["pairs"] else x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            x[..., :r] = z.flatten(-2) if case["pairs"] else z.transpose(-1, -2).flatten(-2)
            out[name] = x
        return out
    store, page, kv, dim = case["store"], case["page"], case["kv_heads"], case["dim"]
    book, pages, slots, width = s["book"].tolist(), s["k"].shape[1], s["slots"], s["width"]
    lens, refs = book[4:4 + slots], book[4 + slots:4 + slots + pages]
    tables = [book[4 + slots + pages + i * width:4 + slots + pages + (i + 1) * width] for i in range(slots)]

    def tokens(i, a, b):
        """K and V of tokens a .. b-1 of sequence i."""
        n = torch.tensor(tables[i][:up(b, page)], dtype=torch.long, device=s["k"].device)
        scale = {x: s[x + "_scale"][0, n].repeat_interleave(BLOCK, 1).reshape(-1, kv) for x in ("k", "v")}
        return [value_of(s[x][0, n].reshape(-1, kv, dim)[a:b], scale[x][a:b], store) for x in ("k", "v")]

    if op == "read":
        both = [tokens(i, 0, n) for i, n in enumerate(lens) if n]
        return {x: torch.cat([t[j] for t in both]) for j, x in enumerate(("k", "v"))}
    if op == "decode":
        q = s["q"].double()
        out, group, cut = torch.zeros_like(q), case["heads"] // kv, case["shared"] // BLOCK * BLOCK
        seqs = s["seqs"].tolist()
        front = tokens(seqs[0], 0, cut) if cut else []
        for i, seq in enumerate(seqs):
            k, v = tokens(seq, cut, lens[seq])
            if cut:
                k, v = torch.cat([front[0], k]), torch.cat([front[1], v])
            for h in range(kv):
                a = torch.softmax(q[i, h * group:(h + 1) * group] @ k[:, h].T / math.sqrt(dim), -1)
                out[i, h * group:(h + 1) * group] = a @ v[:, h]
        return out
    # write: token after token into pages, then block after block
    unused = iter([p for p in range(pages) if refs[p] == 0])
    at, starts = s["offsets"].tolist(), s["starts"].tolist()
    values = {"k": [], "v": []}
    for i in range(slots):
        old, new = lens[i], lens[i] + at[i + 1] - at[i]
        kept = tokens(i, starts[i], old) if starts[i] < old else None
        for c in range(up(old, page), up(new, page)):
            tables[i][c] = p = next(unused)
            refs[p] = 1
        lens[i] = new
        if old == new:
            if kept:
                values["k"].append(kept[0])
                values["v"].append(kept[1])
            continue
        for j, x in enumerate(("k", "v")):
            y = s[x + "_new"][at[i]:at[i + 1]].double()
            lead = old - starts[i]
            padded = torch.zeros((up(lead + len(y), BLOCK) * BLOCK, kv, dim), dtype=torch.float64, device=y.device)
            padded[lead:lead + len(y)] = y
            blocks = padded.view(-1, BLOCK, kv, dim)
            amax = blocks.abs().amax((1, 3))
            e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / TOP[store])).clamp(min=LEAST)
            scale = power64(e)
            scale = torch.where(amax > scale * TOP[store], scale * 2, scale)
            scale = torch.where((amax <= scale / 2 * TOP[store]) & (e > LEAST), scale / 2, scale)
            b = torch.arange(starts[i] // BLOCK, starts[i] // BLOCK + len(blocks), device=y.device)
            number = torch.tensor(tables[i], device=y.device)[b * BLOCK // page]
            part = b * BLOCK % page // BLOCK
            if lead:
                scale[0] = torch.maximum(scale[0], s[x + "_scale"][0, number[0], part[0]].double())
                blocks[0, :lead] = kept[j]
            got = nearest(blocks / scale[:, None, :, None], store) * scale[:, None, :, None]
            s[x + "_scale"][0, number, part] = scale.float()
            values[x].append(got.reshape(-1, kv, dim)[:lead + len(y)])
    flat = [0, 0, 0, 0] + lens + refs + [p for row in tables for p in row]
    return {"k": torch.cat(values["k"]), "v": torch.cat(values["v"]), "book": torch.tensor(flat, dtype=torch.int32),
            "k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double()}
