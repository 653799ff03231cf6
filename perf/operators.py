"""Cases of the serving operators: attention over packed prompts, attention of
single tokens over a paged cache whose sequences share a prefix, and the page
operations of that cache.

``run`` computes a case either in plain torch operations (``own`` false) or
through this framework's calls (``own`` true). The cache's book is one int32
tensor: 4 header words (status bits, pages moved by the last compact, 0, 0),
the length of each sequence slot, the reference count of each page, and the
page table of each slot (-1 where there is no page). Pages are
(layers, pages, page_size, kv_heads, dim), one tensor for K and one for V.
"""
import math
import random

import torch

own = False

DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    def prompt(name, act, heads, kv, dim, lens, packed=False):
        return {"name": name, "op": "prompt", "act": act, "heads": heads, "kv_heads": kv, "dim": dim, "lens": lens,
                "packed": packed}

    def decode(name, act, heads, kv, dim, batch, shared, most, page):
        return {"name": name, "op": "decode", "act": act, "heads": heads, "kv_heads": kv, "dim": dim, "batch": batch,
                "shared": shared, "own": most, "page": page}

    def append(name, act, kv, dim, lens, held, page):
        return {"name": name, "op": "append", "act": act, "kv_heads": kv, "dim": dim, "lens": lens, "held": held,
                "page": page}

    def pages(name, op, act, kv, dim, layers, page, seqs, most):
        return {"name": name, "op": op, "act": act, "kv_heads": kv, "dim": dim, "layers": layers, "page": page,
                "seqs": seqs, "own": most}

    return [
        # a chat turn of a few words: latency
        prompt("prompt short", "bf16", 24, 4, 256, "17"),
        # one prefill step of a serving batch, lengths as they come (an empty and a one-token prompt among them)
        prompt("prompts ragged", "f16", 24, 4, 256, "700,1,333,2049,64,129,0,820"),
        # the same over q, k and v that are slices of one buffer, in heads of 128
        prompt("prompts dim 128", "f16", 48, 8, 128, "5000,1023,2161", True),
        # one long document: compute bound
        prompt("prompt long", "bf16", 24, 4, 256, "16384"),
        # a single user, nothing shared: latency
        decode("decode one", "f16", 24, 4, 256, 1, 0, 1000, 16),
        # a batch of chats behind one system prompt that ends inside a page's tile
        decode("decode sixteen", "bf16", 24, 4, 256, 16, 8240, 600, 16),
        # many chats behind one long document
        decode("decode many", "f16", 24, 4, 256, 64, 65536, 2048, 64),
        # one decode step's new keys and values
        append("append tokens", "bf16", 4, 256, ",".join(["1"] * 64), 900, 16),
        # a prefill step's keys and values
        append("append prompts", "f16", 4, 256, "700,1,333,2049,64,129,0,820", 0, 64),
        # a few pages moved by their numbers
        pages("copy pages", "copy", "f16", 4, 256, 4, 16, 24, 300),
        # branches of a sampled answer: full pages are shared, each partial page is copied
        pages("fork", "fork", "bf16", 4, 256, 16, 64, 32, 3000),
        # chats that ended leave, and the rest moves to the front of the pool
        pages("free and compact", "compact", "f16", 4, 256, 8, 64, 96, 1000),
    ]


LAYOUTS = [(24, 4, 256), (24, 4, 256), (48, 8, 128), (12, 4, 256), (8, 8, 256), (32, 8, 128), (28, 4, 128), (16, 1, 128),
           (16, 16, 128)]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    act = rng.choice(["f16", "bf16"])
    heads, kv, dim = rng.choice(LAYOUTS)
    op = rng.choice(["prompt"] * 4 + ["decode"] * 4 + ["append", "copy", "fork", "compact"])
    if op == "prompt":
        # the plain form's scores are (tokens x tokens) for every head: tokens bounded by the largest case's
        total = log_int(rng, 1, int(16384 * math.sqrt(min(1.0, 24 / heads))))
        n = min(total, rng.choice([1, 1, 2, 3, 7, 20]))
        cuts = sorted(rng.randrange(total + 1) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return {"op": op, "act": act, "heads": heads, "kv_heads": kv, "dim": dim, "lens": ",".join(map(str, lens)),
                "packed": rng.random() < 0.5}
    if op == "decode":
        # a token's keys and values take kv * dim values: no more of them than the largest case reads
        room = 4 * 256 / (kv * dim)
        most = log_int(rng, 1, int(min(1.0, room) * 2000))
        batch = log_int(rng, 1, 64)
        shared = rng.choice([0, 1, 1, 1]) * log_int(rng, 1, int(min(1.0, room) * 60000))
        return {"op": op, "act": act, "heads": heads, "kv_heads": kv, "dim": dim, "batch": batch, "shared": shared,
                "own": most, "page": rng.choice([16, 32, 64, 128])}
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        if rng.random() < 0.5:
            lens = [1] * log_int(rng, 1, 200)
        else:
            lens = [log_int(rng, 1, 3000) for _ in range(rng.choice([1, 2, 5]))]
        return {"op": op, "act": act, "kv_heads": kv, "dim": dim, "lens": ",".join(map(str, lens)),
                "held": rng.choice([0, 1]) * log_int(rng, 1, 1500), "page": page}
    # pools of at most about 1 GB a side
    layers = rng.choice([1, 2, 5, 8])
    tokens = min(60000, (1 << 29) // (layers * kv * dim))
    seqs = log_int(rng, 4, 64)
    return {"op": op, "act": act, "kv_heads": kv, "dim": dim, "layers": layers, "page": page, "seqs": seqs,
            "own": log_int(rng, 8, max(8, min(3000, tokens // seqs)))}


# ---- what a case holds, apart from the values -------------------------------


def ints(text):
    return [int(x) for x in text.split(",")]


def up(a, b):
    return -(-a // b)


def own_lens(case):
    """Tokens that each sequence of a decode batch or a page case has of its own."""
    n = case["batch"] if case["op"] == "decode" else case["seqs"]
    return [1 + (i * 7919 + case["own"] - 1) % case["own"] for i in range(n)]


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


def pool(case, seed):
    """A page case's sequences on scattered pages (the same for every seed): lens, page numbers, pages, width, slots."""
    page, lens = case["page"], own_lens(case)
    need = sum(up(n, page) for n in lens)
    pages = need + need // 4 + 2 * len(lens)
    slots = 2 * len(lens)
    width = up(case["own"], page)
    return lens + [0] * len(lens), spread(case, 0, need, pages), pages, width, slots


def leaving(case):
    """Slots whose sequences end in a free-and-compact case: every other one, from the second."""
    return list(range(1, case["seqs"], 2))


def copied(case):
    """Source and target pages of a copy case: half of the used ones, to unused ones."""
    _, used, pages, _, _ = pool(case, 0)
    unused = sorted(set(range(pages)) - set(used))
    n = min(len(used) // 2 + 1, len(unused))
    return used[:n], unused[:n]


def normal(shape, act, seed, dev, scale=1.0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.empty(shape, dtype=DTYPE[act], device=dev)
    x.normal_(0.0, scale, generator=g)
    return x


def prepare(case, seed):
    dev = torch.device("cuda")
    op, act, kv, dim = case["op"], case["act"], case["kv_heads"], case["dim"]
    s = {"case": dict(case)}
    if op == "prompt":
        lens, heads = ints(case["lens"]), case["heads"]
        total = sum(lens)
        if case["packed"]:
            x = normal((total, heads + 2 * kv, dim), act, 3 * seed, dev)
            q, k, v = x[:, :heads], x[:, heads:heads + kv], x[:, heads + kv:]
            q.mul_(1.5)
        else:
            q = normal((total, heads, dim), act, 3 * seed, dev, 1.5)
            k = normal((total, kv, dim), act, 3 * seed + 1, dev)
            v = normal((total, kv, dim), act, 3 * seed + 2, dev)
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        return s | {"q": q, "k": k, "v": v, "offsets": torch.tensor(at, dtype=torch.int32)}
    page = case["page"]
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
        k = normal((1, pages, page, kv, dim), act, 3 * seed, dev)
        v = normal((1, pages, page, kv, dim), act, 3 * seed + 1, dev)
        if shared % page:  # the copies of the prefix's last page hold the same tokens in every sequence
            own_pages = torch.tensor([row[full] for row in tables], device=dev)
            for x in (k, v):
                x[0, own_pages, :shared % page] = x[0, own_pages[:1], :shared % page].clone()
        q = normal((case["batch"], case["heads"], dim), act, 3 * seed + 2, dev, 1.5)
        order = spread(case, seed + 1, len(lens), len(lens))
        slots, width = len(lens), len(tables[0])
        book = book_of([shared + n for n in lens], refs, tables).to(dev)
        s |= {"q": q, "k": k, "v": v, "book": book, "slots": slots, "width": width,
              "seqs": torch.tensor(order, dtype=torch.int32, device=dev)}
    elif op == "append":
        lens, held = ints(case["lens"]), case["held"]
        before = [held if i % 3 else held // 2 for i in range(len(lens))]
        used = sum(up(n, page) for n in before)
        pages = sum(up(a + n, page) for a, n in zip(before, lens)) + 5
        width = max(up(a + n, page) for a, n in zip(before, lens))
        numbers = spread(case, seed, used, pages)
        refs = [0] * pages
        for p in numbers:
            refs[p] = 1
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        s |= {"k": torch.zeros((2, pages, page, kv, dim), dtype=DTYPE[act], device=dev),
              "v": torch.zeros((2, pages, page, kv, dim), dtype=DTYPE[act], device=dev),
              "k_new": normal((at[-1], kv, dim), act, 3 * seed, dev), "v_new": normal((at[-1], kv, dim), act, 3 * seed + 1, dev),
              "book": book_of(before, refs, tables_of(before, page, width, numbers)).to(dev), "slots": len(lens), "width": width,
              "seqs": torch.arange(len(lens), dtype=torch.int32, device=dev),
              "offsets": torch.tensor(at, dtype=torch.int32, device=dev)}
    else:
        lens, used, pages, width, slots = pool(case, seed)
        refs = [0] * pages
        for p in used:
            refs[p] = 1
        s |= {"k": normal((case["layers"], pages, page, kv, dim), act, 3 * seed, dev),
              "v": normal((case["layers"], pages, page, kv, dim), act, 3 * seed + 1, dev),
              "book": book_of(lens, refs, tables_of(lens, page, width, used)).to(dev), "slots": slots, "width": width}
        n = case["seqs"]
        if op == "copy":
            s["src"], s["dst"] = (torch.tensor(x, dtype=torch.int32, device=dev) for x in copied(case))
        elif op == "fork":
            s["src"] = torch.arange(n, dtype=torch.int32, device=dev)
            s["dst"] = torch.arange(n, 2 * n, dtype=torch.int32, device=dev)
        else:
            s["seqs"] = torch.tensor(leaving(case), dtype=torch.int32, device=dev)
    s["book_before"] = s["book"].clone()
    if own:
        import exl3_trellis_quantized_rot_gb300 as tfx
        s["cache"] = tfx.Cache(s["k"], s["v"], s["slots"], s["width"], book=s["book"])
        tfx.cache_reserve(s["cache"], max_batch=max(1, len(s.get("seqs", ()))), heads=case.get("heads", kv))
    return s


# ---- the plain forms --------------------------------------------------------


def views(s):
    """The book's parts: lengths, reference counts, page tables."""
    book, pages, slots, width = s["book"], s["k"].shape[1], s["slots"], s["width"]
    at = 4 + slots + pages
    return book[4:4 + slots], book[4 + slots:at], book[at:at + slots * width].view(slots, width)


def softmax_parts(scores):
    e = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    return e, e.sum(-1, keepdim=True)


def plain_prompt(s):
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    total, heads, dim = q.shape
    kv = k.shape[1]
    seg = torch.searchsorted(s["offsets"].to(q.device), torch.arange(total, device=q.device, dtype=torch.int32), right=True)
    pos = torch.arange(total, device=q.device)
    hidden = (seg[:, None] != seg[None, :]) | (pos[None, :] > pos[:, None])
    g = q.permute(1, 0, 2).reshape(kv, heads // kv * total, dim)
    scores = (g @ k.permute(1, 2, 0)).mul_(1 / math.sqrt(dim)).view(heads, total, total)
    scores.masked_fill_(hidden, -math.inf)
    e, z = softmax_parts(scores)
    o = (e.view(kv, heads // kv * total, total) @ v.permute(1, 0, 2)).view(heads, total, dim) / z
    return o.permute(1, 0, 2).to(s["q"].dtype)


def plain_decode(s):
    lens, _, tables = views(s)
    c, q = s["case"], s["q"].float()
    batch, heads, dim = q.shape
    page, kv, shared = c["page"], c["kv_heads"], c["shared"]
    seqs, dev = s["seqs"].long(), q.device
    q = q.view(batch, kv, heads // kv, dim)
    kp, vp = s["k"][0].reshape(-1, kv, dim), s["v"][0].reshape(-1, kv, dim)
    at = torch.arange(shared, device=dev)
    at = tables[seqs[0]].long()[at // page] * page + at % page
    ks, vs = kp[at].float(), vp[at].float()
    pos = shared + torch.arange(c["own"], device=dev)
    seen = pos[None, :] < lens[seqs].long()[:, None]
    at = tables[seqs].long()[:, (pos // page).clamp(max=s["width"] - 1)].clamp(min=0) * page + pos % page
    ko, vo = kp[at].float(), vp[at].float()
    scale = 1 / math.sqrt(dim)
    a = torch.einsum("bhgd,lhd->bhgl", q, ks) * scale
    b = torch.einsum("bhgd,blhd->bhgl", q, ko) * scale
    b = torch.where(seen[:, None, None, :], b, torch.full((), -math.inf, device=dev))
    e, z = softmax_parts(torch.cat([a, b], -1))
    o = torch.einsum("bhgl,lhd->bhgd", e[..., :shared], vs) + torch.einsum("bhgl,blhd->bhgd", e[..., shared:], vo)
    return (o / z).reshape(batch, heads, dim).to(s["q"].dtype)


def plain_append(s):
    lens, refs, tables = views(s)
    page, seqs, offsets = s["case"]["page"], s["seqs"].long(), s["offsets"].long()
    add = offsets[1:] - offsets[:-1]
    old = lens[seqs].long()
    have = (old + page - 1) // page
    more = (old + add + page - 1) // page - have
    ends = more.cumsum(0)
    fresh = (refs == 0).nonzero()[:, 0][:int(ends[-1])]
    slot = torch.repeat_interleave(torch.arange(len(seqs), device=seqs.device), more)
    col = have[slot] + torch.arange(len(fresh), device=seqs.device) - (ends - more)[slot]
    tables[seqs[slot], col] = fresh.int()
    refs[fresh] = 1
    lens[seqs] = (old + add).int()
    row = torch.repeat_interleave(torch.arange(len(seqs), device=seqs.device), add)
    pos = old[row] + torch.arange(len(row), device=seqs.device) - offsets[row]
    at = tables[seqs[row], pos // page].long() * page + pos % page
    s["k"][1].view(-1, *s["k_new"].shape[1:])[at] = s["k_new"]
    s["v"][1].view(-1, *s["v_new"].shape[1:])[at] = s["v_new"]
    return {"k": s["k"], "v": s["v"], "book": s["book"]}


def plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    return {"k": s["k"], "v": s["v"]}


def plain_fork(s):
    lens, refs, tables = views(s)
    page, src, dst = s["case"]["page"], s["src"].long(), s["dst"].long()
    n = lens[src].long()
    full, part = n // page, n % page > 0
    cols = torch.arange(tables.shape[1], device=n.device)
    rows = torch.where(cols[None, :] < full[:, None], tables[src], torch.full_like(tables[src], -1))
    held = rows[rows >= 0].long()
    old = tables[src[part], full[part]].long()
    fresh = (refs == 0).nonzero()[:, 0][:len(old)]
    refs.index_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    refs[fresh] = 1
    tables[dst] = rows
    tables[dst[part], full[part]] = fresh.int()
    lens[dst] = n.int()
    s["k"][:, fresh] = s["k"][:, old]
    s["v"][:, fresh] = s["v"][:, old]
    return {"k": s["k"], "v": s["v"], "book": s["book"]}


def plain_compact(s):
    lens, refs, tables = views(s)
    seqs = s["seqs"].long()
    gone = tables[seqs]
    gone = gone[gone >= 0].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    tables[seqs] = -1
    lens[seqs] = 0
    live = refs > 0
    at = torch.arange(len(refs), device=refs.device)
    front = at < live.sum()
    src, dst = at[live & ~front], at[~live & front]
    to = at.clone()
    to[src] = dst
    tables.copy_(torch.where(tables >= 0, to[tables.long().clamp(min=0)].int(), tables))
    refs[dst] = refs[src]
    refs[src] = 0
    s["book"][1] = len(src)
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    return {"k": s["k"], "v": s["v"], "book": s["book"]}


PLAIN = {"prompt": plain_prompt, "decode": plain_decode, "append": plain_append, "copy": plain_copy, "fork": plain_fork,
         "compact": plain_compact}


# ---- one pass ---------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if op in ("append", "fork", "compact"):
        s["book"].copy_(s["book_before"])  # the step begins from the same book each time
    if not own:
        return PLAIN[op](s)
    import exl3_trellis_quantized_rot_gb300 as tfx
    if op == "prompt":
        return tfx.attn_prompt(s["q"], s["k"], s["v"], s["offsets"])
    cache = s["cache"]
    if op == "decode":
        return tfx.attn_decode(cache, 0, s["q"], s["seqs"], shared=s["case"]["shared"])
    if op == "append":
        tfx.cache_extend(cache, s["seqs"], s["offsets"])
        tfx.cache_append(cache, 1, s["k_new"], s["v_new"], s["seqs"], s["offsets"])
    elif op == "copy":
        tfx.cache_copy(cache, s["src"], s["dst"])
        return {"k": s["k"], "v": s["v"]}
    elif op == "fork":
        tfx.cache_fork(cache, s["src"], s["dst"])
    else:
        tfx.cache_free(cache, s["seqs"])
        tfx.cache_compact(cache)
    return {"k": s["k"], "v": s["v"], "book": s["book"]}


def work(case):
    op, kv, dim = case["op"], case["kv_heads"], case["dim"]
    token = 2 * kv * dim * 2  # bytes of one token's K and V
    if op == "prompt":
        lens, heads = ints(case["lens"]), case["heads"]
        return {"bytes": sum(lens) * (token + 2 * heads * dim * 2), "flops": 4 * dim * heads * sum(n * (n + 1) // 2 for n in lens)}
    if op == "decode":
        lens, heads, batch, shared = own_lens(case), case["heads"], case["batch"], case["shared"]
        return {"bytes": (shared + sum(lens)) * token + 2 * batch * heads * dim * 2 + 4 * (up(shared, case["page"]) + batch),
                "flops": 4 * dim * heads * (batch * shared + sum(lens))}
    if op == "append":
        return {"bytes": 2 * sum(ints(case["lens"])) * token, "flops": 0}
    page = case["page"]
    if op == "copy":
        moved = len(copied(case)[0]) * page
    elif op == "fork":
        moved = sum(n % page for n in own_lens(case))  # the tokens that a partial page holds
    else:
        lens, used, _, _, _ = pool(case, 0)
        gone, at, live = set(leaving(case)), 0, []
        for i, n in enumerate(lens):
            k = up(n, page)
            live += [] if i in gone else used[at:at + k]
            at += k
        moved = sum(p >= len(live) for p in live) * page
    return {"bytes": 2 * case["layers"] * moved * token, "flops": 0}


# ---- in 64 bits, from the definitions ---------------------------------------


def attend(q, k, v, seen):
    """q (m, d), k and v (n, d) in 64 bits, seen (m, n): the rows' attention."""
    a = (q @ k.T) / math.sqrt(q.shape[1])
    a[~seen] = -math.inf
    a = torch.exp(a - a.max(1, keepdim=True).values)
    return (a @ v) / a.sum(1, keepdim=True)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prompt":
        q, k, v = s["q"], s["k"].double(), s["v"].double()
        out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        group = case["heads"] // case["kv_heads"]
        at = s["offsets"].tolist()
        for a, b in zip(at, at[1:]):
            for r in range(a, b, 2048):
                e = min(r + 2048, b)
                seen = torch.arange(a, e, device=q.device)[None, :] <= torch.arange(r, e, device=q.device)[:, None]
                for h in range(case["heads"]):
                    out[r:e, h] = attend(q[r:e, h].double(), k[a:e, h // group], v[a:e, h // group], seen)
        return out
    if op == "decode":
        lens, _, tables = views(s)
        q = s["q"].double()
        out = torch.zeros_like(q)
        group, page = case["heads"] // case["kv_heads"], case["page"]
        for i, seq in enumerate(s["seqs"].tolist()):
            n = int(lens[seq])
            at = tables[seq, :up(n, page)].long()
            k, v = (x[0, at].reshape(-1, case["kv_heads"], case["dim"])[:n].double() for x in (s["k"], s["v"]))
            seen = torch.ones((group, n), dtype=torch.bool, device=q.device)
            for h in range(case["kv_heads"]):
                rows = slice(h * group, (h + 1) * group)
                out[i, rows] = attend(q[i, rows], k[:, h], v[:, h], seen)
        return out
    book = s["book"].tolist()
    pages, slots, width = s["k"].shape[1], s["slots"], s["width"]
    lens, refs = book[4:4 + slots], book[4 + slots:4 + slots + pages]
    flat = book[4 + slots + pages:]
    tables = [flat[i * width:(i + 1) * width] for i in range(slots)]
    moves, head, page = [], [0, 0, 0, 0], case["page"]
    if op == "copy":
        moves = list(zip(s["src"].tolist(), s["dst"].tolist()))
    elif op == "fork":
        n = case["seqs"]
        unused = iter([p for p in range(pages) if refs[p] == 0])
        for i in range(n):
            lens[n + i] = lens[i]
            for c in range(up(lens[i], page)):
                p = tables[i][c]
                if (c + 1) * page <= lens[i]:
                    refs[p] += 1
                else:
                    moves.append((p, next(unused)))
                    p = moves[-1][1]
                    refs[p] = 1
                tables[n + i][c] = p
    elif op == "append":
        at = s["offsets"].tolist()
        unused = iter([p for p in range(pages) if refs[p] == 0])
        where = []
        for i, seq in enumerate(s["seqs"].tolist()):
            for _ in range(at[i], at[i + 1]):
                if lens[seq] % page == 0:
                    tables[seq][lens[seq] // page] = p = next(unused)
                    refs[p] = 1
                where.append(tables[seq][lens[seq] // page] * page + lens[seq] % page)
                lens[seq] += 1
        where = torch.tensor(where, device=s["k"].device)
        for x, new in ((s["k"], s["k_new"]), (s["v"], s["v_new"])):
            x[1].view(-1, *new.shape[1:]).index_copy_(0, where, new)
    else:
        for i in leaving(case):
            for p in tables[i]:
                if p >= 0:
                    refs[p] -= 1
            tables[i], lens[i] = [-1] * width, 0
        live = sum(r > 0 for r in refs)
        unused = iter([p for p in range(live) if refs[p] == 0])
        to = {p: next(unused) for p in range(live, pages) if refs[p] > 0}
        for p, q in to.items():
            refs[q], refs[p] = refs[p], 0
        tables = [[to.get(p, p) for p in row] for row in tables]
        moves, head = list(to.items()), [0, len(to), 0, 0]
    for a, b in moves:
        s["k"][:, b].copy_(s["k"][:, a])
        s["v"][:, b].copy_(s["v"][:, a])
    if op == "copy":
        return {"k": s["k"], "v": s["v"]}
    return {"k": s["k"], "v": s["v"], "book": torch.tensor(head + lens + refs + [p for row in tables for p in row], dtype=torch.int32)}
