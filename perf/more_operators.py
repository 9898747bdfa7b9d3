"""Cases for what serving many continuations of one prompt needs around the 8-bit paged cache.

Four operators, each in the plain form (elementary torch operations in 32 bits,
angles in 64) and as the library call a program makes:

* rotate: every head of the queries and keys of a fused projection normalised
  (root mean square, a weight for each dimension) and rotated by its token's
  positions, one axis (text) or several (time, height, width);
* fork: the batch of the next step from the one before: new sequences take over
  (parents named on the device) their parent's pages, share the full ones, copy
  a partly filled one before it is written to, get free pages for the tokens to
  come; sequences without children give theirs back;
* compact: the pages in use moved to the front of the cache, tables following;
* prefix: attention of sequences in groups, each group's common prefix held and
  read once, each sequence's own tokens behind it.

Cache pages: keys [page][head][token][dim], values [page][head][dim][token] in
e4m3, one exponent byte for each page and head of either.  refs[page] is the
number of sequences (and other holders) that hold a page; 0: free.
"""
import math

import torch

own = False


def listed():
    return [
        # one decoded token: latency
        dict(name="rotate_token", op="rotate", tokens=1, q_heads=40, kv_heads=8, dim=128, rot=128, axes=1, pairs="half",
             norm=True, dtype="bf16", out="bf16", first=131071),
        # a long prompt from a projection that keeps 32 bits, part of each wide head rotated, far positions
        dict(name="rotate_prompt", op="rotate", tokens=8191, q_heads=24, kv_heads=4, dim=256, rot=64, axes=1, pairs="half",
             norm=True, dtype="f32", out="bf16", first=120000),
        # the image and text tokens of a diffusion transformer block, batch of 4, three axes
        dict(name="rotate_image", op="rotate", tokens=18432, q_heads=20, kv_heads=20, dim=128, rot=128, axes=3,
             pairs="adjacent", norm=True, dtype="bf16", out="bf16", first=0),
        # reordering the beams of a batch after a step: 16 prompts, 4 beams each
        dict(name="fork_beams", op="fork", groups=16, beams=4, new=4, shared=1537, ctx=2100, grow=1, kv_heads=8, dim=128,
             page=64, spare=200),
        # two long prompts, 100 answers started from each
        dict(name="fork_prompts", op="fork", groups=2, beams=1, new=100, shared=32759, ctx=32759, grow=5, kv_heads=8, dim=128,
             page=16, spare=900),
        # a small cache with few free pages closed up
        dict(name="compact_small", op="compact", seqs=9, ctx=1000, pages=700, kv_heads=4, dim=64, page=16),
        # a pool of twice the pages in use closed up before a part of it is given away
        dict(name="compact_pool", op="compact", seqs=60, ctx=8000, pages=6000, kv_heads=8, dim=128, page=64),
        # a handful of answers behind a short prompt: the smallest call
        dict(name="prefix_few", op="prefix", groups=1, seqs=4, new=1, ctx=70, prefix=1000, q_heads=40, kv_heads=8, dim=128,
             page=16),
        # 64 answers behind one long document
        dict(name="prefix_batch", op="prefix", groups=1, seqs=64, new=1, ctx=500, prefix=32760, q_heads=40, kv_heads=8,
             dim=128, page=64),
        # five drafted tokens of each answer checked, several prompts, small heads
        dict(name="prefix_verify", op="prefix", groups=6, seqs=45, new=5, ctx=900, prefix=8000, q_heads=16, kv_heads=4, dim=64,
             page=32),
        # wide heads, a very long prefix
        dict(name="prefix_wide", op="prefix", groups=2, seqs=16, new=1, ctx=2000, prefix=65000, q_heads=24, kv_heads=4,
             dim=256, page=128),
        # users' prompts behind one system prompt
        dict(name="prefix_prompts", op="prefix", groups=1, seqs=8, new=777, ctx=777, prefix=6001, q_heads=32, kv_heads=8,
             dim=128, page=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotate", "fork", "compact", "prefix", "prefix"))
    if op == "rotate":
        while True:
            tokens, kv_heads = _log_int(rng, 1, 20000), rng.choice((1, 2, 4, 5, 8, 20, 40))
            q_heads, dim = kv_heads * rng.choice((1, 1, 2, 3, 5, 8)), rng.choice((64, 72, 80, 96, 128, 128, 192, 256))
            if q_heads <= 64 and tokens * (q_heads + kv_heads) * dim <= 18432 * 40 * 128:
                rot = rng.choice((dim, dim, 8 * rng.randint(2, dim // 8)))
                return dict(op=op, tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, dim=dim, rot=rot,
                            axes=rng.choice((1, 1, 2, 3)), pairs=rng.choice(("half", "adjacent")), norm=rng.random() < 0.75,
                            dtype=rng.choice(("bf16", "bf16", "f32")), out=rng.choice(("bf16", "bf16", "f32")),
                            first=_log_int(rng, 1, 1000000) - 1)
    kv_heads, dim, page = rng.choice((1, 2, 4, 5, 8)), rng.choice((64, 128, 256)), rng.choice((16, 32, 64, 128))
    if op == "fork":
        while True:
            groups, beams, new = _log_int(rng, 1, 40), rng.choice((1, 2, 4, 5, 8)), _log_int(rng, 1, 100)
            shared = _log_int(rng, 1, 30000)
            ctx = shared + _log_int(rng, 1, 1000) - 1 if beams > 1 else shared
            grow = rng.choice((0, 1, 1, 1, 5, 77))
            need = groups * (shared // page + (beams + new) * ((ctx - shared + grow) // page + 3))
            if need * page * kv_heads * dim <= 2 ** 28 and groups * new * ctx <= 2 * 100 * 32759 * 2:
                return dict(op=op, groups=groups, beams=beams, new=new, shared=shared, ctx=ctx, grow=grow, kv_heads=kv_heads,
                            dim=dim, page=page, spare=_log_int(rng, 1, 500))
    if op == "compact":
        while True:
            seqs, ctx = _log_int(rng, 1, 200), _log_int(rng, 1, 20000)
            used = seqs * -(-ctx // page)
            pages = used + _log_int(rng, 1, 4000)
            if pages * page * kv_heads * dim <= 6000 * 64 * 8 * 128:
                return dict(op=op, seqs=seqs, ctx=ctx, pages=pages, kv_heads=kv_heads, dim=dim, page=page)
    while True:
        groups, step = _log_int(rng, 1, 8), rng.random() < 0.75
        seqs = groups * _log_int(rng, 2, 64 if step else 10) + rng.randint(0, groups - 1)
        new = rng.choice((1, 1, 1, 2, 5)) if step else _log_int(rng, 6, 700)
        ctx, prefix = new + _log_int(rng, 1, 1200) - 1, _log_int(rng, 10, 60000)
        q_heads = kv_heads * rng.choice((1, 2, 3, 5, 6, 8))
        if (q_heads <= 64 and seqs * new * (ctx + prefix) * q_heads * dim <= 8 * 777 * 6778 * 32 * 128
                and (groups * prefix + seqs * ctx) * kv_heads * dim <= 2 ** 28):
            return dict(op=op, groups=groups, seqs=seqs, new=new, ctx=ctx, prefix=prefix, q_heads=q_heads, kv_heads=kv_heads,
                        dim=dim, page=page)


def _ragged(i, least=0.25):
    """A factor in (least, 1], 1 for i = 0."""
    return 1.0 - (1.0 - least) * ((i * 0.6180339887) % 1.0)


def _behind(c):
    """Of a prefix case: sequences and prefix length of each group, new tokens and own tokens of each sequence."""
    g, b = c["groups"], c["seqs"]
    count = [b // g + (1 if i < b % g else 0) for i in range(g)]
    prefix = [max(1, int(c["prefix"] * _ragged(i, 0.5))) for i in range(g)]
    lens = []
    for i in range(b):
        n = max(1, int(c["new"] * _ragged(i)))
        lens.append((n, max(n, int(c["ctx"] * _ragged(i)))))
    return count, prefix, lens


def work(c):
    if c["op"] == "rotate":
        n = c["tokens"] * (c["q_heads"] + c["kv_heads"]) * c["dim"]
        e = (2 if c["dtype"] == "bf16" else 4) + (2 if c["out"] == "bf16" else 4)
        return {"bytes": n * e + 4 * c["tokens"] * c["axes"], "flops": 6 * n}
    if c["op"] == "prefix":
        count, prefix, lens = _behind(c)
        token, row = 2 * c["kv_heads"] * (c["dim"] + 1 / c["page"]), c["q_heads"] * (4 * c["dim"] + 4)
        new = sum(n for n, _ in lens)
        pairs, at = 0, 0
        for m, p in zip(count, prefix):
            pairs += p * sum(n for n, _ in lens[at:at + m])
            at += m
        pairs += sum(n * (t - n) + n * (n + 1) // 2 for n, t in lens)
        return {"bytes": (sum(prefix) + sum(t for _, t in lens)) * token + new * row,
                "flops": 4 * pairs * c["q_heads"] * c["dim"]}
    page = 2 * c["kv_heads"] * (c["page"] * c["dim"] + 1)
    if c["op"] == "compact":
        used = sum(-(-max(1, int(c["ctx"] * _ragged(i))) // c["page"]) for i in range(c["seqs"]))
        # pages in use lie anywhere: those at or behind `used` move
        moved = used * (c["pages"] - used) / c["pages"]
        return {"bytes": 2 * moved * page + 4 * (3 * c["pages"] + 2 * used), "flops": 0}
    old, new = c["groups"] * c["beams"], c["groups"] * c["new"]
    # a partly filled page is kept by one child of each parent with children
    copies = 0
    if c["grow"] and c["ctx"] % c["page"]:
        copies = new - old * (1 - (1 - 1 / c["beams"]) ** c["new"])
    entries = old * -(-c["ctx"] // c["page"]) + new * -(-(c["ctx"] + c["grow"]) // c["page"])
    return {"bytes": 2 * copies * page + 4 * (entries + 2 * _fork_pages(c) + 3 * new), "flops": 0}


def _fork_pages(c):
    P = c["page"]
    full, held = c["shared"] // P, -(-c["ctx"] // P)
    more = -(-(c["ctx"] + c["grow"]) // P) - held + 1
    return c["groups"] * (full + c["beams"] * (held - full) + c["new"] * more) + c["spare"]


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda").contiguous()


def _cache(g, pages, c):
    H, D, P = c["kv_heads"], c["dim"], c["page"]
    out = []
    for shape in ((pages, H, P, D), (pages, H, D, P)):
        t = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
        step = max(1, 2 ** 26 // (H * P * D))
        for i in range(0, pages, step):
            part = _randn(g, min(step, pages - i), *shape[1:])
            t[i:i + step] = part.mul_(90).clamp_(-448, 448).to(torch.float8_e4m3fn)
        out.append(t)
    for _ in range(2):
        out.append(torch.randint(118, 122, (pages, H), device="cuda", generator=g).to(torch.uint8))
    return tuple(out)


def _frequencies(c):
    """Radians a position of each pair, and the pair's axis: every axis has a run of pairs with a geometric
    sequence of its own, the first axis (time) a shorter one."""
    n, axes = c["rot"] // 2, c["axes"]
    size = [n] if axes == 1 else [n // 2, n - n // 2] if axes == 2 else [n // 8, (n - n // 8) // 2]
    if axes == 3:
        size.append(n - sum(size))
    f, a = [], []
    for i, m in enumerate(size):
        base = 1e6 if axes == 1 else 1e4
        f += [base ** (-j / m) for j in range(m)]
        a += [i] * m
    return f, a


def prepare(c, seed):
    g = _gen(seed)
    s = {"case": dict(c)}
    if c["op"] == "rotate":
        T, Hq, H, D = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
        qkv = _randn(g, T, Hq + 2 * H, D)
        qkv *= torch.exp(0.5 * _randn(g, T, 1, 1))
        s["qkv"] = qkv.bfloat16() if c["dtype"] == "bf16" else qkv
        f, a = _frequencies(c)
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        s["pair_axis"] = None if c["axes"] == 1 else _i32(a)
        # text counts on; an image's tokens share the first axis and count rows and columns on the others
        t = torch.arange(T, device="cuda") + c["first"]
        side = max(1, int(math.sqrt(T / 4)))
        grid = [t // (side * side), t // side % side, t % side]
        s["positions"] = _i32(t) if c["axes"] == 1 else torch.stack(grid[3 - c["axes"]:]).to(torch.int32).contiguous()
        for n in ("q_weight", "k_weight"):
            s[n] = 1 + 0.3 * _randn(g, D) if c["norm"] else None
        return s
    P = c["page"]
    if c["op"] == "fork":
        groups, beams, new = c["groups"], c["beams"], c["new"]
        full, held = c["shared"] // P, -(-c["ctx"] // P)
        pages = _fork_pages(c)
        perm = torch.randperm(pages, device="cuda", generator=g)
        mine = groups * beams * (held - full)
        table = torch.full((groups, beams, held + 1), -1, dtype=torch.int64, device="cuda")
        table[:, :, :full] = perm[:groups * full].reshape(groups, 1, full)
        table[:, :, full:held] = perm[groups * full:groups * full + mine].reshape(groups, beams, held - full)
        refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        at = table[:, :, :held].reshape(-1)
        refs.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
        # the first group's prompt stays in a store of prompts
        refs[perm[:full]] += 1
        s["refs"] = refs
        s["page_table"] = table.reshape(groups * beams, held + 1).to(torch.int32)
        s["kv_lens"] = torch.full((groups * beams,), c["ctx"], dtype=torch.int32, device="cuda")
        pick = torch.randint(0, beams, (groups, new), device="cuda", generator=g)
        s["parents"] = (pick + beams * torch.arange(groups, device="cuda")[:, None]).reshape(-1).to(torch.int32)
        s["width"] = -(-(c["ctx"] + c["grow"]) // P)
        s["cache"] = _cache(g, pages, c)
        return s
    if c["op"] == "compact":
        lens = [max(1, int(c["ctx"] * _ragged(i))) for i in range(c["seqs"])]
        held = [-(-n // P) for n in lens]
        perm = torch.randperm(c["pages"], device="cuda", generator=g)
        table = torch.full((c["seqs"], max(held)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(held):
            table[b, :n] = perm[at:at + n]
            at += n
        # the second half of the sequences begins with the first one's first page
        table[c["seqs"] // 2:, 0] = table[0, 0]
        refs = torch.zeros(c["pages"], dtype=torch.int32, device="cuda")
        use = table[table >= 0].long()
        s["refs"] = refs.index_add_(0, use, torch.ones_like(use, dtype=torch.int32))
        s["page_table"], s["kv_lens"] = table, _i32(lens)
        s["cache"] = _cache(g, c["pages"], c)
        return s
    count, prefix, lens = _behind(c)
    B, G = c["seqs"], c["groups"]
    w0, w1 = -(-max(prefix) // P), max(-(-t // P) for _, t in lens)
    pages = G * w0 + B * w1 + 3
    perm = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    s["prefix_table"] = perm[:G * w0].reshape(G, w0).contiguous()
    s["page_table"] = perm[G * w0:G * w0 + B * w1].reshape(B, w1).contiguous()
    s["prefix_lens"], s["kv_lens"] = _i32(prefix), _i32([t for _, t in lens])
    starts = [0]
    for m in count:
        starts.append(starts[-1] + m)
    s["seq_starts"] = _i32(starts)
    rows = [0]
    for n, _ in lens:
        rows.append(rows[-1] + n)
    s["q_starts"] = _i32(rows)
    s["max_q"], s["max_kv"] = max(n for n, _ in lens), max(t for _, t in lens)
    s["max_prefix"], s["max_seqs"] = max(prefix), max(count)
    s["cache"] = _cache(g, pages, c)
    s["q"] = _randn(g, rows[-1], c["q_heads"], c["dim"]).bfloat16()
    # rows of each group, for the plain form
    at = [0]
    for m in count:
        at.append(at[-1] + sum(n for n, _ in lens[starts[len(at) - 1]:starts[len(at) - 1] + m]))
    s["rows"], s["prefix"] = at, prefix
    return s


# ------------------------------------------------- the formulas, in 32 bits


def _rotate_plain(s):
    c = s["case"]
    Hq, H, R = c["q_heads"], c["kv_heads"], c["rot"]
    pos = s["positions"].reshape(c["axes"], c["tokens"]).double()
    at = pos[0][:, None] if s["pair_axis"] is None else pos[s["pair_axis"].long()].t()
    angle = torch.remainder(at * s["freqs"], 2 * math.pi)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x, w in ((s["qkv"][:, :Hq], s["q_weight"]), (s["qkv"][:, Hq:Hq + H], s["k_weight"])):
        y = x.float()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(2, keepdim=True) + 1e-6) * w
        r = y[..., :R]
        a, b = (r[..., :R // 2], r[..., R // 2:]) if c["pairs"] == "half" else (r[..., 0::2], r[..., 1::2])
        u, v = a * cos - b * sin, b * cos + a * sin
        r = torch.cat((u, v), 2) if c["pairs"] == "half" else torch.stack((u, v), 3).flatten(2)
        y = torch.cat((r, y[..., R:]), 2)
        out.append(y.bfloat16() if c["out"] == "bf16" else y)
    return tuple(out)


def _copy_pages(cache, src, dst):
    for t in cache:
        u = t.view(torch.uint8)
        u[dst] = u[src]


def _fork_plain(s):
    c = s["case"]
    P, grow, width = c["page"], c["grow"], s["width"]
    table, lens, parents, refs = s["page_table"].long(), s["kv_lens"].long(), s["parents"].long(), s["refs"].long()
    N, dev = refs.numel(), refs.device
    one = torch.ones((), dtype=torch.int64, device=dev)
    held = (lens + P - 1) // P
    slot = torch.arange(table.shape[1], device=dev)
    old = table[slot < held[:, None]]
    length = lens[parents]
    had = held[parents]
    need = (length + grow + P - 1) // P
    slot = torch.arange(width, device=dev)
    out = torch.full((parents.numel(), width), -1, dtype=torch.int64, device=dev)
    most = min(width, table.shape[1])
    take = slot[:most] < had[:, None]
    out[:, :most][take] = table[parents][:, :most][take]
    r = refs.clone().index_add_(0, old, -one.expand(old.numel()))
    kept = out[out >= 0]
    r.index_add_(0, kept, one.expand(kept.numel()))
    # the partly filled pages to be written: the first child keeps one that nobody else holds
    child = torch.arange(parents.numel(), device=dev)
    write = (length % P != 0) & (grow > 0)
    tail = out.gather(1, (had - 1).clamp(min=0)[:, None])[:, 0]
    writers = torch.zeros(N, dtype=torch.int64, device=dev).index_add_(0, tail[write], one.expand(int(write.sum())))
    first = torch.full((N,), N + child.numel(), dtype=torch.int64, device=dev)
    first.scatter_reduce_(0, tail[write], child[write], "amin")
    copy = write & ~((r[tail] == writers[tail]) & (first[tail] == child))
    # free pages in ascending order to the children in turn: the copy first, then further ones
    count = copy.long() + need - had
    start = count.cumsum(0) - count
    free = torch.nonzero(r == 0)[:, 0]
    fresh = (slot >= had[:, None]) & (slot < need[:, None])
    which = start[:, None] + copy.long()[:, None] + slot - had[:, None]
    out[fresh] = free[which[fresh]]
    src, dst = tail[copy], free[start[copy]]
    out[child[copy], had[copy] - 1] = dst
    r.index_add_(0, src, -one.expand(src.numel()))
    r[out[fresh]] = 1
    r[dst] = 1
    _copy_pages(s["cache"], src, dst)
    failed = (count.sum() - free.numel()).clamp(min=0).to(torch.int32).reshape(1)
    return out.to(torch.int32), (length + grow).to(torch.int32), r.to(torch.int32), failed


def _compact_plain(s):
    P, table, refs = s["case"]["page"], s["page_table"], s["refs"]
    live = refs > 0
    count = live.sum()
    page = torch.arange(refs.numel(), device=refs.device)
    src = page[live & (page >= count)]
    dst = page[~live & (page < count)][:src.numel()]
    to = torch.where(live, page, -torch.ones_like(page))
    to[src] = dst
    _copy_pages(s["cache"], src, dst)
    new = torch.where(page < count, refs, torch.zeros_like(refs))
    new[dst] = refs[src]
    held = torch.arange(table.shape[1], device=refs.device) < ((s["kv_lens"].long() + P - 1) // P)[:, None]
    out = torch.where(held, to[table.long().clamp(min=0)], -torch.ones_like(to[:1]))
    return out.to(torch.int32), new, to.to(torch.int32), count.to(torch.int32).reshape(1)


def _two(e):
    """2^e in 32 bits for whole e from -126 to 127, from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _tokens(s, table):
    """Keys and values [..][heads][tokens][dim] of page numbers [..][pages]."""
    kc, vc, ks, vs = s["cache"]
    t = table.long()
    k = kc.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * _two(ks[t].int() - 127)[..., None, None]
    v = vc.view(torch.uint8)[t].view(torch.float8_e4m3fn).float() * _two(vs[t].int() - 127)[..., None, None]
    d = k.dim()
    lead = list(range(d - 4))
    k = k.permute(*lead, d - 3, d - 4, d - 2, d - 1).flatten(d - 3, d - 2)
    v = v.permute(*lead, d - 3, d - 4, d - 1, d - 2).flatten(d - 3, d - 2)
    return k, v


def _weigh(score, v):
    """Largest score, sum of weights, weighted values."""
    m = score.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = score.sub_(m).exp_()
    return m, p.sum(-1, keepdim=True), torch.matmul(p, v)


def _prefix_plain(s):
    c = s["case"]
    H, D, Hq = c["kv_heads"], c["dim"], c["q_heads"]
    G, q, n = Hq // H, s["q"], s["max_q"]
    T, scale = q.shape[0], 1.0 / math.sqrt(D)
    # the prefixes, group by group: rows [head][query head of it][token]
    parts = []
    for i, length in enumerate(s["prefix"]):
        lo, hi = s["rows"][i], s["rows"][i + 1]
        k, v = _tokens(s, s["prefix_table"][i])
        x = q[lo:hi].float().reshape(hi - lo, H, G, D).permute(1, 2, 0, 3).reshape(H, G * (hi - lo), D)
        w = _weigh(torch.matmul(x, k[:, :length].transpose(1, 2).contiguous()).mul_(scale), v[:, :length].contiguous())
        parts.append([t.reshape(H, G, hi - lo, -1).permute(2, 0, 1, 3).reshape(hi - lo, Hq, -1) for t in w])
    m1, l1, o1 = (torch.cat([p[i] for p in parts]) for i in range(3))
    # each sequence's own tokens
    lens, starts = s["kv_lens"].long(), s["q_starts"].long()
    B, count = lens.numel(), starts[1:] - starts[:-1]
    k, v = _tokens(s, s["page_table"])
    S = k.shape[2]
    i = torch.arange(n, device=q.device)
    row = (starts[:-1, None] + i).clamp(max=T - 1)
    x = q[row].float().reshape(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    sc = torch.matmul(x, k.transpose(2, 3).contiguous()).mul_(scale).reshape(B, H, G, n, S)
    pos, t = (lens - count)[:, None] + i, torch.arange(S, device=q.device)
    see = (t < lens[:, None, None]) & (t <= pos[..., None])
    sc.masked_fill_(~see[:, None, None], -math.inf)
    w = _weigh(sc.reshape(B, H, G * n, S), v)
    b = torch.searchsorted(starts[1:].contiguous(), torch.arange(T, device=q.device), right=True)
    j = torch.arange(T, device=q.device) - starts[b]
    m2, l2, o2 = (t.reshape(B, H, G, n, -1).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, -1)[b, j] for t in w)
    m = torch.maximum(m1, m2)
    a1, a2 = (m1 - m).exp(), (m2 - m).exp()
    z = a1 * l1 + a2 * l2
    return ((a1 * o1 + a2 * o2) / z).bfloat16(), (m + z.log()).squeeze(2)


def run(s):
    c = s["case"]
    if own:
        from ultra_bit_dit_amd import lowbit as lb

        if c["op"] == "rotate":
            Hq = c["q_heads"]
            return lb.qk_norm_rope(s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + c["kv_heads"]], s["positions"], s["freqs"],
                                   q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6, pair_axis=s["pair_axis"],
                                   adjacent=c["pairs"] == "adjacent", y_dtype=lb.BF16 if c["out"] == "bf16" else lb.F32)
        if c["op"] == "fork":
            out = lb.kv8_fork(s["cache"], s["page_table"], s["kv_lens"], s["refs"], s["parents"], grow=c["grow"],
                              width=s["width"])
            return tuple(out) + s["cache"]
        if c["op"] == "compact":
            return tuple(lb.kv8_compact(s["cache"], s["page_table"], s["kv_lens"], s["refs"])) + s["cache"]
        return lb.attention_kv8_prefix(s["q"], s["cache"], s["prefix_table"], s["prefix_lens"], s["page_table"], s["kv_lens"],
                                       seq_starts=s["seq_starts"], q_starts=s["q_starts"], max_q=s["max_q"],
                                       max_kv=s["max_kv"], max_prefix=s["max_prefix"], max_seqs=s["max_seqs"],
                                       return_lse=True)
    if c["op"] == "rotate":
        return _rotate_plain(s)
    if c["op"] == "fork":
        return _fork_plain(s) + s["cache"]
    if c["op"] == "compact":
        return _compact_plain(s) + s["cache"]
    return _prefix_plain(s)


# ------------------------------------- the definitions, in 64 bits, one by one


def _exact_rotate(c, s):
    D, R, Hq = c["dim"], c["rot"], c["q_heads"]
    pos = s["positions"].reshape(c["axes"], -1).double()
    f, a = _frequencies(c)
    # a pair is one complex number, turned by e^(i position frequency)
    turn = torch.stack([torch.polar(torch.ones_like(pos[0]), pos[k] * w) for w, k in zip(f, a)], 1)[:, None]
    first = torch.arange(R // 2, device="cuda") * (1 if c["pairs"] == "half" else 2)
    second = first + (R // 2 if c["pairs"] == "half" else 1)
    out = []
    for lo, hi, w in ((0, Hq, s["q_weight"]), (Hq, Hq + c["kv_heads"], s["k_weight"])):
        x = s["qkv"][:, lo:hi].double()
        if w is not None:
            x = x * w.double() * torch.rsqrt(x.square().sum(2, keepdim=True) / D + 1e-6)
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        out.append(x)
    return tuple(out)


def _move64(cache, moves):
    out = [t.double() for t in cache[:2]] + [t.clone() for t in cache[2:]]
    if moves:
        src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
        for t in out:
            t[dst] = t[src]
    return tuple(out)


def _exact_fork(c, s):
    P, grow = c["page"], c["grow"]
    table, lens, parents = s["page_table"].tolist(), s["kv_lens"].tolist(), s["parents"].tolist()
    refs = s["refs"].tolist()
    for row, n in zip(table, lens):
        for p in row[:-(-n // P)]:
            refs[p] -= 1
    rows = [table[p][:-(-lens[p] // P)] for p in parents]
    for row in rows:
        for p in row:
            refs[p] += 1
    tails = [row[-1] if grow and lens[p] % P else None for row, p in zip(rows, parents)]
    writers = {}
    for p in tails:
        if p is not None:
            writers[p] = writers.get(p, 0) + 1
    shared_out = {p for p, n in writers.items() if refs[p] > n}
    free = iter([p for p, n in enumerate(refs) if n == 0])
    moves, kept = [], set()
    for row, p, parent in zip(rows, tails, parents):
        if p is not None:
            if p in shared_out or p in kept:
                row[-1] = next(free)
                moves.append((p, row[-1]))
                refs[p] -= 1
                refs[row[-1]] = 1
            else:
                kept.add(p)
        while len(row) < -(-(lens[parent] + grow) // P):
            row.append(next(free))
            refs[row[-1]] = 1
    out = [row + [-1] * (s["width"] - len(row)) for row in rows]
    return (_i32(out), _i32([lens[p] + grow for p in parents]), _i32(refs), _i32([0])) + _move64(s["cache"], moves)


def _exact_compact(c, s):
    P, refs = c["page"], s["refs"].tolist()
    count = sum(n > 0 for n in refs)
    holes = iter([p for p in range(count) if refs[p] == 0])
    to = [-1 if n == 0 else p if p < count else next(holes) for p, n in enumerate(refs)]
    new = [0] * len(refs)
    for p, n in enumerate(refs):
        if n:
            new[to[p]] = n
    width = s["page_table"].shape[1]
    out = []
    for row, n in zip(s["page_table"].tolist(), s["kv_lens"].tolist()):
        held = -(-n // P)
        out.append([to[p] for p in row[:held]] + [-1] * (width - held))
    moves = [(p, q) for p, q in enumerate(to) if q >= 0 and q != p]
    return (_i32(out), _i32(new), _i32(to), _i32([count])) + _move64(s["cache"], moves)


def _exact_prefix(c, s):
    P, H, D = c["page"], c["kv_heads"], c["dim"]
    G = c["q_heads"] // H
    kc, vc, ks, vs = s["cache"]
    count, prefix, lens = _behind(c)

    def read(table, n, h):
        pg = table[:-(-n // P)].long()
        two = [torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), e[pg, h].double() - 127)[:, None, None]
               for e in (ks, vs)]
        k = (kc[pg, h].double() * two[0]).reshape(-1, D)[:n]
        v = (vc[pg, h].double() * two[1]).transpose(1, 2).reshape(-1, D)[:n]
        return k, v.contiguous()

    O = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    Z = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for h in range(H):
        b, row = 0, 0
        for i, (m, length) in enumerate(zip(count, prefix)):
            k0, v0 = read(s["prefix_table"][i], length, h)
            n_rows = sum(n for n, _ in lens[b:b + m])
            q = s["q"][row:row + n_rows, h * G:(h + 1) * G].double()
            x0 = torch.matmul(q.reshape(-1, D), k0.t().contiguous()).reshape(n_rows, G, length) * D ** -0.5
            at = 0
            for n, t in lens[b:b + m]:
                k1, v1 = read(s["page_table"][b], t, h)
                x1 = torch.matmul(q[at:at + n].reshape(-1, D), k1.t().contiguous()).reshape(n, G, t) * D ** -0.5
                hide = torch.arange(t, device="cuda")[None] > torch.arange(t - n, t, device="cuda")[:, None]
                x = torch.cat((x0[at:at + n], x1.masked_fill(hide[:, None], -math.inf)), 2)
                z = torch.logsumexp(x, 2)
                p = torch.exp(x - z[..., None]).reshape(n * G, -1)
                o = torch.matmul(p[:, :length].contiguous(), v0) + torch.matmul(p[:, length:].contiguous(), v1)
                O[row + at:row + at + n, h * G:(h + 1) * G] = o.reshape(n, G, D)
                Z[row + at:row + at + n, h * G:(h + 1) * G] = z
                at += n
                b += 1
            row += n_rows
    return O, Z


def exact(c, seed):
    s = prepare(c, seed)
    return {"rotate": _exact_rotate, "fork": _exact_fork, "compact": _exact_compact, "prefix": _exact_prefix}[c["op"]](c, s)
