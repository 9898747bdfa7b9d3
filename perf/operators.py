"""Cases for the microscaled 4-bit products and the 8-bit paged attention cache.

Four operators, each in the plain form (elementary torch operations in 32
bits) and as the library call a program makes:

* quantize: rows of activations or weights to MXFP4 (e2m1 codes, one power of
  two for 32 values), the values the codes stand for beside them;
* product: Y = X W^T with W in MXFP4, X in bf16 or quantized to MXFP4 within
  the call;
* append: new keys and values written into a paged cache of e4m3 codes with
  one power of two for each page and head;
* attention: queries against that cache, single tokens or whole prompts.

Layouts.  MXFP4 rows are tiled by 16; byte ((rb G + g) 64 + r + 16 q) 16 + i
of the codes holds elements 2 i (low nibble) and 2 i + 1 of the 32-value block
4 g + q of row 16 rb + r, G = ceil(K / 128); byte ((rb GQ + g/4) 64 + r + 16 q)
4 + g % 4 of the scales holds that block's exponent + 127, GQ = ceil(G / 4).
Cache pages: keys [page][head][token][dim], values [page][head][dim][token].
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token's hidden state, quantized before a 4-bit product: latency
        dict(name="quantize_token", op="quantize", rows=1, K=5120, dtype="bf16"),
        # a down-projection's weights quantized when a model is loaded
        dict(name="quantize_weights", op="quantize", rows=5120, K=17408, dtype="bf16"),
        # output projection of one decoded token, bf16 activations
        dict(name="product_token", op="product", M=1, N=5120, K=5120, x="bf16", y="f32"),
        # down projection of five tokens (four drafted and the next one)
        dict(name="product_verify", op="product", M=5, N=5120, K=17408, x="bf16", y="bf16"),
        # fused q/k/v of a ragged prompt chunk, bf16 activations
        dict(name="product_chunk", op="product", M=509, N=15360, K=5120, x="bf16", y="bf16"),
        # fused gate/up of a long prompt, activations quantized in the call
        dict(name="product_prompt", op="product", M=4608, N=34816, K=5120, x="mxfp4", y="bf16"),
        # one decoded token of each of 64 sequences into the cache
        dict(name="append_step", op="append", seqs=64, new=1, ctx=4096, kv_heads=8, dim=128, page=64),
        # prompts of odd lengths behind a cached prefix, small pages
        dict(name="append_prompt", op="append", seqs=3, new=4093, ctx=5000, kv_heads=8, dim=128, page=16),
        # one short sequence, one token: the smallest decode call
        dict(name="attention_short", op="attention", seqs=1, new=1, ctx=77, q_heads=40, kv_heads=8, dim=128,
             page=16, causal=True, window=0),
        # a decode batch of ragged contexts, grouped heads
        dict(name="attention_batch", op="attention", seqs=32, new=1, ctx=16384, q_heads=40, kv_heads=8, dim=128,
             page=64, causal=True, window=0),
        # one token against a very long context, wide heads
        dict(name="attention_long", op="attention", seqs=1, new=1, ctx=131071, q_heads=24, kv_heads=4, dim=256,
             page=128, causal=True, window=0),
        # two prompts behind a short cached prefix
        dict(name="attention_prompt", op="attention", seqs=2, new=3999, ctx=4500, q_heads=40, kv_heads=8, dim=128,
             page=64, causal=True, window=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("quantize", "product", "append", "attention"))
    if op == "quantize":
        while True:
            rows, K = _log_int(rng, 1, 20000), 32 * _log_int(rng, 1, 600)
            if rows * K <= 5120 * 17408:
                return dict(op=op, rows=rows, K=K, dtype=rng.choice(("bf16", "f32")))
    if op == "product":
        while True:
            M, N, K = _log_int(rng, 1, 5000), _log_int(rng, 16, 36000), 32 * _log_int(rng, 2, 600)
            if M * N * K <= 4608 * 34816 * 5120 and M * N <= 160_000_000:
                return dict(op=op, M=M, N=N, K=K, x=rng.choice(("bf16", "mxfp4")), y=rng.choice(("bf16", "f32")))
    kv_heads, dim, page = rng.choice((1, 2, 4, 5, 8, 40)), rng.choice((64, 128, 256)), rng.choice((16, 32, 64, 128))
    if op == "append":
        while True:
            seqs, new = _log_int(rng, 1, 96), _log_int(rng, 1, 4200)
            ctx = new + _log_int(rng, 1, 4000)
            if seqs * ctx * kv_heads * dim <= 64 * 4096 * 8 * 128 and seqs * new * kv_heads * dim <= 3 * 4093 * 8 * 128:
                return dict(op=op, seqs=seqs, new=new, ctx=ctx, kv_heads=kv_heads, dim=dim, page=page)
    while True:
        step = rng.random() < 0.5
        seqs = _log_int(rng, 1, 48 if step else 8)
        new = rng.choice((1, 1, 1, 2, 5)) if step else _log_int(rng, 6, 4000)
        ctx = new + _log_int(rng, 1, 30000 if step else 4500)
        q_heads = kv_heads * rng.choice((1, 2, 3, 5, 6, 8))
        if (q_heads <= 64 and seqs * q_heads * new * ctx <= 2 * 40 * 3999 * 4500
                and q_heads * dim * seqs * new * ctx <= 2 * 40 * 128 * 3999 * 4500
                and seqs * ctx * kv_heads * dim <= 32 * 16384 * 8 * 128):
            causal = rng.random() < 0.8
            window = _log_int(rng, 1, ctx) if causal and rng.random() < 0.25 else 0
            return dict(op=op, seqs=seqs, new=new, ctx=ctx, q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page,
                        causal=causal, window=window)


def _lengths(c):
    """(new tokens, length with them) of each sequence: ragged, the first one the longest."""
    out = []
    for i in range(c["seqs"]):
        f = 1.0 - 0.75 * ((i * 0.6180339887) % 1.0)
        n = max(1, int(c["new"] * f))
        out.append((n, max(n, int(c["ctx"] * f))))
    return out


def work(c):
    if c["op"] == "quantize":
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["rows"] * c["K"]
        return {"bytes": n * (2 * e + 0.5 + 1 / 32), "flops": 4 * n}
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K * (0.5 + 1 / 32) + M * K * 2 + M * N * (2 if c["y"] == "bf16" else 4), "flops": 2 * M * N * K}
    new = sum(n for n, _ in _lengths(c))
    hd = c["kv_heads"] * c["dim"]
    if c["op"] == "append":
        pages = sum((t - 1) // c["page"] - (t - n) // c["page"] + 1 for n, t in _lengths(c))
        return {"bytes": 2 * (new * hd * 3 + pages * c["kv_heads"]), "flops": 4 * new * hd}
    pairs, read = 0, 0
    for n, t in _lengths(c):
        w = c["window"]
        if not c["causal"]:
            pairs, read = pairs + n * t, read + t
            continue
        first = t - n  # position of the first query
        pairs += sum(range(first + 1, t + 1)) if not w else sum(min(p + 1, w) for p in range(first, t))
        read += t if not w else min(t, n + w - 1)
    by = read * 2 * (hd + c["kv_heads"] / c["page"]) + new * c["q_heads"] * (4 * c["dim"] + 4)
    return {"bytes": by, "flops": 4 * pairs * c["q_heads"] * c["dim"]}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def prepare(c, seed):
    g = _gen(seed)
    s = {"case": dict(c)}
    if c["op"] == "quantize":
        x = _randn(g, c["rows"], c["K"])
        x *= torch.exp(_randn(g, c["rows"], 1))  # rows of different sizes
        s["x"] = x if c["dtype"] == "f32" else x.bfloat16()
    elif c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        w = _randn(g, N, K).mul_(0.02)
        s["codes"], s["scales"] = _pack(*_quantize(w))
        s["x"] = _randn(g, M, K).bfloat16()
    else:
        lens = _lengths(c)
        B, P, H, D = c["seqs"], c["page"], c["kv_heads"], c["dim"]
        width = max(-(-t // P) for _, t in lens)
        pages = B * width + 3
        perm = torch.randperm(pages, device="cuda", generator=g)[: B * width]
        s["page_table"] = perm.to(torch.int32).reshape(B, width).contiguous()
        s["kv_lens"] = torch.tensor([t for _, t in lens], dtype=torch.int32, device="cuda")
        starts = [0]
        for n, _ in lens:
            starts.append(starts[-1] + n)
        s["q_starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        s["max_q"], s["max_kv"] = max(n for n, _ in lens), max(t for _, t in lens)
        T = starts[-1]
        for n, shape in (("k", (pages, H, P, D)), ("v", (pages, H, D, P))):
            s[n + "_codes"] = _randn(g, *shape).mul_(90).clamp_(-448, 448).to(torch.float8_e4m3fn)
            s[n + "_scales"] = torch.randint(118, 122, (pages, H), device="cuda", generator=g).to(torch.uint8)
        if c["op"] == "append":
            # keys and values lie beside the queries in a fused projection's output
            qkv = _randn(g, T, 3, H, D)
            qkv *= torch.exp2(torch.randint(-1, 3, (T, 1, 1, 1), device="cuda", generator=g).float())
            s["qkv"] = qkv.bfloat16()
        else:
            s["q"] = _randn(g, T, c["q_heads"], D).bfloat16()
    return s


# ------------------------------------------------- the formulas, in 32 bits


def _two(e):
    """2^e in 32 bits for whole e from -127 to 127, exactly (from its bits: a power function may be a step off)."""
    e = e.int()
    return torch.where(e < -126, torch.full_like(e, 1 << 22), (e + 127) << 23).view(torch.float32)


def _quantize(x):
    """Codes (0..15) and biased exponents of blocks of 32: 2^e, e = floor(log2 max|x|) - 2;
    codes are round to nearest, ties to even, of x / 2^e, at most 6."""
    rows, K = x.shape
    b = x.float().reshape(rows, K // 32, 32)
    a = b.abs().amax(2)
    e = (torch.frexp(a)[1] - 3).clamp(min=-127)
    e = torch.where(a == 0, torch.full_like(e, -127), e)
    v = b * _two(-e)[..., None]
    m = v.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    r = ((m / step).round() * step).clamp(max=6.0)
    code = torch.where(r < 2, 2 * r, torch.where(r < 4, r + 2, r / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    return code.reshape(rows, K), (e + 127).to(torch.uint8)


def _dequantize(code, exp):
    rows, K = code.shape
    mag = torch.tensor(E2M1, device=code.device)[(code & 7).long()]
    v = torch.where(code > 7, -mag, mag).reshape(rows, K // 32, 32)
    return (v * _two(exp.int() - 127)[..., None]).reshape(rows, K)


def _pack(code, exp):
    """Dense codes [rows][K] and exponents [rows][K/32] in the tiled layout."""
    rows, K = code.shape
    RB, G = -(-rows // 16), -(-K // 128)
    GQ = -(-G // 4)
    full = torch.zeros(RB * 16, G * 128, dtype=torch.uint8, device=code.device)
    full[:rows, :K] = code
    full = full[:, 0::2] | (full[:, 1::2] << 4)
    pc = full.reshape(RB, 16, G, 4, 16).permute(0, 2, 3, 1, 4).reshape(-1).contiguous()
    se = torch.full((RB * 16, GQ * 16), 127, dtype=torch.uint8, device=code.device)
    se[:rows, : K // 32] = exp
    ps = se.reshape(RB, 16, GQ, 4, 4).permute(0, 2, 4, 1, 3).reshape(-1).contiguous()
    return pc, ps


def _unpack(pc, ps, rows, K):
    RB, G = -(-rows // 16), -(-K // 128)
    GQ = -(-G // 4)
    by = pc.reshape(RB, G, 4, 16, 16).permute(0, 3, 1, 2, 4).reshape(RB * 16, G * 64)
    code = torch.stack((by & 15, by >> 4), 2).reshape(RB * 16, G * 128)[:rows, :K]
    exp = ps.reshape(RB, GQ, 4, 16, 4).permute(0, 3, 1, 4, 2).reshape(RB * 16, GQ * 16)[:rows, : K // 32]
    return code, exp


def _value(codes, scales):
    """Cache pages as numbers: codes [n][H][..][..] times 2^(scale - 127) of each page and head."""
    return codes.float() * _two(scales.int() - 127)[..., None, None]


def _page_exponent(a):
    """The smallest e, at least -127, with a <= 448 * 2^e."""
    m, x = torch.frexp(a)  # a = m 2^x, m in [0.5, 1): 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).int()
    return torch.where(a == 0, torch.full_like(e, -127), e).clamp(min=-127)


def _append_plain(s):
    c = s["case"]
    B, P, H, D = c["seqs"], c["page"], c["kv_heads"], c["dim"]
    T = s["qkv"].shape[0]
    lens, starts = s["kv_lens"].long(), s["q_starts"].long()
    n = starts[1:] - starts[:-1]
    first = lens - n  # position of the first new token
    span = (s["max_q"] + P - 2) // P + 1
    at = torch.minimum(first[:, None] // P + torch.arange(span, device="cuda"), ((lens - 1) // P)[:, None])  # [B][span]
    page = s["page_table"].long().gather(1, at).reshape(-1)
    pos = (at * P)[..., None] + torch.arange(P, device="cuda")  # [B][span][P]
    isnew = ((pos >= first[:, None, None]) & (pos < lens[:, None, None])).reshape(-1, P)
    isold = (pos < first[:, None, None]).reshape(-1, P)
    tok = (starts[:-1, None, None] + pos - first[:, None, None]).clamp(0, T - 1).reshape(-1, P)
    for name, part in (("k", 1), ("v", 2)):
        codes, scales = s[name + "_codes"].view(torch.uint8), s[name + "_scales"]
        old8 = codes[page]
        old = _value(old8.view(torch.float8_e4m3fn), scales[page])
        new = s["qkv"][tok, part].float().permute(0, 2, 1, 3)  # [page][H][P][D]
        mn, mo = isnew[:, None, :, None], isold[:, None, :, None]
        if name == "v":
            new, mn, mo = new.transpose(2, 3), mn.transpose(2, 3), mo.transpose(2, 3)
        e = _page_exponent((new * mn).abs().amax((2, 3)))
        e = torch.where(isold.any(1)[:, None], torch.maximum(e, scales[page].int() - 127), e)
        e = torch.where(isnew.any(1)[:, None], e, scales[page].int() - 127)
        v = torch.where(mn, new, old) * _two(-e)[..., None, None]
        out8 = torch.where(mn | mo, v.to(torch.float8_e4m3fn).view(torch.uint8), old8)
        codes[page] = out8
        scales[page] = (e + 127).to(torch.uint8)


def _attention_plain(s):
    c = s["case"]
    B, P, H, D, Hq = c["seqs"], c["page"], c["kv_heads"], c["dim"], c["q_heads"]
    G, n, q = Hq // H, s["max_q"], s["q"]
    table = s["page_table"].long()
    S = table.shape[1] * P
    k = _value(s["k_codes"].view(torch.uint8)[table].view(torch.float8_e4m3fn), s["k_scales"][table])
    k = k.permute(0, 2, 4, 1, 3).reshape(B, H, D, S)
    v = _value(s["v_codes"].view(torch.uint8)[table].view(torch.float8_e4m3fn), s["v_scales"][table])
    v = v.permute(0, 2, 1, 4, 3).reshape(B, H, S, D)
    lens, starts = s["kv_lens"].long(), s["q_starts"].long()
    count = starts[1:] - starts[:-1]
    i = torch.arange(n, device="cuda")
    row = (starts[:-1, None] + i).clamp(max=q.shape[0] - 1)  # [B][n]
    qf = q[row].float().reshape(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    sc = torch.matmul(qf, k).mul_(1.0 / math.sqrt(D)).reshape(B, H, G, n, S)
    pos = (lens - count)[:, None] + i  # position of each query
    t = torch.arange(S, device="cuda")
    see = t < lens[:, None, None]
    if c["causal"]:
        see = see & (t <= pos[..., None])
    if c["window"]:
        see = see & (t > pos[..., None] - c["window"])
    see = see.expand(B, n, S)[:, None, None]
    sc = sc.masked_fill_(~see, -math.inf)
    m = sc.amax(4, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m0).exp_()
    l = p.sum(4, keepdim=True)
    o = torch.matmul(p.reshape(B, H, G * n, S), v).reshape(B, H, G, n, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m0 + l.log()).squeeze(4)
    b = torch.searchsorted(starts[1:], torch.arange(q.shape[0], device="cuda"), right=True)
    j = torch.arange(q.shape[0], device="cuda") - starts[b]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[b, j]
    lse = lse.permute(0, 3, 1, 2).reshape(B, n, Hq)[b, j]
    return o.bfloat16(), lse


def run(s):
    c = s["case"]
    if own:
        from ultra_bit_dit_amd import lowbit as lb

        if c["op"] == "quantize":
            return lb.quantize_mxfp4(s["x"], values=True)[2]
        if c["op"] == "product":
            y = lb.F32 if c["y"] == "f32" else lb.BF16
            if c["x"] == "bf16":
                return lb.gemm_mxfp4(c["M"], c["N"], c["K"], s["codes"], s["scales"], s["x"], y_dtype=y)
            xc, xs = lb.quantize_mxfp4(s["x"])
            return lb.gemm_mxfp4(c["M"], c["N"], c["K"], s["codes"], s["scales"], xc, x_scales=xs, y_dtype=y)
        cache = (s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
        if c["op"] == "append":
            lb.kv8_append(cache, s["page_table"], s["kv_lens"], s["qkv"][:, 1], s["qkv"][:, 2],
                          q_starts=s["q_starts"], max_q=s["max_q"], max_kv=s["max_kv"])
            return cache
        return lb.attention_kv8(s["q"], cache, s["page_table"], s["kv_lens"], q_starts=s["q_starts"],
                                max_q=s["max_q"], max_kv=s["max_kv"], causal=c["causal"], window=c["window"],
                                return_lse=True)
    if c["op"] == "quantize":
        return _dequantize(*_quantize(s["x"])).to(s["x"].dtype)
    if c["op"] == "product":
        x = s["x"].float() if c["x"] == "bf16" else _dequantize(*_quantize(s["x"]))
        y = torch.matmul(x, _dequantize(*_unpack(s["codes"], s["scales"], c["N"], c["K"])).t())
        return y if c["y"] == "f32" else y.bfloat16()
    if c["op"] == "append":
        _append_plain(s)
        return s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"]
    return _attention_plain(s)


# ------------------------------------- the definitions, in 64 bits, one by one


def _two64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _mx_nearest64(x):
    """MXFP4 values of x in 64 bits, by comparing with the midpoints of the code values."""
    rows, K = x.shape
    b = x.double().reshape(rows, K // 32, 32)
    top = b.abs().amax(2, keepdim=True)
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140)))
    e = torch.where(_two64(e) > top, e - 1, torch.where(_two64(e + 1) <= top, e + 1, e))
    unit = _two64(torch.clamp(e - 2, min=-127.0))
    a = (b / unit).abs()
    idx = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
           + (a >= 3.5).int() + (a > 5.0).int())
    v = torch.tensor(E2M1, dtype=torch.float64, device=x.device)[idx.long()] * torch.sign(b)
    return (v * unit).reshape(rows, K)


def _e4m3_nearest64(x):
    """The e4m3 numbers nearest to x (ties to even), in 64 bits."""
    a = x.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    e = torch.where(_two64(e) > a.clamp(min=2.0 ** -6), e - 1, torch.where(_two64(e + 1) <= a, e + 1, e))
    step = _two64(e - 3)
    return torch.sign(x) * torch.round(a / step) * step


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "quantize":
        return _mx_nearest64(s["x"])
    if c["op"] == "product":
        N, K = c["N"], c["K"]
        n = torch.arange(N, device="cuda")[:, None]
        k = torch.arange(K, device="cuda")[None]
        lane = n % 16 + 16 * ((k // 32) % 4)
        G, GQ = -(-K // 128), -(-(-(-K // 128)) // 4)
        byte = s["codes"][(((n // 16) * G + k // 128) * 64 + lane) * 16 + (k % 32) // 2]
        code = torch.where(k % 2 == 1, byte >> 4, byte & 15)
        exp = s["scales"][(((n // 16) * GQ + k // 512) * 64 + lane) * 4 + (k // 128) % 4]
        w = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")[code.long()]
        w *= _two64(exp.int() - 127)
        x = s["x"].double() if c["x"] == "bf16" else _mx_nearest64(s["x"])
        return x @ w.t().contiguous()
    lens = _lengths(c)
    P, H, D = c["page"], c["kv_heads"], c["dim"]
    table = s["page_table"].tolist()
    if c["op"] == "append":
        k, v = s["k_codes"].double(), s["v_codes"].double().transpose(2, 3).contiguous()
        ke, ve = s["k_scales"].clone(), s["v_scales"].clone()
        t0 = 0
        for b, (n, t) in enumerate(lens):
            for j in range((t - n) // P, (t - 1) // P + 1):
                page, lo, hi = table[b][j], max(t - n, j * P), min(t, (j + 1) * P)
                old = max(0, (t - n) - j * P)
                for part, cc, ee in ((1, k, ke), (2, v, ve)):
                    x = s["qkv"][t0 + lo - (t - n):t0 + hi - (t - n), part].double().transpose(0, 1)  # [H][tokens][D]
                    a = x.abs().amax((1, 2)) / 448
                    e = torch.ceil(torch.log2(a.clamp(min=2.0 ** -127))).clamp(min=-127.0)
                    e = torch.where(_two64(e - 1) >= a, (e - 1).clamp(min=-127.0), torch.where(_two64(e) < a, e + 1, e))
                    was = ee[page].double() - 127
                    e = torch.maximum(e, was) if old else e
                    if old:
                        cc[page, :, :old] = _e4m3_nearest64(cc[page, :, :old] * _two64(was - e)[:, None, None])
                    cc[page, :, lo - j * P:hi - j * P] = _e4m3_nearest64(x / _two64(e)[:, None, None])
                    ee[page] = (e + 127).to(torch.uint8)
            t0 += n
        return k, v.transpose(2, 3).contiguous(), ke, ve
    G = c["q_heads"] // H
    out, lses, t0 = [], [], 0
    for b, (n, t) in enumerate(lens):
        pg = torch.tensor(table[b][: -(-t // P)], device="cuda")
        pos = torch.arange(t - n, t, device="cuda")[:, None]
        key = torch.arange(t, device="cuda")[None]
        hide = (key > pos) if c["causal"] else torch.zeros(n, t, dtype=torch.bool, device="cuda")
        if c["window"]:
            hide = hide | (key <= pos - c["window"])
        os, ls = [], []
        for h in range(H):
            k = (s["k_codes"][pg, h].double() * _two64(s["k_scales"][pg, h].int() - 127)[:, None, None]).reshape(-1, D)[:t]
            v = s["v_codes"][pg, h].double() * _two64(s["v_scales"][pg, h].int() - 127)[:, None, None]
            v = v.transpose(1, 2).reshape(-1, D)[:t].contiguous()
            for g in range(G):
                x = s["q"][t0:t0 + n, h * G + g].double() @ k.t().contiguous() * D ** -0.5
                x = x.masked_fill(hide, -math.inf)
                z = torch.logsumexp(x, 1)
                os.append(torch.exp(x - z[:, None]) @ v)
                ls.append(z)
        out.append(torch.stack(os, 1))
        lses.append(torch.stack(ls, 1))
        t0 += n
    return torch.cat(out), torch.cat(lses)
