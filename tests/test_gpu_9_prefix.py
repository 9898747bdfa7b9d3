"""Attention behind shared prefixes on the GPU against the plain 64-bit form, and
a run of everything that serves many continuations of a prompt."""
import numpy as np
import pytest
import torch

import mx_ref as M
import serve_ref as R
from test_gpu_9_kv8 import Cache, f64, fill, i32, tokens
from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu


class Call:
    """Groups of sequences: prefix lengths, sequences of each group, new tokens and own length of each sequence."""

    def __init__(self, prefix, count, new, own, Hq, H, D, P, seed=0):
        self.prefix, self.count, self.new, self.own = prefix, count, new, own
        self.G, self.B, self.Hq, self.H, self.D, self.P = len(prefix), len(own), Hq, H, D, P
        lens = list(prefix) + list(own)
        self.c = Cache(lens, P, H, D, seed)
        fill(self.c, lens, 100 + seed)
        t = self.c.tables()
        self.prefix_table, self.table = t[:self.G], t[self.G:]
        self.rows = np.concatenate([[0], np.cumsum(new)])
        self.q = tokens(int(self.rows[-1]) + 2, Hq, D, 7 + seed)  # two rows behind the last sequence
        self.starts = np.concatenate([[0], np.cumsum(count)])

    def args(self, **kw):
        a = dict(seq_starts=i32(self.starts), q_starts=i32(self.rows), max_q=max(max(self.new), 1), max_kv=max(max(self.own), 1),
                 max_prefix=max(max(self.prefix), 1), max_seqs=max(max(self.count), 1), return_lse=True)
        a.update(kw)
        return a

    def run(self, **kw):
        O = torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        a = self.args(O=O, lse=lse, **kw)
        return lb.attention_kv8_prefix(self.q, self.c.gpu, self.prefix_table, i32(self.prefix), self.table, i32(self.own), **a)

    def check(self, out, what, causal=True, scale=None, rows=None, some=None):
        O, lse = f64(out[0]), f64(out[1])
        assert np.all(O[self.rows[-1]:] == 7) and np.all(lse[self.rows[-1]:] == 7), f"{what}: rows behind the last sequence"
        scale = self.D ** -0.5 if scale is None else scale
        q = f64(self.q)
        for b in range(self.B):
            if self.new[b] == 0 or (some and b % max(1, self.B // some) and b != self.B - 1):
                continue
            g = int(np.searchsorted(self.starts, b, side="right")) - 1
            Kp, Vp = self.c.read(g, self.prefix[g]) if 0 <= g < self.G else (np.zeros((0, self.H, self.D)),) * 2
            Ko, Vo = self.c.read(self.G + b, self.own[b])
            lo, n = int(self.rows[b]), self.new[b]
            pick = range(n) if rows is None or n <= rows else sorted({0, n - 1, *np.random.default_rng(b).integers(0, n, rows)})
            for i in pick:
                ref, z, A, eps = R.attention_prefix(q[lo + i:lo + i + 1], Kp, Vp, Ko, Vo, self.own[b] - n + i, scale, causal)
                T = len(Kp) + len(Ko)
                err = np.abs(O[lo + i] - ref[0])
                tol = M.attention_tolerance(ref, A, eps, T)[0]
                assert np.all(err <= tol), f"{what}: sequence {b} row {i}: {(err / np.maximum(tol, 1e-300)).max()} of the bound"
                seen = np.isfinite(z[0])
                assert np.all((lse[lo + i] == -np.inf) == ~seen), f"{what}: lse of rows that see nothing"
                e = np.abs(lse[lo + i] - z[0])[seen]
                assert np.all(e <= M.lse_tolerance(z, eps, T)[0][seen]), f"{what}: lse"


CASES = {
    # few rows in all: both launches read the cache straight into registers
    "one": dict(prefix=[37], count=[2], new=[1, 1], own=[1, 30]),
    # prefixes of 0 and 1 token, an empty group, sequences without new or without own tokens, of no group
    "corners": dict(prefix=[0, 1, 50, 64], count=[1, 2, 0, 3], new=[1, 0, 2, 1, 3, 0, 1], own=[5, 9, 2, 0, 3, 0, 40]),
    # whole pages, parts of pages; rows for one tile of a prompt and more
    "tiles": dict(prefix=[200, 333], count=[5, 9], new=[4] * 14, own=[4 + 7 * i for i in range(14)]),
    # many single tokens behind a longer prefix (parts of its steps)
    "batch": dict(prefix=[1500], count=[40], new=[1] * 40, own=[1 + (17 * i) % 150 for i in range(40)]),
    # prompts behind a prefix: many rows of their own
    "prompts": dict(prefix=[130, 600], count=[2, 1], new=[150, 3, 170], own=[150, 90, 400]),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("Hq,H,D,P", [(5, 1, 64, 16), (8, 2, 128, 64), (16, 2, 128, 32), (4, 2, 256, 128), (6, 6, 64, 32)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_prefix(name, Hq, H, D, P, causal):
    print(f"prefix {name} {Hq}/{H} D={D} P={P} causal={causal}", flush=True)
    k = Call(**CASES[name], Hq=Hq, H=H, D=D, P=P, seed=D + P)
    out = k.run(causal=causal)
    k.check(out, name, causal, rows=6)
    again = k.run(causal=causal)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.parametrize("Hq,H,D,P,B,n,L", [(40, 8, 128, 64, 16, 1, 4000), (16, 4, 64, 32, 30, 5, 2500), (12, 2, 256, 128, 9, 2, 3000),
                                            (32, 1, 128, 16, 12, 1, 700)])
def test_sizes_of_plans(Hq, H, D, P, B, n, L):
    """Rows of a group past a tile of 128 and of 256, many parts, several groups of different lengths."""
    print(f"plans {Hq}/{H} D={D} B={B} n={n} L={L}", flush=True)
    k = Call(prefix=[L, L // 3, 10], count=[B - 3, 2, 1], new=[n] * B, own=[n + 11 * (i % 9) for i in range(B)], Hq=Hq, H=H, D=D, P=P)
    k.check(k.run(), "plans", rows=2)
    # loose bounds choose other kernels and parts; the same within the bound
    k.check(k.run(max_q=None, max_seqs=None, max_kv=None, max_prefix=None), "loose bounds", rows=2)


OWN = lambda n, first=30: [first + 11 * (i % 9) for i in range(n)]
LAUNCHES = {
    # one prompt launch, its tiles in parts, uncut, or cut in the last round
    "parts, 64": dict(prefix=[700, 90], count=[3, 2], new=[70, 100, 3, 90, 61], own=[70, 150, 30, 90, 300], Hq=8, H=2, D=64, P=16),
    "parts, 128": dict(prefix=[700, 90], count=[3, 2], new=[30, 20, 3, 30, 31], own=[70, 150, 30, 90, 300], Hq=8, H=2, D=128, P=16),
    "parts, 256": dict(prefix=[500, 90], count=[3, 1], new=[60, 20, 3, 30], own=[70, 150, 30, 90], Hq=4, H=4, D=256, P=64),
    "uncut, 64": dict(prefix=[300], count=[100], new=[130] * 100, own=[130] * 100, Hq=8, H=8, D=64, P=64),
    "uncut, 128": dict(prefix=[150], count=[40], new=[120] * 40, own=[120] * 40, Hq=32, H=8, D=128, P=64),
    "uncut, 256": dict(prefix=[300], count=[40], new=[130] * 40, own=[130] * 40, Hq=8, H=8, D=256, P=64),
    "last round, 128": dict(prefix=[300, 400], count=[10, 30], new=[130] * 40, own=[130] * 40, Hq=32, H=8, D=128, P=64),
    # the groups in prompt tiles of 128 and 256 rows, then the sequences, in pieces or whole
    "groups, 64": dict(prefix=[8000], count=[60], new=[2] * 60, own=OWN(60), Hq=16, H=4, D=64, P=64),
    "groups, pieces": dict(prefix=[20000], count=[24], new=[1] * 24, own=OWN(24, 300), Hq=4, H=4, D=64, P=64),
    "groups, 128": dict(prefix=[9000, 3000], count=[30, 3], new=[1] * 33, own=OWN(33), Hq=16, H=4, D=128, P=64),
    "groups, 256 rows": dict(prefix=[9000, 3000], count=[60, 3], new=[1] * 63, own=OWN(63), Hq=16, H=4, D=128, P=64),
    "groups, 256": dict(prefix=[9000, 500], count=[40, 2], new=[1] * 42, own=OWN(42), Hq=12, H=2, D=256, P=128),
    # the groups in attn_decode too
    "few, 64": dict(prefix=[20000], count=[16], new=[1] * 16, own=OWN(16), Hq=8, H=8, D=64, P=64),
    "few, 64, 32 rows a wave": dict(prefix=[24000], count=[16], new=[1] * 16, own=OWN(16), Hq=32, H=8, D=64, P=64),
    "few, 128": dict(prefix=[30000], count=[16], new=[1] * 16, own=OWN(16, 300), Hq=8, H=8, D=128, P=64),
    "few, 256": dict(prefix=[20000], count=[14], new=[1] * 14, own=OWN(14, 300), Hq=4, H=4, D=256, P=128),
    # again parts and uncut tiles of prompts
    "parts, 64, again": dict(prefix=[3000, 90], count=[3, 2], new=[70, 100, 30, 90, 61], own=[70, 150, 30, 90, 300], Hq=32, H=2, D=64, P=16),
    "parts, 128, again": dict(prefix=[3000, 90], count=[3, 2], new=[32, 32, 3, 32, 31], own=[70, 150, 40, 90, 300], Hq=24, H=6, D=128, P=16),
    "parts, 128, 256 rows": dict(prefix=[1000, 90], count=[3, 2], new=[70, 100, 3, 90, 61], own=[70, 150, 30, 90, 300], Hq=32, H=4, D=128, P=16),
    "uncut, 128, 128 rows": dict(prefix=[100, 90], count=[30, 30], new=[40] * 60, own=[50] * 60, Hq=24, H=8, D=128, P=16),
    # one attn_decode: a workgroup for each tile or several for each, and equal shares
    "tiles, 64": dict(prefix=[900, 90], count=[9, 5], new=[1] * 14, own=OWN(14), Hq=16, H=8, D=64, P=16),
    "pieces, 64": dict(prefix=[2900, 90], count=[9, 5], new=[1] * 14, own=OWN(14), Hq=16, H=8, D=64, P=16),
    "tiles, 64, 32 rows a wave": dict(prefix=[900, 1500], count=[9, 50], new=[5] * 59, own=OWN(59), Hq=32, H=8, D=64, P=32),
    "pieces, 64, 32 rows a wave": dict(prefix=[3000, 800], count=[9, 1], new=[5] * 10, own=OWN(10), Hq=20, H=5, D=64, P=16),
    "tiles, 128": dict(prefix=[700, 800], count=[19, 60], new=[2] * 79, own=OWN(79), Hq=20, H=4, D=128, P=16),
    "pieces, 128": dict(prefix=[3000, 800], count=[9, 1], new=[2] * 10, own=OWN(10), Hq=20, H=4, D=128, P=16),
    "tiles, 256": dict(prefix=[300, 200], count=[19, 30], new=[1] * 49, own=OWN(49), Hq=12, H=4, D=256, P=16),
    "pieces, 256": dict(prefix=[1500, 800], count=[9, 1], new=[1] * 10, own=OWN(10), Hq=4, H=4, D=256, P=16),
    "shares, 64": dict(prefix=[300, 200], count=[100, 130], new=[1] * 230, own=OWN(230), Hq=12, H=4, D=64, P=16),
    "shares, 64, 32 rows a wave": dict(prefix=[60000, 90, 700], count=[2, 1, 3], new=[5] * 6, own=OWN(6), Hq=32, H=8, D=64, P=128),
    "shares, 128": dict(prefix=[300, 200], count=[100, 130], new=[1] * 230, own=OWN(230), Hq=12, H=4, D=128, P=16),
    "shares, 256": dict(prefix=[40000, 90], count=[2, 1], new=[1] * 3, own=OWN(3), Hq=8, H=8, D=256, P=128),
}


@pytest.mark.parametrize("name", LAUNCHES)
def test_every_launch(name):
    """Sizes that take each of the launches by the expected times; softmax scales of both signs and 0; some rows of some
    sequences against the plain form, all of them the same twice."""
    print(f"launch {name}", flush=True)
    k = Call(**LAUNCHES[name])
    for scale in (None, -0.3, 0.0):
        out = k.run(softmax_scale=scale)
        again = k.run(softmax_scale=scale)
        assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
        k.check(out, f"{name} scale {scale}", scale=scale, rows=2, some=6 if scale is None else 2)


def test_equal_groups_without_starts():
    """seq_starts and q_starts None; a softmax scale below zero and at zero."""
    k = Call(prefix=[90, 90], count=[3, 3], new=[2] * 6, own=[2, 5, 9, 30, 2, 17], Hq=4, H=2, D=64, P=16)
    q = k.q[:12].contiguous()
    for scale in (None, -0.2, 0.0):
        a = lb.attention_kv8_prefix(q, k.c.gpu, k.prefix_table, i32(k.prefix), k.table, i32(k.own), softmax_scale=scale, return_lse=True)
        b = k.run(softmax_scale=scale)
        k.check(b, f"scale {scale}", scale=scale)
        pad = [torch.cat((x, y[12:])) for x, y in zip(a, b)]
        k.check(pad, f"scale {scale}, no starts", scale=scale)


def test_nan_and_infinity():
    """A NaN in one group's prefix reaches that group's rows alone, one in a sequence's own tokens
    its rows alone; NaN and infinities in pages behind the lengths reach nobody; an infinite query."""
    k = Call(prefix=[40, 70], count=[2, 3], new=[1] * 5, own=[20, 3, 8, 33, 5], Hq=4, H=1, D=64, P=16)
    clean = [x.clone() for x in k.run()]
    k.check(clean, "clean")
    kc, vc, ks, vs = k.c.gpu
    v = vc.view(torch.uint8)
    page = k.c.table[0, 1]
    v[page, 0, 5, 3] = 0x7F  # group 0, token 19, dim 5
    out = k.run()
    assert out[0][:2, :, 5].isnan().all() and not out[0][:2, :, :5].isnan().any()
    assert torch.equal(out[0][2:], clean[0][2:]) and torch.equal(out[1], clean[1])
    v[page, 0, 5, 3] = 0
    kc.view(torch.uint8)[k.c.table[2 + 3, 2], 0, 0] = 0x7F  # own token 32 of sequence 3: the last one, all of its dims
    out = k.run()
    assert out[0][3].isnan().all() and torch.equal(out[0][[2, 4]], clean[0][[2, 4]])
    k.q[4] = float("inf")
    out = k.run()
    assert out[0][4].isnan().all() and torch.equal(out[0][2], clean[0][2])


def test_bad_pages_and_lengths():
    """Unreadable pages of either table are not seen and counted; lengths past their bounds, starts
    outside the batch stay inside the buffers."""
    k = Call(prefix=[64, 48], count=[2, 2], new=[1, 1, 1, 1], own=[20, 20, 20, 20], Hq=4, H=2, D=128, P=16)
    t = k.c.table
    t[0, 1], t[1, 0], t[2 + 2, 1] = -1, 10 ** 6, 10 ** 9
    tt = k.c.tables()
    k.prefix_table, k.table = tt[:2], tt[2:]
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = k.run(bad_pages=bad)
    assert bad.item() >= 3
    read = k.c.read

    def visible(b, T):  # the readable tokens alone
        ok = [s for s in range(T) if 0 <= t[b, s // 16] < len(k.c.k)]
        safe = np.where((t[b] >= 0) & (t[b] < len(k.c.k)), t[b], 0)
        pg, s = safe[np.arange(T) // 16], np.arange(T) % 16
        K = k.c.k[pg, :, s, :] * np.ldexp(1.0, k.c.ks[pg])[..., None]
        V = k.c.v[pg, :, :, s] * np.ldexp(1.0, k.c.vs[pg])[..., None]
        return K[ok], V[ok]

    k.c.read = visible
    k.own = [20, 20, 16, 20]  # causal: the last token of sequence 2 lies in the unreadable page, as a query it sees the others
    out_own = out
    k.check(out_own, "bad pages")
    k.c.read = read
    k.own = [20] * 4
    for kw in (dict(seq_starts=i32([-3, 9, 2])), dict(seq_starts=i32([4, 0, 4])), dict(q_starts=i32([-1, 9, 2, 50, 3])),
               dict(max_kv=16, max_prefix=16)):
        lb.attention_kv8_prefix(k.q, k.c.gpu, k.prefix_table, i32([1 << 30, -5]), k.table, i32([1 << 30, -1, 20, 3]), **k.args(**kw))
    torch.cuda.synchronize()


@pytest.mark.parametrize("D,prefix,count", [(64, 20000, 24), (64, 900, 24), (128, 100, 8), (128, 20000, 24)])
def test_starts_that_overlap(D, prefix, count):
    """More rows named than there are: tiles that the launch has no room for are left out, the others stay inside the
    buffers, and calls afterwards give what they gave before (in pieces; behind groups and in one launch)."""
    k = Call(prefix=[prefix], count=[count], new=[8] * count, own=[300] * count, Hq=4, H=4, D=D, P=64)
    total = 8 * count + 2
    want = k.run(max_q=total)
    print(f"overlapping starts D={D} prefix={prefix}", flush=True)
    k.run(max_q=total, q_starts=i32([0, total] * (count // 2) + [0]))
    again = k.run(max_q=total)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])
    k.check(again, "after overlapping starts", rows=1, some=3)


def test_strides_streams_and_tables_of_whole_sequences():
    """Queries inside a fused projection's output, outputs strided; the two tables as slices of
    rows that hold prefix and own pages; a call on another stream."""
    P, H, D, Hq, B, n = 16, 2, 64, 6, 5, 2
    shared = 4  # whole pages
    own = [2, 16, 17, 40, 33]
    c = Cache([shared * P + max(own)] * B, P, H, D, seed=3)
    c.table[1:, :shared] = c.table[0, :shared]
    fill_lens = [shared * P + x for x in own]
    for b in range(B):  # one sequence at a time: their first pages are the same
        K, V = tokens(fill_lens[b], H, D, 40 + b), tokens(fill_lens[b], H, D, 60 + b)
        K[:shared * P], V[:shared * P] = tokens(shared * P, H, D, 1), tokens(shared * P, H, D, 2)
        lb.kv8_append(c.gpu, i32(c.table[b:b + 1]), i32([fill_lens[b]]), K, V)
    c.fresh()
    table = c.tables()
    qkv = tokens(B * n, Hq + 2 * H, D, 5)
    q, O = qkv[:, :Hq], torch.zeros(B * n, Hq + 1, D, dtype=torch.bfloat16, device="cuda")
    whole = lb.attention_kv8(q, c.gpu, table, i32(fill_lens), return_lse=True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = lb.attention_kv8_prefix(q, c.gpu, table[:1, :shared], i32([shared * P]), table[:, shared:], i32(own), O=O[:, :Hq],
                                       return_lse=True, stream=s)
    s.synchronize()
    assert not O[:, Hq].any()
    for b in range(B):
        K, V = c.read(b, fill_lens[b])
        ref, z, A, eps = M.attention(f64(q)[b * n:(b + 1) * n], K, V, fill_lens[b] - n, D ** -0.5, True, 0)
        tol = M.attention_tolerance(ref, A, eps, len(K))
        for o, l in ((out, lse), whole):
            assert np.all(np.abs(f64(o)[b * n:(b + 1) * n] - ref) <= tol)
            assert np.all(np.abs(f64(l)[b * n:(b + 1) * n] - z) <= M.lse_tolerance(z, eps, len(K)))


def test_in_a_graph():
    """Captured with its workspace reserved; replays see new lengths, other calls of the same stream between."""
    k = Call(prefix=[300], count=[12], new=[1] * 12, own=[30] * 12, Hq=16, H=2, D=128, P=32)
    q, pl, ow = k.q[:12].contiguous(), i32([300]), i32([30] * 12)
    lens = dict(max_kv=30, max_prefix=300)
    call = lambda **kw: lb.attention_kv8_prefix(q, k.c.gpu, k.prefix_table, pl, k.table, ow, return_lse=True, **lens, **kw)
    O, lse = (torch.zeros_like(x) for x in call())
    need = lb.attention_kv8_prefix_workspace(k.c.gpu, k.prefix_table, pl, k.table, ow, 16, 12, **lens)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        lb.reserve_workspace(need)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(O=O, lse=lse)
    for i in range(4):
        pl.fill_(300 - 77 * i)
        ow.copy_(i32([1 + (7 * j + i) % 30 for j in range(12)]))
        q.copy_(tokens(12, 16, 128, 90 + i))
        torch.cuda.synchronize()
        want = call()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(O, want[0]) and torch.equal(lse, want[1]), i
        with torch.cuda.stream(s):
            call()


@pytest.mark.parametrize("name", ["groups, pieces", "few, 256", "parts, 64, again", "pieces, 128", "shares, 128"])
def test_launches_in_a_graph_beside_another_stream(name):
    """Two launches, parts with their join, pieces and shares: replayed on one stream while another call runs on
    a second, shorter lengths from replay to replay."""
    k, other = Call(**LAUNCHES[name]), Call(**LAUNCHES["tiles, 64"], seed=3)
    pl, ow, a = i32(k.prefix), i32(k.own), k.args()
    call = lambda **kw: lb.attention_kv8_prefix(k.q, k.c.gpu, k.prefix_table, pl, k.table, ow, **{**a, **kw})
    O, lse = (torch.zeros_like(x) for x in call())
    want_other = other.run()
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(O=O, lse=lse)
    print(f"graph {name}", flush=True)
    used = int(k.rows[-1])  # rows behind the last sequence are left as they were
    for i in range(4):
        pl.copy_(i32([max(n - 777 * i, i) for n in k.prefix]))
        ow.copy_(i32([max(n - 5 * i, m) for n, m in zip(k.own, k.new)]))
        torch.cuda.synchronize()
        want = call()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        with torch.cuda.stream(s2):
            out = other.run()
        torch.cuda.synchronize()
        assert torch.equal(O[:used], want[0][:used]) and torch.equal(lse[:used], want[1][:used]), i
        assert torch.equal(out[0], want_other[0]) and torch.equal(out[1], want_other[1]), i


def test_argument_errors():
    k = Call(prefix=[20], count=[2], new=[1, 1], own=[5, 5], Hq=4, H=2, D=64, P=16)
    base = dict(Q=k.q, cache=k.c.gpu, prefix_table=k.prefix_table, prefix_lens=i32([20]), page_table=k.table, kv_lens=i32([5, 5]))
    for kw in (dict(Q=k.q.float()), dict(Q=k.q[..., :32]), dict(prefix_table=k.prefix_table.long()), dict(prefix_lens=i32([1, 2])),
               dict(page_table=k.table.t()), dict(kv_lens=i32([5])), dict(seq_starts=i32([0])), dict(q_starts=i32([0, 1])),
               dict(max_kv=10 ** 6), dict(max_prefix=10 ** 6), dict(prefix_table=k.table[:0]),
               dict(prefix_table=k.c.tables()[:3], prefix_lens=i32([1, 1, 1])),  # two sequences for three groups
               dict(O=torch.zeros(4, 4, 64, device="cuda")), dict(lse=torch.zeros(4, 4, device="cuda")[:, :3]),
               dict(kv_lens=i32([5, 5]).cpu()), dict(bad_pages=torch.zeros(1, device="cuda"))):
        args = dict(base)
        args.update(kw)
        with pytest.raises(ValueError):
            lb.attention_kv8_prefix(**args)
    for kw in (dict(softmax_scale=float("inf")), dict(max_q=0), dict(seq_starts=i32([0, 2]), max_seqs=3)):
        with pytest.raises(lb.LowbitError):
            lb.attention_kv8_prefix(**base, **kw)


def read_pages(cache, row, T):
    """Keys and values of the first T tokens of a table row in 64 bits, [T][H][D], and the exponents of their pages, [T][H]."""
    kc, vc, ks, vs = cache
    t = torch.arange(T, device="cuda")
    P = kc.shape[2]
    pg, s = row[t // P].long(), t % P
    ek, ev = ks[pg].double() - 127, vs[pg].double() - 127
    K = kc.double()[pg, :, s] * torch.exp2(ek)[..., None]
    V = vc.double()[pg, :, :, s] * torch.exp2(ev)[..., None]
    return K.cpu().numpy(), V.cpu().numpy(), np.exp2(ek.cpu().numpy()), np.exp2(ev.cpu().numpy())


def test_serving_many_continuations():
    """A prompt's heads normalised, rotated and cached; six answers to it; five steps of all of them: fork (answers replaced
    by copies of others), heads, cache, attention behind the prompt; once between, the cache closed up.  The cache holds
    what each answer's tokens were, attention is that of the cache's contents, and no page is lost or held twice."""
    P, H, D, Hq, n, L = 16, 2, 64, 8, 6, 3 * 16 + 9
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.rand(D, device="cuda", generator=g) + 0.5
    freqs = torch.tensor([1e4 ** (-i / 32) for i in range(32)], dtype=torch.float64, device="cuda")
    n_pages = 64
    cache = lb.empty_kv8(n_pages, P, H, D)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")

    def heads(rows, positions):
        """A fused projection's output, its queries and keys normalised and rotated."""
        qkv = torch.randn(rows, Hq + 2 * H, D, device="cuda", generator=g).bfloat16()
        q, k = lb.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + H], positions, freqs, w, w)
        return q, k, qkv[:, Hq + H:]

    def holds(row, tokens, what):
        """The cache holds these tokens: each rounded to e4m3 (2^-4 of it, the last time 2^-10 of its page's unit, and
        so each time the exponent rose, the unit being half or less then: 2^-9 in all)."""
        K, V, ek, ev = read_pages(cache, row, tokens[0].shape[0])
        for x, y, e in ((K, tokens[0], ek), (V, tokens[1], ev)):
            y = f64(y)
            assert np.all(np.abs(x - y) <= 2.0 ** -4 * 1.01 * np.abs(y) + 2.0 ** -9 * e[..., None]), what
        return K, V

    # the prompt: pages for it, its tokens
    none = torch.zeros(0, 4, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    pt, pl, refs, failed = lb.kv8_fork(cache, *none, refs, i32([-1]), grow=L, width=4)
    _, k, v = heads(L, torch.arange(L, dtype=torch.int32, device="cuda"))
    lb.kv8_append(cache, pt, pl, k, v)
    prompt = k, v
    # the answers hold no pages yet; the prompt's stay where they are
    table, lens = torch.full((n, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    parents, mirror = list(range(n)), [(k[:0], v[:0])] * n
    for step in range(5):
        table, lens, refs, failed = lb.kv8_fork(cache, table, lens, refs, i32(parents), grow=7, width=3)
        assert failed.item() == 0 and lens.tolist() == [7 * (step + 1)] * n
        q, k, v = heads(7 * n, (L + 7 * step + torch.arange(7, device="cuda")).repeat(n).to(torch.int32))
        lb.kv8_append(cache, table, lens, k, v)
        mirror = [tuple(torch.cat((x, y[7 * b:7 * b + 7])) for x, y in zip(mirror[p], (k, v))) for b, p in enumerate(parents)]
        if step == 3:
            # the rows of the answers and the prompt's in one table
            both = torch.full((n + 1, 4), -1, dtype=torch.int32, device="cuda")
            both[:n, :3], both[n] = table, pt[0]
            both, refs, remap, live = lb.kv8_compact(cache, both, torch.cat((lens, pl)), refs)
            table, pt = both[:n, :3].contiguous(), both[n:].contiguous()
            assert live.item() == len(set(both[both >= 0].tolist())) and both.max().item() < live.item()
        O, lse = lb.attention_kv8_prefix(q, cache, pt, pl, table, lens, return_lse=True)
        Kp, Vp = holds(pt[0], prompt, f"step {step}: prompt")
        for b in range(n):
            Ko, Vo = holds(table[b], mirror[b], f"step {step}: answer {b}")
            ref, z, A, eps = R.attention_prefix(f64(q)[7 * b:7 * b + 7], Kp, Vp, Ko, Vo, 7 * step, D ** -0.5, True)
            T = len(Kp) + len(Ko)
            assert np.all(np.abs(f64(O)[7 * b:7 * b + 7] - ref) <= M.attention_tolerance(ref, A, eps, T)), step
            assert np.all(np.abs(f64(lse)[7 * b:7 * b + 7] - z) <= M.lse_tolerance(z, eps, T)), step
        held = [0] * n_pages
        for p in pt[0].tolist() + [p for row in table.tolist() for p in row[:R.held(7 * (step + 1), P)]]:
            held[p] += 1
        assert refs.tolist() == held, f"step {step}: counts"
        parents = [0, 0, 2, 2, 5, 5] if step % 2 else np.random.default_rng(step).integers(0, n, n).tolist()
