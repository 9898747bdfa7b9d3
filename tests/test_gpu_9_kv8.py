"""The 8-bit paged cache on the GPU: writes bit for bit, attention within the
bound of its roundings, and a layer's products, cache and attention run
together, all against the plain 64-bit forms."""
import numpy as np
import pytest
import torch

import mx_ref as R
from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def codes64(t):
    """e4m3 codes of a cache tensor as numbers."""
    return R.E4M3[t.view(torch.uint8).cpu().numpy()]


class Cache:
    """A cache on the GPU with every byte set (codes at random, NaN codes among
    them), its mirror in 64 bits, and a page table of shuffled pages."""

    def __init__(self, lens, P, H, D, seed=0, spare=2):
        g = np.random.default_rng(seed)
        self.P, self.H, self.D = P, H, D
        self.width = max(1, -(-max(lens) // P))
        n = len(lens) * self.width + spare
        kc, vc, ks, vs = lb.empty_kv8(n, P, H, D)
        for t in (kc, vc):
            t.view(torch.uint8).copy_(torch.from_numpy(g.integers(0, 256, t.shape, dtype=np.uint8)))
        for t in (ks, vs):
            t.copy_(torch.from_numpy(g.integers(0, 256, t.shape, dtype=np.uint8)))
        self.gpu = (kc, vc, ks, vs)
        self.table = g.permutation(n)[:len(lens) * self.width].reshape(len(lens), self.width).astype(np.int32)
        self.fresh()

    def fresh(self):
        kc, vc, ks, vs = self.gpu
        self.k, self.v = codes64(kc), codes64(vc)
        self.ks, self.vs = ks.cpu().numpy().astype(int) - 127, vs.cpu().numpy().astype(int) - 127

    def tables(self):
        return torch.from_numpy(self.table).cuda()

    def append(self, b, first, K, V):
        """Mirror of the write of one sequence's new tokens (float64 [n][H][D])."""
        t = first
        while t < first + len(K):
            lo = t % self.P
            n = min(self.P - lo, first + len(K) - t)
            pg = self.table[b, t // self.P]
            R.append(self.k, self.ks, pg, K[t - first:t - first + n], lo, False)
            R.append(self.v, self.vs, pg, V[t - first:t - first + n], lo, True)
            t += n

    def check(self, what):
        kc, vc, ks, vs = self.gpu
        assert np.array_equal(ks.cpu().numpy().astype(int) - 127, self.ks), f"{what}: key exponents"
        assert np.array_equal(vs.cpu().numpy().astype(int) - 127, self.vs), f"{what}: value exponents"
        assert np.array_equal(codes64(kc), self.k, equal_nan=True), f"{what}: keys"
        assert np.array_equal(codes64(vc), self.v, equal_nan=True), f"{what}: values"

    def read(self, b, T):
        """Keys and values of the first T tokens, [T][H][D]."""
        pg = self.table[b][np.arange(T) // self.P]
        s = np.arange(T) % self.P
        K = self.k[pg, :, s, :] * np.ldexp(1.0, self.ks[pg])[..., None]
        V = self.v[pg, :, :, s] * np.ldexp(1.0, self.vs[pg])[..., None]
        return K, V


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def tokens(T, H, D, seed, dtype=torch.bfloat16):
    g = np.random.default_rng(seed)
    x = g.standard_normal((T, H, D)) * np.exp2(g.integers(-6, 7, (T, 1, 1)))
    return torch.from_numpy(x.astype(np.float32)).cuda().to(dtype)


def fill(c, lens, seed, dtype=torch.bfloat16):
    """Write whole sequences of the given lengths."""
    T = int(sum(lens))
    K, V = tokens(T, c.H, c.D, seed, dtype), tokens(T, c.H, c.D, seed + 1, dtype)
    starts = np.concatenate([[0], np.cumsum(lens)])
    lb.kv8_append(c.gpu, c.tables(), i32(lens), K, V, q_starts=i32(starts), max_q=max(lens))
    for b, n in enumerate(lens):
        c.append(b, 0, f64(K)[starts[b]:starts[b + 1]], f64(V)[starts[b]:starts[b + 1]])


# ------------------------------------------------------------------ writes


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("D,H,dtype", [(64, 3, torch.float32), (128, 2, torch.bfloat16), (256, 1, torch.bfloat16)])
def test_append_prompt_then_tokens(P, D, H, dtype):
    """Prompts of odd lengths, then tokens one by one: pages that fill up, exponents that rise."""
    lens = [1, P - 1, P, P + 1, 3 * P + 5]
    print(f"append P={P} D={D} H={H} {dtype}", flush=True)
    c = Cache([n + 4 for n in lens], P, H, D, seed=P + D)
    fill(c, lens, 11, dtype)
    c.check("prompt")
    for step in range(3):
        B = len(lens)
        K, V = tokens(B, H, D, 50 + step, dtype) * (4.0 ** step), tokens(B, H, D, 70 + step, dtype)
        now = [n + step + 1 for n in lens]
        lb.kv8_append(c.gpu, c.tables(), i32(now), K, V)
        for b in range(B):
            c.append(b, now[b] - 1, f64(K)[b:b + 1], f64(V)[b:b + 1])
        c.check(f"token {step}")
        lb.kv8_append(c.gpu, c.tables(), i32(now), K, V)
        c.check(f"token {step} again")


@pytest.mark.parametrize("P,D", [(16, 128), (64, 128), (128, 128), (32, 256), (128, 256)])
def test_append_fp32_wide_heads(P, D):
    test_append_prompt_then_tokens(P, D, 2, torch.float32)


def test_append_strided_empty_and_special():
    """Keys and values inside a fused projection's output; a sequence without new
    tokens, one of length 0; zeros, subnormals, infinities, NaN."""
    P, H, D = 16, 2, 64
    print("append strided", flush=True)
    lens, new = [20, 9, 0, 33], [7, 0, 0, 33]
    c = Cache(lens, P, H, D, seed=4)
    starts = np.concatenate([[0], np.cumsum(new)])
    T = int(starts[-1])
    qkv = torch.full((T + 2, 5, H, D), float("nan"), device="cuda")
    qkv[:T, 1], qkv[:T, 3] = tokens(T, H, D, 1, torch.float32), tokens(T, H, D, 2, torch.float32)
    qkv[7:23, 1] = 0.0
    qkv[23:39, 1] = 2.0 ** -140
    qkv[10, 3, 1, 3], qkv[11, 3, 1, 4], qkv[12, 3, 0, 5] = float("inf"), float("-inf"), float("nan")
    qkv[39, 1, 0] = float("nan")  # the last page's only key: nothing finite
    K, V = qkv[:T, 1], qkv[:T, 3]
    # earlier tokens of the first sequence
    K0, V0 = tokens(13, H, D, 8), tokens(13, H, D, 9)
    lb.kv8_append(c.gpu, c.tables()[:1], i32([13]), K0, V0)
    c.append(0, 0, f64(K0), f64(V0))
    lb.kv8_append(c.gpu, c.tables(), i32(lens), K, V, q_starts=i32(starts), max_q=33)
    for b in (0, 3):
        c.append(b, lens[b] - new[b], f64(K)[starts[b]:starts[b + 1]], f64(V)[starts[b]:starts[b + 1]])
    c.check("special")


def test_append_bad_pages_are_counted_and_not_written():
    P, H, D = 16, 1, 64
    print("append bad pages", flush=True)
    c = Cache([40, 16], P, H, D, seed=6)
    n = c.gpu[0].shape[0]
    good = c.table.copy()
    c.table[0, 1], c.table[1, 0] = n, -5
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    K, V = tokens(56, H, D, 1), tokens(56, H, D, 2)
    lb.kv8_append(c.gpu, c.tables(), i32([40, 16]), K, V, q_starts=i32([0, 40, 56]), bad_pages=bad)
    k, v = f64(K), f64(V)
    R.append(c.k, c.ks, good[0, 0], k[:16], 0, False)
    R.append(c.v, c.vs, good[0, 0], v[:16], 0, True)
    R.append(c.k, c.ks, good[0, 2], k[32:40], 0, False)
    R.append(c.v, c.vs, good[0, 2], v[32:40], 0, True)
    c.check("bad pages")
    assert int(bad) == 2


def test_append_clamps_lengths_and_rows():
    """Lengths beyond max_kv and rows beyond the tensors (a stale array on the device) stay inside the buffers."""
    P, H, D = 16, 1, 64
    print("append clamps", flush=True)
    c = Cache([32], P, H, D, seed=7)
    K, V = tokens(4, H, D, 1), tokens(4, H, D, 2)
    lb.kv8_append(c.gpu, c.tables(), i32([1000]), K, V, q_starts=i32([0, 4]), max_kv=30)
    c.append(0, 26, f64(K), f64(V))
    c.check("length")
    lb.kv8_append(c.gpu, c.tables(), i32([12]), K, V, q_starts=i32([2, 900]), max_q=4)
    c.append(0, 10, f64(K)[2:], f64(V)[2:])
    c.check("rows")
    lb.kv8_append(c.gpu, c.tables(), i32([-3]), K, V, q_starts=i32([3, 1]))
    c.check("nothing")


# --------------------------------------------------------------- attention


def attend(c, lens, new, G, seed, causal=True, window=0, scale=None, **more):
    """Run and check one call; returns the outputs."""
    T = int(sum(new))
    starts = np.concatenate([[0], np.cumsum(new)])
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(T, c.H * G, c.D, device="cuda", generator=g).bfloat16()
    O, lse = lb.attention_kv8(q, c.gpu, c.tables(), i32(lens), q_starts=i32(starts), max_q=max(new),
                              softmax_scale=scale, causal=causal, window=window, return_lse=True, **more)
    compare(c, q, O, lse, lens, starts, scale, causal, window)
    return q, O, lse


def compare(c, q, O, lse, lens, starts, scale=None, causal=True, window=0):
    scale = float(np.float32(c.D ** -0.5 if scale is None else scale))
    for b, T in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        if lo == hi:
            continue
        K, V = c.read(b, T)
        o, l, A, eps = R.attention(f64(q[lo:hi]), K, V, T - (hi - lo), scale, causal, window)
        got, gl = f64(O[lo:hi]), f64(lse[lo:hi])
        bad = ~(np.abs(got - o) <= R.attention_tolerance(o, A, eps, max(T, 1)))
        assert not bad.any(), (f"sequence {b}: {int(bad.sum())} of {bad.size} off, first at {np.argwhere(bad)[0]}: "
                               f"{got[bad][0]} for {o[bad][0]}")
        inf = np.isneginf(l)
        assert np.array_equal(np.isneginf(gl), inf)
        assert np.all(np.abs(gl - l)[~inf] <= R.lse_tolerance(l, eps, max(T, 1))[~inf]), f"sequence {b}: lse"
        assert np.all(got[inf] == 0)


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("D,H,G", [(64, 2, 3), (128, 3, 1), (128, 1, 8), (256, 1, 6)])
def test_decode(P, D, H, G):
    """One token of each sequence, lengths around the ends of pages and steps."""
    lens = [1, 15, 16, 17, 63, 64, 65, 127, 130, 200]
    print(f"decode P={P} D={D} H={H} G={G}", flush=True)
    c = Cache(lens, P, H, D, seed=P + D + G)
    fill(c, lens, 3)
    attend(c, lens, [1] * len(lens), G, 5)


@pytest.mark.parametrize("P,D,H,G", [(16, 64, 1, 2), (64, 128, 2, 5), (128, 256, 1, 3), (32, 128, 1, 1)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 23), (True, 100), (False, 0), (False, 9)])
def test_prompts(P, D, H, G, causal, window):
    """Several new tokens a sequence, ragged, behind prefixes of any length."""
    lens, new = [70, 33, 150, 5, 64], [70, 1, 37, 5, 64]
    print(f"prompt P={P} D={D} H={H} G={G} causal={causal} window={window}", flush=True)
    c = Cache(lens, P, H, D, seed=P + D)
    fill(c, lens, 3)
    attend(c, lens, new, G, 6, causal=causal, window=window)


@pytest.mark.parametrize("D,G,n", [(64, 4, 300), (128, 1, 260), (128, 5, 129), (256, 2, 131)])
@pytest.mark.parametrize("causal", [True, False])
def test_long_prompts(D, G, n, causal):
    lens, new = [n + 150, n - 60], [n, n - 60]
    print(f"long prompt D={D} G={G} n={n} causal={causal}", flush=True)
    c = Cache(lens, 64, 1, D, seed=D)
    fill(c, lens, 4)
    attend(c, lens, new, G, 8, causal=causal)


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (256, 128)])
def test_long_context_splits(D, P):
    """A context long enough to be split over many workgroups; the same bits twice."""
    lens = [9001, 512, 3]
    print(f"splits D={D} P={P}", flush=True)
    c = Cache(lens, P, 1, D, seed=2)
    fill(c, lens, 9)
    q, O, lse = attend(c, lens, [1, 1, 1], 3, 4)
    for _ in range(3):
        O2, l2 = lb.attention_kv8(q, c.gpu, c.tables(), i32(lens), return_lse=True)
        assert torch.equal(O, O2) and torch.equal(lse, l2)
    # a bound larger than any length changes the split, not the result's bound
    O3, l3 = lb.attention_kv8(q, c.gpu, c.tables(), i32(lens), max_kv=9001, return_lse=True)
    compare(c, q, O3, l3, lens, [0, 1, 2, 3])
    attend(c, lens, [5, 5, 2], 3, 4)
    attend(c, lens, [1, 1, 1], 3, 4, window=2000)


@pytest.mark.parametrize("D,H,G,P", [(64, 2, 4, 16), (128, 2, 5, 64), (256, 1, 4, 128)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 900), (False, 0)])
def test_prompt_parts(D, H, G, P, causal, window):
    """Chunks of rows against contexts long enough to be cut into parts."""
    lens, new = [5003, 1300, 40, 0], [33, 40, 40, 3]
    print(f"parts D={D} G={G} P={P} causal={causal} window={window}", flush=True)
    c = Cache(lens, P, H, D, seed=12)
    fill(c, lens, 13)
    starts = np.concatenate([[0], np.cumsum(new)])
    size = lb.attention_kv8_workspace(c.gpu, c.tables(), i32(lens), H * G, int(starts[-1]), q_starts=i32(starts),
                                      max_q=max(new))
    assert size > 4 * 128 * (D + 2) * 4  # holds more than one part's rows
    q, O, lse = attend(c, lens, new, G, 14, causal=causal, window=window)
    for _ in range(2):
        O2, l2 = lb.attention_kv8(q, c.gpu, c.tables(), i32(lens), q_starts=i32(starts), max_q=max(new),
                                  causal=causal, window=window, return_lse=True)
        assert torch.equal(O, O2) and torch.equal(lse, l2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [300, 3000])
def test_unreadable_pages_and_nan_in_chunks(T, D):
    """Pages that cannot be read in the middle of many rows' context, and a NaN
    value that half of the rows see."""
    P, H, G, n = 32, 2, 2, 70
    print(f"unreadable pages T={T} D={D}", flush=True)
    c = Cache([T], P, H, D, seed=18)
    fill(c, [T], 16)
    keep = c.table.copy()
    gone = np.isin(np.arange(T) // P, (2, 5))
    c.table[0, 2], c.table[0, 5] = c.gpu[0].shape[0] + 7, -1
    at = T - n // 2
    c.gpu[1].view(torch.uint8)[int(c.table[0, at // P]), 1, 5, at % P] = 0x7F
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn(n, H * G, D, device="cuda").bfloat16()
    O = f64(lb.attention_kv8(q, c.gpu, c.tables(), i32([T]), bad_pages=bad))
    assert int(bad) >= 2
    c.table = keep
    K, V = c.read(0, T)
    for i in range(n):
        see = ~gone & (np.arange(T) <= T - n + i)
        o, _, A, eps = R.attention(f64(q[i:i + 1]), K[see], V[see], int(see.sum()) - 1, D ** -0.5, True, 0)
        want = np.zeros((H * G, D), bool)
        want[G:, 5] = T - n + i >= at
        nan = np.isnan(O[i])
        assert np.array_equal(nan, want), i
        assert np.all((np.abs(O[i] - o[0]) <= R.attention_tolerance(o, A, eps, T)[0]) | want), i


@pytest.mark.parametrize("D,P", [(64, 16), (128, 32), (256, 64)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 130), (False, 0)])
@pytest.mark.parametrize("G", [1, 3, 6])
def test_up_to_32_rows_behind_a_wide_table(D, P, causal, window, G):
    """5, 15 and 30 rows a head in calls whose bound on the length is large; table
    entries behind a sequence's pages are anything.  A NaN value in the last
    tokens reaches the rows that see it."""
    lens, new, H = [700, 131, 9, 64], [5, 4, 5, 1], 2
    print(f"wide table D={D} P={P} G={G} causal={causal} window={window}", flush=True)
    c = Cache(lens, P, H, D, seed=52)
    fill(c, lens, 53)
    wide = torch.full((len(lens), 40000 // P), -77, dtype=torch.int32, device="cuda")
    wide[:, :c.width] = c.tables()
    starts = np.concatenate([[0], np.cumsum(new)])
    g = torch.Generator(device="cuda").manual_seed(54)
    q = torch.randn(int(starts[-1]), H * G, D, device="cuda", generator=g).bfloat16()

    def run():
        return lb.attention_kv8(q, c.gpu, wide, i32(lens), q_starts=i32(starts), max_q=5, causal=causal,
                                window=window, return_lse=True)

    O, lse = run()
    compare(c, q, O, lse, lens, starts, causal=causal, window=window)
    t = lens[0] - 3
    c.gpu[1].view(torch.uint8)[int(c.table[0, t // P]), 1, 7, t % P] = 0xFF
    O2, lse2 = run()
    want = torch.zeros_like(O, dtype=torch.bool)
    for i in range(5):
        want[i, G:, 7] = not causal or lens[0] - 5 + i >= t
    assert torch.equal(torch.isnan(O2), want)
    assert torch.equal(torch.where(want, O, O2), O) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_tile_in_very_many_shares(D):
    """One key head and a context that more than 64 workgroups share: joined in groups of many."""
    T, P = 70000, 64
    print(f"one tile, many shares D={D}", flush=True)
    c = Cache([T], P, 1, D, seed=22)
    fill(c, [T], 23)
    attend(c, [T], [1], 2, 24)
    attend(c, [T], [3], 1, 25, window=33000)


@pytest.mark.parametrize("D,G,big", [(64, 2, 3), (128, 1, 130)])
def test_many_sequences(D, G, big):
    """More sequences than threads that number them, empty ones among them; in
    the second case some are prompts."""
    g = np.random.default_rng(31)
    B, P, H = 700, 16, 1
    print(f"many sequences D={D} big={big}", flush=True)
    new = g.integers(0, 3, B)
    new[[5, 300, B - 1]] = big
    lens = np.where(g.random(B) < 0.2, 0, new + g.integers(0, 40, B))
    c = Cache(list(lens), P, H, D, seed=32)
    fill(c, list(map(int, lens)), 33)
    attend(c, list(map(int, lens)), list(map(int, new)), G, 34)


def test_rows_that_see_nothing():
    """Length 0, more new tokens than the sequence holds, and rows behind the last sequence."""
    print("empty rows", flush=True)
    c = Cache([40, 1, 3], 16, 2, 64, seed=3)
    fill(c, [40, 1, 3], 4)
    T = 12
    q = torch.randn(T, 4, 64, device="cuda").bfloat16()
    O = torch.full((T, 4, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((T, 4), 7.0, device="cuda")
    starts = [0, 2, 2, 7]
    lb.attention_kv8(q, c.gpu, c.tables(), i32([0, 1, 3]), q_starts=i32(starts), max_q=5, O=O, lse=lse)
    assert (O[:2] == 0).all() and torch.isneginf(lse[:2]).all()
    compare(c, q, O, lse, [0, 1, 3], starts)  # rows 2, 3 of the last sequence lie before its first token
    assert (O[2:4] == 0).all() and (O[7:] == 7).all() and (lse[7:] == 7).all()


@pytest.mark.parametrize("new", [1, 9, 140])
@pytest.mark.parametrize("P", [16, 128])
def test_nan_reaches_only_rows_that_see_it(new, P):
    """NaN keys and values in the middle: rows before them (causal) and behind
    their window stay exact; rows that see them are NaN."""
    D, H, G, T = 128, 2, 2, 200
    print(f"NaN tokens new={new} P={P}", flush=True)
    c = Cache([T], P, H, D, seed=5)
    fill(c, [T], 6)
    kc, vc = c.gpu[0].view(torch.uint8), c.gpu[1].view(torch.uint8)
    for t, h, what in ((T - new // 2 - 1, 0, "v"), (T - 1, 1, "k"), (20, 1, "v")):
        pg, s = int(c.table[0, t // P]), t % P
        if what == "v":
            vc[pg, h, 5, s] = 0xFF
        else:
            kc[pg, h, s, 9] = 0x7F
    window = 150
    starts = [0, new]
    q = torch.randn(new, H * G, D, device="cuda").bfloat16()
    O, lse = lb.attention_kv8(q, c.gpu, c.tables(), i32([T]), window=window, return_lse=True)
    got = f64(O)
    K, V = c.read(0, T)  # the mirror holds no NaN there
    o, l, A, eps = R.attention(f64(q), K, V, T - new, D ** -0.5, True, window)
    tol = R.attention_tolerance(o, A, eps, T)
    for i in range(new):
        p = T - new + i
        for hq in range(H * G):
            want = np.zeros(D, bool)
            if hq // G == 0 and p >= T - new // 2 - 1 and p - window < T - new // 2 - 1:
                want[5] = True
            if hq // G == 1 and p - window < 20 <= p:
                want[5] = True
            if hq // G == 1 and p >= T - 1:
                want[:] = True
            nan = np.isnan(got[i, hq])
            assert np.array_equal(nan, want), (i, hq, np.nonzero(nan != want)[0][:4])
            ok = np.abs(got[i, hq] - o[i, hq]) <= tol[i, hq]
            assert ok[~want].all(), (i, hq)


def test_unreadable_pages_are_not_seen():
    P, H, D = 16, 2, 64
    print("unreadable pages", flush=True)
    c = Cache([100, 50], P, H, D, seed=8)
    fill(c, [100, 50], 6)
    n = c.gpu[0].shape[0]
    keep = c.table.copy()
    c.table[0, 2], c.table[1, 3] = n + 7, -1
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, D, device="cuda").bfloat16()
    O = lb.attention_kv8(q, c.gpu, c.tables(), i32([100, 50]), bad_pages=bad)
    assert int(bad) >= 2
    c.table = keep
    for b, T in enumerate((100, 50)):
        K, V = c.read(b, T)
        gone = np.arange(T) // P == (2 if b == 0 else 3)
        o, _, A, eps = R.attention(f64(q[b:b + 1]), K[~gone], V[~gone], T, D ** -0.5, True, 0)
        assert np.all(np.abs(f64(O[b:b + 1]) - o) <= R.attention_tolerance(o, A, eps, T))


def test_strides_scale_and_shared_pages():
    """Queries inside a wider tensor, a scale of its own, sequences that share full pages, outputs strided."""
    P, H, D, G = 16, 2, 128, 2
    print("strides", flush=True)
    c = Cache([48, 48, 48], P, H, D, seed=9)
    fill(c, [48, 48, 48], 6)
    c.table[1, :2], c.table[2, 0] = c.table[0, :2], c.table[0, 0]
    wide = torch.randn(3, 3, H * G, D, device="cuda").bfloat16()
    out = torch.full((3, 2, H * G, D), 3.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(3, H * G, device="cuda")
    for scale in (0.03, -0.1, 0.0):
        lb.attention_kv8(wide[:, 1], c.gpu, c.tables(), i32([41, 40, 33]), softmax_scale=scale, O=out[:, 1], lse=lse)
        compare(c, wide[:, 1], out[:, 1], lse, [41, 40, 33], [0, 1, 2, 3], scale)
    assert (out[:, 0] == 3).all()


def test_large_scores_and_spread_exponents():
    """Scores of some hundreds (one token takes all) and pages whose exponents lie far apart."""
    P, H, D = 16, 1, 64
    print("spread", flush=True)
    T = 160
    c = Cache([T], P, H, D, seed=1)
    K, V = tokens(T, H, D, 2), tokens(T, H, D, 3)
    K[16:32] *= 2.0 ** -30
    V[48:64] *= 2.0 ** 40
    V[64:80] *= 2.0 ** -60
    K[100:116] *= 8.0
    lb.kv8_append(c.gpu, c.tables(), i32([T]), K, V)
    c.append(0, 0, f64(K), f64(V))
    for new in (1, 100):
        attend(c, [T], [new], 4, 12, scale=1.0)
        attend(c, [T], [new], 4, 13, window=30)


def test_offsets_beyond_32_bits():
    """Pages more than 4 GiB into the codes."""
    P, H, D = 128, 8, 256
    print("large cache", flush=True)
    n = (5 << 30) // (P * H * D)
    cache = lb.empty_kv8(n, P, H, D)
    table = i32([[n - 1, 0, n - 2]])
    T = 300
    K, V = tokens(T, H, D, 1), tokens(T, H, D, 2)
    lb.kv8_append(cache, table, i32([T]), K, V)
    small = Cache([T], P, H, D, seed=0)
    small.append(0, 0, f64(K), f64(V))
    q = torch.randn(2, 2 * H, D, device="cuda").bfloat16()
    O, lse = lb.attention_kv8(q, cache, table, i32([T]), return_lse=True)
    compare(small, q, O, lse, [T], [0, 2])
    ks, vs = cache[2].cpu().numpy().astype(int) - 127, cache[3].cpu().numpy().astype(int) - 127
    for j, pg in enumerate((n - 1, 0, n - 2)):
        m = small.table[0, j]
        w = min(P, T - j * P)
        assert np.array_equal(codes64(cache[0][pg])[:, :w], small.k[m][:, :w])
        assert np.array_equal(codes64(cache[1][pg])[:, :, :w], small.v[m][:, :, :w])
        assert np.array_equal(ks[pg], small.ks[m]) and np.array_equal(vs[pg], small.vs[m])


def test_decode_step_in_a_graph():
    """Append and attention captured once (one split and many), replayed as the
    sequences grow, with eager calls of other shapes on the stream between."""
    P, H, D, G, B = 16, 2, 128, 3, 2
    print("graph", flush=True)
    lens = [1500, 37]
    c = Cache([1520, 60], P, H, D, seed=3)
    fill(c, lens, 5)
    table, dl = c.tables(), i32(lens)
    K, V = tokens(B, H, D, 1), tokens(B, H, D, 2)
    q = torch.zeros(B, H * G, D, device="cuda", dtype=torch.bfloat16)
    O, lse = torch.empty_like(q), torch.empty(B, H * G, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lb.reserve_workspace(lb.attention_kv8_workspace(c.gpu, table, dl, H * G, B), s)

    def step():
        lb.kv8_append(c.gpu, table, dl, K, V)
        lb.attention_kv8(q, c.gpu, table, dl, O=O, lse=lse)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in range(4):
        lens = [n + 1 for n in lens]
        dl.copy_(i32(lens))
        K.copy_(tokens(B, H, D, 100 + i))
        V.copy_(tokens(B, H, D, 200 + i))
        q.copy_(torch.randn(B, H * G, D, device="cuda"))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
            q2 = torch.randn(1, H, D, device="cuda").bfloat16()
            lb.attention_kv8(q2, c.gpu, table[:1], dl[:1], max_kv=700)
        torch.cuda.synchronize()
        for b in range(B):
            c.append(b, lens[b] - 1, f64(K)[b:b + 1], f64(V)[b:b + 1])
        c.check(f"replay {i}")
        compare(c, q, O, lse, lens, [0, 1, 2])


def test_chunk_in_parts_in_a_graph():
    """A chunk of rows against a long context, captured and replayed as the
    context grows, with eager calls of the same kind between."""
    P, H, D, G, n = 64, 1, 128, 4, 40
    print("graph of parts", flush=True)
    T = 4000
    c = Cache([T + 64], P, H, D, seed=43)
    fill(c, [T], 44)
    table, dl = c.tables(), i32([T])
    q = torch.zeros(n, H * G, D, device="cuda", dtype=torch.bfloat16)
    O, lse = torch.empty_like(q), torch.empty(n, H * G, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lb.reserve_workspace(lb.attention_kv8_workspace(c.gpu, table, dl, H * G, n), s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        lb.attention_kv8(q, c.gpu, table, dl, O=O, lse=lse)
    for i in range(3):
        K, V = tokens(1, H, D, 100 + i), tokens(1, H, D, 200 + i)
        T += 1
        dl.copy_(i32([T]))
        lb.kv8_append(c.gpu, table, dl, K, V)
        c.append(0, T - 1, f64(K), f64(V))
        q.copy_(torch.randn(n, H * G, D, device="cuda"))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
            e = lb.attention_kv8(q, c.gpu, table, dl)
        torch.cuda.synchronize()
        assert torch.equal(e, O)
        compare(c, q, O, lse, [T], [0, n])


def test_two_streams_at_once():
    """The same call on two streams: their workspaces are their own."""
    P, H, D = 64, 2, 128
    print("two streams", flush=True)
    lens = [6000]
    c = Cache(lens, P, H, D, seed=3)
    fill(c, lens, 5)
    table, dl = c.tables(), i32(lens)
    qs = [torch.randn(1, 8, D, device="cuda").bfloat16() for _ in range(2)]
    want = [lb.attention_kv8(q, c.gpu, table, dl) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, q in zip(streams, qs):
            with torch.cuda.stream(s):
                got.append(lb.attention_kv8(q, c.gpu, table, dl))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------ run together


@pytest.mark.parametrize("new,x4", [(1, False), (5, False), (70, True)])
def test_layer(new, x4):
    """x -> MXFP4 q/k/v product -> cache -> attention -> MXFP4 o product, as a
    model's layer calls them, each step checked on the GPU's own input to it."""
    hid, H, G, D, P = 512, 2, 2, 64, 32
    Hq = H * G
    print(f"layer new={new} x4={x4}", flush=True)
    rng = np.random.default_rng(new)

    def weights(n, k):
        w = torch.from_numpy((rng.standard_normal((n, k)) * 0.05).astype(np.float32)).cuda()
        c, s, v = lb.quantize_mxfp4(w, values=True)
        return c, s, f64(v)

    n_qkv = (Hq + 2 * H) * D
    wq, wo = weights(n_qkv, hid), weights(hid, Hq * D)
    lens = [new + 90, new + 3]
    c = Cache(lens, P, H, D, seed=new)
    fill(c, [90, 3], 17)
    T = 2 * new

    def product(x, w, n):
        k = x.shape[1]
        if not x4:
            return lb.gemm_mxfp4(T, n, k, w[0], w[1], x, y_dtype=lb.BF16), f64(x)
        xc, xs, xv = lb.quantize_mxfp4(x, values=True)
        return lb.gemm_mxfp4(T, n, k, w[0], w[1], xc, x_scales=xs, y_dtype=lb.BF16), f64(xv)

    x = torch.randn(T, hid, device="cuda").bfloat16()
    qkv, xv = product(x, wq, n_qkv)
    ref, mag = xv @ wq[2].T, np.abs(xv) @ np.abs(wq[2]).T
    assert np.all(np.abs(f64(qkv) - ref) <= R.product_tolerance(mag, ref, hid, True))
    heads = qkv.view(T, Hq + 2 * H, D)
    q, K, V = heads[:, :Hq], heads[:, Hq:Hq + H], heads[:, Hq + H:]
    table, dl = c.tables(), i32(lens)
    lb.kv8_append(c.gpu, table, dl, K, V)
    for b in range(2):
        c.append(b, lens[b] - new, f64(K)[b * new:(b + 1) * new], f64(V)[b * new:(b + 1) * new])
    c.check("layer")
    o, lse = lb.attention_kv8(q, c.gpu, table, dl, return_lse=True)
    compare(c, q, o, lse, lens, [0, new, 2 * new])
    y, ov = product(o.view(T, Hq * D), wo, hid)
    ref, mag = ov @ wo[2].T, np.abs(ov) @ np.abs(wo[2]).T
    assert np.all(np.abs(f64(y) - ref) <= R.product_tolerance(mag, ref, Hq * D, True))
