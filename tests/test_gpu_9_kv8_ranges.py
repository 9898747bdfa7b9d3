"""The 8-bit cache at the ends of its number ranges: exponents that rise by
any amount, the largest finite values, scales of zero
and next to it, and how finely attention with few rows weighs."""
import numpy as np
import pytest
import torch

import mx_ref as R
from ultra_bit_dit_amd import lowbit as lb
from test_gpu_9_kv8 import Cache, f64, fill, i32, tokens

pytestmark = pytest.mark.gpu


def check_bits(c, what):
    """As Cache.check, and the signs of zeros."""
    c.check(what)
    for t, m in ((c.gpu[0], c.k), (c.gpu[1], c.v)):
        by = t.view(torch.uint8).cpu().numpy()
        assert np.array_equal((by >> 7 == 1) & ~np.isnan(m), np.signbit(m) & ~np.isnan(m)), f"{what}: signs"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("P,D", [(16, 64), (64, 128), (128, 256)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_append_exponent_rises_by_any_amount(P, D, which, dtype):
    """Earlier tokens all zero, or near 2^-120 (exponent -127), then tokens whose
    maximum raises the page's exponent by 1 .. 246; the other side rises by one."""
    H, n = 2, 3
    lo = P // 2 + 3
    tops = [(0.0, t) for t in (448.0, 500.0, 896.0, 897.0, 2.0 ** 60, 2.0 ** 99)]
    tops += [(2.0 ** -120, 448 * 2.0 ** (r - 127)) for r in
             (0, 1, 9, 17, 18, 100, 125, 126, 127, 128, 129, 140, 191, 192, 246)]
    B = len(tops)
    print(f"append far rise {which} P={P} D={D} {dtype}", flush=True)
    c = Cache([lo + n] * B, P, H, D, seed=P)
    g = np.random.default_rng(3)

    def side(T, size, far):
        """[B T][H][D] with the given largest magnitude of each sequence's heads"""
        x = g.uniform(0.25, 1, (B, T, H, D)) * np.where(g.random((B, T, H, D)) < .5, -1, 1)
        x[:, 0, :, 5] = 1.0
        x *= np.array([s[size] for s in tops])[:, None, None, None] if far else 1.0 + size
        return torch.from_numpy(x.reshape(B * T, H, D).astype(np.float32)).cuda().to(dtype)

    for T, first, size in ((lo, 0, 0), (n, lo, 1)):
        K, V = side(T, size, which == "k"), side(T, size, which == "v")
        lb.kv8_append(c.gpu, c.tables(), i32([first + T] * B), K, V)
        for b in range(B):
            c.append(b, first, f64(K)[b * T:(b + 1) * T], f64(V)[b * T:(b + 1) * T])
        check_bits(c, "earlier" if first == 0 else "later")
    assert {1, 127, 128, 246} <= set((c.ks if which == "k" else c.vs)[c.table[:, 0], 0] + 127)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (256, 128)])
@pytest.mark.parametrize("new", [1, 4, 150])
def test_largest_finite_values(D, P, new, dtype):
    """Values near the largest finite number stay finite in the cache (at e = 120 codes
    end at 240) and, in tokens a row does not see, do not reach it."""
    H, G, T = 1, 2, 170
    print(f"largest values D={D} P={P} new={new} {dtype}", flush=True)
    c = Cache([T], P, H, D, seed=2)
    K, V = tokens(T, H, D, 5, dtype), tokens(T, H, D, 6, dtype)
    top = torch.finfo(dtype).max
    at = T - (new + 1) // 2          # half of the rows see it
    V[at, 0, 3], V[at, 0, 4], V[at, 0, 5] = top, -top, float("inf")
    K[at, 0, 7], K[at, 0, 8] = top, -float("inf")
    lb.kv8_append(c.gpu, c.tables(), i32([T]), K, V)
    kc, vc, ks, vs = c.gpu
    pg, s = int(c.table[0, at // P]), at % P
    assert int(vs[pg, 0]) == 247 and int(ks[pg, 0]) == 247
    c.fresh()  # the cache as it is, in 64 bits
    K64, V64 = c.read(0, T)
    q = torch.randn(new, H * G, D, device="cuda").bfloat16()
    q[:, :, 7:9] = 0                 # the large keys do not take part in the scores
    O, lse = lb.attention_kv8(q, c.gpu, c.tables(), i32([T]), return_lse=True)
    o, l, A, eps = R.attention(f64(q), K64, V64, T - new, D ** -0.5, True, 0)
    got = f64(O)
    hidden = np.arange(T - new, T) < at
    tol = R.attention_tolerance(o, A, eps, T)
    assert np.isfinite(got[hidden]).all()
    assert np.all(np.abs(got - o)[hidden] <= tol[hidden])
    rest = np.ones(D, bool)
    rest[3:6] = False
    assert np.all(np.abs(got - o)[~hidden][..., rest] <= tol[~hidden][..., rest])
    assert vc[pg, 0, 3:6, s].float().tolist() == [240, -240, 240]
    assert kc[pg, 0, s, 7:9].float().tolist() == [240, -240]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 150])
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_scale_of_zero_keeps_nan_and_infinity(D, new, scale):
    """0 times a NaN or an infinity of Q is NaN: such a row is NaN, the others
    are the mean of what they see."""
    P, H, G, T = 32, 1, 2, 200
    print(f"scale {scale} D={D} new={new}", flush=True)
    c = Cache([T], P, H, D, seed=4)
    fill(c, [T], 6)
    q = torch.randn(new, H * G, D, device="cuda").bfloat16()
    bad = np.zeros((new, H * G), bool)
    for r, h, v in ((0, 0, float("nan")), (new - 1, 1, float("inf")), (new // 2, 0, float("-inf"))):
        q[r, h, 9] = v
        bad[r, h] = True
    O, lse = lb.attention_kv8(q, c.gpu, c.tables(), i32([T]), softmax_scale=scale, return_lse=True)
    assert np.array_equal(np.isnan(f64(O)).all(2), bad) and np.array_equal(np.isnan(f64(O)).any(2), bad)
    assert np.array_equal(np.isnan(f64(lse)), bad)
    K, V = c.read(0, T)
    clean = torch.where(torch.isfinite(q), q, torch.zeros_like(q))
    o, l, A, eps = R.attention(f64(clean), K, V, T - new, scale, True, 0)
    assert np.all((np.abs(f64(O) - o) <= R.attention_tolerance(o, A, eps, T))[~bad])
    assert np.all((np.abs(f64(lse) - l) <= R.lse_tolerance(l, eps, T))[~bad])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 150])
@pytest.mark.parametrize("scale", [2.0 ** -127, -2.0 ** -127])
def test_subnormal_scale(D, new, scale):
    """A scale below the normal numbers against keys and queries near 2^62 still weighs."""
    P, H, G, T = 32, 1, 2, 200
    print(f"scale {scale} D={D} new={new}", flush=True)
    c = Cache([T], P, H, D, seed=4)
    K, V = tokens(T, H, D, 7), tokens(T, H, D, 8)
    K = (K.float().sign() * 2.0 ** 60).bfloat16()
    lb.kv8_append(c.gpu, c.tables(), i32([T]), K, V)
    c.append(0, 0, f64(K), f64(V))
    q = (torch.randn(new, H * G, D, device="cuda").clamp(-3, 3) * 2.0 ** 63).bfloat16()
    q[:, :, 20:] = 0  # |q k| <= 20 * 3 * 2^123: below 2^128.95, and below 2^128 for sums this far from all alike
    O, lse = lb.attention_kv8(q, c.gpu, c.tables(), i32([T]), softmax_scale=scale, return_lse=True)
    K64, V64 = c.read(0, T)
    o, l, A, eps = R.attention(f64(q), K64, V64, T - new, scale, True, 0)
    s = np.einsum("ihd,jd->ihj", f64(q), K64[:, 0]) * scale
    assert 0.5 < np.abs(s).max() < 1.9  # scores that matter, sums below 2^128
    # scale log2(e) is rounded to a multiple of 2^-149, half a step: 2^-23 of it, and the scores with it
    eps = eps + 2.0 ** -22 * np.abs(s).max()
    assert np.all(np.abs(f64(O) - o) <= R.attention_tolerance(o, A, eps, T))
    assert np.all(np.abs(f64(lse) - l) <= R.lse_tolerance(l, eps, T))


@pytest.mark.parametrize("D,G", [(64, 4), (64, 20), (128, 4), (128, 16), (256, 6)])
@pytest.mark.parametrize("lens", [[16] * 9, [16, 4000, 14, 2, 900]])
def test_single_tokens_are_weighed_finely(D, G, lens):
    """Values that cancel in pairs of keys that are nearly alike: what is left is
    the difference of their weights, far below one weight's half step of bf16.
    Weights enter the second product in two bf16 terms, so a weight is off by at
    most 2^-8 of 2^-8."""
    P, H = 16, 2
    print(f"weights D={D} G={G} lens={lens}", flush=True)
    c = Cache(lens, P, H, D, seed=9)
    B, most = len(lens), max(lens)
    g = np.random.default_rng(D + G)
    K = np.zeros((B, most, H, D))
    for b, n in enumerate(lens):
        base = g.standard_normal((n // 2, H, D)) * 0.1
        K[b, :n] = np.repeat(base, 2, 0) + g.standard_normal((n, H, D)) * 0.02
    V = np.where(np.arange(most) % 2 == 0, 1.0, -1.0)[None, :, None, None] * np.ones((B, 1, H, D))
    starts = np.concatenate([[0], np.cumsum(lens)])
    flat = lambda x: torch.from_numpy(np.concatenate([x[b, :n] for b, n in enumerate(lens)]).astype(np.float32)).cuda()
    Kt, Vt = flat(K), flat(V)
    lb.kv8_append(c.gpu, c.tables(), i32(lens), Kt, Vt, q_starts=i32(starts), max_q=most)
    for b, n in enumerate(lens):
        c.append(b, 0, f64(Kt)[starts[b]:starts[b + 1]], f64(Vt)[starts[b]:starts[b + 1]])
    q = torch.randn(B, H * G, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(G)).bfloat16()
    wide = torch.full((B, 40000 // P), -77, dtype=torch.int32, device="cuda")  # a loose bound: the kernel of few rows
    wide[:, :c.width] = c.tables()
    O = f64(lb.attention_kv8(q, c.gpu, wide, i32(lens)))
    for b, n in enumerate(lens):
        K64, V64 = c.read(b, n)
        o, _, A, eps = R.attention(f64(q[b:b + 1]), K64, V64, n - 1, D ** -0.5, True, 0)
        # scores off by eps, a weight by 2^-16 (and 2^-126 where a term is subnormal), n of them
        # added in fp32, one rounding of the output
        tol = (2.5 * eps[..., None] + 2.0 ** -16 * 1.01 + (n + 64) * 2.0 ** -22) * A + 2.0 ** -8 * np.abs(o) + n * 2.0 ** -126
        bad = ~(np.abs(O[b] - o[0]) <= tol[0])
        assert not bad.any(), f"sequence {b}: {int(bad.sum())} of {bad.size} off, {O[b][bad][0]} for {o[0][bad][0]} +- {tol[0][bad][0]}"
