"""How finely tokens behind shared prefixes are weighed: values that cancel in pairs of
keys that are nearly alike, in each of the launches that calls of few rows take."""
import numpy as np
import pytest
import torch

import serve_ref as R
from test_gpu_9_kv8 import Cache, f64, i32
from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu

# Hq, H, D, P, tokens of a prefix that the call is told, sequences of each group, new tokens of each
CASES = {
    "groups in prompt tiles, 64": (16, 4, 64, 64, 8000, 30, 2),
    "groups in prompt tiles, 128": (16, 4, 128, 64, 9000, 15, 1),
    "groups in prompt tiles of 256 rows, 128": (16, 4, 128, 64, 9000, 30, 2),
    "groups in prompt tiles, 256": (12, 2, 256, 128, 9000, 21, 1),
    "groups in attn_decode, 64": (8, 8, 64, 64, 40000, 8, 1),
    "groups in attn_decode, 128": (8, 8, 128, 64, 60000, 8, 1),
    "drafts, 64": (32, 4, 64, 32, 400, 2, 8),
    "drafts, 128": (10, 2, 128, 16, 200, 100, 5),
    "drafts, 256": (24, 4, 256, 32, 400, 2, 8),
    "single tokens, 64": (8, 2, 64, 16, 300, 3, 1),
    "single tokens, 128": (8, 2, 128, 16, 300, 3, 1),
    "single tokens, 256": (12, 2, 256, 16, 300, 3, 1),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("prefix", [(16, 14), (16, 770)])
def test_few_rows_are_weighed_finely(name, prefix):
    """What is left of such values is the difference of their weights, far below one weight's half step of bf16.
    Weights enter the second product in two bf16 terms, so a weight is off by at most 2^-8 of 2^-8."""
    Hq, H, D, P, told, each, new = CASES[name]
    told = max(told, *prefix)
    B, own = 2 * each, [new + new % 2 + 2 * (b % 4) for b in range(2 * each)]
    print(f"weights {name} {prefix}", flush=True)
    lens = list(prefix) + own
    c = Cache(lens, P, H, D, seed=9)
    most = max(lens)
    g = np.random.default_rng(D + each)
    K, V = np.zeros((len(lens), most, H, D)), np.ones((len(lens), most, H, D))
    for b, n in enumerate(lens):
        K[b, :n] = np.repeat(g.standard_normal((n // 2, H, D)) * 0.1, 2, 0) + g.standard_normal((n, H, D)) * 0.02
    V[:, 1::2] = -1
    starts = np.concatenate([[0], np.cumsum(lens)])
    flat = lambda x: torch.from_numpy(np.concatenate([x[b, :n] for b, n in enumerate(lens)]).astype(np.float32)).cuda()
    Kt, Vt = flat(K), flat(V)
    lb.kv8_append(c.gpu, c.tables(), i32(lens), Kt, Vt, q_starts=i32(starts), max_q=most)
    for b, n in enumerate(lens):
        c.append(b, 0, f64(Kt)[starts[b]:starts[b + 1]], f64(Vt)[starts[b]:starts[b + 1]])
    q = torch.randn(B * new, Hq, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(each)).bfloat16()
    table = c.tables()
    wide = torch.full((2, told // P + 1), -77, dtype=torch.int32, device="cuda")  # a loose bound on the prefixes
    wide[:, :c.width] = table[:2, :wide.shape[1]]
    O = f64(lb.attention_kv8_prefix(q, c.gpu, wide, i32(prefix), table[2:], i32(own), max_kv=max(own), max_prefix=told,
                                    causal=False))
    for b in range(B):
        Kp, Vp = c.read(b // each, prefix[b // each])
        Ko, Vo = c.read(2 + b, own[b])
        o, _, A, eps = R.attention_prefix(f64(q[b * new:(b + 1) * new]), Kp, Vp, Ko, Vo, 0, D ** -0.5, False)
        n = len(Kp) + len(Ko)
        # scores off by eps, a weight by 2^-16 (and 2^-126 where a term is subnormal), n of them
        # added in fp32, one rounding of the output
        tol = (2.5 * eps[..., None] + 2.0 ** -16 * 1.01 + (n + 64) * 2.0 ** -22) * A + 2.0 ** -8 * np.abs(o) + n * 2.0 ** -126
        bad = ~(np.abs(O[b * new:(b + 1) * new] - o) <= tol)
        assert not bad.any(), f"sequence {b}: {int(bad.sum())} of {bad.size} off, {O[b * new:(b + 1) * new][bad][0]} for {o[bad][0]} +- {tol[bad][0]}"
