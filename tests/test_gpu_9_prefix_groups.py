"""Attention behind shared prefixes with many groups, and with more groups than sequences."""
import numpy as np
import pytest

from test_gpu_9_prefix_starts import Told, poison

pytestmark = pytest.mark.gpu


def spread(groups, seqs, seed):
    """Sequences of each group, some of them none."""
    g = np.random.default_rng(seed)
    return np.bincount(g.integers(0, groups, seqs), minlength=groups).tolist()


def case(groups, seqs, told, Hq, H, D, P, new=1, seed=0):
    return dict(prefix=[told] * groups, count=spread(groups, seqs, seed + groups), new=[new] * seqs,
                own=[5 + 11 * (i % 5) for i in range(seqs)], Hq=Hq, H=H, D=D, P=P)


# Whether there are at most 16 groups, at most 64 sequences and at most 64 groups decides how they are found; in one
# launch and behind the groups' own, those in prompt tiles (70 groups) and in attn_decode (65).
GROUPS = {}
for n, B in ((16, 3), (9, 60), (16, 64), (16, 70), (17, 5), (17, 60), (65, 40), (130, 10)):
    for D, told in ((64, 300), (128, 300), (256, 300), (64, 20000), (128, 20000), (256, 20000)):
        H = 4 if D == 64 else 2
        GROUPS[f"{n} groups, {B} sequences, {D}, {told}"] = case(n, B, told, 4 * H, H, D, 32, seed=B)
GROUPS["65 groups, 200 sequences, 64, 20000"] = case(65, 200, 20000, 16, 4, 64, 32, seed=200)
for D in (64, 128, 256):
    GROUPS[f"70 groups, 300 sequences, {D}, 20000"] = case(70, 300, 20000, 8, 1, D, 32, seed=300)


@pytest.mark.parametrize("name", GROUPS)
def test_many_groups(name):
    print(name, flush=True)
    k = Told(**GROUPS[name], short=60)
    if k.told > 1000:
        poison(k)
    out = k.run()
    k.check(out, name, rows=1, some=9)
    assert not out[0][:k.rows[-1]].isnan().any()


@pytest.mark.parametrize("D,told", [(64, 300), (128, 300), (256, 300), (64, 20000), (128, 20000), (256, 20000)])
@pytest.mark.parametrize("counts", [[0] * 13 + [1, 1, 1], [1] + [0] * 14 + [2], [0] * 15 + [1], [0, 0, 2, 0, 0, 1] + [0] * 30])
def test_more_groups_than_sequences(D, told, counts):
    """Groups at lanes that have no sequence; some sequences before the first group or behind the last one have none."""
    print(f"groups {len(counts)} of {sum(counts)} sequences D={D} told={told}", flush=True)
    B = sum(counts)
    k = Told(prefix=[told] * len(counts), count=counts, new=[2] * B, own=[5 + 9 * b for b in range(B)], Hq=8, H=2, D=D, P=16, short=90)
    k.check(k.run(), "groups", rows=2)
    # one sequence more, of no group
    k = Told(prefix=[told] * len(counts), count=counts, new=[2] * (B + 1), own=[5 + 9 * b for b in range(B + 1)], Hq=8, H=2, D=D, P=16,
             short=90)
    k.check(k.run(), "behind the last group", rows=2)
    # and the first sequence before the first group
    k.starts = np.concatenate([[1], 1 + np.cumsum(counts)])
    k.check(k.run(), "before the first group", rows=2)
