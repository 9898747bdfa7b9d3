"""Which launches calls behind shared prefixes take, on a machine without a GPU."""
import ctypes

import pytest

from prefix_launches import every_kind, kind, launches, launches_of
from test_gpu_9_prefix import LAUNCHES
from test_gpu_9_prefix_weights import CASES as FEW_ROWS
from test_prefix_cpu import batch, kv, prefix
from ultra_bit_dit_amd import lowbit as lb


def test_refusals():
    """As the call itself, before anything is read."""
    f, plan = lb.lib().lowbit_attention_kv8_prefix_launches, lb.Kv8PrefixPlan()
    assert f(kv(), prefix(), batch(), 4, None) == lb.E_NULL
    for args, status in (((None, prefix(), batch(), 4), lb.E_NULL), ((kv(), None, batch(), 4), lb.E_NULL),
                         ((kv(head_dim=96), prefix(), batch(), 4), lb.E_UNSUPPORTED), ((kv(), prefix(), batch(), 3), lb.E_SHAPE),
                         ((kv(), prefix(max_len=49), batch(), 4), lb.E_SHAPE)):
        plan.launches = 9
        assert f(*args, ctypes.byref(plan)) == status and plan.launches == 0
    assert f(kv(), prefix(), batch(), 4, ctypes.byref(plan)) == lb.OK and plan.launches in (1, 2)


def test_the_kinds_that_are_run():
    """One launch and two, every kernel of each head size, weights in one term and two."""
    kinds = list(every_kind())
    for D in (64, 128, 256):
        mine = [k for k in kinds if k.startswith(f"D={D} ")]
        for part in ("attn_decode 16 rows, whole", "attn_decode 16 rows, pieces", "attn_decode 16 rows, shares", "prompt tiles of 128, whole",
                     "prompt tiles of 128, cut", "last round cut", "1 terms", "2 terms", "groups: attn_decode", "groups: prompt tiles of 128",
                     "sequences: 16 rows, whole", "sequences: 16 rows, pieces"):
            assert any(part in k for k in mine), (D, part)
    for k in ("D=64 attn_decode 32 rows, pieces", "D=64 attn_decode 32 rows, shares", "D=128 prompt tiles of 256, cut, 1 terms"):
        assert k in kinds, k
    assert any("D=128 groups: prompt tiles of 256" in k for k in kinds) and any("sequences: 32 rows" in k for k in kinds)


def test_sizes_of_the_tests_of_launches():
    """What those sizes are for: one launch and two of every head size, tiles of either kernel."""
    plans = [(c["D"], launches_of(c)) for c in LAUNCHES.values()]
    assert all(p for _, p in plans)
    for D in (64, 128, 256):
        assert {(p["launches"], p["tile_rows"] >= 128) for d, p in plans if d == D} == {(1, False), (1, True), (2, False), (2, True)}
    assert len({kind(D, p) for D, p in plans}) >= 20


@pytest.mark.parametrize("name", FEW_ROWS)
def test_few_rows_have_two_terms(name):
    Hq, H, D, P, told, each, new = FEW_ROWS[name]
    for n in (told, 10 * told):
        for own in (new + new % 2 + 6, 1000):
            p = launches(Hq, H, D, P, n, 2, each, 2 * each, 2 * each * new, new, own, q_starts=False)
            assert p["weight_terms"] == 2 and new * Hq // H <= 64


def test_weight_terms():
    """Two wherever a sequence has at most 64 rows of a key head."""
    for D in (64, 128, 256):
        for G in (1, 4, 8):
            for seqs in (1, 40, 700):
                for told in (10, 3000, 60000):
                    for q in (1, 64 // G, 64 // G + 1, 300):
                        p = launches(2 * G, 2, D, 64, told, 1, seqs, seqs, seqs * q, q, q + 100)
                        assert p["weight_terms"] == 2 or q * G > 64
    assert launches(8, 2, 128, 64, 3000, 1, 8, 8, 8 * 300, 300, 400)["weight_terms"] == 1


@pytest.mark.parametrize("D,G", [(64, 4), (128, 5), (256, 6)])
def test_rows_between_sequences_are_reckoned_with(D, G):
    """A batch padded to many rows a sequence fills as many tiles as one that has them."""
    args = dict(Hq=8 * G, H=8, D=D, P=64, max_prefix=20000, groups=2, max_seqs=32, seqs=64, max_q=1, max_kv=100)
    tight, loose = launches(total_q=64, **args), launches(total_q=64 * 64, **args)
    assert tight["launches"] == 2 and (loose["launches"] == 1 or loose["tile_parts"] < tight["tile_parts"])
    # more than 256 rows of a sequence go by the sequences, which skip those between
    assert launches(total_q=64 * (256 // G + 1), **args)["launches"] == 1


@pytest.mark.parametrize("D", [64, 128, 256])
def test_groups_of_more_rows_than_int_counts(D):
    """More than 2^30 rows of a key head in the batch: a padded group could have them all, so it is not asked for."""
    for H, G, groups, seqs in ((1, 64, 4, 1 << 10), (1, 8, 1, 2), (2, 16, 1 << 10, 1 << 20), (1, 64, 1, 1)):
        for told in (1000, 1 << 28):
            total = (1 << 30) // G + 1
            p = launches(Hq=H * G, H=H, D=D, P=128, max_prefix=told, groups=groups, max_seqs=seqs // groups, seqs=seqs, max_q=1,
                         max_kv=100, total_q=total)
            assert p is None or p["launches"] == 1
