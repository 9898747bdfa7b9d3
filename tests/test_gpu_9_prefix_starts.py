"""Attention behind shared prefixes with rows between the sequences (a padded batch), and with groups of
more sequences than the call was told."""
import numpy as np
import pytest
import torch

from test_gpu_9_kv8 import i32, tokens
from test_gpu_9_prefix import CASES, Call, LAUNCHES, OWN

pytestmark = pytest.mark.gpu


class Told(Call):
    """Prefixes of `short` tokens and fewer, told to be as long as `prefix` says (which sizes the launches), sequence b's
    rows from b * spacing on (0: one after the other)."""

    def __init__(self, prefix, spacing=0, short=100, **kw):
        super().__init__(prefix=[min(n, short - 7 * (g % 8)) for g, n in enumerate(prefix)], **kw)
        self.told = max(prefix)
        wide = torch.full((self.G, -(-self.told // self.P)), -77, dtype=torch.int32, device="cuda")
        n = min(self.prefix_table.shape[1], wide.shape[1])
        wide[:, :n] = self.prefix_table[:, :n]
        self.prefix_table = wide
        if spacing:
            self.rows = np.arange(self.B + 1) * spacing
            self.q = tokens(int(self.rows[-1]) + 2, self.Hq, self.D, 7)

    def args(self, **kw):
        return super().args(**{"max_prefix": self.told, **kw})


def poison(k, **kw):
    """The same call with queries that leave NaN in every sum it writes to the workspace."""
    q = k.q
    k.q = torch.full_like(q, float("nan"))
    k.run(max_q=int(k.rows[-1]), max_seqs=k.B, **kw)
    k.q = q


SPACED = {
    # the groups in prompt tiles, then in attn_decode
    "groups, 64": dict(LAUNCHES["groups, 64"], spacing=8),
    "groups, 128": dict(LAUNCHES["groups, 128"], spacing=8),
    "groups, 256 rows": dict(LAUNCHES["groups, 256 rows"], spacing=3),
    "groups, 256": dict(LAUNCHES["groups, 256"], spacing=5),
    "few, 64": dict(LAUNCHES["few, 64"], spacing=8),
    "few, 64, 32 rows a wave": dict(LAUNCHES["few, 64, 32 rows a wave"], spacing=4),
    "few, 128": dict(LAUNCHES["few, 128"], spacing=8),
    "few, 256": dict(LAUNCHES["few, 256"], spacing=8),
    # one launch
    "pieces, 128": dict(LAUNCHES["pieces, 128"], spacing=6),
    "shares, 64": dict(LAUNCHES["shares, 64"], spacing=2),
    "parts, 128": dict(prefix=[700, 90], count=[3, 2], new=[30] * 5, own=[70, 150, 30, 90, 300], Hq=8, H=2, D=128, P=16, spacing=33),
}


@pytest.mark.parametrize("name", SPACED)
def test_rows_between_sequences(name):
    """Every sequence's first rows see their prefix, wherever they lie; other rows are left as they were."""
    print(f"spaced {name}", flush=True)
    k = Told(**SPACED[name])
    poison(k)
    out = k.run()
    k.check(out, name, rows=2, some=12)
    own = torch.zeros(len(k.q), dtype=torch.bool)
    for b in range(k.B):
        own[k.rows[b]:k.rows[b] + k.new[b]] = True
    assert (out[0][~own] == 7).all() and (out[1][~own] == 7).all()
    assert not out[0][own].isnan().any()
    again = k.run()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.parametrize("name", ["groups, 64", "groups, 128", "groups, 256", "few, 128"])
def test_more_sequences_than_told(name):
    """max_seqs sizes the launch: with one too small the results stay what they are."""
    print(f"max_seqs {name}", flush=True)
    k = Told(**LAUNCHES[name])
    poison(k)
    most = max(k.count)
    for m in (most // 2, 1):
        k.check(k.run(max_seqs=m), f"{name} max_seqs {m}", rows=2, some=12)


def test_equal_groups_with_rows_between():
    """seq_starts None: equally many sequences each, their rows spaced."""
    k = Told(spacing=8, prefix=[9000, 3000], count=[32, 32], new=[1] * 64, own=OWN(64), Hq=16, H=4, D=128, P=64)
    poison(k)
    print("spaced, equal groups", flush=True)
    k.check(k.run(seq_starts=None, max_seqs=None), "equal groups", rows=1, some=12)
    k.check(k.run(), "the same named", rows=1, some=12)


@pytest.mark.parametrize("name", ["corners", "tiles"])
def test_padded_corners(name):
    """Empty sequences, sequences of no group and short ones, every sequence in max_q rows of its own."""
    case = dict(CASES[name])
    case["new"] = [max(case["new"])] * len(case["new"])
    case["own"] = [max(t, case["new"][0]) for t in case["own"]]
    k = Told(spacing=case["new"][0] + 5, Hq=8, H=2, D=128, P=32, **case)
    print(f"padded {name}", flush=True)
    k.check(k.run(), name, rows=4)
