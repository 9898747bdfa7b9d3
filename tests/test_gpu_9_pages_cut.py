"""Children that need more pages than their table rows have are counted on the device."""
import numpy as np
import pytest
import torch

import serve_ref as R
from test_gpu_9_pages import batch, cache_of, i32
from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,B,n_pages", [(1, 1, 40), (9, 4, 90), (2500, 300, 4000), (300, 5000, 40000)])
def test_cut_children_are_counted(n, B, n_pages):
    """Rows that are wide enough for all, some and none; the count is set, whatever it was; the other outputs are those of
    the call without it."""
    P = 16
    rng = np.random.default_rng(n)
    table, lens, refs = batch(rng, n_pages, P, B, 8, 2)
    parents, grow = rng.integers(-1, B + 1, n), rng.choice([0, 1, P, 3 * P + 1], n)
    grow[0], parents[0] = 3 * P + 1, 0
    args = [i32(table), i32(lens), i32(refs), i32(parents)]
    most = int(grow.max())
    print(f"cut n={n} B={B}", flush=True)
    for width in (1, 4, 8, 40):
        cache = cache_of(n_pages, P, 1, 64, n)
        cut = torch.full((1,), 77, dtype=torch.int32, device="cuda")
        out = lb.kv8_fork(cache, *args, grow=i32(grow), max_grow=most, width=width, cut=cut)
        had = [R.Pages(n_pages, P)._cut(lens[p], 8) if 0 <= p < B else 0 for p in parents]
        want = [h + int(g) > width * P for h, g in zip(had, grow)]
        assert cut.item() == sum(want), width
        # what the new lengths say too
        lengths = out[1].cpu().numpy()
        assert [int(x) < h + int(g) for x, h, g in zip(lengths, had, grow)] == want
        again = lb.kv8_fork(cache_of(n_pages, P, 1, 64, n), *args, grow=i32(grow), max_grow=most, width=width)
        if out[3].item() == 0:
            assert all(torch.equal(a, b) for a, b in zip(out, again))
    assert cut.item() == 0


def test_a_full_row_that_would_grow():
    """The default width is the old table's: a sequence that fills its row does not grow, which the count shows."""
    cache = cache_of(8, 16, 1, 64, 1)
    cut = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = i32([[3, 5]]), i32([32]), i32([0, 0, 0, 1, 0, 1, 0, 0]), i32([0, 0])
    out = lb.kv8_fork(cache, *args, grow=1, cut=cut)
    assert cut.item() == 2 and out[1].tolist() == [32, 32] and out[3].item() == 0
    out = lb.kv8_fork(cache, *args, grow=1, cut=cut, width=3)
    assert cut.item() == 0 and out[1].tolist() == [33, 33]
    for bad in (cut.long(), cut.cpu(), torch.zeros(2, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            lb.kv8_fork(cache, *args, grow=1, cut=bad)
