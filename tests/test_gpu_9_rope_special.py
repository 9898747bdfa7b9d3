"""Infinities and NaN in heads that are rotated in part: dims and pairs that do not turn keep what they are."""
import numpy as np
import pytest
import torch

import serve_ref as R
from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


def check(x, y, w, pos, freqs, axis, adjacent, what):
    args = (x.double().cpu().numpy(), None if w is None else w.double().cpu().numpy(), float(np.float32(1e-6)), pos, freqs,
            axis, adjacent)
    with np.errstate(invalid="ignore"):
        ref, mag, turn = R.rotate(*args)
        tol = R.rotate_tolerance(ref, mag, turn, x.shape[2], y.dtype == BF)
    got = y.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: {np.argwhere(np.isnan(got) != np.isnan(ref))[:4].tolist()}"
    far = np.isinf(ref)
    assert np.array_equal(got[far], ref[far]) and np.isfinite(got[~far & ~np.isnan(ref)]).all(), what
    near = np.isfinite(ref)
    assert np.all(np.abs(got[near] - ref[near]) <= np.where(np.isfinite(tol), tol, 0)[near]), what


@pytest.mark.parametrize("D,pairs", [(8, 0), (24, 4), (64, 8), (72, 20), (96, 40), (128, 24), (128, 64), (256, 32), (256, 72)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("axes", [0, 2])
def test_what_does_not_turn_stays(D, pairs, adjacent, axes):
    """Each dim in turn an infinity or NaN, one to a head; with and without a norm; with axes some pairs turn by none."""
    rng = np.random.default_rng(D + pairs)
    axis = None if axes == 0 or pairs == 0 else rng.integers(-1, axes + 1, pairs).astype(np.int32)
    pos = rng.integers(1, 5000, (max(axes, 1), D)).astype(np.int32)
    freqs = 1e4 ** (-np.arange(pairs) / max(pairs, 1))
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
    f = dev(freqs) if pairs else None
    p = dev(pos if axes else pos[0])
    w = torch.from_numpy(rng.random(D).astype(np.float32) + 0.5).cuda()
    for dtype in (F, BF):
        x = torch.from_numpy(rng.standard_normal((D, 4, D)).astype(np.float32)).cuda().to(dtype)
        for t in range(D):
            x[t, 0, t], x[t, 1, t], x[t, 2, t] = float("inf"), float("-inf"), float("nan")
        print(f"special D={D} pairs={pairs} {adjacent} axes={axes} {dtype}", flush=True)
        y, z = lb.qk_norm_rope(x, x.clone(), p, f, None, w, pair_axis=dev(axis), adjacent=adjacent)
        check(x, y, None, pos, freqs, axis, adjacent, "without a norm")
        check(x, z, w, pos, freqs, axis, adjacent, "with a norm")
