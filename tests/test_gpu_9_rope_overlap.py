"""Outputs of the head norms with rotation between other tensors' rows: taken where no byte is shared, refused where one is."""
import random

import pytest
import torch

from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu
D = 8


def test_rows_between_rows():
    """Inputs and outputs at random places and distances of one buffer, against the bytes one by one."""
    rng = random.Random(3)
    f = torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64, device="cuda")
    taken = refused = 0
    print("rows between rows", flush=True)
    while taken < 60:
        T, hq, hk = rng.randint(1, 6), rng.randint(1, 3), rng.randint(1, 3)
        one = 8 * rng.randint(4, 14)
        place = {}
        for name, h in (("q", hq), ("k", hk), ("qo", hq), ("ko", hk)):
            stride = one if rng.random() < 0.7 else D * h + 8 * rng.randint(0, 9)
            place[name] = (8 * rng.randint(0, 40), max(stride, D * h), h)
        if rng.random() < 0.3:
            place["qo"] = place["q"]
        if rng.random() < 0.3:
            place["ko"] = place["k"]
        at = {n: {e for t in range(T) for e in range(p + t * s, p + t * s + D * h)} for n, (p, s, h) in place.items()}
        same = lambda x, y: place[x][0] == place[y][0] and (T == 1 or place[x][1] == place[y][1])
        share = any(at[x] & at[y] and not (ok and same(x, y))
                    for x, y, ok in (("q", "qo", True), ("k", "ko", True), ("q", "ko", False), ("k", "qo", False), ("qo", "ko", False)))
        if share and refused > 3 * taken:
            continue
        buf = torch.randn(1024, device="cuda").bfloat16()
        t = {n: buf.as_strided((T, h, D), (s, D, 1), p) for n, (p, s, h) in place.items()}
        pos = torch.arange(T, dtype=torch.int32, device="cuda")
        before = buf.clone()
        if share:
            with pytest.raises(lb.LowbitError) as e:
                lb.qk_norm_rope(t["q"], t["k"], pos, f, Q_out=t["qo"], K_out=t["ko"])
            assert e.value.status == lb.E_UNSUPPORTED and torch.equal(buf, before)
            refused += 1
            continue
        want = lb.qk_norm_rope(t["q"].clone(), t["k"].clone(), pos, f)
        lb.qk_norm_rope(t["q"], t["k"], pos, f, Q_out=t["qo"], K_out=t["ko"])
        assert torch.equal(t["qo"], want[0]) and torch.equal(t["ko"], want[1])
        rest = [e for e in range(1024) if e not in at["qo"] and e not in at["ko"]]
        assert torch.equal(buf[rest], before[rest])
        taken += 1
    assert refused > 20
