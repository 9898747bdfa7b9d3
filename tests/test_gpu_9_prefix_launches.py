"""Attention behind shared prefixes in every kind of launch that the library's plan has, whatever its numbers are: the
sizes are found by asking it."""
import pytest
import torch

from prefix_launches import every_kind, launches
from test_gpu_9_prefix_starts import Told
from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", list(every_kind()))
def test_every_kind_of_launch(kind):
    print(kind, flush=True)
    k = Told(**every_kind()[kind], short=270)
    out = k.run()
    k.check(out, kind, rows=2, some=6)
    again = k.run()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
    k.check(k.run(causal=False, softmax_scale=-0.2), f"{kind}, all pairs", causal=False, scale=-0.2, rows=1, some=2)


def test_through_the_binding():
    """The plan's fields by name; a loose bound on the new tokens costs the second terms of the weights."""
    cache = lb.empty_kv8(8, 64, 2, 128, device="cuda")
    i32 = lambda *x: torch.zeros(x, dtype=torch.int32, device="cuda")
    args = (cache, i32(1, 500), i32(1), i32(64, 8), i32(64), 8, 64)
    tight = lb.attention_kv8_prefix_launches(*args, q_starts=i32(65), max_q=1, max_kv=500)
    assert tight == launches(8, 2, 128, 64, 500 * 64, 1, 64, 64, 64, 1, 500)
    assert set(tight) == {n for n, _ in lb.Kv8PrefixPlan._fields_} and tight["launches"] == 2 and tight["weight_terms"] == 2
    assert lb.attention_kv8_prefix_launches(*args, q_starts=i32(65), max_kv=500)["weight_terms"] == 1
    with pytest.raises(lb.LowbitError):
        lb.attention_kv8_prefix_launches(*args[:5], 7, 64)
