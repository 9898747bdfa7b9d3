"""Attention behind shared prefixes in every kind of launch that the library's plan has, whatever its numbers are: the
sizes are found by asking it."""
import pytest
import torch

from prefix_launches import every_kind
from test_gpu_9_prefix_starts import Told

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", list(every_kind()))
def test_every_kind_of_launch(kind):
    print(kind, flush=True)
    k = Told(**every_kind()[kind], short=290)
    out = k.run()
    k.check(out, kind, rows=2, some=6)
    again = k.run()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])
    k.check(k.run(causal=False, softmax_scale=-0.2), f"{kind}, all pairs", causal=False, scale=-0.2, rows=1, some=2)
