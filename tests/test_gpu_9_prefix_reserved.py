"""Calls behind shared prefixes captured in the workspace that was reserved for a larger one."""
import pytest
import torch

from test_gpu_9_kv8 import i32
from test_gpu_9_prefix import OWN
from test_gpu_9_prefix_starts import Told
from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,H,D,new", [(40, 8, 128, 1), (16, 4, 64, 2), (12, 2, 256, 1)])
def test_the_largest_batch_reserves_for_all(Hq, H, D, new):
    """One reservation, then graphs of smaller batches behind shorter prefixes on the same stream; each replayed twice."""
    largest = dict(prefix=[32760], count=[80], new=[new] * 80, own=OWN(80, 20))
    k = Told(**largest, Hq=Hq, H=H, D=D, P=64)
    a = k.args()
    a.pop("return_lse")
    torch.cuda.synchronize()
    lb.release_workspaces()
    s = torch.cuda.Stream()
    need = lb.attention_kv8_prefix_workspace(k.c.gpu, k.prefix_table, i32(k.prefix), k.table, i32(k.own), Hq, len(k.q), **a)
    with torch.cuda.stream(s):
        lb.reserve_workspace(need)
    torch.cuda.synchronize()
    for B, told in ((80, 32760), (64, 32760), (32, 32760), (24, 8000), (64, 1000), (3, 8000), (1, 32760), (1, 1)):
        print(f"captured B={B} prefix={told} D={D}", flush=True)
        k = Told(prefix=[told], count=[B], new=[new] * B, own=OWN(B, 20), Hq=Hq, H=H, D=D, P=64)
        pl, ow, a = i32(k.prefix), i32(k.own), k.args()
        call = lambda **kw: lb.attention_kv8_prefix(k.q, k.c.gpu, k.prefix_table, pl, k.table, ow, **{**a, **kw})
        want = [x.clone() for x in call()]  # on the current stream, which has a workspace of its own
        O, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(O=O, lse=lse)
        used = int(k.rows[-1])
        for _ in range(2):
            O.zero_(), lse.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(O[:used], want[0][:used]) and torch.equal(lse[:used], want[1][:used]), (B, told)
