"""A decode layer of the 1..2-bit formats through the cache: packed q/k/v
product, cache write, attention, packed o product, each step checked on the
GPU's own input to it."""
import numpy as np
import pytest
import torch

import synth
from oracle import oracle as O
from ultra_bit_dit_amd import lowbit as lb

from helpers import SEED, assert_within
from test_gpu_3_gemm import bf16_dev, make
from test_gpu_9_kv8 import Cache, compare, f64, fill, i32

pytestmark = pytest.mark.gpu


def bits(t):
    """bf16 tensor -> its uint16 words on the host."""
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("fmt", [1, 2, 3])
@pytest.mark.parametrize("new", [1, 5, 70])
def test_layer_of_packed_products(fmt, new):
    hid, H, G, D, P = 512, 2, 2, 64, 32
    Hq, T = H * G, 2 * new
    n_qkv = (Hq + 2 * H) * D
    print(f"layer fmt={fmt} new={new}", flush=True)
    wq, wo = make(fmt, n_qkv, hid, tid=301), make(fmt, hid, Hq * D, tid=305)

    def product(w, x, n, what):
        y = lb.gemm(fmt, T, n, x.shape[1], w[2], w[3], x, y_dtype=lb.BF16)
        yref, absY = O.matmul(w[0], w[1], O.X_BF16, bits(x))
        assert_within(y.float().cpu().numpy(), yref, absY, bf16_out=True, what=what)
        return y

    lens = [new + 90, new + 3]
    c = Cache(lens, P, H, D, seed=new)
    fill(c, [90, 3], 17)
    heads = product(wq, bf16_dev(synth.normal_bf16(SEED, 303, T, hid)), n_qkv, "q/k/v").view(T, Hq + 2 * H, D)
    q, K, V = heads[:, :Hq], heads[:, Hq:Hq + H], heads[:, Hq + H:]
    table, dl = c.tables(), i32(lens)
    lb.kv8_append(c.gpu, table, dl, K, V)
    for b in range(2):
        c.append(b, lens[b] - new, f64(K)[b * new:(b + 1) * new], f64(V)[b * new:(b + 1) * new])
    c.check("layer")
    o, lse = lb.attention_kv8(q, c.gpu, table, dl, return_lse=True)
    compare(c, q, o, lse, lens, [0, new, 2 * new])
    product(wo, o.view(T, Hq * D), hid, "o")
