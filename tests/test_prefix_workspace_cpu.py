"""The workspace that attention behind shared prefixes asks for, on a machine without a GPU."""
import ctypes
import random

import pytest

from test_prefix_cpu import batch, kv, prefix
from ultra_bit_dit_amd import lowbit as lb


def need(D, H, G, groups, max_seqs, seqs, total_q, max_q, max_kv, max_len):
    n = ctypes.c_size_t()
    c = kv(kv_heads=H, head_dim=D, page_tokens=64, n_pages=1 << 20)
    p = prefix(n_groups=groups, table_width=1 << 16, max_len=max_len, max_seqs=max_seqs)
    b = batch(n_seqs=seqs, q_starts=0x80000, total_q=total_q, max_q=max_q, table_width=1 << 16, max_kv=max_kv)
    assert lb.lib().lowbit_attention_kv8_prefix_workspace(c, p, b, H * G, ctypes.byref(n)) == lb.OK
    return n.value


@pytest.mark.parametrize("D,H,G", [(64, 8, 2), (64, 4, 8), (128, 8, 5), (128, 1, 16), (256, 4, 6), (256, 2, 1)])
def test_smaller_calls_need_no_more(D, H, G):
    """Fewer sequences, groups or rows and closer bounds, one of them or all: a server reserves for its largest batch."""
    rng = random.Random(D + H)
    log = lambda n: max(1, min(n, int(n ** rng.random())))
    for _ in range(1500):
        seqs, max_q = log(2000), log(700)
        big = dict(groups=log(seqs), max_seqs=log(seqs), seqs=seqs, max_q=max_q, total_q=max(max_q, log(2 * seqs * max_q)),
                   max_kv=log(20000), max_len=log(100000))
        small = {k: log(v) if rng.random() < 0.5 else v for k, v in big.items()}
        small["max_seqs"] = min(small["max_seqs"], small["seqs"])
        small["max_q"] = min(small["max_q"], small["total_q"])
        assert need(D, H, G, **small) <= need(D, H, G, **big), (small, big)


def test_one_prefix_of_a_server():
    """The batch of a server shrinks, and its prefix: what was reserved at first holds."""
    at = lambda seqs, n: need(128, 8, 5, 1, seqs, seqs, seqs, 1, 500, n)
    sizes = [at(B, 32760) for B in (1, 2, 7, 32, 64, 80, 200)]
    assert sizes == sorted(sizes) and sizes[-1] < 200 << 20
    sizes = [at(64, n) for n in (10, 1000, 8000, 32760)]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("D,H,G", [(64, 8, 4), (128, 8, 5), (256, 4, 6)])
def test_long_prompts_keep_no_sums(D, H, G):
    """Rows that go by their sequences alone leave no sums: the bytes do not grow with them, padded or not."""
    for seqs, q, padded in ((8, 4096, 4096), (64, 1000, 1000), (64, 1, 1000), (1, 1 << 20, 1 << 20)):
        assert need(D, H, G, 1, seqs, seqs, seqs * padded, q, q, 6001) < 200 << 20
