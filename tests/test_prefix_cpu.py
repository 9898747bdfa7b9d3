"""Attention behind shared prefixes on a machine without a GPU: refusals before any
HIP call, workspace bytes, and the plain form's pin."""
import ctypes

import numpy as np
import pytest

import mx_ref as M
import serve_ref as R
from ultra_bit_dit_amd import lowbit as lb

A16, A4 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)


def kv(**over):
    c = dict(n_pages=4, page_tokens=16, kv_heads=2, head_dim=64, k_codes=0x10000, v_codes=0x20000, k_scales=0x30000,
             v_scales=0x40000)
    c.update(over)
    return lb.Kv8(*[c[f[0]] for f in lb.Kv8._fields_])


def batch(**over):
    b = dict(n_seqs=4, page_table=0x50000, table_width=2, kv_lens=0x60000, q_starts=None, total_q=4, max_q=1, max_kv=32,
             bad_pages=None)
    b.update(over)
    return lb.Kv8Batch(*[b[f[0]] for f in lb.Kv8Batch._fields_])


def prefix(**over):
    p = dict(n_groups=2, page_table=0x50000, table_width=3, lens=0x60000, seq_starts=0x70000, max_seqs=2, max_len=48)
    p.update(over)
    return lb.Kv8Prefix(*[p[f[0]] for f in lb.Kv8Prefix._fields_])


def call(c=None, p=None, b=None, hq=4, Q=A16, qs=256, scale=1.0, O=A16, os=256, lse=None):
    return lb.lib().lowbit_attention_kv8_prefix(kv() if c is None else c, prefix() if p is None else p, batch() if b is None else b,
                                                hq, Q, qs, scale, 1, O, os, lse, None)


@pytest.mark.parametrize("c,p,b,status", [
    (dict(k_codes=None), {}, {}, lb.E_NULL), ({}, dict(page_table=None), {}, lb.E_NULL), ({}, dict(lens=None), {}, lb.E_NULL),
    ({}, {}, dict(kv_lens=None), lb.E_NULL), (dict(page_tokens=48), {}, {}, lb.E_UNSUPPORTED),
    (dict(head_dim=96), {}, {}, lb.E_UNSUPPORTED), ({}, dict(n_groups=0), {}, lb.E_SHAPE),
    ({}, dict(n_groups=(1 << 20) + 1), {}, lb.E_SHAPE), ({}, dict(table_width=0), {}, lb.E_SHAPE),
    ({}, dict(max_len=0), {}, lb.E_SHAPE), ({}, dict(max_len=49), {}, lb.E_SHAPE),  # more than the table holds
    ({}, dict(table_width=1 << 26, max_len=1 << 30), {}, lb.E_SHAPE),  # with the own tokens more than 2^30
    ({}, dict(max_seqs=0), {}, lb.E_SHAPE), ({}, dict(max_seqs=5), {}, lb.E_SHAPE),
    ({}, dict(n_groups=3, seq_starts=None), {}, lb.E_SHAPE),  # four sequences for three groups
    ({}, {}, dict(n_seqs=0), lb.E_SHAPE), ({}, {}, dict(max_kv=33), lb.E_SHAPE),
    ({}, dict(page_table=0x50002), {}, lb.E_ALIGN), ({}, dict(lens=0x60001), {}, lb.E_ALIGN),
    ({}, dict(seq_starts=0x70002), {}, lb.E_ALIGN), ({}, {}, dict(page_table=0x50001), lb.E_ALIGN)])
def test_refusals(c, p, b, status):
    assert call(kv(**c), prefix(**p), batch(**b)) == status
    n = ctypes.c_size_t(5)
    f = lb.lib().lowbit_attention_kv8_prefix_workspace
    assert f(kv(**c), prefix(**p), batch(**b), 4, ctypes.byref(n)) == status and n.value == 0


def test_more_refusals():
    f = lb.lib().lowbit_attention_kv8_prefix
    assert f(None, prefix(), batch(), 4, A16, 256, 1.0, 1, A16, 256, None, None) == lb.E_NULL
    assert f(kv(), None, batch(), 4, A16, 256, 1.0, 1, A16, 256, None, None) == lb.E_NULL
    assert f(kv(), prefix(), None, 4, A16, 256, 1.0, 1, A16, 256, None, None) == lb.E_NULL
    assert call(Q=None) == lb.E_NULL and call(O=None) == lb.E_NULL
    assert lb.lib().lowbit_attention_kv8_prefix_workspace(kv(), prefix(), batch(), 4, None) == lb.E_NULL
    assert call(hq=3) == lb.E_SHAPE and call(hq=0) == lb.E_SHAPE and call(hq=1 << 17, qs=1 << 30, os=1 << 30) == lb.E_SHAPE
    assert call(qs=255) == lb.E_SHAPE and call(os=255) == lb.E_SHAPE and call(qs=1 << 41) == lb.E_SHAPE
    for s in (float("inf"), float("nan"), 3e38):
        assert call(scale=s) == lb.E_UNSUPPORTED
    assert call(Q=A4) == lb.E_ALIGN and call(O=A4) == lb.E_ALIGN and call(qs=260) == lb.E_ALIGN
    assert call(lse=ctypes.c_void_p(0x10002)) == lb.E_ALIGN


def test_launches_that_do_not_fit():
    """Rows of the sequences and of the groups: both sides of what a launch holds."""
    n = ctypes.c_size_t()
    f = lb.lib().lowbit_attention_kv8_prefix_workspace

    def status(B, q, heads):
        # long rows in the place of many: nothing is read here
        c = kv(kv_heads=heads, n_pages=1 << 30)
        return f(c, prefix(n_groups=1, seq_starts=None, table_width=1 << 20, max_len=1 << 24),
                 batch(n_seqs=B, q_starts=0x80000, total_q=B * q, max_q=q, table_width=1 << 20, max_kv=1 << 24), heads, ctypes.byref(n))

    assert status(1 << 10, 1 << 10, 8) == lb.OK
    assert status(1 << 20, 1 << 10, 64) == lb.E_SHAPE
    assert status(1 << 20, 1 << 10, 4096) == lb.E_SHAPE


@pytest.mark.parametrize("D,H,G", [(64, 8, 4), (128, 8, 5), (256, 4, 6)])
def test_workspace_holds_for_smaller_calls(D, H, G):
    """Bytes for the plan of a call; none is negative or beyond what its rows and parts can take."""
    n = ctypes.c_size_t()
    f = lb.lib().lowbit_attention_kv8_prefix_workspace
    for B in (1, 2, 7, 64, 300, 2000):
        for q in (1, 3, 17, 130, 1000):
            for own in (1, 100, 5000):
                for L in (1, 1000, 100000):
                    c = kv(kv_heads=H, head_dim=D, page_tokens=64, n_pages=1 << 20)
                    p = prefix(n_groups=1, table_width=1 << 16, max_len=L, max_seqs=B)
                    b = batch(n_seqs=B, q_starts=0x80000, total_q=B * q, max_q=q, table_width=1 << 16, max_kv=own)
                    assert f(c, p, b, H * G, ctypes.byref(n)) == lb.OK
                    rows = B * q * H * G
                    # sums in parts only where the groups' tiles do not fill the chip (at most 768 tiles of 256 rows at once,
                    # four parts behind that), shares of attn_decode, counters
                    assert n.value <= (4 * rows + 4 * 2 * 768 * 256) * (D + 4) * 4 * 2 + (1 << 28)


def test_plain_form():
    """Behind a prefix of length 0 the plain form is attention over the own tokens; over all
    tokens without a mask it is that over both together."""
    g = np.random.default_rng(4)
    q, Kp, Vp, Ko, Vo = (g.standard_normal((n, h, 8)) for n, h in ((3, 4), (5, 2), (5, 2), (6, 2), (6, 2)))
    none = np.zeros((0, 2, 8))
    for causal in (True, False):
        a = R.attention_prefix(q, none, none, Ko, Vo, 3, 0.3, causal)
        b = M.attention(q, Ko, Vo, 3, 0.3, causal, 0)
        assert all(np.allclose(x, y) for x, y in zip(a, b))
    a = R.attention_prefix(q, Kp, Vp, Ko, Vo, 0, 0.3, False)
    b = M.attention(q, np.concatenate((Kp, Ko)), np.concatenate((Vp, Vo)), 0, 0.3, False, 0)
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])
    # causal: query i sees the prefix and i + 1 own tokens
    a = R.attention_prefix(q, Kp, Vp, Ko, Vo, 0, 0.3, True)
    b = M.attention(q[1:2], np.concatenate((Kp, Ko[:2])), np.concatenate((Vp, Vo[:2])), 0, 0.3, False, 0)
    assert np.allclose(a[0][1], b[0][0])
