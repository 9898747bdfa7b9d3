"""MXFP4 and 8-bit cache entry points on a machine without a GPU: sizes,
refusals (every check runs before any HIP call), and the plain forms the GPU
tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import mx_ref as R
from ultra_bit_dit_amd import lowbit as lb

A16, A4, A1 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004), ctypes.c_void_p(0x10001)


@pytest.mark.parametrize("rows,K", [(1, 32), (16, 128), (17, 160), (5120, 5120), (34816, 5120), (3, 17408)])
def test_mxfp4_bytes(rows, K):
    cb, sb = lb.mxfp4_bytes(rows, K)
    assert (cb, sb) == lb._mx_sizes(rows, K)
    pc, ps = R.mx_pack(np.zeros((rows, K), np.uint8), np.zeros((rows, K // 32), np.uint8)) if rows < 100 else (None, None)
    if pc is not None:
        assert (cb, sb) == (pc.size, ps.size)
    if rows % 16 == 0 and K % 512 == 0:
        assert 8 * (cb + sb) == 4.25 * rows * K


def test_mxfp4_refusals():
    L = lb.lib()
    cb, sb = ctypes.c_size_t(), ctypes.c_size_t()
    f = L.lowbit_mxfp4_bytes
    assert f(1, 32, None, ctypes.byref(sb)) == lb.E_NULL
    for rows, K in ((0, 32), (1, 0), (1, 48), (1, -32), (1 << 31, 32), (1 << 30, 1 << 10), (1, 1 << 31)):
        assert f(rows, K, ctypes.byref(cb), ctypes.byref(sb)) == lb.E_SHAPE
    p = L.lowbit_pack_mxfp4
    assert p(1, 32, None, A16, A16, A16, None) == lb.E_NULL
    assert p(1, 40, A16, A16, A16, A16, None) == lb.E_SHAPE
    assert p(1, 32, A4, A16, A16, A16, None) == lb.E_ALIGN
    q = L.lowbit_quantize_mxfp4
    assert q(1, 32, lb.BF16, None, 32, A16, A16, None, None) == lb.E_NULL
    assert q(1, 32, lb.I8, A16, 32, A16, A16, None, None) == lb.E_UNSUPPORTED
    assert q(1, 32, lb.MXFP4, A16, 32, A16, A16, None, None) == lb.E_UNSUPPORTED
    assert q(1, 33, lb.BF16, A16, 64, A16, A16, None, None) == lb.E_SHAPE
    assert q(1, 32, lb.BF16, A16, 31, A16, A16, None, None) == lb.E_SHAPE
    assert q(2, 32, lb.BF16, A16, 36, A16, A16, None, None) == lb.E_ALIGN
    assert q(2, 32, lb.F32, A16, 34, A16, A16, None, None) == lb.E_ALIGN
    assert q(1, 32, lb.BF16, A4, 32, A16, A16, None, None) == lb.E_ALIGN
    assert q(1, 32, lb.BF16, A16, 32, A16, A16, A4, None) == lb.E_ALIGN
    g = L.lowbit_gemm_mxfp4
    assert g(1, 1, 32, A16, None, lb.BF16, A16, 32, None, lb.F32, A16, None) == lb.E_NULL
    assert g(1, 1, 32, A16, A16, lb.MXFP4, A16, 0, None, lb.F32, A16, None) == lb.E_NULL
    assert g(1, 1, 32, A16, A16, lb.F32, A16, 32, None, lb.F32, A16, None) == lb.E_UNSUPPORTED
    assert g(1, 1, 32, A16, A16, lb.BF16, A16, 32, None, lb.I32, A16, None) == lb.E_UNSUPPORTED
    assert g(0, 1, 32, A16, A16, lb.BF16, A16, 32, None, lb.F32, A16, None) == lb.E_SHAPE
    assert g(1, 1, 30, A16, A16, lb.BF16, A16, 32, None, lb.F32, A16, None) == lb.E_SHAPE
    assert g(1 << 24, 1 << 24, 32, A16, A16, lb.BF16, A16, 32, None, lb.F32, A16, None) == lb.E_SHAPE
    assert g(1, 1, 64, A16, A16, lb.BF16, A16, 32, None, lb.F32, A16, None) == lb.E_SHAPE
    assert g(2, 1, 32, A16, A16, lb.BF16, A16, 36, None, lb.F32, A16, None) == lb.E_ALIGN
    assert g(1, 1, 32, A16, A16, lb.BF16, A16, 32, None, lb.F32, A4, None) == lb.E_ALIGN
    assert g(1, 1, 32, A16, A16, lb.MXFP4, A16, 0, A4, lb.F32, A16, None) == lb.E_ALIGN
    # the group-scaled formats' entry points do not take the new type
    assert L.lowbit_gemm(1, 1, 16, 128, A16, A16, lb.MXFP4, A16, None, lb.F32, A16, None) == lb.E_UNSUPPORTED


def test_product_workspace():
    """Host-only: its refusals, and that K is split only where tiles are few."""
    L = lb.lib()
    n = ctypes.c_size_t(5)
    f = L.lowbit_gemm_mxfp4_workspace
    assert f(1, 16, 32, lb.BF16, None) == lb.E_NULL
    for bad in ((0, 16, 32), (1, 0, 32), (1, 16, 0), (1, 16, 48), (1, (1 << 26) + 1, 32), (1 << 30, 1 << 20, 32)):
        n.value = 5
        assert f(*bad, lb.BF16, ctypes.byref(n)) == lb.E_SHAPE and n.value == 0
    assert f(1, 16, 32, lb.F32, ctypes.byref(n)) == lb.E_UNSUPPORTED
    assert lb.gemm_mxfp4_workspace(40, 130, 17408, lb.BF16) > 0
    assert lb.gemm_mxfp4_workspace(4096, 16384, 5120, lb.BF16) == 0


def kv(**over):
    c = dict(n_pages=4, page_tokens=16, kv_heads=2, head_dim=64, k_codes=0x10000, v_codes=0x20000, k_scales=0x30000,
             v_scales=0x40000)
    c.update(over)
    return lb.Kv8(*[c[f[0]] for f in lb.Kv8._fields_])


def batch(**over):
    b = dict(n_seqs=2, page_table=0x50000, table_width=2, kv_lens=0x60000, q_starts=None, total_q=2, max_q=1, max_kv=32,
             bad_pages=None)
    b.update(over)
    return lb.Kv8Batch(*[b[f[0]] for f in lb.Kv8Batch._fields_])


BAD = [
    (dict(k_codes=None), {}, lb.E_NULL), (dict(v_scales=None), {}, lb.E_NULL), ({}, dict(page_table=None), lb.E_NULL),
    ({}, dict(kv_lens=None), lb.E_NULL), (dict(page_tokens=8), {}, lb.E_UNSUPPORTED),
    (dict(page_tokens=48), {}, lb.E_UNSUPPORTED), (dict(page_tokens=256), {}, lb.E_UNSUPPORTED),
    (dict(head_dim=96), {}, lb.E_UNSUPPORTED), (dict(kv_heads=0), {}, lb.E_SHAPE), (dict(n_pages=0), {}, lb.E_SHAPE),
    (dict(n_pages=1 << 31), {}, lb.E_SHAPE), ({}, dict(n_seqs=0), lb.E_SHAPE), ({}, dict(table_width=0), lb.E_SHAPE),
    ({}, dict(total_q=0), lb.E_SHAPE), ({}, dict(max_q=0), lb.E_SHAPE), ({}, dict(max_q=3), lb.E_SHAPE),
    ({}, dict(total_q=3), lb.E_SHAPE),  # without q_starts every sequence has max_q rows
    ({}, dict(max_kv=0), lb.E_SHAPE), ({}, dict(max_kv=33), lb.E_SHAPE),  # more than the table holds
    (dict(k_codes=0x10004), {}, lb.E_ALIGN), ({}, dict(kv_lens=0x60001), lb.E_ALIGN),
    ({}, dict(q_starts=0x70002), lb.E_ALIGN), ({}, dict(bad_pages=0x70002), lb.E_ALIGN),
]


@pytest.mark.parametrize("c,b,status", BAD)
def test_kv8_refusals(c, b, status):
    L = lb.lib()
    assert L.lowbit_kv8_append(kv(**c), batch(**b), lb.BF16, A16, A16, 128, 128, None) == status
    assert L.lowbit_attention_kv8(kv(**c), batch(**b), 4, A16, 256, 1.0, 1, 0, A16, 256, None, None) == status
    n = ctypes.c_size_t(5)
    assert L.lowbit_attention_kv8_workspace(kv(**c), batch(**b), 4, ctypes.byref(n)) == status and n.value == 0


def test_append_and_attention_refusals():
    L = lb.lib()
    f = L.lowbit_kv8_append
    assert f(None, batch(), lb.BF16, A16, A16, 128, 128, None) == lb.E_NULL
    assert f(kv(), batch(), lb.BF16, A16, None, 128, 128, None) == lb.E_NULL
    assert f(kv(), batch(), lb.I8, A16, A16, 128, 128, None) == lb.E_UNSUPPORTED
    assert f(kv(), batch(), lb.BF16, A16, A16, 127, 128, None) == lb.E_SHAPE
    assert f(kv(), batch(), lb.BF16, A16, A16, 132, 128, None) == lb.E_ALIGN
    assert f(kv(), batch(), lb.F32, A16, A16, 130, 128, None) == lb.E_ALIGN
    assert f(kv(), batch(), lb.BF16, A4, A16, 128, 128, None) == lb.E_ALIGN
    g = L.lowbit_attention_kv8
    inf, nan = float("inf"), float("nan")
    assert g(kv(), batch(), 4, None, 256, 1.0, 1, 0, A16, 256, None, None) == lb.E_NULL
    for heads in (0, 3, -2):
        assert g(kv(), batch(), heads, A16, 256, 1.0, 1, 0, A16, 256, None, None) == lb.E_SHAPE
    assert g(kv(), batch(), 4, A16, 255, 1.0, 1, 0, A16, 256, None, None) == lb.E_SHAPE
    assert g(kv(), batch(), 4, A16, 256, 1.0, 1, -1, A16, 256, None, None) == lb.E_SHAPE
    for scale in (inf, -inf, nan):
        assert g(kv(), batch(), 4, A16, 256, scale, 1, 0, A16, 256, None, None) == lb.E_UNSUPPORTED
    assert g(kv(), batch(), 4, A16, 260, 1.0, 1, 0, A16, 256, None, None) == lb.E_ALIGN
    assert g(kv(), batch(), 4, A16, 256, 1.0, 1, 0, A16, 256, A1, None) == lb.E_ALIGN
    n = ctypes.c_size_t()
    assert L.lowbit_attention_kv8_workspace(kv(), batch(), 4, None) == lb.E_NULL
    assert L.lowbit_attention_kv8_workspace(kv(), batch(), 4, ctypes.byref(n)) == lb.OK and n.value > 0


def test_attention_sizes_beyond_a_grid():
    """Numbers of workgroups that 32 bits do not hold are refused, not cut."""
    L = lb.lib()
    n = ctypes.c_size_t(5)
    many = dict(n_seqs=1 << 20, total_q=1 << 29, max_q=1 << 9, q_starts=0x70000)
    for heads in (4096, 8192):
        c, b = kv(kv_heads=4096), batch(**many)
        assert L.lowbit_attention_kv8_workspace(c, b, heads, ctypes.byref(n)) == lb.E_SHAPE and n.value == 0
        n.value = 5
        row = heads * 64
        assert L.lowbit_attention_kv8(c, b, heads, A16, row, 1.0, 1, 0, A16, row, None, None) == lb.E_SHAPE
    b = batch(n_seqs=1, total_q=1 << 30, max_q=1 << 30, q_starts=0x70000)
    assert L.lowbit_attention_kv8_workspace(kv(), b, 8, ctypes.byref(n)) == lb.E_SHAPE


def test_binding_checks_tensors():
    """The binding refuses wrong shapes, types and layouts before it looks for a device."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lb.quantize_mxfp4(x.t())
    with pytest.raises(lb.LowbitError):
        lb.quantize_mxfp4(x[:, :40])
    c, s = (torch.zeros(n, dtype=torch.uint8) for n in lb.mxfp4_bytes(4, 64))
    with pytest.raises(ValueError):
        lb.gemm_mxfp4(1, 20, 64, c, s, x[:1])
    with pytest.raises(ValueError):
        lb.gemm_mxfp4(1, 4, 64, c, s, x[:1].float())
    with pytest.raises(ValueError):
        lb.gemm_mxfp4(3, 4, 64, c, s, x)
    cache = lb.empty_kv8(3, 16, 2, 64, device="cpu")
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for bad in (dict(K=k[:, :1]), dict(K=k[..., :32]), dict(V=k.float()), dict(kv_lens=lens.long()),
                dict(page_table=table[0]), dict(q_starts=lens)):
        a = dict(cache=cache, page_table=table, kv_lens=lens, K=k, V=k)
        a.update(bad)
        with pytest.raises(ValueError):
            lb.kv8_append(**a)
    with pytest.raises(ValueError):
        lb.attention_kv8(k.float(), cache, table, lens)
    with pytest.raises(ValueError):
        lb.attention_kv8(k, (cache[0], cache[0], cache[2], cache[3]), table, lens)


def test_plain_forms():
    # e2m1: every midpoint goes to the even code
    x = np.zeros((1, 32))
    x[0, :10] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.75, 4.0]
    codes, b = R.mx_quantize(x)
    assert b[0, 0] == 127 and codes[0, :10].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 10, 6]
    # e4m3: the table's numbers are themselves, midpoints go to the even mantissa
    fin = R.E4M3[np.isfinite(R.E4M3)]
    assert np.array_equal(R.e4m3_nearest(fin), fin)
    assert R.e4m3_nearest(17.0) == 16 and R.e4m3_nearest(19.0) == 20 and R.e4m3_nearest(1e9) == 448
    assert R.e4m3_nearest(2.0 ** -10) == 0 and R.e4m3_nearest(3 * 2.0 ** -10) == 2.0 ** -8
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, R.E4M3, equal_nan=True)
    assert R.page_exponent(448.0) == 0 and R.page_exponent(449.0) == 1 and R.page_exponent(0.0) == -127
    # attention: equal scores average the values; a row that sees nothing is 0
    K, V = np.zeros((3, 1, 64)), np.arange(3 * 64, dtype=float).reshape(3, 1, 64)
    O, lse, _, _ = R.attention(np.ones((2, 1, 64)), K, V, -1, 1.0, True, 0)
    assert np.all(O[0] == 0) and lse[0, 0] == -np.inf and np.array_equal(O[1, 0], V[0, 0]) and lse[1, 0] == 0
