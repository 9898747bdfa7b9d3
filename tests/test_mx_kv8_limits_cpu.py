"""Sizes at the ends of what a launch holds (2^32 - 1 threads), on a machine
without a GPU: one more is refused with E_SHAPE.  The largest accepted ones
are shown by the check that comes after the sizes', a misaligned pointer."""
import ctypes

import pytest

from ultra_bit_dit_amd import lowbit as lb
from test_mx_kv8_cpu import A4, A16, batch, kv


@pytest.mark.parametrize("P,D,most", [(128, 256, 1 << 22), (64, 256, 1 << 23), (128, 128, 1 << 23)])
def test_append_workgroups(P, D, most):
    """1024 threads for pages of 32768 elements a head, 512 for 16384."""
    def call(H):
        c = kv(page_tokens=P, kv_heads=H, head_dim=D)
        b = batch(n_seqs=1 << 13, table_width=2, total_q=1 << 13, max_q=1, max_kv=2 * P, q_starts=0x70000)
        return lb.lib().lowbit_kv8_append(c, b, lb.BF16, A4, A16, H * D, H * D, None)

    H = most >> 13  # max_q = 1 touches one page
    assert call(H) == lb.E_SHAPE
    assert call(H - 1) == lb.E_ALIGN


def test_append_workgroups_of_small_pages():
    """The documented bound itself."""
    def call(n):
        c = kv(page_tokens=64, kv_heads=1 << 10, head_dim=128)
        b = batch(n_seqs=n, table_width=2, total_q=n, max_q=1, max_kv=64, q_starts=0x70000)
        return lb.lib().lowbit_kv8_append(c, b, lb.BF16, A4, A16, 1 << 17, 1 << 17, None)

    assert call(1 << 13) == lb.E_ALIGN
    assert call((1 << 13) + 1) == lb.E_SHAPE


def test_quantizer_rows():
    def call(rows, K):
        return lb.lib().lowbit_quantize_mxfp4(rows, K, lb.BF16, A4, K, A16, A16, None, None)

    for K in (32, 256):
        assert call(1 << 30, K) == lb.E_SHAPE
        assert call((1 << 30) - 63, K) == lb.E_SHAPE
        assert call((1 << 30) - 64, K) == lb.E_ALIGN
    assert call(1 << 29, 512) == lb.E_ALIGN


@pytest.mark.parametrize("x,most", [(lb.BF16, (1 << 30) - 128), (lb.MXFP4, 1 << 30)])
def test_product_tiles(x, most):
    """ceil(M/128) ceil(N/128) <= 2^23, with bf16 X (512 threads a tile of 128 rows) < 2^23."""
    L = lb.lib()
    n = ctypes.c_size_t()

    def call(M, N):
        size = L.lowbit_gemm_mxfp4_workspace(M, N, 32, x, ctypes.byref(n))
        run = L.lowbit_gemm_mxfp4(M, N, 32, A16, A16, x, A4, 32, A16, lb.F32, A16, None)
        assert (size, run) in ((lb.OK, lb.E_ALIGN), (lb.E_SHAPE, lb.E_SHAPE)), (M, N, size, run)
        return size

    for M, N in ((most + 1, 16), (most + 1, 128), (1 << 30, 129), (1 << 23, (1 << 14) + 1), (1 << 10, 1 << 27)):
        assert call(M, N) == lb.E_SHAPE
    for M, N in ((most, 16), (most, 128), (1 << 29, 16), ((1 << 29) + 1, 100), (128, 1 << 26), (1 << 20, 1 << 16)):
        assert call(M, N) == lb.OK


@pytest.mark.parametrize("scale,status", [(2.35e38, lb.E_ALIGN), (2.37e38, lb.E_UNSUPPORTED), (-2.37e38, lb.E_UNSUPPORTED),
                                          (3.4e38, lb.E_UNSUPPORTED)])
def test_scale_whose_base_2_form_is_infinite(scale, status):
    """scale log2(e) has to be finite, as 0 times it has to be 0."""
    f = lb.lib().lowbit_attention_kv8
    assert f(kv(), batch(), 4, A4, 256, scale, 1, 0, A16, 256, None, None) == status
