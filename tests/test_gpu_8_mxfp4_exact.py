"""MXFP4 products whose sums are exact in fp32, bit for bit: operands are
whole numbers of a common step and small enough that every partial sum, in any
order, is a multiple of that step below 2^24 of it.  A sum held or joined in
fewer bits anywhere on the way shows."""
import pytest
import torch

from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu

TABLE = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def operand(rows, K, bytes_, g):
    """Random codes with the exponent bytes bytes_ [rows][K/32], packed on the GPU,
    and their values in 64 bits."""
    codes = torch.randint(0, 16, (rows, K), generator=g, device="cuda", dtype=torch.uint8)
    pc, ps = lb.pack_mxfp4((codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous(), bytes_)
    step = ((bytes_.long() + 1023 - 127) << 52).view(torch.float64)  # 2^(byte - 127) from its bits
    return pc, ps, TABLE.cuda()[codes.long()] * step.repeat_interleave(32, 1)


def spread(rows, K, lo, hi, g):
    return torch.randint(lo, hi + 1, (rows, K // 32), generator=g, device="cuda", dtype=torch.uint8)


# few rows, whole and split; small tiles, those that share compute units, large
# tiles; each with K whole and split; K that ends inside a group
SHAPES = [(1, 5120, 17408, False), (5, 640, 17408, False), (16, 48, 17408, False), (3, 5120, 5120, False),
          (40, 130, 17408, False), (300, 700, 17408, False), (50, 34800, 672, False), (64, 2560, 5120, False),
          (2001, 4003, 672, False), (900, 2200, 6176, False), (509, 15360, 5120, False),
          (1, 640, 17408, True), (20, 700, 17408, True), (32, 5120, 5120, True), (70, 100, 17408, True),
          (300, 700, 17408, True), (129, 260, 1184, True), (4001, 4003, 672, True), (392, 4290, 16000, True)]


@pytest.mark.parametrize("M,N,K,x4", SHAPES)
def test_sums_are_exact(M, N, K, x4):
    """|w| <= 12 in halves times |x| <= 8 whole, or times |x| <= 6 in halves: sums
    of 17408 are at most 1.7e6 in steps of 1/2, or 1.3e6 in steps of 1/4: below 2^23."""
    print(f"exact sums M={M} N={N} K={K} x4={x4}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    wc, ws, wv = operand(N, K, spread(N, K, 127, 128, g), g)
    if x4:
        x, xs, xv = operand(M, K, spread(M, K, 127, 127, g), g)
    else:
        xs, xv = None, torch.randint(-8, 9, (M, K), generator=g, device="cuda").double()
        x = xv.bfloat16()
    want = xv @ wv.t().contiguous()
    y = lb.gemm_mxfp4(M, N, K, wc, ws, x, x_scales=xs)
    assert torch.equal(y.double(), want), f"{int((y.double() != want).sum())} of {want.numel()} differ"
    # one rounding to bf16, to nearest even
    y = lb.gemm_mxfp4(M, N, K, wc, ws, x, x_scales=xs, y_dtype=lb.BF16)
    assert torch.equal(y, want.float().bfloat16())


@pytest.mark.parametrize("M,N,K", [(1, 40, 672), (16, 700, 1056), (20, 40, 160), (90, 200, 1056), (300, 600, 672),
                                   (2001, 4003, 672)])
@pytest.mark.parametrize("x4", [False, True])
def test_exponents_at_the_ends(M, N, K, x4):
    """The smallest and the largest powers of two, a row of W each.  With bf16 X,
    weights below 2^-126 may count as 0; everything else counts."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    for ends, other in (((0, 1, 2, 3), 60), ((249, 250, 251, 252), -60)):
        print(f"exponent bytes {ends} M={M} N={N} K={K} x4={x4}", flush=True)
        b = torch.tensor(ends, device="cuda", dtype=torch.uint8)[torch.arange(N, device="cuda") % 4]
        wc, ws, wv = operand(N, K, b[:, None].expand(N, K // 32).contiguous(), g)
        if x4:
            x, xs, xv = operand(M, K, spread(M, K, 127 + other, 127 + other, g), g)
        else:
            xs, xv = None, torch.randint(-8, 9, (M, K), generator=g, device="cuda").double() * 2.0 ** other
            x = xv.bfloat16()
        y = lb.gemm_mxfp4(M, N, K, wc, ws, x, x_scales=xs).double()
        want = xv @ wv.t().contiguous()
        ok = y == want
        if not x4:
            wv = torch.where(wv.abs() < 2.0 ** -126, torch.zeros_like(wv), wv)
            ok |= y == xv @ wv.t().contiguous()
        assert bool(ok.all()), (int((~ok).sum()), y[~ok][:4], want[~ok][:4])


@pytest.mark.parametrize("M,N,K", [(3, 16, 96), (20, 40, 160), (90, 200, 672), (300, 600, 672)])
def test_exponents_of_both_operands_at_the_ends(M, N, K):
    """MXFP4 by MXFP4, the smallest powers of two against the largest."""
    print(f"both ends M={M} N={N} K={K}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(M)
    for w, x in ((0, 254), (254, 0), (1, 253)):
        wc, ws, wv = operand(N, K, spread(N, K, w, w, g), g)
        xc, xs, xv = operand(M, K, spread(M, K, x, x, g), g)
        y = lb.gemm_mxfp4(M, N, K, wc, ws, xc, x_scales=xs)
        assert torch.equal(y.double(), xv @ wv.t().contiguous()), (w, x)


@pytest.mark.parametrize("M,N,K", [(3, 16, 96), (90, 200, 672), (300, 600, 672)])
def test_largest_exponents_with_bf16_x(M, N, K):
    """Bytes 253 and 254, codes whose values are below 2^128: counted exactly."""
    g = torch.Generator(device="cuda").manual_seed(M)
    for byte, top in ((253, 6), (254, 4)):  # magnitudes below 4, below 2
        print(f"byte {byte} M={M} N={N} K={K}", flush=True)
        codes = torch.randint(0, top, (N, K), generator=g, device="cuda", dtype=torch.uint8)
        codes |= torch.randint(0, 2, (N, K), generator=g, device="cuda", dtype=torch.uint8) << 3
        wc, ws = lb.pack_mxfp4((codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous(), spread(N, K, byte, byte, g))
        wv = TABLE.cuda()[codes.long()] * 2.0 ** (byte - 127)
        xv = torch.randint(-8, 9, (M, K), generator=g, device="cuda").double() * 2.0 ** -60
        y = lb.gemm_mxfp4(M, N, K, wc, ws, xv.bfloat16())
        assert torch.equal(y.double(), xv @ wv.t().contiguous())
