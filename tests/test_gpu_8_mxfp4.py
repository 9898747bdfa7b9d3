"""MXFP4 quantizer, packer and products on the GPU against the plain 64-bit
forms: codes, scales and values bit for bit, products within the bound of
their fp32 sums."""
import numpy as np
import pytest
import torch

import mx_ref as R
from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu


def values(rows, K, seed, spread=3.0):
    g = np.random.default_rng(seed)
    return (g.standard_normal((rows, K)) * np.exp2(np.rint(g.standard_normal((rows, 1)) * spread))).astype(np.float32)


def device(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def check_quantized(X, x, pc, ps, vals):
    codes, b = R.mx_quantize(X)
    wc, ws = R.mx_pack(codes, b)
    assert np.array_equal(ps.cpu().numpy(), ws), "scales"
    assert np.array_equal(pc.cpu().numpy(), wc), "codes"
    assert np.array_equal(f64(vals), R.mx_values(codes, b), equal_nan=True), "values"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (17, 160), (33, 512), (16, 544), (40, 1056), (2, 5120)])
def test_quantize(rows, K, dtype):
    print(f"quantize rows={rows} K={K} {dtype}", flush=True)
    x = device(values(rows, K, rows + K), dtype)
    pc, ps, v = lb.quantize_mxfp4(x, values=True)
    check_quantized(f64(x), x, pc, ps, v)
    # the same without the values, from rows that lie in a wider matrix
    wide = torch.full((rows, K + 64), float("nan"), dtype=dtype, device="cuda")
    wide[:, 32:32 + K] = x
    pc2, ps2 = lb.quantize_mxfp4(wide[:, 32:32 + K])
    assert torch.equal(pc, pc2) and torch.equal(ps, ps2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_edges(dtype):
    """Midpoints at many exponents, zeros of both signs, the smallest and the largest numbers, infinities and NaN."""
    print(f"quantize edges {dtype}", flush=True)
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.5, 7.5, 4.0, 6.0, -0.25, -5.0, 0.0, -0.0, 1.0])
    rows = [np.tile(mid, 2) * np.ldexp(1.0, e) for e in (-120, -20, 0, 3, 100)]
    rows += [np.zeros(32), -np.zeros(32), np.full(32, 2.0 ** -133), np.linspace(1, 32, 32) * 2.0 ** -133,
             np.full(32, 3.3e38), np.full(32, 2.0 ** -126), np.full(32, 2.0 ** -125), np.full(32, 1.75 * 2.0 ** -124)]
    for bad in (np.inf, -np.inf, np.nan):
        r = np.ones(32)
        r[7] = bad
        rows.append(r)
    X = np.stack(rows).astype(np.float32)
    X = np.concatenate([X, X[::-1]], 1)  # two blocks a row: a bad one leaves its neighbour alone
    x = device(X, dtype)
    pc, ps, v = lb.quantize_mxfp4(x, values=True)
    check_quantized(f64(x), x, pc, ps, v)


@pytest.mark.parametrize("rows,K", [(1, 32), (17, 160), (35, 672), (16, 2048)])
def test_pack(rows, K):
    print(f"pack rows={rows} K={K}", flush=True)
    g = np.random.default_rng(rows * K)
    codes = g.integers(0, 16, (rows, K), dtype=np.uint8)
    b = g.integers(0, 256, (rows, K // 32), dtype=np.uint8)
    rm = torch.from_numpy(codes[:, 0::2] | (codes[:, 1::2] << 4)).cuda()
    pc, ps = lb.pack_mxfp4(rm, torch.from_numpy(b).cuda())
    wc, ws = R.mx_pack(codes, b)
    assert np.array_equal(pc.cpu().numpy(), wc) and np.array_equal(ps.cpu().numpy(), ws)


def product_case(M, N, K, seed, x4):
    W = device(values(N, K, seed) * 0.05, torch.float32)
    wc, ws, wv = lb.quantize_mxfp4(W, values=True)
    x = device(values(M, K, seed + 1), torch.bfloat16)
    if x4:
        xc, xs, xv = lb.quantize_mxfp4(x, values=True)
        return wc, ws, xc, xs, f64(wv), f64(xv)
    return wc, ws, x, None, f64(wv), f64(x)


def check_product(y, wv, xv, K, bf16_out, what):
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    err, tol = np.abs(f64(y) - ref), R.product_tolerance(mag, ref, K, bf16_out)
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first {i}: {f64(y)[i]} for {ref[i]} +- {tol[i]}")


SHAPES = [(1, 1, 32), (1, 16, 128), (1, 37, 96), (2, 256, 1024), (5, 100, 672), (15, 33, 544), (16, 64, 512), (17, 48, 160),
          (33, 130, 1056), (64, 257, 640), (65, 96, 2080), (100, 520, 384), (129, 260, 1184), (200, 272, 128),
          (257, 129, 2592), (300, 700, 1024), (513, 515, 544), (1, 5120, 17408), (5, 640, 17408), (600, 1056, 5120)]


@pytest.mark.parametrize("x4", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, x4):
    print(f"product M={M} N={N} K={K} x4={x4}", flush=True)
    wc, ws, x, xs, wv, xv = product_case(M, N, K, 7 * M + N + K, x4)
    for yd in (lb.F32, lb.BF16):
        Y = torch.full((M + 1, N), float("nan"), device="cuda", dtype=lb._ytorch(yd))
        y = lb.gemm_mxfp4(M, N, K, wc, ws, x, x_scales=xs, y_dtype=yd, Y=Y[:M])
        check_product(y, wv, xv, K, yd == lb.BF16, f"M={M} N={N} K={K}")
        assert torch.isnan(Y[M]).all(), "the row behind the last one"
        y2 = lb.gemm_mxfp4(M, N, K, wc, ws, x, x_scales=xs, y_dtype=yd)
        assert torch.equal(y, y2), "two runs differ"


@pytest.mark.parametrize("M,N,K", [(17, 16, 32), (25, 300, 17408), (31, 33, 544), (32, 700, 5120), (33, 300, 17408)])
def test_product_of_two_row_blocks(M, N, K):
    """17 to 32 rows of MXFP4 X, and one more; K whole and split."""
    test_product(M, N, K, True)


@pytest.mark.parametrize("K", [96, 672])
def test_product_of_more_tiles_than_compute_units(K):
    """Tiles of 64 rows that share compute units."""
    M, N = 50, 34800
    print(f"product {M}x{N}x{K}", flush=True)
    wc, ws, x, _, wv, xv = product_case(M, N, K, 21, False)
    for yd in (lb.F32, lb.BF16):
        y = lb.gemm_mxfp4(M, N, K, wc, ws, x, y_dtype=yd)
        check_product(y, wv, xv, K, yd == lb.BF16, f"y {yd}")


@pytest.mark.parametrize("M", [1, 7, 80, 300])
def test_product_strided_x(M):
    """Rows of X inside a wider matrix whose other elements are NaN; K ends inside a group."""
    N, K = 144, 928
    print(f"strided product M={M}", flush=True)
    wc, ws, x, _, wv, xv = product_case(M, N, K, 91 + M, False)
    wide = torch.full((M, K + 40), float("nan"), device="cuda", dtype=torch.bfloat16)
    wide[:, 8:8 + K] = x
    y = lb.gemm_mxfp4(M, N, K, wc, ws, wide[:, 8:8 + K])
    check_product(y, wv, xv, K, False, f"strided M={M}")


@pytest.mark.parametrize("M,N", [(3, 40), (90, 200), (300, 600)])
@pytest.mark.parametrize("x4", [False, True])
def test_product_nan_and_infinity_stay_in_their_rows(M, N, x4):
    K = 320
    print(f"NaN rows M={M} N={N} x4={x4}", flush=True)
    wc, ws, x, xs, wv, xv = product_case(M, N, K, 5 * M, x4)
    W = torch.from_numpy(wv).float()
    W[N - 2, 100] = float("nan")
    wc, ws, wv = lb.quantize_mxfp4(W.cuda(), values=True)
    wv = f64(wv)
    X = torch.from_numpy(xv).float()
    X[1, 5] = float("inf")
    if x4:
        x, xs, xv = lb.quantize_mxfp4(X.cuda(), values=True)
        xv = f64(xv)
    else:
        x, xv = X.cuda().bfloat16(), None
    y = f64(lb.gemm_mxfp4(M, N, K, wc, ws, x, x_scales=xs))
    assert np.isnan(y[:, N - 2]).all() and not np.isfinite(y[1]).any()
    keep_m, keep_n = np.arange(M) != 1, np.arange(N) != N - 2
    assert np.isfinite(y[keep_m][:, keep_n]).all()


@pytest.mark.parametrize("M,x4", [(1, False), (512, False), (512, True)])
def test_product_layer_shape_sampled(M, x4):
    """The fused gate/up shape, sampled columns against 64 bits."""
    N, K = 34816, 5120
    print(f"layer product M={M} x4={x4}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    W = torch.randn(N, K, device="cuda", generator=g) * 0.02
    wc, ws, wv = lb.quantize_mxfp4(W, values=True)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    xa, xs, xv = x, None, f64(x)
    if x4:
        xa, xs, xv = lb.quantize_mxfp4(x, values=True)
        xv = f64(xv)
    y = lb.gemm_mxfp4(M, N, K, wc, ws, xa, x_scales=xs)
    cols = np.r_[0:40, np.random.default_rng(3).choice(N, 60, replace=False), N - 40:N]
    at = torch.from_numpy(cols).cuda()
    check_product(y[:, at], f64(wv[at]), xv, K, False, f"layer M={M}")


@pytest.mark.parametrize("M,N,K,x4", [(2001, 4003, 672, False), (900, 2200, 6176, False), (4001, 4003, 672, True),
                                      (392, 4290, 16000, True)])
def test_product_of_large_tiles_sampled(M, N, K, x4):
    """Sizes with odd ends that take the large tiles, whole K and split; sampled columns against 64 bits."""
    print(f"large tiles M={M} N={N} K={K} x4={x4}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(M + N)
    wc, ws, wv = lb.quantize_mxfp4(torch.randn(N, K, device="cuda", generator=g) * 0.02, values=True)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    xa, xs, xv = x, None, f64(x)
    if x4:
        xa, xs, xv = lb.quantize_mxfp4(x, values=True)
        xv = f64(xv)
    cols = np.unique(np.r_[0:33, np.random.default_rng(3).choice(N, 60, replace=False), N - 40:N])
    at = torch.from_numpy(cols).cuda()
    for yd in (lb.F32, lb.BF16):
        y = lb.gemm_mxfp4(M, N, K, wc, ws, xa, x_scales=xs, y_dtype=yd)
        check_product(y[:, at], f64(wv[at]), xv, K, yd == lb.BF16, f"large tiles M={M}")
        assert bool(torch.isfinite(y.float()).all())


def test_stream_and_graph():
    """Quantizing and multiplying on another stream, then captured and replayed
    on new inputs with other work between the replays."""
    M, N, K = 48, 320, 672
    print("graph", flush=True)
    wc, ws, x, _, wv, _ = product_case(M, N, K, 3, False)
    s = torch.cuda.Stream()
    pc, ps = lb.empty_mxfp4(M, K)
    y4 = torch.empty(M, N, device="cuda")
    y16 = torch.empty(M, N, device="cuda")

    def step():
        lb.quantize_mxfp4(x, pcodes=pc, pscales=ps)
        lb.gemm_mxfp4(M, N, K, wc, ws, pc, x_scales=ps, Y=y4)
        lb.gemm_mxfp4(M, N, K, wc, ws, x, Y=y16)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in range(3):
        x.copy_(device(values(M, K, 40 + i), torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        _, _, xv = lb.quantize_mxfp4(x, values=True)
        check_product(y4, wv, f64(xv), K, False, f"replay {i}")
        check_product(y16, wv, f64(x), K, False, f"replay {i}")


def test_split_products_in_a_graph():
    """Products whose K is split over workgroups, captured with a reserved
    workspace and replayed, with eager ones on the stream between."""
    K, cases = 17408, ((3, 48, False), (40, 130, False), (70, 100, True))
    print("graph of split products", flush=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    work = []
    for M, N, x4 in cases:
        size = lb.gemm_mxfp4_workspace(M, N, K, lb.MXFP4 if x4 else lb.BF16)
        assert size > 4 * M * N  # more than one sum for each output
        lb.reserve_workspace(size, s)
        wc, ws, x, _, wv, _ = product_case(M, N, K, 7, False)
        work.append((M, N, x4, wc, ws, x, wv, torch.empty(M, N, device="cuda"), *lb.empty_mxfp4(M, K)))

    def step():
        for M, N, x4, wc, ws, x, _, y, pc, ps in work:
            if x4:
                lb.quantize_mxfp4(x, pcodes=pc, pscales=ps)
                lb.gemm_mxfp4(M, N, K, wc, ws, pc, x_scales=ps, Y=y)
            else:
                lb.gemm_mxfp4(M, N, K, wc, ws, x, Y=y)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in range(3):
        for M, *_, x, _, _, _, _ in work:
            x.copy_(device(values(M, K, 60 + i), torch.bfloat16))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
            first = [w[7].clone() for w in work]
            step()
        torch.cuda.synchronize()
        for (M, N, x4, _, _, x, wv, y, _, _), g in zip(work, first):
            assert torch.equal(y, g)
            xv = lb.quantize_mxfp4(x, values=True)[2] if x4 else x
            check_product(g, wv, f64(xv), K, False, f"replay {i}")


def test_capture_without_a_workspace_is_refused():
    """A stream that is being captured cannot grow its workspace: E_NOMEM, and nothing is recorded."""
    M, N, K = 40, 130, 17408
    print("capture without workspace", flush=True)
    wc, ws, x, _, _, _ = product_case(M, N, K, 8, False)
    y = torch.full((M, N), 7.0, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    lb.release_workspaces()  # the stream may have been another test's
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y.add_(1.0)
        with pytest.raises(lb.LowbitError) as e:
            lb.gemm_mxfp4(M, N, K, wc, ws, x, Y=y)
        assert e.value.status == lb.E_NOMEM
    graph.replay()
    torch.cuda.synchronize()
    assert torch.all(y == 8.0)


@pytest.mark.parametrize("M,x4", [(1, False), (3, True), (20, True), (40, False), (40, True)])
def test_weights_beyond_32_bits(M, x4):
    """Packed codes of more than 4 GiB: rows from both ends against 64 bits."""
    N, K = 1_100_005, 8192
    print(f"large weights M={M} x4={x4}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(9)
    wc, ws = lb.empty_mxfp4(N, K)
    assert wc.numel() > 1 << 32
    wc.random_(0, 256, generator=g)
    ws.random_(118, 130, generator=g)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    xa, xs, xv = x, None, f64(x)
    if x4:
        xa, xs, xv = lb.quantize_mxfp4(x, values=True)
        xv = f64(xv)
    y = lb.gemm_mxfp4(M, N, K, wc, ws, xa, x_scales=xs)
    rows = np.r_[0:3, 65535:65540, N - 40:N]
    codes = wc.view(-1, K // 128, 4, 16, 16)
    scales = ws.view(-1, K // 512, 4, 16, 4)
    wv = np.empty((len(rows), K))
    table = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])
    for i, n in enumerate(rows):
        c = codes[n // 16, :, :, n % 16].cpu().numpy()                       # [group][q][16]
        e = scales[n // 16, :, :, n % 16].permute(0, 2, 1).cpu().numpy()     # [quad][group % 4][q]
        v = table[np.stack([c & 15, c >> 4], -1).reshape(-1, 4, 32)]
        wv[i] = (v * np.exp2(e.reshape(-1, 4, 1).astype(float) - 127)).reshape(-1)
    check_product(y[:, torch.from_numpy(rows).cuda()], wv, xv, K, False, f"large weights M={M}")


def test_quantize_beyond_32_bits():
    """More than 2^32 values, and codes of more than 4 GiB: the last rows like those rows alone."""
    rows, K = (1 << 27) + 77, 32
    print("large quantization", flush=True)
    X = torch.empty(rows, K, device="cuda", dtype=torch.bfloat16)
    X.fill_(1.0)
    tail = torch.randn(93, K, device="cuda").bfloat16()
    X[-93:] = tail
    pc, ps, vals = lb.quantize_mxfp4(X, values=True)
    # the last 93 rows begin a row-block
    assert (rows - 93) % 16 == 0 and pc.numel() > 1 << 32
    c2, s2, v2 = lb.quantize_mxfp4(tail, values=True)
    assert torch.equal(pc[-c2.numel():], c2) and torch.equal(ps[-s2.numel():], s2) and torch.equal(vals[-93:], v2)
    assert bool((vals[:1000] == 1).all()) and bool((vals[-1093:-93] == 1).all())
