"""Head norms with rotation on the GPU against the plain 64-bit form."""
import numpy as np
import pytest
import torch

import serve_ref as R
from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


def freqs_of(n, base=1e4):
    return torch.tensor([base ** (-i / max(n, 1)) for i in range(n)], dtype=torch.float64, device="cuda")


def check(x, y, w, eps, pos, freqs, axis, adjacent, what):
    """Output y of input x, both [T][heads][D] tensors."""
    x64 = x.double().cpu().numpy()
    pos = pos.cpu().numpy().reshape(-1, x.shape[0])
    ref, mag, turn = R.rotate(x64, None if w is None else w.double().cpu().numpy(), eps, pos,
                              [] if freqs is None else freqs.cpu().numpy(), None if axis is None else axis.cpu().numpy(), adjacent)
    tol = R.rotate_tolerance(ref, mag, turn, x.shape[2], y.dtype == BF)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= tol), f"{what}: {(err / tol).max()} of the bound at {np.argmax(err / tol)}"


def data(T, heads, D, dtype, seed, spread=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, heads, D), device="cuda", generator=g)
    if spread:
        x = x * torch.exp2(torch.randint(-8, 9, (T, heads, 1), device="cuda", generator=g).float())
    return x.to(dtype)


SHAPES = [  # D, pairs
    (8, 4), (8, 0), (16, 8), (24, 12), (64, 32), (64, 8), (72, 36), (80, 40), (80, 20), (96, 48), (128, 64), (128, 32), (128, 4),
    (192, 96), (248, 124), (256, 128), (256, 32), (256, 0)]


@pytest.mark.parametrize("D,pairs", SHAPES)
@pytest.mark.parametrize("adjacent", [False, True])
def test_sizes(D, pairs, adjacent):
    """Every width of head, in all four pairs of types, one token and more, odd numbers of heads."""
    for i, (T, Hq, Hk) in enumerate(((1, 5, 1), (7, 3, 2), (67, 1, 1))):
        for xd, yd in ((BF, BF), (BF, F), (F, BF), (F, F)):
            print(f"rope D={D} pairs={pairs} {adjacent} {T}x{Hq}+{Hk} {xd} {yd}", flush=True)
            q, k = data(T, Hq, D, xd, 3 + i), data(T, Hk, D, xd, 5 + i)
            w, v = (torch.rand(D, device="cuda") * 2 - 0.5 for _ in range(2))
            pos = torch.randint(-5000, 200000, (T,), device="cuda", dtype=torch.int32)
            f = freqs_of(pairs) if pairs else None
            qo, ko = lb.qk_norm_rope(q, k, pos, f, w, v, eps=1e-6, adjacent=adjacent, y_dtype=lb.BF16 if yd == BF else lb.F32)
            assert qo.dtype == yd and qo.shape == q.shape and ko.shape == k.shape
            check(q, qo, w, float(np.float32(1e-6)), pos, f, None, adjacent, "q")
            check(k, ko, v, float(np.float32(1e-6)), pos, f, None, adjacent, "k")


@pytest.mark.parametrize("heads", [(1, 0), (8, 8), (40, 8), (64, 1), (33, 11)])
@pytest.mark.parametrize("T", [1, 2, 300, 9000])
def test_heads_and_tokens(heads, T):
    """Few tokens spread over more waves than heads fill, many tokens; no norm for one side."""
    Hq, Hk = heads
    D = 64 if T == 9000 else 128
    print(f"rope heads {heads} T={T}", flush=True)
    q, k = data(T, Hq, D, BF, 1), data(T, Hk, D, BF, 2) if Hk else None
    w = torch.rand(D, device="cuda") + 0.5
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 3
    f = freqs_of(D // 2, 1e6)
    qo, ko = lb.qk_norm_rope(q, k, pos, f, w, None)
    s = slice(None) if T < 1000 else slice(T - 40, T)
    check(q[s], qo[s], w, float(np.float32(1e-6)), pos[s], f, None, False, "q")
    if Hk:
        check(k[s], ko[s], None, 0.0, pos[s], f, None, False, "k")
    else:
        assert ko is None


def test_axes_strides_and_in_place():
    """Three axes in any order over the pairs, an axis outside the range (not rotated);
    queries and keys inside a fused projection's output, written in place; the rest of it untouched."""
    T, Hq, Hk, D = 37, 6, 2, 96
    qkv = torch.randn(T, Hq + 2 * Hk, D, device="cuda").to(BF)
    before = qkv.clone()
    pos = torch.randint(-300, 300, (4, T + 5), device="cuda", dtype=torch.int32)[:3, :T]
    axis = torch.tensor([(i * 7) % 5 - 1 for i in range(40)], dtype=torch.int32, device="cuda")  # -1 .. 3
    f = freqs_of(40)
    w = torch.rand(D, device="cuda")
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    qo, ko = lb.qk_norm_rope(q, k, pos, f, w, w, pair_axis=axis, adjacent=True, Q_out=q, K_out=k)
    assert qo.data_ptr() == qkv.data_ptr()
    check(before[:, :Hq], qo, w, float(np.float32(1e-6)), pos, f, axis, True, "q")
    check(before[:, Hq:Hq + Hk], ko, w, float(np.float32(1e-6)), pos, f, axis, True, "k")
    assert torch.equal(qkv[:, Hq + Hk:], before[:, Hq + Hk:])


def test_far_positions():
    """Positions at the ends of their type keep their angles."""
    T, D = 6, 64
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 123456789, -1, 0], dtype=torch.int32, device="cuda")
    q = data(T, 2, D, F, 9, False)
    f = freqs_of(32)
    qo, _ = lb.qk_norm_rope(q, None, pos, f)
    check(q, qo, None, 0.0, pos, f, None, False, "q")
    # quarter turns are exact to the last rounding
    f = torch.full((32,), np.pi / 2, dtype=torch.float64, device="cuda")
    for p, (c, s) in enumerate(((1, 0), (0, 1), (-1, 0), (0, -1), (1, 0))):
        qo, _ = lb.qk_norm_rope(q, None, torch.full((T,), p, dtype=torch.int32, device="cuda"), f)
        a, b = q[..., :32], q[..., 32:]
        assert torch.allclose(qo, torch.cat((a * c - b * s, b * c + a * s), 2), rtol=0, atol=float(q.abs().max()) * 2.0 ** -23)


def test_special_values():
    """Zero heads, a NaN and an infinity reach their own head alone; large and small
    magnitudes; eps 0."""
    T, H, D = 3, 4, 128
    x = data(T, H, D, F, 4, False)
    x[0, 0] = 0
    x[0, 1, 5], x[1, 2, 70] = float("nan"), float("inf")
    x[2, 3] *= 1e17
    x[2, 1] *= 1e-17
    w = torch.rand(D, device="cuda") + 0.5
    pos, f = torch.arange(T, device="cuda", dtype=torch.int32), freqs_of(64)
    y, _ = lb.qk_norm_rope(x, None, pos, f, w, eps=1e-30)
    assert torch.equal(y[0, 0], torch.zeros_like(y[0, 0]))
    assert y[0, 1].isnan().all() and y[1, 2].isnan().any()
    bad = torch.zeros(T, H, dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[1, 2] = True
    assert torch.isfinite(y[~bad]).all()
    z = torch.where(bad[..., None], torch.zeros_like(x), x)
    check(z, torch.where(bad[..., None], torch.zeros_like(y), y), w, float(np.float32(1e-30)), pos, f, None, False, "x")
    assert lb.qk_norm_rope(x[:1, :1], None, pos[:1], f, w, eps=0.0)[0].isnan().all()  # 0 / 0, as the formula


def test_argument_errors():
    q, k = torch.zeros(2, 4, 64, device="cuda", dtype=BF), torch.zeros(2, 2, 64, device="cuda", dtype=BF)
    pos, f = torch.zeros(2, dtype=torch.int32, device="cuda"), freqs_of(32)
    for kw in (dict(K=k.float()), dict(K=k[:1]), dict(positions=pos[:1]), dict(positions=pos.long()), dict(freqs=f.float()),
               dict(q_weight=torch.ones(32, device="cuda")), dict(k_weight=torch.ones(64, device="cuda", dtype=BF)),
               dict(pair_axis=pos), dict(y_dtype=lb.I8), dict(Q_out=q.float(), y_dtype=lb.BF16), dict(K_out=q),
               dict(freqs=None, pair_axis=pos), dict(K=None, k_weight=torch.ones(64, device="cuda")), dict(freqs=f.cpu()),
               dict(positions=None)):
        args = dict(Q=q, K=k, positions=pos, freqs=f)
        args.update(kw)
        with pytest.raises(ValueError):
            lb.qk_norm_rope(**args)
    with pytest.raises(lb.LowbitError) as e:
        lb.qk_norm_rope(q, k, pos, freqs_of(36))
    assert e.value.status == lb.E_UNSUPPORTED


def test_in_a_graph():
    """Replays see new contents of the inputs."""
    q, k = data(5, 8, 128, BF, 1), data(5, 2, 128, BF, 2)
    pos, f = torch.arange(5, device="cuda", dtype=torch.int32), freqs_of(64)
    w = torch.rand(128, device="cuda")
    qo, ko = lb.qk_norm_rope(q, k, pos, f, w, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lb.qk_norm_rope(q, k, pos, f, w, w, Q_out=qo, K_out=ko)
    for i in range(3):
        q.copy_(data(5, 8, 128, BF, 10 + i))
        pos.add_(1000)
        want = lb.qk_norm_rope(q, k, pos, f, w, w)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


def test_offsets_past_32_bits():
    """Rows further apart than 2^31 elements."""
    D = 64
    big = torch.empty(3 * 2 ** 30 // 2 + 4096, dtype=BF, device="cuda")
    q = big.as_strided((2, 1, D), (3 * 2 ** 29, D, 1))
    q.copy_(data(2, 1, D, BF, 5))
    far = big.as_strided((2, 1, D), (3 * 2 ** 29, D, 1), 2048)
    pos, f = torch.arange(2, device="cuda", dtype=torch.int32), freqs_of(32)
    lb.qk_norm_rope(q, None, pos, f, Q_out=far)
    check(q.clone(), far.clone(), None, 0.0, pos, f, None, False, "q")
