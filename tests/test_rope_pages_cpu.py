"""Head norms with rotation and page calls on a machine without a GPU: every
refusal comes before any HIP call; pins of the plain forms."""
import ctypes

import numpy as np
import pytest

import serve_ref as R
from ultra_bit_dit_amd import lowbit as lb

A16, A8, A4, A1 = (ctypes.c_void_p(0x10000 + k) for k in (0, 8, 4, 1))


def rope(**over):
    r = dict(tokens=3, head_dim=64, n_pairs=32, adjacent=0, n_axes=1, positions=0x20000, pos_stride=3, freqs=0x30000,
             pair_axis=None)
    r.update(over)
    return lb.Rope(*[r[f[0]] for f in lb.Rope._fields_])


def call(r=None, xd=lb.BF16, Q=A16, hq=4, qs=256, qw=None, K=A16, hk=2, ks=128, kw=None, eps=1e-6, yd=lb.BF16, Qo=A16, qos=256,
         Ko=A16, kos=128):
    return lb.lib().lowbit_qk_norm_rope(rope() if r is None else r, xd, Q, hq, qs, qw, K, hk, ks, kw, eps, yd, Qo, qos, Ko, kos,
                                        None)


@pytest.mark.parametrize("kw,status", [
    (dict(Q=None), lb.E_NULL), (dict(Qo=None), lb.E_NULL), (dict(K=None), lb.E_NULL), (dict(Ko=None), lb.E_NULL),
    (dict(r=rope(positions=None)), lb.E_NULL), (dict(r=rope(freqs=None)), lb.E_NULL),
    (dict(xd=lb.I8), lb.E_UNSUPPORTED), (dict(yd=lb.I32), lb.E_UNSUPPORTED),
    (dict(r=rope(head_dim=60)), lb.E_UNSUPPORTED), (dict(r=rope(head_dim=264)), lb.E_UNSUPPORTED),
    (dict(r=rope(head_dim=0)), lb.E_UNSUPPORTED), (dict(r=rope(n_pairs=6)), lb.E_UNSUPPORTED),
    (dict(r=rope(n_pairs=36)), lb.E_UNSUPPORTED), (dict(r=rope(n_pairs=-4)), lb.E_UNSUPPORTED),
    (dict(eps=-1.0), lb.E_UNSUPPORTED), (dict(eps=float("inf")), lb.E_UNSUPPORTED), (dict(eps=float("nan")), lb.E_UNSUPPORTED),
    (dict(r=rope(tokens=0)), lb.E_SHAPE), (dict(r=rope(tokens=(1 << 30) + 1)), lb.E_SHAPE), (dict(r=rope(n_axes=0)), lb.E_SHAPE),
    (dict(r=rope(n_axes=2, pos_stride=2)), lb.E_SHAPE), (dict(hq=0), lb.E_SHAPE), (dict(hq=(1 << 16) + 1), lb.E_SHAPE),
    (dict(hk=-1), lb.E_SHAPE), (dict(qs=248), lb.E_SHAPE), (dict(ks=120), lb.E_SHAPE), (dict(qos=248), lb.E_SHAPE),
    (dict(kos=120), lb.E_SHAPE), (dict(qs=1 << 41), lb.E_SHAPE),
    (dict(Q=A8), lb.E_ALIGN), (dict(Qo=A8), lb.E_ALIGN), (dict(K=A8), lb.E_ALIGN), (dict(Ko=A8), lb.E_ALIGN),
    (dict(qs=260), lb.E_ALIGN), (dict(kos=132), lb.E_ALIGN), (dict(qw=A1), lb.E_ALIGN), (dict(kw=A1), lb.E_ALIGN),
    (dict(r=rope(freqs=0x30004)), lb.E_ALIGN), (dict(r=rope(positions=0x20002)), lb.E_ALIGN),
    (dict(r=rope(pair_axis=0x20002)), lb.E_ALIGN),
])
def test_rope_refusals(kw, status):
    assert call(**kw) == status


def test_rope_outputs_elsewhere_or_in_place():
    """In place: the same type and strides.  Never over the other input, or both outputs in one place."""
    B, C, D = (ctypes.c_void_p(k) for k in (0x40000, 0x50000, 0x60000))
    bad = lb.E_UNSUPPORTED
    assert call(K=B, Ko=C, qos=512) == bad and call(K=B, Ko=C, yd=lb.F32) == bad and call(K=B, Qo=D, Ko=B, kos=256) == bad
    assert call(K=B, Qo=B, Ko=C) == bad and call(K=B, Qo=C, Ko=A16) == bad and call(K=B, Qo=D, Ko=D) == bad


def kv(**over):
    c = dict(n_pages=64, page_tokens=16, kv_heads=2, head_dim=64, k_codes=0x10000, v_codes=0x20000, k_scales=0x30000,
             v_scales=0x40000)
    c.update(over)
    return lb.Kv8(*[c[f[0]] for f in lb.Kv8._fields_])


def caches(*cs):
    return (lb.Kv8 * len(cs))(*cs)


def fork(c=None, nc=1, B=2, pt=A16, w=4, ln=A16, refs=A16, n=3, par=A16, grow=None, mg=1, nt=A16, nw=4, nl=A16, nr=A16, fl=A16):
    return lb.lib().lowbit_kv8_fork(caches(kv()) if c is None else c, nc, B, pt, w, ln, refs, n, par, grow, mg, nt, nw, nl, nr, fl,
                                    None)


def compact(c=None, nc=1, B=2, pt=A16, w=4, ln=A16, refs=A16, nt=A16, nr=A16, rm=A16, lv=A16):
    return lb.lib().lowbit_kv8_compact(caches(kv()) if c is None else c, nc, B, pt, w, ln, refs, nt, nr, rm, lv, None)


@pytest.mark.parametrize("c,nc,status", [
    (caches(kv(k_codes=None)), 1, lb.E_NULL), (caches(kv(), kv(v_scales=None)), 2, lb.E_NULL), (caches(kv()), 0, lb.E_SHAPE),
    (caches(kv()), 4097, lb.E_SHAPE), (caches(kv(page_tokens=24)), 1, lb.E_UNSUPPORTED),
    (caches(kv(head_dim=96)), 1, lb.E_UNSUPPORTED), (caches(kv(n_pages=0)), 1, lb.E_SHAPE),
    (caches(kv(n_pages=(1 << 26) + 1)), 1, lb.E_SHAPE), (caches(kv(kv_heads=0)), 1, lb.E_SHAPE),
    (caches(kv(), kv(n_pages=63)), 2, lb.E_SHAPE), (caches(kv(), kv(page_tokens=32)), 2, lb.E_SHAPE),
    (caches(kv(v_codes=0x20008)), 1, lb.E_ALIGN)])
def test_caches_refusals(c, nc, status):
    assert fork(c, nc) == status and compact(c, nc) == status


def test_fork_refusals():
    assert lb.lib().lowbit_kv8_fork(None, 1, 1, A16, 1, A16, A16, 1, A16, None, 1, A16, 1, A16, A16, A16, None) == lb.E_NULL
    for k in ("pt", "ln", "refs", "par", "nt", "nl", "nr", "fl"):
        assert fork(**{k: None}) == lb.E_NULL, k
    for k in ("pt", "ln", "refs", "par", "grow", "nt", "nl", "fl"):
        assert fork(**{k: A1}) == lb.E_ALIGN, k
    assert fork(nr=A8) == lb.E_ALIGN
    for kw in (dict(B=-1), dict(B=(1 << 20) + 1), dict(n=-1), dict(n=(1 << 20) + 1), dict(w=0), dict(w=(1 << 26) + 1), dict(nw=0),
               dict(nw=(1 << 26) + 1), dict(mg=-1), dict(mg=(1 << 30) + 1), dict(n=1 << 20, mg=1 << 20),
               dict(n=1 << 20, nw=1 << 20)):
        assert fork(**kw) == lb.E_SHAPE, kw
    b = ctypes.c_size_t(7)
    f = lb.lib().lowbit_kv8_fork_workspace
    assert f(64, 16, 1, 1, 1, 1, None) == lb.E_NULL
    assert f(64, 17, 1, 1, 1, 1, ctypes.byref(b)) == lb.E_UNSUPPORTED and b.value == 0
    for bad in ((0, 16, 1, 1, 1, 1), (1 << 27, 16, 1, 1, 1, 1), (64, 16, 1, -1, 1, 1), (64, 16, 1, 1, 1 << 21, 1),
                (64, 16, 1, 1, 1, -1), (64, 16, 1, 1, 1 << 20, 1 << 20), (64, 16, 0, 1, 1, 1), (64, 16, 4097, 1, 1, 1)):
        assert f(*bad, ctypes.byref(b)) == lb.E_SHAPE
    assert lb.kv8_fork_workspace(64, 16, 0, 0, 0) > 0
    # the free pages' list grows with what can be asked for, never past the pages
    assert lb.kv8_fork_workspace(1 << 20, 16, 8, 1 << 10, 1) < lb.kv8_fork_workspace(1 << 20, 16, 8, 1 << 10, 1 << 12)
    assert lb.kv8_fork_workspace(1 << 20, 16, 8, 1 << 10, 1 << 16) == lb.kv8_fork_workspace(1 << 20, 16, 8, 1 << 10, 1 << 17)


def test_page_outputs_overlap_nothing():
    """Refused where one integer is shared."""
    at = {k: 0x100000 * (i + 1) for i, k in enumerate(("pt", "ln", "refs", "par", "grow", "nt", "nl", "nr", "fl", "rm", "lv"))}
    size = dict(pt=8, ln=2, refs=64, par=3, grow=3, nt=12, nl=3, nr=64, fl=1, rm=64, lv=1)
    for f, ins, outs in ((fork, ("pt", "ln", "refs", "par", "grow"), ("nt", "nl", "nr", "fl")),
                         (compact, ("pt", "ln", "refs"), ("nt", "nr", "rm", "lv"))):
        base = {k: ctypes.c_void_p(at[k]) for k in ins + outs}
        n = dict(size, nt=8) if f is compact else size
        for o in outs:
            for i in ins + outs:
                if i == o:
                    continue
                if o != "nr" or f is compact:  # the last integer of i
                    assert f(**dict(base, **{o: ctypes.c_void_p(at[i] + 4 * n[i] - 4)})) == lb.E_UNSUPPORTED, (o, i)
                assert f(**dict(base, **{o: ctypes.c_void_p(at[i])})) == lb.E_UNSUPPORTED, (o, i)


def test_compact_refusals():
    for k in ("pt", "ln", "refs", "nt", "nr", "rm", "lv"):
        assert compact(**{k: None}) == lb.E_NULL, k
        assert compact(**{k: A1}) == lb.E_ALIGN, k
    for kw in (dict(B=-1), dict(B=(1 << 20) + 1), dict(w=0), dict(w=(1 << 26) + 1), dict(B=1 << 20, w=1 << 20)):
        assert compact(**kw) == lb.E_SHAPE, kw
    b = ctypes.c_size_t(7)
    f = lb.lib().lowbit_kv8_compact_workspace
    assert f(64, 1, None) == lb.E_NULL
    assert f(0, 1, ctypes.byref(b)) == lb.E_SHAPE and b.value == 0
    assert f((1 << 26) + 1, 1, ctypes.byref(b)) == lb.E_SHAPE and f(64, 0, ctypes.byref(b)) == lb.E_SHAPE


# ------------------------------------------------------- the plain forms' pins


def test_rotation_keeps_lengths_and_turns_products():
    """A rotation keeps each pair's length, and the product of a rotated query and
    key depends on the difference of their positions alone."""
    g = np.random.default_rng(1)
    q, k = g.standard_normal((2, 1, 1, 16))
    f = 1e4 ** (-np.arange(8) / 8)
    at = lambda x, p, adj: R.rotate(x, None, 0.0, np.array([[p]]), f, None, adj)[0][0, 0]
    for adj in (False, True):
        a = at(q, 7, adj) @ at(k, 3, adj)
        assert abs(a - at(q, 1007, adj) @ at(k, 1003, adj)) < 1e-10
        y = at(q, 5, adj)
        i, j = (0, 1) if adj else (0, 8)
        assert abs(np.hypot(y[i], y[j]) - np.hypot(q[0, 0, i], q[0, 0, j])) < 1e-12
        assert np.allclose(y[[i, j]], [q[0, 0, i] * np.cos(5) - q[0, 0, j] * np.sin(5),
                                       q[0, 0, j] * np.cos(5) + q[0, 0, i] * np.sin(5)])


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((2, 3, 24)) * 9
    y = R.rotate(x, np.ones(24), 0.0, np.zeros((1, 2), int), [], None, False)[0]
    assert np.allclose((y * y).mean(2), 1)


def test_fork_by_hand():
    """Two sequences of 20 tokens in pages of 16: the first one forked in two, the second freed."""
    p = R.Pages(8, 16)
    table, lens, refs = [[3, 5, -1], [3, 1, -1]], [20, 20], [0, 1, 0, 3, 0, 1, 0, 0]  # page 3: one holder more elsewhere
    out = p.fork(table, lens, refs, [0, 0], [1, 1], 3)
    # the first child keeps page 5, the second gets a copy in the lowest free page; page 1 is free again
    assert out == ([[3, 5, -1], [3, 0, -1]], [21, 21], [1, 0, 0, 3, 0, 1, 0, 0], 0, [(5, 0)])
    # without tokens to come nothing is copied; 13 more need a page each
    assert p.fork(table, lens, refs, [0, 0], [0, 0], 3)[0] == [[3, 5, -1], [3, 5, -1]]
    assert p.fork(table, lens, refs, [0, 0], [13, 13], 3)[0] == [[3, 5, 0], [3, 1, 2]]
    assert p.fork(table, lens, refs, [0, -1, 7], [0, 17, 1], 3)[:2] == ([[3, 5, -1], [0, 1, -1], [2, -1, -1]], [20, 17, 1])
    # all of the pages are needed and more
    assert p.fork(table, lens, refs, [-1], [200], 3)[3] == 0 and p.fork(table, lens, refs, [-1], [200], 13)[3] == 6


def test_compact_by_hand():
    p = R.Pages(8, 16)
    out = p.compact([[6, 2], [2, 7]], [17, 32], [0, 0, 2, 0, 0, 0, 1, 1])
    assert out == ([[0, 2], [2, 1]], [1, 1, 2, 0, 0, 0, 0, 0], [-1, -1, 2, -1, -1, -1, 0, 1], 3, [(6, 0), (7, 1)])
