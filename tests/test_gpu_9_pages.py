"""Forking and compacting the cache's pages on the GPU, against plain integers."""
import numpy as np
import pytest
import torch

import serve_ref as R
from ultra_bit_dit_amd import lowbit as lb

pytestmark = pytest.mark.gpu


def i32(x, shape=None):
    t = torch.tensor(np.asarray(x, dtype=np.int64).astype(np.int32), device="cuda")
    return t if shape is None else t.reshape(shape)


def cache_of(n, P, H, D, seed):
    """A cache of random bytes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = lambda *s: torch.randint(0, 256, s, device="cuda", generator=g, dtype=torch.uint8)
    return (u(n, H, P, D).view(torch.float8_e4m3fn), u(n, H, D, P).view(torch.float8_e4m3fn), u(n, H), u(n, H))


def raw(cache):
    return [t.view(torch.uint8).clone() for t in cache]


def check_moves(before, caches, moves, what):
    """Every byte of every layer: the moved pages, and the others as they were."""
    for c, old in zip(caches, before):
        for t, o in zip(c, old):
            if moves:
                src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
                o[dst] = o[src]
            assert torch.equal(t.view(torch.uint8), o), what


def run_fork(caches, P, table, lens, refs, parents, grow, width, what, each=True, single=False):
    n_pages, B, n = caches[0][0].shape[0], len(lens), len(parents)
    before = [raw(c) for c in caches]
    w = len(table[0]) if B else 1
    t, l, r = i32(table, (B, w)), i32(lens, (B,)), i32(refs)
    keep = [x.clone() for x in (t, l, r)]
    g = i32(grow, (n,)) if each else (grow[0] if n else 0)
    out = lb.kv8_fork(caches[0] if single else caches, t, l, r, i32(parents, (n,)), grow=g, width=width,
                      max_grow=max([0] + [int(x) for x in grow]) if each else None)
    got = [x.cpu().numpy() for x in out]
    want = R.Pages(n_pages, P).fork(table, lens, refs, parents, grow, width)
    assert got[3][0] == want[3], what
    check_moves(before, caches, want[4], what)
    for a, b in zip((t, l, r), keep):
        assert torch.equal(a, b), f"{what}: an input changed"
    if want[3] == 0:
        assert got[0].tolist() == want[0] and got[1].tolist() == want[1] and got[2].tolist() == want[2], what
    return out


def batch(rng, n_pages, P, B, width, shared, holders=0.3):
    """Sequences with common first pages and pages of their own, and the counts; bad entries behind their pages."""
    perm = list(rng.permutation(n_pages))
    front = [perm.pop() for _ in range(shared)]
    table, lens, refs = [], [], [0] * n_pages
    for b in range(B):
        own = int(rng.integers(0, min(width - shared, len(perm) // (B - b)) + 1)) if len(perm) > B - b else 0
        row = front + [perm.pop() for _ in range(own)]
        n = len(row) * P - int(rng.integers(0, P)) if row else 0
        h = R.held(n, P)
        for p in row[:h]:
            refs[p] += 1
        table.append([int(p) for p in row] + [int(x) for x in rng.integers(-5, n_pages + 9, width - len(row))])
        lens.append(n)
    for p in range(n_pages):
        if rng.random() < holders and refs[p]:
            refs[p] += 1
    return table, lens, refs


@pytest.mark.parametrize("P,H,D", [(16, 1, 64), (32, 3, 64), (64, 2, 128), (128, 1, 256), (16, 5, 128)])
def test_fork(P, H, D):
    """Random batches: parents with several children and with none, outside the range, tokens to come from none to pages."""
    rng = np.random.default_rng(P + H)
    for i in range(14):
        n_pages, B, width = int(rng.integers(1, 90)), int(rng.integers(1, 9)), int(rng.integers(1, 12))
        shared = int(rng.integers(0, min(width, n_pages) + 1))
        table, lens, refs = batch(rng, n_pages, P, B, width, shared)
        n = int(rng.integers(1, 12))
        parents = rng.integers(-1, B + 1, n)
        grow = rng.choice([0, 1, 1, P - 1, 2 * P + 3], n)
        print(f"fork {i}: pages={n_pages} B={B} n={n} width={width}", flush=True)
        caches = [cache_of(n_pages, P, H, D, i)]
        run_fork(caches, P, table, lens, refs, parents, grow, width + int(rng.integers(0, 3)), f"fork {i}", single=True)
        run_fork(caches, P, table, lens, refs, parents, [1] * n, max(1, width - 2), f"fork {i}, cut", each=False)


def test_fork_corners():
    """Nothing yet, everything freed, negative and too large lengths, unreadable pages, pages that do not suffice."""
    P, n_pages = 16, 12
    c = [cache_of(n_pages, P, 2, 64, 1)]
    print("fork corners", flush=True)
    run_fork(c, P, [], [], [0] * n_pages, [-1, -1, 0], [17, 0, 33], 4, "start")
    run_fork(c, P, [[3, 4, 5]], [40], [0, 0, 0, 1, 1, 2] + [0] * 6, [], [], 4, "free all")
    table, refs = [[3, 4], [5, 6]], [0, 0, 0, 1, 1, 1, 1] + [0] * 5
    run_fork(c, P, table, [-3, 1000], refs, [0, 1, 1], [1, 0, 0], 4, "lengths")
    run_fork(c, P, [[3, 99], [-7, 6]], [20, 20], refs, [0, 0, 1, 1], [1] * 4, 4, "unreadable")
    run_fork(c, P, [[3, 4]], [20], [1] * n_pages, [0, 0], [1, 1], 3, "none free")
    run_fork(c, P, [[3, 4]], [20], [1] * 11 + [0], [0, 0, 0], [1, 13, 1], 3, "too few")
    run_fork(c, P, [[3, 4]], [20], [0] * 3 + [1, 1] + [0] * 7, [0] * 5, [100] * 5, 2, "cut")
    run_fork(c, P, [[3, 4], [3, 4]], [20, 20], [0] * 3 + [2, 2] + [0] * 7, [1, 0], [1, 1], 2, "a tail of two parents")
    run_fork(c, P, [[3, 4], [3, 4]], [20, 20], [0] * 3 + [2, 2] + [0] * 7, [1, 0], [0, 1], 2, "one of them writes")


def test_fork_many():
    """More children than threads of the planning workgroup, long rows, a large pool, many layers."""
    P, n_pages, B, n = 16, 40000, 300, 2500
    rng = np.random.default_rng(3)
    caches = [cache_of(n_pages, P, 1, 64, s) for s in range(2)]
    table, lens, refs = batch(rng, n_pages, P, B, 90, 40)
    print("fork many", flush=True)
    run_fork(caches, P, table, lens, refs, rng.integers(0, B, n), rng.choice([0, 1, 20], n), 95, "many")
    caches = [cache_of(70, P, 1 + s % 2, 64, s) for s in range(35)]
    table, lens, refs = batch(rng, 70, P, 3, 9, 2)
    run_fork(caches, P, table, lens, refs, [0, 0, 2, 2, 1], [1] * 5, 9, "layers")
    one = [cache_of(3000, P, 1, 64, 9)]
    row = [int(x) for x in rng.permutation(3000)[:2500]]
    refs = np.bincount(row, minlength=3000).tolist()
    run_fork(one, P, [row], [2500 * P - 3], refs, [0, 0, 0], [1, 5, 1], 2600, "a long row")


@pytest.mark.parametrize("P,H,D", [(16, 1, 64), (32, 3, 64), (64, 2, 128), (128, 1, 256)])
def test_compact(P, H, D):
    rng = np.random.default_rng(7 * P + H)
    for i in range(12):
        n_pages, B, width = int(rng.integers(1, 120)), int(rng.integers(0, 7)), int(rng.integers(1, 12))
        table, lens, refs = batch(rng, n_pages, P, B, width, int(rng.integers(0, min(width, n_pages) + 1)), 0.2)
        if i == 0:
            refs = [0] * n_pages
        if i == 1:
            refs = [1] * n_pages
        for p in rng.integers(0, n_pages, 3):
            refs[p] += int(i > 1)  # a store's pages, in no row
        print(f"compact {i}: pages={n_pages} B={B}", flush=True)
        run_compact([cache_of(n_pages, P, H, D, i) for _ in range(1 + i % 2)], P, table, lens, refs, width, f"compact {i}")


def run_compact(caches, P, table, lens, refs, width, what):
    before = [raw(c) for c in caches]
    B, n_pages = len(lens), caches[0][0].shape[0]
    ins = i32(table, (B, width)), i32(lens, (B,)), i32(refs)
    keep = [x.clone() for x in ins]
    out = lb.kv8_compact(caches, *ins)
    want = R.Pages(n_pages, P).compact(table, lens, refs)
    assert out[0].cpu().tolist() == want[0] and out[1].cpu().tolist() == want[1] and out[2].cpu().tolist() == want[2], what
    assert out[3].item() == want[3], what
    check_moves(before, caches, want[4], what)
    for a, b in zip(ins, keep):
        assert torch.equal(a, b), f"{what}: an input changed"


def test_compact_many():
    """Several chunks of pages, the border inside one and at its edge."""
    rng = np.random.default_rng(5)
    for n_pages, L in ((20000, 9000), (16384, 8192), (4097, 4096), (4096, 4096), (12289, 1), (28672, 20001), (28673, 16000),
                       (40960, 8192), (36865, 36864), (45000, 0)):
        refs = np.zeros(n_pages, int)
        refs[rng.permutation(n_pages)[:L]] = rng.integers(1, 5, L)
        use = np.nonzero(refs)[0]
        table = [[int(x) for x in rng.choice(use, 1500)] if L else [7] * 1500 for _ in range(3)]
        print(f"compact {n_pages} {L}", flush=True)
        run_compact([cache_of(n_pages, 16, 1, 64, 1)], 16, table, [1500 * 16, 1499 * 16, 5], refs.tolist(), 1500, f"{n_pages} {L}")


def test_pages_past_32_bits():
    """Pages further than 2^32 bytes into the cache."""
    P, H, D = 128, 8, 256
    n_pages = 2 ** 32 // (P * H * D) + 9
    kc = torch.zeros(n_pages, H, P, D, dtype=torch.uint8, device="cuda")
    vc, ks, vs = torch.zeros(n_pages, H, D, P, dtype=torch.uint8, device="cuda"), *torch.zeros(2, n_pages, H, dtype=torch.uint8,
                                                                                             device="cuda")
    c = (kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), ks, vs)
    g = torch.Generator(device="cuda").manual_seed(1)
    last = n_pages - 1
    for t in (kc, vc, ks, vs):
        t[last] = torch.randint(0, 256, t[last].shape, device="cuda", generator=g, dtype=torch.uint8)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[last] = 1
    want = [t[last].clone() for t in (kc, vc, ks, vs)]
    print("pages past 32 bits", flush=True)
    out = lb.kv8_compact(c, i32([[last]]), i32([P]), refs)
    assert out[0].item() == 0 and all(torch.equal(t[0], w) for t, w in zip((kc, vc, ks, vs), want))
    refs = torch.ones(n_pages, dtype=torch.int32, device="cuda")
    refs[last - 1] = 0
    for t in (kc, vc, ks, vs):
        t[0] = 0
    out = lb.kv8_fork(c, i32([[last]]), i32([P - 1]), refs, i32([0, 0]), grow=1)
    assert out[0].cpu().tolist() == [[last], [last - 1]] and all(torch.equal(t[last - 1], w) for t, w in zip((kc, vc, ks, vs), want))


def test_argument_errors():
    c = lb.empty_kv8(8, 16, 2, 64)
    pt, ln, rf, pr = i32([[1, 2]]), i32([20]), i32([0] * 8), i32([0])
    for kw in (dict(page_table=pt.long()), dict(kv_lens=ln[:0]), dict(refs=rf[:7]), dict(parents=pr.long()),
               dict(grow=i32([1])), dict(grow=i32([1, 2]), max_grow=2), dict(cache=[c, lb.empty_kv8(9, 16, 2, 64)]),
               dict(out=(pt, ln, rf)), dict(out=(pt, ln, rf.long(), ln)), dict(refs=rf.cpu())):
        args = dict(cache=c, page_table=pt, kv_lens=ln, refs=rf, parents=pr)
        args.update(kw)
        with pytest.raises(ValueError):
            lb.kv8_fork(**args)
    for kw in (dict(page_table=pt.t()), dict(refs=rf[1:]), dict(out=(pt,))):
        args = dict(cache=c, page_table=pt, kv_lens=ln, refs=rf)
        args.update(kw)
        with pytest.raises(ValueError):
            lb.kv8_compact(**args)
    with pytest.raises(lb.LowbitError) as e:
        lb.kv8_fork(c, pt, ln, rf, pr, grow=-1)
    assert e.value.status == lb.E_SHAPE


def test_in_a_graph():
    """Two steps of forking in one graph, the second from the first's outputs; every replay from new
    parents, other work between; a capture without its workspace is refused."""
    P, n_pages, n = 16, 300, 6
    c = cache_of(n_pages, P, 2, 64, 1)
    table, lens, refs = batch(np.random.default_rng(8), n_pages, P, n, 12, 3, 0)
    t, l, r, p, p2 = i32(table), i32(lens), i32(refs), i32([0] * n), i32([0] * n)
    s = torch.cuda.Stream()
    mk = lambda: (torch.empty(n, 14, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda"),
                  torch.empty(n_pages, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda"))
    a, b, z = mk(), mk(), tuple(mk()[i] for i in (0, 2, 2, 3))  # table, lengths, counts, failed; table, counts, remap, live
    torch.cuda.synchronize()
    lb.release_workspaces()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.capture_begin()
        with pytest.raises(lb.LowbitError) as e:
            lb.kv8_fork(c, t, l, r, p, grow=1, width=14, out=a)
        g.capture_end()
    assert e.value.status == lb.E_NOMEM
    with torch.cuda.stream(s):
        lb.reserve_workspace(max(lb.kv8_fork_workspace(n_pages, P, n, n, 3), lb.kv8_compact_workspace(n_pages)))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lb.kv8_fork(c, t, l, r, p, grow=1, width=14, out=a)
        lb.kv8_fork(c, a[0], a[1], a[2], p2, grow=3, width=14, out=b)
        lb.kv8_compact(c, b[0], b[1], b[2], out=z)
    rng = np.random.default_rng(9)
    fresh = raw(c)
    for i in range(4):
        for x, y in zip(c, fresh):
            x.view(torch.uint8).copy_(y)
        q, q2 = rng.integers(0, n, n), rng.integers(0, n, n)
        p.copy_(i32(q))
        p2.copy_(i32(q2))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        oracle = R.Pages(n_pages, P)
        w = oracle.fork(table, lens, refs, q, [1] * n, 14)
        w2 = oracle.fork(w[0], w[1], w[2], q2, [3] * n, 14)
        w3 = oracle.compact(w2[0], w2[1], w2[2])
        assert a[0].cpu().tolist() == w[0] and b[0].cpu().tolist() == w2[0] and b[2].cpu().tolist() == w2[2], i
        assert z[0].cpu().tolist() == w3[0] and z[1].cpu().tolist() == w3[1] and z[2].cpu().tolist() == w3[2], i
        now = [x.clone() for x in fresh]
        for moves in (w[4], w2[4], w3[4]):
            check = [x.clone() for x in now]
            for src, dst in moves:
                for x, y in zip(now, check):
                    x[dst] = y[src]
        assert all(torch.equal(x.view(torch.uint8), y) for x, y in zip(c, now)), i
        torch.randn(1 << 16, device="cuda").sum().item()
