"""Plain forms of the head norms with rotation and of the cache's page moves
(numpy, Python integers), and the rotation's error bound."""
import numpy as np


def rotate(x, weight, eps, positions, freqs, pair_axis, adjacent):
    """x [T][heads][D] float64, positions [axes][T] integers.  Returns y and, for
    the bound, the largest magnitude that went into each element."""
    T, H, D = x.shape
    y = x.copy()
    if weight is not None:
        y = y / np.sqrt((y * y).mean(2, keepdims=True) + eps) * weight
    mag = np.abs(y)
    turn = np.zeros_like(y)  # radians that went through rounding
    n = len(freqs)
    for i in range(n):
        axis = 0 if pair_axis is None else int(pair_axis[i])
        if not 0 <= axis < len(positions):
            continue
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, n + i)
        t = positions[axis].astype(np.longdouble) * np.longdouble(freqs[i])
        c, s = (f(t).astype(np.float64)[:, None] for f in (np.cos, np.sin))
        u, v = y[:, :, a].copy(), y[:, :, b].copy()
        y[:, :, a], y[:, :, b] = u * c - v * s, v * c + u * s
        mag[:, :, a] = mag[:, :, b] = np.abs(u) + np.abs(v)
        turn[:, :, a] = turn[:, :, b] = np.abs(t).astype(np.float64)[:, None]
    return y, mag, turn


def rotate_tolerance(y, mag, turn, D, bf16_out):
    """The sum of D squares is off by at most D steps of 2^-24 relative (all of one
    sign), its root by half of that, and root, quotient, weight, the angle's last
    rounding (pi/4 2^-24), two series (2^-24 each and their roundings, at most
    eight), two products and their sum add fewer than 24.  An angle of many turns
    is off by 2^-51 of itself (two fp64 products).  Output: half a step."""
    t = mag * ((D / 2 + 24) * 2.0 ** -24 + turn * 2.0 ** -51)
    return t + np.abs(y) * (2.0 ** -8 if bf16_out else 2.0 ** -24) * 1.01 + 2.0 ** -133


def held(n, P):
    return -(-n // P)


class Pages:
    """What lowbit_kv8_fork and lowbit_kv8_compact promise, in Python integers."""

    def __init__(self, n_pages, P):
        self.N, self.P = n_pages, P

    def _cut(self, n, width):
        return max(0, min(int(n), width * self.P, 2 ** 30))

    def fork(self, table, lens, refs, parents, grow, width):
        """Returns (table, lens, refs, failed, moves)."""
        P, N = self.P, self.N
        refs = [int(r) for r in refs]
        old_width = len(table[0]) if len(table) else 1
        lens = [self._cut(n, old_width) for n in lens]

        def ok(p):
            return 0 <= p < N

        for row, n in zip(table, lens):
            for p in row[:held(n, P)]:
                if ok(p):
                    refs[p] -= 1
        kids = []
        for i, q in enumerate(parents):
            q = int(q)
            n = self._cut(lens[q], width) if 0 <= q < len(lens) else 0
            row = [int(p) if ok(p) else -1 for p in (table[q][:held(n, P)] if n else [])]
            total = min(n + max(0, int(grow[i])), width * P, 2 ** 30)
            tail = row[-1] if total > n and n % P and row[-1] >= 0 else None
            kids.append([row, n, total, tail])
            for p in row:
                if p >= 0:
                    refs[p] += 1
        writers = {}
        for k in kids:
            if k[3] is not None:
                writers.setdefault(k[3], []).append(id(k))
        free = [p for p in range(N) if refs[p] == 0]
        need, moves, out = 0, [], []
        take = iter(free)
        after = list(refs)
        for k in kids:
            row, n, total, tail = k
            if tail is not None and not (refs[tail] == len(writers[tail]) and writers[tail][0] == id(k)):
                need += 1
                to = next(take, -1)
                moves.append((tail, to))
                after[tail] -= 1
                if to >= 0:
                    after[to] = 1
                row[-1] = to
            while len(row) < held(total, P):
                need += 1
                to = next(take, -1)
                if to >= 0:
                    after[to] = 1
                row.append(to)
            out.append(row + [-1] * (width - len(row)))
        failed = max(0, need - len(free))
        return out, [k[2] for k in kids], after, failed, [] if failed else moves

    def compact(self, table, lens, refs):
        """Returns (table, refs, remap, live, moves)."""
        N, P = self.N, self.P
        live = [p for p in range(N) if refs[p] > 0]
        L = len(live)
        holes = [p for p in range(L) if refs[p] <= 0]
        movers = [p for p in live if p >= L]
        to = [p if refs[p] > 0 else -1 for p in range(N)]
        new = [int(refs[p]) if p < L else 0 for p in range(N)]
        for p, q in zip(movers, holes):
            to[p] = q
            new[q] = int(refs[p])
        out = []
        for row, n in zip(table, lens):
            h = held(self._cut(n, len(row)), P)
            out.append([to[p] if 0 <= p < N else -1 for p in row[:h]] + [-1] * (len(row) - h))
        return out, new, to, L, list(zip(movers, holes))


def attention_prefix(q, Kp, Vp, Ko, Vo, first, scale, causal):
    """q [n][Hq][D] behind Kp, Vp [prefix][H][D], its own tokens Ko, Vo [T][H][D], query i at own position first + i.
    Returns O, lse and the bound's ingredients, as mx_ref.attention does."""
    import mx_ref
    n, Hq, D = q.shape
    out = []
    for i in range(n):
        hi = max(0, min(len(Ko), first + i + 1)) if causal else len(Ko)
        K, V = np.concatenate((Kp, Ko[:hi])), np.concatenate((Vp, Vo[:hi]))
        out.append(mx_ref.attention(q[i:i + 1], K, V, 0, scale, False, 0))
    return tuple(np.concatenate(x) for x in zip(*out))
