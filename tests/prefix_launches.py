"""Calls of attention behind shared prefixes, by the launches that the library's plan has for them."""
import ctypes
import functools
import math
import random

from ultra_bit_dit_amd import lowbit as lb


def launches(Hq, H, D, P, max_prefix, groups, max_seqs, seqs, total_q, max_q, max_kv, q_starts=True):
    """lowbit_attention_kv8_prefix_launches of these sizes, on a machine without a GPU too (nothing is read); None: refused."""
    c = lb.Kv8(1 << 20, P, H, D, 0x10000, 0x20000, 0x30000, 0x40000)
    p = lb.Kv8Prefix(groups, 0x50000, 1 << 22, 0x60000, 0x70000, max_seqs, max_prefix)
    b = lb.Kv8Batch(seqs, 0x50000, 1 << 22, 0x60000, 0x80000 if q_starts else None, total_q, max_q, max_kv, None)
    plan = lb.Kv8PrefixPlan()
    rc = lb.lib().lowbit_attention_kv8_prefix_launches(c, p, b, Hq, ctypes.byref(plan))
    return None if rc else {n: getattr(plan, n) for n, _ in plan._fields_}


def launches_of(case):
    """Of a case's arguments (prefix, count, new, own, Hq, H, D, P) as test_gpu_9_prefix.Call gives them."""
    return launches(case["Hq"], case["H"], case["D"], case["P"], max(max(case["prefix"]), 1), len(case["prefix"]),
                    max(max(case["count"]), 1), len(case["own"]), sum(case["new"]) + 2, max(max(case["new"]), 1),
                    max(max(case["own"]), 1))


def kind(D, plan):
    """The kernels of a plan, in words."""
    parts = plan["tile_parts"]
    if plan["tile_rows"] <= 32:
        how = f"attn_decode {plan['tile_rows']} rows, " + ("shares" if parts == 0 else "pieces" if parts > 1 else "whole tiles")
    else:
        how = f"prompt tiles of {plan['tile_rows']}, " + ("whole" if parts == 1 else "cut" if plan["whole_tiles"] == 0 else "last round cut")
        how += f", {plan['weight_terms']} terms"
    if plan["launches"] == 1:
        return f"D={D} {how}"
    return f"D={D} groups: {how}; sequences: {plan['own_rows']} rows, " + ("pieces" if plan["own_parts"] > 1 else "whole tiles")


def ragged(groups, seqs, new, own, told, **heads):
    """Sequences and prefixes of different lengths, the first ones the longest."""
    f = lambda i, least: 1.0 - (1.0 - least) * ((i * 0.6180339887) % 1.0)
    n = [max(1, int(new * f(i, 0.6))) for i in range(seqs)]
    return dict(prefix=[max(1, int(told * f(g, 0.5))) for g in range(groups)],
                count=[seqs // groups + (g < seqs % groups) for g in range(groups)], new=n,
                own=[max(n[i], int(own * f(i, 0.3))) for i in range(seqs)], **heads)


@functools.lru_cache(None)
def every_kind(draws=30000, least=3):
    """A small call for each kind of launch that `least` of `draws` random ones take."""
    rng = random.Random(11)
    some = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))
    best, seen = {}, {}
    for _ in range(draws):
        H, G, D = rng.choice((1, 2, 3, 4, 5, 8)), rng.choice((1, 2, 3, 4, 5, 6, 8, 16)), rng.choice((64, 128, 256))
        g, new, P = some(1, 40), some(1, 600), rng.choice((16, 32, 64, 128))
        seqs, own, told = g * some(1, 40), new + some(1, 1000), some(1, 60000)
        cost = (seqs + g) * max(own, 300) * H * D + seqs * new * H * G * D * 4
        if cost > 4e7:
            continue
        case = ragged(g, seqs, new, own, told, Hq=H * G, H=H, D=D, P=P)
        plan = launches_of(case)
        if plan is None:
            continue
        k = kind(D, plan)
        seen[k] = seen.get(k, 0) + 1
        if k not in best or cost < best[k][0]:
            best[k] = cost, case
    return {k: best[k][1] for k in sorted(best) if seen[k] >= least}
