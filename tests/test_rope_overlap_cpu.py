"""Which outputs of the head norms with rotation are refused for sharing bytes, on a machine without a GPU."""
import ctypes
import random

import pytest

from test_rope_pages_cpu import call, rope
from ultra_bit_dit_amd import lowbit as lb

BASE = 1 << 24
P = ctypes.c_void_p
BAD = lb.E_UNSUPPORTED


def at(elements, base=BASE, size=2):
    return P(base + size * elements)


# a fused projection of 4 + 2 + 2 heads of 64, three tokens
FUSED = dict(r=rope(positions=0x2000, freqs=0x3000), Q=at(0), qs=512, K=at(256), ks=512)


@pytest.mark.parametrize("kw", [
    dict(Qo=at(64), qos=512, Ko=at(1 << 16), kos=128),           # shifted by a head
    dict(Qo=at(8), qos=512, Ko=at(1 << 16), kos=128),            # by 16 bytes
    dict(Qo=at(512), qos=512, Ko=at(1 << 16), kos=128),          # by a token
    dict(Qo=at(1 << 16), qos=256, Ko=at(192), kos=512),          # the keys' over the last query head
    dict(Qo=at(1 << 16), qos=256, Ko=at(320), kos=512),          # over half of the keys
    dict(Qo=at(320), qos=512, Ko=at(1 << 16), kos=128),          # the queries' over keys, values and the next token
    dict(Qo=at(1 << 16), qos=256, Ko=at((1 << 16) + 760), kos=128),  # the last head of the other output
    dict(Qo=at(0), qos=520, Ko=at(256), kos=512),                # other strides: the second token no longer in place
    dict(Qo=at(384), qos=384, Ko=at(1 << 16), kos=128),          # rows that meet after some
])
def test_shared_bytes(kw):
    assert call(**{**FUSED, **kw}) == BAD


@pytest.mark.parametrize("name,size", [("positions", 12), ("freqs", 256), ("pair_axis", 128), ("qw", 256), ("kw", 256)])
def test_shared_with_small_inputs(name, size):
    """One element of what says how to turn or to weigh, at either end of either output."""
    far = dict(Qo=at(1 << 16), qos=256, Ko=at(1 << 17), kos=128)
    for out, row in (("Qo", 512), ("Ko", 256)):
        start = far[out].value
        step = 8 if name == "freqs" else 4
        for place in (start + 3 * row - step, start - size + step):
            kw = dict(FUSED, **far)
            if name in ("qw", "kw"):
                kw[name] = P(place)
            else:
                kw["r"] = rope(**{**dict(positions=0x2000, freqs=0x3000), name: place})
            if place % step == 0:
                assert call(**kw) == BAD, (name, out)


def test_second_axis():
    """Positions of the other axes lie pos_stride apart."""
    r = rope(positions=0x2000, freqs=0x3000, n_axes=3, pos_stride=(1 << 20) // 4)
    kw = dict(FUSED, r=r, Ko=at(1 << 17), kos=128)
    assert call(**dict(kw, Qo=P(0x2000 + (2 << 20)), qos=256)) == BAD


def test_rows_against_bytes():
    """The two outputs, random places and distances, against the bytes one by one: what shares one is refused."""
    rng, refused = random.Random(5), 0
    for _ in range(4000):
        T, hq, hk = rng.randint(1, 6), rng.randint(1, 3), rng.randint(1, 3)
        qos, kos = (8 * (h + rng.randint(0, 5)) for h in (hq, hk))
        if rng.random() < 0.5:
            qos = kos = max(qos, kos)
        q, k = BASE, BASE + 16 * rng.randint(-40, 40)
        rows = lambda p, h, s: {b for t in range(T) for b in range(p + 2 * t * s, p + 2 * t * s + 16 * h)}
        if not rows(q, hq, qos) & rows(k, hk, kos):
            continue
        refused += 1
        r = rope(tokens=T, head_dim=8, n_pairs=4, positions=0x2000, freqs=0x3000, pos_stride=T)
        assert call(r=r, Q=at(0, 1 << 28), hq=hq, qs=64, K=at(0, 1 << 29), hk=hk, ks=64, Qo=P(q), qos=qos, Ko=P(k), kos=kos) == BAD
    assert refused > 500


@pytest.mark.parametrize("name", ["qs", "ks", "qos", "kos"])
def test_rows_that_no_memory_has(name):
    """tokens * stride up to 2^46; the places of rows are counted in 64 bits."""
    r = rope(tokens=1 << 30, positions=0x2000, freqs=0x3000, pos_stride=1 << 30)
    strides = dict(qs=512, ks=512, qos=512, kos=512)
    assert call(**{**FUSED, "r": r, **strides, name: (1 << 16) + 8}) == lb.E_SHAPE
    # one less is looked at further: this address is misplaced
    assert call(**{**FUSED, "r": r, "Qo": P(BASE + 8), "Ko": at(1 << 40), **strides, name: 1 << 16}) == lb.E_ALIGN
