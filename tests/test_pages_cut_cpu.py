"""The count of cut children among the outputs of a fork, on a machine without a GPU."""
import ctypes

import pytest

from test_rope_pages_cpu import A1, A16, caches, kv
from ultra_bit_dit_amd import lowbit as lb

P = ctypes.c_void_p


def fork(cut, **kw):
    a = dict(pt=P(0x100000), ln=P(0x200000), refs=P(0x300000), par=P(0x400000), grow=P(0x500000), nt=P(0x600000), nl=P(0x700000),
             nr=P(0x800000), fl=P(0x900000))
    a.update(kw)
    return lb.lib().lowbit_kv8_fork_cut(caches(kv()), 1, 2, a["pt"], 4, a["ln"], a["refs"], 3, a["par"], a["grow"], 1, a["nt"], 4,
                                        a["nl"], a["nr"], a["fl"], cut, None)


def test_refusals():
    assert fork(A1) == lb.E_ALIGN
    for at, ints in ((0x100000, 8), (0x200000, 2), (0x300000, 64), (0x400000, 3), (0x500000, 3), (0x600000, 12), (0x700000, 3),
                     (0x800000, 64), (0x900000, 1)):
        assert fork(P(at)) == lb.E_UNSUPPORTED and fork(P(at + 4 * ints - 4)) == lb.E_UNSUPPORTED, hex(at)


@pytest.mark.parametrize("cut", [None, P(0xA00000)])
def test_the_rest_is_checked_as_without_it(cut):
    assert fork(cut, refs=None) == lb.E_NULL and fork(cut, nr=P(0x800008)) == lb.E_ALIGN
    assert fork(cut, nl=P(0x300000)) == lb.E_UNSUPPORTED and fork(cut, fl=A1) == lb.E_ALIGN
    assert fork(cut, pt=A16, nt=A16) == lb.E_UNSUPPORTED
