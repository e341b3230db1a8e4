"""What copies and swaps of an 8-bit cache's scales refuse (no GPU)."""
import ctypes

import pytest

from paged_kv_cache_245_gb300 import binding
from paged_kv_cache_245_gb300.build import build

FAKE = 0x10000  # aligned, never dereferenced: every call here fails before a launch


@pytest.fixture(scope="module")
def L():
    build()
    return binding.lib()


def pools(*at):
    return (ctypes.c_void_p * len(at))(*at)


def copy(L, pairs=FAKE, n=2, k=None, v=None, layers=1, blocks=10, size=8):
    return L.pkv_q8_scale_copy(pairs, n, k or pools(FAKE), v or pools(FAKE + 4), layers, blocks, size,
                               None)


@pytest.mark.parametrize("over", [dict(pairs=None), dict(pairs=FAKE + 4), dict(n=-1), dict(layers=-1),
                                  dict(k=pools(0)), dict(v=pools(FAKE + 2)), dict(blocks=0),
                                  dict(size=0), dict(size=6), dict(size=-4)])
def test_copy_refuses(L, over):
    assert copy(L, **over) == 1
    assert L.pkv_last_error()


def test_nothing_to_copy(L):
    assert copy(L, n=0, pairs=None) == 0
    assert copy(L, layers=0) == 0


@pytest.mark.parametrize("over", [dict(n=-1), dict(size=10), dict(size=0), dict(src=0), dict(dst=0),
                                  dict(layers=4097), dict(k=None)])
def test_swap_refuses(L, over):
    a = dict(n=2, k=pools(FAKE), src=4, dst=4, layers=1, size=4)
    a.update(over)
    one = pools(FAKE)
    assert L.pkv_q8_scale_swap(FAKE, a["n"], a["k"], one, a["src"], one, one, a["dst"], a["layers"],
                               a["size"], None) == 1


def test_words_are_named(L):
    assert copy(L, size=6) == 1
    assert b"multiple of 4" in L.pkv_last_error()
