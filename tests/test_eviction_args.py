"""The eviction entry points refuse bad arguments on the host before anything is launched (no device is
touched)."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def dsa():
    import __graft_entry__
    __graft_entry__.build()
    import sparse_attention_index_gb300 as m
    return m


# Fake (never dereferenced) 16-byte-aligned addresses: every call below fails validation on the
# host and returns before any CUDA call.
A = 1 << 20
P = ctypes.c_void_p(A)
FAR = ctypes.c_void_p(1 << 44)
MIS = ctypes.c_void_p(A + 4)


def test_cache_mass_refusals(dsa):
    size = dsa.lib.dsa_cache_mass_workspace_size

    def call(Q=P, cache=P, fmt=1, pages=8, page=64, table=P, maxp=4, lens=P, idx=None, k=0, lse=P, B=2,
             Sq=1, H=16, Dc=512, Dr=64, scale=0.1, prev=P, decay=0.5, mass=FAR, n=256, ws=P, nbytes=1 << 40):
        return dsa.lib.dsa_cache_mass(Q, cache, fmt, pages, page, table, maxp, lens, idx, k, lse, B, Sq, H,
                                      Dc, Dr, scale, prev, decay, mass, n, ws, nbytes, None)

    for name in ("Q", "cache", "table", "lens", "lse", "mass"):
        assert call(**{name: None}) == 1 and call(**{name: MIS}) == 1, name
    assert call(prev=MIS) == 1 and call(idx=MIS, k=4) == 1
    for name in ("pages", "page", "maxp", "B", "Sq", "H", "Dc", "n"):
        assert call(**{name: 0}) == 1, name
    assert call(fmt=5) == 1 and call(Dr=-8) == 1
    assert call(k=4) == 1 and call(idx=P) == 1 and call(idx=P, k=-1) == 1   # idx and k go together
    # prev is mass or apart from it
    assert call(mass=ctypes.c_void_p(A + 16)) == 1 and call(mass=ctypes.c_void_p(A + 2 * 256 * 4 - 16)) == 1
    assert call(prev=ctypes.c_void_p((1 << 44) + 16)) == 1
    assert call(Dc=256) == 2 and call(Dr=0) == 2 and call(H=129) == 2
    for scale in (0.0, -1.0, math.inf, math.nan, 2.1e38):
        assert call(scale=scale) == 2
    for decay in (math.inf, -math.inf, math.nan):
        assert call(decay=decay) == 2
    assert call(pages=1 << 26) == 2 and call(maxp=1 << 26) == 2 and call(n=2 ** 30 + 1) == 2
    assert call(B=1 << 20, Sq=1 << 10, n=1) == 2
    assert call(B=1 << 12, n=1, idx=P, k=1 << 20) == 2
    need = size(2, 1, 16, 512, 64, 4)
    assert need == 2 * 4 * 4
    for bad in (dict(ws=None), dict(ws=MIS), dict(nbytes=need - 1)):
        assert call(idx=P, k=4, **bad) == 3
    assert size(2, 1, 16, 512, 64, 0) == 0 and size(2, 1, 129, 512, 64, 4) == 0
    need = size(2, 9, 16, 512, 64, 0)      # sums of more than 128 pairs may be split
    assert need > 0 and call(Sq=9, nbytes=need - 1) == 3 and call(Sq=9, ws=None) == 3


def test_cache_keep_refusals(dsa):
    def call(mass=P, n=100, lens=P, B=2, budget=10, sink=2, recent=3, keep=P, count=P):
        return dsa.lib.dsa_cache_keep(mass, n, lens, B, budget, sink, recent, keep, count, None)

    for name in ("mass", "lens", "keep", "count"):
        assert call(**{name: None}) == 1 and call(**{name: MIS}) == 1, name
    for name in ("n", "B", "budget"):
        assert call(**{name: 0}) == 1, name
    assert call(sink=-1) == 1 and call(recent=-1) == 1
    assert call(sink=11, recent=0) == 1 and call(sink=0, recent=11) == 1 and call(sink=5, recent=6) == 1
    assert call(sink=2 ** 31 - 1, recent=2 ** 31 - 1) == 1      # their sum is past 32 bits
    assert call(n=2 ** 30 + 1) == 2 and call(budget=2 ** 30 + 1) == 2 and call(B=2 ** 27 + 1) == 2


def test_cache_compact_refusals(dsa):
    def call(cache=P, fmt=1, pages=8, page=64, table=P, maxp=4, lens=P, keep=P, budget=10, new=P,
             newp=1, B=2, Dc=512, Dr=64, mass=P, n=100, new_mass=FAR, new_n=10):
        return dsa.lib.dsa_cache_compact(cache, fmt, pages, page, table, maxp, lens, keep, budget, new,
                                         newp, B, Dc, Dr, mass, n, new_mass, new_n, None)

    for name in ("cache", "table", "lens", "keep"):
        assert call(**{name: None}) == 1 and call(**{name: MIS}) == 1, name
    for name in ("new", "mass", "new_mass"):
        assert call(**{name: MIS}) == 1, name
    assert call(mass=None) == 1 and call(new_mass=None) == 1     # both or none
    for name in ("pages", "page", "maxp", "budget", "B", "Dc", "newp", "n"):
        assert call(**{name: 0}) == 1, name
    assert call(fmt=2) == 1 and call(Dr=-8) == 1
    assert call(new_n=9) == 1                                    # weights need room for the budget
    assert call(budget=65, new_n=65) == 1                        # and so do the new pages
    # weights in place have the same columns; any other overlap is refused
    assert call(new_mass=P, new_n=99) == 1
    assert call(new_mass=ctypes.c_void_p(A + 16), new_n=100) == 1
    assert call(mass=ctypes.c_void_p(A + 64), new_mass=P, new_n=100) == 1
    assert call(Dc=500) == 2 and call(Dr=4) == 2
    assert call(pages=1 << 26) == 2 and call(maxp=1 << 26) == 2 and call(newp=1 << 26) == 2
    assert call(budget=2 ** 30 + 1, new_n=2 ** 30 + 1, newp=1 << 25) == 2
    assert call(n=2 ** 30 + 1) == 2 and call(new=None, B=65536) == 2


def test_python_checks(dsa):
    """CPU tensors, wrong types and wrong shapes raise before the library is called."""
    with pytest.raises(TypeError):
        dsa.dsa_cache_mass(torch.zeros(1, 1, 2, 576, dtype=torch.bfloat16), None, None, None, None, 1.0, 8)
    with pytest.raises(TypeError):
        dsa.dsa_cache_keep(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32), 4)
    with pytest.raises(TypeError):
        dsa.dsa_cache_compact(None, None, None, torch.zeros(2, 4, dtype=torch.int32), None, 512, 64)
