"""dsa_latent_attn_shared refuses bad arguments on the host before anything is launched (no device is
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
P = ctypes.c_void_p(1 << 20)
MIS = ctypes.c_void_p((1 << 20) + 4)


def test_refusals(dsa):
    size = dsa.lib.dsa_latent_attn_shared_workspace_size

    def call(Q=P, cache=P, fmt=1, pages=8, page=64, ptable=P, pmax=4, plens=P, starts=P, G=2, table=P,
             maxp=4, lens=P, B=4, Sq=1, H=16, Dc=512, Dr=64, scale=0.1, O=P, lse=P, ws=P, nbytes=1 << 40):
        return dsa.lib.dsa_latent_attn_shared(Q, cache, fmt, pages, page, ptable, pmax, plens, starts, G,
                                              table, maxp, lens, B, Sq, H, Dc, Dr, scale, O, lse, ws,
                                              nbytes, None)

    for name in ("Q", "cache", "ptable", "plens", "starts", "table", "lens", "O", "lse"):
        assert call(**{name: None}) == 1 and call(**{name: MIS}) == 1, name
    for name in ("pages", "page", "pmax", "maxp", "G", "B", "Sq", "H"):
        assert call(**{name: 0}) == 1, name
    assert call(fmt=5) == 1 and call(Dr=-8) == 1
    assert call(Dc=256) == 2 and call(Dr=0) == 2 and call(H=129) == 2 and call(G=65) == 2
    for scale in (0.0, -1.0, math.inf, math.nan, 2.1e38):
        assert call(scale=scale) == 2
    assert call(pages=1 << 26) == 2 and call(maxp=1 << 26) == 2 and call(pmax=1 << 26) == 2
    assert call(B=1 << 20, Sq=1 << 7) == 2
    need = size(4, 1, 16, 2, 512, 64)
    assert call(ws=None) == 3 and call(ws=MIS) == 3 and call(nbytes=need - 1) == 3
    for bad in ((0, 1, 16, 2, 512, 64), (4, 0, 16, 2, 512, 64), (4, 1, 129, 2, 512, 64),
                (4, 1, 16, 0, 512, 64), (4, 1, 16, 65, 512, 64), (4, 1, 16, 2, 256, 64),
                (4, 1, 16, 2, 512, 0), (1 << 23, 1, 128, 2, 512, 64)):
        assert size(*bad) == 0, bad


def test_workspace_holds_every_part(dsa):
    """A part per tile and 80 more of 32 to 128 rows of (512 + 2) fp32: tiles of the groups' rows (each
    group's rounded up) and of the sequences' own."""
    size = dsa.lib.dsa_latent_attn_shared_workspace_size
    for B, Sq, H, G in ((1, 1, 1, 1), (4, 1, 16, 1), (7, 3, 20, 3), (64, 1, 128, 2), (96, 7, 100, 64)):
        rows = B * Sq * H
        tiles = rows // 128 + min(G, B) + B * -(-Sq * H // 128)
        worst = (tiles + 80) * min(128, -(-rows // 32) * 32) * 514 * 4
        assert worst <= size(B, Sq, H, G, 512, 64) <= worst + 8 * tiles + 1024


def test_python_checks(dsa):
    with pytest.raises(TypeError):
        dsa.dsa_latent_attn_shared(torch.zeros(1, 1, 2, 576, dtype=torch.bfloat16), None, None, None, None,
                                   None, None, 1.0)


def test_refusals_agree_with_the_library(dsa):
    """What dsa_decode_layer asks before it writes to the cache is what the library then answers. (Its
    calls below are refused: an accepted set of arguments is not given to the library here.)"""
    A = 1 << 20
    shared = dict(qp=A, cp=A, fmt=1, num_pages=8, page_size=64, gp=A, max_prefix=4, pp=A, sp=A, G=2, tp=A,
                  max_pages=4, lp=A, B=4, Sq=1, H=16, Dc=512, Dr=64, scale=0.1, op=A, ep=A, wp=A,
                  ws_bytes=1 << 40)
    need = dsa.latent_attn_shared_workspace_bytes(4, 1, 16, 2, 512, 64)
    bads = [{name: A + 4} for name in ("qp", "cp", "gp", "pp", "sp", "tp", "lp", "op", "ep", "wp")]
    bads += [{name: 0} for name in ("num_pages", "page_size", "max_prefix", "G", "max_pages", "B", "Sq", "H")]
    bads += [dict(Dc=256), dict(Dr=0), dict(H=129), dict(G=65), dict(scale=0.0), dict(scale=math.nan),
             dict(scale=2.1e38), dict(num_pages=1 << 26), dict(max_pages=1 << 26), dict(max_prefix=1 << 26),
             dict(B=1 << 20, Sq=1 << 7), dict(wp=None), dict(ws_bytes=need - 1)]
    mass = dict(qp=A, cp=A, fmt=1, num_pages=8, page_size=64, tp=A, max_pages=4, lp=A, ip=None, k=0, ep=A, B=2,
                Sq=9, H=16, Dc=512, Dr=64, scale=0.1, pp=A, decay=0.5, mp=A, n=256, wp=A, ws_bytes=1 << 40)
    need = dsa.cache_mass_workspace_bytes(2, 9, 16, 512, 64)
    more = [{name: A + 4} for name in ("qp", "cp", "tp", "lp", "ep", "mp", "wp")]
    more += [{name: 0} for name in ("num_pages", "page_size", "max_pages", "B", "Sq", "H", "n")]
    more += [dict(ip=A + 4, k=4), dict(Dc=256), dict(Dr=0), dict(H=129), dict(scale=0.0), dict(scale=-1.0),
             dict(scale=math.inf), dict(scale=2.1e38), dict(decay=math.nan), dict(decay=1e300),
             dict(num_pages=1 << 26), dict(max_pages=1 << 26), dict(n=2 ** 30 + 1), dict(B=1 << 20, Sq=1 << 10, n=1),
             dict(ip=A, k=1 << 20, B=1 << 12, Sq=1, n=1), dict(wp=None), dict(ws_bytes=need - 1),
             dict(ip=A, k=4, wp=None)]
    for good, refusal, call, wrong in ((shared, dsa._shared_refusal, dsa.lib.dsa_latent_attn_shared, bads),
                                       (mass, dsa._mass_refusal, dsa.lib.dsa_cache_mass, more)):
        assert refusal(**good) == dsa.DSA_OK
        for bad in wrong:
            args = {**good, **bad}
            if call is dsa.lib.dsa_cache_mass:
                args["pp"] = args["mp"]
            want = refusal(**args)
            assert want != dsa.DSA_OK, bad
            assert call(*args.values(), None) == want, bad
