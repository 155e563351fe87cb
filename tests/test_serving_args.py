"""The serving entry points refuse bad arguments on the host before anything is launched (no
device is touched), and the frequencies of the scaled rotary positions."""
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
FAR = ctypes.c_void_p(1 << 40)
MIS = ctypes.c_void_p(A + 4)


def test_rope_refusals(dsa):
    def rope(x=P, y=FAR, dtype=0, pos=P, inv=P, T=4, H=2, D=192, off=128, rot=64, layout=0):
        return dsa.lib.dsa_rope(x, y, dtype, pos, inv, T, H, D, off, rot, layout, 1.0, 0, None)

    for name in ("x", "y", "pos", "inv"):
        assert rope(**{name: None}) == 1, name
        assert rope(**{name: MIS}) == 1, name
    assert rope(dtype=2) == 1 and rope(layout=2) == 1 and rope(layout=-1) == 1
    assert rope(T=0) == 1 and rope(H=0) == 1 and rope(D=0) == 1 and rope(rot=0) == 1
    assert rope(off=-8) == 1 and rope(off=136) == 1 and rope(off=200) == 1   # past the head's end
    assert rope(D=1032, off=0) == 2 and rope(D=196) == 2
    assert rope(off=124) == 2 and rope(rot=24) == 2 and rope(rot=8) == 2
    # overlapping, but not the same, input and output
    n = 5 * 2 * 192 * 2
    assert rope(T=5, y=ctypes.c_void_p(A + 16)) == 1
    assert rope(T=5, y=ctypes.c_void_p(A + n - 16)) == 1
    assert rope(T=5, x=ctypes.c_void_p(A + n - 16), y=P) == 1
    assert rope(T=2 ** 31 - 1, H=2 ** 31 - 1) == 2


def test_cache_row_bytes(dsa):
    assert dsa.cache_row_bytes(512, 64, "bf16") == 1152
    assert dsa.cache_row_bytes(512, 64, "e4m3") == 512 + 16 + 128
    assert dsa.cache_row_bytes(128, 0, "e4m3") == 128 + 16
    assert dsa.cache_row_bytes(640, 8, "e4m3") == 640 + 32 + 16
    for Dc, Dr in ((0, 64), (64, 64), (500, 64), (1152, 0), (512, 4), (512, 264), (512, -8)):
        assert dsa.cache_row_bytes(Dc, Dr) == 0
    assert dsa.lib.dsa_cache_row_bytes(2, 512, 64) == 0
    with pytest.raises(ValueError):
        dsa.cache_row_bytes(512, 64, "fp4")


@pytest.mark.parametrize("write", [True, False])
def test_cache_refusals(dsa, write):
    def call(kv=P, slots=P, cache=P, n=4, Dc=512, Dr=64, fmt=1, num=64):
        if write:
            return dsa.lib.dsa_cache_write(kv, slots, n, Dc, Dr, fmt, cache, num, None)
        return dsa.lib.dsa_cache_read(cache, num, fmt, slots, n, Dc, Dr, kv, None)

    for name in ("kv", "slots", "cache"):
        assert call(**{name: None}) == 1 and call(**{name: MIS}) == 1, name
    assert call(n=0) == 1 and call(Dc=0) == 1 and call(Dr=-8) == 1 and call(num=0) == 1
    assert call(fmt=2) == 1
    assert call(Dc=500) == 2 and call(Dr=4) == 2 and call(Dc=2048) == 2
    assert call(num=1 << 31) == 2


def test_latent_attn_refusals(dsa):
    size = dsa.lib.dsa_latent_attn_workspace_size

    def call(Q=P, cache=P, fmt=1, pages=8, page=64, table=P, maxp=4, lens=P, idx=None, k=0, B=2,
             Sq=1, H=16, Dc=512, Dr=64, scale=0.1, O=P, lse=P, ws=P, nbytes=None):
        if nbytes is None:
            nbytes = 1 << 40
        return dsa.lib.dsa_latent_attn(Q, cache, fmt, pages, page, table, maxp, lens, idx, k, B, Sq,
                                       H, Dc, Dr, scale, O, lse, ws, nbytes, None)

    for name in ("Q", "cache", "table", "lens", "O", "lse"):
        assert call(**{name: None}) == 1 and call(**{name: MIS}) == 1, name
    assert call(idx=MIS, k=4) == 1
    for name in ("pages", "page", "maxp", "B", "Sq", "H"):
        assert call(**{name: 0}) == 1, name
    assert call(fmt=5) == 1
    assert call(k=4) == 1 and call(idx=P) == 1 and call(idx=P, k=-1) == 1   # idx and k go together
    assert call(Dc=256) == 2 and call(Dr=0) == 2 and call(H=129) == 2
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=scale) == 2
    assert call(pages=1 << 26, page=64) == 2 and call(maxp=1 << 26) == 2
    assert call(B=1 << 20, Sq=1 << 10) == 2
    need = size(2, 1, 16, 512, 64, 0)
    if need:
        assert call(ws=None) == 3 and call(ws=MIS) == 3 and call(nbytes=need - 1) == 3
    assert size(0, 1, 16, 512, 64, 0) == 0 and size(1, 1, 129, 512, 64, 0) == 0
    assert size(1, 1, 16, 256, 64, 0) == 0 and size(1, 1, 16, 512, 64, -1) == 0


def test_python_checks(dsa):
    """CPU tensors, wrong types and wrong shapes raise before the library is called."""
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        dsa.dsa_rope(x, torch.zeros(4, dtype=torch.int32), torch.zeros(16))
    with pytest.raises(TypeError):
        dsa.dsa_rope(x.half(), torch.zeros(4, dtype=torch.int32), torch.zeros(16))
    with pytest.raises(ValueError):
        dsa.dsa_rope(x, torch.zeros(4, dtype=torch.int32), torch.zeros(16), layout="neox")
    with pytest.raises(TypeError):
        dsa.dsa_cache_write(torch.zeros(4, 576, dtype=torch.bfloat16), None, None, 512)
    with pytest.raises(TypeError):
        dsa.dsa_cache_read(None, torch.zeros(4, dtype=torch.int32), 512, 64)
    with pytest.raises(TypeError):
        dsa.dsa_latent_attn(torch.zeros(1, 1, 2, 576, dtype=torch.bfloat16), None, None, None, 1.0)


def test_rope_frequencies(dsa):
    """Against the formulas, frequency by frequency."""
    rot, base, factor, length = 64, 10000.0, 40.0, 4096
    plain, m = dsa.rope_frequencies(rot, base, device="cpu")
    assert m == 1.0 and plain.dtype == torch.float32 and plain.shape == (32,)
    want = [base ** (-2 * i / rot) for i in range(32)]
    # one rounding to fp32
    assert all(abs(a - b) <= 2 ** -24 * b for a, b in zip(plain.tolist(), want))
    lin, _ = dsa.rope_frequencies(rot, base, "linear", factor, device="cpu")
    assert all(abs(a - b / factor) <= 2 ** -24 * b / factor for a, b in zip(lin.tolist(), want))
    ntk, _ = dsa.rope_frequencies(rot, base, "ntk", factor, device="cpu")
    assert ntk[0] == 1.0
    assert abs(ntk[31].item() * factor / want[31] - 1) < 1e-6       # the lowest: divided by factor
    yarn, m = dsa.rope_frequencies(rot, base, "yarn", factor, length, device="cpu")
    assert abs(m - (0.1 * math.log(factor) + 1)) < 1e-15
    turns = [length * f / (2 * math.pi) for f in want]
    for f, w, n in zip(yarn.tolist(), want, turns):
        if n >= 32 * 1.4:    # one index further than the (floored) border: untouched
            assert abs(f - w) <= 2 ** -24 * w
        elif n <= 1 / 1.4:
            assert abs(f - w / factor) <= 2 ** -23 * w / factor
        else:
            assert w / factor * (1 - 1e-6) <= f <= w * (1 + 1e-6)
    _, m = dsa.rope_frequencies(rot, base, "yarn", factor, length, attention_factor=0.5, device="cpu")
    assert m == 0.5
    for bad in (dict(rot=7), dict(rot=0), dict(rot=64, scaling="dynamic"), dict(rot=64, base=1.0),
                dict(rot=64, factor=0.5), dict(rot=2, scaling="ntk"),
                dict(rot=64, scaling="yarn", beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(ValueError):
            dsa.rope_frequencies(**bad, device="cpu")


@pytest.mark.parametrize("rot,base,length,fast,slow", [
    (64, 10000.0, 4096, 32.0, 1.0),        # both borders among the frequencies
    (64, 10000.0, 65536, 32.0, 1.0),       # the ramp ends behind the last one
    (64, 10000.0, 131072, 32.0, 1.0),
    (64, 500.0, 131072, 32.0, 1.0),        # all of it between the last frequency and rot - 1
    (64, 10000.0, 100, 32.0, 1.0),         # it begins in front of the first one
    (128, 1e6, 32768, 8.0, 0.25),
    (64, 10000.0, 1 << 30, 4.0, 1.0),      # every frequency turns more than beta_fast times
    (32, 10000.0, 4, 32.0, 1.0)])          # every frequency turns less than beta_slow times
def test_yarn_frequencies_against_the_ramp(dsa, rot, base, length, fast, slow):
    """Each frequency against the published ramp: from floor(d(beta_fast)) to ceil(d(beta_slow)), cut
    to [0, rot - 1], where d(n) is the index at which base^(-2d/rot) turns n times in `length`."""
    factor = 8.0
    got = dsa.rope_frequencies(rot, base, "yarn", factor, length, fast, slow, device="cpu")[0].tolist()
    d = lambda n: rot / 2 * math.log(length / (2 * math.pi * n)) / math.log(base)  # noqa: E731
    lo, hi = max(math.floor(d(fast)), 0), min(math.ceil(d(slow)), rot - 1)
    for i, f in enumerate(got):
        w = base ** (-2 * i / rot)
        turns = length * w / (2 * math.pi)
        if turns <= slow:
            t = 1.0
        elif i <= lo:
            t = 0.0
        else:
            t = min(max((i - lo) / (hi - lo), 0.0), 1.0) if hi > lo else 0.0
        want = w * (1.0 - t) + w / factor * t
        # one rounding to fp32, and the 64-bit arithmetic in front of it
        assert abs(f - want) <= 2.0 ** -23 * want, (i, f, want)
        if turns > slow * 1.001 and t < 1.0:
            assert f > w / factor, i          # not fully divided
        if turns <= slow:
            assert f <= w / factor * (1 + 2.0 ** -23), i


def test_latent_refusal_agrees_with_the_library(dsa):
    """What dsa_decode_layer asks before it writes to the cache is what the library then answers. (Its
    calls below are refused: an accepted set of arguments is not given to the library here.)"""
    good = dict(qp=A, cp=A, fmt=1, num_pages=8, page_size=64, tp=A, max_pages=4, lp=A, ip=None, k=0, B=2,
                Sq=1, H=16, Dc=512, Dr=64, scale=0.1, op=A, ep=A, wp=A, ws_bytes=1 << 40)
    assert dsa._latent_refusal(**good) == dsa.DSA_OK
    need = dsa.latent_attn_workspace_bytes(2, 1, 16, 512, 64)
    assert dsa._latent_refusal(**{**good, "ws_bytes": need}) == dsa.DSA_OK
    assert dsa._latent_refusal(**{**good, "scale": 2.0e38}) == dsa.DSA_OK
    bads = [{name: A + 4} for name in ("qp", "cp", "tp", "lp", "op", "ep", "wp")]
    bads += [{name: 0} for name in ("num_pages", "page_size", "max_pages", "B", "Sq", "H")]
    bads += [dict(ip=A + 4, k=4), dict(Dc=256), dict(Dr=0), dict(H=129), dict(scale=0.0),
             dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(scale=2.1e38),
             dict(scale=1e-60), dict(num_pages=1 << 26), dict(max_pages=1 << 26),
             dict(B=1 << 20, Sq=1 << 10), dict(wp=None), dict(ws_bytes=need - 1)]
    for bad in bads:
        args = {**good, **bad}
        want = dsa._latent_refusal(**args)
        assert want != dsa.DSA_OK, bad
        assert dsa.lib.dsa_latent_attn(*args.values(), None) == want, bad


def test_sizes_are_32_bit(dsa):
    dsa._int32(0, -1, 2 ** 31 - 1, -2 ** 31)
    for bad in (2 ** 31, -2 ** 31 - 1, 2 ** 32 + 5):
        with pytest.raises(ValueError):
            dsa._int32(1, bad)
        with pytest.raises(ValueError):
            dsa.cache_row_bytes(512, bad)
