"""Rotary positions, the paged latent cache and the attention over it, against plain definitions in
64 bits.

Tolerances. A rounding to bf16 is off by at most 2^-8 of the value, one to fp32 by 2^-24.

* rope: |y - ref| <= r |ref| + 1e-6 m (|a| + |b|), r the rounding of the output type. The second
  term covers the angle (1.9e-7 rad for its 64-bit fraction at the farthest position, 1.9e-7 for its
  conversion to fp32), the 2 ulp of sine and cosine (2.4e-7) and four fp32 roundings (2.4e-7).
* cache: the same bytes as the definition.
* attention: el bounds the error of a logit: 576 exact products added in fp32, each addition off by
  at most 2^-23 (truncation) of the sum of magnitudes. Weights are exp(l - m) with relative error
  2 el + 2^-18 (both l and m move; the fast exponential and its fp32 argument), rounded to bf16
  (2^-8) for the product with the rows, whose fp32 sums lose at most keys * 2^-23. So
  |O - ref| <= 2^-8 |ref| + (4 el + 2^-8 + 2^-17 + keys 2^-22) sum_j p_j |v_j|
  (numerator and denominator), and |lse - ref| <= 2 el + 2^-17 + keys 2^-23 + 2^-22 |ref|. The
  roundings of the weights are independent of the values, so the norm of the error stays within
  2^-7 of the norm of O.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DC, DR, D = 512, 64, 576


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_index_gb300 as m
    m.dsa_get_last_device_error()
    return m


def no_error(dsa):
    assert dsa.dsa_get_last_device_error() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------------------------- rope


def rope_ref(x, pos, inv_freq, off, rot, layout, mscale, inverse):
    """(ref, |a| + |b| of each rotated element's pair, 0 elsewhere) in 64 bits."""
    x = x.double()
    i = torch.arange(rot // 2, device=x.device)
    a, b = (off + 2 * i, off + 2 * i + 1) if layout == "interleaved" else (off + i, off + rot // 2 + i)
    ang = pos.double()[..., None] * inv_freq.double()
    # turns reduced before the sine, which would itself lose nothing at these sizes
    c, s = torch.cos(ang)[..., None, :], torch.sin(ang)[..., None, :]
    if inverse:
        s = -s
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., a] = mscale * (x[..., a] * c - x[..., b] * s)
    y[..., b] = mscale * (x[..., a] * s + x[..., b] * c)
    mag[..., a] = mag[..., b] = abs(mscale) * (x[..., a].abs() + x[..., b].abs())
    return y, mag


def rope_close(got, ref, mag):
    r = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    err = (got.double() - ref).abs()
    assert bool((err <= r * ref.abs() + 1e-6 * mag).all()), float((err - r * ref.abs() - 1e-6 * mag).max())


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,D_,off,rot", [
    (1, 1, 16, 0, 16), (1, 128, 192, 128, 64), (37, 3, 24, 8, 16), (513, 1, 64, 0, 32),
    (5, 7, 128, 0, 128), (700, 2, 576, 512, 64), (3, 1, 1024, 0, 1024), (129, 16, 40, 24, 16),
    (2, 5, 1000, 8, 992)])
def test_rope(dsa, layout, dtype, T, H, D_, off, rot):
    g = gen(T * 1000 + H)
    x = torch.randn(T, H, D_, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    inv, _ = dsa.rope_frequencies(rot)
    for inverse, m in ((False, 1.0), (True, 1.3688879454113936)):
        ref, mag = rope_ref(x, pos, inv, off, rot, layout, m, inverse)
        y = dsa.dsa_rope(x, pos, inv, off=off, layout=layout, mscale=m, inverse=inverse)
        rope_close(y, ref, mag)
        # dims outside the rotated part are the same bits; in place gives the same bits too
        keep = torch.ones(D_, dtype=torch.bool, device="cuda")
        keep[off:off + rot] = False
        assert torch.equal(y[..., keep], x[..., keep])
        z = x.clone()
        assert dsa.dsa_rope(z, pos, inv, off=off, layout=layout, mscale=m, inverse=inverse,
                            out=z) is z
        assert torch.equal(z, y)
    no_error(dsa)


@pytest.mark.parametrize("layout,rot", [("interleaved", 64), ("half", 64), ("half", 48)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_more_than_l2_holds(dsa, layout, rot, dtype):
    T, H, D_, off = 5003, 37, 192, 128
    g = gen(9)
    x = torch.randn(T, H, D_, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    inv, _ = dsa.rope_frequencies(rot)
    y = dsa.dsa_rope(x, pos, inv, off=off, layout=layout)
    for t0 in range(0, T, 1000):
        part = slice(t0, t0 + 1000)
        ref, mag = rope_ref(x[part], pos[part], inv, off, rot, layout, 1.0, False)
        rope_close(y[part], ref, mag)
    assert torch.equal(y[..., :off], x[..., :off])
    assert torch.equal(y[..., off + rot:], x[..., off + rot:])
    assert torch.equal(dsa.dsa_rope(x, pos, inv, off=off, layout=layout, out=x), y)   # in place
    no_error(dsa)


def test_rope_far_and_negative_positions(dsa):
    pos = i32([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 999999937, 131071])
    x = torch.randn(8, 2, 64, generator=gen(1), device="cuda")
    for rot, scaling in ((64, None), (64, "yarn"), (32, "linear")):
        inv, m = dsa.rope_frequencies(rot, scaling=scaling, factor=32.0)
        ref, mag = rope_ref(x, pos, inv, 0, rot, "half", m, False)
        rope_close(dsa.dsa_rope(x, pos, inv, layout="half", mscale=m), ref, mag)


def test_rope_is_relative_and_its_inverse_is_the_gradient(dsa):
    g = gen(2)
    inv, _ = dsa.rope_frequencies(64)
    T, H = 50, 4
    x = torch.randn(T, H, 192, generator=g, device="cuda")
    dy = torch.randn(T, H, 192, generator=g, device="cuda")
    pos = torch.randint(0, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
    kw = dict(off=128, layout="interleaved", mscale=1.25)
    y = dsa.dsa_rope(x, pos, inv, **kw)
    dx = dsa.dsa_rope(dy, pos, inv, inverse=True, **kw)
    # <dy, J x> = <J^T dy, x>; each side sums 192 H T products with relative errors <= 2e-6
    lhs, rhs = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    scale = (dy.double().abs() * y.double().abs()).sum() + (dx.double().abs() * x.double().abs()).sum()
    assert abs(lhs - rhs) <= 2e-6 * scale
    # against differences: the map is linear, so a step of any size gives the derivative up to
    # the rounding of its two values
    h = torch.randn(T, H, 192, generator=g, device="cuda")
    diff = (dsa.dsa_rope(x + h, pos, inv, **kw).double() - y.double())
    ref, mag = rope_ref((x + h).double() - x.double(), pos, inv, 128, 64, "interleaved", 1.25, False)
    room = 2.0 ** -23 * (y.double().abs() + diff.abs()) + 1e-6 * 4 * (mag + 4)
    assert bool(((diff - ref).abs() <= room).all())
    # scores depend on the distance alone: <R(p) a, R(q) b> = <R(p + s) a, R(q + s) b>
    for s in (1, 4096, 10 ** 9):
        a, b = x[:, :1].contiguous(), dy[:, :1].contiguous()
        p, q = pos % 1000, (pos + 7) % 1000
        dot = lambda u, v: (u.double() * v.double()).sum(-1)  # noqa: E731
        one = dot(dsa.dsa_rope(a, p, inv, off=128), dsa.dsa_rope(b, q, inv, off=128))
        two = dot(dsa.dsa_rope(a, p + s, inv, off=128), dsa.dsa_rope(b, q + s, inv, off=128))
        room = 8e-6 * (a.double().norm(dim=-1) * b.double().norm(dim=-1))
        assert bool(((one - two).abs() <= room).all())


def test_rope_leading_shapes_streams_and_refusals(dsa):
    g = gen(3)
    inv, _ = dsa.rope_frequencies(32)
    x = torch.randn(2, 9, 3, 64, generator=g, device="cuda")
    pos = torch.randint(0, 4096, (2, 9), generator=g, device="cuda", dtype=torch.int32)
    y = dsa.dsa_rope(x, pos, inv, off=32)
    assert torch.equal(y.view(18, 3, 64), dsa.dsa_rope(x.view(18, 3, 64), pos.view(18), inv, off=32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = dsa.dsa_rope(x, pos, inv, off=32, stream=side)
    side.synchronize()
    assert torch.equal(z, y)
    for bad in (dict(pos=pos.view(18)), dict(pos=pos.long()), dict(inv_freq=inv.double()),
                dict(x=x.transpose(0, 1)), dict(out=torch.empty_like(x)[:1]), dict(layout="other"),
                dict(off=40), dict(off=4)):
        kw = dict(x=x, pos=pos, inv_freq=inv, off=32)
        kw.update(bad)
        with pytest.raises((TypeError, ValueError, dsa.DsaError)):
            dsa.dsa_rope(**kw)


# ------------------------------------------------------------------------------------- cache


def e4m3_values():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[(b & 0x7f) == 0x7f] = np.nan
    return np.where(b & 0x80, -v, v)


def encode_ref(kv, Dc, fmt):
    """The bytes of cache rows for kv bf16 [T, Dc + Dr] (CPU tensors), from the definition."""
    T = kv.shape[0]
    raw = kv.view(torch.int16).numpy().view(np.uint8).reshape(T, -1)
    if fmt == "bf16":
        return raw.copy()
    x = kv[:, :Dc].double().numpy().reshape(T, Dc // 128, 128)
    amax = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    with np.errstate(all="ignore"):
        k = np.ceil(np.log2(amax / 448.0))
    k = np.where(amax == 0, 0, np.maximum(k, -120))
    k = np.where(bad, 0, k)
    vals = e4m3_values()
    pos = vals[:127]                                     # 0 .. 448, ascending
    y = np.where(np.isfinite(x), x, 0) / 2.0 ** k[..., None]
    mid = (pos[1:] + pos[:-1]) / 2
    lo = np.searchsorted(mid, np.abs(y), side="left")    # ties to the lower code ...
    tie = (lo < 126) & (np.abs(y) == mid[np.minimum(lo, 125)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo)     # ... unless the upper one is even
    code = (code | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)
    scale = np.where(bad, np.nan, 2.0 ** k).astype(np.float32)
    pad = np.zeros((T, (Dc // 128 + 3) // 4 * 4), np.float32)
    pad[:, :Dc // 128] = scale
    return np.concatenate([code.reshape(T, Dc), pad.view(np.uint8), raw[:, 2 * Dc:]], 1), bad


def cache_inputs(T, Dc, Dr, seed):
    g = torch.Generator().manual_seed(seed)
    kv = torch.randn(T, Dc + Dr, generator=g)
    kv *= torch.exp2(torch.randint(-30, 30, (T, 1), generator=g).float())
    return kv.to(torch.bfloat16)


@pytest.mark.parametrize("Dc,Dr", [(512, 64), (128, 0), (128, 64), (640, 8), (1024, 256), (256, 136)])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("T", [1, 7, 130])
def test_cache_write_and_read(dsa, Dc, Dr, fmt, T):
    kv = cache_inputs(T, Dc, Dr, T + Dc)
    if T == 7:   # a group of zeros, one of the largest values, one of the smallest
        kv[1, :128] = 0
        kv[2, :128] = torch.finfo(torch.bfloat16).max
        kv[3, :128] = 2.0 ** -133
        kv[4, :128] = -448.0
    pages, page = 9, 19
    row = dsa.cache_row_bytes(Dc, Dr, fmt)
    start = torch.randint(0, 256, (pages, page, row), dtype=torch.uint8)
    cache = start.cuda()
    slots = torch.randperm(pages * page)[:T].to(torch.int32)
    if T > 1:
        slots[T // 2] = -1
    assert dsa.dsa_cache_write(kv.cuda(), slots.cuda(), cache, Dc, fmt=fmt) is cache
    want = start.view(-1, row).clone().numpy()
    ref = encode_ref(kv, Dc, fmt)
    ref = ref if fmt == "bf16" else ref[0]
    live = slots.numpy() >= 0
    want[slots.numpy()[live]] = ref[live]
    assert np.array_equal(cache.view(-1, row).cpu().numpy(), want)   # every other byte unchanged
    back = dsa.dsa_cache_read(cache, slots.cuda(), Dc, Dr, fmt=fmt).double().cpu().numpy()
    x = kv.double().numpy()
    assert np.array_equal(back[~live], np.zeros_like(back[~live]))
    if fmt == "bf16":
        assert np.array_equal(back[live], x[live])
    else:
        assert np.array_equal(back[:, Dc:][live], x[:, Dc:][live])
        sc = np.repeat(ref[:, Dc:Dc + 4 * (Dc // 128)].copy().view(np.float32).astype(np.float64), 128, 1)
        exact = e4m3_values()[ref[:, :Dc]] * sc
        # exact in bf16, but for what rounds up past its largest value (2^128)
        with np.errstate(invalid="ignore"):   # NaN codes in the rows that were skipped
            held = np.where(np.abs(exact) < 2.0 ** 128, exact, np.sign(exact) * np.inf)
        assert np.array_equal(back[:, :Dc][live], held[live])
        err = np.abs(exact - x[:, :Dc])
        assert (err <= np.maximum(2.0 ** -4 * np.abs(x[:, :Dc]), 2.0 ** -10 * sc)).all()
    # repeats are allowed when reading
    twice = torch.cat([slots, slots]).cuda()
    again = dsa.dsa_cache_read(cache, twice, Dc, Dr, fmt=fmt).double().cpu().numpy()
    assert np.array_equal(again[:T], back) and np.array_equal(again[T:], back)
    no_error(dsa)


def test_cache_values_that_are_not_finite(dsa):
    kv = cache_inputs(4, 512, 64, 5)
    kv[0, 3] = math.inf
    kv[1, 200] = math.nan
    kv[2, 511] = -math.inf
    kv[3, 512 + 9] = math.nan          # a positional dim: kept as it is
    cache = torch.zeros(1, 4, 656, dtype=torch.uint8, device="cuda")
    slots = i32([0, 1, 2, 3])
    dsa.dsa_cache_write(kv.cuda(), slots, cache, 512)
    back = dsa.dsa_cache_read(cache, slots, 512, 64).float().cpu()
    nan = torch.isnan(back)
    want = torch.zeros_like(nan)
    want[0, :128] = want[1, 128:256] = want[2, 384:512] = True
    want[3, 512 + 9] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_cache_many_rows(dsa, fmt):
    """Many rows in one call give the bytes and values of calls of a few hundred each."""
    T, page = 18003, 16
    g = gen(71)
    kv = torch.randn(T, D, generator=g, device="cuda").to(torch.bfloat16)
    shape = (T // page + 3, page, dsa.cache_row_bytes(DC, DR, fmt))
    slots = torch.randperm(shape[0] * page, generator=g, device="cuda")[:T].to(torch.int32)
    slots[::97] = -1
    one = torch.full(shape, 0x5a, dtype=torch.uint8, device="cuda")
    many = one.clone()
    dsa.dsa_cache_write(kv, slots, one, DC, fmt=fmt)
    back = dsa.dsa_cache_read(one, slots, DC, DR, fmt=fmt)
    for t0 in range(0, T, 400):
        part = slice(t0, t0 + 400)
        dsa.dsa_cache_write(kv[part], slots[part], many, DC, fmt=fmt)
        assert torch.equal(dsa.dsa_cache_read(many, slots[part], DC, DR, fmt=fmt), back[part])
    assert torch.equal(one, many)
    assert not back[::97].any()
    no_error(dsa)


def test_cache_bad_slots(dsa):
    """A slot outside the cache is recorded and skipped, the others are served."""
    kv = cache_inputs(5, 512, 64, 6).cuda()
    for fmt in ("bf16", "e4m3"):
        row = dsa.cache_row_bytes(512, 64, fmt)
        cache = torch.full((2, 3, row), 7, dtype=torch.uint8, device="cuda")
        dsa.dsa_cache_write(kv, i32([5, 6, -2, 0, 2 ** 31 - 1]), cache, 512, fmt=fmt)
        assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_CACHE | dsa.DSA_DEVERR_BAD_INDEX
        untouched = cache.view(6, row)[1:5]
        assert bool((untouched == 7).all())
        got = dsa.dsa_cache_read(cache, i32([0, 5, -1]), 512, 64, fmt=fmt)
        no_error(dsa)
        bad = dsa.dsa_cache_read(cache, i32([0, 6, 5, -7]), 512, 64, fmt=fmt)
        assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_CACHE | dsa.DSA_DEVERR_BAD_INDEX
        assert torch.equal(bad[0], got[0]) and torch.equal(bad[2], got[1])
        assert not bad[1].any() and not bad[3].any() and not got[2].any()


# --------------------------------------------------------------------------------- attention


def make_cache(dsa, lens, page, fmt, seed, scale=1.0, spare=2):
    """A paged cache holding random rows for each sequence, its pages shuffled; the rows behind
    each sequence and the spare pages hold NaN. -> (cache, table, rows fp64 by sequence)."""
    g = gen(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g, device="cuda").tolist()
    row = dsa.cache_row_bytes(DC, DR, fmt)
    cache = torch.full((total, page, row), 0xff, dtype=torch.uint8, device="cuda")   # NaN everywhere
    table = torch.full((len(lens), max(max(need), 1) + 1), 2 ** 30, dtype=torch.int32)  # never read
    rows, first = [], 0
    for b, n in enumerate(lens):
        mine = order[first:first + need[b]]
        first += need[b]
        table[b, :need[b]] = torch.tensor(mine, dtype=torch.int32)
        n = max(n, 0)
        kv = (torch.randn(n, D, generator=g, device="cuda") * scale).to(torch.bfloat16)
        if n:
            at = torch.arange(n)
            slots = (torch.tensor(mine)[at // page] * page + at % page).to(torch.int32).cuda()
            dsa.dsa_cache_write(kv, slots, cache, DC, fmt=fmt)
            kv = dsa.dsa_cache_read(cache, slots, DC, DR, fmt=fmt)
        rows.append(kv.double())
    return cache, table.cuda(), rows


def attn_check(O, lse, Q, rows, lens, scale, idx=None):
    """Holds (O, lse) to the definition in 64 bits within the tolerances above."""
    B, Sq, H, _ = Q.shape
    err2 = ref2 = 0.0
    for b in range(B):
        n = max(int(lens[b]), 0)
        for i in range(Sq):
            lim = n - Sq + i + 1
            keys = rows[b][:max(lim, 0)]
            if idx is not None:
                t = idx[b, i].long()
                keys = rows[b][t[(t >= 0) & (t < lim)]]
            got, gl = O[b, i].double(), lse[b, i].double()
            if len(keys) == 0:
                assert not got.any() and bool((gl == -math.inf).all())
                continue
            q = Q[b, i].double()
            l = scale * (q @ keys.T)
            ref_l = torch.logsumexp(l, -1)
            p = torch.exp(l - ref_l[:, None])
            ref = p @ keys[:, :DC]
            el = D * 2.0 ** -23 * scale * (q.abs() @ keys.abs().T).amax(-1)
            pv = p @ keys[:, :DC].abs()
            nk = len(keys)
            tol = 2.0 ** -8 * ref.abs() + (4 * el[:, None] + 2.0 ** -8 + 2.0 ** -17 + nk * 2.0 ** -22) * pv
            assert bool(((got - ref).abs() <= tol).all()), (b, i, float(((got - ref).abs() / tol).max()))
            assert bool(((gl - ref_l).abs() <= 2 * el + 2.0 ** -17 + nk * 2.0 ** -23
                         + 2.0 ** -22 * ref_l.abs()).all()), (b, i, float((gl - ref_l).abs().max()))
            err2 += float(((got - ref) ** 2).sum())
            ref2 += float((ref ** 2).sum())
    assert err2 <= (2.0 ** -7) ** 2 * ref2, math.sqrt(err2 / max(ref2, 1e-300))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,Sq,H,lens,page", [
    (1, 1, 1, [1], 16), (1, 1, 128, [1], 1), (1, 1, 16, [489], 64), (3, 1, 128, [47, 48, 49], 7),
    (4, 1, 20, [0, 1, 97, 0], 16), (2, 4, 16, [3, 130], 16), (2, 3, 128, [2, 700], 100),
    (1, 7, 5, [7], 64), (5, 2, 64, [96, 1000, 1, 31, 2049], 32), (1, 1, 128, [20000], 64),
    (2, 1, 33, [-5, 64], 16), (1, 70, 3, [200], 16)])
def test_latent_attn(dsa, fmt, B, Sq, H, lens, page):
    cache, table, rows = make_cache(dsa, lens, page, fmt, 11)
    no_error(dsa)
    Q = torch.randn(B, Sq, H, D, generator=gen(12), device="cuda").to(torch.bfloat16)
    scale = 192 ** -0.5
    O = torch.full((B, Sq, H, DC), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Sq, H), math.nan, device="cuda")
    dsa.dsa_latent_attn(Q, cache, table, i32(lens), scale, fmt=fmt, O=O, lse=lse)
    want = dsa.DSA_STAGE_LATENT | dsa.DSA_DEVERR_BAD_PAGE if min(lens) < 0 else 0
    assert dsa.dsa_get_last_device_error() == want
    attn_check(O, lse, Q, rows, lens, scale)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("Sq,H,page", [(1, 128, 64), (2, 100, 48), (4, 16, 100)])
def test_latent_attn_many_ragged(dsa, fmt, Sq, H, page):
    """Enough keys that several tiles lie in one cluster's range and one tile in several."""
    lens = [9000 - 371 * b if b % 6 else (0, 1, 30011, 48)[b // 6 % 4] for b in range(24)]
    cache, table, rows = make_cache(dsa, lens, page, fmt, 81)
    Q = torch.randn(24, Sq, H, D, generator=gen(82), device="cuda").to(torch.bfloat16)
    O, lse = dsa.dsa_latent_attn(Q, cache, table, i32(lens), 192 ** -0.5, fmt=fmt)
    no_error(dsa)
    attn_check(O, lse, Q, rows, lens, 192 ** -0.5)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,Sq,H,lens,k", [
    (1, 1, 128, [300], 1), (2, 1, 16, [64, 5000], 48), (3, 2, 128, [1, 0, 777], 100),
    (1, 1, 7, [40], 64), (40, 1, 128, [2500] * 40, 2048), (1, 130, 2, [130], 33),
    (2, 5, 64, [900, 3], 17)])
def test_latent_attn_selected(dsa, fmt, B, Sq, H, lens, k):
    """Lists as the top-k gives them (ascending, -1 behind), and lists with holes, entries above
    the diagonal and rows that list nothing."""
    cache, table, rows = make_cache(dsa, lens, 64, fmt, 21)
    g = gen(22)
    Q = torch.randn(B, Sq, H, D, generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.full((B, Sq, k), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for i in range(Sq):
            lim = n - Sq + i + 1
            pick = torch.randperm(max(n if (i + b) % 3 == 1 else lim, 0))[:k].sort().values
            idx[b, i, :len(pick)] = pick.to(torch.int32)
            if (i + b) % 3 == 2:
                idx[b, i, ::2] = -1
            if (i + b) % 7 == 6:
                idx[b, i] = -1
    idx = idx.cuda()
    O, lse = dsa.dsa_latent_attn(Q, cache, table, i32(lens), 192 ** -0.5, fmt=fmt, idx=idx)
    no_error(dsa)
    attn_check(O, lse, Q, rows, lens, 192 ** -0.5, idx)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_latent_attn_bad_lists_pages_and_lengths(dsa, fmt):
    """What points outside the cache is recorded and skipped; the rest of the row is computed."""
    lens = [200, 100]
    cache, table, rows = make_cache(dsa, lens, 16, fmt, 31)
    Q = torch.randn(2, 1, 16, D, generator=gen(32), device="cuda").to(torch.bfloat16)
    idx = i32([[[3, 5, 200, 9, -2, 2 ** 31 - 1, -1, 199]], [[0, 1, 2, 99, 100, -1, -1, -1]]])
    O, lse = dsa.dsa_latent_attn(Q, cache, table, i32(lens), 0.07, fmt=fmt, idx=idx)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_LATENT | dsa.DSA_DEVERR_BAD_INDEX
    ok = idx.clone()
    ok[(ok >= i32(lens)[:, None, None]) | (ok < -1)] = -1
    attn_check(O, lse, Q, rows, lens, 0.07, ok)
    # a page outside the cache: its 16 keys are not there
    bad = table.clone()
    bad[0, 2], bad[1, 6] = -3, cache.shape[0]
    O, lse = dsa.dsa_latent_attn(Q, cache, bad, i32(lens), 0.07, fmt=fmt)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_LATENT | dsa.DSA_DEVERR_BAD_PAGE
    left = [torch.cat([rows[0][:32], rows[0][48:]]), rows[1][:96]]
    attn_check(O, lse, Q, left, [len(x) for x in left], 0.07)
    # a length behind the page table is cut to it
    full = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    dsa.dsa_cache_write(rows[0][:64].to(torch.bfloat16), i32(range(64)), cache, DC, fmt=fmt)
    kept = dsa.dsa_cache_read(cache, i32(range(64)), DC, DR, fmt=fmt).double()
    O, lse = dsa.dsa_latent_attn(Q[:1], cache, full, i32([10 ** 9]), 0.07, fmt=fmt)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_LATENT | dsa.DSA_DEVERR_BAD_PAGE
    attn_check(O, lse, Q[:1], [kept], [64], 0.07)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_latent_attn_large_and_small_logits(dsa, fmt):
    """Logits far apart (the running maximum moves by more than any exponent holds), all equal, and
    a key far above the rest at the very end."""
    n = 700
    cache, table, rows = make_cache(dsa, [n], 64, fmt, 41)
    Q = torch.randn(1, 1, 16, D, generator=gen(42), device="cuda")
    Q[0, 0, 0] = 0.0
    Q[0, 0, 1] = rows[0][n - 1] * 4
    Q[0, 0, 2] = rows[0][0] * 4
    Q[0, 0, 3] = -rows[0][n - 1] * 4
    Q[0, 0, 4:8] *= 1e-3
    Q = Q.to(torch.bfloat16)
    for scale in (0.07, 3.0):
        O, lse = dsa.dsa_latent_attn(Q, cache, table, i32([n]), scale, fmt=fmt)
        attn_check(O, lse, Q, rows, [n], scale)
    # all logits zero: n weights of one
    assert bool((lse[0, 0, 0] - math.log(n)).abs() <= 2.0 ** -17 + n * 2.0 ** -23)


def test_latent_attn_non_finite_rows_outside(dsa):
    """NaN in rows behind the sequence, in unlisted rows and in pages of others changes nothing;
    an infinity in a seen row shows in the result of that sequence alone."""
    lens = [100, 90]
    cache, table, rows = make_cache(dsa, lens, 64, "bf16", 51)
    Q = torch.randn(2, 1, 16, D, generator=gen(52), device="cuda").to(torch.bfloat16)
    O, lse = dsa.dsa_latent_attn(Q, cache, table, i32(lens), 0.07, fmt="bf16")
    attn_check(O, lse, Q, rows, lens, 0.07)
    at = int(table[0, 0]) * 64 + 5
    bad = cache.clone().view(-1, 1152).view(torch.bfloat16)
    bad[at, 3] = math.nan
    bad = bad.view(torch.uint8).view_as(cache)
    O2, lse2 = dsa.dsa_latent_attn(Q, bad, table, i32(lens), 0.07, fmt="bf16")
    assert torch.equal(O2[1], O[1]) and torch.equal(lse2[1], lse[1])
    assert bool(torch.isnan(lse2[0]).all()) and bool(torch.isnan(O2[0]).all())
    idx = i32([[[0, 1, 2, 3, 4, 6, 7, -1]], [[0, 1, 2, 3, 4, 5, 6, 7]]])
    O3, lse3 = dsa.dsa_latent_attn(Q, bad, table, i32(lens), 0.07, fmt="bf16", idx=idx)
    attn_check(O3, lse3, Q, rows, lens, 0.07, idx)


@pytest.mark.parametrize("H", [16, 128])
@pytest.mark.parametrize("group", [0, 1, 2, 3])
def test_latent_attn_wide_and_nan_scales(dsa, group, H):
    """e4m3 rows of which one group of 128 dims has scales from 2^-108 to 2^106 and Q is zero there,
    so that the weights stay ordinary ones; and a row whose group is NaN, seen and not listed."""
    n, dims = 330, slice(128 * group, 128 * group + 128)
    g = gen(61)
    kv = torch.randn(n, D, generator=g, device="cuda")
    shift = torch.tensor([0, 15, 16, 17, 18, 60, 112, -100])[torch.arange(n) % 8]
    kv[:, dims] *= torch.exp2(shift.float())[:, None].cuda()
    cache = torch.full((8, 64, dsa.cache_row_bytes(DC, DR, "e4m3")), 0xff, dtype=torch.uint8,
                       device="cuda")
    table = i32([[7, 2, 0, 5, 3, 6]])
    at = torch.arange(n, device="cuda")
    slots = (table[0][at // 64] * 64 + at % 64).to(torch.int32)
    dsa.dsa_cache_write(kv.to(torch.bfloat16), slots, cache, DC, fmt="e4m3")
    rows = [dsa.dsa_cache_read(cache, slots, DC, DR, fmt="e4m3").double()]
    Q = torch.randn(1, 1, H, D, generator=g, device="cuda")
    Q[..., dims] = 0.0
    Q = Q.to(torch.bfloat16)
    O, lse = dsa.dsa_latent_attn(Q, cache, table, i32([n]), 0.07, fmt="e4m3")
    no_error(dsa)
    attn_check(O, lse, Q, rows, [n], 0.07)
    # a group of NaN: all of a row that sees it, nothing of a row that does not list it
    kv[5, dims.start + 77] = math.nan
    dsa.dsa_cache_write(kv[5:6].to(torch.bfloat16), slots[5:6].clone(), cache, DC, fmt="e4m3")
    O, lse = dsa.dsa_latent_attn(Q, cache, table, i32([n]), 0.07, fmt="e4m3")
    assert bool(torch.isnan(O).all()) and bool(torch.isnan(lse).all())
    idx = i32([[[j for j in range(n) if j != 5]]])
    O, lse = dsa.dsa_latent_attn(Q, cache, table, i32([n]), 0.07, fmt="e4m3", idx=idx)
    no_error(dsa)
    attn_check(O, lse, Q, rows, [n], 0.07, idx)


def test_latent_attn_same_bits_every_time_and_on_any_stream(dsa):
    """No atomics: repeated, concurrent (own workspaces) and captured calls give the same bits."""
    lens = [3000, 1, 700]
    cache, table, _ = make_cache(dsa, lens, 64, "e4m3", 61)
    Q = torch.randn(3, 2, 32, D, generator=gen(62), device="cuda").to(torch.bfloat16)
    n = i32(lens)
    O, lse = dsa.dsa_latent_attn(Q, cache, table, n, 0.07)
    torch.cuda.synchronize()
    outs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                outs.append(dsa.dsa_latent_attn(Q, cache, table, n, 0.07))
    torch.cuda.synchronize()
    for o, e in outs:
        assert torch.equal(o, O) and torch.equal(e, lse)
    ws = torch.empty(max(dsa.latent_attn_workspace_bytes(3, 2, 32, DC, DR), 16), dtype=torch.uint8,
                     device="cuda")
    graphs, got = [], []
    for _ in range(2):   # two graphs on one workspace, replayed in turn
        g = torch.cuda.CUDAGraph()
        o, e = torch.empty_like(O), torch.empty_like(lse)
        with torch.cuda.graph(g):
            dsa.dsa_latent_attn(Q, cache, table, n, 0.07, O=o, lse=e, ws=ws)
        graphs.append(g)
        got.append((o, e))
    for _ in range(3):
        ws.fill_(0xff)
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, e in got:
        assert torch.equal(o, O) and torch.equal(e, lse)
    # a replay reads the lengths and the table of that moment
    n.copy_(i32([5, 3000 // 64 * 64 + 1, 0]))
    table[1, :47] = table[0, :47].clone()
    graphs[0].replay()
    torch.cuda.synchronize()
    O2, lse2 = dsa.dsa_latent_attn(Q, cache, table, n, 0.07)
    assert torch.equal(O2, got[0][0]) and torch.equal(lse2, got[0][1])
    no_error(dsa)


def test_latent_attn_slots_past_32_bits(dsa):
    """A cache of more than 2^31 bytes: rows at its far end."""
    page, pages = 64, 60000   # 60000 * 64 * 1152 bytes = 4.4e9
    cache = torch.empty(pages, page, 1152, dtype=torch.uint8, device="cuda")
    table = i32([[pages - 1, pages - 2, 0]])
    n = 150
    kv = torch.randn(n, D, generator=gen(71), device="cuda").to(torch.bfloat16)
    at = torch.arange(n, device="cuda")
    slots = (table[0].long()[at // page] * page + at % page).to(torch.int32)
    dsa.dsa_cache_write(kv, slots, cache, DC, fmt="bf16")
    assert torch.equal(dsa.dsa_cache_read(cache, slots, DC, DR, fmt="bf16"), kv)
    Q = torch.randn(1, 1, 16, D, generator=gen(72), device="cuda").to(torch.bfloat16)
    O, lse = dsa.dsa_latent_attn(Q, cache, table, i32([n]), 0.07, fmt="bf16")
    no_error(dsa)
    attn_check(O, lse, Q, [kv.double()], [n], 0.07)


def test_latent_attn_refusals(dsa):
    cache, table, _ = make_cache(dsa, [64], 64, "e4m3", 81)
    Q = torch.zeros(1, 1, 16, D, dtype=torch.bfloat16, device="cuda")
    good = dict(Q=Q, cache=cache, page_table=table, lens=i32([64]), scale=0.1)
    dsa.dsa_latent_attn(**good)
    idx = i32([[[0, 1]]])
    for bad in (dict(fmt="bf16"), dict(fmt="fp4"), dict(scale=0.0), dict(lens=i32([64, 64])),
                dict(lens=i32([64]).long()), dict(page_table=table[0]), dict(Q=Q.float()),
                dict(Q=Q[..., :500].contiguous()), dict(Q=torch.cat([Q] * 9, 2)),
                dict(cache=cache.view(-1, 656)), dict(idx=idx[..., :0]), dict(idx=idx[0]),
                dict(idx=idx.long()), dict(lens=i32([64]).cpu()), dict(O=Q), dict(Dc=256),
                dict(Q=Q.expand(1, 2, 16, D)), dict(lse=torch.empty(1, 16, 1, device="cuda"))):
        with pytest.raises((TypeError, ValueError, dsa.DsaError)):
            dsa.dsa_latent_attn(**{**good, **bad})
    no_error(dsa)


# --------------------------------------------------------------------------- used together


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_decode_steps(dsa, fmt):
    """A prompt, then tokens one by one: rotary positions into the rows, the rows into the cache,
    attention over it; each token against the same attention computed from scratch."""
    B, H, page, steps = 3, 16, 16, 4
    prompt = [33, 1, 64]
    inv, m = dsa.rope_frequencies(DR, scaling="yarn", factor=4.0)
    g = gen(91)
    total = [p + steps for p in prompt]
    raw = [torch.randn(n, 1, D, generator=g, device="cuda").to(torch.bfloat16) for n in total]
    table = torch.arange(B * 5, dtype=torch.int32, device="cuda").flip(0).view(B, 5)
    cache = torch.zeros(B * 5, page, dsa.cache_row_bytes(DC, DR, fmt), dtype=torch.uint8, device="cuda")

    def store(b, first, last):
        pos = torch.arange(first, last, dtype=torch.int32, device="cuda")
        kv = dsa.dsa_rope(raw[b][first:last].contiguous(), pos, inv, off=DC, mscale=m)
        slots = (table[b].long()[pos.long() // page] * page + pos % page).to(torch.int32)
        dsa.dsa_cache_write(kv.view(-1, D), slots, cache, DC, fmt=fmt)
        return slots

    all_slots = [[store(b, 0, prompt[b])] for b in range(B)]
    for s in range(steps):
        lens = [p + s + 1 for p in prompt]
        for b in range(B):
            all_slots[b].append(store(b, lens[b] - 1, lens[b]))
        q = torch.randn(B, 1, H, D, generator=g, device="cuda").to(torch.bfloat16)
        q = dsa.dsa_rope(q, i32([[n - 1] for n in lens]), inv, off=DC, mscale=m)
        O, lse = dsa.dsa_latent_attn(q, cache, table, i32(lens), 192 ** -0.5, fmt=fmt)
        rows = [dsa.dsa_cache_read(cache, torch.cat(all_slots[b]), DC, DR, fmt=fmt).double()
                for b in range(B)]
        attn_check(O, lse, q, rows, lens, 192 ** -0.5)
    no_error(dsa)


def test_prompt_with_the_selection_of_the_top_k(dsa):
    """A prompt in the absorbed form: the indexer's scores and the top-k of the whole sequence
    give the lists, all of its tokens attend as the newest ones of the sequence."""
    S, H, k = 200, 8, 32
    g = gen(95)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    scores = dsa.dsa_index_scores(bf(1, S, 64, 128), bf(1, S, 128),
                                  torch.rand(1, S, 64, generator=g, device="cuda"))
    idx, _ = dsa.dsa_topk(scores, k, S=S)
    cache, table, rows = make_cache(dsa, [S], 64, "bf16", 96)
    Q = bf(1, S, H, D)
    O, lse = dsa.dsa_latent_attn(Q, cache, table, i32([S]), 192 ** -0.5, fmt="bf16", idx=idx)
    no_error(dsa)
    attn_check(O, lse, Q, rows, [S], 192 ** -0.5, idx)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("side", [False, True])
def test_decode_layer(dsa, fmt, side):
    """One serving step gives what its parts give, in a padded batch, on any stream."""
    B, Sq, H, page, lens = 4, 2, 16, 16, [37, 0, 2, 160]
    cache, table, rows = make_cache(dsa, lens, page, fmt, 101)
    inv, m = dsa.rope_frequencies(DR, scaling="yarn", factor=8.0)
    g = gen(102)
    Q = torch.randn(B, Sq, H, D, generator=g, device="cuda").to(torch.bfloat16)
    kv = torch.randn(B, Sq, D, generator=g, device="cuda").to(torch.bfloat16)
    n = i32(lens)
    pos = (n[:, None] - Sq + torch.arange(Sq, device="cuda")).clamp(min=0).to(torch.int32)
    at = pos.long()
    slots = (table.long().gather(1, at // page) * page + at % page).to(torch.int32)
    slots[1] = -1                                    # the padded sequence
    Q0, kv0 = Q.clone(), kv.clone()
    one = cache.clone()
    stream = None
    if side:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
    O, lse = dsa.dsa_decode_layer(Q, kv, pos, inv, slots, one, table, n, 0.07, fmt=fmt, mscale=m,
                                  stream=stream)
    if side:
        torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(Q, Q0) and torch.equal(kv, kv0)
    rot = dsa.dsa_rope(kv[:, :, None].contiguous(), pos, inv, off=DC, mscale=m)
    dsa.dsa_cache_write(rot.view(-1, D), slots.view(-1), cache, DC, fmt=fmt)
    q = dsa.dsa_rope(Q, pos, inv, off=DC, mscale=m)
    O2, lse2 = dsa.dsa_latent_attn(q, cache, table, n, 0.07, fmt=fmt)
    assert torch.equal(one, cache) and torch.equal(O, O2) and torch.equal(lse, lse2)
    no_error(dsa)
    assert not O[1].any() and bool((lse[1] == -math.inf).all())
    new = dsa.dsa_cache_read(cache, slots.view(-1), DC, DR, fmt=fmt).double().view(B, Sq, D)
    for b, k in enumerate(lens):
        if k:
            rows[b][k - Sq:] = new[b]
    attn_check(O, lse, q, rows, lens, 0.07)


def test_concurrent_calls(dsa):
    """Two streams with a workspace each, e4m3 calls on one and bf16 calls on the other at once."""
    cases = []
    for fmt, H, lens in (("e4m3", 128, [5000, 300]), ("bf16", 16, [7, 2000, 64])):
        cache, table, rows = make_cache(dsa, lens, 64, fmt, 111)
        Q = torch.randn(len(lens), 1, H, D, generator=gen(112), device="cuda").to(torch.bfloat16)
        cases.append((Q, cache, table, i32(lens), fmt, rows, lens))
    wss = [torch.empty(dsa.latent_attn_workspace_bytes(c[0].shape[0], 1, c[0].shape[2], DC, DR),
                       dtype=torch.uint8, device="cuda") for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for _ in range(5):
        for st, ws, (Q, cache, table, n, fmt, _, _) in zip(streams, wss, cases):
            O = torch.empty(*Q.shape[:3], DC, dtype=torch.bfloat16, device="cuda")
            outs.append((O, torch.empty(Q.shape[:3], device="cuda")))
    torch.cuda.synchronize()
    for i, (O, lse) in enumerate(outs):
        Q, cache, table, n, fmt, _, _ = cases[i % 2]
        dsa.dsa_latent_attn(Q, cache, table, n, 0.07, fmt=fmt, O=O, lse=lse, ws=wss[i % 2],
                            stream=streams[i % 2])
    torch.cuda.synchronize()
    for i, (O, lse) in enumerate(outs):
        assert torch.equal(O, outs[i % 2][0]) and torch.equal(lse, outs[i % 2][1])
    for (O, lse), (Q, _, _, _, _, rows, lens) in zip(outs, cases):
        attn_check(O, lse, Q, rows, lens, 0.07)
    no_error(dsa)


@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_calls_on_another_stream(dsa, handle):
    """Workspaces and outputs that a call on a side stream allocates are not handed to work that is
    queued on the current stream meanwhile."""
    lens = [4000, 900]
    cache, table, rows = make_cache(dsa, lens, 64, "bf16", 121)
    Q = torch.randn(2, 1, 128, D, generator=gen(122), device="cuda").to(torch.bfloat16)
    n = i32(lens)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    size = dsa.latent_attn_workspace_bytes(2, 1, 128, DC, DR)
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        outs.append(dsa.dsa_latent_attn(Q, cache, table, n, 0.07, fmt="bf16", stream=stream))
        for _ in range(3):
            torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")   # on the current stream
    torch.cuda.synchronize()
    for O, lse in outs:
        assert torch.equal(O, outs[0][0]) and torch.equal(lse, outs[0][1])
    attn_check(*outs[0], Q, rows, lens, 0.07)
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [100, 5000])
def test_latent_attn_logits_past_fp32(dsa, fmt, n):
    """Logits whose product with scale, or with scale log2(e), is past fp32, from finite Q . row: the
    differences decide, and lse is the nearest fp32 (an infinity where it is past its range). Dim 0 of
    the keys is +-2^10 and Q is zero elsewhere, so that the weights are 0 and 1 exactly; the
    sums of at most n rows lose n * 2^-23 of their magnitudes, O one rounding to bf16."""
    cache, table, _ = make_cache(dsa, [n], 64, fmt, 131)
    kv = torch.randn(n, D, generator=gen(132), device="cuda")
    up = torch.arange(n, device="cuda") % 3 != 0
    kv[:, 0] = torch.where(up, 1024.0, -1024.0)
    at = torch.arange(n, device="cuda")
    slots = (table[0].long()[at // 64] * 64 + at % 64).to(torch.int32)
    dsa.dsa_cache_write(kv.to(torch.bfloat16), slots, cache, DC, fmt=fmt)
    rows = dsa.dsa_cache_read(cache, slots, DC, DR, fmt=fmt).double()
    assert bool((rows[:, 0].abs() == 1024).all())
    q0 = [2.0 ** 100, -2.0 ** 100, 0.0, 2.0 ** 60]
    Q = torch.zeros(1, 1, 4, D, dtype=torch.bfloat16, device="cuda")
    Q[0, 0, :, 0] = torch.tensor(q0)
    for scale in (1.5 * 2.0 ** 17, 2.0 ** 30, 2.0 ** 127):
        O, lse = dsa.dsa_latent_attn(Q, cache, table, i32([n]), scale, fmt=fmt)
        no_error(dsa)
        for h, q in enumerate(q0):
            seen = rows if q == 0 else rows[up if q > 0 else ~up]
            ref, mag = seen[:, :DC].mean(0), seen[:, :DC].abs().mean(0)
            err = (O[0, 0, h].double() - ref).abs()
            assert bool((err <= 2.0 ** -8 * ref.abs() + n * 2.0 ** -22 * mag).all()), (scale, h)
            want = abs(q) * 1024 * scale + math.log(len(seen))
            got = float(lse[0, 0, h])
            if want > torch.finfo(torch.float32).max:
                assert got == math.inf, (scale, h, got)
            else:
                assert abs(got - want) <= 2.0 ** -21 * want, (scale, h, got, want)
    # every logit far below zero: still the mean, not the zeros of a token without a key
    neg = torch.zeros(1, 1, 4, D, dtype=torch.bfloat16, device="cuda")
    neg[..., 0] = -2.0 ** 100
    idx = torch.nonzero(up)[:, 0].to(torch.int32).view(1, 1, -1).contiguous()
    O, lse = dsa.dsa_latent_attn(neg, cache, table, i32([n]), 1.5 * 2.0 ** 17, fmt=fmt, idx=idx)
    seen = rows[up][:, :DC]
    err = (O[0, 0].double() - seen.mean(0)).abs()
    assert bool((err <= 2.0 ** -8 * seen.mean(0).abs() + n * 2.0 ** -22 * seen.abs().mean(0)).all())
    want = -1.5 * 2.0 ** 127 + math.log(len(seen))
    assert bool(((lse.double() - want).abs() <= 2.0 ** -21 * abs(want)).all())
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("Sq,H,lens", [
    (2, 16, [100, 49]), (4, 16, [49, 3, 500]), (7, 5, [7, 96]), (3, 128, [2, 50, 4000]),
    (70, 3, [200]), (4, 33, [20011])])
def test_latent_attn_non_finite_rows_behind_a_token(dsa, fmt, Sq, H, lens):
    """A NaN in the row of a new token, or an infinity that gives a logit of +inf, reaches that token and
    the later ones, and none in front of it."""
    cache, table, rows = make_cache(dsa, lens, 16, fmt, 141)
    Q = torch.randn(len(lens), Sq, H, D, generator=gen(142), device="cuda").to(torch.bfloat16)
    for j, dim, value in ((Sq - 1, 3, math.nan), (1, 300, math.nan), (Sq // 2, 511, math.inf),
                          (Sq - 1, 0, -math.inf), (1, 530, math.nan), (Sq - 1, 575, math.inf)):
        bad = cache.clone()
        kv = torch.randn(len(lens), D, generator=gen(143), device="cuda").to(torch.bfloat16)
        kv[:, dim] = value
        at = torch.tensor([n - Sq + j for n in lens], device="cuda")
        slots = (table.long().gather(1, (at.clamp(min=0) // 16)[:, None])[:, 0] * 16 + at % 16)
        slots = torch.where(at >= 0, slots, -1).to(torch.int32)
        dsa.dsa_cache_write(kv, slots, bad, DC, fmt=fmt)
        O, lse = dsa.dsa_latent_attn(Q, bad, table, i32(lens), 0.07, fmt=fmt)
        no_error(dsa)
        attn_check(O[:, :j], lse[:, :j], Q[:, :j], rows, [n - (Sq - j) for n in lens], 0.07)
        for b, n in enumerate(lens):
            for i in range(j, Sq):
                if n - Sq + j < 0:       # no such row
                    continue
                if math.isnan(value) or (fmt == "e4m3" and dim < DC):
                    assert bool(O[b, i].isnan().all()) and bool(lse[b, i].isnan().all()), (b, i)
                else:    # a logit of +inf; one of -inf is a weight of zero
                    up = Q[b, i, :, dim] * value > 0
                    assert bool(O[b, i][up].isnan().all()) and bool(lse[b, i][up].isnan().all()), (b, i)


def test_decode_layer_refused_steps_leave_the_cache(dsa):
    """A step that is refused writes nothing."""
    B, Sq, H = 2, 1, 16
    cache, table, _ = make_cache(dsa, [20, 33], 16, "e4m3", 191)
    inv, _ = dsa.rope_frequencies(DR)
    Q = torch.zeros(B, Sq, H, D, dtype=torch.bfloat16, device="cuda")
    good = dict(Q=Q, kv=torch.ones(B, Sq, D, dtype=torch.bfloat16, device="cuda"), pos=i32([[20], [33]]),
                inv_freq=inv, slots=i32([[3], [7]]), cache=cache.clone(), page_table=table,
                lens=i32([21, 34]), scale=0.1)
    wide = torch.zeros(2 * table.numel() + 4, dtype=torch.int32, device="cuda")
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    need = dsa.latent_attn_workspace_bytes(B, Sq, H, DC, DR)
    odd = torch.empty(need + 32, dtype=torch.uint8, device="cuda")[4:]
    for bad in (dict(Q=Q[:1].contiguous()), dict(Q=Q.float()), dict(Q=Q[..., :512].contiguous()),
                dict(Q=torch.zeros(B, Sq, 129, D, dtype=torch.bfloat16, device="cuda")), dict(scale=0.0),
                dict(scale=math.nan), dict(scale=3e38), dict(lens=i32([21])), dict(lens=i32([21, 34]).long()),
                dict(lens=i32([0, 0, 21, 34, 0])[1:3]), dict(page_table=table[0]),
                dict(page_table=table[:1].contiguous()), dict(page_table=table[:, :0].contiguous()),
                dict(page_table=wide[1:1 + table.numel()].view(table.shape)),
                dict(page_table=table.cpu()), dict(ws=small), dict(ws=odd), dict(ws=small.cpu()),
                dict(idx=i32([[[1]]])), dict(idx=i32([[[1]], [[1]]]).long()),
                dict(idx=i32([[[]], [[]]])), dict(idx=wide[1:3].view(2, 1, 1)), dict(layout="other"),
                dict(fmt="bf16"), dict(slots=i32([[3]])), dict(pos=i32([[20]])),
                dict(cache=cache.view(-1, cache.shape[-1]))):
        kw = {**good, **bad}
        before = kw["cache"].clone()
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            dsa.dsa_decode_layer(**kw)
        torch.cuda.synchronize()
        assert torch.equal(kw["cache"], before), bad
    dsa.dsa_decode_layer(**good)
    assert not torch.equal(good["cache"], cache)   # the same step, not refused
    no_error(dsa)


def block_counts(lims, blocks=DC, size=64):
    """How many of the positions below each limit lie in each block of `size`, the blocks in turn."""
    d = torch.arange(blocks, device="cuda")
    full = (lims[..., None] - d * size).clamp(0, size)
    assert int(lims.max()) <= blocks * size
    return full.double()


def every_key_once(dsa, fmt, lens, Sq, H, page, idx=None, times=2):
    """Q = 0: every weight is 1, lse is log(keys) up to the logarithm's rounding (2^-22 of it), and
    with rows that are 1 in the dim of their block of 64 positions O counts the keys of each block:
    integers, their quotient (2^-22) and one rounding to bf16 (2^-8). A key left out or counted twice
    changes its block by 2^-6 and lse by 1 / keys."""
    B = len(lens)
    cache, table, _ = make_cache(dsa, lens, page, fmt, 151)
    n = i32(lens)
    kv = torch.zeros(max(max(lens), 1), D, dtype=torch.bfloat16, device="cuda")
    p = torch.arange(len(kv), device="cuda")
    kv[p, (p // 64) % DC] = 1.0
    for b in range(B):
        if lens[b] > 0:
            q = p[:lens[b]]
            slots = (table[b].long()[q // page] * page + q % page).to(torch.int32)
            dsa.dsa_cache_write(kv[:lens[b]], slots, cache, DC, fmt=fmt)
    Q = torch.zeros(B, Sq, H, D, dtype=torch.bfloat16, device="cuda")
    lims = (n[:, None] - Sq + 1 + torch.arange(Sq, device="cuda")).clamp(min=0)
    if idx is None:
        counts = block_counts(lims)
    else:
        counts = torch.zeros(B, Sq, DC + 1, dtype=torch.float64, device="cuda")
        t = idx.long()
        seen = (t >= 0) & (t < lims[..., None])
        counts.scatter_add_(2, torch.where(seen, t // 64, DC), torch.ones_like(t, dtype=torch.float64))
        counts = counts[..., :DC]
    keys = counts.sum(-1)
    ref = (counts / keys.clamp(min=1)[..., None])[:, :, None]
    ref_lse = torch.where(keys > 0, keys.log(), -math.inf)[..., None]
    first = None
    for _ in range(times):
        O = torch.full((B, Sq, H, DC), math.nan, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((B, Sq, H), math.nan, device="cuda")
        dsa.dsa_latent_attn(Q, cache, table, n, 0.07, fmt=fmt, idx=idx, O=O, lse=lse)
        no_error(dsa)
        if first is None:
            first = O, lse
        assert torch.equal(O, first[0]) and torch.equal(lse, first[1])
    for b in range(B):
        err = (O[b].double() - ref[b]).abs()
        assert bool((err <= (2.0 ** -8 + 2.0 ** -22) * ref[b]).all()), (b, float(err.max()))
        off = torch.where(keys[b, :, None] > 0, (lse[b].double() - ref_lse[b]).abs(), 0.0)
        assert bool((off <= 2.0 ** -22 * ref_lse[b].abs() + 1e-30).all()), (b, float(off.max()))
        assert bool((lse[b][(keys[b] == 0)] == -math.inf).all())


RAGGED = [9000 - 371 * b if b % 6 else (0, 1, 30011, 48)[b // 6 % 4] for b in range(24)]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,Sq,H,page", [
    (RAGGED, 1, 128, 64), (RAGGED, 2, 100, 48), (RAGGED, 4, 16, 100), ([32768], 1, 16, 64),
    ([20000, 5], 7, 128, 64), ([31000, 32000, 30500, 29000], 1, 8, 16),
    ([(7 * b * b + 13 * b) % 401 for b in range(600)], 1, 128, 16),     # a thread splits several tiles
    ([(11 * b) % 97 for b in range(1300)], 1, 1, 16), ([900, 777], 700, 128, 64),
    ([1500], 1500, 64, 64)])
def test_latent_attn_every_key_once(dsa, fmt, lens, Sq, H, page):
    every_key_once(dsa, fmt, lens, Sq, H, page)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,Sq,H,k", [
    ([5000, 300, 0, 20000], 1, 128, 2048), ([700] * 600, 1, 16, 100), ([1100], 1100, 8, 130)])
def test_latent_attn_every_listed_key_once(dsa, fmt, lens, Sq, H, k):
    g = torch.Generator()
    g.manual_seed(161)
    idx = torch.full((len(lens), Sq, k), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        for i in range(Sq):
            pick = torch.randperm(max(n - Sq + i + 1, 0), generator=g)[:k].sort().values.to(torch.int32)
            at = torch.randperm(k, generator=g)[:len(pick)].sort().values   # holes anywhere
            idx[b, i, at] = pick
    every_key_once(dsa, fmt, lens, Sq, H, 64, idx.cuda())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("Sq,H,page", [(1, 128, 64), (2, 100, 48), (4, 16, 100)])
def test_latent_attn_many_ragged_each_sequence(dsa, fmt, Sq, H, page):
    """As test_latent_attn_many_ragged, the norm of the error held for every sequence by itself (a few
    short sequences have nearly all of the norm of O)."""
    cache, table, rows = make_cache(dsa, RAGGED, page, fmt, 81)
    Q = torch.randn(24, Sq, H, D, generator=gen(83), device="cuda").to(torch.bfloat16)
    O, lse = dsa.dsa_latent_attn(Q, cache, table, i32(RAGGED), 192 ** -0.5, fmt=fmt)
    no_error(dsa)
    for b in range(24):
        one = slice(b, b + 1)
        attn_check(O[one], lse[one], Q[one], rows[one], RAGGED[one], 192 ** -0.5)


@pytest.mark.parametrize("turned", [False, True])
def test_latent_attn_every_code_and_scale(dsa, turned):
    """A token that lists one key has its row as the output, bit for bit as dsa_cache_read has it: every
    finite e4m3 code, at scales from 2^-120 to 2^120 (2^7 is the largest that widens in one step), the
    key at any place of a list."""
    code = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()   # 0 to 448
    scales = [-120, -119, -118, -100, -60, -9, -1, 0, 1, 6, 7, 8, 9, 15, 60, 112, 113, 118, 119, 120]
    rows = []
    for k in scales:
        v = code.clamp(max=240.0) if k == 120 else code      # 1.875 * 2^127: above it, an infinity
        top = v[-1:]
        groups = [torch.cat([v, -top]), torch.cat([-v, top]), torch.cat([top, v.flip(0)]),
                  torch.cat([-top, -v.flip(0)])]
        if turned:
            groups = groups[2:] + groups[:2]
        rows.append(torch.cat(groups) * 2.0 ** k)
    n = len(rows)
    kv = torch.zeros(n, D)
    kv[:, :DC] = torch.stack(rows).float()
    cache = torch.full((2, 16, dsa.cache_row_bytes(DC, DR, "e4m3")), 0xff, dtype=torch.uint8,
                       device="cuda")
    slots = i32(range(n))
    dsa.dsa_cache_write(kv.to(torch.bfloat16).cuda(), slots, cache, DC, fmt="e4m3")
    held = cache.view(32, -1)[:n, DC:DC + 16].contiguous().view(torch.float32)
    assert torch.equal(held.cpu().double(), torch.tensor([[2.0 ** k] * 4 for k in scales]).double())
    want = dsa.dsa_cache_read(cache, slots, DC, DR, fmt="e4m3")
    assert torch.equal(want.cpu(), kv.to(torch.bfloat16))     # nothing was rounded
    for first in (0, 7, 29):
        idx = torch.full((1, n, 60), -1, dtype=torch.int32, device="cuda")
        for i in range(n):
            idx[0, i, (first + 11 * i) % 60] = i
        Q = torch.zeros(1, n, 16, D, dtype=torch.bfloat16, device="cuda")
        O, lse = dsa.dsa_latent_attn(Q, cache, i32([[0, 1]]), i32([n]), 0.07, fmt="e4m3", idx=idx)
        no_error(dsa)
        bad = (O[0] != want[:, None, :DC]).any(-1).any(-1)
        assert not bool(bad.any()), [scales[i] for i in torch.nonzero(bad)[:, 0].tolist()]
        assert not lse.any()


def test_a_longer_prompt_with_the_selection_of_the_top_k(dsa):
    """As test_prompt_with_the_selection_of_the_top_k, with more tokens than one batch of tiles."""
    S, H, k = 900, 16, 256
    g = gen(171)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    idx, _ = dsa.dsa_topk(dsa.dsa_index_scores(bf(1, S, 64, 128), bf(1, S, 128),
                                               torch.rand(1, S, 64, generator=g, device="cuda")), k, S=S)
    for fmt in ("bf16", "e4m3"):
        cache, table, rows = make_cache(dsa, [S], 64, fmt, 172)
        Q = bf(1, S, H, D)
        O, lse = dsa.dsa_latent_attn(Q, cache, table, i32([S]), 192 ** -0.5, fmt=fmt, idx=idx)
        no_error(dsa)
        for i in range(0, S, 50):        # the norm of the error held for 50 tokens at a time
            part = slice(i, i + 50)
            attn_check(O[:, part], lse[:, part], Q[:, part], rows, [i + 50], 192 ** -0.5, idx[:, part])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_decode_layer_captured(dsa, fmt):
    """A serving step captured once and replayed for the steps that follow: its positions, slots and
    lengths change in place."""
    B, Sq, H, page = 3, 1, 16, 16
    lens = [30, 47, 0]
    cache, table, _ = make_cache(dsa, [40, 60, 0], page, fmt, 181)
    mine = cache.clone()
    inv, m = dsa.rope_frequencies(DR, scaling="yarn", factor=8.0)
    g = gen(182)
    Q = torch.empty(B, Sq, H, D, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(B, Sq, D, dtype=torch.bfloat16, device="cuda")
    pos, slots, n = i32([[0]] * B), i32([[-1]] * B), i32(lens)

    def step(s):
        Q.copy_(torch.randn(Q.shape, generator=g, device="cuda"))
        kv.copy_(torch.randn(kv.shape, generator=g, device="cuda"))
        at = [k + s if k else 0 for k in lens]
        pos.copy_(i32([[a] for a in at]))
        slots.copy_(i32([[int(table[b, a // page]) * page + a % page if lens[b] else -1]
                         for b, a in enumerate(at)]))
        n.copy_(i32([k + s + 1 if k else 0 for k in lens]))

    step(0)
    dsa.dsa_decode_layer(Q, kv, pos, inv, slots, cache, table, n, 0.07, fmt=fmt, mscale=m)
    mine.copy_(cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O, lse = dsa.dsa_decode_layer(Q, kv, pos, inv, slots, mine, table, n, 0.07, fmt=fmt, mscale=m)
    for s in range(1, 8):
        step(s)
        O.fill_(math.nan)
        graph.replay()
        O2, lse2 = dsa.dsa_decode_layer(Q, kv, pos, inv, slots, cache, table, n, 0.07, fmt=fmt, mscale=m)
        assert torch.equal(O, O2) and torch.equal(lse, lse2) and torch.equal(mine, cache)
    no_error(dsa)


def test_sizes_past_32_bits_are_refused(dsa):
    """The library counts in 32-bit integers: what does not fit is refused, not cut."""
    inv, _ = dsa.rope_frequencies(64)
    x = torch.ones(2, 1, 128, device="cuda")
    cache = torch.zeros(2, 4, dsa.cache_row_bytes(DC, DR), dtype=torch.uint8, device="cuda")
    kv = torch.zeros(2, D, dtype=torch.bfloat16, device="cuda")
    Q = torch.zeros(1, 1, 4, D, dtype=torch.bfloat16, device="cuda")
    for wrap in (1 << 32, -(1 << 32), 1 << 40):
        for call in (lambda: dsa.dsa_rope(x, i32([3, 5]), inv, off=wrap + 64),
                     lambda: dsa.dsa_cache_write(kv, i32([0, 1]), cache, wrap + DC),
                     lambda: dsa.dsa_cache_read(cache, i32([0, 1]), wrap + DC, DR, kv=kv),
                     lambda: dsa.dsa_cache_read(cache, i32([0, 1]), DC, wrap + DR, kv=kv),
                     lambda: dsa.dsa_latent_attn(Q, cache, i32([[0, 1]]), i32([3]), 0.1, Dc=wrap + DC),
                     lambda: dsa.cache_row_bytes(wrap + DC, DR)):
            with pytest.raises(ValueError):
                call()
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_latent_attn_as_long_as_it_can_be(dsa, fmt):
    """2^31 - 2 keys, the most that pages of more than one row can hold: a page table that names two
    pages in turn, each of one row many times. The logits are all equal, so the weights are 1, and the
    values small integers: a cluster's sums (of 2^31 / 70 keys at most) are multiples of their
    smallest term below 2^24 of it, exact in fp32. What is rounded is the join of up to 80 parts (2^-17),
    the division and O (2^-8), and lse (2^-22 of it)."""
    page = 662
    pages = (2 ** 31 - 2) // page
    n = page * pages
    assert n == 2 ** 31 - 2
    cache = torch.zeros(2, page, dsa.cache_row_bytes(DC, DR, fmt), dtype=torch.uint8, device="cuda")
    kv = torch.zeros(2 * page, D, dtype=torch.bfloat16, device="cuda")
    kv[:, 0] = 1.0
    kv[:page, 300], kv[page:, 511] = 4.0, -2.0
    dsa.dsa_cache_write(kv, torch.arange(2 * page, dtype=torch.int32, device="cuda"), cache, DC, fmt=fmt)
    table = (torch.arange(pages, device="cuda") % 2).to(torch.int32)[None].contiguous()
    Q = torch.zeros(1, 2, 2, D, dtype=torch.bfloat16, device="cuda")
    Q[:, :, 1, 0] = 8.0
    O, lse = dsa.dsa_latent_attn(Q, cache, table, i32([n]), 1.0, fmt=fmt)
    no_error(dsa)
    for i in range(2):
        keys = n - 1 + i
        even = (pages - pages // 2) * page - (1 - i)     # the last page is an even one
        ref = torch.zeros(DC, dtype=torch.float64, device="cuda")
        ref[0], ref[300], ref[511] = 1.0, 4.0 * even / keys, -2.0 * (keys - even) / keys
        for h in range(2):
            err = (O[0, i, h].double() - ref).abs()
            assert bool((err <= (2.0 ** -8 + 2.0 ** -16) * ref.abs()).all()), (h, i, O[0, i, h][[0, 300, 511]])
            want = math.log(keys) + 8.0 * h
            assert abs(float(lse[0, i, h]) - want) <= 2.0 ** -17 + 2.0 ** -22 * want, (h, i, float(lse[0, i, h]), want)
