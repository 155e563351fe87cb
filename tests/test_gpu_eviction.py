"""Eviction from the paged latent cache by attention weight, against plain definitions.

Which positions stay and where their rows go are whole numbers and copied bytes: they are equal to the
definition's, with no tolerance.

Weights: el bounds the error of a logit l (576 exact products added in fp32, each addition off by at most
2^-23 of the sum of magnitudes). exp(l - lse) takes that error, those of the subtraction and of the change
of base (2^-24 |l - lse| each, 2^-22 with the second's own constant) and the exponential's (2^-22, and
2^-22 for the others' product). A sum of c such weights, all positive, in fp32, with decay * prev in front
of it, is off by at most (c + 3) 2^-24 of the whole (c + 3 roundings, each of at most half a step of a
partial sum).
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_serving import D, gen, i32, make_cache, no_error

pytestmark = pytest.mark.gpu

DC, DR = 512, 64


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_index_gb300 as m
    m.dsa_get_last_device_error()
    return m


# -------------------------------------------------------------------------------- what stays


def keep_ref(mass, lens, budget, sink, recent):
    """The definition: first ones, newest ones, and the others by (-mass, position); a NaN first."""
    keep = np.full((len(lens), budget), -1, np.int32)
    count = np.zeros(len(lens), np.int32)
    for b, n in enumerate(lens):
        n = min(max(n, 0), mass.shape[1])
        if n <= budget:
            got = np.arange(n)
        else:
            mid = np.arange(sink, n - recent)
            m = mass[b, mid].astype(np.float64)
            nan = np.isnan(m)
            order = np.lexsort((mid, np.where(nan, 0.0, -m), ~nan))
            chosen = mid[order[:budget - sink - recent]]
            got = np.sort(np.concatenate([np.arange(sink), np.arange(n - recent, n), chosen]))
        keep[b, :len(got)] = got
        count[b] = len(got)
    return keep, count


def check_keep(dsa, mass, lens, budget, sink, recent):
    keep, count = dsa.dsa_cache_keep(mass, i32(lens), budget, sink=sink, recent=recent)
    want, n = keep_ref(mass.cpu().numpy(), lens, budget, sink, recent)
    assert np.array_equal(count.cpu().numpy(), n)
    assert np.array_equal(keep.cpu().numpy(), want)


@pytest.mark.parametrize("n,budget,sink,recent", [
    (1, 1, 0, 0), (1, 4, 1, 1), (2, 1, 0, 0), (33, 32, 0, 0), (33, 32, 16, 16), (100, 1, 1, 0),
    (100, 1, 0, 1), (1000, 999, 3, 5), (2047, 100, 4, 16), (8192, 2048, 4, 128), (8193, 8192, 0, 0),
    (40001, 5000, 64, 1024), (131072, 16384, 64, 1024)])
@pytest.mark.parametrize("kind", ["lognormal", "ties", "equal", "narrow", "signed"])
def test_keep(dsa, n, budget, sink, recent, kind):
    g = gen(n + budget)
    B = 5
    m = torch.randn(B, n, generator=g, device="cuda")
    if kind == "lognormal":
        m = torch.exp(2 * m)
    elif kind == "ties":
        m = (torch.exp(2 * m) * 4).round() / 4
    elif kind == "equal":
        m = torch.full_like(m, 0.25)
    elif kind == "narrow":        # a few last bits apart
        m = (torch.full_like(m, 1.5).view(torch.int32)
             + torch.randint(0, 40, m.shape, generator=g, device="cuda", dtype=torch.int32)).view(torch.float32)
    check_keep(dsa, m, [n, max(n - 7, 0), min(n, budget), min(n, budget + 1), n // 2], budget, sink, recent)
    no_error(dsa)


def test_keep_orders_zeros_infinities_and_nans(dsa):
    v = torch.tensor([0.0, -0.0, 1.0, float("inf"), float("nan"), -float("inf"), -1.0, 1e-45, -1e-45,
                      3.4e38, -3.4e38], device="cuda")
    neg = (torch.full((1,), float("nan"), device="cuda").view(torch.int32) | -(1 << 31)).view(torch.float32)
    v = torch.cat([v, neg])
    g = gen(1)
    for n in (12, 500):
        m = v[torch.randint(0, len(v), (4, n), generator=g, device="cuda")]
        for budget in (1, 3, 7, 11):
            check_keep(dsa, m, [n, n - 1, 11, 5], budget, 0, 0)
    no_error(dsa)


@pytest.mark.parametrize("B,n", [(1, 5000), (3, 400000), (37, 3000), (160, 9000), (400, 700)])
def test_keep_batches(dsa, B, n):
    """Every cluster size, and more weights than shared memory holds."""
    g = gen(B)
    m = (torch.exp(torch.randn(B, n, generator=g, device="cuda")) * 64).round() / 64
    lens = [max(0, n - 13 * b) for b in range(B)]
    check_keep(dsa, m, lens, n // 3, 5, 17)
    no_error(dsa)


def test_keep_lengths_outside(dsa):
    m = torch.rand(3, 50, generator=gen(2), device="cuda")
    check_keep(dsa, m, [0, 50, 20], 10, 1, 2)
    no_error(dsa)
    check_keep(dsa, m, [-5, 99, 50], 10, 1, 2)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_EVICT | dsa.DSA_DEVERR_BAD_PAGE


# ---------------------------------------------------------------------------- the rows moved


def setup_rows(dsa, B, lens, budget, page, fmt, seed, dims=(DC, DR)):
    g = gen(seed)
    row = dsa.cache_row_bytes(*dims, fmt)
    need = [max(1, -(-n // page)) for n in lens]
    new = -(-budget // page)
    total = sum(need) + B * new + 2
    cache = torch.randint(0, 256, (total, page, row), generator=g, device="cuda", dtype=torch.uint8)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(need)), -7, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return cache, table, order[at:at + B * new].view(B, new).clone(), g


def slots_of(table, page, at):
    return table[at // page].astype(np.int64) * page + at % page


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,budget,page", [
    ([1], 1, 64), ([70], 33, 16), ([0, 5, 300], 40, 7), ([500, 499, 37, 2000], 256, 64),
    ([3000] * 3, 1000, 100), ([9000], 4097, 1)])
@pytest.mark.parametrize("place", ["new", "same"])
def test_compact(dsa, fmt, lens, budget, page, place):
    B = len(lens)
    cache, table, new_table, g = setup_rows(dsa, B, lens, budget, page, fmt, budget)
    n = max(lens) + 3
    mass = torch.rand(B, n, generator=g, device="cuda")
    keep, count = dsa.dsa_cache_keep(mass, i32(lens), budget, sink=min(2, budget), recent=min(5, budget - min(2, budget)))
    want = cache.cpu().numpy().reshape(-1, cache.shape[-1]).copy()
    old = want.copy()
    to = (new_table if place == "new" else table).cpu().numpy()
    t, k, m = table.cpu().numpy(), keep.cpu().numpy(), mass.cpu().numpy()
    want_mass = np.zeros((B, budget + 5), np.float32)
    for b in range(B):
        kept = k[b][k[b] >= 0]
        want[slots_of(to[b], page, np.arange(len(kept)))] = old[slots_of(t[b], page, kept)]
        want_mass[b, :len(kept)] = m[b, kept]
    new_mass = torch.full((B, budget + 5), -1.0, device="cuda")
    got = dsa.dsa_cache_compact(cache, table, i32(lens), keep, new_table if place == "new" else None, DC, DR,
                                fmt=fmt, mass=mass, new_mass=new_mass)
    assert got is new_mass
    assert np.array_equal(cache.cpu().numpy().reshape(want.shape), want)
    assert np.array_equal(new_mass.cpu().numpy(), want_mass)
    no_error(dsa)


@pytest.mark.parametrize("place", ["new", "same"])
@pytest.mark.parametrize("B,n,budget", [(1, 20000, 7000), (5, 900, 450), (3, 10, 10), (90, 300, 100)])
def test_compact_weights_in_place(dsa, place, B, n, budget):
    lens = [max(1, n - 11 * b) for b in range(B)]
    cache, table, new_table, g = setup_rows(dsa, B, lens, budget, 32, "e4m3", n, dims=(128, 8))
    mass = torch.rand(B, n, generator=g, device="cuda")
    keep, _ = dsa.dsa_cache_keep(mass, i32(lens), budget, sink=1, recent=3)
    rows = cache.cpu().numpy().reshape(-1, cache.shape[-1]).copy()
    k, m, t = keep.cpu().numpy(), mass.cpu().numpy(), table.cpu().numpy()
    want = np.zeros((B, n), np.float32)
    moved = rows.copy()
    to = new_table.cpu().numpy() if place == "new" else t
    for b in range(B):
        kept = k[b][k[b] >= 0]
        want[b, :len(kept)] = m[b, kept]
        moved[slots_of(to[b], 32, np.arange(len(kept)))] = rows[slots_of(t[b], 32, kept)]
    dsa.dsa_cache_compact(cache, table, i32(lens), keep, new_table if place == "new" else None, 128, 8,
                          mass=mass, new_mass=mass)
    assert np.array_equal(mass.cpu().numpy(), want)
    assert np.array_equal(cache.cpu().numpy().reshape(moved.shape), moved)
    no_error(dsa)


def test_compact_bad_entries_and_pages(dsa):
    """They move nothing and are recorded; everything else moves."""
    lens = [60, 60]
    for place in ("new", "same"):
        cache, table, new_table, _ = setup_rows(dsa, 2, lens, 10, 16, "e4m3", 3)
        old = cache.cpu().numpy().reshape(-1, cache.shape[-1]).copy()
        t = table.cpu().numpy()
        to = new_table.cpu().numpy() if place == "new" else t
        keep = i32([[3, 9, 60, 21, -2, 30, 31, 32, 1 << 30, 59], [0, 1, 2, 3, 4, 5, 6, 7, 58, -1]])
        want = old.copy()
        for b, row in enumerate(keep.cpu().numpy()):
            for j, e in enumerate(row):
                if 0 <= e < 60:
                    want[slots_of(to[b], 16, np.array([j]))] = old[slots_of(t[b], 16, np.array([e]))]
        dsa.dsa_cache_compact(cache, table, i32(lens), keep, new_table if place == "new" else None, DC, DR)
        assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_EVICT | dsa.DSA_DEVERR_BAD_INDEX
        assert np.array_equal(cache.cpu().numpy().reshape(old.shape), want), place
        # the third page of the first sequence is not one of the cache
        cache.copy_(torch.from_numpy(old).view(cache.shape))
        table[0, 2] = cache.shape[0]
        keep = i32([[3, 33, 34, 50], [1, 33, 34, 50]])
        want = old.copy()
        for b, row in enumerate(keep.cpu().numpy()):
            for j, e in enumerate(row):
                if b == 1 or e // 16 != 2:
                    want[slots_of(to[b], 16, np.array([j]))] = old[slots_of(t[b], 16, np.array([e]))]
        dsa.dsa_cache_compact(cache, table, i32(lens), keep, new_table if place == "new" else None, DC, DR)
        assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_EVICT | dsa.DSA_DEVERR_BAD_PAGE
        assert np.array_equal(cache.cpu().numpy().reshape(old.shape), want), place


@pytest.mark.parametrize("place", ["new", "same"])
def test_compact_entries_behind_the_end(dsa, place):
    """A list that goes on behind a short sequence's end names rows that are not there."""
    cache, table, new_table, _ = setup_rows(dsa, 2, [5, 700], 600, 16, "e4m3", 5)
    keep = torch.full((2, 600), -1, dtype=torch.int32, device="cuda")
    keep[0, :3] = i32([0, 2, 4])
    keep[1] = torch.arange(50, 650, device="cuda")
    old = cache.view(-1, cache.shape[-1]).cpu().numpy().copy()
    t = table.cpu().numpy()
    to = new_table.cpu().numpy() if place == "new" else t
    want = old.copy()
    for b, kept in enumerate((np.array([0, 2, 4]), np.arange(50, 650))):
        want[slots_of(to[b], 16, np.arange(len(kept)))] = old[slots_of(t[b], 16, kept)]
    keep[0, 599] = 3
    dsa.dsa_cache_compact(cache, table, i32([5, 700]), keep, new_table if place == "new" else None, DC, DR)
    got = cache.view(-1, cache.shape[-1]).cpu().numpy()
    if place == "new":       # a row that is there, to a place that is there
        want[slots_of(to[0], 16, np.array([599]))] = old[slots_of(t[0], 16, np.array([3]))]
        no_error(dsa)
    else:
        assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_EVICT | dsa.DSA_DEVERR_BAD_INDEX
    assert np.array_equal(got, want)
    keep[0, 599] = 5
    dsa.dsa_cache_compact(cache, table, i32([5, 700]), keep, new_table if place == "new" else None, DC, DR)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_EVICT | dsa.DSA_DEVERR_BAD_INDEX


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,n,budget", [(1, 9000, 5000), (3, 4000, 3999), (70, 600, 300), (200, 90, 64)])
def test_compact_in_place_of_many(dsa, fmt, B, n, budget):
    """Every block size and slice, lists that move by one row and by many."""
    lens = [max(1, n - 7 * b) for b in range(B)]
    cache, table, _, g = setup_rows(dsa, B, lens, budget, 64, fmt, n)
    keep = torch.full((B, budget), -1, dtype=torch.int32, device="cuda")
    for b, m in enumerate(lens):
        c = min(m, budget)
        if b % 3 == 0:                              # the last ones: every row by the same step
            keep[b, :c] = torch.arange(m - c, m, device="cuda")
        else:
            keep[b, :c] = torch.randperm(m, generator=g, device="cuda")[:c].sort().values.to(torch.int32)
    old = cache.view(-1, cache.shape[-1]).clone()
    page = torch.arange(max(n, budget), device="cuda") // 64
    off = torch.arange(max(n, budget), device="cuda") % 64
    want = old.clone()
    for b in range(B):
        kept = keep[b][keep[b] >= 0].long()
        slot = lambda j: table[b].long()[page[j]] * 64 + off[j]  # noqa: E731,B023
        want[slot(torch.arange(len(kept), device="cuda"))] = old[slot(kept)]
    dsa.dsa_cache_compact(cache, table, i32(lens), keep, None, DC, DR, fmt=fmt)
    assert torch.equal(cache.view(old.shape), want)
    no_error(dsa)


def test_python_refusals(dsa):
    m, lens = torch.zeros(2, 8, device="cuda"), i32([8, 8])
    with pytest.raises(ValueError):
        dsa.dsa_cache_keep(m, lens, 0)
    with pytest.raises(ValueError):
        dsa.dsa_cache_keep(m[0], lens, 4)
    with pytest.raises(ValueError):
        dsa.dsa_cache_keep(m, i32([8]), 4)
    with pytest.raises(ValueError):
        dsa.dsa_cache_keep(m.t(), lens, 4)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_cache_keep(m, lens, 4, sink=3, recent=2)
    cache, table, new_table, _ = setup_rows(dsa, 2, [8, 8], 4, 16, "e4m3", 1)
    keep = i32([[0, 1, 2, 3]] * 2)
    before = cache.clone()
    with pytest.raises(ValueError):
        dsa.dsa_cache_compact(cache, table, lens, keep, new_table, DC, DR, fmt="bf16")
    with pytest.raises(ValueError):
        dsa.dsa_cache_compact(cache, table, lens, keep, new_table, DC, DR, new_mass=m)
    with pytest.raises(dsa.DsaError):
        dsa.dsa_cache_compact(cache, table, lens, keep, new_table, DC, DR, mass=m, new_mass=torch.zeros(2, 3, device="cuda"))
    with pytest.raises(ValueError):
        dsa.dsa_cache_compact(cache, table, lens, i32([0, 1]), new_table, DC, DR)
    assert torch.equal(cache, before)
    no_error(dsa)


# ------------------------------------------------------------------------------- the weights


def mass_inputs(dsa, lens, Sq, H, page, fmt, seed, k=0):
    """A cache, queries, lists and the attention's lse (the definition's, rounded to fp32)."""
    cache, table, rows = make_cache(dsa, lens, page, fmt, seed)
    g, B = gen(seed + 1), len(lens)
    Q = torch.randn(B, Sq, H, D, generator=g, device="cuda").to(torch.bfloat16)
    scale = 192 ** -0.5
    idx = None
    if k:
        idx = torch.full((B, Sq, k), -1, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            for i in range(Sq):
                at = torch.randperm(max(n, 1), generator=g, device="cuda")[:min(k, max(n, 0))].sort().values
                idx[b, i, :len(at)] = at.to(torch.int32)          # entries behind the token among them
    lse = torch.full((B, Sq, H), -math.inf, device="cuda")
    for b in range(B):
        for i in range(Sq):
            at = seen(lens[b], Sq, i, None if idx is None else idx[b, i])
            if len(at):
                l = scale * (Q[b, i].double() @ rows[b][at].T)
                lse[b, i] = torch.logsumexp(l, -1).float()
    return Q, cache, table, i32(lens), lse, scale, idx, rows


def seen(n, Sq, i, listed):
    """The positions that token i of a sequence of n sees."""
    limit = max(n, 0) - Sq + i + 1
    if listed is None:
        return torch.arange(max(limit, 0), device="cuda")
    t = listed.long()
    return t[(t >= 0) & (t < limit)]


def mass_check(got, Q, rows, lens, lse, scale, idx=None, prev=None, decay=1.0):
    B, Sq, H, _ = Q.shape
    n = got.shape[1]
    for b in range(B):
        m = min(max(int(lens[b]), 0), n)
        ref = torch.zeros(n, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(ref)
        if prev is not None:
            ref[:m] = decay * prev[b, :m].double()
        base = ref.clone()
        for i in range(Sq):
            at = seen(int(lens[b]), Sq, i, None if idx is None else idx[b, i])
            at = at[at < n]
            if len(at) == 0:
                continue
            q, kv = Q[b, i].double(), rows[b][at]
            x = scale * (q @ kv.T) - lse[b, i].double()[:, None]
            x[lse[b, i] == -math.inf] = -math.inf
            w = torch.exp(x)
            el = D * 2.0 ** -23 * scale * (q.abs() @ kv.abs().T)
            r = torch.where(w > 0, torch.expm1(el + x.abs() * 2.0 ** -22 + 2.0 ** -21), torch.zeros_like(w))
            ref.index_add_(0, at, w.sum(0))
            tol.index_add_(0, at, (w * r).sum(0))
        tol += (Sq * H + 3) * 2.0 ** -24 * (ref - base + base.abs())
        err = (got[b].double() - ref).abs()
        assert bool((err <= tol).all()), (b, float((err - tol).max()), int((err - tol).argmax()))
        assert not got[b, m:].any()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,Sq,H,page", [
    ([1], 1, 1, 16), ([489], 1, 16, 64), ([127, 128, 129], 1, 128, 7), ([0, 1, 97, 0], 1, 20, 16),
    ([3, 130], 4, 16, 16), ([2, 700], 3, 128, 100), ([7], 7, 5, 64), ([96, 1000, 1, 31, 2049], 2, 64, 32),
    ([20000], 1, 128, 64), ([300, 40], 33, 128, 16), ([1500], 32, 128, 64), ([200], 70, 3, 16),
    ([4000, 257], 9, 57, 1)])
def test_mass(dsa, fmt, lens, Sq, H, page):
    Q, cache, table, ln, lse, scale, _, rows = mass_inputs(dsa, lens, Sq, H, page, fmt, 11)
    n = max(lens) + 5
    prev = torch.rand(len(lens), n, generator=gen(12), device="cuda")
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, n, fmt=fmt)
    mass_check(got, Q, rows, lens, lse, scale)
    both = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, n, fmt=fmt, prev=prev, decay=0.875)
    mass_check(both, Q, rows, lens, lse, scale, None, prev, 0.875)
    again = prev.clone()
    assert dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, n, fmt=fmt, prev=again, decay=0.875, mass=again) is again
    assert torch.equal(again, both)                                       # the same bits
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,Sq,H,page,k", [
    ([1], 1, 1, 16, 1), ([489], 1, 16, 64, 100), ([50, 0, 3], 2, 20, 16, 64), ([700, 2000], 3, 128, 100, 500),
    ([5000, 4097, 9000], 1, 128, 64, 2048), ([300], 9, 8, 16, 129), ([20000, 1], 2, 33, 16, 300)])
def test_mass_of_lists(dsa, fmt, lens, Sq, H, page, k):
    Q, cache, table, ln, lse, scale, idx, rows = mass_inputs(dsa, lens, Sq, H, page, fmt, 21, k)
    n = max(lens) + 1
    prev = torch.rand(len(lens), n, generator=gen(22), device="cuda")
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, n, fmt=fmt, idx=idx)
    mass_check(got, Q, rows, lens, lse, scale, idx)
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, n, fmt=fmt, idx=idx, prev=prev, decay=-0.5, mass=prev.clone())
    mass_check(got, Q, rows, lens, lse, scale, idx, prev, -0.5)
    twice = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, n, fmt=fmt, idx=idx, prev=prev, decay=-0.5)
    assert torch.equal(got, twice)
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("Sq,H", [(1, 128), (1, 16), (4, 100)])
def test_mass_many_ragged(dsa, fmt, Sq, H):
    lens = [5000 - 371 * b if b % 6 else (0, 1, 20011, 128)[b // 6 % 4] for b in range(13)] * 3
    lens = [max(n, 0) for n in lens]
    Q, cache, table, ln, lse, scale, _, rows = mass_inputs(dsa, lens, Sq, H, 64, fmt, 31)
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, max(lens), fmt=fmt)
    mass_check(got, Q, rows, lens, lse, scale)
    no_error(dsa)


def test_mass_of_attention_sums_to_the_tokens(dsa):
    """With the lse that the attention gives, the weights of a token and head sum to one."""
    lens, Sq, H = [700, 33, 2, 1500], 2, 48
    Q, cache, table, ln, _, scale, idx, _ = mass_inputs(dsa, lens, Sq, H, 16, "e4m3", 41, 200)
    for lists in (None, idx):
        lse = dsa.dsa_latent_attn(Q, cache, table, ln, scale, idx=lists)[1]
        got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, max(lens), idx=lists)
        # each weight within 2^-12 (the bounds of both logits and of lse), tokens without a key add none
        tokens = torch.tensor([[float(bool((lse[b, i] > -math.inf).all())) for i in range(Sq)] for b in range(4)])
        assert (got.double().sum(-1).cpu() - H * tokens.sum(-1)).abs().max() <= 2.0 ** -12 * H * Sq
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("H", [16, 128])
def test_mass_values_that_are_not_finite(dsa, fmt, H):
    """A NaN row is NaN in its own place alone; a token's lse of NaN in all that it sees, of -inf in none;
    an infinite row has the weight of its logit: 0 or what exp gives."""
    lens, Sq = [200, 150], 2
    Q, cache, table, ln, lse, scale, _, rows = mass_inputs(dsa, lens, Sq, H, 16, fmt, 51)
    clean = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 200, fmt=fmt)
    for b, j in ((0, 40), (0, 199), (1, 149)):        # 199: seen by the last token alone
        slot = int(table[b, j // 16]) * 16 + j % 16
        dsa.dsa_cache_write(torch.full((1, D), math.nan, dtype=torch.bfloat16, device="cuda"), i32([slot]),
                            cache, DC, fmt=fmt)
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 200, fmt=fmt)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[0, 40] = hit[0, 199] = hit[1, 149] = True
    assert torch.equal(torch.isnan(got), hit) and torch.equal(got[~hit], clean[~hit])
    # the rows again, and the first token's lse
    bad = lse.clone()
    bad[1, 0, H // 2] = math.nan
    bad[0, 0] = -math.inf
    cache2, table2, rows2 = make_cache(dsa, lens, 16, fmt, 51)
    got = dsa.dsa_cache_mass(Q, cache2, table2, ln, bad, scale, 200, fmt=fmt)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[1, :149] = True
    assert torch.equal(torch.isnan(got), hit)
    mass_check(got[:1], Q[:1], rows2[:1], lens[:1], bad[:1], scale)
    # positional dims of plus and minus infinity: logits of infinite size
    row = torch.zeros(1, D, dtype=torch.bfloat16, device="cuda")
    row[0, DC] = math.inf
    slot = int(table2[0, 0]) * 16
    dsa.dsa_cache_write(row, i32([slot]), cache2, DC, fmt=fmt)
    Q[0, :, :, DC] = -Q[0, :, :, DC].abs() - 1
    got = dsa.dsa_cache_mass(Q, cache2, table2, ln, lse, scale, 200, fmt=fmt)
    assert float(got[0, 0]) == 0.0
    Q[0, :, 0, DC] = 1.0
    got = dsa.dsa_cache_mass(Q, cache2, table2, ln, lse, scale, 200, fmt=fmt)
    assert float(got[0, 0]) == math.inf
    no_error(dsa)


def test_mass_bad_entries_pages_and_lengths(dsa):
    lens, Sq, H = [100, 90], 1, 16
    Q, cache, table, ln, lse, scale, idx, rows = mass_inputs(dsa, lens, Sq, H, 16, "e4m3", 61, 20)
    idx[0, 0, 3], idx[1, 0, 0] = 100, -2
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 100, idx=idx)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_EVICT | dsa.DSA_DEVERR_BAD_INDEX
    mass_check(got, Q, rows, lens, lse, scale, idx)
    # a page that is none: its keys are not there
    broken = table.clone()
    broken[0, 2] = cache.shape[0]
    whole = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 100)
    no_error(dsa)
    got = dsa.dsa_cache_mass(Q, cache, broken, ln, lse, scale, 100)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_EVICT | dsa.DSA_DEVERR_BAD_PAGE
    want = whole.clone()
    want[0, 32:48] = 0
    assert torch.equal(got, want)
    # room for fewer positions than there are
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 37)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_EVICT | dsa.DSA_DEVERR_BAD_PAGE
    assert torch.equal(got, whole[:, :37])
    got = dsa.dsa_cache_mass(Q, cache, table, i32([-3, 90]), lse, scale, 100)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_EVICT | dsa.DSA_DEVERR_BAD_PAGE
    assert not got[0].any() and torch.equal(got[1], whole[1])


def test_mass_of_an_entry_twice(dsa):
    """An entry listed twice counts twice, the same bits every time."""
    Q, cache, table, ln, lse, scale, idx, rows = mass_inputs(dsa, [300], 2, 16, 16, "bf16", 71, 40)
    idx[0, 0, 5] = idx[0, 0, 4]
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 300, fmt="bf16", idx=idx)
    mass_check(got, Q, rows, [300], lse, scale, idx)
    for _ in range(3):
        assert torch.equal(got, dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 300, fmt="bf16", idx=idx))
    no_error(dsa)


# ---------------------------------------------------------------------------------- together


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("place", ["new", "same"])
def test_steps_with_eviction(dsa, fmt, place):
    """Attention, its weights, the positions that stay, their rows moved; then the next step's attention
    over what is left is that over the kept rows."""
    lens, Sq, H, page, budget = [300, 40, 777, 128], 1, 32, 16, 100
    Q, cache, table, ln, _, scale, _, rows = mass_inputs(dsa, lens, Sq, H, page, fmt, 81)
    n = 800
    mass = torch.zeros(4, n, device="cuda")
    for _ in range(2):
        O, lse = dsa.dsa_latent_attn(Q, cache, table, ln, scale, fmt=fmt)
        dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, n, fmt=fmt, prev=mass, decay=0.5, mass=mass)
    keep, count = dsa.dsa_cache_keep(mass, ln, budget, sink=2, recent=10)
    want, _ = keep_ref(mass.cpu().numpy(), lens, budget, 2, 10)
    assert np.array_equal(keep.cpu().numpy(), want)
    new_table = table
    if place == "new":
        spare = torch.zeros(4 * 7, page, cache.shape[-1], dtype=torch.uint8, device="cuda")
        new_table = (cache.shape[0] + torch.randperm(28, device="cuda").to(torch.int32)).view(4, 7).contiguous()
        cache = torch.cat([cache, spare])
    dsa.dsa_cache_compact(cache, table, ln, keep, new_table if place == "new" else None, DC, DR, fmt=fmt, mass=mass,
                          new_mass=mass)
    from test_gpu_serving import attn_check
    O, lse = dsa.dsa_latent_attn(Q, cache, new_table, count, scale, fmt=fmt)
    kept = [rows[b][keep[b][keep[b] >= 0].long()] for b in range(4)]
    attn_check(O, lse, Q, kept, [len(r) for r in kept], scale)
    got = dsa.dsa_cache_mass(Q, cache, new_table, count, lse, scale, n, fmt=fmt, prev=mass)
    mass_check(got, Q, kept, [len(r) for r in kept], lse, scale, None, mass)
    no_error(dsa)


def test_captured_step(dsa):
    """A whole step captured into a graph and replayed with other lengths."""
    lens, H, page, budget = [300, 200, 60], 16, 16, 64
    Q, cache, table, ln, _, scale, _, _ = mass_inputs(dsa, lens, 1, H, page, "e4m3", 91)
    start = cache.clone()

    def step():
        O, lse = dsa.dsa_latent_attn(Q, cache, table, ln, scale)
        mass = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 300)
        keep, count = dsa.dsa_cache_keep(mass, ln, budget, recent=4)
        new_mass = dsa.dsa_cache_compact(cache, table, ln, keep, None, DC, DR, mass=mass)
        return O, lse, mass, keep, count, new_mass

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for other in (lens, [100, 64, 1]):
        ln.copy_(i32(other))
        cache.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs] + [cache.clone()]
        cache.copy_(start)
        for a, b in zip(got, list(step()) + [cache]):
            assert torch.equal(a, b)
    # on another stream than the current one
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mass = dsa.dsa_cache_mass(Q, start, table, ln, got[1], scale, 300, stream=s)
    keep, count = dsa.dsa_cache_keep(mass, ln, budget, recent=4, stream=s)
    new_mass = dsa.dsa_cache_compact(start, table, ln, keep, None, DC, DR, mass=mass, stream=s)
    s.synchronize()
    for a, b in zip((mass, keep, count, new_mass, start), got[2:]):
        assert torch.equal(a, b)
    no_error(dsa)


@pytest.mark.parametrize("Sq,H,k", [(1, 16, 0), (2, 80, 0), (1, 128, 1), (3, 20, 70)])
def test_mass_of_many_short_sequences(dsa, Sq, H, k):
    """More sequences than clusters, empty ones among them."""
    lens = [(b * 37) % 300 if b % 5 else 0 for b in range(300)]
    Q, cache, table, ln, lse, scale, idx, rows = mass_inputs(dsa, lens, Sq, H, 32, "e4m3", 111, k)
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 301, idx=idx)
    mass_check(got, Q, rows, lens, lse, scale, idx)
    no_error(dsa)


@pytest.mark.parametrize("Sq", [1, 40])
def test_mass_into_other_widths(dsa, Sq):
    """Rows of mass at every alignment, and the room behind the sequences cleared in all of them."""
    lens, H = [260, 1 + Sq, 513], 16
    Q, cache, table, ln, lse, scale, _, rows = mass_inputs(dsa, lens, Sq, H, 16, "bf16", 121)
    want = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 513, fmt="bf16")
    mass_check(want, Q, rows, lens, lse, scale)
    for n in (514, 515, 517, 100003):
        mass = torch.full((3, n), math.nan, device="cuda")
        got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, n, fmt="bf16", mass=mass)
        assert torch.equal(got[:, :513], want) and not got[:, 513:].any()
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_cache_of_more_than_2_to_the_31_bytes(dsa, fmt):
    """Rows whose offsets do not fit 32 bits: attention over a shared prefix, weights, and rows moved to
    and fro, against the same rows in a small cache."""
    row, page = dsa.cache_row_bytes(DC, DR, fmt), 1024
    pages = (1 << 32) // (row * page) + 8
    big = torch.zeros(pages, page, row, dtype=torch.uint8, device="cuda")
    lens, Sq, H = [1500, 900], 1, 16
    Q, cache, table, ln, lse, scale, _, rows = mass_inputs(dsa, lens, Sq, H, page, fmt, 131)
    far = table.clone()
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            far[b, j] = pages - 1 - (2 * b + j)
            big[int(far[b, j])] = cache[int(table[b, j])]
    want = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 1500, fmt=fmt)
    got = dsa.dsa_cache_mass(Q, big, far, ln, lse, scale, 1500, fmt=fmt)
    assert torch.equal(got, want)
    starts, plen = i32([0, 2]), i32([1500])
    a = dsa.dsa_latent_attn_shared(Q, cache, table[:1].clone(), plen, starts, table, ln, scale, fmt=fmt)
    b = dsa.dsa_latent_attn_shared(Q, big, far[:1].clone(), plen, starts, far, ln, scale, fmt=fmt)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    keep, _ = dsa.dsa_cache_keep(want, ln, 700, recent=5)
    near = i32([[0], [1]])
    dsa.dsa_cache_compact(big, far, ln, keep, near, DC, DR, fmt=fmt)
    dsa.dsa_cache_compact(big, far, ln, keep, None, DC, DR, fmt=fmt)
    for s in range(2):
        old = cache[table[s, :-(-lens[s] // page)].long()].view(-1, row)[keep[s].long()]
        assert torch.equal(big[s, :700], old) and torch.equal(big[int(far[s, 0]), :700], old)
    no_error(dsa)


def test_two_streams_at_once(dsa):
    """Calls on two streams, each with its own workspace and outputs, do not reach one another."""
    lens, H = [700, 900], 128
    sets = [mass_inputs(dsa, lens, Sq, H, 16, "e4m3", 141 + Sq) for Sq in (2, 3)]
    want = [dsa.dsa_cache_mass(*t[:3], t[3], t[4], t[5], 900) for t in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, t in enumerate(sets):
            m = dsa.dsa_cache_mass(*t[:3], t[3], t[4], t[5], 900, stream=streams[i])
            keep, count = dsa.dsa_cache_keep(m, t[3], 300, recent=3, stream=streams[i])
            got[i].append((m, keep, count))
    torch.cuda.synchronize()
    for i in range(2):
        keep, count = dsa.dsa_cache_keep(want[i], sets[i][3], 300, recent=3)
        for m, k, c in got[i]:
            assert torch.equal(m, want[i]) and torch.equal(k, keep) and torch.equal(c, count)
    no_error(dsa)
