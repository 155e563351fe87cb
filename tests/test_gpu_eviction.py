"""Eviction from the paged latent cache by attention weight, against plain definitions.

Which positions stay and where their rows go are whole numbers and copied bytes: they are equal to the
definition's, with no tolerance.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DC, DR = 512, 64


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
