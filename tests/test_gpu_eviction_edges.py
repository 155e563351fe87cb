"""Eviction from the paged latent cache where its arguments are at the edge of the contract: lists that do
not ascend, and entries that the weights have no room for."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from test_gpu_eviction import DC, DR, mass_check, mass_inputs, setup_rows, slots_of
from test_gpu_serving import D, attn_check, gen, i32, no_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_index_gb300 as m
    m.dsa_get_last_device_error()
    return m


def bad_index(dsa):
    return dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_EVICT | dsa.DSA_DEVERR_BAD_INDEX


def moved(cache, table, to, keep, page):
    """The cache's rows after every entry of keep has moved."""
    old = cache.cpu().numpy().reshape(-1, cache.shape[-1])
    want = old.copy()
    t, to = table.cpu().numpy(), to.cpu().numpy()
    for b, row in enumerate(keep.cpu().numpy()):
        for j, e in enumerate(row):
            if e >= 0:
                want[slots_of(to[b], page, np.array([j]))] = old[slots_of(t[b], page, np.array([e]))]
    return want


@pytest.mark.parametrize("aliased", [False, True])
def test_list_that_does_not_ascend_to_new_pages(dsa, aliased):
    """Every row moves. The weights move in place from higher places to lower ones alone: one that would not
    is zero there and recorded; into another buffer all of them move."""
    cache, table, new_table, g = setup_rows(dsa, 2, [60, 60], 6, 16, "e4m3", 11)
    keep = i32([[7, 0, 9, 30, -1, -1], [2, 3, 5, 8, 13, 21]])
    want = moved(cache, table, new_table, keep, 16)
    mass = torch.rand(2, 60, generator=g, device="cuda") + 1
    want_mass = torch.zeros(2, 60, device="cuda")
    for b in range(2):
        for j, e in enumerate(keep[b].tolist()):
            if e >= (j if aliased else 0):
                want_mass[b, j] = mass[b, e]
    out = mass if aliased else torch.full_like(mass, -1.0)
    dsa.dsa_cache_compact(cache, table, i32([60, 60]), keep, new_table, DC, DR, mass=mass, new_mass=out)
    if aliased:
        assert bad_index(dsa)
    else:
        no_error(dsa)
    assert torch.equal(out, want_mass)
    assert np.array_equal(cache.cpu().numpy().reshape(want.shape), want)


@pytest.mark.parametrize("place", ["new", "same"])
@pytest.mark.parametrize("aliased", [False, True])
def test_entries_behind_the_weights(dsa, place, aliased):
    """An entry at or behind n moves its row; it has no weight, which is recorded."""
    cache, table, new_table, g = setup_rows(dsa, 2, [60, 60], 6, 16, "bf16", 12)
    keep = i32([[1, 4, 9, 10, 40, 59], [0, 2, 5, 6, 8, 9]])
    to = new_table if place == "new" else table
    want = moved(cache, table, to, keep, 16)
    mass = torch.rand(2, 10, generator=g, device="cuda") + 1
    want_mass = torch.zeros(2, 10, device="cuda")
    for b in range(2):
        for j, e in enumerate(keep[b].tolist()):
            if e < 10:
                want_mass[b, j] = mass[b, e]
    out = mass if aliased else torch.full_like(mass, -1.0)
    dsa.dsa_cache_compact(cache, table, i32([60, 60]), keep, new_table if place == "new" else None, DC, DR,
                          fmt="bf16", mass=mass, new_mass=out)
    assert bad_index(dsa)
    assert torch.equal(out, want_mass)
    assert np.array_equal(cache.cpu().numpy().reshape(want.shape), want)
    # without those entries nothing is recorded
    keep[0, 3:] = -1
    dsa.dsa_cache_compact(cache, table, i32([60, 60]), keep, new_table if place == "new" else None, DC, DR,
                          fmt="bf16", mass=out, new_mass=out)
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("Sq", [1, 9])
def test_weights_of_calls_that_follow_at_once(dsa, fmt, Sq):
    """Blocks that end with their last products, one launch behind the other: the same bits every time."""
    lens = [Sq + b for b in range(20)] + [300, 513]
    Q, cache, table, ln, lse, scale, _, rows = mass_inputs(dsa, lens, Sq, 16, 16, fmt, 151)
    want = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 520, fmt=fmt)
    mass_check(want, Q, rows, lens, lse, scale)
    got = [dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 520, fmt=fmt) for _ in range(200)]
    assert all(torch.equal(m, want) for m in got)
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("Sq,H,k", [
    (1, 1, 0), (1, 16, 0), (1, 31, 0), (1, 32, 0), (1, 33, 0), (3, 16, 0), (1, 49, 0), (5, 16, 0), (1, 65, 0),
    (7, 16, 0), (1, 97, 0), (1, 127, 0), (129, 1, 0), (2, 15, 30), (2, 17, 30), (2, 48, 30), (2, 80, 30),
    (2, 112, 30)])
def test_weights_of_every_number_of_pairs(dsa, fmt, Sq, H, k):
    """Numbers of (token, head) pairs on both sides of every width of the products."""
    lens = [Sq, Sq + 40, 300]
    Q, cache, table, ln, lse, scale, idx, rows = mass_inputs(dsa, lens, Sq, H, 16, fmt, 161, k)
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 301, fmt=fmt, idx=idx)
    mass_check(got, Q, rows, lens, lse, scale, idx)
    no_error(dsa)


FIRST_CALLS = """
import threading, torch
import sparse_attention_index_gb300 as dsa
B, Sq, H, n = 2, 1, 16, 100
dev = torch.device("cuda:0")
g = torch.Generator(device=dev).manual_seed(5)
Q = torch.randn(B, Sq, H, 576, generator=g, device=dev).to(torch.bfloat16)
cache = torch.zeros(14, 16, 1152, dtype=torch.uint8, device=dev)
rows = torch.randn(14 * 16, 576, generator=g, device=dev).to(torch.bfloat16)
cache.view(-1, 1152).copy_(rows.view(torch.uint8).view(-1, 1152))
table = torch.arange(14, dtype=torch.int32, device=dev).view(2, 7)
lens = torch.tensor([100, 60], dtype=torch.int32, device=dev)
lse = torch.full((B, Sq, H), 3.0, device=dev)
torch.cuda.synchronize()
got, gate = [None] * 8, threading.Barrier(8)
def work(i):
    s = torch.cuda.Stream()
    gate.wait()
    got[i] = dsa.dsa_cache_mass(Q, cache, table, lens, lse, 0.05, n, fmt="bf16", stream=s)
    s.synchronize()
threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
for t in threads: t.start()
for t in threads: t.join()
want = dsa.dsa_cache_mass(Q, cache, table, lens, lse, 0.05, n, fmt="bf16")
assert all(torch.equal(m, want) for m in got)
assert bool(want[0].gt(0).all()) and not want[1, 60:].any()
assert dsa.dsa_get_last_device_error() == 0
"""


def test_first_calls_from_several_threads(dsa):
    """A process whose first calls come from eight host threads at once."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("place", ["new", "same"])
@pytest.mark.parametrize("fmt,dims", [("bf16", (128, 0)), ("bf16", (1024, 256)), ("bf16", (640, 72)),
                                      ("e4m3", (128, 0)), ("e4m3", (1024, 256)), ("e4m3", (384, 200))])
def test_rows_of_every_width(dsa, place, fmt, dims):
    """The narrowest and the widest rows, and odd numbers of 16-byte pieces."""
    lens, budget, page = [90, 301, 77], 80, 16
    cache, table, new_table, g = setup_rows(dsa, 3, lens, budget, page, fmt, sum(dims), dims)
    keep = torch.full((3, budget), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        at = torch.randperm(n, generator=g, device="cuda")[:budget].sort().values
        keep[b, :len(at)] = at.to(torch.int32)
    want = moved(cache, table, new_table if place == "new" else table, keep, page)
    dsa.dsa_cache_compact(cache, table, i32(lens), keep, new_table if place == "new" else None, *dims, fmt=fmt)
    assert np.array_equal(cache.cpu().numpy().reshape(want.shape), want)
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_serving_goes_on_after_a_cut(dsa, fmt):
    """The steps that a user makes: one with the weights kept, the cut in place with the indexer's keys along,
    and the next one, whose positions go on from the old length and whose lengths from the new one."""
    lens, H, page, budget, n, scale = [300, 40, 777, 129], 16, 16, 100, 800, 192 ** -0.5
    _, cache, table, _, _, _, _, rows = mass_inputs(dsa, lens, 1, H, page, fmt, 171)
    g, B = gen(172), len(lens)
    inv, m = dsa.rope_frequencies(64, scaling="yarn", factor=8.0)
    Q = torch.randn(B, 1, H, D, generator=g, device="cuda").to(torch.bfloat16)
    kv = torch.randn(B, 1, D, generator=g, device="cuda").to(torch.bfloat16)
    keys = torch.randn(B, n, 128, generator=g, device="cuda").to(torch.bfloat16)
    mass = torch.zeros(B, n, device="cuda")

    def step(pos, at, count):
        slots = (table.long().gather(1, (at // page).long()[:, None]) * page + (at % page)[:, None]).to(torch.int32)
        O, lse = dsa.dsa_decode_layer(Q, kv, pos[:, None].contiguous(), inv, slots, cache, table, count, scale,
                                      fmt=fmt, mscale=m, mass=mass, decay=0.5)
        new = dsa.dsa_cache_read(cache, slots.view(-1), DC, DR, fmt=fmt).double()
        return O, lse, new, dsa.dsa_rope(Q, pos[:, None].contiguous(), inv, off=DC, mscale=m)

    # the newest row of each sequence is that of the first step
    ln = i32(lens)
    O, lse, new, q = step(ln - 1, ln - 1, ln)
    have = [torch.cat([rows[b][:lens[b] - 1], new[b:b + 1]]) for b in range(B)]
    attn_check(O, lse, q, have, lens, scale)
    mass_check(mass, q, have, lens, lse, scale)
    keep, count = dsa.dsa_cache_keep(mass, ln, budget, sink=2, recent=10)
    before, old_keys = mass.clone(), keys.clone()
    dsa.dsa_cache_compact(cache, table, ln, keep, None, DC, DR, fmt=fmt, mass=mass, new_mass=mass)
    # the indexer's keys: a cache of one page a sequence, without positional dims
    dsa.dsa_cache_compact(keys.view(torch.uint8).view(B, n, 256), torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous(),
                          ln, keep, None, 128, 0, fmt="bf16")
    kept = [keep[b][keep[b] >= 0].long() for b in range(B)]
    for b in range(B):
        assert torch.equal(keys[b, :len(kept[b])], old_keys[b, kept[b]])
        assert torch.equal(keys[b, len(kept[b]):], old_keys[b, len(kept[b]):])
        assert torch.equal(mass[b, :len(kept[b])], before[b, kept[b]]) and not mass[b, len(kept[b]):].any()
    # the next token: its position as if nothing had been cut, its place behind what was kept
    prev, now = mass.clone(), [len(k) + 1 for k in kept]
    O, lse, new, q = step(ln, count, count + 1)
    have = [torch.cat([have[b][kept[b]], new[b:b + 1]]) for b in range(B)]
    attn_check(O, lse, q, have, now, scale)
    mass_check(mass, q, have, now, lse, scale, None, prev, 0.5)
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_decode_layer_with_lists_and_weights(dsa, fmt):
    """A serving step over selected positions that keeps their weights, in place, gives what its parts give."""
    lens, Sq, H, k, n = [300, 41], 2, 24, 64, 310
    Q, cache, table, ln, _, scale, idx, _ = mass_inputs(dsa, lens, Sq, H, 16, fmt, 181, k)
    g = gen(182)
    inv, m = dsa.rope_frequencies(64)
    kv = torch.randn(2, Sq, D, generator=g, device="cuda").to(torch.bfloat16)
    at = (ln[:, None] - Sq + torch.arange(Sq, device="cuda")).to(torch.int32)
    slots = (table.long().gather(1, (at // 16).long()) * 16 + at % 16).to(torch.int32)
    mass = torch.rand(2, n, generator=g, device="cuda")
    other, prev = cache.clone(), mass.clone()
    O, lse = dsa.dsa_decode_layer(Q, kv, at, inv, slots, cache, table, ln, scale, fmt=fmt, idx=idx, mscale=m,
                                  mass=mass, decay=0.75)
    rot = dsa.dsa_rope(kv[:, :, None].contiguous(), at, inv, off=DC, mscale=m)
    dsa.dsa_cache_write(rot.view(-1, D), slots.view(-1), other, DC, fmt=fmt)
    q = dsa.dsa_rope(Q, at, inv, off=DC, mscale=m)
    O2, lse2 = dsa.dsa_latent_attn(q, other, table, ln, scale, fmt=fmt, idx=idx)
    want = dsa.dsa_cache_mass(q, other, table, ln, lse2, scale, n, fmt=fmt, idx=idx, prev=prev, decay=0.75)
    assert torch.equal(O, O2) and torch.equal(lse, lse2) and torch.equal(mass, want) and torch.equal(cache, other)
    rows = [dsa.dsa_cache_read(other, (table[b].long()[torch.arange(x, device="cuda") // 16] * 16
                                       + torch.arange(x, device="cuda") % 16).to(torch.int32), DC, DR, fmt=fmt).double()
            for b, x in enumerate(lens)]
    mass_check(want, q, rows, lens, lse2, scale, idx, prev, 0.75)
    no_error(dsa)


@pytest.mark.parametrize("place", ["new", "same"])
@pytest.mark.parametrize("aliased", [False, True])
def test_weight_of_a_row_without_a_page(dsa, place, aliased):
    """A page that is none of the cache's moves no row; the weights move as they would."""
    cache, table, new_table, g = setup_rows(dsa, 1, [60], 20, 16, "e4m3", 13)
    table[0, 2] = cache.shape[0]
    before = cache.clone().view(-1, cache.shape[-1])
    keep = i32([[33, 34] + [-1] * 18])
    mass = torch.rand(1, 60, generator=g, device="cuda") + 1
    want = torch.zeros(1, 60, device="cuda")
    want[0, :2] = mass[0, 33:35]
    out = mass if aliased else torch.full_like(mass, -1.0)
    dsa.dsa_cache_compact(cache, table, i32([60]), keep, new_table if place == "new" else None, DC, DR, mass=mass,
                          new_mass=out)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_EVICT | dsa.DSA_DEVERR_BAD_PAGE
    assert torch.equal(out, want) and torch.equal(cache.view(before.shape), before)
