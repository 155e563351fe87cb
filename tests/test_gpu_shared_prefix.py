"""Attention of sequences that share cached prefixes, against the definition in 64 bits: each token's
keys are its group's prefix and its own positions, and its output is held to the tolerances of
test_gpu_serving (the join adds fp32 parts, as that of a split sequence does)."""
import math

import pytest
import torch

from test_gpu_serving import D, DC, attn_check, gen, i32, make_cache, no_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_index_gb300 as m
    m.dsa_get_last_device_error()
    return m


class Batch:
    """A cache with the rows of G prefixes and B sequences, and the tables to call with."""

    def __init__(self, dsa, starts, prefixes, lens, Sq, H, page, fmt, seed, scale=1.0):
        G, B = len(prefixes), len(lens)
        self.cache, table, self.rows = make_cache(dsa, prefixes + lens, page, fmt, seed, scale)
        self.prefix_table, self.table = table[:G].clone(), table[G:].clone()
        self.prefixes, self.lens, self.starts = prefixes, lens, starts
        self.G, self.B, self.Sq, self.H, self.fmt = G, B, Sq, H, fmt
        self.Q = torch.randn(B, Sq, H, D, generator=gen(seed + 1), device="cuda").to(torch.bfloat16)
        self.scale = 192 ** -0.5
        self.args = (self.Q, self.cache, self.prefix_table, i32(prefixes), i32(starts), self.table, i32(lens),
                     self.scale)

    def run(self, dsa, **more):
        O = torch.full((self.B, self.Sq, self.H, DC), math.nan, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.B, self.Sq, self.H), math.nan, device="cuda")
        return dsa.dsa_latent_attn_shared(*self.args, fmt=self.fmt, O=O, lse=lse, **more)

    def keys(self, b, i):
        """The rows that token i of sequence b sees."""
        end = max(self.lens[b], 0) - self.Sq + i + 1
        if end < 1:
            return self.rows[self.G + b][:0]
        s = self.starts
        g = [g for g in range(self.G) if s[g] <= b < s[g + 1]]
        mine = self.rows[self.G + b][:end]
        return torch.cat([self.rows[g[0]], mine]) if g else mine

    def check(self, O, lse):
        for b in range(self.B):
            for i in range(self.Sq):
                keys = self.keys(b, i)
                at = (slice(b, b + 1), slice(i, i + 1))
                attn_check(O[at], lse[at], self.Q[at], [keys], [len(keys)], self.scale)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("starts,prefixes,lens,Sq,H,page", [
    ([0, 1], [1], [1], 1, 1, 16),                               # one key in each part
    ([0, 4], [489], [33, 1, 17, 33], 1, 16, 64),
    ([0, 3], [5000], [700, 1, 49], 1, 128, 64),
    ([0, 9], [100], [3] * 9, 1, 20, 7),                         # a sequence's rows in two prefix tiles
    ([0, 2, 2, 7], [48, 500, 97], [5, 60, 1, 47, 48, 49, 200], 2, 16, 16),   # an empty group
    ([1, 4, 6], [300, 0], [9, 10, 11, 12, 13, 14, 15], 1, 33, 32),           # no prefix: first, last, len 0
    ([0, 5], [200], [0, 3, 1, 2, 50], 3, 16, 16),               # tokens without a place
    ([0, 2], [150], [0, -4], 2, 5, 16),                         # padding alone
    ([0, 2], [97], [130, 7], 7, 100, 100),                      # several own tiles a sequence
    ([0, 130], [60], [1 + b % 5 for b in range(130)], 1, 8, 4),
    ([0, 1], [30000], [1], 1, 128, 64)])
def test_shared(dsa, fmt, starts, prefixes, lens, Sq, H, page):
    t = Batch(dsa, starts, prefixes, lens, Sq, H, page, fmt, 21)
    no_error(dsa)
    O, lse = t.run(dsa)
    want = dsa.DSA_STAGE_LATENT | dsa.DSA_DEVERR_BAD_PAGE if min(lens) < 0 else 0
    assert dsa.dsa_get_last_device_error() == want
    t.check(O, lse)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_many_groups_and_long_parts(dsa, fmt):
    """Enough keys that several tiles lie in one cluster's range and one tile in several."""
    B, G = 40, 13
    starts = [0] + [min(B, 1 + g * g // 4) for g in range(1, G)] + [B]
    t = Batch(dsa, starts, [(g * 977) % 9000 + 1 for g in range(G)], [1 + (b * 379) % 2500 for b in range(B)],
              2, 24, 64, fmt, 31)
    O, lse = t.run(dsa)
    no_error(dsa)
    t.check(O, lse)
    again = t.run(dsa)
    assert torch.equal(again[0], O) and torch.equal(again[1], lse)       # the same bits


def test_most_groups(dsa):
    t = Batch(dsa, list(range(65)), [1 + g % 50 for g in range(64)], [2] * 64, 1, 16, 16, "e4m3", 41)
    t.check(*t.run(dsa))
    no_error(dsa)


def test_agrees_with_one_table(dsa):
    """Prefix pages in front of the own pages in one table give the same attention."""
    page, P = 16, 160                                                     # the prefix ends with a page
    t = Batch(dsa, [0, 6], [P], [5, 40, 1, 300, 17, 2], 1, 16, page, "bf16", 51)
    table = torch.cat([t.prefix_table[:, :P // page].expand(6, -1), t.table], 1).contiguous()
    O, lse = t.run(dsa)
    O1, lse1 = dsa.dsa_latent_attn(t.Q, t.cache, table, i32([P + n for n in t.lens]), t.scale, fmt="bf16")
    # both are within 2^-7 of the definition's norm
    assert float((O.double() - O1.double()).norm()) <= 2.0 ** -6 * float(O1.double().norm())
    assert float((lse - lse1).abs().max()) <= 1e-4
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_nan_stays_with_those_that_see_it(dsa, fmt):
    t = Batch(dsa, [0, 2, 5], [70, 70], [9, 8, 7, 0, 6], 2, 16, 16, fmt, 61)
    clean = t.run(dsa)
    # a row of the second group's prefix, and the newest row of sequence 0
    for table, j in ((t.prefix_table[1], 33), (t.table[0], 8)):
        slot = int(table[j // 16]) * 16 + j % 16
        bad = torch.full((1, D), math.nan, dtype=torch.bfloat16, device="cuda")
        dsa.dsa_cache_write(bad, i32([slot]), t.cache, DC, fmt=fmt)
    O, lse = t.run(dsa)
    hit = torch.zeros(5, 2, dtype=torch.bool)
    hit[2:] = True
    hit[3] = False                                   # padding
    hit[0, 1] = True                                 # the token itself, not the one in front of it
    for b in range(5):
        for i in range(2):
            if hit[b, i]:
                assert bool(torch.isnan(O[b, i]).all()) and bool(torch.isnan(lse[b, i]).all())
            else:
                assert torch.equal(O[b, i], clean[0][b, i]) and torch.equal(lse[b, i], clean[1][b, i])
    no_error(dsa)


def test_bad_starts_and_pages(dsa):
    """They are taken as the nearest that are right, or skipped, and recorded."""
    t = Batch(dsa, [0, 2, 4], [40, 50], [5, 6, 7, 8], 1, 16, 16, "e4m3", 71)
    want = t.run(dsa)
    args = list(t.args)
    args[4] = i32([-3, 2, 99])
    O, lse = dsa.dsa_latent_attn_shared(*args)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_LATENT | dsa.DSA_DEVERR_BAD_INDEX
    assert torch.equal(O, want[0]) and torch.equal(lse, want[1])
    args[4] = i32([0, 4, 1])                          # goes down: the second group is empty
    O, lse = dsa.dsa_latent_attn_shared(*args)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_LATENT | dsa.DSA_DEVERR_BAD_INDEX
    t.starts = [0, 4, 4]
    t.check(O, lse)
    # the second group's second page is none of the cache's: its keys are not there
    t.starts = [0, 2, 4]
    args = list(t.args)
    args[2] = t.prefix_table.clone()
    args[2][1, 1] = t.cache.shape[0]
    O, lse = dsa.dsa_latent_attn_shared(*args)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_LATENT | dsa.DSA_DEVERR_BAD_PAGE
    t.rows[1] = torch.cat([t.rows[1][:16], t.rows[1][32:]])
    t.check(O, lse)
    # a prefix's length past its table is taken as what the table holds
    args[3] = i32([10 ** 6, -1])
    args[2] = t.prefix_table.clone()
    args[2][0, 3:] = args[2][0, 0]
    O, lse = dsa.dsa_latent_attn_shared(*args)
    assert dsa.dsa_get_last_device_error() == dsa.DSA_STAGE_LATENT | dsa.DSA_DEVERR_BAD_PAGE


def test_captured_and_on_other_streams(dsa):
    """Two captured calls with workspaces of their own replay with new lengths, and a call on another
    stream than the current one gives the same bits."""
    t = Batch(dsa, [0, 6], [700], [5, 40, 1, 300, 17, 2], 1, 16, 16, "e4m3", 81)
    u = Batch(dsa, [0, 1, 3], [90, 800], [30, 20, 10], 2, 64, 16, "bf16", 82)
    want = t.run(dsa), u.run(dsa)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    O, lse = dsa.dsa_latent_attn_shared(*t.args, fmt=t.fmt, stream=s)
    s.synchronize()
    assert torch.equal(O, want[0][0]) and torch.equal(lse, want[0][1])
    outs = []
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs.append(dsa.dsa_latent_attn_shared(*t.args, fmt=t.fmt))
        outs.append(dsa.dsa_latent_attn_shared(*u.args, fmt=u.fmt))
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    t.lens[3] = 120
    t.args[6].copy_(i32(t.lens))
    graph.replay()
    torch.cuda.synchronize()
    t.check(*outs[0])
    no_error(dsa)


def test_python_refusals(dsa):
    t = Batch(dsa, [0, 2], [40], [5, 6], 1, 16, 16, "e4m3", 91)
    names = ("Q", "cache", "prefix_table", "prefix_lens", "starts", "page_table", "lens", "scale")
    good = dict(zip(names, t.args))
    for bad in (dict(starts=i32([0])), dict(prefix_lens=i32([1, 2])), dict(lens=i32([1])),
                dict(prefix_table=t.prefix_table[0]), dict(page_table=t.table[:1].clone()),
                dict(cache=t.cache.view(-1, 656)), dict(fmt="bf16"),
                dict(O=torch.empty(2, 1, 16, 64, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            dsa.dsa_latent_attn_shared(**{**good, **bad})
    for bad in (dict(starts=t.args[4].long()), dict(Q=t.Q.float()), dict(lse=torch.empty(2, 1, 16))):
        with pytest.raises(TypeError):
            dsa.dsa_latent_attn_shared(**{**good, **bad})
    with pytest.raises(dsa.DsaError):
        dsa.dsa_latent_attn_shared(**good, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("shared", [True, False])
def test_decode_layer_with_prefix_and_weights(dsa, fmt, shared):
    """One serving step over shared prefixes that keeps the positions' weights gives what its parts give."""
    t = Batch(dsa, [0, 2, 4], [90, 200], [37, 2, 0, 160], 2, 16, 16, fmt, 101)
    inv, m = dsa.rope_frequencies(64, scaling="yarn", factor=8.0)
    g = gen(102)
    Q = torch.randn(4, 2, 16, D, generator=g, device="cuda").to(torch.bfloat16)
    kv = torch.randn(4, 2, D, generator=g, device="cuda").to(torch.bfloat16)
    n = i32(t.lens)
    at = (n[:, None] - 2 + torch.arange(2, device="cuda")).clamp(min=0).long()
    slots = (t.table.long().gather(1, at // 16) * 16 + at % 16).to(torch.int32)
    slots[2] = -1                                       # the padded sequence
    pos = at.to(torch.int32)
    mass = torch.rand(4, 170, generator=g, device="cuda")
    one, mine = t.cache.clone(), mass.clone()
    prefix = (t.prefix_table, i32(t.prefixes), i32(t.starts))
    for _ in range(2):                                  # the second with the same rows again
        O, lse = dsa.dsa_decode_layer(Q, kv, pos, inv, slots, one, t.table, n, 0.07, fmt=fmt, mscale=m,
                                      prefix=prefix if shared else None, mass=mine, decay=0.5)
    rot = dsa.dsa_rope(kv[:, :, None].contiguous(), pos, inv, off=DC, mscale=m)
    dsa.dsa_cache_write(rot.view(-1, D), slots.view(-1), t.cache, DC, fmt=fmt)
    q = dsa.dsa_rope(Q, pos, inv, off=DC, mscale=m)
    if shared:
        O2, lse2 = dsa.dsa_latent_attn_shared(q, t.cache, *prefix, t.table, n, 0.07, fmt=fmt)
    else:
        O2, lse2 = dsa.dsa_latent_attn(q, t.cache, t.table, n, 0.07, fmt=fmt)
    for _ in range(2):
        mass = dsa.dsa_cache_mass(q, t.cache, t.table, n, lse2, 0.07, 170, fmt=fmt, prev=mass, decay=0.5)
    assert torch.equal(one, t.cache) and torch.equal(O, O2) and torch.equal(lse, lse2)
    assert torch.equal(mine, mass)
    # refused steps leave the cache and the weights
    before = one.clone()
    good = dict(Q=Q, kv=kv, pos=pos, inv_freq=inv, slots=slots, cache=one, page_table=t.table, lens=n, scale=0.07,
                fmt=fmt, prefix=prefix, mass=mine)
    many = tuple(torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((65, 1), (65,), (66,)))
    for bad in (dict(prefix=many), dict(prefix=(prefix[0], prefix[1], prefix[2][:2].clone())), dict(decay=math.inf),
                dict(mass=mine[0]), dict(mass=mine.double()), dict(idx=torch.zeros(4, 2, 3, dtype=torch.int32, device="cuda")),
                dict(scale=0.0), dict(ws=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((dsa.DsaError, ValueError, TypeError)):
            dsa.dsa_decode_layer(**{**good, **bad})
    assert torch.equal(one, before) and torch.equal(mine, mass)
    no_error(dsa)
