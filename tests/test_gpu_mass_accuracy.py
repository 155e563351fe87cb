"""How accurate the weights of cached positions are on ordinary values, and on logits far from zero.

test_gpu_eviction bounds them for any values at all (each of 576 products as large as they come). Here the
error follows the arithmetic that is stated for them, with S = q . row, x = scale S - lse, w = exp(x):

* S is two fp32 accumulators, of dims 0 to 319 and 320 to 575, which take 16 dims at a time. A step may cut
  off what is behind the last bit of the largest number in it (the accumulator in front of it or behind it,
  or a product), once where the products are lined up and once in the result: 2 * 2^-23 of that number. Adding
  the two accumulators up is one rounding, 2^-24 |S|.
* x is one rounding (2^-24 |x|), its change of base another, log2(e) itself is off by less than 2^-24: no more
  than 3 * 2^-24 |x|. The exponential is off by at most 2^-22 of w. The scale is the fp32 number that the
  kernel gets.
* A position's sum adds a sixteenth of up to 64 pairs at a time to each of four sums, then these, the other 64
  pairs, one number for each further 128 pairs, and with lists one for each token: at most
  16 + 5 + ceil(pairs / 128) + Sq roundings of 2^-24 of the whole, all weights being positive.

The norm of all errors is held to a few times the relative error that is stated for them, 7e-7: a cut is half
a bit on average and only the accumulator's own, which leaves 3e-6 as room.
"""
import math

import pytest
import torch

from test_gpu_eviction import mass_inputs, seen
from test_gpu_serving import D, DC, DR, gen, i32, no_error

pytestmark = pytest.mark.gpu

SPLIT = 320


@pytest.fixture(scope="module")
def dsa():
    import sparse_attention_index_gb300 as m
    m.dsa_get_last_device_error()
    return m


def f32(x):
    return float(torch.tensor(x, dtype=torch.float32))


def cut_off(q, kv):
    """What may be cut off S [H, n], as above."""
    lost = torch.zeros(q.shape[0], kv.shape[0], dtype=torch.float64, device=q.device)
    for first, end in ((0, SPLIT), (SPLIT, D)):
        acc = torch.zeros_like(lost)
        for d in range(first, end, 16):
            p = q[:, None, d:d + 16] * kv[None, :, d:d + 16]
            now = acc + p.sum(-1)
            lost += torch.maximum(torch.maximum(acc.abs(), now.abs()), p.abs().amax(-1))
            acc = now
    return 2.0 ** -22 * lost


def accurate(got, Q, rows, lens, lse, scale, idx=None, exact=False):
    """Every weight within the bound; exact: nothing can be cut off S."""
    scale, (B, Sq, H, _) = f32(scale), Q.shape
    depth = 16 + 5 + -(-Sq * H // 128) + Sq
    err2 = ref2 = 0.0
    for b in range(B):
        ref = torch.zeros(got.shape[1], dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(ref)
        for i in range(Sq):
            at = seen(lens[b], Sq, i, None if idx is None else idx[b, i])
            if len(at) == 0:
                continue
            q, kv = Q[b, i].double(), rows[b][at]
            S = q @ kv.T
            x = scale * S - lse[b, i].double()[:, None]
            off = 3 * 2.0 ** -24 * x.abs() + 2.0 ** -22
            if not exact:
                off += scale * (cut_off(q, kv) + 2.0 ** -24 * S.abs())
            w = torch.exp(x)
            ref.index_add_(0, at, w.sum(0))
            tol.index_add_(0, at, (w * torch.expm1(off)).sum(0))
        tol += depth * 2.0 ** -24 * ref
        err = (got[b].double() - ref).abs()
        assert bool((err <= tol).all()), (b, float((err / ref.clamp(min=1e-300)).max()), float((err - tol).max()))
        err2 += float((err * err).sum())
        ref2 += float((ref * ref).sum())
    return math.sqrt(err2 / ref2)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,Sq,H,k", [
    ([489, 130], 1, 16, 0), ([300], 1, 128, 0), ([257, 64], 3, 40, 0), ([700, 65], 2, 128, 0), ([200], 20, 16, 0),
    ([900, 77], 1, 16, 200), ([300], 2, 128, 100)])
def test_ordinary_values(dsa, fmt, lens, Sq, H, k):
    Q, cache, table, ln, lse, scale, idx, rows = mass_inputs(dsa, lens, Sq, H, 16, fmt, 201, k)
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, max(lens), fmt=fmt, idx=idx)
    assert accurate(got, Q, rows, lens, lse, scale, idx) <= 3e-6
    no_error(dsa)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("Sq,H,k", [(1, 16, 0), (1, 128, 0), (9, 16, 0), (2, 24, 150)])
@pytest.mark.parametrize("far", [0, 125, -125])
def test_logits_far_from_zero(dsa, fmt, Sq, H, k, far):
    """Logits around 0, 1000 and -1000 whose S is a multiple of 2^-4 below 2^15, which no addition cuts
    anything off: what is left is the arithmetic behind it, where lse (as large) has to be taken off first.
    Taken off behind the change of base, it would move the weights by 1e-4."""
    B, n, scale = 2, 500, 0.0625
    lens, g = [n, n - 131], gen(211)
    Q = (torch.randint(-8, 9, (B, Sq, H, D), generator=g, device="cuda") / 4).to(torch.bfloat16)
    kv = (torch.randint(-8, 9, (B, n, D), generator=g, device="cuda") / 4).to(torch.bfloat16)
    Q[..., D - 1] = 128.0
    kv[..., D - 1] = far                                    # a positional dim, bf16 in either format
    cache = torch.zeros(40 * B, 16, dsa.cache_row_bytes(DC, DR, fmt), dtype=torch.uint8, device="cuda")
    table = torch.randperm(40 * B, generator=g, device="cuda").to(torch.int32).view(B, 40)
    at = torch.arange(n, device="cuda")
    for b in range(B):
        slots = (table[b].long()[at // 16] * 16 + at % 16).to(torch.int32)
        dsa.dsa_cache_write(kv[b], slots, cache, DC, fmt=fmt)
        assert torch.equal(dsa.dsa_cache_read(cache, slots, DC, DR, fmt=fmt), kv[b])
    idx = None
    if k:
        idx = torch.stack([torch.randperm(lens[b], generator=g, device="cuda")[:k].sort().values
                           for b in range(B) for _ in range(Sq)]).to(torch.int32).view(B, Sq, k)
    rows = [kv[b, :lens[b]].double() for b in range(B)]
    lse = torch.full((B, Sq, H), -math.inf, device="cuda")
    for b in range(B):
        for i in range(Sq):
            keys = rows[b][seen(lens[b], Sq, i, None if idx is None else idx[b, i])]
            lse[b, i] = torch.logsumexp(scale * (Q[b, i].double() @ keys.T), -1).float()
    if far:
        assert float(lse.abs().min()) > 900
    got = dsa.dsa_cache_mass(Q, cache, table, i32(lens), lse, scale, n, fmt=fmt, idx=idx)
    accurate(got, Q, rows, lens, lse, scale, idx, exact=True)
    no_error(dsa)


def test_lse_of_plus_infinity(dsa):
    """A token whose logits are past fp32 (lse = +inf) adds nothing where Q . row is finite."""
    Q, cache, table, ln, lse, scale, _, rows = mass_inputs(dsa, [200], 2, 16, 16, "bf16", 221)
    lse[0, 0] = math.inf
    got = dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 200, fmt="bf16")
    lse[0, 0] = -math.inf                     # a token that has no key adds nothing either
    assert torch.equal(got, dsa.dsa_cache_mass(Q, cache, table, ln, lse, scale, 200, fmt="bf16"))
    no_error(dsa)
