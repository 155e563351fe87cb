"""Measured cases of the operators around a full serving cache: attention of a batch that shares long
prefixes, and eviction from the cache by accumulated attention weight.

Four operators, each with its plain form in elementary torch operations and the call that a user makes:

* ``shared``  - attention of the newest tokens of each sequence over its group's cached prefix and its
  own cached rows (a prefix is stored once for all sequences of its group);
* ``mass``    - the attention weight that each cached position receives from the newest tokens, summed
  over tokens and heads and added to the (decayed) weight of earlier steps;
* ``keep``    - the positions that stay when a sequence is cut to a budget: the first ones, the newest
  ones and the heaviest of the others;
* ``compact`` - the kept rows moved to pages of their own, and their weights with them.

A cache row holds 512 latent dims and 64 positional dims. "bf16": all of them in bf16. "e4m3": the latent
dims in e4m3, one fp32 power-of-two scale per 128 of them, then the positional dims in bf16.
"""
import math

import torch

own = False

DEV = "cuda"
DC, DR, GROUP = 512, 64, 128
D = DC + DR


# ------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # four answers to one short question on a rank with 16 of the heads: latency
        dict(name="shared_few_short", op="shared", G=1, B=4, Sq=1, H=16, prefix=489, len=33, ragged=True, loose=0, page=64, fmt="bf16"),
        # a batch of questions about one long document, 16 heads
        dict(name="shared_document_bf16", op="shared", G=1, B=64, Sq=1, H=16, prefix=32768, len=1024, ragged=True, loose=0, page=64, fmt="bf16"),
        # three groups of unequal size with prefixes of their own, four drafted tokens each
        dict(name="shared_groups_e4m3", op="shared", G=3, B=48, Sq=4, H=16, prefix=16000, len=500, ragged=True, loose=1, page=16, fmt="e4m3"),
        # all heads on one GPU, a long system prompt
        dict(name="shared_heads_e4m3", op="shared", G=1, B=32, Sq=1, H=128, prefix=8192, len=512, ragged=True, loose=0, page=64, fmt="e4m3"),
        # one short sequence on a rank with 16 of the heads: latency
        dict(name="mass_one_short", op="mass", B=1, Sq=1, H=16, len=489, ragged=False, page=64, fmt="bf16", k=0, prev=True),
        # a ragged decode batch, weights of earlier steps decayed
        dict(name="mass_batch_e4m3", op="mass", B=32, Sq=1, H=128, len=8192, ragged=True, page=64, fmt="e4m3", k=0, prev=True),
        # the last 32 tokens of a prompt look over it before it is cut
        dict(name="mass_window_bf16", op="mass", B=2, Sq=32, H=128, len=16384, ragged=False, page=64, fmt="bf16", k=0, prev=False),
        # the weights of the selected 2048 keys of each token
        dict(name="mass_selected_e4m3", op="mass", B=128, Sq=1, H=128, len=4096, ragged=False, page=64, fmt="e4m3", k=2048, prev=True),
        # a decode batch cut to 2048 positions
        dict(name="keep_batch", op="keep", B=64, len=8192, ragged=True, budget=2048, sink=4, recent=128, ties=False),
        # few long contexts, many equal weights
        dict(name="keep_long", op="keep", B=2, len=131072, ragged=False, budget=16384, sink=64, recent=1024, ties=True),
        # the batch's rows moved
        dict(name="compact_batch_e4m3", op="compact", B=64, len=8192, ragged=True, budget=2048, sink=4, recent=128, page=64, fmt="e4m3"),
        # the long contexts' rows moved
        dict(name="compact_long_bf16", op="compact", B=2, len=131072, ragged=False, budget=16384, sink=64, recent=1024, page=64, fmt="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "mass", "mass", "keep", "compact"])
    fmt = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 32, 64, 100])
    ragged = rng.random() < 0.7
    if op == "shared":
        H = rng.choice([8, 16, 20, 32, 64, 128])
        Sq = rng.choice([1, 1, 1, 2, 4, 7])
        B = _log(rng, 1, 96)
        G = rng.choice([1, 1, 2, 3, 7])
        most = 36_000_000 // (B * Sq * H)                       # keys a sequence
        prefix = _log(rng, 1, min(65536, most, 2_000_000 // B))
        return dict(op=op, G=G, B=B, Sq=Sq, H=H, prefix=prefix, len=_log(rng, Sq, min(2048, most)), ragged=ragged,
                    loose=rng.choice([0, 0, 1, 2]) if B > 4 else 0, page=page, fmt=fmt)
    if op == "mass":
        H = rng.choice([8, 16, 20, 32, 64, 128])
        Sq = rng.choice([1, 1, 1, 2, 5, 16, 32])
        k = rng.choice([0, 0, 0, 64, 500, 2048])
        B = _log(rng, 1, 128 // Sq if k else 128)
        n = _log(rng, Sq, max(Sq + 1, min(131072, 160000 // (B * Sq) if k else 160000 // B, 134_000_000 // (B * Sq * H))))
        return dict(op=op, B=B, Sq=Sq, H=H, len=n, ragged=ragged, page=page, fmt=fmt, k=k, prev=rng.random() < 0.6)
    B = _log(rng, 1, 128)
    n = _log(rng, 1, min(131072, 260000 // B) if op == "keep" else 80000 // B)
    budget = _log(rng, 1, n + n // 4 + 1)
    sink = rng.randrange(0, min(64, budget) + 1)
    recent = _log(rng, 1, budget - sink) if budget > sink else 0
    c = dict(op=op, B=B, len=n, ragged=ragged, budget=budget, sink=sink, recent=recent)
    return {**c, "ties": rng.random() < 0.5} if op == "keep" else {**c, "page": page, "fmt": fmt}


def row_bytes(fmt):
    return 2 * D if fmt == "bf16" else DC + 16 + 2 * DR


def lens_of(c):
    """Each sequence's own cached tokens, its new ones among them: a ramp where ragged."""
    least = c.get("Sq", 1)
    if not c["ragged"]:
        return [c["len"]] * c["B"]
    return [max(least, c["len"] * (b + 1) // c["B"]) for b in range(c["B"])]


def groups_of(c):
    """(first sequence of each group and the end of the last, prefix of each group): groups grow in size and length."""
    G, n = c["G"], c["B"] - c["loose"]
    return [n * g * g // (G * G) for g in range(G + 1)], [max(1, c["prefix"] * (g + 1) // G) for g in range(G)]


def work(c):
    lens, n = lens_of(c), c["B"]
    if c["op"] == "keep":
        return {"bytes": 4 * sum(lens) + 4 * n + 4 * n * (c["budget"] + 1), "flops": 0}
    if c["op"] == "compact":
        kept = sum(min(c["budget"], x) for x in lens)
        return {"bytes": kept * (2 * row_bytes(c["fmt"]) + 4) + 4 * n * (2 * c["budget"] + 1)
                + 8 * sum(-(-x // c["page"]) for x in lens), "flops": 0}
    Sq, H = c["Sq"], c["H"]
    tokens = n * Sq
    pages = 4 * sum(-(-x // c["page"]) for x in lens)
    seen = [[x - Sq + i + 1 for i in range(Sq)] for x in lens]
    if c["op"] == "shared":
        starts, prefixes = groups_of(c)
        pairs = sum(sum(s) for s in seen) + sum((b - a) * Sq * p for a, b, p in zip(starts, starts[1:], prefixes))
        rows = sum(lens) + sum(p for a, b, p in zip(starts, starts[1:], prefixes) if b > a)
        return {"bytes": rows * row_bytes(c["fmt"]) + tokens * H * (2 * D + 2 * DC + 4) + pages + 4 * n
                + 4 * sum(-(-p // c["page"]) for p in prefixes), "flops": 2 * pairs * H * (D + DC)}
    if c["k"]:
        seen = [[min(c["k"], x) for x in s] for s in seen]
    rows = sum(min(x, sum(s)) if c["k"] else x for x, s in zip(lens, seen))
    return {"bytes": rows * row_bytes(c["fmt"]) + tokens * H * (2 * D + 4) + pages + 4 * n + 4 * tokens * c["k"]
            + 4 * n * max(lens) + (4 * sum(lens) if c["prev"] else 0), "flops": 2 * sum(sum(s) for s in seen) * H * D}


# ----------------------------------------------------------------------------------------- inputs


def quantised(x):
    """fp32 [n, D] -> (codes float8 [n, DC], scales fp32 [n, DC / 128], rest bf16 [n, DR])."""
    g = x[:, :DC].reshape(-1, DC // GROUP, GROUP)
    mant, expo = torch.frexp(g.abs().amax(-1))           # amax = mant * 2^expo, mant in [1/2, 1)
    # the smallest power of two that brings amax to at most 448 = 0.875 * 2^9; 1 where all is zero
    k = torch.where(mant > 0.875, expo - 8, expo - 9)
    k = torch.where(mant == 0, torch.zeros_like(k), k).clamp(min=-120)
    scales = torch.ldexp(torch.ones_like(mant), k)
    codes = (g / scales[..., None]).to(torch.float8_e4m3fn)
    return codes.reshape(-1, DC), scales, x[:, DC:].to(torch.bfloat16)


def parts(cache, fmt):
    """The cache's rows [n, row] bytes as the values it holds: views, no copies."""
    if fmt == "bf16":
        return {"row": cache.view(torch.bfloat16)}
    return {"codes": cache[:, :DC].view(torch.float8_e4m3fn), "scales": cache[:, DC:DC + 16].view(torch.float32),
            "rest": cache[:, DC + 16:].view(torch.bfloat16)}


def fill(cache, fmt, at, x):
    """Writes rows x (fp32) at the slots `at`, in the plain form."""
    p = parts(cache, fmt)
    if fmt == "bf16":
        p["row"][at] = x.to(torch.bfloat16)
        return
    codes, scales, rest = quantised(x)
    p["codes"].view(torch.uint8)[at] = codes.view(torch.uint8)
    p["scales"][at] = scales
    p["rest"][at] = rest


def values(cache, fmt, at):
    """fp32 values of the rows at the slots `at` (any shape)."""
    p = parts(cache[at.reshape(-1)], fmt)
    if fmt == "bf16":
        v = p["row"].float()
    else:
        v = p["codes"].float().view(-1, DC // GROUP, GROUP) * p["scales"][..., None]
        v = torch.cat([v.reshape(-1, DC), p["rest"].float()], -1)
    return v.view(*at.shape, D)


def slots(table, page, at):
    """The slots of positions at [B, ...] through the page table [B, pages]."""
    return table.long().gather(1, (at // page).reshape(len(at), -1)).view_as(at) * page + at % page


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    lens, B = lens_of(c), c["B"]
    s = {"case": c, "lens": torch.tensor(lens, dtype=torch.int32, device=DEV)}
    if c["op"] in ("keep", "compact"):
        mass = torch.exp(2.0 * normal(B, max(lens)))     # a few positions hold most of the weight
        if c.get("ties"):
            mass = (mass * 8).round() / 8                # and many hold next to none
        s["mass"] = mass
        if c["op"] == "keep":
            return s
        s["keep"] = keep_plain(mass, s["lens"], c["budget"], c["sink"], c["recent"])["keep"]
    fmt, page = c["fmt"], c["page"]
    new = [min(x, c["budget"]) for x in lens] if c["op"] == "compact" else []
    starts, prefixes = groups_of(c) if c["op"] == "shared" else ([], [])
    need = [-(-n // page) for n in lens + new + prefixes]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)

    def table(counts, first):
        t = torch.zeros(len(counts), max(counts), dtype=torch.int32, device=DEV)
        for b, n in enumerate(counts):
            t[b, :n] = order[first:first + n]
            first += n
        return t

    cache = torch.zeros(total * page, row_bytes(fmt), dtype=torch.uint8, device=DEV)
    for a in range(0, total * page, 131072):
        e = min(total * page, a + 131072)
        fill(cache, fmt, torch.arange(a, e, device=DEV), normal(e - a, D))
    s.update(cache=cache.view(total, page, -1), table=table(need[:B], 0))
    if c["op"] == "compact":
        s["new_table"] = table([-(-c["budget"] // page)] * B, 0) * 0
        t = table(need[B:], sum(need[:B]))
        s["new_table"][:, :t.shape[1]] = t
        return s
    Sq, H = c["Sq"], c["H"]
    s.update(q=normal(B, Sq, H, D).to(torch.bfloat16), scale=192 ** -0.5)
    if c["op"] == "shared":
        s.update(prefix_table=table(need[B:], sum(need[:B])), prefix_lens=torch.tensor(prefixes, dtype=torch.int32, device=DEV),
                 starts=torch.tensor(starts, dtype=torch.int32, device=DEV))
        return s
    s["idx"] = None
    if c["k"]:
        n = max(lens)
        limit = s["lens"][:, None] - Sq + 1 + torch.arange(Sq, device=DEV)
        r = torch.rand(B, Sq, n, generator=g, device=DEV)
        r.masked_fill_(torch.arange(n, device=DEV) >= limit[..., None], -1.0)
        top = r.topk(min(c["k"], n), -1)
        at = torch.where(top.values >= 0, top.indices, n).sort(-1).values
        idx = torch.full((B, Sq, c["k"]), -1, dtype=torch.int32, device=DEV)
        idx[..., :at.shape[-1]] = torch.where(at < n, at, -1).to(torch.int32)
        s["idx"] = idx
    # the attention's own log-sum-exp, as the step has it
    s["lse"] = torch.logsumexp(logits_plain(s["q"], s["cache"], fmt, s["table"], s["lens"], s["scale"], s["idx"], max(lens))[0], -1)
    s["prev"] = torch.exp(2.0 * normal(B, max(lens))) * (torch.arange(max(lens), device=DEV) < s["lens"][:, None] - Sq) if c["prev"] else None
    return s


# ------------------------------------------------------------------------------------ plain forms


def logits_plain(q, cache, fmt, table, lens, scale, idx, n):
    """(logits [B, Sq, H, keys], -inf where a token does not see a key; the rows; the keys' positions)."""
    B, Sq, H, _ = q.shape
    pages, page, _ = cache.shape
    limit = lens[:, None] - Sq + 1 + torch.arange(Sq, device=q.device)      # keys each token sees
    if idx is None:
        at = torch.arange(n, device=q.device)[None, None]
        seen = at < limit[..., None]                                         # [B, Sq, n]
    else:
        at = idx.long()
        seen = (at >= 0) & (at < limit[..., None])
        at = at.clamp(min=0)
    at = at.expand(B, -1, -1)                                                # [B, 1 or Sq, keys]
    rows = values(cache.view(pages * page, -1), fmt, slots(table, page, at))   # [B, 1 or Sq, keys, D]
    if idx is None:
        logits = torch.matmul(q.float().view(B, 1, Sq * H, -1), rows.transpose(-1, -2)).view(B, Sq, H, -1)
    else:
        logits = torch.matmul(q.float(), rows.transpose(-1, -2))
    return (logits * scale).masked_fill_(~seen[:, :, None], -math.inf), rows, at


def shared_plain(q, cache, fmt, prefix_table, prefix_lens, starts, table, lens, scale, np, n):
    B, Sq, H, _ = q.shape
    pages, page, _ = cache.shape
    mine, rows, _ = logits_plain(q, cache, fmt, table, lens, scale, None, n)
    b = torch.arange(B, device=q.device)
    group = torch.bucketize(b, starts, right=True) - 1                       # -1 or G: none
    grouped = (group >= 0) & (group < len(prefix_lens))
    group = group.clamp(0, len(prefix_lens) - 1)
    at = torch.arange(np, device=q.device)
    before = values(cache.view(pages * page, -1), fmt, slots(prefix_table, page, at.expand(len(prefix_lens), -1)))[group]
    seen = (at < prefix_lens[group][:, None]) & grouped[:, None]             # [B, np]
    theirs = torch.matmul(q.float().view(B, Sq * H, -1), before.transpose(-1, -2)).view(B, Sq, H, -1) * scale
    theirs.masked_fill_(~seen[:, None, None], -math.inf)
    top = torch.maximum(mine.amax(-1, keepdim=True), theirs.amax(-1, keepdim=True))
    mine, theirs = torch.exp(mine - top), torch.exp(theirs - top)
    total = mine.sum(-1, keepdim=True) + theirs.sum(-1, keepdim=True)
    o = torch.matmul(mine.view(B, Sq * H, -1), rows[:, 0, :, :DC]) + torch.matmul(theirs.view(B, Sq * H, -1), before[..., :DC])
    return {"O": (o.view(B, Sq, H, DC) / total).to(torch.bfloat16), "lse": (top + total.log()).squeeze(-1)}


def mass_plain(q, cache, fmt, table, lens, lse, scale, idx, prev, decay, n):
    B = len(lens)
    logits, _, at = logits_plain(q, cache, fmt, table, lens, scale, idx, n)
    w = torch.exp(logits - lse[..., None]).sum(2)                            # [B, Sq, keys]
    base = torch.zeros(B, n, device=q.device)
    if prev is not None:
        base += decay * prev * (torch.arange(n, device=q.device) < lens[:, None])
    return base + w.sum(1) if idx is None else base.scatter_add(1, at.reshape(B, -1), w.view(B, -1))


def keep_plain(mass, lens, budget, sink, recent):
    B, n = mass.shape
    at = torch.arange(n, device=mass.device)[None].expand(B, -1)
    end = lens.long()[:, None]
    whole = end <= budget
    free = (at >= sink) & (at < end - recent)                                # these go by their weight
    order = torch.where(free, mass, -math.inf).sort(dim=-1, descending=True, stable=True).indices
    place = torch.empty_like(order).scatter_(1, order, at)                   # 0: the heaviest
    kept = (at < end) & (whole | ~free | (place < budget - sink - recent))
    where = torch.where(kept, at, n).sort(-1).values[:, :budget]
    keep = torch.full((B, budget), -1, dtype=torch.int32, device=mass.device)
    keep[:, :where.shape[1]] = torch.where(where < n, where, -1).to(torch.int32)
    return {"keep": keep, "count": kept.sum(-1, dtype=torch.int32)}


def compact_plain(cache, table, keep, new_table, mass):
    pages, page, _ = cache.shape
    flat = cache.view(pages * page, -1)
    held = keep >= 0
    j = torch.arange(keep.shape[1], device=keep.device).expand_as(keep)
    src, dst = slots(table, page, keep.long().clamp(min=0)), slots(new_table, page, j)
    flat[dst[held]] = flat[src[held]]
    return mass.gather(1, keep.long().clamp(min=0)) * held


def run(s):
    c, n = s["case"], int(s["case"]["len"])
    if own:
        import sparse_attention_index_gb300 as dsa
    if c["op"] == "shared":
        if own:
            O, lse = dsa.dsa_latent_attn_shared(s["q"], s["cache"], s["prefix_table"], s["prefix_lens"], s["starts"],
                                                s["table"], s["lens"], s["scale"], fmt=c["fmt"])
            return {"O": O, "lse": lse}
        return shared_plain(s["q"], s["cache"], c["fmt"], s["prefix_table"], s["prefix_lens"], s["starts"], s["table"],
                            s["lens"], s["scale"], max(1, c["prefix"]), n)
    if c["op"] == "mass":
        if own:
            return dsa.dsa_cache_mass(s["q"], s["cache"], s["table"], s["lens"], s["lse"], s["scale"], n, fmt=c["fmt"],
                                      idx=s["idx"], prev=s["prev"], decay=0.875)
        return mass_plain(s["q"], s["cache"], c["fmt"], s["table"], s["lens"], s["lse"], s["scale"], s["idx"], s["prev"],
                          0.875, n)
    if c["op"] == "keep":
        if own:
            keep, count = dsa.dsa_cache_keep(s["mass"], s["lens"], c["budget"], sink=c["sink"], recent=c["recent"])
            return {"keep": keep, "count": count}
        return keep_plain(s["mass"], s["lens"], c["budget"], c["sink"], c["recent"])
    if own:
        mass = dsa.dsa_cache_compact(s["cache"], s["table"], s["lens"], s["keep"], s["new_table"], DC, DR, fmt=c["fmt"],
                                     mass=s["mass"])
    else:
        mass = compact_plain(s["cache"], s["table"], s["keep"], s["new_table"], s["mass"])
    return {"mass": mass, **parts(s["cache"].view(-1, row_bytes(c["fmt"])), c["fmt"])}


# ---------------------------------------------------------------------- the definitions in 64 bits


def e4m3_table():
    """The value of each e4m3 byte: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    b = torch.arange(256, device=DEV)
    sign = 1.0 - 2.0 * (b >> 7).double()
    e, m = (b >> 3) & 15, (b & 7).double()
    return sign * torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.pow(2.0, e.double() - 7))


def bf16_bits(b):
    """bf16 values of little-endian byte pairs [..., 2n], in 64 bits."""
    h = b[..., 0::2].int() | (b[..., 1::2].int() << 8)
    return (h << 16).view(torch.float32).double()


def held(rows, fmt):
    """What the bytes of cache rows [n, row] hold, in 64 bits, part by part."""
    if fmt == "bf16":
        return {"row": bf16_bits(rows)}
    sc = rows[:, DC:DC + 16].reshape(-1, 4, 4).int()
    sc = (sc[..., 0] | sc[..., 1] << 8 | sc[..., 2] << 16 | sc[..., 3] << 24).view(torch.float32).double()
    return {"codes": e4m3_table()[rows[:, :DC].long()], "scales": sc, "rest": bf16_bits(rows[:, DC + 16:])}


def rows_of(cache, fmt, pages, n):
    """The first n rows of a list of pages, in 64 bits."""
    p = held(torch.cat([cache[i] for i in pages.tolist()])[:n], fmt)
    return p["row"] if fmt == "bf16" else torch.cat([p["codes"] * p["scales"].repeat_interleave(GROUP, 1), p["rest"]], 1)


def exact(c, seed):
    s = prepare(c, seed)
    lens, page = lens_of(c), c.get("page", 1)
    if c["op"] == "keep":
        return None                                       # whole numbers only
    if c["op"] == "compact":
        flat = s["cache"].view(-1, row_bytes(c["fmt"]))
        mass = torch.zeros(c["B"], c["budget"], dtype=torch.float64, device=DEV)
        new = flat.clone()
        for b in range(c["B"]):
            kept = s["keep"][b][s["keep"][b] >= 0].long()
            mass[b, :len(kept)] = s["mass"][b, kept].double()
            old = torch.cat([s["cache"][i] for i in s["table"][b].tolist()])[kept]
            for j in range(0, len(kept), page):
                at = int(s["new_table"][b, j // page]) * page
                new[at:at + min(page, len(kept) - j)] = old[j:j + page]
        return {"mass": mass, **held(new, c["fmt"])}
    B, Sq, H, _ = s["q"].shape
    q = s["q"].double() * s["scale"]
    own_rows = lambda b: rows_of(s["cache"], c["fmt"], s["table"][b, :-(-lens[b] // page)], lens[b])  # noqa: E731
    if c["op"] == "shared":
        starts, prefixes = groups_of(c)
        O = torch.zeros(B, Sq, H, DC, dtype=torch.float64, device=DEV)
        lse = torch.zeros(B, Sq, H, dtype=torch.float64, device=DEV)
        before = [rows_of(s["cache"], c["fmt"], s["prefix_table"][g, :-(-p // page)], p) for g, p in enumerate(prefixes)]
        for b in range(B):
            g = [i for i in range(c["G"]) if starts[i] <= b < starts[i + 1]]
            kv = torch.cat([before[g[0]], own_rows(b)]) if g else own_rows(b)
            for i in range(Sq):
                kv_i = kv[:len(kv) - Sq + i + 1]
                w = q[b, i] @ kv_i.T
                lse[b, i] = torch.logsumexp(w, -1)
                O[b, i] = torch.exp(w - lse[b, i][:, None]) @ kv_i[:, :DC]
        return {"O": O, "lse": lse}
    mass = torch.zeros(B, max(lens), dtype=torch.float64, device=DEV)
    for b in range(B):
        kv = own_rows(b)
        if c["prev"]:
            mass[b, :lens[b]] = 0.875 * s["prev"][b, :lens[b]].double()
        for i in range(Sq):
            t = torch.arange(lens[b] - Sq + i + 1, device=DEV)
            if c["k"]:
                t = s["idx"][b, i].long()
                t = t[t >= 0]
            w = torch.exp(q[b, i] @ kv[t].T - s["lse"][b, i].double()[:, None]).sum(0)
            mass[b].index_add_(0, t, w)
    return mass
