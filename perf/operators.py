"""Measured cases of the serving operators: rotary positions, the paged latent cache and the attention
that reads it.

Four operators, each with its plain form in elementary torch operations and the call that a user makes:

* ``rope``   - rotary positions on part of each head, interleaved or half layout, forward and inverse;
* ``write``  - latent rows into the slots of a paged cache, kept as bf16 or quantised to e4m3;
* ``read``   - rows of the cache back as bf16;
* ``attn``   - attention of the newest tokens of each sequence over its cached rows (keys: the whole
  row, values: its latent part), over every cached key or over a selected list.

A cache row holds Dc latent dims and Dr positional dims. "bf16": all of them in bf16. "e4m3": the Dc
dims in e4m3, one fp32 power-of-two scale per 128 of them (padded to 16 bytes), then the Dr dims in
bf16.
"""
import math

import torch

own = False

DEV = "cuda"
DC, DR, GROUP = 512, 64, 128


# ------------------------------------------------------------------------------------------ cases


def listed():
    return [
        # the rotary part of the queries of a decode batch of 8 tokens: latency
        dict(name="rope_decode_q", op="rope", T=8, H=128, D=192, off=128, rot=64, layout="interleaved", dtype="bf16", inverse=False, far=131072),
        # the queries of a long prompt
        dict(name="rope_prefill_q", op="rope", T=16384, H=128, D=192, off=128, rot=64, layout="interleaved", dtype="bf16", inverse=False, far=16384),
        # training: fp32 gradient of the indexer queries back through their rotation
        dict(name="rope_indexer_grad", op="rope", T=4097, H=64, D=128, off=0, rot=64, layout="half", dtype="f32", inverse=True, far=131072),
        # a decode batch of 128 tokens written to the cache
        dict(name="write_decode_e4m3", op="write", T=128, slots=8192, dc=DC, dr=DR, fmt="e4m3"),
        # a prompt written to the cache
        dict(name="write_prefill_e4m3", op="write", T=16385, slots=32768, dc=DC, dr=DR, fmt="e4m3"),
        # a short prefix fetched for a prompt that continues it, kept as bf16
        dict(name="read_prefix_bf16", op="read", N=489, slots=4096, dc=DC, dr=DR, fmt="bf16"),
        # a long cached prompt dequantised
        dict(name="read_long_e4m3", op="read", N=131072, slots=140000, dc=DC, dr=DR, fmt="e4m3"),
        # one short sequence on a rank with 16 of the heads: latency
        dict(name="attn_one_short", op="attn", B=1, Sq=1, H=16, len=489, ragged=False, page=64, fmt="bf16", k=0),
        # a ragged decode batch, every cached key
        dict(name="attn_batch_bf16", op="attn", B=32, Sq=1, H=128, len=8192, ragged=True, page=64, fmt="bf16", k=0),
        # four new tokens a sequence (drafted tokens verified together), 16 heads
        dict(name="attn_draft_bf16", op="attn", B=16, Sq=4, H=16, len=16000, ragged=True, page=16, fmt="bf16", k=0),
        # the selected 2048 keys of each token, quantised cache
        dict(name="attn_selected_e4m3", op="attn", B=128, Sq=1, H=128, len=4096, ragged=False, page=64, fmt="e4m3", k=2048),
        # few long contexts, quantised cache
        dict(name="attn_long_e4m3", op="attn", B=4, Sq=1, H=128, len=131072, ragged=False, page=64, fmt="e4m3", k=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn"])
    if op == "rope":
        H = rng.choice([1, 2, 8, 16, 64, 128])
        D, off, rot = rng.choice([(192, 128, 64), (128, 0, 64), (128, 0, 128), (576, 512, 64), (64, 0, 32)])
        T = _log(rng, 1, max(1, min(65536, 200_000_000 // (H * D))))
        return dict(op=op, T=T, H=H, D=D, off=off, rot=rot, layout=rng.choice(["interleaved", "half"]),
                    dtype=rng.choice(["bf16", "f32"]), inverse=rng.random() < 0.5, far=rng.choice([4096, 131072, 1 << 20]))
    dc, dr = rng.choice([(512, 64), (512, 64), (128, 64), (128, 0)])
    fmt = rng.choice(["bf16", "e4m3"])
    if op == "write":
        T = _log(rng, 1, 65536)
        return dict(op=op, T=T, slots=T + rng.randrange(1, 9000), dc=dc, dr=dr, fmt=fmt)
    if op == "read":
        N = _log(rng, 1, 131072)
        return dict(op=op, N=N, slots=rng.randrange(1, 100000), dc=dc, dr=dr, fmt=fmt)
    H = rng.choice([8, 16, 20, 32, 64, 128])
    Sq = rng.choice([1, 1, 1, 2, 4, 7])
    k = rng.choice([0, 0, 0, 64, 500, 2048])
    B = _log(rng, 1, 128)
    n = _log(rng, Sq, max(Sq + 1, min(131072, 400000 // (B * Sq))))
    return dict(op=op, B=B, Sq=Sq, H=H, len=n, ragged=rng.random() < 0.7, page=rng.choice([16, 32, 64, 100]), fmt=fmt, k=k)


def row_bytes(fmt, dc, dr):
    if fmt == "bf16":
        return 2 * (dc + dr)
    return dc + (4 * (dc // GROUP) + 15) // 16 * 16 + 2 * dr


def lens_of(c):
    """Cached tokens of each sequence, its new ones among them: a ramp where ragged."""
    if not c["ragged"]:
        return [c["len"]] * c["B"]
    return [max(c["Sq"], c["len"] * (b + 1) // c["B"]) for b in range(c["B"])]


def work(c):
    if c["op"] == "rope":
        size = 2 if c["dtype"] == "bf16" else 4
        n = c["T"] * c["H"]
        return {"bytes": 2 * n * c["D"] * size + 4 * c["T"] + 2 * c["rot"], "flops": 3 * n * c["rot"]}
    if c["op"] in ("write", "read"):
        n = c["T"] if c["op"] == "write" else c["N"]
        d = c["dc"] + c["dr"]
        return {"bytes": n * (2 * d + row_bytes(c["fmt"], c["dc"], c["dr"]) + 4), "flops": 2 * n * d}
    rows = pairs = 0
    for n in lens_of(c):
        seen = [n - c["Sq"] + i + 1 for i in range(c["Sq"])]
        if c["k"]:
            seen = [min(c["k"], s) for s in seen]
        pairs += sum(seen)
        rows += min(n, sum(seen)) if c["k"] else n
    tokens = c["B"] * c["Sq"]
    return {"bytes": rows * row_bytes(c["fmt"], DC, DR) + tokens * c["H"] * (2 * (DC + DR) + 2 * DC + 4)
            + 4 * c["B"] + 4 * tokens * c["k"] + 4 * sum(-(-n // c["page"]) for n in lens_of(c)),
            "flops": 2 * pairs * c["H"] * (2 * DC + DR)}


# ----------------------------------------------------------------------------------------- inputs


def quantised(x, dc, dr):
    """fp32 [n, dc + dr] -> (codes float8 [n, dc], scales fp32 [n, dc / 128], rest bf16 [n, dr])."""
    g = x[:, :dc].reshape(-1, dc // GROUP, GROUP)
    mant, expo = torch.frexp(g.abs().amax(-1))           # amax = mant * 2^expo, mant in [1/2, 1)
    # the smallest power of two that brings amax to at most 448 = 0.875 * 2^9; 1 where all is zero
    k = torch.where(mant > 0.875, expo - 8, expo - 9)
    k = torch.where(mant == 0, torch.zeros_like(k), k).clamp(min=-120)
    scales = torch.ldexp(torch.ones_like(mant), k)
    codes = (g / scales[..., None]).to(torch.float8_e4m3fn)
    return codes.reshape(-1, dc), scales, x[:, dc:].to(torch.bfloat16)


def parts(cache, fmt, dc, dr):
    """The cache's rows [n, row] bytes as the values it holds: views, no copies."""
    if fmt == "bf16":
        return {"row": cache.view(torch.bfloat16)}
    pad = (4 * (dc // GROUP) + 15) // 16 * 16
    got = {"codes": cache[:, :dc].view(torch.float8_e4m3fn),
           "scales": cache[:, dc:dc + 4 * (dc // GROUP)].view(torch.float32)}
    if dr:
        got["rest"] = cache[:, dc + pad:].view(torch.bfloat16)
    return got


def fill(cache, fmt, dc, dr, at, x):
    """Writes rows x (fp32) at the slots `at`, in the plain form."""
    p = parts(cache, fmt, dc, dr)
    if fmt == "bf16":
        p["row"][at] = x.to(torch.bfloat16)
        return
    codes, scales, rest = quantised(x, dc, dr)
    p["codes"].view(torch.uint8)[at] = codes.view(torch.uint8)
    p["scales"][at] = scales
    if dr:
        p["rest"][at] = rest


def values(cache, fmt, dc, dr, at):
    """fp32 values of the rows at the slots `at` (any shape)."""
    p = parts(cache[at.reshape(-1)], fmt, dc, dr)
    if fmt == "bf16":
        v = p["row"].float()
    else:
        v = p["codes"].float().view(-1, dc // GROUP, GROUP) * p["scales"][..., None]
        v = v.reshape(-1, dc)
        if dr:
            v = torch.cat([v, p["rest"].float()], -1)
    return v.view(*at.shape, dc + dr)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    s = {"case": c}
    if c["op"] == "rope":
        x = normal(c["T"], c["H"], c["D"])
        s["x"] = x.to(torch.bfloat16) if c["dtype"] == "bf16" else x
        # tokens of packed sequences anywhere in a long context
        s["pos"] = torch.randint(0, c["far"], (c["T"],), generator=g, device=DEV, dtype=torch.int32)
        i = torch.arange(c["rot"] // 2, dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-2.0 * i / c["rot"])).float().to(DEV)
        s["mscale"] = 1.0
        return s
    fmt = c["fmt"]
    if c["op"] == "attn":
        lens = lens_of(c)
        page, B, Sq = c["page"], c["B"], c["Sq"]
        need = [-(-n // page) for n in lens]
        total = sum(need) + 3
        order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros(B, max(need), dtype=torch.int32, device=DEV)
        first = 0
        for b, n in enumerate(need):
            table[b, :n] = order[first:first + n]
            first += n
        cache = torch.zeros(total * page, row_bytes(fmt, DC, DR), dtype=torch.uint8, device=DEV)
        for a in range(0, total * page, 131072):
            e = min(total * page, a + 131072)
            fill(cache, fmt, DC, DR, torch.arange(a, e, device=DEV), normal(e - a, DC + DR))
        s.update(cache=cache.view(total, page, -1), table=table, scale=192 ** -0.5,
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 q=normal(B, Sq, c["H"], DC + DR).to(torch.bfloat16), idx=None)
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
        return s
    d = c["dc"] + c["dr"]
    s["cache"] = torch.zeros(c["slots"], row_bytes(fmt, c["dc"], c["dr"]), dtype=torch.uint8, device=DEV)
    if c["op"] == "write":
        s["kv"] = normal(c["T"], d).to(torch.bfloat16)
        s["slots"] = torch.randperm(c["slots"], generator=g, device=DEV)[:c["T"]].to(torch.int32)
    else:
        fill(s["cache"], fmt, c["dc"], c["dr"], torch.arange(c["slots"], device=DEV), normal(c["slots"], d))
        s["slots"] = torch.randint(0, c["slots"], (c["N"],), generator=g, device=DEV, dtype=torch.int32)
    return s


# ------------------------------------------------------------------------------------ plain forms


def rope_plain(x, pos, inv_freq, off, rot, layout, mscale, inverse):
    ang = pos.double()[:, None] * inv_freq.double()      # far positions: 32 bits would lose the angle
    cos, sin = (mscale * ang.cos()).float()[:, None], (mscale * ang.sin()).float()[:, None]
    if inverse:
        sin = -sin
    v = x.float()
    r = v[..., off:off + rot]
    if layout == "interleaved":
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([v[..., :off], turned, v[..., off + rot:]], -1).to(x.dtype)


def attn_plain(q, cache, fmt, table, lens, scale, idx):
    B, Sq, H, _ = q.shape
    pages, page, _ = cache.shape
    limit = lens[:, None] - Sq + 1 + torch.arange(Sq, device=q.device)      # keys each token sees
    if idx is None:
        at = torch.arange(table.shape[1] * page, device=q.device)[None, None]
        seen = at < limit[..., None]                                         # [B, Sq, L]
    else:
        at = idx.long()
        seen = (at >= 0) & (at < limit[..., None])
        at = at.clamp(min=0)
    at = at.expand(B, -1, -1)                                                # [B, 1 or Sq, keys]
    slot = table.long().gather(1, (at // page).reshape(B, -1)).view_as(at) * page + at % page
    rows = values(cache.view(pages * page, -1), fmt, DC, DR, slot)           # [B, 1 or Sq, keys, DC + DR]
    if idx is None:
        logits = torch.matmul(q.float().view(B, 1, Sq * H, -1), rows.transpose(-1, -2)).view(B, Sq, H, -1)
    else:
        logits = torch.matmul(q.float(), rows.transpose(-1, -2))
    logits = (logits * scale).masked_fill_(~seen[:, :, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - top.masked_fill(top == -math.inf, 0.0))           # a row without keys: zeros
    total = p.sum(-1, keepdim=True)
    v = rows[..., :DC]
    o = torch.matmul(p.view(B, 1, Sq * H, -1), v).view(B, Sq, H, DC) if idx is None else torch.matmul(p, v)
    o = o / total.masked_fill(total == 0, 1.0)
    return {"O": o.to(torch.bfloat16), "lse": (top + total.log()).squeeze(-1)}


def run(s):
    c = s["case"]
    if own:
        import sparse_attention_index_gb300 as dsa
    if c["op"] == "rope":
        if own:
            return dsa.dsa_rope(s["x"], s["pos"], s["inv_freq"], off=c["off"], layout=c["layout"],
                                mscale=s["mscale"], inverse=c["inverse"])
        return rope_plain(s["x"], s["pos"], s["inv_freq"], c["off"], c["rot"], c["layout"], s["mscale"], c["inverse"])
    if c["op"] == "write":
        if own:
            dsa.dsa_cache_write(s["kv"], s["slots"], s["cache"], c["dc"], fmt=c["fmt"])
        else:
            fill(s["cache"], c["fmt"], c["dc"], c["dr"], s["slots"].long(), s["kv"].float())
        return parts(s["cache"], c["fmt"], c["dc"], c["dr"])
    if c["op"] == "read":
        if own:
            return dsa.dsa_cache_read(s["cache"], s["slots"], c["dc"], c["dr"], fmt=c["fmt"])
        return values(s["cache"], c["fmt"], c["dc"], c["dr"], s["slots"].long()).to(torch.bfloat16)
    if own:
        O, lse = dsa.dsa_latent_attn(s["q"], s["cache"], s["table"], s["lens"], s["scale"], fmt=c["fmt"], idx=s["idx"])
        return {"O": O, "lse": lse}
    return attn_plain(s["q"], s["cache"], c["fmt"], s["table"], s["lens"], s["scale"], s["idx"])


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


def stored(rows, fmt, dc):
    """What the bytes of cache rows [n, row] stand for, in 64 bits."""
    if fmt == "bf16":
        return bf16_bits(rows)
    n = dc // GROUP
    sc = rows[:, dc:dc + 4 * n].reshape(-1, n, 4).int()
    sc = (sc[..., 0] | sc[..., 1] << 8 | sc[..., 2] << 16 | sc[..., 3] << 24).view(torch.float32).double()
    v = e4m3_table()[rows[:, :dc].long()] * sc.repeat_interleave(GROUP, 1)
    return torch.cat([v, bf16_bits(rows[:, dc + (4 * n + 15) // 16 * 16:])], 1)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        # each pair (x_a, x_b) as a complex number, turned by e^(+-i pos f)
        x, o, r = s["x"].double(), c["off"], c["rot"]
        i = torch.arange(r // 2, device=DEV)
        a, b = (o + 2 * i, o + 2 * i + 1) if c["layout"] == "interleaved" else (o + i, o + r // 2 + i)
        angle = torch.outer(s["pos"].double(), s["inv_freq"].double()) * (-1.0 if c["inverse"] else 1.0)
        z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.full_like(angle, s["mscale"]), angle)[:, None]
        x[..., a], x[..., b] = z.real, z.imag
        return x
    if c["op"] == "write":
        at, x, dc = s["slots"].long(), s["kv"].double(), c["dc"]
        if c["fmt"] == "bf16":
            full = torch.zeros(c["slots"], dc + c["dr"], dtype=torch.float64, device=DEV)
            full[at] = x
            return {"row": full}
        g = x[:, :dc].view(len(x), -1, GROUP)
        scale = torch.pow(2.0, torch.ceil(torch.log2(g.abs().amax(-1) / 448.0)))
        got = {"codes": (g / scale[..., None]).reshape(len(x), dc), "scales": scale}
        if c["dr"]:
            got["rest"] = x[:, dc:]
        full = {k: torch.zeros(c["slots"], v.shape[1], dtype=torch.float64, device=DEV) for k, v in got.items()}
        for k, v in got.items():
            full[k][at] = v
        return full
    if c["op"] == "read":
        return stored(s["cache"][s["slots"].long()], c["fmt"], c["dc"])
    pages, page, _ = s["cache"].shape
    B, Sq, H, D = s["q"].shape
    O = torch.zeros(B, Sq, H, DC, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Sq, H), -math.inf, dtype=torch.float64, device=DEV)
    flat, q = s["cache"].view(pages * page, -1), s["q"].double()
    for b, n in enumerate(lens_of(c)):
        p = torch.arange(n, device=DEV)
        kv = stored(flat[s["table"][b].long()[p // page] * page + p % page], c["fmt"], DC)   # [n, D]
        for i in range(Sq):
            keys = n - Sq + i + 1
            if keys < 1:
                continue
            rows = kv[:keys]
            if c["k"]:
                t = s["idx"][b, i].long()
                rows = kv[t[(t >= 0) & (t < keys)]]
            w = (q[b, i] @ rows.T) * s["scale"]
            lse[b, i] = torch.logsumexp(w, -1)
            O[b, i] = torch.exp(w - lse[b, i][:, None]) @ rows[:, :DC]
    return {"O": O, "lse": lse}
