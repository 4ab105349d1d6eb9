"""Cases of the serving-cache operators: rotary positions, the append into a cache held in 8 bits, the attention
over that cache, and the eviction of its least attended tokens.

The cache is paged, [num_pages, Hkv, page, d] e4m3 bytes for K and for V, with one fp32 scale for each block of
`sb` consecutive tokens of a page and kv head.  ``run`` computes each operator in its plain form (elementary torch
operations in 32 bits; angles of positions in 64) or, with ``own`` set, by the framework's calls.  e4m3 bytes are
returned as float8_e4m3fn tensors beside their scales.
"""
import math
import random

import torch

own = False
DEV = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one serving step's queries, at far positions of a context stretched eightfold
        dict(name="rope_step_B32", op="rope", B=32, H=32, N=1, d=128, rot=128, inter=False, layout="bhnd",
             stretch="yarn", far=131072, grad=False),
        # a prompt's queries as the projection leaves them (token-major), into the attention's head-major layout
        dict(name="rope_prompt_8k", op="rope", B=1, H=32, N=8192, d=128, rot=128, inter=False, layout="bnhd",
             stretch="none", far=0, grad=False),
        # the gradient of interleaved rotation of half of a 64-wide head, odd length, out of a training batch
        dict(name="rope_grad_part", op="rope", B=2, H=32, N=4093, d=64, rot=32, inter=True, layout="bhnd",
             stretch="linear", far=0, grad=True),
        # one token of each of 32 sequences, rotated and written
        dict(name="append_step_B32", op="append", B=32, Hkv=8, N=1, d=128, page=16, sb=16, have=4096, rot=128,
             inter=False, layout="bhnd"),
        # ragged prompts, packed beside the queries as one projection leaves them
        dict(name="append_prompt_2k", op="append", B=8, Hkv=8, N=2048, d=128, page=64, sb=32, have=100, rot=128,
             inter=False, layout="packed"),
        # one short sequence: the latency of a step
        dict(name="decode_one_777", op="decode", B=1, Hkv=8, group=4, Nq=1, N=777, d=128, page=16, sb=16,
             ragged=False, weights=False),
        # the ordinary batch of a server
        dict(name="decode_B32_4k", op="decode", B=32, Hkv=8, group=4, Nq=1, N=4096, d=128, page=64, sb=64,
             ragged=True, weights=False),
        # one very long context
        dict(name="decode_long_128k", op="decode", B=1, Hkv=8, group=4, Nq=1, N=131072, d=128, page=128, sb=64,
             ragged=False, weights=False),
        # 64-wide heads without sharing, accumulating the weights that eviction reads
        dict(name="decode_d64_weights", op="decode", B=16, Hkv=16, group=1, Nq=1, N=3001, d=64, page=48, sb=24,
             ragged=True, weights=True),
        # four drafted tokens checked at once, groups of eight heads, weights accumulated
        dict(name="decode_draft_weights", op="decode", B=8, Hkv=4, group=8, Nq=4, N=8000, d=128, page=32, sb=32,
             ragged=True, weights=True),
        # a batch whose contexts reached their budget
        dict(name="evict_B32_4k", op="evict", B=32, Hkv=8, N=4096, d=128, page=64, sb=64, keep=1024, recent=128),
        # one long context cut to an eighth
        dict(name="evict_long_64k", op="evict", B=1, Hkv=8, N=65521, d=128, page=128, sb=32, keep=8192, recent=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _page(rng):
    page = rng.choice([8, 16, 20, 32, 48, 64, 128, 256])
    return page, rng.choice([s for s in (4, 8, 16, 20, 24, 32, 64, 128) if page % s == 0])


def draw(rng):
    op = rng.choice(["rope", "append", "append", "decode", "decode", "decode", "evict"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    if op == "rope":
        H = rng.choice([1, 2, 8, 12, 32, 40])
        N = _log(rng, 1, 16384)
        B = _log(rng, 1, max(1, min(64, 32 * 8192 // (H * N))))
        return dict(op=op, B=B, H=H, N=N, d=d, rot=rng.choice([16, 32, 48, d // 2, d, d]), inter=rng.random() < 0.5,
                    layout=rng.choice(["bhnd", "bnhd", "packed"]), stretch=rng.choice(["none", "linear", "ntk", "yarn"]),
                    far=rng.choice([0, 5000, 131072, 1000000]), grad=rng.random() < 0.5)
    page, sb = _page(rng)
    if op == "append":
        N = 1 if rng.random() < 0.4 else _log(rng, 2, 8192)
        B = _log(rng, 1, max(1, min(64, 8 * 8 * 2048 // (Hkv * N))))
        return dict(op=op, B=B, Hkv=Hkv, N=N, d=d, page=page, sb=sb, have=rng.choice([0, 1, 100, 1000]),
                    rot=rng.choice([0, 32, d, d]), inter=rng.random() < 0.5,
                    layout=rng.choice(["bhnd", "bnhd", "packed"]))
    if op == "decode":
        N = _log(rng, 1, 131072)
        B = _log(rng, 1, max(1, min(64, 32 * 8 * 4096 // (Hkv * N))))
        return dict(op=op, B=B, Hkv=Hkv, group=rng.choice([1, 2, 3, 4, 5, 8, 16]), Nq=rng.choice([1, 1, 1, 2, 5]), N=N, d=d,
                    page=page, sb=sb, ragged=rng.random() < 0.7, weights=rng.random() < 0.4)
    N = _log(rng, 64, 65521)
    B = _log(rng, 1, max(1, min(32, 32 * 8 * 4096 // (Hkv * N))))
    keep = max(1, min(int(N * rng.uniform(0.1, 0.9)), 32 * 8 * 1024 // (B * Hkv)))
    return dict(op=op, B=B, Hkv=Hkv, N=N, d=d, page=page, sb=sb, keep=keep, recent=int(keep * rng.uniform(0, 1)))


def _lengths(case, most):
    """Tokens of each sequence: all `most`, or spread from empty or half full up to it.  A function of the case alone."""
    B = case["B"]
    if not case.get("ragged", True) or B == 1:
        return [most] * B
    r = random.Random(B * 1000003 + most)
    lens = [r.randint(most // 2, most) for _ in range(B)]
    lens[0] = most
    if B > 3 and case["op"] == "decode":
        lens[B // 2] = 0  # a slot of the batch without a sequence
    return lens


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(DEV).manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _frequencies(rot, stretch):
    """Angle per position of each pair, float64 [rot/2], and the factor on cos and sin: plain rotary frequencies, or
    stretched for a context eight times as long by interpolation, by a larger base, or by parts (long waves
    interpolated, short ones kept, with the factor 0.1 ln 8 + 1)."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if stretch == "ntk" and rot > 2:
        return (10000.0 * 8.0 ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    f = 10000.0 ** (-2.0 * i / rot)
    if stretch == "linear":
        return f / 8.0, 1.0
    if stretch == "yarn":
        turns = 4096.0 * f / (2 * math.pi)  # turns within the original context
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f * keep + f / 8.0 * (1.0 - keep), 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def _turns(freq):
    """Turns per position as 64-bit fixed-point fractions (the table the framework's rotation takes)."""
    t = [int(round(f / (2 * math.pi) * 2.0 ** 64)) % (1 << 64) for f in freq.tolist()]
    return torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in t], dtype=torch.int64, device=DEV)


def _rotary(s, rot, stretch):
    f, s["mag"] = _frequencies(rot, stretch)
    s["freq"], s["turns"] = f.to(DEV), _turns(f)


def _activations(g, B, H, N, d, layout):
    """bf16 [B, H, N, d] as the program holds it: head-major, token-major, or inside a wider projection's output.
    Two columns of a head are far larger than the others, as in trained models."""
    x = _randn(g, B, N, H, d)
    x[..., 3] *= 9.0
    x[..., d // 2 + 5] *= 5.0
    x = x.to(torch.bfloat16)
    if layout == "bhnd":
        return x.transpose(1, 2).contiguous()
    if layout == "packed":
        wide = torch.empty((B, N, H + 4, d), dtype=torch.bfloat16, device=DEV)
        wide[:, :, 2:2 + H] = x
        return wide[:, :, 2:2 + H].transpose(1, 2)
    return x.transpose(1, 2)


def _pool(g, s, case, pages):
    """Page pools and power-of-two scales, full of tokens whose blocks differ in size."""
    shape = (pages, case["Hkv"], case["page"], case["d"])
    nb = case["page"] // case["sb"]
    for n in ("k", "v"):
        x = _randn(g, *shape)
        x[..., 3] *= 6.0
        x = x.reshape(shape[0], shape[1], nb, case["sb"] * case["d"])
        amax = x.abs().amax(-1, keepdim=True).clamp_min(1e-20)
        s[n] = (x / amax * E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8).reshape(shape)
        up = torch.exp2(torch.randint(-2, 2, amax.shape, generator=g, device=DEV).float())
        if n == "k":
            up = up * 0.5
        s[n + "s"] = (torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX))) * up).squeeze(-1).contiguous()


def _table(g, B, maxp, first, pages):
    """int32 [B, maxp] of distinct pages in [first, pages), shuffled as a server's allocator leaves them."""
    p = torch.randperm(pages - first, generator=g, device=DEV)[:B * maxp] + first
    return p.reshape(B, maxp).to(torch.int32)


def prepare(case, seed):
    c, g, s = dict(case), _gen(seed), {}
    s["case"] = c
    B, d = c["B"], c["d"]
    if c["op"] == "rope":
        x = _activations(g, B, c["H"], c["N"], d, c["layout"])
        s["x"] = x
        start = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device=DEV)
        s["pos"] = (start + torch.arange(c["N"], device=DEV)).to(torch.int32).contiguous()
        _rotary(s, c["rot"], c["stretch"])
        return s
    if c["op"] == "append":
        have = _lengths(c, c["have"])
        new = _lengths(c, c["N"])
        new = [max(1, n) for n in new]
        maxp = -(-(max(have) + c["N"]) // c["page"])
        s["k_new"] = _activations(g, B, c["Hkv"], c["N"], d, c["layout"])
        s["v_new"] = _activations(g, B, c["Hkv"], c["N"], d, c["layout"])
        _pool(g, s, c, B * maxp + 3)
        s["table"], s["lens"], s["new"] = _table(g, B, maxp, 0, B * maxp + 3), _ints(have), _ints(new)
        s["pos"] = (s["lens"][:, None] + torch.arange(c["N"], device=DEV, dtype=torch.int32) + 11).contiguous()
        if c["rot"]:
            _rotary(s, c["rot"], "none")
        return s
    maxp = -(-c["N"] // c["page"])
    lens = _lengths(c, c["N"])
    s["lens"] = _ints(lens)
    if c["op"] == "decode":
        _pool(g, s, c, B * maxp + 3)
        s["table"] = _table(g, B, maxp, 0, B * maxp + 3)
        s["q"] = (_randn(g, B, c["Hkv"] * c["group"], c["Nq"], d)).to(torch.bfloat16)
        if c["weights"]:
            s["w"] = 0.01 * torch.rand((B, c["Hkv"], maxp * c["page"]), generator=g, device=DEV)
        return s
    newp = -(-c["keep"] // c["page"])
    _pool(g, s, c, B * (maxp + newp))
    both = _table(g, B, maxp + newp, 0, B * (maxp + newp))
    s["table"], s["new_table"] = both[:, :maxp].contiguous(), both[:, maxp:].contiguous()
    # accumulated weights: a few heavy tokens over a long light tail, as attention leaves them, coarse enough for ties
    w = torch.exp(3.0 * _randn(g, B, c["Hkv"], maxp * c["page"]))
    s["w"] = torch.round(w * 256) / 256
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, pos, s, inter, inverse):
    """fp32 rotation of x [B, H, N, d] (any strides) by pos [B, N]; angles in 64 bits."""
    half = s["freq"].numel()
    a = pos.double()[:, None, :, None] * s["freq"]
    cos, sin = (torch.cos(a) * s["mag"]).float(), (torch.sin(a) * s["mag"]).float()
    sin = -sin if inverse else sin
    x = x.float()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if inter:
        x1, x2 = r[..., 0::2], r[..., 1::2]
        return torch.cat([torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2), rest], -1)
    x1, x2 = r[..., :half], r[..., half:]
    return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin, rest], -1)


def _power_of_two_scale(amax):
    """Smallest power of two s >= 2^-126 with amax / s <= 448, exactly (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), torch.full_like(e, -126)).clamp_min(-126)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _value(b):
    return b.view(torch.float8_e4m3fn).float()


def _append(s, c, pages, scales, x):
    """Writes x [B, Hkv, N, d] (fp32) at positions lens.. of the paged cache, block by block."""
    P, S, B, N = c["page"], c["sb"], c["B"], c["N"]
    lens, new, table = s["lens"].long(), s["new"].long(), s["table"].long()
    blocks = (N + S - 2) // S + 1
    blk = (lens // S)[:, None] + torch.arange(blocks, device=DEV)
    pos = blk[..., None] * S + torch.arange(S, device=DEV)                       # [B, blocks, S]
    end = (lens + new)[:, None, None]
    here, old = pos < end, pos < lens[:, None, None]
    fresh = here & ~old
    b = torch.arange(B, device=DEV)[:, None, None]
    page = table[b, (pos // P).clamp_max(table.shape[1] - 1)]
    was = pages[page, :, pos % P]                                                # [B, blocks, S, Hkv, d]
    sc = scales[page[..., 0], :, (pos[..., 0] % P) // S]                         # [B, blocks, Hkv]
    val = x.transpose(1, 2)[b, (pos - lens[:, None, None]).clamp(0, N - 1)]      # [B, blocks, S, Hkv, d]
    size = torch.where(fresh[..., None, None] & val.isfinite(), val.abs(), torch.zeros_like(val)).amax((2, 4))
    need = _power_of_two_scale(size)
    to = torch.where((blk * S < lens[:, None])[..., None], torch.maximum(sc, need), need)
    by = to[:, :, None, :, None]
    got = torch.where(fresh[..., None, None], _e4m3(val / by), _e4m3(_value(was) * sc[:, :, None, :, None] / by))
    pages[page[here], :, (pos % P)[here]] = got[here]
    use = here[..., 0]
    scales[page[..., 0][use], :, ((pos[..., 0] % P) // S)[use]] = to[use]


def _gathered(pages, scales, table, P, S):
    """fp32 values [B, Hkv, tokens, d] of the pages that a table names."""
    t = table.long()
    x = _value(pages[t].view(torch.uint8)) * scales[t].repeat_interleave(S, -1)[..., None]
    B, mp, Hkv, _, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, mp * P, d)


def _decode(s, c):
    P, S, B, Hkv, G, Nq, d = c["page"], c["sb"], c["B"], c["Hkv"], c["group"], c["Nq"], c["d"]
    k = _gathered(s["k"], s["ks"], s["table"], P, S)
    v = _gathered(s["v"], s["vs"], s["table"], P, S)
    q = s["q"].float().reshape(B, Hkv, G * Nq, d)
    x = q @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    tok = torch.arange(Nq, device=DEV).repeat(G)
    last = s["lens"][:, None] - Nq + tok                                         # the last key that a row sees
    seen = torch.arange(x.shape[-1], device=DEV) <= last[:, None, :, None]
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, torch.ones_like(l))
    v = v.masked_fill((torch.arange(x.shape[-1], device=DEV) >= s["lens"][:, None])[:, None, :, None], 0.0)
    o = (p @ v).to(torch.bfloat16).reshape(B, Hkv * G, Nq, d)
    out = [o, (m + torch.log(l)).reshape(B, Hkv * G, Nq)]
    if c["weights"]:
        s["w"] += p.sum(2)
        out.append(s["w"])
    return out


def _evict(s, c):
    P, S, B, Hkv = c["page"], c["sb"], c["B"], c["Hkv"]
    T, C = s["table"].shape[1] * P, s["new_table"].shape[1] * P
    j = torch.arange(T, device=DEV)
    n = s["lens"].long()[:, None, None]
    rank = torch.where(j < n - c["recent"], s["w"], torch.full_like(s["w"], math.inf))
    rank = rank.masked_fill(j >= n, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :c["keep"]]
    order = torch.where(torch.arange(order.shape[-1], device=DEV) < n, order, torch.full_like(order, T))
    order = torch.nn.functional.pad(order.sort(-1).values, (0, C - order.shape[-1]), value=T)
    there = order < T
    src = order.clamp_max(T - 1)
    b, h = torch.arange(B, device=DEV)[:, None, None], torch.arange(Hkv, device=DEV)[None, :, None]
    page = s["table"].long()[b, src // P]
    to = torch.arange(C, device=DEV).expand(B, Hkv, C)
    to_page = s["new_table"].long()[b, to // P]
    hh = h.expand(B, Hkv, C)
    for pages, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        sc = scales[page, h, src % P // S]
        by = torch.where(there, sc, torch.zeros_like(sc)).reshape(B, Hkv, C // S, S).amax(-1).repeat_interleave(S, -1)
        got = _e4m3(_value(pages[page, h, src % P]) * sc[..., None] / by[..., None])
        pages[to_page[there], hh[there], (to % P)[there]] = got[there]
        scales[to_page[there], hh[there], (to % P // S)[there]] = by[there]
    w = torch.where(there, s["w"].gather(-1, src), torch.zeros_like(src, dtype=torch.float32))
    return torch.minimum(s["lens"], torch.full_like(s["lens"], c["keep"])), w, torch.where(there, order, -torch.ones_like(order)).int()


def _cache(s):
    return [s["k"].view(torch.float8_e4m3fn), s["ks"], s["v"].view(torch.float8_e4m3fn), s["vs"]]


def run(state):
    s, c = state, state["case"]
    if own:
        import exact_tiled_attention_21_gb300 as fa
        if c["op"] == "rope":
            return fa.rope(s["x"], s["turns"], s["pos"], interleaved=c["inter"], magnitude=s["mag"], inverse=c["grad"])
        if c["op"] == "append":
            fa.cache_append_fp8(s["k_new"], s["v_new"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"],
                                new_lens=s["new"], turns=s.get("turns"), positions=s["pos"], interleaved=c["inter"])
            return _cache(s)
        if c["op"] == "decode":
            o, lse = fa.decode_paged_fp8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"],
                                         weights=s.get("w"))
            return [o, lse, s["w"]] if c["weights"] else [o, lse]
        lens, w, kept = fa.cache_evict_fp8(s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"], s["w"],
                                           s["new_table"], keep=c["keep"], recent=c["recent"])
        return _cache(s) + [lens, w, kept]
    if c["op"] == "rope":
        return _rotate(s["x"], s["pos"], s, c["inter"], c["grad"]).to(torch.bfloat16)
    if c["op"] == "append":
        k = s["k_new"]
        k = _rotate(k, s["pos"], s, c["inter"], False).to(torch.bfloat16) if c["rot"] else k
        _append(s, c, s["k"], s["ks"], k.float())
        _append(s, c, s["v"], s["vs"], s["v_new"].float())
        return _cache(s)
    if c["op"] == "decode":
        return _decode(s, c)
    return _cache(s) + list(_evict(s, c))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "rope":
        n = c["B"] * c["H"] * c["N"] * c["d"]
        return {"bytes": 4.0 * n + 4.0 * c["B"] * c["N"] + 4.0 * c["rot"], "flops": 3.0 * n * c["rot"] / c["d"]}
    d, Hkv = c["d"], c["Hkv"]
    if c["op"] == "append":
        t = sum(max(1, n) for n in _lengths(c, c["N"])) * Hkv
        return {"bytes": t * (4.0 * d + 2.0 * d + 8.0 / c["sb"]), "flops": t * 6.0 * d}
    lens = _lengths(c, c["N"])
    if c["op"] == "decode":
        rows = c["group"] * c["Nq"]
        t = sum(lens) * Hkv
        io = c["B"] * Hkv * rows * (4.0 * d + 4.0)
        return {"bytes": t * (2.0 * d + 8.0 / c["sb"] + (8.0 if c["weights"] else 0.0)) + io, "flops": 4.0 * t * rows * d}
    t = sum(lens) * Hkv
    kept = sum(min(n, c["keep"]) for n in lens) * Hkv
    return {"bytes": 4.0 * t + kept * (4.0 * d + 16.0 / c["sb"] + 8.0), "flops": 4.0 * kept * d}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_turned(x, pos, freq, mag, inter, sign):
    x = x.double().clone()
    y = x.clone()
    half = len(freq)
    for i in range(half):
        ang = pos.double() * float(freq[i])
        c, sn = torch.cos(ang)[:, None] * mag, torch.sin(ang)[:, None] * (mag * sign)
        p, q = (2 * i, 2 * i + 1) if inter else (i, i + half)
        y[..., p] = c * x[..., p] - sn * x[..., q]
        y[..., q] = sn * x[..., p] + c * x[..., q]
    return y


def _exact_scale(big):
    if big <= 0:
        return 2.0 ** -126
    e = math.ceil(math.log2(big / 448.0))
    while 448.0 * 2.0 ** (e - 1) >= big:
        e -= 1
    while 448.0 * 2.0 ** e < big:
        e += 1
    return 2.0 ** max(e, -126)


def _exact_round(x):
    """Nearest e4m3 value (ties to even), saturated; float64 in and out."""
    a = x.abs().clamp_max(448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3.0)
    return torch.copysign((torch.round(a / step) * step).clamp_max(448.0), x)


def _exact_append(s, c, vals, scales, x):
    lens, new, table = s["lens"].tolist(), s["new"].tolist(), s["table"].tolist()
    P, S = c["page"], c["sb"]
    for b in range(c["B"]):
        t = lens[b]
        while t < lens[b] + new[b]:
            first = t // S * S
            stop = min(first + S, lens[b] + new[b])
            page, at = table[b][t // P], t % P
            rows = x[b, :, t - lens[b]:stop - lens[b]]
            big = rows.abs().amax((1, 2)).tolist()
            for h in range(c["Hkv"]):
                sc = _exact_scale(big[h])
                if t > first:
                    before = float(scales[page, h, first % P // S])
                    sc = max(sc, before)
                    o = vals[page, h, first % P:at]
                    if sc != before:
                        vals[page, h, first % P:at] = _exact_round(o * before / sc)
                vals[page, h, at:at + stop - t] = _exact_round(rows[h] / sc)
                scales[page, h, first % P // S] = sc
            t = stop


def exact(case, seed):
    s, c = prepare(case, seed), dict(case)
    if c["op"] == "rope":
        return _exact_turned(s["x"], s["pos"], s["freq"].tolist(), s["mag"], c["inter"], -1.0 if c["grad"] else 1.0)
    if c["op"] == "append":
        S, N = c["sb"], c["N"]
        if c["B"] * c["Hkv"] * (N // S + 2) > 12000:
            return None  # block by block in 64 bits: too many blocks for 20 seconds
        k = s["k_new"].double()
        if c["rot"]:
            k = _exact_turned(k, s["pos"], s["freq"].tolist(), s["mag"], c["inter"], 1.0).to(torch.bfloat16).double()
        out = []
        for n, x in (("k", k), ("v", s["v_new"].double())):
            vals, sc = s[n].view(torch.float8_e4m3fn).double(), s[n + "s"].double()
            _exact_append(s, c, vals, sc, x)
            out += [vals, sc]
        return out
    P, S, Hkv, d = c["page"], c["sb"], c["Hkv"], c["d"]
    lens, table = s["lens"].tolist(), s["table"].long()
    if c["op"] == "decode":
        G, Nq = c["group"], c["Nq"]
        q = s["q"].double()
        o, lse = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=DEV)
        w = s["w"].double() if c["weights"] else None
        for b in range(c["B"]):
            n = lens[b]
            pg = table[b, :-(-n // P)]
            for h in range(Hkv if n else 0):
                K, V = ((s[m][pg, h].view(torch.float8_e4m3fn).double().reshape(-1, S, d)
                         * s[m + "s"][pg, h].double().reshape(-1, 1, 1)).reshape(-1, d)[:n] for m in ("k", "v"))
                for t in range(Nq):
                    sees = n - Nq + t + 1
                    if sees <= 0:
                        continue
                    x = (q[b, h * G:(h + 1) * G, t] @ K[:sees].T) / math.sqrt(d)
                    z = torch.logsumexp(x, -1)
                    p = torch.exp(x - z[:, None])
                    o[b, h * G:(h + 1) * G, t], lse[b, h * G:(h + 1) * G, t] = p @ V[:sees], z
                    if w is not None:
                        w[b, h, :sees] += p.sum(0)
        return [o, lse, w] if c["weights"] else [o, lse]
    C = s["new_table"].shape[1] * P
    w = torch.zeros((c["B"], Hkv, C), dtype=torch.float64, device=DEV)
    pools = {m: (s[m].view(torch.float8_e4m3fn).double(), s[m + "s"].double()) for m in ("k", "v")}
    for b in range(c["B"]):
        n, spare = lens[b], max(0, lens[b] - c["recent"])
        for h in range(Hkv):
            idx = torch.arange(n, device=DEV)
            if n > c["keep"]:
                heavy = torch.argsort(-s["w"][b, h, :spare].double(), stable=True)[:c["keep"] - c["recent"]]
                idx = torch.cat([heavy, idx[spare:]]).sort().values
            m = idx.numel()
            w[b, h, :m] = s["w"][b, h, idx].double()
            to = torch.arange(m, device=DEV)
            sp, tp = table[b, idx // P], s["new_table"].long()[b, to // P]
            for vals, sc in pools.values():
                one = sc[sp, h, idx % P // S]
                top = torch.zeros(C // S, dtype=torch.float64, device=DEV).scatter_reduce(0, to // S, one, "amax")
                vals[tp, h, to % P] = _exact_round(vals[sp, h, idx % P] * (one / top[to // S])[:, None])
                sc[tp, h, to % P // S] = top[to // S]
    return list(pools["k"]) + list(pools["v"]) + [None, w, None]
