"""Cases of the long-context operators of the bf16 paged cache: the append with the position rotation applied on the
way and bounds of each block's keys kept, the selection of blocks by a score from those bounds, the attention over
the selected blocks, and the attention of a batch whose sequences share a prefix.

The cache is paged, [num_pages, Hkv, page, d] bf16 for K and for V; the bounds are bf16 [num_pages, Hkv, page / block,
2, d], the smallest and the largest key element of each column over the block's tokens.  ``run`` computes each
operator in its plain form (elementary torch operations in 32 bits; angles of positions, and the scores that decide
which blocks are taken, in 64) or, with ``own`` set, by the framework's calls.
"""
import math
import random

import torch

own = False
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token of each of 32 sequences, rotated and written, the bounds of its block widened
        dict(name="append_step_B32", op="append", B=32, Hkv=8, N=1, d=128, page=16, block=16, have=4096, rot=128,
             inter=False, layout="bhnd"),
        # ragged prompts, packed beside the queries as one projection leaves them
        dict(name="append_prompt_2k", op="append", B=8, Hkv=8, N=2048, d=128, page=64, block=32, have=100, rot=128,
             inter=False, layout="packed"),
        # chunks of odd lengths into a cache without bounds, half of a 64-wide head rotated
        dict(name="append_plain_d64", op="append", B=4, Hkv=16, N=777, d=64, page=48, block=0, have=1000, rot=32,
             inter=True, layout="bnhd"),
        # the ordinary batch of a server: 64 of up to 256 blocks
        dict(name="select_B32_4k", op="select", B=32, Hkv=8, group=4, Nq=1, N=4096, d=128, page=16, block=16, keep=64,
             first=1, recent=2),
        # one very long context
        dict(name="select_long_128k", op="select", B=1, Hkv=8, group=4, Nq=1, N=131072, d=128, page=128, block=32,
             keep=128, first=1, recent=4),
        # four drafted tokens of 64-wide heads in groups of eight, blocks of 24 tokens
        dict(name="select_draft_d64", op="select", B=8, Hkv=4, group=8, Nq=4, N=8000, d=64, page=48, block=24, keep=50,
             first=0, recent=3),
        # 1024 of up to 4096 tokens
        dict(name="blocks_B32_4k", op="blocks", B=32, Hkv=8, group=4, Nq=1, N=4096, d=128, page=16, block=16, keep=64),
        # 4096 of 128k tokens
        dict(name="blocks_long_128k", op="blocks", B=1, Hkv=8, group=4, Nq=1, N=131072, d=128, page=128, block=32,
             keep=128),
        # drafted tokens, odd blocks
        dict(name="blocks_draft_d64", op="blocks", B=8, Hkv=4, group=8, Nq=4, N=8000, d=64, page=48, block=24, keep=50),
        # a few short questions about one page of text
        dict(name="shared_B4_777", op="shared", B=4, Hkv=8, group=4, Nq=1, shared=777, N=100, d=128, page=16),
        # a server's system prompt
        dict(name="shared_B32_8k", op="shared", B=32, Hkv=8, group=4, Nq=1, shared=8192, N=512, d=128, page=64),
        # many samples of one long document, two drafted tokens each
        dict(name="shared_B64_32k", op="shared", B=64, Hkv=8, group=4, Nq=2, shared=32768, N=1000, d=128, page=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _page(rng):
    page = rng.choice([8, 16, 20, 32, 48, 64, 128, 256])
    return page, rng.choice([s for s in (4, 8, 16, 20, 24, 32, 64, 128) if page % s == 0])


def draw(rng):
    op = rng.choice(["append", "append", "select", "select", "blocks", "blocks", "shared", "shared", "shared"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    page, block = _page(rng)
    if op == "append":
        N = 1 if rng.random() < 0.4 else _log(rng, 2, 8192)
        B = _log(rng, 1, max(1, min(64, 8 * 8 * 2048 // (Hkv * N))))
        return dict(op=op, B=B, Hkv=Hkv, N=N, d=d, page=page, block=block if rng.random() < 0.7 else 0,
                    have=rng.choice([0, 1, 100, 1000]), rot=rng.choice([0, 32, d, d]), inter=rng.random() < 0.5,
                    layout=rng.choice(["bhnd", "bnhd", "packed"]))
    group, Nq = rng.choice([1, 2, 3, 4, 5, 8, 16]), rng.choice([1, 1, 1, 2, 5])
    if op == "shared":
        group = min(group, 8)
        B = _log(rng, 2, 128)
        most = 64 * 8 * 4 * 2 * 32768 // (B * Hkv * group * Nq)  # key times query row products, as the largest listed
        shared = _log(rng, 64, max(64, min(65536, most // 2, 8 * 32768 // Hkv)))
        N = _log(rng, 1, max(1, min(2048, 64 * 8 * 1000 // (B * Hkv))))
        return dict(op=op, B=B, Hkv=Hkv, group=group, Nq=Nq, shared=shared, N=max(N, Nq), d=d,
                    page=rng.choice([8, 16, 32, 48, 64, 128, 256]))
    N = _log(rng, 16 * block if op == "select" else 1, 131072)
    B = _log(rng, 1, max(1, min(64, 32 * 8 * 4096 // (Hkv * N))))
    blocks = -(-N // block)
    first, recent = rng.choice([0, 0, 1, 2]), rng.choice([1, 1, 2, 4])
    keep = max(first + recent + 1, min(int(blocks * rng.uniform(0.02, 0.7)), 32 * 8 * 1024 // (B * Hkv * block)))
    c = dict(op=op, B=B, Hkv=Hkv, group=group, Nq=Nq, N=N, d=d, page=page, block=block, keep=keep)
    return dict(c, first=first, recent=recent) if op == "select" else c


def _lengths(case, most):
    """Tokens of each sequence: spread from half full up to `most`.  A function of the case alone."""
    B = case["B"]
    if B == 1:
        return [most]
    r = random.Random(B * 1000003 + most)
    lens = [r.randint(most // 2, most) for _ in range(B)]
    lens[0] = most
    if B > 3 and case["op"] != "append":
        lens[B // 2] = 0  # a slot of the batch without a sequence
    return lens


def _shared_lengths(case):
    """Lengths with the shared tokens: own tokens spread from the drafts up to N, a slot without a sequence."""
    r = random.Random(case["B"] * 1000003 + case["N"])
    lens = [case["shared"] + r.randint(case["Nq"], case["N"]) for _ in range(case["B"])]
    if case["B"] > 3:
        lens[case["B"] // 2] = 0
    return lens


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(DEV).manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _turns(freq):
    """Turns per position as 64-bit fixed-point fractions (the table the framework's rotation takes)."""
    t = [int(round(f / (2 * math.pi) * 2.0 ** 64)) % (1 << 64) for f in freq]
    return torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in t], dtype=torch.int64, device=DEV)


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


def _pool(g, case, pages):
    """Page pools full of tokens; two columns of the keys are larger than the others."""
    shape = (pages, case["Hkv"], case["page"], case["d"])
    k, v = (torch.empty(shape, dtype=torch.bfloat16, device=DEV) for _ in "kv")
    step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = _randn(g, n, *shape[1:])
        x[..., 3] *= 6.0
        k[i:i + n] = x
        v[i:i + n] = _randn(g, n, *shape[1:])
    return k, v


def _extremes(g, pages, case):
    """Bounds as blocks of real keys have them: the keys of a block lie around a common mean."""
    shape = (pages, case["Hkv"], case["page"] // case["block"], case["d"])
    mean, lo, hi = 0.7 * _randn(g, *shape), 1.6 + 0.4 * _randn(g, *shape), 1.6 + 0.4 * _randn(g, *shape)
    x = torch.stack([mean - lo.abs(), mean + hi.abs()], 3)
    x[..., 3] *= 6.0
    return x.to(torch.bfloat16)


def _table(g, B, maxp, pages):
    """int32 [B, maxp] of distinct pages, shuffled as a server's allocator leaves them."""
    return torch.randperm(pages, generator=g, device=DEV)[:B * maxp].reshape(B, maxp).to(torch.int32)


def _lists(g, c, lens):
    """Ascending distinct blocks of each sequence and kv head, its last one among them, -1 behind them."""
    many = -(-c["N"] // c["block"])
    n = ((lens.long() + c["block"] - 1) // c["block"])[:, None, None]
    j = torch.arange(many, device=DEV)
    rank = torch.rand((c["B"], c["Hkv"], many), generator=g, device=DEV)
    rank = torch.where(j == n - 1, torch.full_like(rank, 2.0), rank).masked_fill(j >= n, -1.0)
    top = torch.topk(rank, min(c["keep"], many), -1)
    out = torch.where(top.values >= 0, top.indices, torch.full_like(top.indices, many)).sort(-1).values
    out = torch.nn.functional.pad(out, (0, c["keep"] - out.shape[-1]), value=many)
    return torch.where(out < many, out, -torch.ones_like(out)).to(torch.int32).contiguous()


def prepare(case, seed):
    c, g, s = dict(case), _gen(seed), {}
    s["case"] = c
    B, d, P = c["B"], c["d"], c["page"]
    if c["op"] == "append":
        have = _lengths(c, c["have"])
        new = [max(1, n) for n in _lengths(c, c["N"])]
        maxp = -(-(max(have) + c["N"]) // P)
        s["k_new"] = _activations(g, B, c["Hkv"], c["N"], d, c["layout"])
        s["v_new"] = _activations(g, B, c["Hkv"], c["N"], d, c["layout"])
        s["k"], s["v"] = _pool(g, c, B * maxp + 3)
        if c["block"]:
            s["bounds"] = _extremes(g, B * maxp + 3, c)
        s["table"], s["lens"], s["new"] = _table(g, B, maxp, B * maxp + 3), _ints(have), _ints(new)
        s["pos"] = (s["lens"][:, None] + torch.arange(c["N"], device=DEV, dtype=torch.int32) + 11).contiguous()
        if c["rot"]:
            freq = [10000.0 ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)]
            s["freq"], s["turns"] = torch.tensor(freq, dtype=torch.float64, device=DEV), _turns(freq)
        return s
    s["q"] = _randn(g, B, c["Hkv"] * c["group"], c["Nq"], d).to(torch.bfloat16)
    if c["op"] == "shared":
        # the shared pages stand first in every row; the page that the prefix ends in is each sequence's own copy
        lens, full = _shared_lengths(c), c["shared"] // P
        own_pages = -(-max(lens) // P) - full
        pages = full + B * own_pages + 2
        s["k"], s["v"] = _pool(g, c, pages)
        p = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.cat([p[:full].expand(B, full), p[full:full + B * own_pages].reshape(B, own_pages)], 1).contiguous()
        rest = c["shared"] - full * P
        if rest:
            at = s["table"][:, full].long()
            for n in "kv":
                s[n][at, :, :rest] = s[n][at[0], :, :rest]
        s["lens"], s["shared"] = _ints(lens), _ints([c["shared"]])
        return s
    maxp = -(-c["N"] // P)
    s["lens"] = _ints(_lengths(c, c["N"]))
    s["table"] = _table(g, B, maxp, B * maxp + 3)
    if c["op"] == "select":
        s["bounds"] = _extremes(g, B * maxp + 3, c)
        return s
    s["k"], s["v"] = _pool(g, c, B * maxp + 3)
    s["blocks"] = _lists(g, c, s["lens"])
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, pos, freq, inter):
    """fp32 rotation of x [B, H, N, d] (any strides) by pos [B, N]; angles in 64 bits."""
    half = freq.numel()
    a = pos.double()[:, None, :, None] * freq
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    x = x.float()
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    if inter:
        x1, x2 = r[..., 0::2], r[..., 1::2]
        return torch.cat([torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2), rest], -1)
    x1, x2 = r[..., :half], r[..., half:]
    return torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin, rest], -1)


def _append(s, c):
    k = s["k_new"]
    if c["rot"]:
        k = _rotate(k, s["pos"], s["freq"], c["inter"]).to(torch.bfloat16)
    P, S, B, N = c["page"], c["block"], c["B"], c["N"]
    lens, new, table = s["lens"].long(), s["new"].long(), s["table"].long()
    i = torch.arange(N, device=DEV)
    fresh = i < new[:, None]                                                       # [B, N]
    b, n = fresh.nonzero(as_tuple=True)
    t = lens[b] + n
    page = table[b, t // P]
    s["k"][page, :, t % P] = k[b, :, n]
    s["v"][page, :, t % P] = s["v_new"][b, :, n]
    if not S:
        return
    many = (N + S - 2) // S + 1
    blk = (lens // S)[:, None] + torch.arange(many, device=DEV)                    # [B, many]
    pos = blk[..., None] * S + torch.arange(S, device=DEV)
    new_here = (pos >= lens[:, None, None]) & (pos < (lens + new)[:, None, None])  # [B, many, S]
    at = (pos - lens[:, None, None]).clamp(0, N - 1)
    val = k.transpose(1, 2)[torch.arange(B, device=DEV)[:, None, None], at].float()  # [B, many, S, Hkv, d]
    lo = val.masked_fill(~new_here[..., None, None], math.inf).amin(2)
    hi = val.masked_fill(~new_here[..., None, None], -math.inf).amax(2)
    use = new_here.any(-1)
    page = table[torch.arange(B, device=DEV)[:, None], (blk * S // P).clamp_max(table.shape[1] - 1)]
    slot = blk * S % P // S
    was = s["bounds"][page, :, slot].float()                                       # [B, many, Hkv, 2, d]
    old = (blk * S < lens[:, None])[..., None, None]
    lo = torch.where(old, torch.minimum(lo, was[..., 0, :]), lo)
    hi = torch.where(old, torch.maximum(hi, was[..., 1, :]), hi)
    s["bounds"][page[use], :, slot[use]] = torch.stack([lo, hi], 3)[use].to(torch.bfloat16)


def _select(s, c):
    """Blocks by the largest score that a row of the group can have with a key within the bounds."""
    S, B, Hkv, d, keep = c["block"], c["B"], c["Hkv"], c["d"], c["keep"]
    x = s["bounds"][s["table"].long()].transpose(1, 2).flatten(2, 3).double()      # [B, Hkv, blocks, 2, d]
    q = s["q"].double().reshape(B, Hkv, -1, d)
    score = (q.clamp_min(0.0) @ x[..., 1, :].transpose(-1, -2) + q.clamp_max(0.0) @ x[..., 0, :].transpose(-1, -2)).amax(2)
    j = torch.arange(score.shape[-1], device=DEV)
    n = ((s["lens"].long() + S - 1) // S)[:, None, None]
    score = score.masked_fill((j < c["first"]) | (j >= n - c["recent"]), math.inf).masked_fill(j >= n, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]
    order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=score.shape[-1])
    order = torch.where(order < n, order, torch.full_like(order, score.shape[-1])).sort(-1).values
    return torch.where(order < n, order, -torch.ones_like(order)).to(torch.int32)


def _softmax(x):
    """Weights and natural log-sum-exp of masked scores; rows without keys get weights of zero."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(x - m)
    l = p.sum(-1, keepdim=True)
    return p / torch.where(l > 0, l, torch.ones_like(l)), (m + torch.log(l)).squeeze(-1)


def _blocks(s, c):
    P, S, B, Hkv, G, Nq, d = c["page"], c["block"], c["B"], c["Hkv"], c["group"], c["Nq"], c["d"]
    blk = s["blocks"].long()
    tok = (blk[..., None] * S + torch.arange(S, device=DEV)).flatten(2)            # [B, Hkv, keep * S]
    there = (blk >= 0).repeat_interleave(S, -1) & (tok < s["lens"].long()[:, None, None])
    tok = torch.where(there, tok, torch.zeros_like(tok))
    b, h = torch.arange(B, device=DEV)[:, None, None], torch.arange(Hkv, device=DEV)[None, :, None]
    page = s["table"].long()[b, tok // P]
    k, v = (s[n][page, h, tok % P].float().masked_fill(~there[..., None], 0.0) for n in "kv")
    q = s["q"].float().reshape(B, Hkv, G * Nq, d)
    last = s["lens"].long()[:, None] - Nq + torch.arange(Nq, device=DEV).repeat(G)   # the last key that a row sees
    seen = there[:, :, None] & (tok[:, :, None] <= last[:, None, :, None])
    p, lse = _softmax((q @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))).masked_fill(~seen, -math.inf))
    return (p @ v).to(torch.bfloat16).reshape(B, Hkv * G, Nq, d), lse.reshape(B, Hkv * G, Nq)


def _shared(s, c):
    """The prefix against the rows of all sequences at once, each sequence's own tokens behind it."""
    P, B, Hkv, G, Nq, d, many = c["page"], c["B"], c["Hkv"], c["group"], c["Nq"], c["d"], c["shared"]
    table, scale = s["table"].long(), 1.0 / math.sqrt(d)
    q = s["q"].float().reshape(B, Hkv, G * Nq, d)
    first = table[0, :-(-many // P)]
    k, v = (s[n][first].transpose(0, 1).flatten(1, 2)[:, :many].float() for n in "kv")   # [Hkv, shared, d]
    last = (s["lens"].long()[:, None] - Nq + torch.arange(Nq, device=DEV).repeat(G))[:, None]  # [B, 1, rows]
    x = q.transpose(0, 1).reshape(Hkv, B * G * Nq, d) @ k.transpose(-1, -2) * scale
    x = x.reshape(Hkv, B, G * Nq, many).transpose(0, 1)
    x = x.masked_fill(torch.arange(many, device=DEV) > last[..., None], -math.inf)
    skip = many // P                                                               # own tokens: from this page on
    tail = table[:, skip:]
    tok = skip * P + torch.arange(tail.shape[1] * P, device=DEV)
    kt, vt = (s[n][tail].transpose(1, 2).flatten(2, 3).float() for n in "kv")      # [B, Hkv, tokens, d]
    mine = (tok >= many) & (tok < s["lens"].long()[:, None])                       # [B, tokens]
    vt = vt.masked_fill(~mine[:, None, :, None], 0.0)
    y = q @ kt.transpose(-1, -2) * scale
    y = y.masked_fill(~(mine[:, None, None] & (tok <= last[..., None])), -math.inf)
    p, lse = _softmax(torch.cat([x, y], -1))
    o = (p[..., :many].transpose(0, 1).reshape(Hkv, B * G * Nq, many) @ v).reshape(Hkv, B, G * Nq, d).transpose(0, 1)
    o = o + p[..., many:] @ vt
    return o.to(torch.bfloat16).reshape(B, Hkv * G, Nq, d), lse.reshape(B, Hkv * G, Nq)


def run(state):
    s, c = state, state["case"]
    if own:
        import exact_tiled_attention_21_gb300 as fa
        if c["op"] == "append":
            fa.cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], new_lens=s["new"],
                            turns=s.get("turns"), positions=s["pos"], interleaved=c["inter"], bounds=s.get("bounds"))
            return [s["k"], s["v"]] + ([s["bounds"]] if c["block"] else [])
        if c["op"] == "select":
            return fa.select_blocks(s["q"], s["bounds"], s["table"], s["lens"], block=c["block"], keep=c["keep"],
                                    first=c["first"], recent=c["recent"])
        if c["op"] == "blocks":
            return fa.decode_blocks(s["q"], s["k"], s["v"], s["table"], s["lens"], s["blocks"], block=c["block"])
        return fa.decode_shared(s["q"], s["k"], s["v"], s["table"], s["lens"], s["shared"])
    if c["op"] == "append":
        _append(s, c)
        return [s["k"], s["v"]] + ([s["bounds"]] if c["block"] else [])
    return {"select": _select, "blocks": _blocks, "shared": _shared}[c["op"]](s, c)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, d, Hkv = case, case["d"], case["Hkv"]
    if c["op"] == "append":
        new = [max(1, n) for n in _lengths(c, c["N"])]
        t = sum(new) * Hkv
        touched = 0.0
        if c["block"]:  # a block's bounds are written, and read where it holds earlier tokens
            for have, n in zip(_lengths(c, c["have"]), new):
                touched += (have + n - 1) // c["block"] - have // c["block"] + 1 + (1 if have % c["block"] else 0)
        return {"bytes": 8.0 * d * t + 4.0 * d * Hkv * touched, "flops": 3.0 * t * c["rot"]}
    rows = c["group"] * c["Nq"]
    io = c["B"] * Hkv * rows * (4.0 * d + 4.0)
    if c["op"] == "shared":
        lens = _shared_lengths(c)
        t = sum(max(0, n - c["shared"]) for n in lens)
        return {"bytes": 4.0 * d * Hkv * (c["shared"] + t) + io, "flops": 4.0 * d * rows * Hkv * sum(lens)}
    n = [-(-x // c["block"]) for x in _lengths(c, c["N"])]
    if c["op"] == "select":
        return {"bytes": 4.0 * d * Hkv * sum(n) + c["B"] * Hkv * (2.0 * rows * d + 4.0 * c["keep"]),
                "flops": 4.0 * d * rows * Hkv * sum(n)}
    t = sum(min(x, c["keep"]) * c["block"] for x in n) * Hkv
    return {"bytes": 4.0 * d * t + io + 4.0 * c["B"] * Hkv * c["keep"], "flops": 4.0 * d * rows * t}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_append(s, c):
    k, v = s["k_new"].double(), s["v_new"].double()
    if c["rot"]:
        y = k.clone()
        for i in range(c["rot"] // 2):
            ang = s["pos"].double() * float(s["freq"][i])
            cs, sn = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
            p, r = (2 * i, 2 * i + 1) if c["inter"] else (i, i + c["rot"] // 2)
            y[..., p] = cs * k[..., p] - sn * k[..., r]
            y[..., r] = sn * k[..., p] + cs * k[..., r]
        k = y
    kc, vc = s["k"].double(), s["v"].double()
    bd = s["bounds"].double() if c["block"] else None
    P, S = c["page"], c["block"]
    lens, new, table = s["lens"].tolist(), s["new"].tolist(), s["table"].tolist()
    for b in range(c["B"]):
        t = lens[b]
        while t < lens[b] + new[b]:  # page by page, or block by block
            unit = S or P
            stop = min((t // unit + 1) * unit, lens[b] + new[b])
            page, at = table[b][t // P], t % P
            rows = k[b, :, t - lens[b]:stop - lens[b]]
            kc[page, :, at:at + stop - t] = rows
            vc[page, :, at:at + stop - t] = v[b, :, t - lens[b]:stop - lens[b]]
            if S:
                ends = torch.stack([rows.amin(1), rows.amax(1)], 1)
                if t % S:
                    was = bd[page, :, at // S]
                    ends = torch.stack([torch.minimum(ends[:, 0], was[:, 0]), torch.maximum(ends[:, 1], was[:, 1])], 1)
                bd[page, :, at // S] = ends
            t = stop
    return [kc, vc] + ([bd] if S else [])


def exact(case, seed):
    c = dict(case)
    if c["op"] == "select":
        return None  # whole numbers: which blocks, decided in 64 bits by the plain form too
    if c["op"] == "append" and c["B"] * (c["N"] // (c["block"] or c["page"]) + 2) > 20000:
        return None  # block by block: too many for 20 seconds
    s = prepare(case, seed)
    if c["op"] == "append":
        return _exact_append(s, c)
    P, Hkv, G, Nq, d = c["page"], c["Hkv"], c["group"], c["Nq"], c["d"]
    lens, table = s["lens"].tolist(), s["table"].long()
    q = s["q"].double()
    o, lse = torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    for b in range(c["B"]):
        n = lens[b]
        for h in range(Hkv if n else 0):
            idx = torch.arange(n, device=DEV)
            if c["op"] == "blocks":
                mine = s["blocks"][b, h].long()
                idx = (mine[mine >= 0][:, None] * c["block"] + torch.arange(c["block"], device=DEV)).flatten()
                idx = idx[idx < n]
            K, V = (s[m][table[b, idx // P], h, idx % P].double() for m in "kv")
            x = torch.einsum("gtd,jd->gtj", q[b, h * G:(h + 1) * G], K) / math.sqrt(d)
            for t in range(Nq):
                sees = idx <= n - Nq + t
                if not bool(sees.any()):
                    continue
                y = x[:, t][:, sees]
                z = torch.logsumexp(y, -1)
                lse[b, h * G:(h + 1) * G, t] = z
                o[b, h * G:(h + 1) * G, t] = torch.exp(y - z[:, None]) @ V[sees]
    return [o, lse]
