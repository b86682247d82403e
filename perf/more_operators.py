"""Performance cases of the operators of a round whose drafts form a tree over
a paged cache: the tree's masks (`tree`), the cache as it is written
(`KeyCache.write`), the attention over it (`KeyCache.attend`), the verification
of the tree (`verify_tree`) and the accepted path's move (`KeyCache.move`).

`run` computes an operator in its plain form (elementary torch operations)
unless `own` is set; then it makes the calls a user makes of
`drafter_vocab_top_amd.topk_cols`.  `prepare` builds what the caller has in
hand, from the seed alone; `exact` restates the operators that give computed
numbers in 64 bits.

Lane l owns the columns col_start[l] .. col_start[l+1]-1.  Its column 0 is the
last committed token, the others are drafts; column j hangs below column
parents[j] < j of the lane.  Column j's key and value lie at position
lens[l] + j of the lane, in slot table[l][p / block] * block + p % block.
"""
import math

import torch

own = False


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one lane's anchor and seven drafts, as one drafter pass proposes them
        dict(name="tree one lane", op="tree", lanes=1, most=8, chain=False),
        # a large batch of 64-column trees, every lane with as many drafts as it could use
        dict(name="tree batch", op="tree", lanes=512, most=64, chain=False),
        # a decoding round of eight lanes: 64 new tokens of one layer join an 8-bit cache
        dict(name="write decode", op="write", lanes=8, most=8, heads=8, dim=128, block=16, cache="fp8", dtype="bf16"),
        # a chunk of prompts, 16,384 tokens
        dict(name="write prompts", op="write", lanes=8, most=2048, heads=8, dim=128, block=64, cache="fp8", dtype="bf16"),
        # one lane of the drafter: a 2,048-position window at the end of a long chat
        dict(name="attend one lane", op="attend", lanes=1, most=8, context=32768, window=2048, heads=8, group=4, dim=128,
             block=16, cache="bf16", chain=False),
        # the target's layer over 64 lanes, small trees, an 8-bit cache
        dict(name="attend batch", op="attend", lanes=64, most=16, context=8192, window=0, heads=8, group=4, dim=128,
             block=64, cache="fp8", chain=False),
        # two lanes at the end of very long documents
        dict(name="attend long", op="attend", lanes=2, most=8, context=131072, window=0, heads=8, group=4, dim=128,
             block=32, cache="bf16", chain=True),
        # wide trees: the products count as much as the cache's bytes
        dict(name="attend wide trees", op="attend", lanes=16, most=64, context=8192, window=0, heads=8, group=4, dim=128,
             block=16, cache="bf16", chain=False),
        # one lane's tree of 15 sampled drafts (T 1, top_p 0.95, k 20)
        dict(name="verify one tree", op="verify", lanes=1, most=16, k=20, kq=20, dtype="bf16", temperature=1.0, top_p=0.95),
        # a large batch of wide trees, long lists
        dict(name="verify trees", op="verify", lanes=512, most=64, k=64, kq=64, dtype="f32", temperature=0.8, top_p=0.9),
        # one lane's accepted path closes up, in every layer
        dict(name="move one lane", op="move", lanes=1, most=16, layers=32, heads=8, dim=128, block=16, cache="bf16"),
        # the same for a batch of wide trees
        dict(name="move batch", op="move", lanes=64, most=64, layers=32, heads=4, dim=128, block=32, cache="fp8"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tree", "write", "attend", "attend", "attend", "verify", "move"])
    heads, dim = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
    block, cache = rng.choice([1, 13, 16, 16, 32, 64, 256]), rng.choice(["bf16", "fp8"])
    if op == "tree":
        return dict(op=op, lanes=_log_int(rng, 1, 512), most=_log_int(rng, 1, 64), chain=rng.random() < 0.2)
    if op == "write":
        lanes = _log_int(rng, 1, 64)
        return dict(op=op, lanes=lanes, most=_log_int(rng, 1, max(1, 8_000_000 // (lanes * heads * dim))), heads=heads, dim=dim,
                    block=block, cache=cache, dtype=rng.choice(["bf16", "f32"]))
    if op == "attend":
        lanes, most, group = _log_int(rng, 1, 64), _log_int(rng, 1, 64), rng.choice([1, 2, 4, 5, 8])
        bytes_ = 2 if cache == "bf16" else 1
        room = min(1_000_000_000 // (2 * lanes * heads * dim * bytes_), 1_000_000_000 // (2 * lanes * heads * dim),
                   100_000_000_000 // (4 * lanes * most * heads * group * dim))
        return dict(op=op, lanes=lanes, most=most, context=_log_int(rng, 1, max(1, min(room, 131072))),
                    window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), heads=heads, group=group, dim=dim, block=block,
                    cache=cache, chain=rng.random() < 0.3)
    if op == "verify":
        return dict(op=op, lanes=_log_int(rng, 1, 512), most=_log_int(rng, 1, 64), k=rng.randint(1, 64),
                    kq=rng.choice([0, rng.randint(1, 64)]), dtype=rng.choice(["bf16", "f32"]),
                    temperature=rng.choice([0.0, 0.6, 1.0, 1.7]), top_p=rng.choice([0.5, 0.9, 0.95, 1.0]))
    lanes, most = _log_int(rng, 1, 64), _log_int(rng, 2, 64)
    layers = _log_int(rng, 1, max(1, min(32, 60_000_000 // (lanes * (most + block + 16) * heads * dim))))
    return dict(op=op, lanes=lanes, most=most, layers=layers, heads=heads, dim=dim, block=block, cache=cache)


# ----------------------------------------------------------------- inputs ---

def _starts(n):
    s = torch.zeros(n.numel() + 1, dtype=torch.int32, device=n.device)
    s[1:] = torch.cumsum(n, 0)
    return s


def _columns(c, g):
    """col_start, and for each of the C columns its lane, its place there (0 where it is nobody's: the last ones)
    and whether it is a lane's."""
    L, most = c["lanes"], c["most"]
    n = torch.randint((most + 1) // 2, most + 1, (L,), generator=g, device="cuda")
    cs = _starts(n)
    at = torch.arange(L * most, device="cuda", dtype=torch.int32)
    lane = torch.searchsorted(cs[1:].contiguous(), at, right=True).clamp(max=L - 1)
    owned = at < cs[-1]
    return cs, lane, torch.where(owned, at - cs[lane], 0).long(), owned


def _parents(c, g, place):
    """Each column below an earlier one of its lane: the one before (a chain), or any."""
    if c.get("chain"):
        return (place - 1).to(torch.int32)
    u = torch.rand(place.shape, generator=g, device="cuda", dtype=torch.float64)
    return torch.where(place > 0, (u * place).long(), -1).to(torch.int32)


def _masks(parents, place, owned, cs, lane, most):
    """Ancestors of each column as truth values (C, most), and its depth."""
    C = parents.numel()
    seen = torch.zeros((C, most), dtype=torch.bool, device="cuda")
    rows = torch.arange(C, device="cuda")
    first = cs[lane].long()
    at, depth = place.clone(), torch.zeros(C, dtype=torch.int32, device="cuda")
    for _ in range(most):
        live = owned & (at >= 0)
        seen[rows, at.clamp(0, most - 1)] |= live
        up = torch.where(live, parents[(first + at.clamp(min=0)).clamp(max=C - 1)].long(), -1)
        depth += (live & (up >= 0)).int()
        at = up
    return seen, depth


def _pack(b):
    """Rows of truth values as rows of 32-bit words, entry i in bit i % 32 of word i / 32."""
    n, v = b.shape
    w = (v + 31) // 32
    b = torch.nn.functional.pad(b, (0, w * 32 - v)).view(n, w, 32)
    words = (b.to(torch.int64) << torch.arange(32, device=b.device)).sum(2)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _table(c, g, tokens, slack):
    """Blocks of the lanes in any order: (table, number of blocks)."""
    L, bs = c["lanes"], c["block"]
    width = (tokens + bs - 1) // bs + slack
    blocks = L * width
    return torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).view(L, width), blocks


def _rows(g, shape):
    """Keys or values as a layer gives them: rows of different sizes, a few large channels."""
    x = torch.empty(shape, device="cuda").normal_(0, 1, generator=g)
    x *= torch.empty(shape[:-1] + (1,), device="cuda").normal_(0, 0.5, generator=g).exp_()
    x[..., ::17] *= 4
    return x


def _quantised(x):
    """x as e4m3 values and the exponent byte of each row's scale."""
    a = x.abs().amax(-1, keepdim=True)
    mantissa, e = torch.frexp(a)  # a = mantissa * 2^e, mantissa in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(a > 0, (e - 9 + (mantissa > 0.875)).clamp(-126, 127), -126)
    q = torch.ldexp(x, -e).to(torch.float8_e4m3fn)
    return q, (e[..., 0] + 127).to(torch.uint8)


def _fill_cache(s, c, g, layers, blocks):
    """The cache's tensors, filled: (layers, blocks, block, heads, dim), scales without the last."""
    shape = (layers, blocks, c["block"], c["heads"], c["dim"])
    for n in ("keys", "values"):
        if c["cache"] == "bf16":
            s[n] = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
        else:
            bits = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
            # e4m3 patterns from 16 to 240, as rows scaled by their largest element have, and scales of 2^-8 to 2^-5
            s[n] = ((bits & 0x87) | (0x58 + (bits & 0x18))).view(torch.float8_e4m3fn)
            s[n + "_scales"] = torch.randint(119, 123, shape[:-1], generator=g, device="cuda", dtype=torch.uint8)


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    op, L, most = c["op"], c["lanes"], c["most"]
    cs, lane, place, owned = _columns(c, g)
    s = dict(case=c, col_start=cs)
    if op == "tree":
        s["parents"] = _parents(c, g, place)
        s["lens"] = torch.randint(0, 32768, (L,), generator=g, device="cuda", dtype=torch.int32)
        s["mask"] = torch.zeros((L * most, (most + 31) // 32), dtype=torch.int32, device="cuda")
        s["positions"] = torch.full((L * most,), -1, dtype=torch.int32, device="cuda")
    elif op == "write":
        table, blocks = _table(c, g, most, 1)
        slots = table[lane, place // c["block"]].long() * c["block"] + place % c["block"]
        s["slots"] = torch.where(owned, slots, -1)
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        # as the projections leave them: keys and values side by side in one tensor
        kv = _rows(g, (L * most, 2 * c["heads"], c["dim"])).to(dt)
        s["k"], s["v"] = kv[:, :c["heads"]], kv[:, c["heads"]:]
        _fill_cache(s, c, g, 1, blocks)
    elif op == "attend":
        ctx, H, G, D = c["context"], c["heads"], c["group"], c["dim"]
        s["lens"] = torch.randint((ctx + 1) // 2, ctx + 1, (L,), generator=g, device="cuda", dtype=torch.int32)
        s["table"], blocks = _table(c, g, ctx + most, 0)
        _fill_cache(s, c, g, 1, blocks)
        s["q"] = torch.empty((L * most, H * G, D), device="cuda").normal_(0, 1.5, generator=g).to(torch.bfloat16)
        s["parents"] = _parents(c, g, place)
        seen, depth = _masks(s["parents"], place, owned, cs, lane, most)
        s["mask"], s["positions"] = _pack(seen), s["lens"][lane] + depth
        s["out"] = torch.zeros((L * most, H * G, D), dtype=torch.bfloat16, device="cuda")
    elif op == "verify":
        _prepare_verify(s, c, g, place, owned, lane)
    else:
        s["lens"] = torch.randint(0, c["block"] + 8, (L,), generator=g, device="cuda", dtype=torch.int32)
        s["table"], blocks = _table(c, g, c["block"] + 8 + most, 0)
        _fill_cache(s, c, g, c["layers"], blocks)
        # a path down a random tree: an accepted draft lies somewhere behind the one before it
        step = torch.rand((L, most), generator=g, device="cuda", dtype=torch.float64) ** 2 * 8
        path = torch.cumsum(1 + step.long(), 1) - 1 - step[:, :1].long()
        s["columns"] = torch.where(path < cs.diff()[:, None], path, -1).to(torch.int32)
    return s


def _prepare_verify(s, c, g, place, owned, lane):
    C, k, kq = place.numel(), c["k"], c["kq"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32

    def values(width):
        return torch.randn((C, width), generator=g, device="cuda").mul_(2).sort(1, descending=True)[0].to(dt)

    def tokens():  # 64 different ones of the 128 that a position is likely to take
        return (torch.rand((C, 128), generator=g, device="cuda").argsort(1)[:, :64] * 1009 % 248_046).to(torch.int32)

    base = tokens()
    s["target_values"], s["target_ids"] = values(k), base[:, :k].contiguous()
    s["parents"] = _parents(c, g, place)
    above = (s["col_start"][lane] + s["parents"]).clamp(0, C - 1).long()
    likely = torch.rand(C, generator=g, device="cuda") ** 3
    if kq:  # drafters mostly agree with their target
        near = torch.rand((C, 1), generator=g, device="cuda") < 0.7
        s["draft_values"], s["draft_ids"] = values(kq), torch.where(near, base, tokens())[:, :kq].contiguous()
        s["tokens"] = s["draft_ids"][above, (likely * kq).long().clamp(max=kq - 1)]
    else:
        s["tokens"] = s["target_ids"][above, (likely * k).long().clamp(max=k - 1)]
    s["uniforms"] = torch.rand((C, 2), generator=g, device="cuda")
    L = c["lanes"]
    s["out_tokens"], s["out_columns"] = (torch.zeros((L, c["most"]), dtype=torch.int32, device="cuda") for _ in range(2))
    s["out_count"] = torch.zeros(L, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ plain forms ---

def _tree(s):
    """Ancestors by squaring: after r steps the 2^r nearest, and the one 2^r above."""
    c, cs, parents = s["case"], s["col_start"], s["parents"]
    C, most = parents.numel(), c["most"]
    at = torch.arange(C, device=cs.device, dtype=torch.int32)
    lane = torch.searchsorted(cs[1:].contiguous(), at, right=True).clamp(max=c["lanes"] - 1)
    owned = at < cs[-1]
    j, first = torch.where(owned, at - cs[lane], 0).long(), cs[lane].long()
    seen = torch.nn.functional.one_hot(j, most).bool()
    up = torch.where(owned & (parents >= 0) & (parents < j), first + parents, -1)
    for _ in range(max(1, (most - 1).bit_length())):
        live, above = up >= 0, up.clamp(min=0)
        seen |= seen[above] & live[:, None]
        up = torch.where(live, up[above], -1)
    s["mask"].copy_(torch.where(owned[:, None], _pack(seen), s["mask"]))
    s["positions"].copy_(torch.where(owned, s["lens"][lane] + seen.sum(1, dtype=torch.int32) - 1, s["positions"]))
    return s["mask"], s["positions"]


def _write(s):
    c = s["case"]
    take = torch.nonzero(s["slots"] >= 0)[:, 0]
    slots = s["slots"][take]
    for n, x in (("keys", s["k"]), ("values", s["v"])):
        rows = x[take].float()
        if c["cache"] == "bf16":
            s[n].view(-1, c["heads"], c["dim"])[slots] = rows.to(torch.bfloat16)
        else:
            q, e = _quantised(rows)
            s[n].view(torch.uint8).view(-1, c["heads"], c["dim"])[slots] = q.view(torch.uint8)
            s[n + "_scales"].view(-1, c["heads"])[slots] = e
    return {n: s[n] for n in ("keys", "values", "keys_scales", "values_scales") if n in s}


def _rows_at(s, n, slots):
    """Rows (.., heads, dim) of the cache in 32 bits."""
    c = s["case"]
    if c["cache"] == "bf16":
        return s[n].view(-1, c["heads"], c["dim"])[slots].float()
    x = s[n].view(torch.uint8).view(-1, c["heads"], c["dim"])[slots].view(torch.float8_e4m3fn).float()
    return torch.ldexp(x, s[n + "_scales"].view(-1, c["heads"])[slots][..., None].int() - 127)


def _attend(s):
    c = s["case"]
    L, most, H, G, D, bs = c["lanes"], c["most"], c["heads"], c["group"], c["dim"], c["block"]
    cs, lens, table = s["col_start"], s["lens"].long(), s["table"]
    n = cs.diff().long()
    first = (lens - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    span = (min(c["context"], c["window"] - 1) if c["window"] else c["context"]) + most
    p = first[:, None] + torch.arange(span, device=cs.device)
    slots = table.gather(1, (p // bs).clamp(max=table.shape[1] - 1)).long() * bs + p % bs
    k = _rows_at(s, "keys", slots).permute(0, 2, 3, 1).reshape(L * H, D, span).contiguous()
    v = _rows_at(s, "values", slots).permute(0, 2, 1, 3).reshape(L * H, span, D).contiguous()
    j = torch.arange(most, device=cs.device)
    col = (cs[:-1, None] + j).clamp(max=L * most - 1).long()
    q = s["q"][col].float().view(L, most, H, G, D).permute(0, 2, 1, 3, 4).reshape(L * H, most * G, D)
    scores = torch.bmm(q, k).view(L, H, most, G, span) / math.sqrt(D)
    i = (p - lens[:, None]).clamp(0, most - 1)
    bit = (s["mask"][col].gather(2, (i // 32)[:, None, :].expand(-1, most, -1)) >> (i % 32)[:, None, :].int()) & 1
    seen = torch.where((p < lens[:, None])[:, None, :],
                       p[:, None, :] > (s["positions"][col].long()[:, :, None] - (c["window"] or 1 << 40)),
                       (bit != 0) & (p < (lens + n)[:, None])[:, None, :])
    scores = scores.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    scores = (scores - scores.amax(-1, keepdim=True).clamp(min=-1e38)).exp_()
    total = scores.sum(-1)
    o = torch.bmm(scores.view(L * H, most * G, span), v).view(L, H, most, G, D)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    live = j < n[:, None]
    s["out"][col[live]] = o.permute(0, 2, 1, 3, 4).reshape(L, most, H * G, D)[live].to(torch.bfloat16)
    return s["out"]


def _distribution(values, temperature, top_p):
    """The sampler's probabilities over a top-k list, in 64 bits."""
    v = values.double()
    k = v.shape[1]
    first = torch.arange(k, device=v.device) == 0
    if temperature == 0:
        return first.double().expand(v.shape)
    w = ((v - v[:, :1]) / temperature).exp()
    S = w.cumsum(1)
    n = (S < top_p * S[:, -1:]).sum(1, keepdim=True).clamp(max=k - 1)
    p = torch.where(torch.arange(k, device=v.device) <= n, w / S.gather(1, n), 0.0)
    return torch.where(v[:, :1].isfinite(), p, first.double())


def _verify(s):
    c, cs, parents = s["case"], s["col_start"], s["parents"]
    L, most, C = c["lanes"], c["most"], parents.numel()
    at = torch.arange(C, device=cs.device)
    lane = torch.searchsorted(cs[1:].contiguous(), at.int(), right=True).clamp(max=L - 1)
    p, ids = _distribution(s["target_values"], c["temperature"], c["top_p"]), s["target_ids"]
    u = s["uniforms"].double()
    if c["kq"]:
        q = _distribution(s["draft_values"], c["temperature"], c["top_p"])
        q_at = (q[:, None, :] * (ids[:, :, None] == s["draft_ids"][:, None, :])).sum(2)  # of each target token
    # the children of each column, in order
    draft = (at < cs[-1]) & (parents >= 0)
    above = torch.where(draft, cs[lane].long() + parents, C)
    order = torch.argsort(above, stable=True)
    sorted_above = above[order].contiguous()
    first = torch.searchsorted(sorted_above, at)
    kids = torch.searchsorted(sorted_above, at, right=True) - first
    w, W = p.clone(), torch.ones(C, dtype=torch.float64, device=cs.device)
    chosen = torch.full_like(at, -1)
    for r in range(int(kids.amax())):  # one child of every column after another
        judged = (chosen < 0) & (r < kids)
        x = order[(first + r).clamp(max=C - 1)]
        same = ids == s["tokens"][x][:, None]
        q_x = (q * (s["draft_ids"] == s["tokens"][x][:, None])).sum(1) if c["kq"] else 1.0
        yes = judged & (u[x, 0] * q_x * W < (w * same).sum(1))
        chosen = torch.where(yes, x, chosen)
        rest = (w - W[:, None] * (q_at if c["kq"] else same.double())).clamp(min=0)
        total = rest.sum(1)
        no, none = judged & ~yes, total == 0
        w = torch.where(no[:, None], torch.where(none[:, None], p, rest), w)
        W = torch.where(no, torch.where(none, 1.0, total), W)
    S = w.cumsum(1)
    pick = (S <= u[:, 1:] * S[:, -1:]).sum(1, keepdim=True)
    last = (w > 0).to(torch.int64).mul(torch.arange(1, p.shape[1] + 1, device=cs.device)).amax(1, keepdim=True) - 1
    new = ids.gather(1, torch.minimum(pick, last))[:, 0]
    # down the accepted children, and that column's token
    now, live = cs[:-1].long(), cs.diff() > 0
    s["out_tokens"].fill_(-1)
    s["out_columns"].fill_(-1)
    s["out_count"].zero_()
    t = 0
    while bool(live.any()):
        here = now.clamp(max=C - 1)
        down = torch.where(live, chosen[here], -1)
        s["out_columns"][:, t] = torch.where(live, (now - cs[:-1]).int(), -1)
        s["out_tokens"][:, t] = torch.where(live, torch.where(down >= 0, s["tokens"][down.clamp(min=0)], new[here]), -1)
        s["out_count"] += live.int()
        now, live, t = torch.where(down >= 0, down, now), live & (down >= 0), t + 1
    return s["out_tokens"], s["out_columns"], s["out_count"]


def _move(s):
    c, columns, lens = s["case"], s["columns"].long(), s["lens"].long()
    i = torch.arange(columns.shape[1], device=lens.device)

    def slot(p):
        p = p.clamp(max=s["table"].shape[1] * c["block"] - 1)
        return s["table"].gather(1, p // c["block"]).long() * c["block"] + p % c["block"]

    moved = columns > i
    src = slot(lens[:, None] + columns.clamp(min=0))[moved]
    dst = slot((lens[:, None] + i).expand_as(columns))[moved]
    for n in ("keys", "values", "keys_scales", "values_scales"):
        if n in s:
            flat = s[n] if s[n].dtype != torch.float8_e4m3fn else s[n].view(torch.uint8)
            flat = flat.view(c["layers"], -1, *flat.shape[3:])
            flat[:, dst] = flat[:, src]
    return {n: s[n] for n in ("keys", "values", "keys_scales", "values_scales") if n in s}


# ------------------------------------------------------- the framework's ---

def _own(s):
    from drafter_vocab_top_amd import topk_cols as T
    c = s["case"]
    if c["op"] == "tree":
        return T.tree(s["parents"], s["lens"], s["col_start"], mask=s["mask"], positions=s["positions"])
    if c["op"] == "verify":
        return T.verify_tree(s["target_values"], s["target_ids"], s["col_start"], s["tokens"], s["parents"], s["uniforms"],
                             draft_values=s.get("draft_values"), draft_ids=s.get("draft_ids"), temperature=c["temperature"],
                             top_p=c["top_p"], out_tokens=s["out_tokens"], out_columns=s["out_columns"], out_count=s["out_count"])
    if "handle" not in s:  # the descriptor of the cache that a program keeps
        s["handle"] = T.KeyCache(s["keys"], s["values"], s.get("keys_scales"), s.get("values_scales"))
    cache = s["handle"]
    if c["op"] == "attend":
        return cache.attend(s["q"], s["lens"], s["table"], col_start=s["col_start"], mask=s["mask"], positions=s["positions"],
                            window=c["window"], out=s["out"])
    if c["op"] == "write":
        cache.write(s["k"], s["v"], s["slots"])
    else:
        cache.move(s["lens"], s["table"], s["columns"])
    return {n: s[n] for n in ("keys", "values", "keys_scales", "values_scales") if n in s}


def run(state):
    if own:
        return _own(state)
    return dict(tree=_tree, write=_write, attend=_attend, verify=_verify, move=_move)[state["case"]["op"]](state)


# ------------------------------------------------------------------- work ---

def work(case):
    c = case
    C = 0.75 * c["lanes"] * c["most"]
    e = 2 if c.get("cache") == "bf16" else 1
    scale = 0 if c.get("cache") == "bf16" else 1
    if c["op"] == "tree":
        return {"bytes": C * (8 + 4 * ((c["most"] + 31) // 32)) + 8 * c["lanes"], "flops": 0}
    if c["op"] == "write":
        x = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": C * (2 * c["heads"] * (c["dim"] * (x + e) + scale) + 8), "flops": 0}
    if c["op"] == "attend":
        span = 0.75 * c["context"]
        span = min(span, c["window"]) if c["window"] else span
        tokens = c["lanes"] * (span + 0.75 * c["most"])
        hq = c["heads"] * c["group"]
        return {"bytes": tokens * (2 * c["heads"] * (c["dim"] * e + scale) + 4 / c["block"]) + C * hq * c["dim"] * 4,
                "flops": 4 * C * hq * c["dim"] * (span + 0.375 * c["most"])}
    if c["op"] == "verify":
        x = 2 if c["dtype"] == "bf16" else 4
        path = c["lanes"] * 2.0  # columns on the accepted path
        return {"bytes": path * (c["k"] + c["kq"]) * (x + 4) + C * 12 + c["lanes"] * c["most"] * 8,
                "flops": path * (40 * (c["k"] + c["kq"]) + 2 * c["k"] * max(1, c["kq"]))}
    moved = c["lanes"] * max(0.2, 0.2 * c["most"])
    return {"bytes": 2 * moved * c["layers"] * 2 * c["heads"] * (c["dim"] * e + scale) + 4 * c["lanes"] * c["most"], "flops": 0}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    """Attention lane by lane in 64 bits, the tree followed through its parents; the written cache before
    its rounding.  The other operators give whole numbers or copies."""
    c = case
    if c["op"] == "write":
        return _exact_write(c, prepare(c, seed))
    if c["op"] != "attend":
        return None
    s = prepare(c, seed)
    H, G, D, bs = c["heads"], c["group"], c["dim"], c["block"]
    out = s["out"].double()
    cs, lens = s["col_start"].tolist(), s["lens"].tolist()
    parents = s["parents"].tolist()
    for lane in range(c["lanes"]):
        b, n, length = cs[lane], cs[lane + 1] - cs[lane], lens[lane]
        p = torch.arange(length + n, device="cuda")
        page = s["table"][lane][p // bs].long()
        rows = []
        for name in ("keys", "values"):
            x = s[name][0][page, p % bs].double()
            if c["cache"] == "fp8":
                x = x * torch.exp2(s[name + "_scales"][0][page, p % bs].double() - 127.0)[..., None]
            rows.append(x)
        seen = torch.zeros((n, length + n), dtype=torch.bool)
        for j in range(n):
            line = []
            a = j
            while a >= 0:
                line.append(length + a)
                a = parents[b + a]
            seen[j, line] = True
            position = length + len(line) - 1
            seen[j, max(0, position - c["window"] + 1) if c["window"] else 0:length] = True
        seen = seen.cuda()
        for h in range(H):
            q = s["q"][b:b + n, h * G:(h + 1) * G].double().reshape(n * G, D)
            a = (q @ rows[0][:, h].t().contiguous()) * D ** -0.5
            a = torch.where(seen.repeat_interleave(G, 0), a, torch.tensor(-math.inf, device="cuda", dtype=torch.float64))
            a = torch.softmax(a, 1)
            out[b:b + n, h * G:(h + 1) * G] = (a @ rows[1][:, h].contiguous()).view(n, G, D)
    return out


def _exact_write(c, s):
    got = {}
    slots = s["slots"].tolist()
    take = [i for i, x in enumerate(slots) if x >= 0]
    where = torch.tensor([slots[i] for i in take], device="cuda")
    for n, x in (("keys", s["k"]), ("values", s["v"])):
        y = s[n].double().view(-1, c["heads"], c["dim"])
        rows = x[torch.tensor(take, device="cuda")].double()
        if c["cache"] == "fp8":
            largest = rows.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(largest / 448.0))
            e = torch.where(largest > 448.0 * torch.exp2(e), e + 1, e)
            e = torch.where(largest <= 448.0 * torch.exp2(e - 1), e - 1, e)
            rows = rows * torch.exp2(-e.clamp(-126, 127))
            got[n + "_scales"] = None
        y[where] = rows
        got[n] = y.view(s[n].shape)
    return got
