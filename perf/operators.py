"""Performance cases of the operators around a drafting round's top-k: the
logit rules (`AdjustRules`), the token history they read (`count_tokens`), the
verification of drafts (`verify`) and the batch plan (`plan`).

`run` computes an operator in its plain form (elementary torch operations)
unless `own` is set; then it makes the calls a user makes of
`drafter_vocab_top_amd.topk_cols`.  `prepare` builds what the caller has in
hand, from the seed alone; `exact` restates the logit rules in 64 bits.

A round's matrix has one column per position and a lane owns contiguous
columns: 7 drafts of a lane give 7 columns of the drafter's logits and 8 of
the target's (the drafts and the position behind them).
"""
import math

import numpy as np
import torch

own = False

VOCAB = 248_046       # the drafter's vocabulary
SHORTLIST = 131_072   # the shortlist head's rows
FLAG = -(1 << 31)     # bit 31 of a history word: the token occurs in the prompt


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one lane's target logits, penalties over a chat of 2,000 tokens and the drafts before each column;
        # the raw logits are kept for reported probabilities, so the result goes elsewhere
        dict(name="adjust one lane", op="adjust", V=VOCAB, lanes=1, cols=8, dtype="bf16", layout="col", pad=0,
             in_place=False, hist=2000, bias=0, mask="none", keep=1.0, drafts=True, ragged=False),
        # eight lanes' drafter logits, penalised where they lie
        dict(name="adjust in place", op="adjust", V=VOCAB, lanes=8, cols=7, dtype="bf16", layout="col", pad=0,
             in_place=True, hist=4000, bias=0, mask="none", keep=1.0, drafts=False, ragged=False),
        # constrained output: every column has a grammar mask that leaves little, plus a user's bias list
        dict(name="adjust grammar", op="adjust", V=VOCAB, lanes=8, cols=7, dtype="bf16", layout="col", pad=18,
             in_place=True, hist=600, bias=300, mask="column", keep=0.02, drafts=False, ragged=True),
        # the shortlist head in fp32 with every rule, lanes with fewer drafts than they may have
        dict(name="adjust shortlist f32", op="adjust", V=SHORTLIST, lanes=8, cols=8, dtype="f32", layout="col", pad=0,
             in_place=False, hist=1500, bias=100, mask="lane", keep=0.9, drafts=True, ragged=True),
        # the largest batch, rows interleaved
        dict(name="adjust interleaved", op="adjust", V=VOCAB, lanes=64, cols=7, dtype="bf16", layout="row", pad=0,
             in_place=False, hist=1000, bias=50, mask="lane", keep=0.5, drafts=False, ragged=False),
        # the end of a round: up to 8 committed tokens a lane join the histories
        dict(name="count commit", op="count", V=VOCAB, lanes=64, prompt=0, output=8, fresh=0.0),
        # lanes admitted with their prompts, some resumed with output they had already
        dict(name="count admit", op="count", V=VOCAB, lanes=8, prompt=32768, output=2000, fresh=1.0),
        # one lane's 7 sampled drafts against the target: the sampling recipe of the drafter (T 1, top_p 0.95, k 20)
        dict(name="verify one lane", op="verify", lanes=1, drafts=7, k=20, kq=20, dtype="bf16", temperature=1.0,
             top_p=0.95, greedy_drafts=False),
        # a large batch of 15-token drafts, long lists
        dict(name="verify batch", op="verify", lanes=512, drafts=15, k=64, kq=64, dtype="f32", temperature=0.8,
             top_p=0.9, greedy_drafts=False),
        # drafts taken greedily, checked under sampling
        dict(name="verify one-hot drafts", op="verify", lanes=64, drafts=7, k=20, kq=0, dtype="bf16", temperature=1.0,
             top_p=0.95, greedy_drafts=True),
        # a decoding round of 64 lanes: anchor and up to 7 drafts each, padded to the full batch
        dict(name="plan decode", op="plan", lanes=64, most=8, context=32768, block=16, spare=1.0, room=1.0),
        # prompts arriving in chunks among decoding lanes: about half a million tokens, not quite all of their blocks free
        dict(name="plan prefill", op="plan", lanes=512, most=2048, context=65536, block=64, spare=0.9, room=0.55),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["adjust", "adjust", "count", "verify", "plan"])
    if op == "adjust":
        V = _log_int(rng, 500, VOCAB)
        lanes = _log_int(rng, 1, 64)
        cols = rng.randint(1, 16)
        while V * lanes * cols > VOCAB * 200:
            lanes = max(1, lanes // 2)
        layout = rng.choice(["col", "col", "row"])
        return dict(op="adjust", V=V, lanes=lanes, cols=cols, dtype=rng.choice(["bf16", "f32"]), layout=layout,
                    pad=rng.choice([0, 0, 1, 2, 10, 64]), in_place=rng.random() < 0.4,
                    hist=rng.choice([0, 1, _log_int(rng, 2, 8000)]), bias=rng.choice([0, 0, _log_int(rng, 1, 500)]),
                    mask=rng.choice(["none", "column", "lane"]), keep=rng.choice([0.0, 0.01, 0.5, 0.95, 1.0]),
                    drafts=rng.random() < 0.5, ragged=rng.random() < 0.5)
    if op == "count":
        lanes = _log_int(rng, 1, 64)
        return dict(op="count", V=_log_int(rng, 500, VOCAB), lanes=lanes, prompt=_log_int(rng, 1, 262144 // lanes),
                    output=rng.choice([0, 1, _log_int(rng, 1, 4000)]), fresh=rng.choice([0.0, 0.5, 1.0]))
    if op == "verify":
        greedy = rng.random() < 0.3
        return dict(op="verify", lanes=_log_int(rng, 1, 512), drafts=rng.randint(0, 15), k=rng.randint(1, 64),
                    kq=0 if greedy else rng.randint(1, 64), dtype=rng.choice(["bf16", "f32"]),
                    temperature=rng.choice([0.0, 0.6, 1.0, 1.7]), top_p=rng.choice([0.5, 0.9, 0.95, 1.0]),
                    greedy_drafts=greedy)
    lanes, block = _log_int(rng, 1, 2000), rng.choice([1, 13, 16, 32, 64, 256])
    return dict(op="plan", lanes=lanes, most=_log_int(rng, 1, 262144 // lanes + 1),
                context=_log_int(rng, 1, min(65536, 4_000_000 * block // lanes)), block=block,
                spare=rng.choice([0.5, 0.9, 1.0]), room=rng.choice([0.4, 0.6, 1.0]))


# ----------------------------------------------------------------- inputs ---

def _tokens(g, n, V):
    """Token ids whose frequency falls with the id, as a vocabulary sorted by use gives."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return torch.clamp((u * math.log(V)).exp().to(torch.int32) - 1, 0, V - 1)


def _starts(n):
    s = torch.zeros(n.numel() + 1, dtype=torch.int32, device=n.device)
    s[1:] = torch.cumsum(n, 0)
    return s


def _pack(b):
    """Rows of truth values as rows of 32-bit words, row r in bit r % 32 of word r / 32."""
    n, v = b.shape
    w = (v + 31) // 32
    b = torch.nn.functional.pad(b, (0, w * 32 - v)).view(n, w, 32)
    words = (b.to(torch.int64) << torch.arange(32, device=b.device)).sum(2)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _bits(words, V):
    b = (words[:, :, None] >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1
    return b.reshape(words.shape[0], -1)[:, :V] != 0


def _prepare_adjust(c, g):
    V, L, n = c["V"], c["lanes"], c["cols"]
    C = L * n
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    shape = (C, V + c["pad"]) if c["layout"] == "col" else (V, C + c["pad"])
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0, 4, generator=g).to(dt)
    s = dict(x=x, out=x if c["in_place"] else torch.zeros_like(x))
    have = torch.randint(0, n + 1, (L,), generator=g, device="cuda") if c["ragged"] else torch.full((L,), n, device="cuda")
    s["col_start"] = _starts(have)
    s["draft_start"] = _starts((have - 1).clamp(min=0))
    s["draft_ids"] = _tokens(g, C, V)
    counts = torch.zeros((L, V), dtype=torch.int32, device="cuda")
    if c["hist"]:
        h = c["hist"]
        lane = torch.arange(L, device="cuda").repeat_interleave(h) * V
        counts.view(-1).index_add_(0, lane + _tokens(g, L * h, V), torch.ones(L * h, dtype=torch.int32, device="cuda"))
        prompt = torch.zeros(L * V, dtype=torch.bool, device="cuda")
        prompt[lane + _tokens(g, L * h, V)] = True
        counts = torch.where(prompt.view(L, V), counts | FLAG, counts)
    s["counts"], s["seen"] = counts, _pack(counts != 0)
    s["repetition"] = 1.0 + 0.5 * torch.rand(L, generator=g, device="cuda")
    s["presence"] = torch.rand(L, generator=g, device="cuda")
    s["frequency"] = 0.3 * torch.rand(L, generator=g, device="cuda")
    b = c["bias"]
    s["bias_start"] = _starts(torch.full((L,), b, device="cuda"))
    s["bias_ids"] = _tokens(g, L * b, V)
    s["bias_values"] = 4 * torch.randn(L * b, generator=g, device="cuda")
    masks = dict(none=0, lane=L, column=C)[c["mask"]]
    if masks:
        words = [_pack(torch.rand((min(16, masks - i), V), generator=g, device="cuda") < c["keep"]) for i in range(0, masks, 16)]
        s["mask"] = torch.cat(words)
        s["mask_index"] = torch.arange(C, dtype=torch.int32, device="cuda") // (C // masks)
        if c["mask"] == "lane":  # a lane without a grammar
            s["mask_index"][:n] = -1 if L > 1 else 0
    return s


def _prepare_count(c, g):
    V, L = c["V"], c["lanes"]
    p = torch.randint((c["prompt"] + 1) // 2, c["prompt"] + 1, (L,), generator=g, device="cuda")
    o = torch.randint(min(1, c["output"]), c["output"] + 1, (L,), generator=g, device="cuda")
    start = _starts(p + o)
    ids = _tokens(g, L * (c["prompt"] + c["output"]), V)
    ids[torch.rand(ids.numel(), generator=g, device="cuda") < 0.01] = -1  # padding, as a verification leaves it
    counts = torch.zeros((L, V), dtype=torch.int32, device="cuda")
    counts.view(-1)[torch.arange(L, device="cuda") * V + _tokens(g, L, V)] = 3
    fresh = (torch.rand(L, generator=g, device="cuda") < c["fresh"]).to(torch.int32)
    return dict(ids=ids, start=start, prompt_len=p.to(torch.int32), counts=counts, seen=_pack(counts != 0), fresh=fresh)


def _prepare_verify(c, g):
    L, D, k, kq = c["lanes"], c["drafts"], c["k"], c["kq"]
    V = VOCAB
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    have = torch.randint((D + 1) // 2, D + 1, (L,), generator=g, device="cuda")
    ds, cs = _starts(have), _starts(have + 1)
    Cd, Ct = L * D, L * (D + 1)

    def values(n, width):
        return torch.randn((n, width), generator=g, device="cuda").mul_(2).sort(1, descending=True)[0].to(dt)

    def tokens(n):  # 64 different ones of the 128 that a position is likely to take
        return (torch.rand((n, 128), generator=g, device="cuda").argsort(1)[:, :64] * 1009 % V).to(torch.int32)

    tv, base = values(Ct, k), tokens(Ct)
    ti = base[:, :k].contiguous()
    s = dict(col_start=cs, draft_start=ds, target_values=tv, target_ids=ti)
    lane = torch.searchsorted(ds[1:].contiguous(), torch.arange(Cd, device="cuda", dtype=torch.int32), right=True).clamp(max=L - 1)
    at = (torch.arange(Cd, device="cuda") + lane).clamp(max=Ct - 1)  # the column that judges a draft
    if c["greedy_drafts"]:
        likely = (torch.rand(Cd, generator=g, device="cuda") ** 3 * k).long().clamp(max=k - 1)
        s["drafts"] = ti[at, likely] if Cd else torch.zeros(0, dtype=torch.int32, device="cuda")
    else:
        near = torch.rand((Cd, 1), generator=g, device="cuda") < 0.7  # drafters mostly agree with their target
        qv, qi = values(Cd, kq), torch.where(near, base[at], tokens(Cd))[:, :kq].contiguous()
        pick = (torch.rand(Cd, generator=g, device="cuda") ** 3 * kq).long().clamp(max=kq - 1)
        s.update(draft_values=qv, draft_ids=qi, drafts=qi[torch.arange(Cd, device="cuda"), pick])
    s["drafts"] = torch.cat([s["drafts"], s["drafts"].new_zeros(1)]).contiguous()  # never empty
    s["seed"], s["offset"] = int(torch.randint(0, 2**31, (1,), generator=g, device="cuda")), 11
    s["uniforms"] = torch.from_numpy(_uniforms(s["seed"], s["offset"], Ct)).cuda()
    s["out_tokens"] = torch.zeros((L, D + 1), dtype=torch.int32, device="cuda")
    s["out_count"] = torch.zeros(L, dtype=torch.int32, device="cuda")
    return s


def _uniforms(seed, offset, n):
    """The two uniforms of each target column: Philox4x32-10 with counter (offset, column, 1 or 2) and the seed as key."""
    out = np.empty((2, n))
    for which in (1, 2):
        c = [np.full(n, offset & 0xFFFFFFFF, np.uint64), np.full(n, offset >> 32, np.uint64),
             np.arange(n, dtype=np.uint64), np.full(n, which, np.uint64)]
        k = [seed & 0xFFFFFFFF, seed >> 32]
        for _ in range(10):
            a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
            low = np.uint64(0xFFFFFFFF)
            c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
            k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
        out[which - 1] = (((c[0] << np.uint64(32)) | c[1]) >> np.uint64(11)).astype(np.float64) * 2.0**-53
    return out


def _capacity(c):
    return int(c["lanes"] * c["most"] * c["room"]) + 1


def _prepare_plan(c, g):
    L, bs = c["lanes"], c["block"]
    lens = (torch.rand(L, generator=g, device="cuda") * c["context"]).to(torch.int32)
    add = torch.randint(0, c["most"] + 1, (L,), generator=g, device="cuda", dtype=torch.int32)
    held = (lens + bs - 1) // bs
    ahead = torch.rand(L, generator=g, device="cuda") < 0.3  # blocks left from refused drafts
    held = (held + ahead.int()).to(torch.int32)
    width = (c["context"] + c["most"]) // bs + 2
    need = ((lens + add + bs - 1) // bs - held).clamp(min=0)
    total = int(held.sum()) + int(need.sum()) + 8
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((L, width), -1, dtype=torch.int32, device="cuda")
    first = torch.cumsum(held, 0) - held
    at = torch.arange(width, device="cuda")
    filled = at[None, :] < held[:, None]
    table = torch.where(filled, order[(first[:, None] + at[None, :]).clamp(max=total - 1)], table)
    free_ids = order[int(held.sum()):].contiguous()
    free = torch.tensor([int(int(need.sum()) * c["spare"])], dtype=torch.int32, device="cuda")
    cap = _capacity(c)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    out = dict(held=i32(L), free_count=i32(1), refused=i32(1), col_start=i32(L + 1), col_lane=i32(cap), col_pos=i32(cap),
               slots=torch.zeros(cap, dtype=torch.int64, device="cuda"))
    return dict(lens=lens, add=add, held=held, table=table, free_ids=free_ids, free_count=free, capacity=cap, out=out)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = dict(adjust=_prepare_adjust, count=_prepare_count, verify=_prepare_verify, plan=_prepare_plan)[case["op"]]
    return dict(make(case, g), case=case)


# ------------------------------------------------------------ plain forms ---

def _column_lanes(start, C):
    """Lane of each column, its place in the lane and whether it belongs to one."""
    c = torch.arange(C, device=start.device, dtype=torch.int32)
    lane = torch.searchsorted(start[1:].contiguous(), c, right=True).clamp(max=start.numel() - 2)
    return lane, c - start[lane], c < start[-1]


def _adjust(s):
    c = s["case"]
    V, C = c["V"], c["lanes"] * c["cols"]
    col = c["layout"] == "col"
    x = s["x"][:, :V].float() if col else s["x"][:, :C].float().t()
    lane, j, active = _column_lanes(s["col_start"], C)
    word = s["counts"][lane]
    n, prompt = word & 0x7FFFFFFF, word < 0
    if c["drafts"]:
        most = torch.arange(c["cols"] - 1, device=x.device)
        at = s["draft_start"][lane][:, None] + most[None, :]
        before = (most[None, :] < j[:, None]) & active[:, None]
        ids = s["draft_ids"][at.clamp(max=C - 1).long()].long()
        n = n.scatter_add(1, ids, before.to(torch.int32))
    r = s["repetition"][lane][:, None]
    y = torch.where(prompt | (n > 0), torch.where(x > 0, x / r, x * r), x)
    y = torch.where(n > 0, y - (s["frequency"][lane][:, None] * n + s["presence"][lane][:, None]), y)
    if c["bias"]:
        L, b = c["lanes"], c["bias"]
        place = torch.arange(L, device=x.device).repeat_interleave(b) * V + s["bias_ids"]
        last = torch.full((L * V,), -1, dtype=torch.int64, device=x.device)
        last.scatter_reduce_(0, place, torch.arange(L * b, device=x.device), "amax")  # of two entries the later counts
        last = last.view(L, V)
        bias = torch.where(last >= 0, s["bias_values"][last.clamp(min=0)], 0.0)
        y = y + bias[lane]
    if "mask" in s:
        m = s["mask_index"]
        allowed = _bits(s["mask"], V)[m.clamp(min=0)] | (m < 0)[:, None]
        y = torch.where(allowed, y, -math.inf)
    out = s["out"][:, :V] if col else s["out"][:, :C].t()
    out.copy_(torch.where(active[:, None], y, out.float()))
    return s["out"]


def _count(s):
    counts, seen, start, V = s["counts"], s["seen"], s["start"], s["case"]["V"]
    if s["case"]["fresh"]:
        counts.masked_fill_(s["fresh"][:, None] != 0, 0)
        seen.masked_fill_(s["fresh"][:, None] != 0, 0)
    at = torch.arange(s["ids"].numel(), device=start.device, dtype=torch.int32)
    lane = torch.searchsorted(start[1:].contiguous(), at, right=True).clamp(max=start.numel() - 2)
    real = (at < start[-1]) & (s["ids"] >= 0)
    prompt = real & (at - start[lane] < s["prompt_len"][lane])
    place = lane * V + s["ids"].clamp(min=0)
    flat = counts.view(-1)
    flat.index_add_(0, place, (real & ~prompt).to(torch.int32))
    word = flat[place]
    flat.scatter_reduce_(0, place, torch.where(prompt, word | FLAG, word), "amin")  # the flag makes a word negative
    W = seen.shape[1]
    group = s["ids"].clamp(min=0) // 32
    rows = group[:, None] * 32 + torch.arange(32, device=start.device)
    words = torch.where(rows < V, flat[lane[:, None] * V + rows.clamp(max=V - 1)], 0)
    seen.view(-1)[lane * W + group] = _pack(words != 0)[:, 0]
    return counts, seen


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
    c = s["case"]
    L, D = c["lanes"], c["drafts"]
    Ct, Cd = L * (D + 1), L * D
    dev = s["col_start"].device
    p, pid = _distribution(s["target_values"], c["temperature"], c["top_p"]), s["target_ids"]
    lane, j, active = _column_lanes(s["col_start"], Ct)
    m = (s["draft_start"].diff())[lane]
    row = (s["draft_start"][lane] + j).clamp(max=max(Cd - 1, 0)).long()
    d = s["drafts"][row]
    judged = active & (j < m)
    if Cd and not c["greedy_drafts"]:
        q = _distribution(s["draft_values"], c["temperature"], c["top_p"])[row]
        same = pid[:, :, None] == s["draft_ids"][row][:, None, :]
        q_at = (q[:, None, :] * same).sum(2)  # of each target token
        q_d = (q * (s["draft_ids"][row] == d[:, None])).sum(1)
    else:
        q_at, q_d = (pid == d[:, None]).double(), torch.ones(Ct, device=dev, dtype=torch.float64)
    p_d = (p * (pid == d[:, None])).sum(1)
    ok = judged & (s["uniforms"][0] * q_d < p_d)
    rest = (p - q_at).clamp(min=0)
    rest = torch.where((judged & (rest.sum(1) > 0))[:, None], rest, p)
    S = rest.cumsum(1)
    pick = (S <= s["uniforms"][1][:, None] * S[:, -1:]).sum(1, keepdim=True)
    last = (rest > 0).to(torch.int64).mul(torch.arange(1, p.shape[1] + 1, device=dev)).amax(1, keepdim=True) - 1
    new = pid.gather(1, torch.minimum(pick, last))[:, 0]
    # per lane: drafts up to the first refused one, then that column's token
    at = (s["col_start"][:-1, None] + torch.arange(D + 1, device=dev)).clamp(max=Ct - 1).long()
    place = torch.arange(D + 1, device=dev)
    lasting = (ok[at] & (place < s["draft_start"].diff()[:, None])).to(torch.int64).cumprod(1)
    taken = lasting.sum(1, keepdim=True)
    tokens = torch.where(place < taken, d[at], torch.where(place == taken, new[at], -1))
    s["out_tokens"].copy_(tokens)
    s["out_count"].copy_(taken[:, 0] + 1)
    return s["out_tokens"], s["out_count"]


def _plan(s):
    bs, cap = s["case"]["block"], s["capacity"]
    lens, add, held, table = s["lens"].long(), s["add"].long(), s["held"].long(), s["table"]
    L, width = table.shape
    free = s["free_count"].long()
    total = (lens + add + bs - 1) // bs
    want = (add > 0) & (total <= width)
    need = torch.where(want, (total - held).clamp(min=0), 0)
    taken = need.cumsum(0)
    ok = want & ((need == 0) | (taken <= free))
    ends = torch.where(ok, add, 0).cumsum(0)
    ok = ok & (ends <= cap)
    ends = torch.where(ok, add, 0).cumsum(0)
    col_start = torch.cat([ends.new_zeros(1), ends])
    # new blocks come from the end of the free list
    at = torch.arange(width, device=table.device)
    grown = ok[:, None] & (at >= held[:, None]) & (at < torch.maximum(total, held)[:, None])
    source = free - 1 - (taken - need - held)[:, None] - at
    table.copy_(torch.where(grown, s["free_ids"][source.clamp(0, s["free_ids"].numel() - 1)], table))
    t = torch.arange(cap, device=table.device)
    lane = torch.searchsorted(ends, t, right=True).clamp(max=L - 1)
    live = t < ends[-1]
    pos = lens[lane] + t - col_start[lane]
    slot = table[lane, (pos // bs).clamp(max=width - 1)].long() * bs + pos % bs
    return dict(table=table, held=torch.where(ok, torch.maximum(total, held), held).int(),
                free_count=free.int() - torch.where(ok & (need > 0), taken, 0).amax().int(),
                refused=((add > 0) & ~ok).sum().int()[None], col_start=col_start.int(),
                col_lane=torch.where(live, lane, -1).int(), col_pos=torch.where(live, pos, -1).int(),
                slots=torch.where(live, slot, -1))


# ------------------------------------------------------- the framework's ---

def _own(s):
    from drafter_vocab_top_amd import topk_cols as T
    c = s["case"]
    if c["op"] == "adjust":
        if "rules" not in s:  # the descriptor of the buffers that a program keeps from round to round
            more = dict(drafts=s["draft_ids"], draft_start=s["draft_start"]) if c["drafts"] else {}
            if c["bias"]:
                more.update(bias_start=s["bias_start"], bias_ids=s["bias_ids"], bias_values=s["bias_values"])
            if "mask" in s:
                more.update(mask=s["mask"], mask_index=s["mask_index"])
            s["rules"] = T.AdjustRules(c["V"], c["lanes"] * c["cols"], c["dtype"], c["layout"], s["x"].shape[1],
                                       lanes=c["lanes"], col_start=s["col_start"], counts=s["counts"], seen=s["seen"],
                                       repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"], **more)
        return s["rules"].apply(s["x"], s["out"])
    if c["op"] == "count":
        return T.count_tokens(s["counts"], s["seen"], c["V"], s["ids"], s["start"], prompt_len=s["prompt_len"],
                              fresh=s["fresh"] if c["fresh"] else None)
    if c["op"] == "verify":
        return T.verify(s["target_values"], s["target_ids"], s["col_start"], s["drafts"], s["draft_start"],
                        draft_values=s.get("draft_values"), draft_ids=s.get("draft_ids"), temperature=c["temperature"],
                        top_p=c["top_p"], seed=s["seed"], offset=s["offset"], out_tokens=s["out_tokens"],
                        out_count=s["out_count"])
    got = T.plan(s["lens"], s["add"], s["held"], s["table"], s["free_ids"], s["free_count"], c["block"], s["capacity"],
                 out=s["out"])
    return dict(got, table=s["table"])


def run(state):
    if own:
        return _own(state)
    return dict(adjust=_adjust, count=_count, verify=_verify, plan=_plan)[state["case"]["op"]](state)


# ------------------------------------------------------------------- work ---

def work(case):
    c = case
    if c["op"] == "adjust":
        e = 2 if c["dtype"] == "bf16" else 4
        share = 0.5 if c["ragged"] else 1.0
        C = max(1.0, share * c["lanes"] * c["cols"])
        # tokens drawn log-uniformly over the ids: about this many different ones among h
        distinct = lambda h: min(c["V"], h) * 0.5  # noqa: E731
        touched = C * (distinct(2 * c["hist"]) + distinct(c["bias"]))
        masks = dict(none=0.0, lane=min(c["lanes"], C), column=C)[c["mask"]]
        bits = c["V"] / 8 * (masks + c["lanes"])
        if c["in_place"]:
            changed = min(C * c["V"], touched + (C * c["V"] * (1 - c["keep"]) if masks else 0))
            moved = changed * e + touched * e
        else:
            moved = 2 * C * c["V"] * e
        return {"bytes": moved + bits + c["lanes"] * distinct(2 * c["hist"]) * 4, "flops": 4 * touched}
    if c["op"] == "count":
        ids = c["lanes"] * (0.75 * c["prompt"] + 0.5 * c["output"])
        cleared = c["fresh"] * c["lanes"] * c["V"] * (4 + 1 / 8)
        return {"bytes": 4 * ids + cleared + (1 - c["fresh"]) * ids * 16, "flops": 0}
    if c["op"] == "verify":
        e = 2 if c["dtype"] == "bf16" else 4
        drafts = c["lanes"] * 0.75 * c["drafts"]
        lists = (drafts + c["lanes"]) * c["k"] + drafts * c["kq"]
        return {"bytes": lists * (e + 4) + drafts * 8 + c["lanes"] * 16, "flops": 40 * lists + 2 * drafts * c["k"] * max(1, c["kq"])}
    tokens = c["lanes"] * c["most"] / 2
    return {"bytes": c["lanes"] * 24 + _capacity(c) * 16 + tokens / c["block"] * 12 + 16, "flops": 0}


# ------------------------------------------------------------------ exact ---

def exact(case, seed):
    """The logit rules column by column in 64 bits.  The other operators give whole numbers only."""
    if case["op"] != "adjust":
        return None
    c = case
    s = {k: v.double().cpu().numpy() if torch.is_tensor(v) and v.is_floating_point() else v.cpu().numpy() if torch.is_tensor(v) else v
         for k, v in prepare(case, seed).items()}
    V, n = c["V"], c["lanes"] * c["cols"]
    out = s["out"].copy()
    cs, ds = s["col_start"], s["draft_start"]
    for lane in range(c["lanes"]):
        word = s["counts"][lane].view(np.uint32)
        for col in range(cs[lane], cs[lane + 1]):
            times = (word & np.uint32(0x7FFFFFFF)).astype(np.int64)
            if c["drafts"]:
                first = ds[lane]
                np.add.at(times, s["draft_ids"][first:first + col - cs[lane]], 1)
            y = (s["x"][col, :V] if c["layout"] == "col" else s["x"][:, col]).copy()
            known = np.flatnonzero((word >> np.uint32(31) != 0) | (times > 0))
            rep = s["repetition"][lane]
            y[known] = np.where(y[known] > 0, y[known] / rep, y[known] * rep)
            again = np.flatnonzero(times)
            y[again] -= s["frequency"][lane] * times[again] + s["presence"][lane]
            entries = {}
            for e in range(s["bias_start"][lane], s["bias_start"][lane + 1]):
                entries[int(s["bias_ids"][e])] = s["bias_values"][e]
            for r, b in entries.items():
                y[r] += b
            if "mask" in s and s["mask_index"][col] >= 0:
                bits = np.unpackbits(s["mask"][s["mask_index"][col]].view(np.uint8), bitorder="little")[:V]
                y[bits == 0] = -np.inf
            if c["layout"] == "col":
                out[col, :V] = y
            else:
                out[:, col] = y
    assert n >= cs[-1]
    return out
