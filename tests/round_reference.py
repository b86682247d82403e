"""Plain 64-bit implementations of the steps around the top-k (numpy and
Python floats, one element or token at a time), written from the header's
definitions; and the bounds the logit rules are held to."""
import math

import numpy as np

from drafter_vocab_top_amd import workloads as W

FLAG = np.uint32(1 << 31)
# Half a step of the type relative to the value, and half its smallest subnormal.
HALF_STEP = {W.BF16: 2.0**-8, W.F32: 2.0**-24}
HALF_LEAST = {W.BF16: 2.0**-134, W.F32: 2.0**-150}


def widen(patterns, dtype):
    """The real values of storage patterns."""
    p = np.ascontiguousarray(patterns)
    f = W.f32_from_bf16_bits(p.view(np.uint16)) if dtype == W.BF16 else p.view(np.float32)
    with np.errstate(invalid="ignore"):
        return f.astype(np.float64)


def parts(start, total, lanes):
    """(begin, end) of each lane: by start (cut to [0, total]) or evenly."""
    if start is None:
        return [(l * (total // lanes), (l + 1) * (total // lanes)) for l in range(lanes)]
    cut = [min(max(int(s), 0), total) for s in start]
    return [(b, max(b, e)) for b, e in zip(cut, cut[1:])]


def allowed_rows(mask_row, V):
    return np.unpackbits(np.ascontiguousarray(mask_row).view(np.uint8), bitorder="little")[:V] != 0


def adjust(x, V, C, lanes, dtype, col_start=None, counts=None, repetition=None, presence=None, frequency=None,
           drafts=None, draft_start=None, bias_start=None, bias_ids=None, bias_values=None, mask=None,
           mask_index=None):
    """x: (C, V) storage patterns.  Returns {column: (values, touched, size)}:
    the exact values of the columns that belong to a lane, which elements a
    step changed and the sum of the magnitudes that entered each."""
    out = {}
    spans = parts(col_start, C, lanes)
    draft_spans = parts(draft_start, 0 if drafts is None else len(drafts), lanes)
    bias_spans = parts(bias_start, 0 if bias_ids is None else len(bias_ids), lanes)
    penalties = not (repetition is None and presence is None and frequency is None)
    for l, (cb, ce) in enumerate(spans):
        rep = 1.0 if repetition is None else float(repetition[l])
        pres = 0.0 if presence is None else float(presence[l])
        freq = 0.0 if frequency is None else float(frequency[l])
        word = np.zeros(V, np.uint32) if counts is None else counts[l, :V].view(np.uint32)
        prompt = (word & FLAG) != 0
        biases = {}
        for e in range(*bias_spans[l]):
            if 0 <= bias_ids[e] < V:
                biases[int(bias_ids[e])] = float(bias_values[e])
        db, de = draft_spans[l]
        for c in range(cb, ce):
            y = widen(x[c], dtype)
            size = np.abs(y)
            touched = np.zeros(V, bool)
            n = (word & ~FLAG).astype(np.int64)
            for d in range(db, min(de, db + c - cb)):
                if drafts is not None and 0 <= drafts[d] < V:
                    n[drafts[d]] += 1
            if penalties:
                for r in np.flatnonzero(prompt | (n > 0)):
                    touched[r] = True
                    y[r] = y[r] / rep if y[r] > 0 else y[r] * rep
                    size[r] = abs(y[r])
                    if n[r]:
                        y[r] -= freq * n[r] + pres
                        size[r] += abs(freq) * n[r] + abs(pres)
            for r, b in biases.items():
                touched[r] = True
                y[r] += b
                size[r] += abs(b)
            if mask is not None:
                m = c if mask_index is None else int(mask_index[c])
                if 0 <= m < mask.shape[0]:
                    no = ~allowed_rows(mask[m], V)
                    y[no] = -np.inf
                    touched[no] = True
            out[c] = (y, touched, size)
    return out


def check_adjusted(got, x, dtype, c, expect):
    """One column of results (storage patterns) against adjust()'s: untouched
    elements keep their bits; a changed one is off by half a step of its type,
    plus its binary32 rounding (2^-24) and the chain's binary64 roundings (at
    most 8 half steps of 2^-53 of the magnitudes involved)."""
    y, touched, size = expect
    st = np.uint16 if dtype == W.BF16 else np.uint32
    g, s = got.view(st), x.view(st)
    assert np.array_equal(g[~touched], s[~touched]), f"column {c}: an untouched element changed"
    v = widen(got, dtype)[touched]
    y, size = y[touched], size[touched]
    assert np.array_equal(np.isnan(v), np.isnan(y)), f"column {c}: NaN"
    fine = np.isfinite(y)
    assert np.array_equal(v[~fine & ~np.isnan(y)], y[~fine & ~np.isnan(y)]), f"column {c}: infinities"
    off = np.abs(v[fine] - y[fine])
    bound = np.abs(y[fine]) * (HALF_STEP[dtype] + 2.0**-23) + HALF_LEAST[dtype] + size[fine] * 2.0**-50
    assert (off <= bound).all(), f"column {c}: off by {np.max(off / bound)} times the bound"


def count(counts, seen, V, ids, start, prompt_len=None, fresh=None):
    """New (counts, seen) as uint32 arrays."""
    lanes = counts.shape[0]
    counts, seen = counts.view(np.uint32).copy(), seen.view(np.uint32).copy()
    for l, (b, e) in enumerate(parts(start, len(ids), lanes)):
        if fresh is not None and fresh[l]:
            counts[l, :V] = 0
            seen[l, :(V + 31) // 32] = 0
        for i in range(b, e):
            t = int(ids[i])
            if 0 <= t < V:
                if prompt_len is not None and i - b < prompt_len[l]:
                    counts[l, t] |= FLAG
                else:
                    counts[l, t] += np.uint32(1)
                seen[l, t // 32] |= np.uint32(1 << (t % 32))
    return counts, seen


def philox_uniform(seed, offset, column, stream):
    c = [offset & 0xFFFFFFFF, offset >> 32, column, stream]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return (((c[0] << 32) | c[1]) >> 11) * 2.0**-53


def running(xs):
    s, out = 0.0, []
    for x in xs:
        s += x
        out.append(s)
    return out


def distribution(values, temperature, top_p):
    k = len(values)
    if temperature == 0 or not math.isfinite(values[0]):
        return [1.0] + [0.0] * (k - 1)
    w = [math.exp((v - values[0]) / temperature) for v in values]
    s = running(w)
    n = next(m for m in range(1, k + 1) if s[m - 1] >= top_p * s[-1])
    return [w[j] / s[n - 1] if j < n else 0.0 for j in range(k)]


def verify(target_values, target_ids, spans, drafts, draft_spans, draft_values, draft_ids, temperature, top_p, seed,
           offset, max_tokens):
    """(tokens, count); values are float arrays.  Also returns the smallest
    relative distance of a decision from its border."""
    lanes = len(spans)
    tokens = np.full((lanes, max_tokens), -1, np.int32)
    count_ = np.zeros(lanes, np.int32)
    margin = 1.0
    for l, (cb, ce) in enumerate(spans):
        if ce <= cb:
            continue
        db, de = draft_spans[l]
        m = min(de - db, ce - cb - 1, max_tokens - 1)
        t = 0
        while True:
            c = cb + t
            ids = [int(i) for i in target_ids[c]]
            p = distribution([float(v) for v in target_values[c]], temperature, top_p)
            rest = p
            if t < m:
                d = int(drafts[db + t])
                if draft_values is None:
                    q_of = {d: 1.0}
                else:
                    q = distribution([float(v) for v in draft_values[db + t]], temperature, top_p)
                    q_of = {}
                    for i, v in zip(draft_ids[db + t], q):
                        q_of.setdefault(int(i), v)
                p_d = next((v for i, v in zip(ids, p) if i == d), 0.0)
                a = philox_uniform(seed, offset, c, 1) * q_of.get(d, 0.0)
                if max(a, p_d) > 0:
                    margin = min(margin, abs(a - p_d) / max(a, p_d))
                if a < p_d:
                    tokens[l, t] = d
                    t += 1
                    continue
                rest = [max(v - q_of.get(i, 0.0), 0.0) for i, v in zip(ids, p)]
                if not any(rest):
                    rest = p
            s = running(rest)
            target = philox_uniform(seed, offset, c, 2) * s[-1]
            i = next((i for i in range(len(s)) if s[i] > target), max(j for j in range(len(s)) if rest[j] > 0))
            margin = min([margin] + [abs(v - target) / s[-1] for v in s if s[-1] > 0])
            tokens[l, t] = ids[i]
            count_[l] = t + 1
            break
    return tokens, count_, margin


def plan(lens, add, held, table, free_ids, free_count, block_size, capacity):
    """The plan of a round, lane by lane, as a dict; table is a new array."""
    lanes, width = table.shape
    table = table.copy()
    free = min(max(int(free_count), 0), len(free_ids))
    out = dict(held=[], refused=0, col_start=[0], col_lane=[-1] * capacity, col_pos=[-1] * capacity,
               slots=[-1] * capacity)
    wanted = columns = taken = 0
    for l in range(lanes):
        n, a, h = max(int(lens[l]), 0), max(int(add[l]), 0), min(max(int(held[l]), 0), width)
        total = -(-(n + a) // block_size)
        ok = a > 0 and total <= width and n + a <= 2**31 - 1
        need = max(0, total - h) if ok else 0
        wanted += need
        ok = ok and (need == 0 or wanted <= free)
        columns += a if ok else 0
        ok = ok and columns <= capacity
        at = out["col_start"][-1]
        if ok:
            for b in range(need):
                table[l, h + b] = free_ids[free - 1 - taken - b]
            taken += need
            for i in range(a):
                p = n + i
                out["col_lane"][at + i] = l
                out["col_pos"][at + i] = p
                out["slots"][at + i] = int(table[l, p // block_size]) * block_size + p % block_size
            at += a
        elif a > 0:
            out["refused"] += 1
        out["col_start"].append(at)
        out["held"].append(max(total, h) if ok else h)
    out["free_count"] = free - taken
    out["table"] = table
    return out
