"""Plain 64-bit implementations of the operators of tree rounds over a paged
cache, written from their definitions.  Host arrays in, host arrays out."""
import math

import numpy as np

from round_reference import distribution

E4M3 = np.array([(-1.0 if b >> 7 else 1.0) * ((b & 7) / 8 * 2.0**-6 if (b >> 3) & 15 == 0 else (1 + (b & 7) / 8) * 2.0 ** (((b >> 3) & 15) - 7))
                 for b in range(256)])
E4M3[[0x7F, 0xFF]] = np.nan


def spans_of(col_start, lanes, C):
    """(first, end) of each lane's columns."""
    if col_start is None:
        return [(l * (C // lanes), (l + 1) * (C // lanes)) for l in range(lanes)]
    cut = [min(max(int(s), 0), C) for s in col_start]
    return [(b, max(b, e)) for b, e in zip(cut, cut[1:])]


def line(parents, b, j):
    """Column j of the lane at b and its ancestors."""
    got = [j]
    while 0 <= parents[b + j] < j:
        j = int(parents[b + j])
        got.append(j)
    return got


def tree(spans, parents, lens, mask, positions):
    """Fills mask (rows of uint32 words) and positions."""
    for l, (b, e) in enumerate(spans):
        for j in range(e - b):
            mask[b + j] = 0
            up = line(parents, b, j)
            for i in up:
                if i // 32 < mask.shape[1]:
                    mask[b + j, i // 32] |= np.uint32(1 << (i % 32))
            positions[b + j] = max(int(lens[l]), 0) + len(up) - 1


def e4m3(x):
    """Nearest e4m3 patterns of float64 values of magnitude up to 448 (ties to the even pattern)."""
    top = E4M3[:0x7F]
    i = np.searchsorted(top, np.abs(x))
    hi = np.minimum(i, 0x7E)
    lo = np.maximum(hi - 1, 0)
    a = np.abs(x)
    dl, dh = a - top[lo], top[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(top[hi] == a, hi, pick)
    return (pick | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)


def quantise(row):
    """Patterns and scale byte of one row (float64)."""
    finite = np.isfinite(row)
    a = np.abs(row[finite]).max() if finite.any() else 0.0
    e = -126
    while a > math.ldexp(448.0, e):
        e += 1
    q = e4m3(np.where(finite, np.ldexp(np.where(finite, row, 0.0), -e), 0.0))
    q[~finite] = 0x7F
    return q, e + 127


def slot_of(place, table_row, block_size, blocks):
    """(block, slot in it) of a place, or None beyond the table; block ids are cut."""
    b = place // block_size
    if b >= len(table_row):
        return None
    return min(max(int(table_row[b]), 0), blocks - 1), place % block_size


def visible(j, n, length, window, position, words):
    """Places that column j of n sees; words: its mask row, or None."""
    lo = -math.inf if not window else max(position, length) - window + 1
    got = [p for p in range(length) if p >= lo]
    for i in range(n):
        if words is None:
            seen = i <= j and (not window or j - i < window)
        else:
            seen = i // 32 < len(words) and (int(words[i // 32]) >> (i % 32)) & 1
        if seen:
            got.append(length + i)
    return got


def attend(q, keys, values, spans, lens, table, block_size, group, scale, window=0, positions=None, mask=None, out=None):
    """keys, values: (blocks, block_size, heads, dim) float64, q (C, heads * group, dim).  Returns out and, for each
    element, a bound of what roundings to bfloat16 of weights and result move it by (half a step each)."""
    blocks = keys.shape[0]
    bound = np.zeros(out.shape)
    eps = 2.0**-8  # half a bfloat16 step, relative to the value
    for l, (b, e) in enumerate(spans):
        n, length = e - b, max(int(lens[l]), 0)
        at = [slot_of(p, table[l], block_size, blocks) for p in range(min(length + n, len(table[l]) * block_size))]
        for j in range(n):
            position = length + j if positions is None else int(positions[b + j])
            places = [p for p in visible(j, n, length, window, position, None if mask is None else mask[b + j]) if p < len(at)]
            if not places:
                out[b + j] = 0
                continue
            rows = np.array([at[p] for p in places])
            for h in range(q.shape[1]):
                k = keys[rows[:, 0], rows[:, 1], h // group]
                v = values[rows[:, 0], rows[:, 1], h // group]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (k @ q[b + j, h])
                    spread = abs(scale) * (np.abs(k) @ np.abs(q[b + j, h]))
                    top = s.max()
                    if top == -math.inf:
                        out[b + j, h] = 0
                        continue
                    w = np.exp(s - top)
                    total = w.sum()
                    out[b + j, h] = (w @ v) / total
                    # a weight: one rounding to bfloat16; its score, a binary32 sum of dim products, scaled, less a
                    # maximum; the exponentials.  Then the sums over places in binary32 and the result's rounding.
                    dim = k.shape[1]
                    rel = eps + (dim + 8) * 2.0**-24 * (spread + np.abs(s)) + 2.0**-22 * np.abs(top) + 2.0**-20
                    rel = np.where(s == -math.inf, eps, rel)  # weight 0, exactly
                    moved = ((w * rel) @ np.abs(v)) / total + np.abs(out[b + j, h]) * ((w * (rel - eps)).sum() / total)
                    sums = (len(places) + 16) * 2.0**-23 * (w @ np.abs(v)) / total
                    bound[b + j, h] = moved + sums + (np.abs(out[b + j, h]) + moved + sums) * eps
    return out, bound


def verify_tree(target_values, target_ids, spans, tokens, parents, uniforms, draft_values, draft_ids, temperature, top_p,
                max_tokens):
    """(tokens, columns, count) and the smallest relative distance of a decision from its border."""
    lanes = len(spans)
    out = np.full((lanes, max_tokens), -1, np.int32)
    columns = np.full((lanes, max_tokens), -1, np.int32)
    count = np.zeros(lanes, np.int32)
    margin = 1.0
    for l, (b, e) in enumerate(spans):
        if e <= b:
            continue
        j, t = 0, 0
        while True:
            c = b + j
            columns[l, t] = j
            ids = [int(i) for i in target_ids[c]]
            p = distribution([float(v) for v in target_values[c]], temperature, top_p)
            w, W, down = list(p), 1.0, -1
            kids = [x for x in range(j + 1, e - b) if parents[b + x] == j] if t + 1 < max_tokens else []
            for x in kids:
                d = int(tokens[b + x])
                if draft_values is None:
                    q_of = {d: 1.0}
                else:
                    q_of = {}
                    for i, v in zip(draft_ids[c], distribution([float(v) for v in draft_values[c]], temperature, top_p)):
                        q_of.setdefault(int(i), v)
                w_d = next((v for i, v in zip(ids, w) if i == d), 0.0)
                a = float(uniforms[b + x, 0]) * q_of.get(d, 0.0) * W
                if max(a, w_d) > 0:
                    margin = min(margin, abs(a - w_d) / max(a, w_d))
                if a < w_d:
                    down = x
                    break
                rest = [max(v - W * q_of.get(i, 0.0), 0.0) for i, v in zip(ids, w)]
                w, W = (rest, sum(rest)) if sum(rest) > 0 else (list(p), 1.0)
            if down >= 0:
                out[l, t] = tokens[b + down]
                j, t = down, t + 1
                continue
            s, run = 0.0, []
            for v in w:
                s += v
                run.append(s)
            target = float(uniforms[c, 1]) * s
            i = next((i for i in range(len(run)) if w[i] > 0 and run[i] > target), max(i for i in range(len(w)) if w[i] > 0))
            margin = min([margin] + [abs(v - target) / s for v in run])
            out[l, t] = ids[i]
            count[l] = t + 1
            break
    return out, columns, count, margin


def move(rows, lens, table, columns, block_size):
    """rows: (layers, blocks, block_size, ..), changed in place."""
    for l in range(len(lens)):
        length = max(int(lens[l]), 0)
        for i, c in enumerate(columns[l]):
            if c <= i:
                continue
            where = []
            for p in (length + int(c), length + i):
                b = p // block_size
                if b < table.shape[1] and 0 <= table[l, b] < rows.shape[1]:
                    where.append((table[l, b], p % block_size))
            if len(where) == 2:
                (sb, sr), (db, dr) = where
                rows[:, db, dr] = rows[:, sb, sr]
