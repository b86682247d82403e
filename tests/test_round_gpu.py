"""GPU tests of the steps around the top-k, each against the plain 64-bit
implementation in round_reference.py, and of a whole round as it is used."""
import numpy as np
import pytest

import round_reference as R
from drafter_vocab_top_amd import workloads as W

pytestmark = pytest.mark.gpu

STORAGE = {W.BF16: np.uint16, W.F32: np.uint32}
SIGNED = {W.BF16: np.int16, W.F32: np.int32}
SENTINEL = {W.BF16: 0x1234, W.F32: 0x12345678}


def dev(torch, a, offset=0):
    """A host array on the GPU, `offset` elements into its allocation."""
    a = np.ascontiguousarray(a)
    if a.dtype in (np.uint16, np.uint32):
        a = a.view(np.int16 if a.dtype == np.uint16 else np.int32)
    t = torch.from_numpy(a)
    buf = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    buf[offset:].copy_(t.reshape(-1))
    return buf[offset:].reshape(t.shape)


def host(t, dtype=None):
    a = t.cpu().numpy()
    return a if dtype is None else a.view(STORAGE[dtype])


def split(rng, lanes, most, empty=0.2):
    """Starts of lanes with 0 to `most` entries each."""
    n = rng.integers(1, most + 1, lanes) * (rng.random(lanes) >= empty)
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def zipf(rng, n, V):
    return np.minimum((V ** rng.random(n)).astype(np.int64) - 1, V - 1).clip(0).astype(np.int32)


def packed(rows_allowed):
    n, V = rows_allowed.shape
    b = np.zeros((n, (V + 31) // 32 * 32), np.uint8)
    b[:, :V] = rows_allowed
    # bits past the last row are set: they must not matter
    b[:, V:] = 1
    return np.packbits(b, axis=1, bitorder="little").view(np.uint32)


class Case:
    """A random matrix with every rule that is asked for."""

    def __init__(self, seed, V, lanes, most, dtype, layout, pad=0, out_pad=0, ragged=True, hist=0, penalties="all",
                 drafts=False, bias=0, mask=None, special=False, gap=0, empty=0.2):
        rng = np.random.default_rng(seed)
        self.V, self.lanes, self.dtype, self.layout = V, lanes, dtype, layout
        self.col_start = split(rng, lanes, most, empty) if ragged else None
        used = int(self.col_start[-1]) if ragged else lanes * most
        self.C = max(used, 1) + (gap if ragged else 0)  # the last `gap` columns are nobody's
        C = self.C
        self.ld = (V if layout == W.COL else C) + pad
        self.out_ld = (V if layout == W.COL else C) + out_pad
        x = (rng.standard_normal((C, V)) * 4).astype(np.float32)
        if special:
            for v in (np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-40, -1e-40, 3e38, -3e38):
                x[rng.random((C, V)) < 0.04] = v
        if dtype == W.BF16:
            nan = np.isnan(x)
            bits = W.bf16_bits_from_f32(np.where(nan, 0, x))
            bits[nan] = rng.choice([0x7FC0, 0xFFC1, 0x7F81, 0xFFFF], nan.sum())
        else:
            bits = x.view(np.uint32).copy()
            nan = np.isnan(x)
            bits[nan] = rng.choice([0x7FC00000, 0xFFC00001, 0x7F800001, 0xFFFFFFFF], nan.sum())
        self.x = bits
        self.rules = r = {}
        if self.col_start is not None:
            r["col_start"] = self.col_start
        if hist:
            counts = np.zeros((lanes, V + 3), np.uint32)
            for l in range(lanes):
                np.add.at(counts[l], zipf(rng, hist, V), 1)
                counts[l, zipf(rng, hist, V)] |= R.FLAG
            counts[:, V:] = 7  # beyond V: not a row
            seen = np.zeros((lanes, (V + 31) // 32 + 1), np.uint32)
            seen[:, :-1] = packed(counts[:, :V] != 0)
            r["counts"], r["seen"] = counts.view(np.int32), seen.view(np.int32)
        if penalties in ("all", "repetition"):
            r["repetition"] = (0.6 + rng.random(lanes)).astype(np.float32)
        if penalties in ("all", "presence"):
            r["presence"] = rng.standard_normal(lanes).astype(np.float32)
        if penalties in ("all", "frequency"):
            r["frequency"] = rng.random(lanes).astype(np.float32)
        if drafts:
            if ragged:
                r["draft_start"] = np.concatenate([[0], np.cumsum(np.maximum(np.diff(self.col_start) - 1, 0))]).astype(np.int32)
            # the same token several times, ids that are none
            d = rng.choice(np.concatenate([zipf(rng, 4, V), [V - 1, -1, V]]), max(1, lanes * max(most - 1, 1)))
            if not ragged:
                d = d[:lanes * (most - 1)]
            if len(d):
                r["drafts"] = d.astype(np.int32)
        if bias:
            r["bias_start"] = split(rng, lanes, bias)
            n = max(int(r["bias_start"][-1]), 1)
            ids = np.concatenate([zipf(rng, n, V), [0, V - 1, 0, -1, V]])
            r["bias_ids"] = rng.permutation(ids)[:n].astype(np.int32)
            r["bias_values"] = (rng.standard_normal(n) * 5).astype(np.float32)
        if mask:
            n = dict(column=C, lane=lanes, shared=2)[mask]
            keep = rng.choice([0.0, 0.03, 0.5, 0.97, 1.0], (n, 1))
            words = packed(rng.random((n, V)) < keep)
            r["mask"] = np.concatenate([words, np.zeros((n, 2), np.uint32)], 1).view(np.int32)
            if mask != "column":
                r["mask_index"] = rng.integers(-1, n + 1, C).astype(np.int32)  # -1 and n: no mask

    def matrix(self, ld, patterns):
        """The (C, V) patterns in the layout, the padding filled."""
        shape = (self.C, ld) if self.layout == W.COL else (self.V, ld)
        m = np.full(shape, SENTINEL[self.dtype], STORAGE[self.dtype])
        if patterns is not None:
            if self.layout == W.COL:
                m[:, :self.V] = patterns
            else:
                m[:, :self.C] = patterns.T
        return m

    def columns(self, m):
        return m[:, :self.V] if self.layout == W.COL else np.ascontiguousarray(m[:, :self.C].T)

    def device_rules(self, gpu, out_ld=None):
        torch, T = gpu
        return T.AdjustRules(self.V, self.C, self.dtype, self.layout, self.ld, out_ld if out_ld else self.out_ld,
                             lanes=self.lanes, **{k: dev(torch, v) for k, v in self.rules.items()})

    def expected(self):
        r = {k: (v.view(np.uint32) if k in ("counts", "mask") else v) for k, v in self.rules.items() if k != "seen"}
        return R.adjust(self.x, self.V, self.C, self.lanes, self.dtype, **r)

    def check(self, got, before):
        """got, before: whole matrices (patterns) after and before the call."""
        g, b = self.columns(got), self.columns(before)
        expect = self.expected()
        for c in range(self.C):
            if c in expect:
                R.check_adjusted(g[c].copy(), self.x[c], self.dtype, c, expect[c])
            else:
                assert np.array_equal(g[c], b[c]), f"column {c} is nobody's and was written"
        pad = got[:, self.V:] if self.layout == W.COL else got[:, self.C:]
        assert (pad == SENTINEL[self.dtype]).all(), "the padding was written"


def run_adjust(gpu, case, in_place, offset=0):
    torch, T = gpu
    x = case.matrix(case.ld, case.x)
    dx = dev(torch, x, offset)
    if in_place:
        out, before = dx, x
    else:
        before = case.matrix(case.out_ld, None)
        out = dev(torch, before, offset)
    case.device_rules(gpu, case.ld if in_place else None).apply(dx, out)
    torch.cuda.synchronize()
    case.check(host(out, case.dtype), before)
    if not in_place:
        assert np.array_equal(host(dx, case.dtype), x), "the logits were written"


ADJUST = [
    # V, lanes, most columns of a lane, other settings
    (1, 1, 1, dict(ragged=False, hist=2, mask="column")),
    (1, 3, 2, dict(hist=1, drafts=True, bias=2, mask="lane")),
    (5, 2, 3, dict(hist=3, drafts=True, bias=3, mask="shared", special=True)),
    (31, 4, 5, dict(hist=9, bias=4, mask="column", pad=1, out_pad=2)),
    (32, 3, 4, dict(hist=9, drafts=True, mask="lane", gap=3)),
    (33, 5, 9, dict(hist=20, drafts=True, bias=5, mask="column", pad=7, gap=1)),
    (255, 1, 8, dict(ragged=False, hist=60, drafts=True)),
    (257, 70, 2, dict(hist=10, penalties="repetition", mask="lane")),
    (2047, 2, 16, dict(hist=500, drafts=True, bias=300, special=True, mask="column")),
    (8191, 3, 7, dict(hist=200, penalties="presence", bias=40)),
    (8192, 2, 7, dict(hist=2000, penalties="frequency", drafts=True, mask="shared")),
    (8193, 2, 7, dict(hist=1, bias=1, mask="column", pad=3, out_pad=1, gap=2)),
    (20011, 3, 8, dict(hist=1500, drafts=True, bias=100, mask="lane", special=True, pad=5)),
    (40009, 1, 8, dict(ragged=False, drafts=True)),
    (40009, 2, 3, dict(penalties=None, bias=30, mask="column")),
    (30001, 2, 2, dict(penalties=None, mask="column", out_pad=6)),
    (9001, 300, 1, dict(hist=5, mask="shared")),
    (1021, 6, 100, dict(hist=50, drafts=True, bias=9, mask="lane", gap=11)),
    (1532, 41, 9, dict(hist=6000, bias=20, drafts=True)),      # nearly every row touched
    (4097, 3, 5, dict(hist=9000, bias=60, mask="column", gap=3)),
]


@pytest.mark.parametrize("layout", [W.COL, W.ROW])
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("n", range(len(ADJUST)))
def test_adjust(gpu, n, dtype, layout):
    V, lanes, most, more = ADJUST[n]
    print(f"[round] adjust V={V} lanes={lanes} {dtype} {layout} {more}", flush=True)
    case = Case(100 + n, V, lanes, most, dtype, layout, **more)
    for offset in (0, 1):
        run_adjust(gpu, case, False, offset)
        if case.out_ld >= case.ld:
            run_adjust(gpu, case, True, offset)


@pytest.mark.parametrize("layout", [W.COL, W.ROW])
def test_adjust_a_matrix_larger_than_the_caches(gpu, layout):
    """More than 256 MB read and written, with lanes and columns left over."""
    print(f"[round] adjust, large {layout}", flush=True)
    case = Case(77, 56001, 300, 8, W.BF16, layout, hist=60, drafts=True, bias=5, mask="lane", gap=2, out_pad=3, empty=0.02)
    assert 2 * 2 * case.V * case.C > 256 << 20
    run_adjust(gpu, case, False)


@pytest.mark.parametrize("ragged", [True, False])
def test_adjust_in_place_by_few_workgroups(gpu, ragged):
    """Columns in place that share one list of touched rows, several after each other."""
    print(f"[round] adjust, 150 lanes of 13 columns in place, ragged={ragged}", flush=True)
    run_adjust(gpu, Case(79, 4097, 150, 13, W.F32, W.COL, hist=40, drafts=True, bias=4, ragged=ragged, empty=0.02), True)


@pytest.mark.parametrize("layout", [W.COL, W.ROW])
def test_adjust_more_lanes_than_a_grid_is_high(gpu, layout):
    print(f"[round] adjust, 66,000 lanes {layout}", flush=True)
    run_adjust(gpu, Case(78, 40, 66000, 1, W.F32, layout, hist=3, bias=1, mask="shared", gap=1), False)


@pytest.mark.parametrize("n", [0, 1, 2])
@pytest.mark.parametrize("layout", [W.COL, W.ROW])
def test_adjust_columns_on_cache_lines(gpu, layout, n):
    """Columns (or rows) that start on cache lines, at sizes on both sides of
    a thread's rows and a workgroup's tile."""
    V, lanes, most = ((2048 * 3 + 64, 3, 8), (64 * 33, 5, 32), (262144, 8, 4))[n]
    dtype = (W.BF16, W.F32, W.BF16)[n]
    print(f"[round] adjust, aligned V={V} {layout}", flush=True)
    run_adjust(gpu, Case(300 + n, V, lanes, most, dtype, layout, ragged=n == 1, hist=700, drafts=True, bias=40, mask="column"), False)


@pytest.mark.parametrize("layout", [W.COL, W.ROW])
def test_adjust_offsets_past_32_bits(gpu, layout):
    """Elements, history words and mask words more than 2^32 bytes into their
    arrays."""
    torch, T = gpu
    V, lanes, ld = 70, 3, 2**31 // 2 + 8
    rng = np.random.default_rng(4)
    rows, width = (lanes, V) if layout == W.COL else (V, lanes)
    if layout == W.ROW:
        ld = 2**32 // 2 // (V - 1) + 1   # the last row begins past 2^32 bytes
    x = W.bf16_bits_from_f32((rng.standard_normal((lanes, V)) * 4).astype(np.float32))
    m = x if layout == W.COL else np.ascontiguousarray(x.T)
    word = rng.integers(0, 3, (lanes, V)).astype(np.int32)
    mask = packed(rng.random((lanes, V)) < 0.7)
    wide = 2**30 + 4  # words: 4 GiB and more to a row
    print(f"[round] adjust, offsets past 32 bits {layout}", flush=True)

    def spread(a, columns, dtype):
        t = torch.zeros((a.shape[0], columns), dtype=dtype, device="cuda")
        t[:, :a.shape[1]] = torch.from_numpy(a.view(np.int16 if a.itemsize == 2 else np.int32)).cuda()
        return t
    dx = spread(m, ld, torch.int16)
    rules = dict(repetition=np.float32([1.5, 0.5, 2.0]), presence=np.float32([0.1, 0.2, 0.3]))
    seen = packed(word != 0)
    r = T.AdjustRules(V, lanes, W.BF16, layout, ld, lanes=lanes, counts=spread(word, wide, torch.int32),
                      seen=dev(torch, seen), mask=spread(mask, wide, torch.int32),
                      **{k: dev(torch, v) for k, v in rules.items()})
    r.apply(dx, dx)
    torch.cuda.synchronize()
    got = host(dx[:, :width].contiguous(), W.BF16)
    assert int((dx[:, width:] != 0).sum()) == 0
    got = got if layout == W.COL else np.ascontiguousarray(got.T)
    expect = R.adjust(x, V, lanes, lanes, W.BF16, counts=word, mask=mask, **rules)
    for c in range(lanes):
        R.check_adjusted(got[c].copy(), x[c], W.BF16, c, expect[c])


def test_adjust_with_no_rule_copies(gpu):
    torch, T = gpu
    case = Case(7, 5003, 2, 3, W.BF16, W.COL, penalties=None, special=True)
    run_adjust(gpu, case, False)
    run_adjust(gpu, case, True)
    # histories without a penalty change nothing, NaN patterns included
    case = Case(8, 5003, 2, 3, W.BF16, W.COL, hist=500, penalties=None, special=True)
    run_adjust(gpu, case, False)


@pytest.mark.parametrize("layout", [W.COL, W.ROW])
def test_adjust_offsets_outside_their_arrays_are_cut(gpu, layout):
    """col_start, draft_start and bias_start that run past their arrays, run
    backwards or are negative are cut (checked on the host first)."""
    torch, T = gpu
    case = Case(9, 3001, 4, 3, W.BF16, layout, hist=100, drafts=True, bias=20, mask="column")
    C = case.C
    case.col_start = case.rules["col_start"] = np.array([-5, 1, 2, 1, 2**31 - 1], np.int32)  # the third: none
    case.rules["draft_start"] = np.array([-7, 2**31 - 1, -2**31, 1, 5], np.int32)
    case.rules["bias_start"] = np.array([2**31 - 1, 0, -3, 2, 2**31 - 1], np.int32)
    assert R.parts(case.col_start, C, 4) == [(0, min(1, C)), (min(1, C), min(2, C)), (min(2, C), min(2, C)), (min(1, C), C)]
    case.col_start[3] = 2  # lanes must not overlap
    print("[round] adjust, cut offsets", flush=True)
    run_adjust(gpu, case, False)


def test_adjust_at_the_largest_values(gpu):
    """Results past the largest finite value become infinite; a bias on an
    infinity leaves it; a penalty on -Inf keeps -Inf."""
    torch, T = gpu
    V = 64
    x = np.full((1, V), 3.0e38, np.float32)
    x[0, 1], x[0, 2], x[0, 3] = -3.0e38, np.inf, -np.inf
    counts, seen = np.zeros((1, V), np.int32), np.zeros((1, 2), np.int32)
    counts[0, :4], seen[0, 0] = 2, 15
    r = T.AdjustRules(V, 1, "f32", lanes=1, counts=dev(torch, counts), seen=dev(torch, seen),
                      repetition=dev(torch, np.float32([2.0])), presence=dev(torch, np.float32([-1e38])))
    y = r.apply(dev(torch, x)).cpu().numpy()[0]
    assert y[1] == -np.inf and y[2] == np.inf and y[3] == -np.inf
    assert y[0] == np.float32(np.float64(np.float32(3.0e38)) / 2 + np.float64(np.float32(1e38)))
    assert (y[4:] == x[0, 4:]).all()


def test_adjust_in_place_more_lanes_than_a_launch_takes(gpu):
    """2^20 lanes of five tiles of rows each; three of them own a column."""
    torch, T = gpu
    V, lanes, C = 16411, 1 << 20, 3
    owners = [0, 838865, lanes - 1]
    rng = np.random.default_rng(61)
    col_start, bias_start = np.zeros(lanes + 1, np.int32), np.zeros(lanes + 1, np.int32)
    for l in owners:
        col_start[l + 1:] += 1
        bias_start[l + 1:] += 4
    x = rng.integers(-99, 99, (V, C)).astype(np.float32)
    ids = np.stack([rng.choice(V, 4, False) for _ in owners]).astype(np.int32)
    values = rng.integers(1, 9, ids.shape).astype(np.float32)
    allowed = rng.random((C, V)) < 0.7
    expect = x.copy()
    for c in range(C):
        expect[ids[c], c] += values[c]  # small whole numbers: exact
    expect[~allowed.T] = -np.inf
    print(f"[round] adjust in place, lanes={lanes}", flush=True)
    r = T.AdjustRules(V, C, "f32", "row", lanes=lanes, col_start=dev(torch, col_start), bias_start=dev(torch, bias_start),
                      bias_ids=dev(torch, ids.ravel()), bias_values=dev(torch, values.ravel()),
                      mask=dev(torch, packed(allowed).view(np.int32)))
    t = dev(torch, x)
    r.apply(t, t)
    torch.cuda.synchronize()
    assert np.array_equal(host(t), expect)


# ------------------------------------------------------------------ count ---

COUNT = [
    # V, lanes, most tokens of a lane, prompts, fresh
    (1, 1, 1, False, False),
    (33, 3, 40, True, True),
    (1000, 1, 700, True, False),
    (1000, 64, 8, False, False),
    (20011, 5, 3000, True, True),
    (40001, 2, 20000, True, True),
    (131072, 3, 9000, False, True),
    (257, 300, 5, True, True),
    (35, 66000, 2, True, True),
    (35, 66000, 2, True, False),
    (30281, 5, 3400, True, False),
    (130001, 1, 4000, True, False),
    (1183, 13, 600, True, False),
    (50003, 90, 60, True, False),
]


@pytest.mark.parametrize("n", range(len(COUNT)))
def test_count(gpu, n):
    torch, T = gpu
    V, lanes, most, prompts, fresh = COUNT[n]
    rng = np.random.default_rng(n)
    start = split(rng, lanes, most)
    ids = zipf(rng, int(start[-1]) + 5, V)
    bad = rng.random(len(ids)) < 0.05
    ids[bad] = rng.choice([-1, V, 2**31 - 1, -2**31], bad.sum())
    counts = np.zeros((lanes, V + 2), np.int32)
    counts[:, V:] = 9
    counts[np.arange(lanes).repeat(50), zipf(rng, 50 * lanes, V)] = rng.integers(1, 5, 50 * lanes)
    seen = np.zeros((lanes, (V + 31) // 32 + 1), np.uint32)
    seen[:, :-1] = packed(counts[:, :V] != 0)
    if V % 32:
        seen[:, -2] &= np.uint32((1 << V % 32) - 1)
    seen[:, -1] = 77
    prompt_len = rng.integers(-1, most + 2, lanes).astype(np.int32) if prompts else None
    new = rng.integers(0, 2, lanes).astype(np.int32) if fresh else None
    dc, ds = dev(torch, counts), dev(torch, seen)
    more = dict(prompt_len=None if prompt_len is None else dev(torch, prompt_len),
                fresh=None if new is None else dev(torch, new))
    print(f"[round] count V={V} lanes={lanes} tokens={len(ids)}", flush=True)
    for step in range(2):  # the second call adds to what the first left
        T.count_tokens(dc, ds, V, dev(torch, ids), dev(torch, start), **more)
        counts, seen = R.count(counts, seen, V, ids, start, prompt_len, new)
        torch.cuda.synchronize()
        assert np.array_equal(host(dc).view(np.uint32), counts), step
        assert np.array_equal(host(ds).view(np.uint32), seen), step


def test_count_evenly_and_nothing(gpu):
    torch, T = gpu
    V, lanes = 501, 3
    counts, seen = T.history(V, lanes)
    ids = np.arange(12, dtype=np.int32) % 5
    T.count_tokens(counts, seen, V, dev(torch, ids))
    c, s = R.count(np.zeros((lanes, V), np.int32), np.zeros((lanes, 16), np.uint32), V, ids, None)
    assert np.array_equal(host(counts).view(np.uint32), c) and np.array_equal(host(seen).view(np.uint32), s)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    T.count_tokens(counts, seen, V, none)
    assert np.array_equal(host(counts).view(np.uint32), c)
    fresh = dev(torch, np.int32([0, 1, 0]))
    T.count_tokens(counts, seen, V, none, fresh=fresh)
    c[1], s[1] = 0, 0
    assert np.array_equal(host(counts).view(np.uint32), c) and np.array_equal(host(seen).view(np.uint32), s)
    # starts that are negative, past the ids or backwards are cut
    start = np.array([-3, 5, 4, 2**31 - 1], np.int32)
    T.count_tokens(counts, seen, V, dev(torch, ids), dev(torch, np.array([0, 5, 5, 2**31 - 1], np.int32)))
    c, s = R.count(c, s, V, ids, np.array([0, 5, 5, 12]))
    assert np.array_equal(host(counts).view(np.uint32), c) and np.array_equal(host(seen).view(np.uint32), s)
    assert R.parts(start, 12, 3)[2] == (4, 12)


# ----------------------------------------------------------------- verify ---

def lists(rng, n, k, dtype, universe):
    v = -np.sort(-rng.standard_normal((n, k)) * 2, axis=1).astype(np.float32)
    if dtype == W.BF16:
        bits = W.bf16_bits_from_f32(v)
        return bits, W.f32_from_bf16_bits(bits), np.argsort(rng.random((n, universe)), 1)[:, :k].astype(np.int32)
    return v.view(np.uint32), v, np.argsort(rng.random((n, universe)), 1)[:, :k].astype(np.int32)


VERIFY = [
    # lanes, most drafts, k, kq (0: greedy drafts), temperature, top_p
    (1, 7, 20, 20, 1.0, 0.95),
    (1, 0, 1, 1, 1.0, 1.0),
    (5, 1, 1, 1, 1.0, 0.5),
    (40, 7, 20, 20, 1.0, 0.95),
    (40, 7, 20, 0, 1.0, 0.95),
    (30, 15, 64, 64, 0.7, 0.9),
    (30, 15, 64, 64, 0.0, 0.9),
    (9, 40, 33, 5, 1.6, 1.0),
    (9, 40, 5, 33, 0.05, 0.3),
    (200, 3, 8, 0, 0.0, 1.0),
]


@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
@pytest.mark.parametrize("n", range(len(VERIFY)))
def test_verify(gpu, n, dtype):
    torch, T = gpu
    lanes, most, k, kq, temperature, top_p = VERIFY[n]
    rng = np.random.default_rng(50 + n)
    have = rng.integers(0, most + 1, lanes) if most else np.zeros(lanes, int)
    cols = have + 1
    cols[rng.random(lanes) < 0.1] = 0  # lanes that sit the round out
    cs = np.concatenate([[0], np.cumsum(cols)]).astype(np.int32)
    ds = np.concatenate([[0], np.cumsum(have)]).astype(np.int32)
    C, D = int(cs[-1]) + 2, int(ds[-1])
    tb, tv, ti = lists(rng, C, k, dtype, 70)
    for c in range(0, C, 17):  # tops that are not finite, lists that end in -Inf
        tv[c, 0 if c % 2 else slice(1, None)] = np.inf if c % 2 else -np.inf
    tb = W.bf16_bits_from_f32(tv) if dtype == W.BF16 else tv.view(np.uint32)
    if kq:
        qb, qv, qi = lists(rng, max(D, 1), kq, dtype, 70)
        drafts = qi[np.arange(max(D, 1)), rng.integers(0, kq, max(D, 1))]
        # many lists equal to the target's, as good drafters' are
        for l in range(lanes):
            for j in range(min(have[l], max(cols[l] - 1, 0))):
                if rng.random() < 0.6 and kq == k:
                    qb[ds[l] + j], qv[ds[l] + j], qi[ds[l] + j] = tb[cs[l] + j], tv[cs[l] + j], ti[cs[l] + j]
                    drafts[ds[l] + j] = ti[cs[l] + j, int(rng.random() ** 3 * k)]
        args = dict(draft_values=dev(torch, qb), draft_ids=dev(torch, qi))
    else:
        qv = qi = None
        drafts = rng.integers(0, 70, max(D, 1)).astype(np.int32)
        for l in range(lanes):
            for j in range(min(have[l], max(cols[l] - 1, 0))):
                if rng.random() < 0.8:
                    drafts[ds[l] + j] = ti[cs[l] + j, 0]
        args = {}
    for rep, limit in enumerate((most + 1, 3)):
        seed, offset = 2**40 + n, 2**33 + rep
        tokens = torch.full((lanes, limit), 99, dtype=torch.int32, device="cuda")
        print(f"[round] verify {VERIFY[n]} {dtype}", flush=True)
        got, cnt = T.verify(dev(torch, tb), dev(torch, ti), dev(torch, cs), dev(torch, drafts), dev(torch, ds),
                            temperature=temperature, top_p=top_p, seed=seed, offset=offset, out_tokens=tokens, **args)
        torch.cuda.synchronize()
        want, count, margin = R.verify(tv, ti, R.parts(cs, C, lanes), drafts, R.parts(ds, len(drafts), lanes), qv, qi,
                                       temperature, top_p, seed, offset, limit)
        # exp differs by a few 2^-52 between the two sides and 64 terms are summed: 2^-40 is far from both,
        # except where both sides are equal by construction
        assert temperature == 0 or margin > 2.0**-40
        assert np.array_equal(host(cnt), count) and np.array_equal(host(got), want)


@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_verify_with_repeated_ids(gpu, dtype):
    """Lists in which ids occur several times (rows mapped to the same token):
    the first entry of an id counts."""
    torch, T = gpu
    rng = np.random.default_rng(21)
    lanes, most, k = 50, 6, 12
    have = rng.integers(0, most + 1, lanes)
    cs = np.concatenate([[0], np.cumsum(have + 1)]).astype(np.int32)
    ds = np.concatenate([[0], np.cumsum(have)]).astype(np.int32)
    C, D = int(cs[-1]), max(int(ds[-1]), 1)
    tb, tv, _ = lists(rng, C, k, dtype, 70)
    qb, qv, _ = lists(rng, D, k, dtype, 70)
    ti, qi = rng.integers(0, 5, (C, k)).astype(np.int32), rng.integers(0, 6, (D, k)).astype(np.int32)
    drafts = rng.integers(0, 6, D).astype(np.int32)
    for sampled in (True, False):
        args = dict(draft_values=dev(torch, qb), draft_ids=dev(torch, qi)) if sampled else {}
        got, cnt = T.verify(dev(torch, tb), dev(torch, ti), dev(torch, cs), dev(torch, drafts), dev(torch, ds), top_p=0.9,
                            seed=-3, offset=1, max_tokens=most + 1, **args)
        want, count, margin = R.verify(tv, ti, R.parts(cs, C, lanes), drafts, R.parts(ds, D, lanes), qv if sampled else None,
                                       qi if sampled else None, 1.0, 0.9, 2**64 - 3, 1, most + 1)
        assert margin > 2.0**-40
        assert np.array_equal(host(cnt), count) and np.array_equal(host(got), want)


def test_binding_refuses_on_the_gpu(gpu):
    """What the binding and the library refuse when the tensors are on the GPU."""
    torch, T = gpu
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.zeros((14, 100), dtype=torch.bfloat16, device="cuda")
    rules = T.AdjustRules(100, 14, lanes=2)
    for args in ((x[:13],), (x.float(),), (x, x[:13]), (x, torch.zeros(28, 50, dtype=torch.bfloat16, device="cuda").t()),
                 (x.cpu(),), (x, x.cpu()), (x.half(),), (x, x.half())):
        with pytest.raises((ValueError, TypeError)):
            rules.apply(*args)
    with pytest.raises(ValueError):
        T.AdjustRules(100, 14, lanes=2, out_ld=101).apply(x)      # out is needed
    with pytest.raises(T.TopkError):
        T.AdjustRules(100, 14, lanes=3).apply(x)                  # lanes do not divide the columns
    with pytest.raises(T.TopkError):
        T.AdjustRules(100, 14, lanes=2, counts=i32(2, 100)).apply(x)   # counts without seen
    with pytest.raises(T.TopkError):
        T.count_tokens(i32(2, 100), i32(2, 4), 101, i32(6))       # more rows than counts has
    with pytest.raises(T.TopkError):
        T.count_tokens(i32(2, 100), i32(2, 4), 100, i32(7))       # lanes do not divide the tokens
    with pytest.raises(ValueError):
        T.count_tokens(i32(2, 100), i32(2, 4), 100, i32(6).long())
    values, ids = torch.zeros((16, 8), device="cuda"), i32(16, 8)
    with pytest.raises(T.TopkError):
        T.verify(values, ids, None, i32(14), None, lanes=2, temperature=-1.0)
    with pytest.raises(ValueError):
        T.verify(torch.zeros((16, 65), device="cuda"), i32(16, 65), None, i32(14), None, lanes=2)
    with pytest.raises(ValueError):
        T.verify(values, ids, None, i32(14), None, draft_values=torch.zeros((14, 8), device="cuda"), lanes=2)
    with pytest.raises(ValueError):
        T.verify(values.half(), ids, None, i32(14), None, draft_values=torch.zeros((14, 8), device="cuda"),
                 draft_ids=i32(14, 8), lanes=2)
    with pytest.raises(ValueError):
        T.verify(values.half(), ids, None, i32(14), None, lanes=2)      # float16 is not bfloat16
    with pytest.raises(ValueError):
        T.plan(i32(2), i32(2), i32(2), i32(2, 4), i32(4), i32(1), 0, 8)
    out = T.plan(i32(2), i32(2), i32(2), i32(2, 4), i32(4), i32(1), 16, 8)
    with pytest.raises(T.TopkError):
        T.plan(i32(2), i32(2), out["held"], i32(2, 4), i32(4), i32(1), 16, 8, out=out)   # written over its input
    with pytest.raises(ValueError):
        T.plan(i32(2), i32(2), i32(2), i32(2, 4), i32(4), i32(1), 16, 9, out=out)        # outputs too short
    torch.cuda.synchronize()


def test_verify_keeps_the_targets_distribution(gpu):
    """The committed first token of many lanes is distributed as the target's
    nucleus, whatever the drafter's list: chi-square over 4 tokens."""
    torch, T = gpu
    lanes, k = 20000, 4
    tv = np.tile(np.float32([1.0, 0.5, 0.2, -0.3]), (2 * lanes, 1))
    ti = np.tile(np.int32([5, 6, 7, 8]), (2 * lanes, 1))
    qv = np.tile(np.float32([1.5, 0.9, 0.1, -1.0]), (lanes, 1))
    qi = np.tile(np.int32([8, 5, 9, 6]), (lanes, 1))
    q = np.array(R.distribution([float(v) for v in qv[0]], 1.0, 1.0))
    rng = np.random.default_rng(3)
    drafts = qi[0][np.searchsorted(np.cumsum(q), rng.random(lanes)).clip(max=3)].astype(np.int32)
    got, cnt = T.verify(dev(torch, tv), dev(torch, ti), None, dev(torch, drafts), None, dev(torch, qv), dev(torch, qi),
                        top_p=1.0, seed=5, offset=6, lanes=lanes, max_tokens=2)
    p = np.array(R.distribution([float(v) for v in tv[0]], 1.0, 1.0))
    first = host(got)[:, 0]
    seen = np.array([(first == t).sum() for t in ti[0]])
    assert seen.sum() == lanes
    chi = ((seen - p * lanes) ** 2 / (p * lanes)).sum()
    assert chi < 21.1  # 3 degrees of freedom: exceeded with probability 1e-4
    rate = np.minimum(p, [q[1], q[3], 0, q[0]]).sum()  # accepted with probability sum of min(p, q)
    assert abs((host(cnt) == 2).mean() - rate) < 5 * np.sqrt(rate * (1 - rate) / lanes)


# ------------------------------------------------------------------- plan ---

def plan_inputs(rng, lanes, most, context, bs, width_short=0, spare=1.0):
    lens = rng.integers(0, context + 1, lanes).astype(np.int32)
    add = (rng.integers(0, most + 1, lanes) - (rng.random(lanes) < 0.1) * most).astype(np.int32)
    held = (-(-lens // bs) + (rng.random(lanes) < 0.3) * rng.integers(0, 4, lanes)).astype(np.int32)
    width = max(1, -(-(context + most) // bs) + 2 - width_short)
    need = np.maximum(-(-(lens + np.maximum(add, 0)) // bs) - held, 0)
    free = int(need.sum() * spare)
    ids = rng.permutation(int(held.sum()) + free + 7).astype(np.int32)
    table = np.full((lanes, width), -7, np.int32)
    at = 0
    for l in range(lanes):
        n = min(held[l], width)
        table[l, :n] = ids[at:at + n]
        at += n
    return lens, add, held, table, ids[len(ids) - free - 3:].copy(), free


PLAN = [
    # lanes, most new tokens, context, block size, capacity, table short by, share of the blocks free
    (1, 1, 0, 1, 1, 0, 1.0),
    (1, 8, 100, 16, 20, 0, 1.0),
    (64, 8, 2000, 16, 512, 0, 1.0),
    (64, 8, 2000, 16, 200, 0, 1.0),
    (64, 8, 2000, 13, 512, 0, 0.5),
    (50, 300, 1000, 64, 20000, 0, 0.7),
    (33, 100, 500, 7, 2500, 30, 0.9),
    (1023, 5, 50, 4, 4000, 0, 0.8),
    (1024, 2, 50, 4, 700, 0, 1.0),
    (1025, 9, 90, 8, 9000, 3, 0.9),
    (3000, 4, 40, 1, 9000, 0, 0.97),
    (3, 5000, 9000, 256, 15001, 0, 1.0),
    (66000, 2, 20, 4, 60000, 0, 0.99),
]


@pytest.mark.parametrize("n", range(len(PLAN)))
def test_plan(gpu, n):
    torch, T = gpu
    lanes, most, context, bs, capacity, short, spare = PLAN[n]
    rng = np.random.default_rng(80 + n)
    lens, add, held, table, free_ids, free = plan_inputs(rng, lanes, most, context, bs, short, spare)
    want = R.plan(lens, add, held, table, free_ids, free, bs, capacity)
    if n in (3, 4, 6, 8):
        assert want["refused"] > 0  # the case is about refusals
    dt = dev(torch, table)
    print(f"[round] plan {PLAN[n]}", flush=True)
    got = T.plan(dev(torch, lens), dev(torch, add), dev(torch, held), dt, dev(torch, free_ids),
                 dev(torch, np.int32([free])), bs, capacity)
    torch.cuda.synchronize()
    for name in ("held", "col_start", "col_lane", "col_pos", "slots"):
        assert np.array_equal(host(got[name]), np.array(want[name])), name
    assert int(got["free_count"]) == want["free_count"] and int(got["refused"]) == want["refused"]
    assert np.array_equal(host(dt), want["table"])


def test_plan_with_values_out_of_range(gpu):
    """Negative lengths, held blocks beyond the table, a free count beyond the
    list, tokens whose positions pass 2^31 - 1, and slots past 32 bits."""
    torch, T = gpu
    lens = np.int32([-5, 10, 2**31 - 3, 2**31 - 3, 0, 7])
    add = np.int32([3, 4, 2, 3, 2**31 - 1, -2**31])
    held = np.int32([-1, 99, 1, 1, 0, 2])
    bs, width = 2**30, 4
    table = np.arange(24, dtype=np.int32).reshape(6, width) + 100
    free_ids = np.int32([2**31 - 1, 2**31 - 2, 2**31 - 3, 2**31 - 4])
    want = R.plan(lens, add, held, table, free_ids, 9, bs, 20)
    assert max(want["slots"]) > 2**60
    dt = dev(torch, table)
    print("[round] plan, values out of range", flush=True)
    got = T.plan(dev(torch, lens), dev(torch, add), dev(torch, held), dt, dev(torch, free_ids), dev(torch, np.int32([9])),
                 bs, 20)
    for name in ("held", "col_start", "col_lane", "col_pos", "slots"):
        assert np.array_equal(host(got[name]), np.array(want[name])), name
    assert int(got["free_count"]) == want["free_count"] and int(got["refused"]) == want["refused"]
    assert np.array_equal(host(dt), want["table"])


# -------------------------------------------------------------- together ---

def test_rounds_together_in_a_graph(gpu):
    """Rounds as they are used, captured once and replayed: plan, rules on the
    target's logits, top-k, verification, history.  Every replay is checked
    against the plain implementations, with eager work between the replays."""
    import oracle
    torch, T = gpu
    rng = np.random.default_rng(11)
    lanes, V, k, bs, width, drafts_most = 5, 9001, 8, 4, 40, 3
    capacity, limit = lanes * (drafts_most + 1), drafts_most + 1
    dtype = W.BF16
    i32 = lambda a: dev(torch, np.asarray(a, np.int32))  # noqa: E731
    # what a serving loop keeps
    lens, held, free = np.int32([0, 9, 30, 3, 16]), np.int32([0, 3, 8, 2, 4]), 60
    table = np.full((lanes, width), -1, np.int32)
    ids = rng.permutation(200).astype(np.int32)
    for l in range(lanes):
        table[l, :held[l]] = ids[100 + 10 * l:100 + 10 * l + held[l]]
    free_ids = ids[:free]
    d = dict(lens=i32(lens), add=i32(np.zeros(lanes)), held=i32(held), table=i32(table), free_ids=i32(free_ids),
             free=i32([free]), drafts=i32(np.zeros(lanes * drafts_most)), draft_start=i32(np.zeros(lanes + 1)),
             x=dev(torch, np.zeros((capacity, V), np.uint16)), y=dev(torch, np.zeros((capacity, V), np.uint16)),
             mask=i32(np.zeros((capacity, (V + 31) // 32))))
    counts, seen = T.history(V, lanes)
    hc, hs = host(counts).view(np.uint32), host(seen).view(np.uint32)
    pen = dict(repetition=np.float32([1.0, 1.3, 1.1, 2.0, 0.9]), presence=np.float32([0, 0.5, 1, 0.1, 2]),
               frequency=np.float32([0.1, 0.2, 0.3, 0, 0.5]))
    out = T.plan(d["lens"], d["add"], d["held"], d["table"], d["free_ids"], d["free"], bs, capacity)
    rules = T.AdjustRules(V, capacity, dtype, lanes=lanes, col_start=out["col_start"], counts=counts, seen=seen,
                          drafts=d["drafts"], draft_start=d["draft_start"], mask=d["mask"],
                          **{n: dev(torch, v) for n, v in pen.items()})
    handle = T.TopkCols(V, capacity, k, dtype)
    vals = torch.empty((capacity, k), dtype=torch.int16, device="cuda")
    tids = torch.empty((capacity, k), dtype=torch.int32, device="cuda")
    tokens = torch.empty((lanes, limit), dtype=torch.int32, device="cuda")
    cnt = torch.empty(lanes, dtype=torch.int32, device="cuda")

    def one_round():
        T.plan(d["lens"], d["add"], d["held"], d["table"], d["free_ids"], d["free"], bs, capacity, out=out)
        rules.apply(d["x"], d["y"])
        handle.run(d["y"], vals, tids)
        T.verify(vals, tids, out["col_start"], d["drafts"], d["draft_start"], top_p=0.9, seed=3, offset=4,
                 out_tokens=tokens, out_count=cnt)
        T.count_tokens(counts, seen, V, tokens)
        d["lens"].add_(cnt)
        d["held"].copy_(out["held"])
        d["free"].copy_(out["free_count"])

    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        one_round()
    for rnd in range(6):
        n = rng.integers(0, drafts_most + 1, lanes)
        active = rng.random(lanes) < 0.8
        n = np.where(active, n, 0)
        add = np.where(active, n + 1, 0).astype(np.int32)
        ds = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        x = (rng.standard_normal((capacity, V)) * 2).astype(np.float32)
        x[np.arange(capacity), rng.integers(0, 50, capacity)] += 12
        x = W.bf16_bits_from_f32(x)
        allowed = rng.random((capacity, V)) < rng.choice([0.0, 0.5, 1.0], (capacity, 1))
        drafts = np.zeros(lanes * drafts_most, np.int32)
        start = np.concatenate([[0], np.cumsum(add)])
        f = W.f32_from_bf16_bits(x)
        for l in range(lanes):
            for j in range(n[l]):
                drafts[ds[l] + j] = f[start[l] + j].argmax()
        for name, v in (("add", add), ("draft_start", ds), ("drafts", drafts), ("mask", packed(allowed))):
            d[name].copy_(i32(v.view(np.int32) if v.dtype == np.uint32 else v))
        d["x"].copy_(dev(torch, x))
        d["y"].fill_(SENTINEL[dtype])
        torch.cuda.synchronize()
        print(f"[round] replay {rnd}", flush=True)
        graph.replay()
        torch.cuda.synchronize()
        # the same round, plainly
        p = R.plan(lens, add, held, table, free_ids, free, bs, capacity)
        assert p["refused"] == 0
        for name in ("held", "col_start", "col_lane", "col_pos", "slots"):
            assert np.array_equal(host(out[name]), np.array(p[name])), name
        table, held, free = p["table"], np.int32(p["held"]), p["free_count"]
        assert np.array_equal(host(d["table"]), table) and int(d["free"]) == free
        cs = np.int32(p["col_start"])
        exact = R.adjust(x, V, capacity, lanes, dtype, col_start=cs, counts=hc, drafts=drafts, draft_start=ds,
                         mask=packed(allowed), **pen)
        y = host(d["y"], dtype)
        for c in range(capacity):
            if c in exact:
                R.check_adjusted(y[c].copy(), x[c], dtype, c, exact[c])
            else:
                assert (y[c] == SENTINEL[dtype]).all()
        ov, oi = oracle.topk_cols(y, V, capacity, k, oracle.BF16, oracle.COL_CONTIG, V)
        assert np.array_equal(host(tids), oi) and np.array_equal(host(vals, dtype), ov)
        want, count, margin = R.verify(W.f32_from_bf16_bits(ov), oi, R.parts(cs, capacity, lanes), drafts,
                                       R.parts(ds, len(drafts), lanes), None, None, 1.0, 0.9, 3, 4, limit)
        assert margin > 2.0**-40
        assert np.array_equal(host(tokens), want) and np.array_equal(host(cnt), count)
        hc, hs = R.count(hc, hs, V, want.reshape(-1), None)
        assert np.array_equal(host(counts).view(np.uint32), hc) and np.array_equal(host(seen).view(np.uint32), hs)
        lens = lens + count
        assert np.array_equal(host(d["lens"]), lens)
    assert handle.check() == T.TOPK_OK
    handle.close()


def test_calls_on_two_streams(gpu):
    """The entry points keep nothing between calls: two streams at once give
    what each gives alone."""
    torch, T = gpu
    cases = [Case(200 + i, 30011, 3, 6, W.BF16, layout, hist=800, drafts=True, bias=50, mask="column")
             for i, layout in enumerate((W.COL, W.ROW))]
    work = []
    for c in cases:
        before = c.matrix(c.out_ld, None)
        work.append((c, c.device_rules(gpu), dev(torch, c.matrix(c.ld, c.x)), dev(torch, before), before,
                     torch.cuda.Stream()))
    torch.cuda.synchronize()
    print("[round] two streams", flush=True)
    for _ in range(20):
        for c, rules, x, out, before, stream in work:
            rules.apply(x, out, stream=stream)
    torch.cuda.synchronize()
    for c, rules, x, out, before, stream in work:
        c.check(host(out, c.dtype), before)
