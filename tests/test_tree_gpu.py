"""GPU tests of tree rounds over a paged cache, each operator against the plain
64-bit implementation in tree_reference.py, and of a whole round as it is used."""
import numpy as np
import pytest

import tree_reference as R

pytestmark = pytest.mark.gpu


def dev(torch, a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view({np.dtype(np.uint32): np.int32}.get(a.dtype, a.dtype))).cuda()


def starts(rng, lanes, most, empty=0.2):
    n = rng.integers(1, most + 1, lanes) * (rng.random(lanes) >= empty)
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def random_parents(rng, spans, C, chain=False):
    p = np.full(C, -1, np.int32)
    for b, e in spans:
        for j in range(1, e - b):
            p[b + j] = j - 1 if chain else rng.integers(0, j)
    return p


# ------------------------------------------------------------------- tree ---

TREES = [dict(lanes=1, most=1), dict(lanes=1, most=8), dict(lanes=5, most=64), dict(lanes=33, most=17, gap=5),
         dict(lanes=3, most=64, chain=True), dict(lanes=2, most=200), dict(lanes=2, most=150, chain=True, words=9),
         dict(lanes=4, most=100, words=1), dict(lanes=300, most=3, empty=0.5), dict(lanes=2, most=65, empty=0.0)]


@pytest.mark.parametrize("c", TREES, ids=str)
def test_tree(gpu, c):
    torch, T = gpu
    rng = np.random.default_rng(11)
    cs = starts(rng, c["lanes"], c["most"], c.get("empty", 0.2))
    C = int(cs[-1]) + c.get("gap", 0) + 1
    spans = R.spans_of(cs, c["lanes"], C)
    parents = random_parents(rng, spans, C, c.get("chain"))
    if c["most"] > 10 and not c.get("chain"):
        parents[rng.random(C) < 0.05] = 1 << 20  # follow none
        parents[rng.random(C) < 0.05] = -7
    lens = rng.integers(-3, 5000, c["lanes"]).astype(np.int32)
    words = c.get("words", (c["most"] + 31) // 32)
    mask, positions = np.full((C, words), 0xABCD, np.uint32), np.full(C, 77, np.int32)
    gm, gp = T.tree(dev(torch, parents), dev(torch, lens), dev(torch, cs), mask=dev(torch, mask), positions=dev(torch, positions))
    R.tree(spans, parents, lens, mask, positions)
    assert np.array_equal(gm.cpu().numpy().view(np.uint32), mask)
    assert np.array_equal(gp.cpu().numpy(), positions)


def test_tree_evenly_and_without_lens(gpu):
    torch, T = gpu
    rng = np.random.default_rng(2)
    spans = R.spans_of(None, 6, 60)
    parents = random_parents(rng, spans, 60)
    gm, gp = T.tree(dev(torch, parents), lanes=6, words=1)
    mask, positions = np.zeros((60, 1), np.uint32), np.zeros(60, np.int32)
    R.tree(spans, parents, np.zeros(6, np.int32), mask, positions)
    assert np.array_equal(gm.cpu().numpy().view(np.uint32), mask) and np.array_equal(gp.cpu().numpy(), positions)
    gm, _ = T.tree(dev(torch, parents), lanes=6)  # words for any lane
    assert gm.shape == (60, 2) and np.array_equal(gm.cpu().numpy().view(np.uint32)[:, :1], mask) and not gm[:, 1].any()


def test_tree_starts_out_of_order_and_out_of_range(gpu):
    torch, T = gpu
    cs = np.array([20, 5, 12, -4, 4, 99], np.int32)  # lanes 20..5 (none), 5..12, 12..-4 (none), 0..4, 4..30
    spans = R.spans_of(cs, 5, 30)
    spans[4] = (0, 0)
    cs[5] = 3  # 4..3: none
    parents = random_parents(np.random.default_rng(1), spans, 30)
    mask, positions = np.full((30, 1), 5, np.uint32), np.full(30, 5, np.int32)
    gm, gp = T.tree(dev(torch, parents), None, dev(torch, cs), mask=dev(torch, mask), positions=dev(torch, positions))
    R.tree(spans, parents, np.zeros(5, np.int32), mask, positions)
    assert np.array_equal(gm.cpu().numpy().view(np.uint32), mask) and np.array_equal(gp.cpu().numpy(), positions)


# ------------------------------------------------------------------ cache ---

def make_cache(gpu, rng, fp8, layers, blocks, block_size, heads, dim, layout="slots", fill="random"):
    """(KeyCache, its tensors).  layout: slots (block, slot, head), heads (block, head, slot), or padded rows."""
    torch, T = gpu
    order = dict(slots=(0, 1, 2, 3, 4), heads=(0, 1, 3, 2, 4), padded=(0, 1, 2, 3, 4))[layout]
    shape = (layers, blocks, block_size, heads, dim)
    stored = [shape[i] for i in order]
    if layout == "padded":
        stored[3:] = [heads + 1, dim + 32]
    out = []
    for _ in range(2):
        if fill == "nan":
            x = torch.full(stored, 0x7F if fp8 else 0x7FFF, dtype=torch.uint8 if fp8 else torch.int16, device="cuda")
        elif fp8:
            x = dev(torch, (rng.integers(0, 256, stored) & 0xBF | 0x20).astype(np.uint8))  # ordinary values
        else:
            x = dev(torch, rng.standard_normal(stored).astype(np.float32)).to(torch.bfloat16)
        x = x.view(torch.float8_e4m3fn if fp8 else torch.bfloat16) if x.dtype != torch.bfloat16 else x
        x = x[..., :heads, :dim] if layout == "padded" else x.permute(*[order.index(i) for i in range(5)])
        assert tuple(x.shape) == shape
        out.append(x)
    scales = []
    if fp8:
        for _ in range(2):
            s = dev(torch, rng.integers(120, 130, stored[:-1]).astype(np.uint8))
            s = s[..., :heads] if layout == "padded" else s.permute(*[order[:-1].index(i) for i in range(4)])
            scales.append(s)
    return T.KeyCache(*out, *scales), out + scales


def whole(torch, t):
    """Bytes of a cache tensor (as a host array of its shape)."""
    t = t.contiguous()
    return (t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.uint8)).cpu().numpy()


def real(torch, tensors):
    """Keys and values that a cache stands for, float64."""
    if len(tensors) == 2:
        return [t.double().cpu().numpy() for t in tensors]
    return [R.E4M3[whole(torch, t)] * np.exp2(whole(torch, s).astype(np.float64) - 127)[..., None]
            for t, s in zip(tensors[:2], tensors[2:])]


WRITES = [dict(fp8=fp8, dtype=dtype, dim=dim, heads=heads, layout=layout)
          for fp8 in (False, True) for dtype in ("bf16", "f32")
          for dim, heads, layout in ((128, 8, "slots"), (64, 1, "heads"), (16, 3, "padded"), (80, 2, "heads"), (256, 2, "slots"),
                                     (208, 3, "padded"))]


@pytest.mark.parametrize("c", WRITES, ids=str)
def test_cache_write(gpu, c):
    torch, T = gpu
    rng = np.random.default_rng(5)
    layers, blocks, bs, H, D = 2, 7, 13, c["heads"], c["dim"]
    cache, tensors = make_cache(gpu, rng, c["fp8"], layers, blocks, bs, H, D, c["layout"])
    before = [whole(torch, t) for t in tensors]
    C = 41
    slots = rng.permutation(blocks * bs)[:C].astype(np.int64)
    slots[[3, 9, 20, 33]] = [-1, blocks * bs, 1 << 40, -(1 << 40)]
    x = (rng.standard_normal((2, C, H, D)) * np.exp2(rng.integers(-20, 20, (2, C, H, 1)))).astype(np.float32)
    x[:, 5] = 0.0
    x[:, 6, :, ::3] = 0.0
    x[:, 7, 0, :4] = [np.inf, -np.inf, np.nan, 3.0]
    x[:, 8] = np.nan
    x[:, 10] = 1e-40  # subnormal
    x[:, 11] = 3.3e38
    x[:, 12, :, 0] = 448.0
    x[:, 13, :, 0] = 449.0
    x[:, 14] = -np.float32(2.0**-126)
    x[:, 15, 0, 1:] = x[:, 15, 0, :1] / 1e6  # far below the row's largest
    x[:, 16, 0, :2] = [448 * 2.0**-9, 3.5 * 2.0**-9 - 2.0**-20]
    t = dev(torch, x).to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
    if c["layout"] == "padded":  # side by side in one tensor
        kv = torch.cat([t[0], t[1]], dim=1)
        k, v = kv[:, :H], kv[:, H:]
    else:
        k, v = t[0], t[1]
    cache.write(k, v, dev(torch, slots), layer=1)
    torch.cuda.synchronize()
    after = [whole(torch, y) for y in tensors]
    given = t.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        rounded = whole(torch, t.cpu().to(torch.bfloat16))
    for i, s in enumerate(slots):
        if not 0 <= s < blocks * bs:
            continue
        for n in range(2):
            for h in range(H):
                at = (1, s // bs, s % bs, h)
                if c["fp8"]:
                    want, scale = R.quantise(given[n, i, h])
                    got = after[n][at]
                    nan = np.isnan(R.E4M3[want])
                    assert np.array_equal(np.isnan(R.E4M3[got]), nan) and np.array_equal(got[~nan], want[~nan]), (i, h)
                    assert after[2 + n][at] == scale, (i, h)
                    before[2 + n][at] = after[2 + n][at]
                else:
                    nan = np.isnan(given[n, i, h])
                    got = after[n][at]
                    assert np.array_equal(got[~nan], rounded[n, i, h][~nan]), (i, h)
                    assert ((got[nan].astype(np.int64) & 0x7FFF) > 0x7F80).all()
                before[n][at] = after[n][at]
    for a, b in zip(after, before):  # everything else as it was
        assert np.array_equal(a, b)


def test_cache_write_many_columns(gpu):
    torch, T = gpu
    cache, tensors = make_cache(gpu, np.random.default_rng(1), True, 1, 300, 64, 8, 128)
    x = torch.randn(19000, 2, 8, 128, device="cuda")
    slots = torch.randperm(300 * 64, device="cuda")[:19000]
    cache.write(x[:, 0], x[:, 1], slots)
    for n in range(2):
        a = x[:, n].abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(a.double() / 448))
        got = tensors[n].view(torch.uint8).view(-1, 8, 128)[slots]
        assert torch.equal(tensors[2 + n].view(-1, 8)[slots].double(), e[..., 0] + 127)
        assert torch.equal(got, torch.ldexp(x[:, n], -e.int()).to(torch.float8_e4m3fn).view(torch.uint8))


MOVES = [dict(fp8=False, layers=1, lanes=1, heads=2, dim=128, bs=16, width=8, layout="slots"),
         dict(fp8=True, layers=3, lanes=5, heads=3, dim=80, bs=1, width=17, layout="heads"),
         dict(fp8=False, layers=2, lanes=7, heads=1, dim=16, bs=13, width=64, layout="padded"),
         dict(fp8=True, layers=2, lanes=4, heads=8, dim=256, bs=64, width=33, layout="slots"),
         dict(fp8=True, layers=1, lanes=3, heads=1, dim=16, bs=5, width=1, layout="slots")]


@pytest.mark.parametrize("c", MOVES, ids=str)
def test_cache_move(gpu, c):
    torch, T = gpu
    rng = np.random.default_rng(8)
    L, bs, width = c["lanes"], c["bs"], c["width"]
    row = (90 + 80) // bs + 1
    blocks = L * row + 3
    cache, tensors = make_cache(gpu, rng, c["fp8"], c["layers"], blocks, bs, c["heads"], c["dim"], c["layout"])
    table = rng.permutation(blocks)[:L * row].reshape(L, -1).astype(np.int32)
    lens = rng.integers(0, 90, L).astype(np.int32)
    columns = np.full((L, width), -1, np.int32)
    for l in range(L):
        path = np.sort(rng.permutation(80)[:rng.integers(1, width + 1)])
        path[0] = 0 if l % 2 == 0 else path[0]
        columns[l, :len(path)] = path
    if L > 2:
        lens[1] = -5                           # counts as 0
        lens[2] = row * bs - 10                # the last columns lie beyond the table
        table[0, -1], table[L - 1, 0] = -1, blocks  # no blocks
    want = [whole(torch, t) for t in tensors]
    cache.move(dev(torch, lens), dev(torch, table), dev(torch, columns))
    for w in want:
        R.move(w, lens, table, columns, bs)
    for t, w in zip(tensors, want):
        assert np.array_equal(whole(torch, t), w)


def test_cache_move_long_paths(gpu):
    """More entries than a workgroup has threads, an entry twice, and lanes without any."""
    torch, T = gpu
    rng = np.random.default_rng(18)
    cache, tensors = make_cache(gpu, rng, True, 2, 200, 16, 2, 64)
    table = rng.permutation(200)[:180].reshape(3, 60).astype(np.int32)
    lens = np.array([5, 100, 30], np.int32)
    columns = np.full((3, 600), -1, np.int32)
    for l, n in enumerate((600, 0, 300)):
        path = np.sort(rng.permutation(900)[:n])
        columns[l, :n] = path
    columns[2, 7] = columns[2, 8]
    want = [whole(torch, t) for t in tensors]
    cache.move(dev(torch, lens), dev(torch, table), dev(torch, columns))
    for w, t in zip(want, tensors):
        R.move(w, lens, table, columns, 16)
        assert np.array_equal(whole(torch, t), w)


def test_cache_move_the_last_places(gpu):
    """Places up to 2^31 - 2 are places; those from 2^31 - 1 on are none, whatever the table has room for."""
    torch, T = gpu
    bs = 1 << 20
    keys = torch.zeros(1, 2, bs, 1, 16, dtype=torch.bfloat16, device="cuda")
    values = torch.zeros_like(keys)
    cache = T.KeyCache(keys, values)
    table = torch.full((1, 4096), -1, dtype=torch.int32, device="cuda")
    table[0, 2047], table[0, 2048] = 0, 1  # places 2^31 - 2^20 .. 2^31 + 2^20 - 1
    keys[0, 0, bs - 2], keys[0, 1, 2] = 3.0, 5.0
    before = keys.clone()
    cache.move(torch.tensor([2**31 - 3], dtype=torch.int32, device="cuda"), table,
               torch.tensor([[1, 5]], dtype=torch.int32, device="cuda"))
    before[0, 0, bs - 3] = 3.0
    assert torch.equal(keys, before)


# ----------------------------------------------------------------- attend ---

def attend_case(gpu, c, seed=0):
    """Runs a case; returns (got, want, bound, out before)."""
    torch, T = gpu
    rng = np.random.default_rng(seed)
    L, most, H, G, D, bs = c["lanes"], c["most"], c["heads"], c["group"], c["dim"], c["bs"]
    cs = starts(rng, L, most, c.get("empty", 0.2)) if c.get("ragged", True) else None
    C = (int(cs[-1]) if cs is not None else L * most) + (c.get("gap", 0) if cs is not None else 0)
    C = max(C, 1)
    spans = R.spans_of(cs, L, C)
    ctx = c["ctx"]
    lens = rng.integers(c.get("ctx_min", 0), ctx + 1, L).astype(np.int32)
    if "lens" in c:
        lens = np.resize(np.array(c["lens"], np.int32), L)
    width = (ctx + most) // bs + 1
    blocks = L * width + 2
    table = rng.permutation(blocks)[:L * width].reshape(L, width).astype(np.int32)
    if c.get("room"):  # for more places, which decides how the work is cut
        table = np.concatenate([table, np.full((L, c["room"] // bs), -1, np.int32)], axis=1)
    cache, tensors = make_cache(gpu, rng, c["fp8"], 2, blocks, bs, H, D, c.get("layout", "slots"), fill="nan")
    # what lies in the lanes' places; everywhere else there is NaN
    for l, (b, e) in enumerate(spans):
        p = np.arange(lens[l] + e - b)
        where = (1, dev(torch, table[l][p // bs]).long(), dev(torch, p % bs).long())
        for n in range(2):
            if c["fp8"]:
                bits = (rng.integers(0, 256, (len(p), H, D)) & 0x87 | rng.integers(9, 14, (len(p), H, D)) << 3).astype(np.uint8)
                tensors[n].view(torch.uint8)[where] = dev(torch, bits)
                tensors[2 + n][where] = dev(torch, rng.integers(121, 127, (len(p), H)).astype(np.uint8))
            else:
                tensors[n][where] = dev(torch, rng.standard_normal((len(p), H, D)).astype(np.float32)).to(torch.bfloat16)
    q = dev(torch, (rng.standard_normal((C, H * G, D)) * c.get("sharp", 1.0)).astype(np.float32)).to(torch.bfloat16)
    if c.get("odd_queries"):
        for x in (np.nan, np.inf, -np.inf):
            q[int(rng.integers(0, C)), int(rng.integers(0, H * G)), int(rng.integers(0, D))] = x
    mask = positions = None
    if not c.get("chain"):
        parents = random_parents(rng, spans, C)
        mask, positions = np.zeros((C, c.get("words", (most + 31) // 32)), np.uint32), np.zeros(C, np.int32)
        R.tree(spans, parents, lens, mask, positions)
        if c.get("blind"):
            mask[rng.random(C) < c["blind"]] = 0
    window = c.get("window", 0)
    before = dev(torch, rng.standard_normal((C, H * G, D)).astype(np.float32)).to(torch.bfloat16)
    scale = c.get("scale", D ** -0.5)
    poison = c.get("poison")
    if poison and mask is not None:  # NaN and infinities in rows that some columns do not see
        for l, (b, e) in enumerate(spans):
            for j in range(1, e - b):
                if rng.random() < 0.3:
                    p = int(lens[l]) + j
                    where = (1, int(table[l][p // bs]), p % bs)
                    for n in range(2):
                        t = tensors[n].view(torch.uint8) if c["fp8"] else tensors[n].view(torch.int16)
                        d = rng.integers(0, D, 3)
                        t[where][:, dev(torch, d).long()] = 0x7F if c["fp8"] else int(rng.choice([0x7FC0, 0x7F80, -0x80]))
    out = before.clone()
    got = cache.attend(q, dev(torch, lens), dev(torch, table), col_start=None if cs is None else dev(torch, cs),
                       mask=None if mask is None else dev(torch, mask), positions=None if positions is None else dev(torch, positions),
                       window=window, scale=c.get("scale"), layer=1, out=out)
    torch.cuda.synchronize()
    keys, values = (x[1] for x in real(torch, tensors))
    want, bound = R.attend(q.double().cpu().numpy(), keys, values, spans, lens, table, bs, G, scale, window, positions, mask,
                           before.double().cpu().numpy())
    return got.double().cpu().numpy(), want, bound, spans


def check(got, want, bound):
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{(np.isnan(got) != nan).sum()} of {nan.size} are NaN on one side only"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    fine = ~nan & ~inf
    off = np.abs(got - want)[fine] - bound[fine]
    assert (off <= 0).all(), f"{(off > 0).sum()} of {off.size} off, the worst by {np.abs(got - want)[fine][off.argmax()]} of {bound[fine][off.argmax()]}"


ATTENDS = [
    dict(lanes=1, most=1, ctx=0, heads=1, group=1, dim=64, bs=16),
    dict(lanes=1, most=1, ctx=1, ctx_min=1, heads=1, group=1, dim=128, bs=1),
    dict(lanes=1, most=8, ctx=300, heads=2, group=4, dim=128, bs=16, chain=True, ragged=False),
    dict(lanes=5, most=8, ctx=200, heads=2, group=4, dim=128, bs=16, gap=7),
    dict(lanes=4, most=64, ctx=150, heads=1, group=4, dim=128, bs=32, empty=0.0),
    dict(lanes=3, most=64, ctx=700, heads=2, group=8, dim=64, bs=13),
    dict(lanes=2, most=100, ctx=90, heads=1, group=2, dim=128, bs=64),
    dict(lanes=2, most=150, ctx=40, heads=1, group=1, dim=64, bs=16, chain=True),
    dict(lanes=9, most=5, ctx=140, heads=3, group=5, dim=80, bs=7),
    dict(lanes=3, most=9, ctx=260, heads=1, group=3, dim=96, bs=16, layout="heads"),
    dict(lanes=3, most=20, ctx=260, heads=2, group=2, dim=256, bs=16, layout="padded"),
    dict(lanes=2, most=33, ctx=130, heads=1, group=8, dim=192, bs=256),
    dict(lanes=2, most=4, ctx=90, heads=1, group=1, dim=16, bs=16),
    dict(lanes=2, most=4, ctx=90, heads=2, group=2, dim=240, bs=3),
    dict(lanes=6, most=16, ctx=400, heads=1, group=4, dim=128, bs=16, window=100),
    dict(lanes=6, most=16, ctx=400, heads=1, group=4, dim=128, bs=16, window=100, chain=True),
    dict(lanes=4, most=40, ctx=80, heads=1, group=2, dim=64, bs=16, window=7, chain=True),
    dict(lanes=4, most=10, ctx=80, heads=1, group=2, dim=64, bs=16, window=1),
    dict(lanes=4, most=12, ctx=30, heads=1, group=4, dim=64, bs=16, blind=0.5, ctx_min=0),
    dict(lanes=8, most=12, ctx=0, heads=1, group=4, dim=128, bs=16, blind=0.5),
    dict(lanes=3, most=40, ctx=100, heads=1, group=2, dim=64, bs=16, words=1),
    dict(lanes=2, most=8, ctx=300, heads=1, group=4, dim=128, bs=16, sharp=30.0),
    dict(lanes=2, most=8, ctx=300, heads=1, group=4, dim=128, bs=16, scale=0.0),
    dict(lanes=2, most=8, ctx=300, heads=1, group=4, dim=128, bs=16, scale=-0.3),
    dict(lanes=2, most=8, ctx=9000, ctx_min=8900, heads=1, group=4, dim=128, bs=16),
    dict(lanes=1, most=3, ctx=30000, ctx_min=30000, heads=1, group=1, dim=64, bs=64),
    dict(lanes=40, most=4, ctx=500, heads=2, group=1, dim=64, bs=16),
    dict(lanes=300, most=2, ctx=60, heads=1, group=2, dim=64, bs=16),
    dict(lanes=2, most=64, ctx=2100, heads=2, group=8, dim=128, bs=32, empty=0.0),
    dict(lanes=5, most=24, ctx=70, heads=2, group=3, dim=128, bs=16, poison=True),
    dict(lanes=3, most=60, ctx=70, heads=1, group=2, dim=64, bs=16, poison=True),
    dict(lanes=3, most=20, ctx=70, heads=1, group=2, dim=256, bs=16, poison=True),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("c", ATTENDS, ids=str)
def test_attend(gpu, c, fp8):
    for room in (0, 4000000 // c["lanes"]):
        got, want, bound, spans = attend_case(gpu, dict(c, fp8=fp8, room=room))
        check(got, want, bound)


# Every size class of an item's rows (columns times query heads of a key head: 16, 32, 64, 128, 256), at dims that fill
# a kernel's 64, 128 or 256 and dims that do not, with steps that all rows see whole and steps that they do not.  Little
# work is cut into small items, so the table has room for 4,000,000 places (384 MB of one e4m3 head of dim 48).
CLASSES = [dict(rows=rows, dim=dim, room=room) for rows in (16, 32, 64, 128, 256) for dim in (64, 48, 128, 112, 256, 208)
           for room in (0, 2000000)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("c", CLASSES, ids=str)
def test_attend_sizes(gpu, c, fp8):
    rows, dim = c["rows"], c["dim"]
    for i, extra in enumerate((dict(), dict(window=90), dict(poison=True), dict(chain=True, odd_queries=True))):
        got, want, bound, _ = attend_case(gpu, dict(lanes=2, most=rows // 4, ctx=420, ctx_min=250, heads=1, group=4, dim=dim, bs=16,
                                                    room=c["room"], ragged=False, fp8=fp8, **extra), seed=i)
        check(got, want, bound)


MIXES = [dict(lanes=70, most=16, ctx=150, heads=1, group=4, dim=64, bs=16),              # more lanes than a wave has threads
         dict(lanes=70, most=64, ctx=90, heads=1, group=1, dim=128, bs=32),
         dict(lanes=1, most=64, ctx=4000, ctx_min=4000, heads=1, group=2, dim=64, bs=16),  # one item in many pieces
         dict(lanes=1, most=48, ctx=3000, ctx_min=3000, heads=1, group=4, dim=128, bs=64),
         dict(lanes=24, most=3, ctx=12000, heads=1, group=2, dim=64, bs=64, lens=[12000] + [5] * 23),  # pieces few and many
         dict(lanes=24, most=24, ctx=9000, heads=1, group=2, dim=64, bs=64, lens=[3, 9000, 700, 0]),
         dict(lanes=600, most=2, ctx=300, heads=1, group=1, dim=16, bs=16, lens=[1, 300, 20]),
         dict(lanes=6, most=20, ctx=40, heads=2, group=8, dim=64, bs=16, words=3, odd_queries=True),
         dict(lanes=3, most=5, ctx=300, heads=2, group=4, dim=128, bs=16, gap=300),       # a padded batch: few rows in large items
         dict(lanes=3, most=2, ctx=300, heads=1, group=1, dim=64, bs=16, gap=150, window=40),
         dict(lanes=9, most=150, ctx=120, heads=1, group=3, dim=128, bs=16, empty=0.8),    # many rows in small items
         dict(lanes=70, most=90, ctx=60, heads=1, group=1, dim=64, bs=16, empty=0.95)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("c", MIXES, ids=str)
def test_attend_mixed_lengths(gpu, c, fp8):
    for room in (0, 4000000 // c["lanes"]):
        got, want, bound, _ = attend_case(gpu, dict(c, fp8=fp8, room=room))
        check(got, want, bound)


@pytest.mark.parametrize("most", [4, 24], ids=["few rows", "many rows"])
def test_attend_captured(gpu, most):
    """Two captured calls replayed in turn, with other lengths, queries and cache contents each time and eager work
    between: each replay gives the eager call's bits."""
    torch, T = gpu
    rng = np.random.default_rng(31)
    cache, tensors = make_cache(gpu, rng, True, 1, 260, 16, 2, 128)
    table = torch.randperm(260, device="cuda").int()[:240].view(3, 80)
    states, graphs = [], []
    parents = dev(torch, random_parents(rng, R.spans_of(None, 3, 3 * most), 3 * most))
    for _ in range(2):
        s = dict(q=torch.randn(3 * most, 8, 128, device="cuda").to(torch.bfloat16), lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
        call = lambda s=s: cache.attend(s["q"], s["lens"], table, None, *T.tree(parents, s["lens"], lanes=3))  # noqa: E731
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s["out"] = call()
        states.append(dict(s, call=call))
        graphs.append(graph)
    for i in range(5):
        tensors[2].copy_(dev(torch, rng.integers(120, 128, tuple(tensors[2].shape)).astype(np.uint8)))
        for s in states:
            s["lens"].copy_(dev(torch, rng.integers(0, 1200, 3).astype(np.int32)))
            s["q"].copy_(torch.randn(3 * most, 8, 128, device="cuda").to(torch.bfloat16))
        want = [s["call"]() for s in states]
        for g in graphs if i % 2 else graphs[::-1]:
            g.replay()
        assert torch.randn(500, 500, device="cuda").sum().isfinite()
        for s, w in zip(states, want):
            assert torch.equal(s["out"], w), i


def test_attend_nothing_to_do(gpu):
    """No lane has a column: nothing is written."""
    torch, T = gpu
    cache, _ = make_cache(gpu, np.random.default_rng(1), False, 1, 4, 16, 2, 64)
    for C in (1, 100):
        q = torch.randn(C, 4, 64, device="cuda").to(torch.bfloat16)
        out = q.clone()
        lens, table = torch.tensor([9, 3], dtype=torch.int32, device="cuda"), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
        cache.attend(q, lens, table, col_start=torch.zeros(3, dtype=torch.int32, device="cuda"), out=out)
        assert torch.equal(q, out)


def test_attend_repeats_bit_for_bit(gpu):
    torch, T = gpu
    rng = np.random.default_rng(3)
    cache, _ = make_cache(gpu, rng, False, 1, 600, 16, 2, 128)
    table = torch.randperm(600, device="cuda")[:400].view(4, 100).int()
    lens = torch.tensor([1500, 3, 800, 1555], dtype=torch.int32, device="cuda")
    q = torch.randn(32, 8, 128, device="cuda").to(torch.bfloat16)
    one = cache.attend(q, lens, table)
    for _ in range(3):
        assert torch.equal(cache.attend(q, lens, table), one)


def test_attend_tables_and_lengths_out_of_range(gpu):
    """Lengths beyond the table's row, block ids outside the cache, negative lengths, empty lanes."""
    torch, T = gpu
    rng = np.random.default_rng(6)
    cache, tensors = make_cache(gpu, rng, False, 1, 6, 16, 1, 64)
    table = np.array([[0, 1], [-3, 9], [2, 3], [4, 5]], np.int32)
    lens = np.array([1000, 20, -9, 30], np.int32)
    cs = np.array([0, 3, 6, 6, 10], np.int32)
    q = torch.randn(12, 2, 64, device="cuda").to(torch.bfloat16)
    out = torch.full((12, 2, 64), 7.0, device="cuda").to(torch.bfloat16)
    cache.attend(q, dev(torch, lens), dev(torch, table), col_start=dev(torch, cs), out=out)
    keys, values = (x[0] for x in real(torch, tensors))
    want, bound = R.attend(q.double().cpu().numpy(), keys, values, R.spans_of(cs, 4, 12), lens, table, 16, 2, 64 ** -0.5,
                           out=np.full((12, 2, 64), 7.0))
    check(out.double().cpu().numpy(), want, bound)


def test_attend_strided_queries_and_outputs(gpu):
    torch, T = gpu
    rng = np.random.default_rng(7)
    cache, tensors = make_cache(gpu, rng, False, 1, 10, 16, 2, 64, "heads")
    lens, table = torch.tensor([70, 33], dtype=torch.int32, device="cuda"), torch.arange(10, device="cuda").int().view(2, 5)
    qkv = torch.randn(6, 8, 64, device="cuda").to(torch.bfloat16)
    wide = torch.full((6, 5, 96), 2.0, device="cuda").to(torch.bfloat16)
    a = cache.attend(qkv[:, :4], lens, table)
    b = cache.attend(qkv[:, :4], lens, table, out=wide[:, 1:, 32:])
    assert torch.equal(a, b) and (wide[:, 0] == 2).all() and (wide[:, :, :32] == 2).all()
    c = torch.zeros(4, 6, 64, device="cuda").to(torch.bfloat16)
    cache.attend(qkv[:, :4].transpose(0, 1).contiguous().transpose(0, 1), lens, table, out=c.transpose(0, 1))
    assert torch.equal(a, c.transpose(0, 1))


def test_attend_a_cache_past_32_bits(gpu):
    """Blocks that lie further than 2^32 bytes and elements into the cache."""
    torch, T = gpu
    blocks, H, D, bs = (1 << 32) // (64 * 128 * 16) + 40, 16, 128, 64
    keys, values = (torch.empty(blocks, bs, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert keys.numel() > 1 << 32
    cache = T.KeyCache(keys, values)
    far = torch.tensor([[blocks - 1, 0, blocks - 2]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[3, 1, 2]], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(150, H, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    p = torch.arange(150, device="cuda")
    q = torch.randn(2, H, D, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([148], dtype=torch.int32, device="cuda")
    got = []
    for table in (near, far):
        cache.write(k, v, table[0][p // bs].long() * bs + p % bs)
        got.append(cache.attend(q, lens, table))
    assert torch.equal(got[0], got[1])
    columns = torch.tensor([[0, 1, 2], ], dtype=torch.int32, device="cuda") + torch.tensor([0, 30, 100], device="cuda").int()
    cache.move(torch.tensor([10], dtype=torch.int32, device="cuda"), far, columns)
    flat = far[0][p // bs].long() * bs + p % bs
    assert torch.equal(keys.view(-1, H, D)[flat[11]], k[41]) and torch.equal(values.view(-1, H, D)[flat[12]], v[112])
    del keys, values


# ------------------------------------------------------------ verify_tree ---

def lists(rng, n, k, universe):
    values = -np.sort(-rng.standard_normal((n, k)) * 2, axis=1)
    ids = np.array([rng.permutation(universe)[:k] for _ in range(n)]).astype(np.int32)
    return values.astype(np.float32), ids


def as_stored(torch, values, dtype):
    t = dev(torch, values)
    return t.to(torch.bfloat16) if dtype == "bf16" else t


VERIFIES = [dict(lanes=1, most=1, k=1, kq=1), dict(lanes=1, most=8, k=20, kq=20), dict(lanes=30, most=16, k=64, kq=64),
            dict(lanes=20, most=64, k=8, kq=5, bushy=True), dict(lanes=20, most=40, k=5, kq=0, bushy=True),
            dict(lanes=8, most=150, k=6, kq=6, bushy=True), dict(lanes=8, most=150, k=3, kq=0, chain=True),
            dict(lanes=40, most=12, k=10, kq=7, temperature=0.0), dict(lanes=40, most=12, k=10, kq=0, temperature=0.0),
            dict(lanes=25, most=9, k=12, kq=9, top_p=0.4, temperature=0.6), dict(lanes=25, most=30, k=4, kq=4, same=True),
            dict(lanes=300, most=6, k=3, kq=3, empty=0.4, gap=9), dict(lanes=10, most=20, k=6, kq=6, chain=True, cut=4, same=True),
            dict(lanes=10, most=20, k=6, kq=0, cut=1), dict(lanes=300, most=90, k=4, kq=4, bushy=True, same=True),
            dict(lanes=260, most=150, k=3, kq=3, chain=True, same=True), dict(lanes=4, most=150, k=3, kq=3, chain=True, same=True),
            dict(lanes=256, most=70, k=5, kq=0, bushy=True), dict(lanes=12, most=200, k=4, kq=4, wide=True),
            dict(lanes=270, most=130, k=4, kq=2, wide=True), dict(lanes=30, most=33, k=7, kq=7, top_p=1.0, special=True)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", VERIFIES, ids=str)
def test_verify_tree(gpu, c, dtype):
    torch, T = gpu
    rng = np.random.default_rng(21)
    L, most, k, kq = c["lanes"], c["most"], c["k"], c["kq"]
    cs = starts(rng, L, most, c.get("empty", 0.1))
    C = max(int(cs[-1]), 1) + c.get("gap", 0)
    spans = R.spans_of(cs, L, C)
    if c.get("bushy"):
        parents = np.full(C, -1, np.int32)
        for b, e in spans:
            for j in range(1, e - b):
                parents[b + j] = (j - 1) // 5
    elif c.get("wide"):  # children of a column far behind it
        parents = np.full(C, -1, np.int32)
        for b, e in spans:
            for j in range(1, e - b):
                parents[b + j] = j % 3 if j > 2 else 0
    else:
        parents = random_parents(rng, spans, C, c.get("chain"))
    universe = max(k, kq) + 3
    tv, ti = lists(rng, C, k, universe)
    if c.get("special"):
        tv[rng.random(C) < 0.2, 0] = np.inf
        tv[rng.random(C) < 0.2, -1] = -np.inf
    tv = as_stored(torch, tv, dtype)
    qv = qi = None
    if kq:
        qv, qi = lists(rng, C, kq, universe)
        qv = as_stored(torch, qv, dtype)
        if c.get("same"):
            qv, qi = tv.clone(), ti.copy()
    tokens = rng.integers(0, universe, C).astype(np.int32)
    for b, e in spans:
        for j in range(1, e - b):
            source = ti if not kq else qi
            if rng.random() < 0.9:
                tokens[b + j] = rng.choice(source[b + max(parents[b + j], 0)])
    uniforms = rng.random((C, 2), dtype=np.float32)
    uniforms[rng.random((C, 2)) < 0.05] = 0.0
    temperature, top_p = c.get("temperature", 1.0), c.get("top_p", 0.95)
    most_tokens = c.get("cut", most)
    got = T.verify_tree(tv, dev(torch, ti), dev(torch, cs), dev(torch, tokens), dev(torch, parents), dev(torch, uniforms),
                        draft_values=qv, draft_ids=None if qi is None else dev(torch, qi), temperature=temperature,
                        top_p=top_p, max_tokens=most_tokens)
    want = R.verify_tree(tv.double().cpu().numpy(), ti, spans, tokens, parents, uniforms,
                         None if qv is None else qv.double().cpu().numpy(), qi, temperature, top_p, most_tokens)
    # (decisions nearer to their border than rounding could be read either way; exact ties are decided alike)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w), want[3]


def test_verify_tree_evenly_in_place_of_a_chain(gpu):
    """A chain, judged by verify with the same random numbers: the same tokens."""
    torch, T = gpu
    rng = np.random.default_rng(4)
    L, n, k = 50, 8, 12
    tv, ti = lists(rng, L * n, k, 14)
    qv, qi = lists(rng, L * n, k, 14)
    tv, qv = as_stored(torch, tv, "bf16"), as_stored(torch, qv, "bf16")
    drafts = qi[:, 0].copy()  # of each column's list, a token for the column behind it
    from round_reference import philox_uniform
    uniforms = np.zeros((L * n, 2), np.float32)
    for c in range(L * n):
        # the draft that column c judges sits in column c + 1
        uniforms[c, 1] = philox_uniform(9, 2, c, 2)
        if c % n + 1 < n:
            uniforms[c + 1, 0] = philox_uniform(9, 2, c, 1)
    tokens = np.full(L * n, -1, np.int32)
    parents = np.full(L * n, -1, np.int32)
    for c in range(L * n):
        if c % n:
            tokens[c], parents[c] = drafts[c - 1], c % n - 1
    inner = [c for c in range(L * n) if c % n + 1 < n]
    a = T.verify(tv, dev(torch, ti), None, dev(torch, drafts[inner]), None, draft_values=qv[inner].contiguous(),
                 draft_ids=dev(torch, qi[inner]), seed=9, offset=2, lanes=L, max_tokens=n)
    b = T.verify_tree(tv, dev(torch, ti), None, dev(torch, tokens), dev(torch, parents), dev(torch, uniforms), draft_values=qv,
                      draft_ids=dev(torch, qi), lanes=L, max_tokens=n)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[2])
    columns = torch.arange(n, device="cuda", dtype=torch.int32).expand(L, n)
    assert torch.equal(b[1], torch.where(columns < b[2][:, None], columns, -1))


# ----------------------------------------------------------------- refusals ---

def test_the_binding_refuses_on_the_gpu(gpu):
    torch, T = gpu
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    u8 = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    f8 = lambda *n: u8(*n).view(torch.float8_e4m3fn)  # noqa: E731
    with pytest.raises(ValueError):
        T.KeyCache(bf(4, 16, 2, 64).half(), bf(4, 16, 2, 64).half())
    with pytest.raises(ValueError):
        T.KeyCache(bf(4, 16, 2, 64), bf(4, 16, 2, 32))
    with pytest.raises(ValueError):
        T.KeyCache(f8(4, 16, 2, 64), f8(4, 16, 2, 64))
    with pytest.raises(ValueError):
        T.KeyCache(bf(4, 16, 2, 64), bf(4, 16, 2, 64), u8(4, 16, 2), u8(4, 16, 2))
    with pytest.raises(ValueError):
        T.KeyCache(f8(4, 16, 2, 64), f8(4, 16, 2, 64), u8(4, 16, 2), u8(4, 16, 3))
    with pytest.raises(ValueError):  # strides that differ, or are not of 16 bytes
        T.KeyCache(bf(4, 16, 2, 64), bf(4, 2, 16, 64).transpose(1, 2))
    with pytest.raises(ValueError):
        T.KeyCache(bf(4, 16, 2, 68)[..., :64], bf(4, 16, 2, 68)[..., :64])
    with pytest.raises(ValueError):
        T.KeyCache(bf(4, 16, 64, 2).transpose(2, 3), bf(4, 16, 64, 2).transpose(2, 3))
    cache = T.KeyCache(bf(4, 16, 2, 64), bf(4, 16, 2, 64))
    lens, table, q = i32(2), i32(2, 2), bf(6, 4, 64)
    slots = torch.zeros(6, dtype=torch.int64, device="cuda")
    bad = [lambda: cache.write(bf(6, 2, 64), bf(5, 2, 64), slots), lambda: cache.write(bf(6, 2, 64), bf(6, 2, 64), slots[:5]),
           lambda: cache.write(bf(6, 2, 64), bf(6, 2, 64).float(), slots), lambda: cache.write(bf(6, 3, 64), bf(6, 3, 64), slots),
           lambda: cache.write(bf(6, 2, 64), bf(6, 2, 64), slots.int()),
           lambda: cache.attend(q.float(), lens, table), lambda: cache.attend(bf(6, 4, 32), lens, table),
           lambda: cache.attend(q, lens, i32(1, 2)), lambda: cache.attend(q, lens.long(), table),
           lambda: cache.attend(q, lens, table, mask=i32(5, 1)), lambda: cache.attend(q, lens, table, positions=i32(5)),
           lambda: cache.attend(q, lens, table, out=bf(5, 4, 64)), lambda: cache.attend(q, lens, table, out=bf(6, 3, 64)),
           lambda: cache.attend(q, lens, table, window=-1), lambda: cache.attend(q, i32(1), table, col_start=i32(3)),
           lambda: cache.move(lens, table, i32(1, 4)), lambda: cache.move(lens, table, i32(2)),
           lambda: T.tree(i32(6), lens, i32(3), mask=i32(5, 1)), lambda: T.tree(i32(6), i32(1), i32(3)),
           lambda: T.verify_tree(bf(6, 4), i32(6, 4), None, i32(6), i32(6), torch.zeros(6, 2, device="cuda")),
           lambda: T.verify_tree(bf(6, 4), i32(6, 4), i32(3), i32(6), i32(6), torch.zeros(5, 2, device="cuda")),
           lambda: T.verify_tree(bf(6, 4), i32(6, 4), i32(3), i32(6), i32(6), torch.zeros(6, 2, device="cuda").double()),
           lambda: T.verify_tree(bf(6, 4), i32(6, 4), i32(3), i32(6), i32(6), torch.zeros(6, 2, device="cuda"), draft_values=bf(5, 4), draft_ids=i32(5, 4)),
           lambda: T.verify_tree(bf(6, 4), i32(6, 4), i32(3), i32(6), i32(6), torch.zeros(6, 2, device="cuda"), draft_ids=i32(6, 4))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: cache.write(bf(6, 2, 64), bf(6, 2, 64), slots, layer=1), lambda: cache.attend(bf(6, 3, 64), lens, table),
                 lambda: cache.attend(q, lens, table, layer=-1), lambda: cache.attend(bf(5, 4, 64), lens, table),
                 lambda: cache.attend(q, lens, table, scale=float("nan")), lambda: cache.write(bf(0, 2, 64), bf(0, 2, 64), slots),
                 lambda: cache.write(bf(6, 2, 68)[..., :64], bf(6, 2, 64), slots)):
        with pytest.raises(T.TopkError):
            call()


# ------------------------------------------------------------------ rounds ---

class Serving:
    """Lanes that decode with trees over a paged cache, as a program would: one attention layer of random
    projections stands for the model."""

    def __init__(self, gpu, fp8, lanes=5, nodes=9, bs=16):
        torch, T = self.torch, self.T = gpu
        g = torch.Generator(device="cuda").manual_seed(5)
        self.lanes, self.nodes, self.bs, self.V = lanes, nodes, bs, 16  # (few tokens: drafts are accepted)
        blocks = lanes * 12
        rnd = lambda *n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
        shape = (2, blocks, bs, 2, 64)
        if fp8:
            kv = [torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
            self.cache = T.KeyCache(*kv, *(torch.full(shape[:-1], 127, dtype=torch.uint8, device="cuda") for _ in range(2)))
        else:
            kv = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            self.cache = T.KeyCache(*kv)
        self.embed, self.qkv, self.head = rnd(self.V, 64), rnd(64, 512) / 8, rnd(256, self.V) / 8
        self.free = torch.randperm(blocks, generator=g, device="cuda").int()
        self.table = torch.full((lanes, 12), -1, dtype=torch.int32, device="cuda")
        i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.lens, self.held, self.anchor = i32(lanes), i32(lanes), i32(lanes) + torch.arange(lanes, device="cuda").int() * 3
        self.free_count = torch.tensor([blocks], dtype=torch.int32, device="cuda")
        self.add = torch.full((lanes,), nodes, dtype=torch.int32, device="cuda")
        self.cap = lanes * nodes
        self.parents = torch.tensor([-1, 0, 0, 1, 1, 2, 3, 6, 0][:nodes] * lanes, dtype=torch.int32, device="cuda")
        self.tokens, self.uniforms = i32(self.cap), torch.zeros(self.cap, 2, device="cuda")
        self.top = T.TopkCols(self.V, self.cap, 8, "f32", "col")
        self.out = None
        self.history = T.history(self.V, lanes)

    def round(self):
        torch, T = self.torch, self.T
        plan = T.plan(self.lens, self.add, self.held, self.table, self.free, self.free_count, self.bs, self.cap)
        self.tokens.view(self.lanes, self.nodes)[:, 0] = self.anchor
        mask, positions = T.tree(self.parents, self.lens, plan["col_start"], words=1)
        x = self.embed[self.tokens.long()] + torch.sin(positions[:, None].float() / 10)
        for layer in range(2):
            qkv = (x @ self.qkv).to(torch.bfloat16).view(self.cap, 8, 64)
            self.cache.write(qkv[:, 4:6], qkv[:, 6:], plan["slots"], layer=layer)
            o = self.cache.attend(qkv[:, :4], self.lens, self.table, col_start=plan["col_start"], mask=mask, positions=positions,
                                  layer=layer)
            x = x + o.float().view(self.cap, 4, 64).sum(1) / 2
        logits = (o.float().view(self.cap, 256) @ self.head).contiguous()
        values, ids = self.top.run(logits)
        tokens, columns, count = T.verify_tree(values, ids, plan["col_start"], self.tokens, self.parents, self.uniforms, max_tokens=6)
        self.cache.move(self.lens, self.table, columns)
        T.count_tokens(*self.history, self.V, tokens.view(-1))
        # the state of the next round
        self.anchor.copy_(tokens.gather(1, (count[:, None] - 1).long())[:, 0])
        self.lens.add_(count)
        self.held.copy_(plan["held"])
        self.free_count.copy_(plan["free_count"])
        return tokens, count, o

    def state(self):
        return [t.clone() for t in (self.lens, self.anchor, self.held, self.table, *self.history)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_rounds_together_in_a_graph(gpu, fp8):
    """Six rounds, eager and as replays of one captured round: the same tokens, outputs and state."""
    torch, T = gpu
    eager, captured = Serving(gpu, fp8), Serving(gpu, fp8)
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    draws = [torch.rand(eager.cap, 2, device="cuda") * 0.3 for _ in range(6)]
    g = torch.Generator(device="cuda").manual_seed(1)
    start = captured.state(), [t.clone() for t in captured.cache._tensors]
    with torch.cuda.stream(stream):  # warm
        captured.round()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = captured.round()
    for t, s in zip((captured.lens, captured.anchor, captured.held, captured.table, *captured.history), start[0]):
        t.copy_(s)
    for t, s in zip(captured.cache._tensors, start[1]):
        (t.view(torch.uint8) if fp8 else t).copy_(s.view(torch.uint8) if fp8 else s)
    captured.free_count.fill_(len(captured.free))
    lengths = 0
    for i, u in enumerate(draws):
        guess = torch.randint(0, eager.V, (eager.cap,), generator=g, device="cuda").int()
        for s in (eager, captured):
            s.uniforms.copy_(u)
            s.tokens.copy_(guess)
        want = eager.round()
        graph.replay()
        junk = torch.randn(1000, 1000, device="cuda").sum().item()  # eager work between the replays
        assert junk == junk
        for a, b in zip(want, got):
            assert torch.equal(a, b), i
        for a, b in zip(eager.state(), captured.state()):
            assert torch.equal(a, b), i
        lengths += int(want[1].sum())
    assert lengths > 6 * eager.lanes  # some drafts were accepted


def test_paths_keep_the_text(gpu):
    """After accepted trees have been moved, the cache holds what writing the committed tokens in order holds."""
    torch, T = gpu
    rng = np.random.default_rng(12)
    lanes, nodes, bs, H, D = 3, 7, 4, 2, 64
    blocks = 60
    cache, tensors = make_cache(gpu, rng, False, 1, blocks, bs, H, D)
    table = torch.randperm(blocks, device="cuda").int().view(lanes, 20)
    lens = torch.zeros(lanes, dtype=torch.int32, device="cuda")
    text = [[] for _ in range(lanes)]
    rows = torch.randn(1000, 2, H, D, device="cuda").to(torch.bfloat16)
    for _ in range(8):
        parents = np.concatenate([[-1] + [rng.integers(0, j) for j in range(1, nodes)] for _ in range(lanes)]).astype(np.int32)
        ids = rng.integers(0, 1000, lanes * nodes)
        place = lens.repeat_interleave(nodes) + torch.arange(nodes, device="cuda").repeat(lanes)
        lane = torch.arange(lanes, device="cuda").repeat_interleave(nodes)
        slots = table[lane, (place // bs).long()].long() * bs + place % bs
        kv = rows[dev(torch, ids)]
        cache.write(kv[:, 0], kv[:, 1], slots)
        columns = np.full((lanes, nodes), -1, np.int32)
        for l in range(lanes):
            path = R.line(parents, l * nodes, rng.integers(0, nodes))[::-1]
            columns[l, :len(path)] = path
            text[l] += [ids[l * nodes + i] for i in path]
        cache.move(lens, table, dev(torch, columns))
        lens += dev(torch, (columns >= 0).sum(1).astype(np.int32))
    for l in range(lanes):
        p = torch.arange(len(text[l]), device="cuda")
        at = table[l][p // bs].long() * bs + p % bs
        for n in range(2):
            assert torch.equal(tensors[n].view(-1, H, D)[at], rows[dev(torch, np.array(text[l]))][:, n])


def test_calls_on_another_stream(gpu):
    """Outputs and workspace of calls on a given stream come from its memory, and calls on two streams do not meet."""
    torch, T = gpu
    rng = np.random.default_rng(14)
    cache, _ = make_cache(gpu, rng, False, 1, 400, 16, 2, 128)
    table = torch.randperm(400, device="cuda").int().view(4, 100)
    lens = torch.tensor([1590, 1000, 1500, 700], dtype=torch.int32, device="cuda")
    q = [torch.randn(16, 8, 128, device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [cache.attend(x, lens, table) for x in q]
    parents = torch.tensor([-1, 0, 0, 1] * 4, dtype=torch.int32, device="cuda")
    mask, positions = T.tree(parents, lens, lanes=4)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        got = [cache.attend(x, lens, table, stream=s) for x, s in zip(q, streams)]
        trees = [T.tree(parents, lens, lanes=4, stream=s) for s in streams]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)
        for m, p in trees:
            assert torch.equal(m, mask) and torch.equal(p, positions)
