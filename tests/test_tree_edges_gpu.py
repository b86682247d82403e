"""GPU tests of attention over the paged cache where a step of places is seen in
part, in every size class of an item's rows, against the definition in 64 bits."""
import math

import pytest

import tree_reference as R

pytestmark = pytest.mark.gpu


def stored(torch, shape, fp8, g):
    """Ordinary random keys or values of a cache: (elements, scale bytes or None, the float64 values they stand for)."""
    if not fp8:
        x = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        return x, None, x.double()
    sign = torch.randint(0, 2, shape, generator=g, device="cuda") << 7
    bits = sign | torch.randint(9, 14, shape, generator=g, device="cuda") << 3 | torch.randint(0, 8, shape, generator=g, device="cuda")
    scales = torch.randint(121, 127, shape[:-1], generator=g, device="cuda").to(torch.uint8)
    return bits.to(torch.uint8).view(torch.float8_e4m3fn), scales, worth(torch, bits, scales)


def worth(torch, bits, scales):
    return torch.from_numpy(R.E4M3).cuda()[bits.long()] * torch.exp2(scales.double() - 127)[..., None]


def dense(torch, q, k, v, see, scale):
    """The columns q (n, heads, group, dim) of one lane over its places k, v (places, heads, dim), all float64; see
    (n, places).  Returns out and, for each element, what roundings move it by at most: a weight is rounded to bfloat16
    (half a step, 2^-8), its score is a binary32 sum of dim products, scaled, less a maximum; then exponentials.  Weights
    w (1 + r) with |r| <= rel move sum w v / sum w by at most (sum w rel |v| + |out| sum w rel) / sum w, but for products
    of these.  Then the sums over places in binary32, and the result's own rounding."""
    n, heads, group, dim = q.shape
    eps = 2.0**-8
    s = scale * torch.matmul(q.permute(1, 0, 2, 3).reshape(heads, n * group, dim), k.permute(1, 2, 0)).view(heads, n, group, -1)
    spread = abs(scale) * torch.matmul(q.abs().permute(1, 0, 2, 3).reshape(heads, n * group, dim), k.abs().permute(1, 2, 0)).view_as(s)
    seen = see[None, :, None, :]
    s = torch.where(seen, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    # (a weight of 0 of a place that is not visible removes it, whatever the value)
    values = v.permute(1, 0, 2)[:, None].expand(heads, n, -1, dim)
    values = torch.where(see[None, :, :, None], values, 0.0)
    out = torch.matmul(w, values) / total
    rel = eps + (dim + 8) * 2.0**-24 * (spread + s.abs()) + 2.0**-22 * top.abs() + 2.0**-20
    rel = torch.where(s == -math.inf, eps, rel)
    moved = (torch.matmul(w * rel, values.abs()) + out.abs() * (w * rel).sum(-1, keepdim=True)) / total * (1 + 2.0**-6)
    sums = (see.sum(-1)[None, :, None, None] + 16) * 2.0**-23 * torch.matmul(w, values.abs()) / total
    bound = moved + sums + (out.abs() + moved + sums) * eps
    none = total == 0
    back = lambda x: torch.where(none, 0.0, x).permute(1, 0, 2, 3).reshape(n, heads * group, dim)  # noqa: E731
    return back(out), back(bound)


def check(torch, got, want, bound, what):
    got = got.double()
    nan, inf = want.isnan(), want.isinf()
    assert torch.equal(got.isnan(), nan), f"{what}: {int((got.isnan() != nan).sum())} of {nan.numel()} are NaN on one side only"
    assert torch.equal(got[inf], want[inf]), what
    fine = ~nan & ~inf
    off = ((got - want).abs() - bound)[fine]
    assert not (off > 0).any(), f"{what}: {int((off > 0).sum())} of {off.numel()} off, the worst by {float(off.max())} more than {float(bound[fine][off.argmax()])}"


def words_of(torch, bits):
    """Rows of truth values (C, n) as rows of 32-bit words."""
    C, n = bits.shape
    b = torch.nn.functional.pad(bits, (0, -n % 32)).view(C, -1, 32).long()
    w = (b << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


ROWS = (16, 32, 64, 128, 256)


def lanes_for(rows, dim, fp8, heads, places):
    """So many lanes that items get `rows` rows: little work goes to smaller items, the limits are 150 MB of keys and
    values read for more than 16 rows and 300 MB for more than 32."""
    each = 2 * (1 if fp8 else 2) * dim * heads * places
    return max(6, math.ceil(1.2 * 300e6 / each / math.ceil(rows / 32)) if rows > 32 else math.ceil(1.2 * 150e6 / each / 2) if rows > 16 else 0)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("dim", [64, 112, 128, 256])
@pytest.mark.parametrize("rows", ROWS)
def test_attend_lengths_beyond_the_tables_row(gpu, rows, dim, fp8):
    """The table's row ends inside a step of places; lengths go on far behind it."""
    torch, T = gpu
    g = torch.Generator(device="cuda").manual_seed(rows + dim)
    H, group = 64, 2
    n = rows // group
    for bs, width in ((13, 3), (13, 5), (16, 5), (100, 1)):
        places = bs * width
        L = lanes_for(rows, dim, fp8, H, places)
        blocks = L * width
        shape = (blocks, bs, H, dim)
        (k, ks, kd), (v, vs, vd) = (stored(torch, shape, fp8, g) for _ in range(2))
        cache = T.KeyCache(k, v, *([ks, vs] if fp8 else []))
        table = torch.randperm(blocks, generator=g, device="cuda").view(L, width).int()
        some = [places + 64, 5 * places, places - n // 2, places, places + 1, 2**31 - 1, 0, places - n]
        lens = torch.tensor([some[l % len(some)] for l in range(L)], dtype=torch.int64, device="cuda").clamp(min=0)
        q = torch.randn(L * n, H * group, dim, generator=g, device="cuda").to(torch.bfloat16)
        tree = torch.randint(0, 2, (L * n, n), generator=g, device="cuda").bool()
        for mask in (None, words_of(torch, tree)):
            out = torch.full_like(q, 7.0)
            cache.attend(q, lens.int(), table, mask=mask, out=out)
            for l in list(range(min(L, 16))) + [L - 1]:
                at, own = table[l].long(), slice(l * n, (l + 1) * n)
                lane_k, lane_v = (x[at].view(places, H, dim) for x in (kd, vd))
                p, j = torch.arange(places, device="cuda")[None], torch.arange(n, device="cuda")[:, None]
                i = (p - lens[l]).expand(n, -1)
                seen = i <= j if mask is None else (i < 0) | ((i < n) & tree[own].gather(1, i.clamp(0, n - 1)))
                want, bound = dense(torch, q[own].double().view(n, H, group, dim), lane_k, lane_v, seen, dim**-0.5)
                check(torch, out[own], want, bound, f"blocks of {bs}, {width} of them, length {int(lens[l])}, mask {mask is not None}")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("dim", [64, 48, 128, 112, 256, 208])
@pytest.mark.parametrize("rows", ROWS)
def test_attend_values_that_are_not_finite_before_the_columns(gpu, rows, dim, fp8):
    """NaN and infinities in places that are seen by all rows of an item or, at a window's edge, by some: for lengths at
    every offset of a step."""
    torch, T = gpu
    g = torch.Generator(device="cuda").manual_seed(rows + dim)
    L, bs, group, H = 64, 16, 4, 1
    n = rows // group
    lens = 128 + torch.arange(L, device="cuda")
    width = (128 + L + n) // bs + 1
    blocks = L * width
    room = 4_000_000 // L // bs  # decides the items' sizes
    table = torch.full((L, room), -1, dtype=torch.int32, device="cuda")
    table[:, :width] = torch.randperm(blocks, generator=g, device="cuda").view(L, width)
    (k, ks, kd), (v, vs, vd) = (stored(torch, (blocks, bs, H, dim), fp8, g) for _ in range(2))
    cache = T.KeyCache(k, v, *([ks, vs] if fp8 else []))
    # one value that is not finite in every eighth place of a lane, each in a dim of its own
    flat = (v.view(torch.uint8) if fp8 else v.view(torch.int16)).view(-1, dim)
    kinds = [0x7F, 0xFF] if fp8 else [0x7FC0, 0x7F80, -0x80]
    for l in range(L):
        p = torch.arange(l % 8, int(lens[l]), 8, device="cuda")
        d = torch.randperm(dim, generator=g, device="cuda")[:len(p)]
        at = table[l, p // bs].long() * bs + p % bs
        kind = torch.tensor(kinds, device="cuda")[torch.randint(0, len(kinds), (len(p),), generator=g, device="cuda")]
        flat[at, d] = kind.to(flat.dtype)
    vd = worth(torch, v.view(torch.uint8), vs) if fp8 else v.double()
    q = torch.randn(L * n, H * group, dim, generator=g, device="cuda").to(torch.bfloat16)
    tree = torch.randint(0, 2, (L * n, n), generator=g, device="cuda").bool()
    depth = torch.randint(0, n, (L * n,), generator=g, device="cuda")
    for window, mask in ((0, None), (0, words_of(torch, tree)), (70, None), (100, words_of(torch, tree)), (33, None)):
        positions = None if mask is None else (lens.repeat_interleave(n) + depth).int()
        out = cache.attend(q, lens.int(), table, mask=mask, positions=positions, window=window)
        for l in range(L):
            own, places = slice(l * n, (l + 1) * n), int(lens[l]) + n
            p, j = torch.arange(places, device="cuda"), torch.arange(n, device="cuda")[:, None]
            at = table[l, p // bs].long() * bs + p % bs
            lane_k, lane_v = (x.reshape(-1, H, dim)[at] for x in (kd, vd))
            i = (p[None] - lens[l]).expand(n, -1)
            position = (lens[l] + j) if positions is None else positions[own].long()[:, None]
            before = (i < 0) & ((p[None] > position - window) if window else True)
            if mask is None:
                seen = before | ((i >= 0) & (i <= j) & ((j - i < window) if window else True))
            else:
                seen = before | ((i >= 0) & tree[own].gather(1, i.clamp(0, n - 1)))
            want, bound = dense(torch, q[own].double().view(n, H, group, dim), lane_k, lane_v, seen, dim**-0.5)
            check(torch, out[own], want, bound, f"length {int(lens[l])}, window {window}, mask {mask is not None}")


PROMPTS = [dict(n=[700, 0, 1, 333], lens=[0, 40, 300, 65], heads=2, group=4, dim=128, bs=16),
           dict(n=[513, 2, 64], lens=[1, 64, 0], heads=1, group=2, dim=64, bs=13),
           dict(n=[1100], lens=[900], heads=1, group=8, dim=96, bs=64),
           dict(n=[300, 5], lens=[77, 200], heads=1, group=5, dim=256, bs=7),
           dict(n=[1, 1, 600] + [1] * 70, lens=[400, 0, 33] + [129] * 70, heads=1, group=1, dim=80, bs=32)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("c", PROMPTS, ids=lambda c: f"{len(c['n'])} lanes to {max(c['n'])} columns, dim {c['dim']}")
def test_attend_prompts(gpu, c, fp8):
    """Hundreds of columns in a lane, next to lanes that decode: as chains, with windows that are shorter than the
    prompt, and under masks of many words."""
    torch, T = gpu
    g = torch.Generator(device="cuda").manual_seed(3)
    H, group, dim, bs = c["heads"], c["group"], c["dim"], c["bs"]
    n, lens = c["n"], torch.tensor(c["lens"], device="cuda")
    cs = torch.zeros(len(n) + 1, dtype=torch.int32, device="cuda")
    cs[1:] = torch.cumsum(torch.tensor(n, device="cuda"), 0)
    L, C, most = len(n), sum(n), max(n)
    width = max(a + b for a, b in zip(n, c["lens"])) // bs + 1
    blocks = L * width
    (k, ks, kd), (v, vs, vd) = (stored(torch, (blocks, bs, H, dim), fp8, g) for _ in range(2))
    cache = T.KeyCache(k, v, *([ks, vs] if fp8 else []))
    q = torch.randn(C + 3, H * group, dim, generator=g, device="cuda").to(torch.bfloat16)
    tree = torch.randint(0, 2, (C + 3, most), generator=g, device="cuda").bool()
    for room in (0, 4_000_000 // L // bs):  # decides the items' sizes
        table = torch.full((L, width + room), -1, dtype=torch.int32, device="cuda")
        table[:, :width] = torch.randperm(blocks, generator=g, device="cuda").view(L, width)
        for window, mask in ((0, None), (45, None), (300, None), (0, words_of(torch, tree))):
            out = torch.full_like(q, 7.0)
            cache.attend(q, lens.int(), table, cs, mask=mask, window=window, out=out)
            assert (out[C:] == 7).all()
            for l in range(L):
                if n[l] == 0:
                    continue
                own, p = slice(int(cs[l]), int(cs[l + 1])), torch.arange(int(lens[l]) + n[l], device="cuda")
                j, at = torch.arange(n[l], device="cuda")[:, None], table[l, p // bs].long() * bs + p % bs
                lane_k, lane_v = (x.reshape(-1, H, dim)[at] for x in (kd, vd))
                i = (p[None] - lens[l]).expand(n[l], -1)
                if mask is None:
                    seen = (i <= j) & ((j - i < window) if window else True)
                else:
                    seen = (i < 0) | tree[own].gather(1, i.clamp(0, most - 1))
                want, bound = dense(torch, q[own].double().view(n[l], H, group, dim), lane_k, lane_v, seen, dim**-0.5)
                check(torch, out[own], want, bound, f"lane {l}, window {window}, mask {mask is not None}, room {room}")


@pytest.mark.parametrize("group", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("dim", [16, 64, 128, 256])
def test_attend_reads_every_pattern_and_scale(gpu, dim, group):
    """Each of the 256 e4m3 patterns with each of the 256 scale bytes: a place that is alone has weight 1, so its value
    comes out as it stands for (times below 2^-126 may be 0; a byte of 255 stands for NaN)."""
    torch, T = gpu
    H, bs = 256 // dim, 16
    patterns = torch.arange(256, device="cuda").to(torch.uint8).view(1, 1, H, dim).expand(256, bs, H, dim).contiguous()
    scales = torch.arange(256, device="cuda").to(torch.uint8).view(256, 1, 1).expand(256, bs, H).contiguous()
    cache = T.KeyCache(torch.zeros_like(patterns).view(torch.float8_e4m3fn), patterns.view(torch.float8_e4m3fn),
                       torch.full_like(scales, 127), scales)
    table = torch.full((256, 40000), -1, dtype=torch.int32, device="cuda")  # (the room decides the items' sizes)
    table[:, 0] = torch.arange(256, device="cuda").int()
    want = worth(torch, patterns[:, 0], scales[:, 0])
    want[255] = math.nan
    # all rows of an item see the place; or only the columns before the last do, which leave it out as if it were masked
    lens = torch.zeros(256, dtype=torch.int32, device="cuda")
    for n, bits in ((1, [1]), (16, [1] * 16), (16, [1] * 15 + [0])):
        mask = torch.tensor(bits, dtype=torch.int32, device="cuda").repeat(256).view(-1, 1)
        q = torch.randn(256 * n, H * group, dim, device="cuda").to(torch.bfloat16)
        out = cache.attend(q, lens, table, mask=mask).view(256, n, H, group, dim)
        for j in range(n):
            for h in range(group):
                got = out[:, j, :, h].double()
                value = want if bits[j] else torch.zeros_like(want)
                rounded = value.float().to(torch.bfloat16).double()
                same = (got == rounded) | (got.isnan() & rounded.isnan()) | ((value.abs() < 2.0**-126) & (got == 0))
                assert same.all(), (n, j, h, (~same).nonzero()[:5].tolist())


@pytest.mark.parametrize("group", [1, 4, 16])
def test_attend_windows_and_masks(gpu, group):
    """A window cuts the lane's tokens by the column's position, and a chain's columns; a mask says by itself which
    columns are seen.  So a chain's mask whose far ancestors are cleared gives the chain's bits, and as tree makes it
    shows all ancestors."""
    torch, T = gpu
    g = torch.Generator(device="cuda").manual_seed(1)
    n, H, dim, bs = 12, 2, 64, 16
    lens = torch.tensor([100, 3, 0], device="cuda")
    L = len(lens)
    (k, _, kd), (v, _, vd) = (stored(torch, (L * 8, bs, H, dim), False, g) for _ in range(2))
    cache, table = T.KeyCache(k, v), torch.randperm(L * 8, generator=g, device="cuda").view(L, 8).int()
    q = torch.randn(L * n, H * group, dim, generator=g, device="cuda").to(torch.bfloat16)
    parents = (torch.arange(L * n, device="cuda") % n - 1).int()
    mask, positions = T.tree(parents, lens.int(), lanes=L, words=1)
    i, j = torch.arange(n, device="cuda")[None], torch.arange(n, device="cuda")[:, None]
    for window in (1, 2, 5, 11, 12, 40):
        chain = cache.attend(q, lens.int(), table, window=window)
        cut = words_of(torch, ((i <= j) & (j - i < window)).repeat(L, 1))
        assert torch.equal(cache.attend(q, lens.int(), table, mask=cut, positions=positions, window=window), chain)
        whole = cache.attend(q, lens.int(), table, mask=mask, positions=positions, window=window)
        for l in range(L):
            own, p = slice(l * n, (l + 1) * n), torch.arange(int(lens[l]) + n, device="cuda")
            lane_k, lane_v = (x.reshape(-1, H, dim)[table[l, p // bs].long() * bs + p % bs] for x in (kd, vd))
            column = (p[None] - lens[l]).expand(n, -1)
            near = j - column < window
            for out, seen in ((chain, (column <= j) & near), (whole, (column <= j) & (near | (column >= 0)))):
                want, bound = dense(torch, q[own].double().view(n, H, group, dim), lane_k, lane_v, seen, dim**-0.5)
                check(torch, out[own], want, bound, f"lane {l}, window {window}")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("dim", [64, 112, 128, 208])
@pytest.mark.parametrize("rows", ROWS)
def test_attend_a_scale_of_zero(gpu, rows, dim, fp8):
    """All places weigh alike, but for queries that are not finite: 0 times them is NaN."""
    torch, T = gpu
    g = torch.Generator(device="cuda").manual_seed(2)
    L, bs, group, H = 2, 16, 4, 2
    n = rows // group
    lens = torch.tensor([70, 0], device="cuda")
    width = (70 + n) // bs + 1
    (k, ks, kd), (v, vs, vd) = (stored(torch, (L * width, bs, H, dim), fp8, g) for _ in range(2))
    cache = T.KeyCache(k, v, *([ks, vs] if fp8 else []))
    table = torch.full((L, 2_000_000 // bs), -1, dtype=torch.int32, device="cuda")  # (the room decides the items' sizes)
    table[:, :width] = torch.randperm(L * width, generator=g, device="cuda").view(L, width)
    q = torch.randn(L * n, H * group, dim, generator=g, device="cuda").to(torch.bfloat16)
    for x in (math.nan, math.inf, -math.inf):
        q[int(torch.randint(0, L * n, (), generator=g, device="cuda")), int(torch.randint(0, H * group, (), generator=g, device="cuda")), dim // 3] = x
    for scale in (0.0, -0.0):
        out = cache.attend(q, lens.int(), table, scale=scale)
        for l in range(L):
            own, p = slice(l * n, (l + 1) * n), torch.arange(int(lens[l]) + n, device="cuda")
            lane_k, lane_v = (x.reshape(-1, H, dim)[table[l, p // bs].long() * bs + p % bs] for x in (kd, vd))
            seen = p[None] - lens[l] <= torch.arange(n, device="cuda")[:, None]
            want, bound = dense(torch, q[own].double().view(n, H, group, dim), lane_k, lane_v, seen, scale)
            check(torch, out[own], want, bound, f"lane {l}, scale {scale}")


def test_caches_of_sizes_past_32_bits_are_refused(gpu):
    """Sizes whose fields are 32-bit numbers are not cut to them."""
    torch, T = gpu
    row = torch.zeros(1, 1, 1, 1, 16, dtype=torch.bfloat16, device="cuda")
    for dim in (2, 3):
        shape = [1, 1, 1, 1, 16]
        shape[dim] = 2**32 + 16
        with pytest.raises(ValueError):
            T.KeyCache(row.expand(shape), row.expand(shape))
    T.KeyCache(row.expand(1, 1, 16, 16, 16), row.expand(1, 1, 16, 16, 16))


def test_rounds_of_very_many_lanes(gpu):
    """More lanes than a grid is high, of two columns each: masks, attention, verification, moves."""
    torch, T = gpu
    g = torch.Generator(device="cuda").manual_seed(1)
    L, n, bs, dim = 70000, 2, 4, 64
    cs = torch.cumsum(torch.randint(0, n + 1, (L,), generator=g, device="cuda"), 0)  # some lanes have none
    cs = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), cs]).int()
    (k, _, kd), (v, _, vd) = (stored(torch, (2 * L, bs, 1, dim), False, g) for _ in range(2))
    cache = T.KeyCache(k, v)
    table = torch.randperm(2 * L, generator=g, device="cuda").int().view(L, 2)
    lens = torch.randint(0, 7, (L,), generator=g, device="cuda").int()
    C = int(cs[-1])
    lane = torch.repeat_interleave(torch.arange(L, device="cuda"), cs.diff().long())
    j = torch.arange(C, device="cuda") - cs[lane].long()
    mask, positions = T.tree((j - 1).int(), lens, cs, words=1)
    assert torch.equal(mask[:, 0], torch.where(j == 0, 1, 3).int()) and torch.equal(positions, lens[lane] + j.int())
    q = torch.randn(C, 2, dim, generator=g, device="cuda").to(torch.bfloat16)
    out = cache.attend(q, lens, table, cs, mask=mask, positions=positions)
    p = torch.arange(2 * bs, device="cuda")
    at = table[:, p // bs].long() * bs + p % bs
    lane_k, lane_v = (x.view(-1, dim)[at][lane] for x in (kd, vd))  # (C, places, dim)
    seen = p[None] <= (lens[lane] + j)[:, None]
    for part in range(0, C, 20000):
        own = slice(part, min(part + 20000, C))
        s = torch.matmul(q[own].double(), lane_k[own].transpose(1, 2)) * dim**-0.5
        w = torch.softmax(torch.where(seen[own][:, None], s, -math.inf), -1)
        want, size = torch.matmul(w, lane_v[own]), torch.matmul(w, lane_v[own].abs())
        # weights are rounded to bfloat16 in the sum over values and in their own, the result once more, 2^-8 each; scores
        # (64 products in binary32, 72 roundings of at most 16 in all magnitudes) and the products of errors are below 2^-13
        assert ((out[own].double() - want).abs() <= (size + 2 * want.abs()) * (2.0**-8 + 2.0**-13)).all()
    columns = torch.full((L, 2), -1, dtype=torch.int32, device="cuda")
    columns[:, 0] = torch.randint(0, 2, (L,), generator=g, device="cuda").int()
    flat = k.view(-1, dim).clone()
    l = (columns[:, 0] == 1).nonzero()[:, 0]
    to, of = (at[l, (lens[l] + i).long()] for i in (0, 1))  # the place behind the lane's tokens gets the next one's row
    flat[to] = flat[of]
    cache.move(lens, table, columns)
    assert torch.equal(k.view(-1, dim), flat)
    values = torch.sort(torch.randn(C, 4, generator=g, device="cuda"), descending=True)[0]
    ids = torch.arange(4, device="cuda").int().expand(C, 4).contiguous()
    tokens = torch.randint(0, 4, (C,), generator=g, device="cuda").int()
    _, _, count = T.verify_tree(values, ids, cs, tokens, (j - 1).int(), torch.rand(C, 2, generator=g, device="cuda"),
                                temperature=0.0, max_tokens=2)
    accepted = torch.zeros(L, dtype=torch.int32, device="cuda")
    accepted[lane[(j == 1) & (tokens == 0)]] = 1  # greedy: token 0 is every list's first
    assert torch.equal(count, accepted + (cs.diff() > 0).int())
