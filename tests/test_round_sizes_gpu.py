"""GPU tests of the logit rules and the plan at sizes on both sides of every
rule that chooses a kernel: against the formulas in binary64 (torch's
elementary operations), bit for bit."""
import numpy as np
import pytest

import round_reference as R
from test_round_gpu import dev, host, plan_inputs

pytestmark = pytest.mark.gpu

CACHES = 256 << 20   # matrices that, read and written, exceed this go past the caches
EPV = dict(bf16=8, f32=4)
INTS = dict(bf16="int16", f32="int32")


def col_choice(V, C, lanes, dtype, x, out, ld, out_ld):
    """How the column-contiguous kernel is chosen: (what becomes of the matrix, columns of a workgroup)."""
    es, rows = 16 // EPV[dtype], 256 * EPV[dtype]
    wgs = -(-V // rows) * max(C, lanes)
    u = 1 if wgs <= 2048 or C < 2 * lanes else 4
    if x.data_ptr() == out.data_ptr():
        return "in place", u
    if 2 * V * C * es > CACHES:
        return "past the caches", u
    lines = all(v % 128 == 0 for v in (x.data_ptr(), out.data_ptr(), ld * es, out_ld * es))
    return "short runs" if lines else "long runs", u


def row_choice(V, C, dtype, in_place):
    """How the interleaved kernels are chosen: (what becomes of the matrix, rows of a thread)."""
    es, vecs = 16 // EPV[dtype], -(-C // EPV[dtype])
    return ("in place" if in_place else "past the caches" if 2 * V * C * es > CACHES else "long runs",
            16 if V * vecs >= 1 << 20 else 4)


class Matrix:
    """Logits and rules on the GPU, made there."""

    def __init__(self, torch, seed, V, have, dtype, layout, ld_to=1, gap=0, bias=False, mask=False, drafts=True, dense=False):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.torch, self.V, self.dtype, self.layout, self.have = torch, V, dtype, layout, have
        self.lanes, self.C = len(have), int(sum(have)) + gap
        lanes, C = self.lanes, self.C
        rows, width = (C, V) if layout == "col" else (V, C)
        self.width, self.ld = width, -(-width // ld_to) * ld_to
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.ints = getattr(torch, INTS[dtype])
        self.x = torch.empty((rows, self.ld), device="cuda").normal_(0, 4, generator=g).to(dt)
        flat = self.x.view(-1)
        at = torch.randint(0, flat.numel(), (flat.numel() // 50,), generator=g, device="cuda")
        some = torch.tensor([np.inf, -np.inf, 0.0, -0.0, 1e-40, 3e38], device="cuda").to(dt)
        flat[at] = some[torch.arange(at.numel(), device="cuda") % 6]

        def uniform(*n):
            return torch.rand(n, generator=g, device="cuda")

        def pack(b):
            words = -(-V // 32)
            b = torch.nn.functional.pad(b, (0, words * 32 - V), value=True).view(b.shape[0], words, 32).to(torch.int64)
            w = (b << torch.arange(32, device="cuda")).sum(2)
            return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32).contiguous()
        words = torch.zeros((lanes, V), dtype=torch.int32, device="cuda")
        for part in range(0, lanes, 64):   # (in parts: V x lanes may be large)
            w = words[part:part + 64]
            u = uniform(*w.shape)
            w += torch.where(u < (0.97 if dense else 0.01), 1 + (u * 1e4).to(torch.int32) % 5, 0)
            w |= torch.where(uniform(*w.shape) < 0.005, -(1 << 31), 0).to(torch.int32)
        self.words = words
        seen = torch.cat([pack(words[p:p + 64] != 0) for p in range(0, lanes, 64)])
        i32 = lambda a: dev(torch, np.asarray(a, np.int32))  # noqa: E731
        self.col_start = np.concatenate([[0], np.cumsum(have)])
        self.scalars = [(0.5 + rng.random(lanes)).astype(np.float32), rng.standard_normal(lanes).astype(np.float32),
                        rng.random(lanes).astype(np.float32)]
        rep, pres, freq = (dev(torch, a) for a in self.scalars)
        self.rules = dict(col_start=i32(self.col_start), counts=words, seen=seen, repetition=rep, presence=pres, frequency=freq)
        self.drafts = [[] for _ in have]
        if drafts:
            tokens = rng.choice([0, 1, 2, V // 2, V - 1, -1, V], 7)
            self.drafts = [rng.choice(tokens, max(n - 1, 0)).tolist() for n in have]
            if sum(map(len, self.drafts)):
                self.rules.update(drafts=i32(sum(self.drafts, [])),
                                  draft_start=i32(np.concatenate([[0], np.cumsum([len(d) for d in self.drafts])])))
        self.biases = [[] for _ in have]
        if bias:
            for l in range(lanes):
                ids = rng.integers(0, V, 6).tolist() + [0, V - 1, 0, V]
                self.biases[l] = list(zip(ids, (rng.standard_normal(10) * 5).astype(np.float32).tolist()))
            self.rules.update(bias_start=i32(10 * np.arange(lanes + 1)), bias_ids=i32([i for b in self.biases for i, _ in b]),
                              bias_values=dev(torch, np.float32([v for b in self.biases for _, v in b])))
        self.allowed = None
        if mask:
            n = min(C, 9)
            keep = torch.tensor(rng.choice([0.02, 0.5, 0.95, 1.0, 0.0], n), device="cuda")[:, None]
            self.allowed = uniform(n, V) < keep
            self.allowed[0, ::7] = True
            self.mask_index = rng.integers(-1, n + 1, C)
            self.rules.update(mask=pack(self.allowed), mask_index=i32(self.mask_index))

    def apply(self, T, in_place):
        """The result and what it is to be, as (C, V) patterns; padding and columns of nobody are checked."""
        torch = self.torch
        x = self.x.clone()
        out = x if in_place else torch.full_like(x, 7.0)
        before = out.clone()
        r = T.AdjustRules(self.V, self.C, self.dtype, self.layout, self.ld, lanes=self.lanes, **self.rules)
        if self.layout == "col":
            self.choice = col_choice(self.V, self.C, self.lanes, self.dtype, x, out, self.ld, self.ld)
        else:
            self.choice = row_choice(self.V, self.C, self.dtype, in_place)
        r.apply(x, out)
        torch.cuda.synchronize()
        if not in_place:
            assert torch.equal(x.view(self.ints), self.x.view(self.ints)), "the logits were written"
        assert torch.equal(out[:, self.width:].view(self.ints), before[:, self.width:].view(self.ints)), "the padding was written"

        def columns(m):
            m = m[:, :self.width]
            return m if self.layout == "col" else m.t().contiguous()
        got, x, before = columns(out), columns(self.x), columns(before)
        for l, n in enumerate(self.have):
            for j in range(n):
                c = int(self.col_start[l]) + j
                assert torch.equal(got[c].view(self.ints), self.expect(x[c], l, j, c).view(self.ints)), f"lane {l}, column {j}"
        nobody = got[int(self.col_start[-1]):], before[int(self.col_start[-1]):]
        assert torch.equal(nobody[0].contiguous().view(self.ints), nobody[1].contiguous().view(self.ints))

    def expect(self, x, l, j, c):
        torch = self.torch
        rep, pres, freq = (float(a[l]) for a in self.scalars)
        n = (self.words[l] & 0x7FFFFFFF).double()
        for t in self.drafts[l][:j]:
            if 0 <= t < self.V:
                n[t] += 1
        seen = (self.words[l] != 0) | (n > 0)
        y = x.double()
        y = torch.where(seen, torch.where(y > 0, y / rep, y * rep), y)
        y = torch.where(n > 0, y - (freq * n + pres), y)
        changed = seen
        last = {i: v for i, v in self.biases[l] if 0 <= i < self.V}
        if last:
            at = torch.tensor(list(last), device="cuda")
            y[at] += torch.tensor(list(last.values()), dtype=torch.float64, device="cuda")
            changed = changed.clone()
            changed[at] = True
        y = torch.where(changed, y.float().to(x.dtype), x)
        if self.allowed is not None and 0 <= self.mask_index[c] < self.allowed.shape[0]:
            y = torch.where(self.allowed[int(self.mask_index[c])], y, -np.inf)
        return y


def ragged(rng, lanes, most, empty=1):
    have = [most] * lanes
    for l in rng.choice(lanes, max(lanes // 4, 1), replace=False):
        have[l] = int(rng.integers(1, most + 1))
    for l in rng.choice(lanes, min(empty, lanes - 1), replace=False):
        have[l] = 0
    return have


# (what becomes of the matrix, columns of a workgroup): rows in bf16 (half as many in fp32), lanes, columns of a lane
COLUMNS = {
    ("in place", 1): (9001, 3, 5),
    ("in place", 4): (112001, 4, 14),
    ("short runs", 1): (9001, 3, 5),
    ("short runs", 4): (112001, 4, 14),
    ("long runs", 1): (9001, 3, 5),
    ("long runs", 4): (112001, 4, 14),
    ("past the caches", 1): (240001, 300, 1),
    ("past the caches", 4): (280001, 20, 16),
}


@pytest.mark.parametrize("mask", [False, True], ids=["", "mask"])
@pytest.mark.parametrize("bias", [False, True], ids=["", "bias"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("choice", COLUMNS, ids=lambda c: f"{c[0]}-{c[1]}")
def test_adjust_columns(gpu, choice, dtype, bias, mask):
    torch, T = gpu
    V, lanes, most = COLUMNS[choice]
    if dtype == "f32":
        V = V // 2 + 1
    have = ragged(np.random.default_rng(5), lanes, most)
    print(f"[round] {choice} V={V} lanes={lanes} {dtype} bias={bias} mask={mask}", flush=True)
    m = Matrix(torch, 31, V, have, dtype, "col", ld_to=128 if choice[0] == "short runs" else 1, gap=2, bias=bias, mask=mask)
    m.apply(T, choice[0] == "in place")
    assert m.choice == choice


# (what becomes of the matrix, rows of a thread): rows, columns in bf16 (half as many in fp32, several tiles of
# columns where there are more than 512), of which the last vector is moved up or, 3 past a tile, cut
ROWS = {
    ("in place", 4): [(3001, 41)],
    ("in place", 16): [(16001, 530), (16388, 515)],
    ("long runs", 4): [(3001, 41)],
    ("long runs", 16): [(16001, 530), (16388, 515)],
    ("past the caches", 16): [(131003, 530)],
}


@pytest.mark.parametrize("mask", [False, True], ids=["", "mask"])
@pytest.mark.parametrize("bias", [False, True], ids=["", "bias"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("choice,n", [(c, i) for c in ROWS for i in range(len(ROWS[c]))], ids=lambda c: str(c))
def test_adjust_rows(gpu, choice, n, dtype, bias, mask):
    """Every lane's columns: all of them a lane's but the last two of some."""
    torch, T = gpu
    V, C = ROWS[choice][n]
    if dtype == "f32":
        C = C // 2 + (C % 8 > 2)  # past a tile of 256 by 3 as the others are past one of 512
    rng = np.random.default_rng(6)
    gap = 2 * (n == 0)
    have = []
    while sum(have) < C - gap:
        have.append(min(int(rng.integers(0, 9)), C - gap - sum(have)))
    print(f"[round] {choice} V={V} C={C} lanes={len(have)} {dtype} bias={bias} mask={mask}", flush=True)
    m = Matrix(torch, 32, V, have, dtype, "row", ld_to=1 + n, gap=gap, bias=bias, mask=mask)
    assert m.C == C
    m.apply(T, choice[0] == "in place")
    assert m.choice == choice


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_adjust_dense_histories(gpu, dtype, layout):
    """Nearly every row in every history, in place, with masks."""
    torch, T = gpu
    print(f"[round] dense histories {dtype} {layout}", flush=True)
    have = ragged(np.random.default_rng(7), 70, 9, empty=3)
    Matrix(torch, 33, 16500, have, dtype, layout, mask=True, dense=True).apply(T, True)


PLANS = [
    # lanes, most new tokens, context, block size, capacity: columns for the lanes and some more
    (100, 5400, 40000, 64, 270001),
    (300, 9, 300, 16, 1700),
    (512, 5, 90, 4, 2048),
    (400, 1500, 9000, 16, 300000),
    (1500, 400, 3000, 16, 290007),
]


@pytest.mark.parametrize("n", range(len(PLANS)))
def test_plan_sizes(gpu, n):
    """Lanes to a thread and columns to a thread: one, two and four, one and four."""
    torch, T = gpu
    lanes, most, context, bs, capacity = PLANS[n]
    rng = np.random.default_rng(90 + n)
    lens, add, held, table, free_ids, free = plan_inputs(rng, lanes, most, context, bs, 0, 0.95)
    want = R.plan(lens, add, held, table, free_ids, free, bs, capacity)
    assert 0 < want["refused"] < lanes
    dt = dev(torch, table)
    print(f"[round] plan {PLANS[n]}", flush=True)
    got = T.plan(dev(torch, lens), dev(torch, add), dev(torch, held), dt, dev(torch, free_ids), dev(torch, np.int32([free])),
                 bs, capacity)
    torch.cuda.synchronize()
    for name in ("held", "col_start", "col_lane", "col_pos", "slots"):
        assert np.array_equal(host(got[name]), np.array(want[name])), name
    assert int(got["free_count"]) == want["free_count"] and int(got["refused"]) == want["refused"]
    assert np.array_equal(host(dt), want["table"])
