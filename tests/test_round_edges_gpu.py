"""GPU tests of calls around the top-k at the edges of what is documented."""
import numpy as np
import pytest

import round_reference as R
from drafter_vocab_top_amd import workloads as W
from test_round_gpu import dev, host, packed, zipf

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ count ---

STARTS = {
    "backwards": [4, 2, 0, 4],
    "upper half first": [4, 8, 0, 4],
    "negative": [-7, 3, 3, 2**31 - 1],
    "padded": [0, 3, 5, 5],
    "past the end first": [2**31 - 1, 0, 6, -2**31],
    "nobody": [5, 3, 1, -4],
}


@pytest.mark.parametrize("own", [False, True], ids=["few tokens", "owned rows"])
@pytest.mark.parametrize("name", STARTS)
def test_count_starts_in_any_order(gpu, name, own):
    """Starts that are negative, past the ids or run backwards are cut alike
    by both ways of counting (a `fresh` array chooses the second)."""
    torch, T = gpu
    V, start = 100, np.array(STARTS[name], np.int32)
    ids = np.arange(12, dtype=np.int32) * 3 % 7
    counts, seen = T.history(V, 3)
    print(f"[round] count, starts {name} own={own}", flush=True)
    T.count_tokens(counts, seen, V, dev(torch, ids), dev(torch, start),
                   fresh=dev(torch, np.zeros(3, np.int32)) if own else None)
    c, s = R.count(np.zeros((3, V), np.int32), np.zeros((3, 4), np.uint32), V, ids, start)
    assert np.array_equal(host(counts).view(np.uint32), c) and np.array_equal(host(seen).view(np.uint32), s)


@pytest.mark.parametrize("order", ["ascending", "halves exchanged"])
@pytest.mark.parametrize("lanes", [7, 255, 601, 1023, 5001, 66001])
def test_count_starts_of_many_lanes(gpu, lanes, order):
    """Few tokens for each of many lanes, in buffers with tokens of nobody at
    both ends: in ascending order, and with the lanes that own the second half
    of the tokens first."""
    torch, T = gpu
    rng = np.random.default_rng(lanes)
    V, h = 300, lanes // 2
    n = rng.integers(0, 6, lanes - 1)
    at = 333 + np.concatenate([[0], np.cumsum(n)])   # lanes - 1 ranges; one lane is empty
    if order == "ascending":
        start = np.concatenate([[at[0]], at])
    else:
        start = np.concatenate([at[h:], at[:h + 1]])  # (the lane between the halves runs backwards: it is empty)
    assert len(start) == lanes + 1
    start = start.astype(np.int32)
    ids = zipf(rng, int(at[-1]) + 600, V)
    prompt = rng.integers(0, 4, lanes).astype(np.int32)
    counts, seen = T.history(V, lanes)
    print(f"[round] count, starts of {lanes} lanes {order}", flush=True)
    T.count_tokens(counts, seen, V, dev(torch, ids), dev(torch, start), prompt_len=dev(torch, prompt))
    c, s = R.count(np.zeros((lanes, V), np.int32), np.zeros((lanes, 10), np.uint32), V, ids, start, prompt)
    assert np.array_equal(host(counts).view(np.uint32), c) and np.array_equal(host(seen).view(np.uint32), s)


# ----------------------------------------------------------------- adjust ---

def to_storage(y, dtype):
    """binary64 values rounded to binary32 and, for bf16, from there to bf16."""
    f = y.astype(np.float32)
    return W.bf16_bits_from_f32(f) if dtype == W.BF16 else f.view(np.uint32)


@pytest.mark.parametrize("layout", [W.COL, W.ROW])
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_adjust_divides(gpu, dtype, layout):
    """x / repetition is a division: where a penalty cancels the quotient,
    what is left is zero, not the error of a reciprocal."""
    torch, T = gpu
    V, lanes = 70, 128
    rng = np.random.default_rng(8)
    rep = (1 + np.arange(lanes) / 128).astype(np.float32) if dtype == W.BF16 else (1 + rng.random(lanes)).astype(np.float32)
    assert ((1.0 / rep.astype(np.float64)) * rep != 1.0).any()
    times = np.tile(np.float64([1, 2, 4, 0.5, -1]), V // 5)
    x = to_storage(rep[:, None] * times, dtype)
    assert np.array_equal(R.widen(x, dtype), rep[:, None] * times)  # stored exactly
    ones = np.ones((lanes, V), np.int32)
    r = T.AdjustRules(V, lanes, dtype, layout, lanes=lanes, counts=dev(torch, ones), seen=dev(torch, packed(ones != 0)),
                      repetition=dev(torch, rep), presence=dev(torch, np.ones(lanes, np.float32)))
    y = rep.astype(np.float64)[:, None] * np.where(times > 0, 0, times * rep[:, None]) + np.where(times > 0, times, 0) - 1.0
    m = x if layout == W.COL else np.ascontiguousarray(x.T)
    got = host(r.apply(dev(torch, m)), dtype)
    got = got if layout == W.COL else np.ascontiguousarray(got.T)
    assert (got[:, 0::5] == 0).all()
    assert np.array_equal(got, to_storage(y, dtype))


@pytest.mark.parametrize("layout", [W.COL, W.ROW])
def test_adjust_divides_the_largest_and_smallest(gpu, layout):
    """Subnormal, largest and infinite logits and penalties."""
    torch, T = gpu
    rep = np.float32([1e-45, 1.5e-42, 1.1754944e-38, 0.7, 1, 1.7, 3.4028235e38, np.inf])
    row = np.float32([1e-45, 7e-45, 1.1754944e-38, 0.3, 1, 2.9, 3.4028235e38, np.inf, -1e-45, -3.4028235e38, -np.inf, 0.0, -0.0])
    lanes, V = len(rep), len(row)
    ones = np.ones((lanes, V), np.int32)
    r = T.AdjustRules(V, lanes, "f32", layout, lanes=lanes, counts=dev(torch, ones), seen=dev(torch, packed(ones != 0)),
                      repetition=dev(torch, rep))
    x = np.tile(row, (lanes, 1))
    with np.errstate(all="ignore"):
        a, b = x.astype(np.float64), rep.astype(np.float64)[:, None]
        y = (np.where(a > 0, a / b, a * b) - 0.0).astype(np.float32)
    got = host(r.apply(dev(torch, x if layout == W.COL else np.ascontiguousarray(x.T))))
    got = got if layout == W.COL else np.ascontiguousarray(got.T)
    assert np.array_equal(np.isnan(got), np.isnan(y))
    assert np.array_equal(got[~np.isnan(y)].view(np.uint32), y[~np.isnan(y)].view(np.uint32))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("layout", [W.COL, W.ROW])
@pytest.mark.parametrize("dtype", [W.BF16, W.F32])
def test_adjust_rounds_as_written(gpu, dtype, layout, in_place):
    """The chain in binary64, operation by operation, and one rounding: the
    result is that of the formula bit for bit, for counts up to 2^31 - 1."""
    torch, T = gpu
    V, lanes = 3001, 5
    rng = np.random.default_rng(18)
    x = to_storage(rng.standard_normal((lanes, V)) * 4, dtype)
    n = np.minimum(2.0 ** rng.uniform(0, 31, (lanes, V)), 2**31 - 1).astype(np.int64) * (rng.random((lanes, V)) < 0.8)
    prompt = rng.random((lanes, V)) < 0.3
    words = n.astype(np.uint32) | np.where(prompt, R.FLAG, np.uint32(0))
    rep, pres, freq = ((0.4 + rng.random(lanes) * 2).astype(np.float32) for _ in range(3))
    freq[2:] *= np.float32(2.0**-20)
    bias = (rng.standard_normal((lanes, V)) * 3).astype(np.float32)
    r = T.AdjustRules(V, lanes, dtype, layout, lanes=lanes, counts=dev(torch, words.view(np.int32)),
                      seen=dev(torch, packed(words != 0)), repetition=dev(torch, rep), presence=dev(torch, pres),
                      frequency=dev(torch, freq), bias_start=dev(torch, np.arange(lanes + 1, dtype=np.int32) * V),
                      bias_ids=dev(torch, np.tile(np.arange(V, dtype=np.int32), lanes)), bias_values=dev(torch, bias.ravel()))
    rep, pres, freq = (v.astype(np.float64)[:, None] for v in (rep, pres, freq))
    y = R.widen(x, dtype)
    y = np.where(words != 0, np.where(y > 0, y / rep, y * rep), y)
    y = np.where(n > 0, y - (freq * n + pres), y) + bias
    m = dev(torch, x if layout == W.COL else np.ascontiguousarray(x.T))
    got = host(r.apply(m, m if in_place else None), dtype)
    got = got if layout == W.COL else np.ascontiguousarray(got.T)
    assert np.array_equal(got, to_storage(y, dtype))


# ----------------------------------------------------------------- verify ---

def test_verify_refuses_lists_it_would_misplace(gpu):
    """Without draft_start the drafts are split evenly, and so are their
    lists: fewer lists than drafts belong to no lane in particular.  With
    draft_start, drafts past the lists are not judged."""
    torch, T = gpu
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    values, ids = torch.zeros((16, 8), device="cuda"), i32(16, 8)
    for n in (12, 13, 0):
        with pytest.raises(ValueError, match="draft_start"):
            T.verify(values, ids, None, i32(14), None, torch.zeros((n, 8), device="cuda"), i32(n, 8), lanes=2, max_tokens=8)
    # more lists than drafts: the rest is unused
    tokens, count = T.verify(values, ids, None, i32(14), None, torch.zeros((20, 8), device="cuda"), i32(20, 8), lanes=2,
                             max_tokens=8)
    assert count.tolist() == [8, 8]
    start = dev(torch, np.int32([0, 7, 14]))
    tokens, count = T.verify(values, ids, None, i32(14), start, torch.zeros((12, 8), device="cuda"), i32(12, 8), lanes=2,
                             max_tokens=8)
    assert count.tolist() == [8, 6]


def test_verify_refuses_half_a_list(gpu):
    torch, T = gpu
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    values, ids = torch.zeros((16, 8), device="cuda"), i32(16, 8)
    with pytest.raises(ValueError, match="draft_ids"):
        T.verify(values, ids, None, i32(14), None, draft_ids=i32(14, 8), lanes=2, max_tokens=8)


# ---------------------------------------------------------------- streams ---

def stream_of(torch, t):
    """The stream whose memory a tensor lies in."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])


def test_outputs_made_for_another_stream(gpu):
    """Calls on a side stream that allocate their outputs: these lie in that
    stream's memory, and hold what the calls on the current stream give."""
    torch, T = gpu
    rng = np.random.default_rng(4)
    V, lanes, n, k = 5003, 4, 3, 8
    C = lanes * n
    x = dev(torch, W.random_matrix(3, V, C, W.BF16, W.COL, kind="normal")).view(torch.bfloat16).reshape(C, V)
    i32 = lambda a: dev(torch, np.asarray(a, np.int32))  # noqa: E731
    drafts = i32(rng.integers(0, V, lanes * (n - 1)))
    rules = T.AdjustRules(V, C, lanes=lanes, presence=dev(torch, np.ones(lanes, np.float32)), drafts=drafts)
    inputs = [i32(a) for a in (np.full(lanes, 5), np.full(lanes, n), np.full(lanes, 2), rng.integers(0, 9, (lanes, 4)),
                               np.arange(9), [9])]
    handle = T.TopkCols(V, C, k)

    def calls(stream):
        y = rules.apply(x, stream=stream)
        v, i = handle.run(y, stream=stream)
        v2, i2 = T.run_noalloc(y, V, C, k, stream=stream)
        s = T.sample(v, i, seed=1, stream=stream)
        t = T.verify(v, i, None, drafts, None, lanes=lanes, max_tokens=n, stream=stream)
        p = T.plan(*inputs, 4, C, stream=stream)
        return [y, v, i, v2, i2, *s, *t, *p.values()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    here = calls(None)
    torch.cuda.synchronize()
    print("[round] outputs made for another stream", flush=True)
    there = calls(side)
    side.synchronize()
    assert len(here) == 16
    for a, b in zip(here, there):
        assert stream_of(torch, a) == 0 and stream_of(torch, b) == side.cuda_stream
        assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                           b.view(torch.int16) if b.dtype == torch.bfloat16 else b)
    handle.close()
