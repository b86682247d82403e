"""GPU tests of calls around the top-k at the edges of what is documented."""
import numpy as np
import pytest

import round_reference as R
from test_round_gpu import dev, host, zipf

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
