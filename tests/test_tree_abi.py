"""The entry points of tree rounds and of the paged cache refuse bad arguments
before any launch (no device is needed), the binding refuses tensors that do
not fit, and the structures of header and binding agree.  Also pins the plain
implementations that the GPU tests compare with."""
import ctypes
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import tree_reference as R
from drafter_vocab_top_amd import topk_cols as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 256  # an aligned address that is never read
BAD, LARGE = T.TOPK_ERR_INVALID_ARG, T.TOPK_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return T.load()


CACHE = dict(layers=2, blocks=10, block_size=16, heads=2, dim=64, format=0, keys=P, values=P, layer_stride=20480,
             block_stride=2048, slot_stride=128, head_stride=64)
FP8 = dict(CACHE, format=1, key_scales=1, value_scales=1, scale_layer_stride=320, scale_block_stride=32,
           scale_slot_stride=2, scale_head_stride=1)
BAD_CACHES = [dict(CACHE, **kw) for kw in (
    dict(layers=0), dict(blocks=0), dict(block_size=0), dict(heads=0), dict(dim=0), dict(dim=8), dict(dim=72),
    dict(format=2), dict(format=-1), dict(keys=None), dict(values=None), dict(keys=P + 8), dict(values=P + 2),
    dict(layer_stride=-8), dict(block_stride=4), dict(slot_stride=127), dict(head_stride=-64))]
BAD_CACHES += [dict(FP8, **kw) for kw in (
    dict(key_scales=None), dict(value_scales=None), dict(scale_layer_stride=-1), dict(scale_block_stride=-1),
    dict(scale_slot_stride=-1), dict(scale_head_stride=-1), dict(head_stride=8))]
LARGE_CACHES = [dict(CACHE, **kw) for kw in (
    dict(dim=272), dict(blocks=1 << 27), dict(blocks=1 << 31, block_size=1), dict(layers=1 << 20),
    dict(block_stride=1 << 34), dict(slot_stride=1 << 33))] + [dict(FP8, scale_block_stride=1 << 29), dict(FP8, block_stride=1 << 33)]

WRITE = dict(C=8, layer=0, dtype=0, keys=P, values=P, key_stride=128, key_head_stride=64, value_stride=128,
             value_head_stride=64, slots=P)
ATTEND = dict(lanes=2, C=8, layer=0, heads=4, window=0, scale=0.1, q=P, q_stride=256, q_head_stride=64, col_start=P,
              lens=P, table=P, table_ld=4, mask=P, mask_ld=1, positions=P, out=P, out_stride=256, out_head_stride=64,
              workspace=P, workspace_bytes=1 << 40)
VERIFY = dict(lanes=2, dtype=0, k=8, kq=8, C=16, col_start=P, target_values=P, target_ids=P, tokens=P, parents=P,
              draft_values=P, draft_ids=P, uniforms=P, temperature=1.0, top_p=0.9, max_tokens=8, out_tokens=P,
              out_columns=P, out_count=P)


def write(lib, cache=CACHE, **kw):
    return lib.topk_cols_cache_write(ctypes.byref(T.CacheArgs(**cache)), ctypes.byref(T.CacheWriteArgs(**{**WRITE, **kw})), None)


def attend(lib, cache=CACHE, **kw):
    return lib.topk_cols_attend(ctypes.byref(T.CacheArgs(**cache)), ctypes.byref(T.AttendArgs(**{**ATTEND, **kw})), None)


def workspace(lib, cache=CACHE, **kw):
    n = ctypes.c_int64(-1)
    rc = lib.topk_cols_attend_workspace(ctypes.byref(T.CacheArgs(**cache)), ctypes.byref(T.AttendArgs(**{**ATTEND, **kw})),
                                        ctypes.byref(n))
    return rc, n.value


def move(lib, cache=CACHE, lanes=2, lens=P, table=P, table_ld=4, columns=P, width=8):
    return lib.topk_cols_cache_move(ctypes.byref(T.CacheArgs(**cache)), lanes, lens, table, table_ld, columns, width, None)


@pytest.mark.parametrize("cache", BAD_CACHES, ids=lambda c: "-".join(f"{k}={v}" for k, v in c.items() if v != {**FP8, **CACHE}.get(k)))
def test_bad_caches_are_refused(lib, cache):
    assert write(lib, cache) == attend(lib, cache) == move(lib, cache) == BAD
    assert workspace(lib, cache) == (BAD, 0)


def test_caches_beyond_the_limits_are_refused(lib):
    for cache in LARGE_CACHES:
        assert write(lib, cache) == attend(lib, cache) == move(lib, cache) == LARGE, cache
        assert workspace(lib, cache) == (LARGE, 0)


def test_cache_write_refuses(lib):
    for kw in (dict(C=0), dict(C=-1), dict(layer=-1), dict(layer=2), dict(dtype=2), dict(keys=None), dict(values=None),
               dict(slots=None), dict(keys=P + 8), dict(values=P + 4), dict(slots=P + 4), dict(key_stride=4),
               dict(key_head_stride=-8), dict(value_stride=2), dict(value_head_stride=12), dict(dtype=1, key_stride=2)):
        assert write(lib, **kw) == BAD, kw
    assert write(lib, C=(1 << 25) + 1) == LARGE
    assert lib.topk_cols_cache_write(None, ctypes.byref(T.CacheWriteArgs(**WRITE)), None) == BAD
    assert lib.topk_cols_cache_write(ctypes.byref(T.CacheArgs(**CACHE)), None, None) == BAD


def test_attend_refuses(lib):
    sizes = [dict(lanes=0), dict(C=0), dict(layer=-1), dict(layer=2), dict(heads=0), dict(heads=3), dict(window=-1),
             dict(scale=math.inf), dict(scale=math.nan), dict(q_stride=4), dict(q_head_stride=-8), dict(out_stride=12),
             dict(out_head_stride=2), dict(table_ld=0), dict(lanes=3, col_start=None), dict(col_start=P + 2)]
    pointers = [dict(q=None), dict(q=P + 8), dict(lens=None), dict(lens=P + 2), dict(table=None), dict(table=P + 1),
                dict(out=None), dict(out=P + 8), dict(mask=P + 2), dict(mask_ld=0), dict(positions=P + 2),
                dict(workspace=P + 128)]
    for kw in sizes:
        assert attend(lib, **kw) == BAD, kw
        assert workspace(lib, **kw) == (BAD, 0), kw
    for kw in pointers:
        assert attend(lib, **kw) == BAD, kw
    for kw in (dict(lanes=(1 << 20) + 1), dict(table_ld=1 << 31), dict(mask_ld=1 << 31), dict(C=(1 << 24) + 1)):
        assert attend(lib, **kw) == LARGE, kw
    rc, need = workspace(lib, q=None, lens=None, table=None, out=None, workspace=None)
    assert rc == T.TOPK_OK and need >= 0
    if need:
        assert attend(lib, workspace=None) == BAD
        assert attend(lib, workspace_bytes=need - 1) == BAD
    assert lib.topk_cols_attend(None, ctypes.byref(T.AttendArgs(**ATTEND)), None) == BAD
    assert lib.topk_cols_attend(ctypes.byref(T.CacheArgs(**CACHE)), None, None) == BAD
    assert lib.topk_cols_attend_workspace(ctypes.byref(T.CacheArgs(**CACHE)), ctypes.byref(T.AttendArgs(**ATTEND)), None) == BAD


def test_cache_move_refuses(lib):
    for kw in (dict(lanes=0), dict(lens=None), dict(lens=P + 2), dict(table=None), dict(table=P + 1), dict(table_ld=0),
               dict(columns=None), dict(columns=P + 2), dict(width=0)):
        assert move(lib, **kw) == BAD, kw
    for kw in (dict(lanes=(1 << 20) + 1), dict(table_ld=1 << 31), dict(width=1 << 31)):
        assert move(lib, **kw) == LARGE, kw


def test_tree_refuses(lib):
    good = dict(lanes=2, C=8, col_start=P, parents=P, lens=P, mask=P, mask_ld=1, positions=P)

    def call(**kw):
        return lib.topk_cols_tree(*{**good, **kw}.values(), None)
    for kw in (dict(lanes=0), dict(C=0), dict(lanes=3, col_start=None), dict(col_start=P + 2), dict(parents=None),
               dict(parents=P + 2), dict(lens=P + 1), dict(mask=None), dict(mask=P + 2), dict(mask_ld=0),
               dict(positions=None), dict(positions=P + 3)):
        assert call(**kw) == BAD, kw
    for kw in (dict(lanes=(1 << 20) + 1), dict(C=1 << 31), dict(mask_ld=1 << 31)):
        assert call(**kw) == LARGE, kw


def test_verify_tree_refuses(lib):
    def call(**kw):
        return lib.topk_cols_verify_tree(ctypes.byref(T.VerifyTreeArgs(**{**VERIFY, **kw})), None)
    bad = [dict(lanes=0), dict(C=0), dict(dtype=2), dict(k=0), dict(k=65), dict(kq=0), dict(kq=65), dict(col_start=P + 1),
           dict(lanes=3, col_start=None), dict(target_values=P + 1), dict(dtype=1, target_values=P + 2),
           dict(draft_values=None), dict(draft_ids=None), dict(draft_values=P + 1), dict(temperature=-0.5),
           dict(temperature=math.inf), dict(temperature=math.nan), dict(top_p=0.0), dict(top_p=1.01),
           dict(top_p=math.nan), dict(max_tokens=0)]
    for n in ("target_values", "target_ids", "tokens", "parents", "uniforms", "out_tokens", "out_columns", "out_count"):
        bad.append({n: None})
        if n != "target_values":
            bad.append({n: P + 2})
    for kw in bad:
        assert call(**kw) == BAD, kw
    for kw in (dict(lanes=(1 << 20) + 1), dict(C=1 << 31), dict(max_tokens=1 << 31)):
        assert call(**kw) == LARGE, kw
    assert lib.topk_cols_verify_tree(None, None) == BAD


def test_structures_match_the_header(tmp_path):
    names = {"topk_cache": T.CacheArgs, "topk_cache_write_args": T.CacheWriteArgs, "topk_attend_args": T.AttendArgs,
             "topk_verify_tree_args": T.VerifyTreeArgs}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "topk_cols.h"', "int main(void) {"]
    expect = []
    for name, cls in names.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        expect.append(ctypes.sizeof(cls))
        for field, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {field}));')
            expect.append(getattr(cls, field).offset)
    lines.append("return 0; }")
    src, exe = tmp_path / "s.c", tmp_path / "s"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"), str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(g) for g in got] == expect


def test_the_binding_refuses_host_tensors():
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16)  # noqa: E731
    b = T._round_binding()
    c = T.CacheArgs(**CACHE)
    at = ctypes.addressof(c)
    v = torch.zeros(8, 4)
    calls = [
        lambda: T.tree(i32(8), i32(2)), lambda: T.tree(i32(8)),
        lambda: T.verify_tree(v, i32(8, 4), None, i32(8), i32(8), torch.zeros(8, 2)),
        lambda: T.verify_tree(v, i32(8, 4), i32(3), i32(8), i32(8), torch.zeros(8, 2)),
        lambda: T.KeyCache(bf(2, 4, 2, 64), bf(2, 4, 2, 64)),
        lambda: b.tree(0, 2, i32(8), i32(2), i32(3), i32(7, 1), i32(8)),
        lambda: b.tree(0, 2, i32(8), i32(2), i32(3), i32(8, 1), i32(8)),
        lambda: b.cache_write(0, at, 0, bf(8, 2, 64), bf(8, 2, 64), torch.zeros(8, dtype=torch.int64), 0),
        lambda: b.cache_write(0, at, -1, bf(8, 2, 32), bf(8, 2, 64), torch.zeros(8, dtype=torch.int64), 0),
        lambda: b.cache_write(0, at, -1, bf(8, 2, 64).half(), bf(8, 2, 64).half(), torch.zeros(8, dtype=torch.int64), 0),
        lambda: b.attend(0, at, 0, bf(8, 4, 64), i32(2), i32(2, 4), None, None, None, 0, 0.1, 0, bf(8, 4, 64)),
        lambda: b.attend(0, at, -1, bf(8, 4, 64).float(), i32(2), i32(2, 4), None, None, None, 0, 0.1, 0, bf(8, 4, 64)),
        lambda: b.attend(0, at, -1, bf(8, 4, 64), i32(2), i32(2, 4), None, None, None, 1 << 31, 0.1, 0, bf(8, 4, 64)),
        lambda: b.cache_move(0, at, 0, i32(2), i32(2, 4), i32(2, 8)),
        lambda: b.cache_move(0, at, 0, i32(3), i32(2, 4), i32(3, 8)),
        lambda: b.tree(0, 2),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            print(i)
    with pytest.raises(TypeError):
        b.tree(0, 2, None, i32(2), i32(3), i32(8, 1), i32(8))


def test_entry_points_without_a_device_fail_cleanly():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    code = ("import ctypes; import sys; sys.path.insert(0, 'tests'); import test_tree_abi as A; from drafter_vocab_top_amd import topk_cols as T;"
            "lib = T.load(); E = T.TOPK_ERR_HIP;"
            "assert A.write(lib) == E; assert A.write(lib, A.FP8) == E; assert A.attend(lib) == E; assert A.move(lib) == E;"
            "assert lib.topk_cols_tree(2, 8, 256, 256, None, 256, 1, 256, None) == E;"
            "assert lib.topk_cols_verify_tree(ctypes.byref(T.VerifyTreeArgs(**A.VERIFY)), None) == E")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)


# ------------------------------------------------------ the plain forms ---

def test_reference_e4m3_is_the_type():
    pattern = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(R.E4M3, pattern.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 20011), np.linspace(-0.05, 0.05, 20011), R.E4M3[np.isfinite(R.E4M3)],
                        (R.E4M3[:126] + R.E4M3[1:127]) / 2])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn)
    exact = torch.from_numpy(x).float().double().numpy()
    assert np.array_equal(R.e4m3(exact), want.view(torch.uint8).numpy())


def test_reference_quantise_by_hand():
    q, b = R.quantise(np.array([448.0, -0.5, 0.0, 1.0]))
    assert b == 127 and R.E4M3[q].tolist() == [448.0, -0.5, 0.0, 1.0]
    q, b = R.quantise(np.array([449.0, np.inf, np.nan, 2.0]))
    assert b == 128 and R.E4M3[q[0]] == 224.0 and np.isnan(R.E4M3[q[1:3]]).all() and R.E4M3[q[3]] == 1.0
    assert R.quantise(np.zeros(4))[1] == 1 and R.quantise(np.full(4, np.nan))[1] == 1


def test_reference_tree_by_hand():
    mask, pos = np.zeros((6, 1), np.uint32), np.zeros(6, np.int32)
    R.tree([(0, 5), (5, 6)], [-1, 0, 0, 1, 7, 0], [10, -3], mask, pos)
    assert mask[:, 0].tolist() == [1, 0b11, 0b101, 0b1011, 0b10000, 1] and pos.tolist() == [10, 11, 11, 12, 10, 0]


def test_reference_attend_by_hand():
    k = np.zeros((1, 4, 1, 16))
    v = np.arange(4.0).reshape(1, 4, 1, 1) * np.ones(16)
    q = np.zeros((2, 1, 16))
    out, _ = R.attend(q, k, v, [(0, 2)], [2], np.zeros((1, 1), int), 4, 1, 1.0, out=np.zeros((2, 1, 16)))
    assert out[:, 0, 0].tolist() == [1.0, 1.5]  # places 0, 1, 2 and 0 to 3
    mask = np.array([[1], [2]], np.uint32)
    out, _ = R.attend(q, k, v, [(0, 2)], [2], np.zeros((1, 1), int), 4, 1, 1.0, window=2, mask=mask, out=out)
    assert out[:, 0, 0].tolist() == [1.5, 3.0]  # places 1, 2 and 3


def test_reference_verify_tree_keeps_the_distribution():
    """One anchor with two children sampled from q: the committed tokens follow p."""
    rng = np.random.default_rng(3)
    p_values, q_values = np.array([1.0, 0.5, 0.2, -1.0]), np.array([2.0, 1.9, 0.0, -0.5])
    ids, qids = [3, 5, 7, 9], [5, 3, 9, 11]
    p = np.exp(p_values) / np.exp(p_values).sum()
    q = np.exp(q_values) / np.exp(q_values).sum()
    seen, n = {i: 0 for i in ids}, 20000
    for _ in range(n):
        tokens = [0] + [qids[i] for i in rng.choice(4, 2, p=q)]
        got, _, _, _ = R.verify_tree(np.tile(p_values, (3, 1)), np.tile(ids, (3, 1)), [(0, 3)], tokens, [-1, 0, 0],
                                     rng.random((3, 2)), np.tile(q_values, (3, 1)), np.tile(qids, (3, 1)), 1.0, 1.0, 3)
        seen[int(got[0, 0])] += 1
    chi2 = sum((seen[i] - n * x) ** 2 / (n * x) for i, x in zip(ids, p))
    assert chi2 < 16.3  # 3 degrees of freedom, one in a thousand
