"""The entry points around the top-k refuse bad arguments before any launch
(no device is needed: pointers are never read on the host), the binding
refuses tensors that do not fit, and the structures of header and binding
agree."""
import ctypes
import os
import subprocess
import sys

import pytest

from drafter_vocab_top_amd import topk_cols as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 64  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    return T.load()


def rules(**kw):
    a = dict(V=100, C=14, lanes=2, dtype=0, layout=0, ld=100, out_ld=100)
    a.update(kw)
    return T.AdjustRulesArgs(**a)


BIAS = dict(bias_start=P, bias_ids=P, bias_values=P, n_bias=3)
BAD_RULES = [
    dict(V=0), dict(C=0), dict(lanes=0), dict(lanes=3), dict(dtype=2), dict(layout=2), dict(ld=99), dict(out_ld=99),
    dict(layout=1, ld=13), dict(col_start=P + 2),
    dict(counts=P, counts_ld=100), dict(seen=P, seen_ld=4), dict(counts=P, counts_ld=99, seen=P, seen_ld=4),
    dict(counts=P, counts_ld=100, seen=P, seen_ld=3), dict(counts=P + 1, counts_ld=100, seen=P, seen_ld=4),
    dict(repetition=P + 2), dict(presence=P + 1), dict(frequency=P + 3),
    dict(n_drafts=2), dict(draft_start=P), dict(drafts=P, n_drafts=-1), dict(drafts=P, n_drafts=3),
    dict(drafts=P + 1, n_drafts=2),
    dict(BIAS, bias_start=0), dict(BIAS, bias_ids=0), dict(BIAS, bias_values=0), dict(BIAS, n_bias=-1),
    dict(BIAS, bias_values=P + 2), dict(n_bias=3),
    dict(mask=P, mask_ld=3, mask_count=14), dict(mask=P, mask_ld=4, mask_count=13), dict(mask=P, mask_ld=4),
    dict(mask=P + 2, mask_ld=4, mask_count=14), dict(mask=P, mask_ld=4, mask_count=1, mask_index=P + 1),
    dict(mask_index=P),
]


@pytest.mark.parametrize("kw", BAD_RULES, ids=lambda kw: "-".join(kw))
def test_adjust_refuses(lib, kw):
    assert lib.topk_cols_adjust(ctypes.byref(rules(**kw)), P, 2 * P, None) == T.TOPK_ERR_INVALID_ARG


def test_adjust_refuses_pointers_and_limits(lib):
    ok = ctypes.byref(rules())
    for args in ((None, P, P), (ok, None, P), (ok, P, None), (ok, P + 1, P), (ok, P, P + 1)):
        assert lib.topk_cols_adjust(*args, None) == T.TOPK_ERR_INVALID_ARG
    assert lib.topk_cols_adjust(ctypes.byref(rules(out_ld=101)), P, P, None) == T.TOPK_ERR_INVALID_ARG  # in place
    assert lib.topk_cols_adjust(ctypes.byref(rules(dtype=1)), P + 2, P, None) == T.TOPK_ERR_INVALID_ARG
    big = 1 << 24
    for kw in (dict(V=big, ld=big, out_ld=big), dict(C=1 << 31), dict(lanes=(1 << 20) + 1, col_start=P),
               dict(BIAS, n_bias=1 << 31), dict(drafts=P, n_drafts=1 << 31),
               dict(mask=P, mask_ld=4, mask_count=1 << 31)):
        assert lib.topk_cols_adjust(ctypes.byref(rules(**kw)), P, 2 * P, None) == T.TOPK_ERR_UNSUPPORTED, kw


def test_count_refuses(lib):
    good = dict(V=100, lanes=2, ids=P, n_ids=6, start=P, prompt_len=P, fresh=P, counts=P, counts_ld=100, seen=P,
                seen_ld=4)

    def call(**kw):
        return lib.topk_cols_count(*{**good, **kw}.values(), None)
    for kw in (dict(V=0), dict(lanes=0), dict(ids=None), dict(n_ids=-1), dict(start=P + 1), dict(start=None, n_ids=5),
               dict(prompt_len=P + 2), dict(fresh=P + 2), dict(counts=None), dict(counts=P + 2), dict(counts_ld=99),
               dict(seen=None), dict(seen=P + 1), dict(seen_ld=3), dict(ids=P + 1)):
        assert call(**kw) == T.TOPK_ERR_INVALID_ARG, kw
    for kw in (dict(V=1 << 24, counts_ld=1 << 24, seen_ld=1 << 20), dict(lanes=(1 << 20) + 1), dict(n_ids=1 << 31)):
        assert call(**kw) == T.TOPK_ERR_UNSUPPORTED, kw


def test_verify_refuses(lib):
    good = dict(lanes=2, dtype=0, k=8, kq=8, C=16, col_start=P, target_values=P, target_ids=P, n_drafts=14,
                draft_start=P, drafts=P, draft_values=P, draft_ids=P, temperature=1.0, top_p=0.9, seed=0, offset=0,
                max_tokens=8, out_tokens=P, out_count=P)

    def call(**kw):
        return lib.topk_cols_verify(ctypes.byref(T.VerifyArgs(**{**good, **kw})), None)
    for kw in (dict(lanes=0), dict(C=0), dict(dtype=2), dict(k=0), dict(k=65), dict(kq=0), dict(kq=65),
               dict(col_start=P + 1), dict(lanes=3, col_start=None), dict(lanes=4, draft_start=None),
               dict(target_values=None), dict(target_values=P + 1), dict(dtype=1, target_values=P + 2),
               dict(target_ids=None), dict(target_ids=P + 2), dict(n_drafts=-1), dict(drafts=None),
               dict(drafts=P + 1), dict(draft_values=None), dict(draft_ids=None), dict(draft_ids=P + 2),
               dict(draft_values=P + 1), dict(draft_start=P + 2), dict(temperature=-0.5),
               dict(temperature=float("inf")), dict(temperature=float("nan")), dict(top_p=0.0), dict(top_p=1.01),
               dict(top_p=float("nan")), dict(max_tokens=0), dict(out_tokens=None), dict(out_tokens=P + 2),
               dict(out_count=None), dict(out_count=P + 1)):
        assert call(**kw) == T.TOPK_ERR_INVALID_ARG, kw
    for kw in (dict(lanes=(1 << 20) + 1), dict(C=1 << 31), dict(n_drafts=1 << 31), dict(max_tokens=1 << 31)):
        assert call(**kw) == T.TOPK_ERR_UNSUPPORTED, kw
    assert lib.topk_cols_verify(None, None) == T.TOPK_ERR_INVALID_ARG


PLAN = dict(lanes=2, capacity=16, block_size=16, lens=P, add=P, held=P, table=P, table_ld=4, free_ids=P, n_free_ids=8,
            free_count=P, out_held=2 * P, out_free_count=2 * P, out_refused=P, out_col_start=P, out_col_lane=P,
            out_col_pos=P, out_slots=P)


def test_plan_refuses(lib):
    def call(**kw):
        return lib.topk_cols_plan(ctypes.byref(T.PlanArgs(**{**PLAN, **kw})), None)
    bad = [dict(lanes=0), dict(capacity=0), dict(block_size=0), dict(table_ld=0), dict(n_free_ids=-1),
           dict(out_held=P), dict(out_free_count=P), dict(out_slots=P + 4)]
    pointers = [n for n, t in T.PlanArgs._fields_ if t is ctypes.c_void_p]
    bad += [{n: None} for n in pointers] + [{n: P + 2} for n in pointers]
    for kw in bad:
        assert call(**kw) == T.TOPK_ERR_INVALID_ARG, kw
    for n, most in (("lanes", 1 << 20), ("capacity", 2**31 - 1), ("table_ld", 2**31 - 1), ("n_free_ids", 2**31 - 1)):
        assert call(**{n: most + 1}) == T.TOPK_ERR_UNSUPPORTED, n
    assert lib.topk_cols_plan(None, None) == T.TOPK_ERR_INVALID_ARG


def test_structures_match_the_header(tmp_path):
    """Sizes and offsets of every field, as a C compiler sees the header."""
    names = {"topk_adjust_rules": T.AdjustRulesArgs, "topk_verify_args": T.VerifyArgs, "topk_plan_args": T.PlanArgs}
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


def test_binding_refuses_tensors_that_do_not_fit():
    import torch
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):        # host tensors
        T.AdjustRules(100, 14, lanes=2, col_start=i32(3))
    with pytest.raises(ValueError):
        T.AdjustRules(100, 14, "f64")
    with pytest.raises(ValueError):        # too narrow
        T.AdjustRules(100, 14, lanes=2, counts=i32(2, 99), seen=i32(2, 4))
    with pytest.raises(ValueError):        # a lane short
        T.AdjustRules(100, 14, lanes=2, counts=i32(1, 100), seen=i32(1, 4))
    with pytest.raises(ValueError):
        T.AdjustRules(100, 14, lanes=2, bias_start=i32(3), bias_ids=i32(4), bias_values=torch.zeros(3))
    with pytest.raises(ValueError):
        T.AdjustRules(100, 14, lanes=2).apply(torch.zeros(14, 100, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        T.count_tokens(i32(2, 100), i32(1, 4), 100, i32(6))
    with pytest.raises(ValueError):
        T.verify(torch.zeros(8, 4), i32(8, 4), None, i32(7), None)
    with pytest.raises(ValueError):
        T.plan(i32(2), i32(2), i32(2), i32(1, 4), i32(4), i32(1), 16, 8)


def test_compiled_binding_refuses_before_it_calls():
    """Host tensors, wrong types and missing tensors: Python errors, no call."""
    import torch
    b = T._round_binding()
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    v = torch.zeros(8, 4)
    outs = [i32(2), i32(1), i32(1), i32(3), i32(8), i32(8), torch.zeros(8, dtype=torch.int64)]
    x = torch.zeros(14, 100, dtype=torch.bfloat16)
    calls = [
        (b.adjust, (0, 0, x, x, 2, 1400, 1400, 0)),
        (b.adjust, (0, 0, x, x, 4, 1400, 1400, 0)),
        (b.count, (0, 100, i32(2, 100), i32(2, 4), i32(6), None, None, None)),
        (b.count, (0, 100, i32(2, 100), i32(1, 4), i32(6), None, None, None)),
        (b.count, (0, 100)),
        (b.verify, (0, 1, v, i32(8, 4), None, i32(7), None, None, None, 1.0, 0.9, 0, 0, i32(1, 8), i32(1))),
        (b.verify, (0, 1, v, i32(8, 3), None, i32(7), None, None, None, 1.0, 0.9, 0, 0, i32(1, 8), i32(1))),
        (b.plan, (0, i32(2), i32(2), i32(2), i32(2, 4), i32(4), i32(1), 16, 8, *outs)),
        (b.plan, (0, i32(2), i32(2), i32(2), i32(2, 4), i32(4), i32(1), 0, 8, *outs)),
        (b.plan, (0, i32(2), i32(2), i32(2), i32(2, 4), i32(4), i32(1), 16, 1 << 40, *outs)),
    ]
    for f, args in calls:
        with pytest.raises(ValueError):
            f(*args)
    with pytest.raises(TypeError):
        b.count(0, 100, None, i32(2, 4), i32(6), None, None, None)
    with pytest.raises(TypeError):
        b.plan(0, [1, 2], i32(2), i32(2), i32(2, 4), i32(4), i32(1), 16, 8, *outs)
    with pytest.raises(TypeError):
        b.plan(0, i32(2), i32(2), i32(2), i32(2, 4), i32(4), i32(1), "16", 8, *outs)


def test_entry_points_without_a_device_fail_cleanly():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    code = ("import ctypes; from drafter_vocab_top_amd import topk_cols as T; lib = T.load();"
            "a = T.AdjustRulesArgs(V=100, C=14, lanes=2, ld=100, out_ld=100);"
            "assert lib.topk_cols_adjust(ctypes.byref(a), 64, 128, None) == T.TOPK_ERR_HIP;"
            "assert lib.topk_cols_count(100, 2, 64, 6, None, None, None, 64, 100, 64, 4, None) == T.TOPK_ERR_HIP")
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)
