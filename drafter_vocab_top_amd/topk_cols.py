"""ctypes binding of libtopk_cols.so, the HIP column-wise top-k library.

The binding only marshals arguments.  It passes raw device pointers and the
current HIP stream to the C ABI in include/topk_cols.h; every step of the
selection runs in the library's kernels.  PyTorch supplies the device buffers
and the stream.

    h = TopkCols(V, C, k, "bf16", "col", ld)
    values, ids = h.run(x)            # x: torch tensor on the GPU
    h.close()

Calls are enqueued on the current stream unless they are given one (stream=).
Outputs that a call allocates then belong to that stream, as if it were the
current one; what is passed in has to be ready there, and kept until the
call is done.

Loading fails loudly when the library is missing or cannot be loaded.  There
is no fallback path.  (The calls around the top-k go through a compiled
module, _round_binding, that reads their many tensors faster than Python does.)
"""
from __future__ import annotations

import contextlib
import ctypes
import os

LIBRARY = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtopk_cols.so")

TOPK_OK = 0
TOPK_ERR_INVALID_ARG = -1
TOPK_ERR_UNSUPPORTED = -2
TOPK_ERR_HIP = -3
TOPK_ERR_OUT_OF_MEMORY = -4
TOPK_ERR_TIMEOUT = -5
TOPK_MAX_K = 64
TOPK_MAX_V = (1 << 24) - 1

TOPK_MAX_LANES = 1 << 20

DTYPES = {"bf16": 0, "f32": 1}
LAYOUTS = {"col": 0, "row": 1}

EXPORTED = ("topk_cols_create", "topk_cols_create_with_segments", "topk_cols_create_tuned",
            "topk_cols_run", "topk_cols_run_n", "topk_cols_run_mapped", "topk_cols_sample",
            "topk_cols_destroy", "topk_cols_status_string", "topk_cols_query", "topk_cols_check",
            "topk_cols_debug_fail_waits", "topk_cols_run_noalloc", "topk_cols_adjust", "topk_cols_count",
            "topk_cols_verify", "topk_cols_plan", "topk_cols_tree", "topk_cols_cache_write", "topk_cols_cache_move",
            "topk_cols_attend", "topk_cols_attend_workspace", "topk_cols_verify_tree")
# kernel families of the column-contiguous layout ("one_wave": the baseline
# design with one wave per column and no vocabulary split)
ALGOS = {"auto": 0, "workgroup": 1, "one_wave": 3}

_lib = None


def _struct(name: str, fields: str):
    """A structure of the header, from "type name" pairs in its order."""
    types = {"p": ctypes.c_void_p, "i64": ctypes.c_int64, "i32": ctypes.c_int32, "u64": ctypes.c_uint64,
             "f64": ctypes.c_double, "f32": ctypes.c_float}
    pairs = [f.split() for f in fields.split(",")]
    return type(name, (ctypes.Structure,), {"_fields_": [(n, types[t]) for t, n in pairs]})


AdjustRulesArgs = _struct("topk_adjust_rules", (
    "i64 V, i64 C, i64 lanes, i32 dtype, i32 layout, i64 ld, i64 out_ld, p col_start, p counts, i64 counts_ld, "
    "p seen, i64 seen_ld, p repetition, p presence, p frequency, p drafts, p draft_start, i64 n_drafts, "
    "p bias_start, p bias_ids, p bias_values, i64 n_bias, p mask, i64 mask_ld, i64 mask_count, p mask_index"))
VerifyArgs = _struct("topk_verify_args", (
    "i64 lanes, i32 dtype, i32 k, i32 kq, i64 C, p col_start, p target_values, p target_ids, i64 n_drafts, "
    "p draft_start, p drafts, p draft_values, p draft_ids, f64 temperature, f64 top_p, u64 seed, u64 offset, "
    "i64 max_tokens, p out_tokens, p out_count"))
PlanArgs = _struct("topk_plan_args", (
    "i64 lanes, i64 capacity, i32 block_size, p lens, p add, p held, p table, i64 table_ld, p free_ids, "
    "i64 n_free_ids, p free_count, p out_held, p out_free_count, p out_refused, p out_col_start, p out_col_lane, "
    "p out_col_pos, p out_slots"))

CacheArgs = _struct("topk_cache", (
    "i64 layers, i64 blocks, i32 block_size, i32 heads, i32 dim, i32 format, p keys, p values, i64 layer_stride, "
    "i64 block_stride, i64 slot_stride, i64 head_stride, p key_scales, p value_scales, i64 scale_layer_stride, "
    "i64 scale_block_stride, i64 scale_slot_stride, i64 scale_head_stride"))
CacheWriteArgs = _struct("topk_cache_write_args", (
    "i64 C, i64 layer, i32 dtype, p keys, p values, i64 key_stride, i64 key_head_stride, i64 value_stride, "
    "i64 value_head_stride, p slots"))
AttendArgs = _struct("topk_attend_args", (
    "i64 lanes, i64 C, i64 layer, i32 heads, i32 window, f32 scale, p q, i64 q_stride, i64 q_head_stride, p col_start, "
    "p lens, p table, i64 table_ld, p mask, i64 mask_ld, p positions, p out, i64 out_stride, i64 out_head_stride, "
    "p workspace, i64 workspace_bytes"))
VerifyTreeArgs = _struct("topk_verify_tree_args", (
    "i64 lanes, i32 dtype, i32 k, i32 kq, i64 C, p col_start, p target_values, p target_ids, p tokens, p parents, "
    "p draft_values, p draft_ids, p uniforms, f64 temperature, f64 top_p, i64 max_tokens, p out_tokens, p out_columns, "
    "p out_count"))


class TopkError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def load(path: str = LIBRARY):
    """Load the library (once) and declare its C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise OSError(f"{path} is missing: build it with `python -m drafter_vocab_top_amd.build`")
    lib = ctypes.CDLL(path)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.topk_cols_create.argtypes = [ctypes.POINTER(p), i64, i64, i32, i32, i32, i64]
    lib.topk_cols_create.restype = ctypes.c_int
    lib.topk_cols_create_with_segments.argtypes = [ctypes.POINTER(p), i64, i64, i32, i32, i32, i64, i64]
    lib.topk_cols_create_with_segments.restype = ctypes.c_int
    lib.topk_cols_create_tuned.argtypes = [ctypes.POINTER(p), i64, i64, i32, i32, i32, i64, i64, i32]
    lib.topk_cols_create_tuned.restype = ctypes.c_int
    lib.topk_cols_run.argtypes = [p, p, p, p, p]
    lib.topk_cols_run.restype = ctypes.c_int
    lib.topk_cols_run_n.argtypes = [p, i64, p, p, p, p]
    lib.topk_cols_run_n.restype = ctypes.c_int
    lib.topk_cols_run_mapped.argtypes = [p, i64, p, p, p, p, p]
    lib.topk_cols_run_mapped.restype = ctypes.c_int
    lib.topk_cols_sample.argtypes = [p, p, i64, i32, i32, ctypes.c_double, ctypes.c_double,
                                     ctypes.c_uint64, ctypes.c_uint64, p, p, p]
    lib.topk_cols_sample.restype = ctypes.c_int
    lib.topk_cols_destroy.argtypes = [p]
    lib.topk_cols_destroy.restype = ctypes.c_int
    lib.topk_cols_status_string.argtypes = [ctypes.c_int]
    lib.topk_cols_status_string.restype = ctypes.c_char_p
    lib.topk_cols_query.argtypes = [p, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i64),
                                    ctypes.POINTER(i32)]
    lib.topk_cols_query.restype = ctypes.c_int
    lib.topk_cols_check.argtypes = [p]
    lib.topk_cols_check.restype = ctypes.c_int
    lib.topk_cols_debug_fail_waits.argtypes = [p, i32]
    lib.topk_cols_debug_fail_waits.restype = ctypes.c_int
    lib.topk_cols_run_noalloc.argtypes = [i64, i64, i32, i32, i32, i64, p, p, p, p]
    lib.topk_cols_run_noalloc.restype = ctypes.c_int
    lib.topk_cols_adjust.argtypes = [p, p, p, p]
    lib.topk_cols_adjust.restype = ctypes.c_int
    lib.topk_cols_count.argtypes = [i64, i64, p, i64, p, p, p, p, i64, p, i64, p]
    lib.topk_cols_count.restype = ctypes.c_int
    lib.topk_cols_verify.argtypes = [p, p]
    lib.topk_cols_verify.restype = ctypes.c_int
    lib.topk_cols_plan.argtypes = [p, p]
    lib.topk_cols_plan.restype = ctypes.c_int
    lib.topk_cols_tree.argtypes = [i64, i64, p, p, p, p, i64, p, p]
    lib.topk_cols_tree.restype = ctypes.c_int
    lib.topk_cols_cache_write.argtypes = [p, p, p]
    lib.topk_cols_cache_write.restype = ctypes.c_int
    lib.topk_cols_cache_move.argtypes = [p, i64, p, p, i64, p, i64, p]
    lib.topk_cols_cache_move.restype = ctypes.c_int
    lib.topk_cols_attend.argtypes = [p, p, p]
    lib.topk_cols_attend.restype = ctypes.c_int
    lib.topk_cols_attend_workspace.argtypes = [p, p, ctypes.POINTER(i64)]
    lib.topk_cols_attend_workspace.restype = ctypes.c_int
    lib.topk_cols_verify_tree.argtypes = [p, p]
    lib.topk_cols_verify_tree.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().topk_cols_status_string(int(status)).decode()


def _torch_dtype(dtype: str):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


_HERE = contextlib.nullcontext()


def _allocate(stream):
    """A context in which outputs are allocated for a call on `stream` (None:
    the current one): from that stream's memory.  Memory of another stream
    may still be in use there, and goes back to it as soon as the tensor is
    dropped, with the call still writing."""
    if stream is None:
        return _HERE
    import torch
    return torch.cuda.stream(stream)


class TopkCols:
    """One top-k shape on the current GPU (a handle of the C library)."""

    def __init__(self, V: int, C: int, k: int, dtype: str = "bf16", layout: str = "col",
                 ld: int | None = None, segments: int = 0, algo: str = "auto"):
        if dtype not in DTYPES or layout not in LAYOUTS or algo not in ALGOS:
            raise ValueError(f"dtype must be one of {list(DTYPES)}, layout one of {list(LAYOUTS)}, "
                             f"algo one of {list(ALGOS)}")
        self.V, self.C, self.k, self.dtype, self.layout = V, C, k, dtype, layout
        self.ld = ld if ld is not None else (V if layout == "col" else C)
        lib = load()
        self._h = ctypes.c_void_p()
        if segments == 0 and algo == "auto":
            rc = lib.topk_cols_create(ctypes.byref(self._h), V, C, k, DTYPES[dtype], LAYOUTS[layout], self.ld)
        else:
            rc = lib.topk_cols_create_tuned(ctypes.byref(self._h), V, C, k, DTYPES[dtype],
                                            LAYOUTS[layout], self.ld, segments, ALGOS[algo])
        if rc != TOPK_OK:
            raise TopkError(rc, "topk_cols_create")

    def query(self) -> dict:
        s, b, w, a = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32()
        rc = load().topk_cols_query(self._h, ctypes.byref(s), ctypes.byref(b), ctypes.byref(w), ctypes.byref(a))
        if rc != TOPK_OK:
            raise TopkError(rc, "topk_cols_query")
        names = {v: n for n, v in ALGOS.items()}
        return {"segments": s.value, "blocks": b.value, "workspace_bytes": w.value, "algo": names.get(a.value)}

    def check(self) -> int:
        """topk_cols_check: synchronizes the device; TOPK_OK, or TOPK_ERR_TIMEOUT
        when a run's cross-workgroup wait gave up (the workspace is then reset)."""
        rc = load().topk_cols_check(self._h)
        if rc not in (TOPK_OK, TOPK_ERR_TIMEOUT):
            raise TopkError(rc, "topk_cols_check")
        return rc

    def debug_fail_waits(self, on: bool) -> None:
        """Tests of the error path only (topk_cols_debug_fail_waits)."""
        rc = load().topk_cols_debug_fail_waits(self._h, 1 if on else 0)
        if rc != TOPK_OK:
            raise TopkError(rc, "topk_cols_debug_fail_waits")

    def run_ptr(self, x_ptr: int, values_ptr: int, ids_ptr: int, stream_ptr: int,
                n_cols: int | None = None, id_map_ptr: int | None = None) -> None:
        """Enqueue one run on raw device pointers and a raw HIP stream handle.

        n_cols: active columns (topk_cols_run_n); None runs all C columns.
        id_map_ptr: device row -> id table (topk_cols_run_mapped), or None.
        """
        lib = load()
        if id_map_ptr is not None:
            rc = lib.topk_cols_run_mapped(self._h, self.C if n_cols is None else n_cols, x_ptr, id_map_ptr,
                                          values_ptr, ids_ptr, stream_ptr)
            what = "topk_cols_run_mapped"
        elif n_cols is not None:
            rc = lib.topk_cols_run_n(self._h, n_cols, x_ptr, values_ptr, ids_ptr, stream_ptr)
            what = "topk_cols_run_n"
        else:
            rc = lib.topk_cols_run(self._h, x_ptr, values_ptr, ids_ptr, stream_ptr)
            what = "topk_cols_run"
        if rc != TOPK_OK:
            raise TopkError(rc, what)

    def run(self, x, values=None, ids=None, stream=None, n_cols: int | None = None, id_map=None):
        """Enqueue one run on torch tensors (on the current stream by default).

        x: GPU tensor holding the matrix (bf16 or fp32, or int16/uint16/int32
           bit patterns of the same width), laid out as given at creation.
        values/ids: optional preallocated outputs (C*k elements each).
        n_cols: select over the first n_cols columns only (None: all C).
        id_map: optional int32 GPU tensor of V entries; the ids returned are
           id_map[row] (selection and tie order are unchanged).
        Returns (values, ids) shaped (C, k); with n_cols, rows n_cols.. of
        freshly allocated outputs are left uninitialised.
        """
        import torch
        if not x.is_cuda:
            raise ValueError("x must be a GPU tensor")
        need = (self.C - 1) * self.ld + self.V if self.layout == "col" else (self.V - 1) * self.ld + self.C
        if x.numel() < need or x.element_size() != (2 if self.dtype == "bf16" else 4):
            raise ValueError("x does not hold the matrix described at creation")
        if not x.is_contiguous():
            raise ValueError("x must be contiguous")
        if values is None or ids is None:
            with _allocate(stream):
                if values is None:
                    values = torch.empty((self.C, self.k), dtype=x.dtype, device=x.device)
                if ids is None:
                    ids = torch.empty((self.C, self.k), dtype=torch.int32, device=x.device)
        if values.numel() < self.C * self.k or ids.numel() < self.C * self.k:
            raise ValueError("output buffers are too small")
        map_ptr = None
        if id_map is not None:
            if not id_map.is_cuda or id_map.dtype != torch.int32 or id_map.numel() < self.V \
                    or not id_map.is_contiguous():
                raise ValueError("id_map must be a contiguous int32 GPU tensor of V entries")
            map_ptr = id_map.data_ptr()
        s = stream if stream is not None else torch.cuda.current_stream(x.device)
        self.run_ptr(x.data_ptr(), values.data_ptr(), ids.data_ptr(), s.cuda_stream, n_cols, map_ptr)
        return values, ids

    def close(self) -> None:
        if getattr(self, "_h", None) and self._h.value:
            rc = load().topk_cols_destroy(self._h)
            self._h = ctypes.c_void_p()
            if rc != TOPK_OK:
                raise TopkError(rc, "topk_cols_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def sample(values, ids, temperature: float = 1.0, top_p: float = 0.95, seed: int = 0, offset: int = 0,
           out_ids=None, out_pos=None, stream=None):
    """One sampled draft per column from top-k outputs (topk_cols_sample).

    values: (C, k) GPU tensor as a run wrote it (bf16 or fp32, or 16/32-bit
    patterns); ids: (C, k) int32 GPU tensor.  Returns (ids, positions), each
    (C,) int32 on the GPU; enqueued on the current stream by default.
    """
    import torch
    if values.dim() != 2 or ids.shape != values.shape or ids.dtype != torch.int32:
        raise ValueError("values and ids must be (C, k) tensors, ids int32")
    if not (values.is_cuda and ids.is_cuda and values.is_contiguous() and ids.is_contiguous()):
        raise ValueError("values and ids must be contiguous GPU tensors")
    C, k = values.shape
    dtype = 0 if values.element_size() == 2 else 1
    if out_ids is None or out_pos is None:
        with _allocate(stream):
            if out_ids is None:
                out_ids = torch.empty(C, dtype=torch.int32, device=values.device)
            if out_pos is None:
                out_pos = torch.empty(C, dtype=torch.int32, device=values.device)
    s = stream if stream is not None else torch.cuda.current_stream(values.device)
    rc = load().topk_cols_sample(values.data_ptr(), ids.data_ptr(), C, k, dtype, float(temperature),
                                 float(top_p), int(seed), int(offset), out_ids.data_ptr(), out_pos.data_ptr(),
                                 s.cuda_stream)
    if rc != TOPK_OK:
        raise TopkError(rc, "topk_cols_sample")
    return out_ids, out_pos


def run_noalloc(x, V: int, C: int, k: int, dtype: str = "bf16", layout: str = "col", ld=None,
                values=None, ids=None, stream=None):
    """topk_cols_run_noalloc: one run with no handle and no device allocation
    by the library (the outputs are allocated here when not given).  Returns
    (values, ids) shaped (C, k); enqueued on the current stream by default."""
    import torch
    if dtype not in DTYPES or layout not in LAYOUTS:
        raise ValueError(f"dtype must be one of {list(DTYPES)}, layout one of {list(LAYOUTS)}")
    ld = ld if ld is not None else (V if layout == "col" else C)
    if not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous GPU tensor")
    need = (C - 1) * ld + V if layout == "col" else (V - 1) * ld + C
    if x.numel() < need or x.element_size() != (2 if dtype == "bf16" else 4):
        raise ValueError("x does not hold the matrix described")
    if values is None or ids is None:
        with _allocate(stream):
            if values is None:
                values = torch.empty((C, k), dtype=x.dtype, device=x.device)
            if ids is None:
                ids = torch.empty((C, k), dtype=torch.int32, device=x.device)
    if values.numel() < C * k or ids.numel() < C * k:
        raise ValueError("output buffers are too small")
    s = stream if stream is not None else torch.cuda.current_stream(x.device)
    rc = load().topk_cols_run_noalloc(V, C, k, DTYPES[dtype], LAYOUTS[layout], ld, x.data_ptr(), values.data_ptr(),
                                      ids.data_ptr(), s.cuda_stream)
    if rc != TOPK_OK:
        raise TopkError(rc, "topk_cols_run_noalloc")
    return values, ids


def _need(name: str, t, numel: int, index: int, dtype) -> int:
    """Address of a contiguous tensor of at least numel elements on GPU
    `index` (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != index or t.numel() < numel or not t.is_contiguous() or index < 0:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of at least {numel} elements on GPU {index}")
    return t.data_ptr()


_round = None


def _round_binding():
    """The compiled part of the binding: it takes tensors apart for
    AdjustRules.apply, count_tokens, verify, plan, tree, verify_tree and
    KeyCache, and calls the loaded library."""
    global _round
    if _round is None:
        import torch  # noqa: F401  (the module needs its libraries in the process)
        lib = load()
        try:
            from . import _round_binding as module
        except ImportError as e:
            raise OSError(f"_round_binding is missing or does not load ({e}): build it with "
                          "`python -m drafter_vocab_top_amd.build`") from e
        from . import build
        if module.built_for != build.built_for():
            raise OSError(f"_round_binding was built for {module.built_for}, this is {build.built_for()}: build it again "
                          "with `python -m drafter_vocab_top_amd.build`")
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                      for f in (lib.topk_cols_adjust, lib.topk_cols_count, lib.topk_cols_verify, lib.topk_cols_plan,
                                lib.topk_cols_tree, lib.topk_cols_cache_write, lib.topk_cols_cache_move, lib.topk_cols_attend,
                                lib.topk_cols_attend_workspace, lib.topk_cols_verify_tree)))
        _round = module
    return _round


def _raw_stream(index: int, stream) -> int:
    """The raw handle of a stream, by default the current one of GPU `index`."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    if index < 0:
        raise ValueError("the tensors must be on a GPU")
    return torch._C._cuda_getCurrentRawStream(index)


def _launch(what: str, function, index: int, *args) -> None:
    """function(*args) with GPU `index` current."""
    import torch
    if index < 0:
        raise ValueError("the tensors must be on a GPU")
    if index == torch._C._cuda_getDevice():
        rc = function(*args)
    else:
        with torch.cuda.device(index):
            rc = function(*args)
    if rc != TOPK_OK:
        raise TopkError(rc, what)


def history(V: int, lanes: int, device="cuda"):
    """Empty token histories of `lanes` lanes: (counts, seen) as AdjustRules
    reads and count_tokens updates them, zeroed int32 tensors (lanes, V) and
    (lanes, ceil(V / 32))."""
    import torch
    return (torch.zeros((lanes, V), dtype=torch.int32, device=device),
            torch.zeros((lanes, (V + 31) // 32), dtype=torch.int32, device=device))


class AdjustRules:
    """Penalties, biases and masks for logits (topk_cols_adjust).

    Describes buffers that the caller keeps (and may update between calls):
    the object holds references to the tensors and no state of its own.  All
    are contiguous GPU tensors on one device, int32 unless said otherwise.

    V, C, dtype, layout, ld: the matrix, as for TopkCols; out_ld: the
        result's leading dimension (default: ld).
    lanes, col_start: lane l owns columns col_start[l]..col_start[l+1]-1
        (lanes + 1 entries), or C / lanes each without col_start.
    counts (lanes, >= V), seen (lanes, >= ceil(V/32)): histories.
    repetition, presence, frequency: (lanes,) float32.
    drafts, draft_start: token ids of the lanes' drafts, packed; column j of
        a lane takes its first j drafts as further output.
    bias_start, bias_ids, bias_values (float32): packed lists per lane.
    mask (masks, >= ceil(V/32)): bit r % 32 of word r / 32 allows row r;
        mask_index (C,): the mask of each column, none where it is outside
        the range (without it: mask c for column c).
    """

    def __init__(self, V: int, C: int, dtype: str = "bf16", layout: str = "col", ld: int | None = None,
                 out_ld: int | None = None, lanes: int = 1, col_start=None, counts=None, seen=None, repetition=None,
                 presence=None, frequency=None, drafts=None, draft_start=None, bias_start=None, bias_ids=None,
                 bias_values=None, mask=None, mask_index=None):
        if dtype not in DTYPES or layout not in LAYOUTS:
            raise ValueError(f"dtype must be one of {list(DTYPES)}, layout one of {list(LAYOUTS)}")
        self.V, self.C, self.dtype, self.layout = V, C, dtype, layout
        self.ld = ld if ld is not None else (V if layout == "col" else C)
        self.out_ld = out_ld if out_ld is not None else self.ld
        self._tensors = tensors = dict(
            col_start=col_start, counts=counts, seen=seen, repetition=repetition, presence=presence,
            frequency=frequency, drafts=drafts, draft_start=draft_start, bias_start=bias_start, bias_ids=bias_ids,
            bias_values=bias_values, mask=mask, mask_index=mask_index)
        import torch
        devices = {t.get_device() for t in tensors.values() if t is not None}
        if len(devices) > 1:
            raise ValueError("the rules' tensors must be on one GPU")
        self._index = devices.pop() if devices else None
        words = (V + 31) // 32
        for name, t, least in (("counts", counts, V), ("seen", seen, words), ("mask", mask, words)):
            if t is not None and (t.dim() != 2 or t.shape[1] < least or (name != "mask" and t.shape[0] < lanes)):
                raise ValueError(f"{name} must be a matrix with rows of at least {least} entries"
                                 + ("" if name == "mask" else " for every lane"))
        if mask is not None and mask.shape[0] == 0:  # (its address is NULL, which means no mask)
            raise ValueError("mask must have at least one row")
        if (bias_ids is None) != (bias_values is None) or \
                (bias_ids is not None and bias_ids.numel() != bias_values.numel()):
            raise ValueError("bias_ids and bias_values must have the same length")
        sizes = dict(col_start=lanes + 1, repetition=lanes, presence=lanes, frequency=lanes, draft_start=lanes + 1,
                     bias_start=lanes + 1, mask_index=C)
        floats = ("repetition", "presence", "frequency", "bias_values")
        at = {n: _need(n, t, sizes.get(n, 0), self._index, torch.float32 if n in floats else torch.int32)
              for n, t in tensors.items()}
        # an empty tensor has no address; an empty list is the same as none
        if bias_ids is not None and bias_ids.numel() == 0:
            at.update(bias_start=0, bias_ids=0, bias_values=0)
        if drafts is not None and drafts.numel() == 0:
            at.update(drafts=0, draft_start=0)
        self._args = AdjustRulesArgs(
            V=V, C=C, lanes=lanes, dtype=DTYPES[dtype], layout=LAYOUTS[layout], ld=self.ld, out_ld=self.out_ld,
            counts_ld=counts.shape[1] if counts is not None else 0, seen_ld=seen.shape[1] if seen is not None else 0,
            n_drafts=drafts.numel() if drafts is not None else 0,
            n_bias=bias_ids.numel() if bias_ids is not None else 0,
            mask_ld=mask.shape[1] if mask is not None else 0, mask_count=mask.shape[0] if mask is not None else 0, **at)
        self._address = ctypes.addressof(self._args)
        self._size = 2 if dtype == "bf16" else 4
        rows, width = (C, V) if layout == "col" else (V, C)
        self._numel = (rows - 1) * self.ld + width
        self._out_numel = (rows - 1) * self.out_ld + width

    def apply(self, x, out=None, stream=None):
        """Enqueue the rules on logits x; returns out (allocated like x when
        not given: its padding, and columns of no lane, are then
        uninitialised).  out=x works in place.  x and out are contiguous GPU
        tensors of the matrix (bf16 or fp32, or patterns of the same width)."""
        if out is None:
            import torch
            if self.out_ld != self.ld:
                raise ValueError("out is needed when out_ld differs from ld")
            with _allocate(stream):
                out = torch.empty_like(x)
        index = x.get_device()
        if self._index not in (None, index):
            raise ValueError("x, out and the rules' tensors must be on one GPU")
        _launch("topk_cols_adjust", _round_binding().adjust, index, _raw_stream(index, stream), self._address, x, out,
                self._size, self._numel, self._out_numel, index)
        return out


def count_tokens(counts, seen, V: int, ids, start=None, prompt_len=None, fresh=None, stream=None):
    """Add packed token ids to the lanes' histories (topk_cols_count).

    counts (lanes, >= V), seen (lanes, >= ceil(V/32)): int32, updated in place.
    ids: int32; lane l's are ids[start[l]:start[l+1]] (evenly many without
        start).  Ids outside [0, V) are skipped.
    prompt_len (lanes,): how many of a lane's tokens, from the first, are
        prompt (none without it).  fresh (lanes,): lanes to clear first.
    Returns (counts, seen).
    """
    index = counts.get_device()
    _launch("topk_cols_count", _round_binding().count, index, _raw_stream(index, stream), V, counts, seen, ids, start,
            prompt_len, fresh)
    return counts, seen


def verify(target_values, target_ids, col_start, drafts, draft_start, draft_values=None, draft_ids=None,
           temperature: float = 1.0, top_p: float = 0.95, seed: int = 0, offset: int = 0, lanes: int | None = None,
           max_tokens: int | None = None, out_tokens=None, out_count=None, stream=None):
    """Verify drafts against the target's top-k lists (topk_cols_verify).

    target_values, target_ids: (C, k), as a run on the target's logits wrote
        them; lane l's columns are col_start[l]..col_start[l+1]-1 (one more
        than its drafts).
    drafts: packed token ids, lane l's at draft_start[l]..draft_start[l+1]-1.
    draft_values, draft_ids: (n, kq), the lists the drafts were sampled from;
        without them drafts count as certain (greedy drafts).  Drafts past the
        n lists are not judged (the padding of a buffer); without draft_start
        there must be a list for every draft.
    temperature 0 verifies greedily.  col_start and draft_start None: the same
        number for each of `lanes` lanes.
    Returns (tokens, count): lane l commits tokens[l, :count[l]], the accepted
    drafts and one token more; -1 follows.  max_tokens: the row length when
    out_tokens is not given (default: one more than all drafts, which is
    enough for any lane; pass the round's draft limit + 1).
    """
    index = target_values.get_device()
    if lanes is None:
        if col_start is None:
            raise ValueError("lanes is needed without col_start")
        lanes = col_start.numel() - 1
    if out_tokens is None or out_count is None:
        import torch
        with _allocate(stream):
            if out_tokens is None:
                out_tokens = torch.empty((lanes, max_tokens or drafts.numel() + 1), dtype=torch.int32,
                                         device=target_values.device)
            if out_count is None:
                out_count = torch.empty(lanes, dtype=torch.int32, device=target_values.device)
    _launch("topk_cols_verify", _round_binding().verify, index, _raw_stream(index, stream), lanes, target_values, target_ids,
            col_start, drafts, draft_start, draft_values, draft_ids, temperature, top_p, seed, offset, out_tokens, out_count)
    return out_tokens, out_count


def plan(lens, add, held, table, free_ids, free_count, block_size: int, capacity: int, out=None, stream=None) -> dict:
    """Plan a round: columns, cache blocks and slots (topk_cols_plan).

    lens, add, held: (lanes,) int32, the lanes' tokens in the cache, the
        columns they want and the blocks they hold.
    table: (lanes, width) int32 block ids, extended in place.
    free_ids: int32 stack of free blocks, its first free_count[0] are free.
    capacity: columns of the round, at most.
    Returns a dict (or fills `out`, one an earlier call returned) of int32
    tensors held (lanes,), free_count (1,), refused (1,), col_start
    (lanes + 1,), col_lane, col_pos (capacity,) and int64 slots (capacity,).
    """
    index = lens.get_device()
    if out is None:
        import torch
        lanes = lens.numel()
        sizes = dict(held=lanes, free_count=1, refused=1, col_start=lanes + 1, col_lane=capacity, col_pos=capacity,
                     slots=capacity)
        with _allocate(stream):
            out = {n: torch.empty(size, dtype=torch.int64 if n == "slots" else torch.int32, device=lens.device)
                   for n, size in sizes.items()}
    _launch("topk_cols_plan", _round_binding().plan, index, _raw_stream(index, stream), lens, add, held, table, free_ids,
            free_count, block_size, capacity, out["held"], out["free_count"], out["refused"], out["col_start"],
            out["col_lane"], out["col_pos"], out["slots"])
    return out


def tree(parents, lens=None, col_start=None, lanes: int | None = None, words: int | None = None, mask=None,
         positions=None, stream=None):
    """Masks and positions of a round's trees (topk_cols_tree).

    parents (C,): int32, for each column the column of its lane that it
        follows (-1: none, as for a lane's column 0).
    lens (lanes,): int32, the lanes' tokens before their columns (0 without).
    col_start (lanes + 1,), or C / lanes columns for each of `lanes` lanes.
    words: 32-bit words of a mask's row when mask is not given, at least a
        32nd of the columns that a lane can have (default: C / 32).
    Returns (mask, positions): int32 (C, words), bit i % 32 of word i / 32 set
    for column i itself and its ancestors, and int32 (C,).  Rows of columns of
    no lane are not written.
    """
    index = parents.get_device()
    lanes = _lanes(col_start, lanes, lens)
    if mask is None or positions is None:
        import torch
        C = parents.numel()
        with _allocate(stream):
            if mask is None:
                mask = torch.empty((C, words or (C + 31) // 32), dtype=torch.int32, device=parents.device)
            if positions is None:
                positions = torch.empty(C, dtype=torch.int32, device=parents.device)
    _launch("topk_cols_tree", _round_binding().tree, index, _raw_stream(index, stream), lanes, parents, lens, col_start, mask,
            positions)
    return mask, positions


def verify_tree(target_values, target_ids, col_start, tokens, parents, uniforms, draft_values=None, draft_ids=None,
                temperature: float = 1.0, top_p: float = 0.95, lanes: int | None = None, max_tokens: int | None = None,
                out_tokens=None, out_columns=None, out_count=None, stream=None):
    """Verify trees of drafts against the target's top-k lists
    (topk_cols_verify_tree).

    target_values, target_ids: (C, k), as a run on the target's logits wrote
        them; lane l's columns are col_start[l]..col_start[l+1]-1, the first
        its anchor (col_start None: the same number for each of `lanes`).
    tokens, parents: (C,) int32, each column's token and the column that it
        follows (see tree).
    uniforms: (C, 2) float32 in [0, 1): the first judges the column's draft, the
        second draws the token behind the column.
    draft_values, draft_ids: (C, kq), row c the list that the children of column
        c were sampled from; without them drafts count as certain.
    Returns (tokens, columns, count): lane l commits tokens[l, :count[l]], the
    accepted drafts and one token more; columns[l, :count[l]] are the columns
    whose keys stay (KeyCache.move), the anchor's first; -1 follows.  max_tokens:
    the row length when outputs are not given (default: C; pass the deepest path
    + 1).
    """
    index = target_values.get_device()
    lanes = _lanes(col_start, lanes)
    if out_tokens is None or out_columns is None or out_count is None:
        import torch
        device = target_values.device
        given = out_tokens if out_tokens is not None else out_columns
        width = given.shape[-1] if given is not None else max_tokens or target_values.shape[0]
        with _allocate(stream):
            if out_tokens is None:
                out_tokens = torch.empty((lanes, width), dtype=torch.int32, device=device)
            if out_columns is None:
                out_columns = torch.empty((lanes, width), dtype=torch.int32, device=device)
            if out_count is None:
                out_count = torch.empty(lanes, dtype=torch.int32, device=device)
    _launch("topk_cols_verify_tree", _round_binding().verify_tree, index, _raw_stream(index, stream), lanes, target_values,
            target_ids, col_start, tokens, parents, uniforms, draft_values, draft_ids, temperature, top_p, out_tokens,
            out_columns, out_count)
    return out_tokens, out_columns, out_count


def _lanes(col_start, lanes, per_lane=None) -> int:
    if lanes is not None:
        return lanes
    if col_start is not None:
        return col_start.numel() - 1
    if per_lane is not None:
        return per_lane.numel()
    raise ValueError("lanes is needed without col_start")


class KeyCache:
    """A paged cache of keys and values (topk_cache), whose slots plan gives out.

    Describes tensors that the caller keeps: the object holds references to
    them and no state of its own.  All are on one GPU.

    keys, values: (layers, blocks, block_size, heads, dim), or without the
        first for one layer; bfloat16, or float8_e4m3fn.  Any strides that are
        multiples of 16 bytes (so heads may also lie outside of a block's
        slots), the last 1; the same for both.  dim: a multiple of 16, at most
        256.
    key_scales, value_scales: with float8_e4m3fn, uint8 (or float8_e8m0fnu) of
        the shape without dim, any strides, the same for both: a row stands for
        its elements times 2^(scale - 127), with 255 for NaN.
    """

    def __init__(self, keys, values, key_scales=None, value_scales=None):
        import torch
        formats = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}
        if keys.dim() not in (4, 5) or values.shape != keys.shape or keys.dtype not in formats \
                or values.dtype != keys.dtype or keys.numel() == 0:
            raise ValueError("keys and values must be (layers, blocks, block_size, heads, dim) tensors, bfloat16 or "
                             "float8_e4m3fn")
        fp8 = keys.dtype == torch.float8_e4m3fn
        if (key_scales is None) == fp8 or (value_scales is None) == fp8:
            raise ValueError("float8_e4m3fn needs key_scales and value_scales, bfloat16 has none")
        self._tensors = tensors = [t for t in (keys, values, key_scales, value_scales) if t is not None]
        self._index = keys.get_device()
        if self._index < 0 or any(t.get_device() != self._index for t in tensors):
            raise ValueError("the cache's tensors must be on one GPU")
        if fp8 and any(t.shape != keys.shape[:-1] or t.dtype not in (torch.uint8, torch.float8_e8m0fnu)
                       for t in (key_scales, value_scales)):
            raise ValueError("scales must be uint8 tensors of the keys' shape without dim")
        shape = tuple(keys.shape) if keys.dim() == 5 else (1, *keys.shape)
        self.layers, self.blocks, self.block_size, self.heads, self.dim = shape
        if max(shape[2:]) > 2**31 - 1:  # (their fields are 32-bit numbers)
            raise ValueError("block_size, heads and dim must be at most 2^31 - 1")

        def strides(a, b, what):
            # (a dimension of one entry has no stride)
            s, t = ([0 if n == 1 else st for n, st in zip(x.shape, x.stride())] for x in (a, b))
            if s != t:
                raise ValueError(f"{what} must have the same strides")
            return s if a.dim() == len(shape) - (what == "scales") else [0, *s]

        layer, block, slot, head, last = strides(keys, values, "keys and values")
        unit = 16 // keys.element_size()
        if last != 1 or any(s % unit for s in (layer, block, slot, head)):
            raise ValueError("keys and values must have strides of multiples of 16 bytes, the last 1")
        scale = strides(key_scales, value_scales, "scales") if fp8 else [0, 0, 0, 0]
        self._args = CacheArgs(
            layers=self.layers, blocks=self.blocks, block_size=self.block_size, heads=self.heads, dim=self.dim,
            format=formats[keys.dtype], keys=keys.data_ptr(), values=values.data_ptr(), layer_stride=layer,
            block_stride=block, slot_stride=slot, head_stride=head,
            key_scales=key_scales.data_ptr() if fp8 else 0, value_scales=value_scales.data_ptr() if fp8 else 0,
            scale_layer_stride=scale[0], scale_block_stride=scale[1], scale_slot_stride=scale[2], scale_head_stride=scale[3])
        self._address = ctypes.addressof(self._args)

    def write(self, k, v, slots, layer: int = 0, stream=None) -> None:
        """Write the columns' keys and values, (C, heads, dim) bf16 or fp32 with
        any strides of multiples of 16 bytes (the last 1), into the slots (C,)
        int64 that plan gave them; negative slots (the padding) are skipped
        (topk_cols_cache_write)."""
        _launch("topk_cols_cache_write", _round_binding().cache_write, self._index, _raw_stream(self._index, stream),
                self._address, self._index, k, v, slots, layer)

    def attend(self, q, lens, table, col_start=None, mask=None, positions=None, window: int = 0, scale=None,
               layer: int = 0, out=None, stream=None):
        """Attention of the columns over their lanes' tokens and ancestors
        (topk_cols_attend); returns out.

        q: (C, query heads, dim) bf16, any strides of multiples of 16 bytes (the
            last 1); query head h reads key head h / (query heads / heads).
        lens (lanes,), table (lanes, width): int32, as plan takes them: the
            tokens before this round's, and the lanes' blocks.
        col_start (lanes + 1,), or the same number of columns for each lane.
        mask, positions: as tree gives them.  Without a mask the columns are a
            chain (or a prompt); without positions column j's is lens + j.
        window: only this many places up to the column's own, 0 for all: of the
            lane's tokens those less than window before its position, and
            without a mask of the columns likewise.  A mask says by itself
            which columns are seen: ancestors whose bits are set are, at any
            distance.
        scale: of the products, default dim ** -0.5.
        out: like q, overlapping neither q nor the cache (default: allocated;
            columns of no lane are then uninitialised).
        """
        if scale is None:
            scale = self.dim ** -0.5
        if out is None:
            import torch
            with _allocate(stream):
                out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        with _allocate(stream):  # (the workspace)
            _launch("topk_cols_attend", _round_binding().attend, self._index, _raw_stream(self._index, stream),
                    self._address, self._index, q, lens, table, col_start, mask, positions, window, scale, layer, out)
        return out

    def move(self, lens, table, columns, stream=None) -> None:
        """Close up the accepted paths, in all layers (topk_cols_cache_move):
        what lies at place lens[l] + columns[l, i] of lane l goes to lens[l] + i.
        columns (lanes, width): int32, as verify_tree gives them; lens (lanes,)
        and table as for attend (lens without the accepted tokens)."""
        _launch("topk_cols_cache_move", _round_binding().cache_move, self._index, _raw_stream(self._index, stream),
                self._address, self._index, lens, table, columns)


def topk_cols(x, V: int, C: int, k: int, dtype: str = "bf16", layout: str = "col", ld=None):
    """One-shot convenience: create, run, synchronize, destroy."""
    import torch
    with TopkCols(V, C, k, dtype, layout, ld) as h:
        v, i = h.run(x)
        torch.cuda.current_stream(x.device).synchronize()
        return v, i
