// CPython module behind AdjustRules.apply, count_tokens, verify, plan, tree,
// verify_tree and KeyCache of the binding: takes their tensors apart, checks
// them and calls the C ABI.
//
// A round's calls run kernels of 3 to 5 us; checking a dozen tensors from
// Python takes as long.  Reading them here takes a call from 7 - 9 us to 4 - 5,
// of which the runtime's launch is 2.6.  Nothing else happens here, but for the
// workspace of attend: the checks are the binding's (each tensor's type,
// device, size and contiguity), every other argument is checked by the library.
//
// The library's functions are bound at load time (bind), so that the binding
// keeps choosing which library is in use.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include "topk_cols.h"

namespace {

decltype(&topk_cols_adjust) g_adjust = nullptr;
decltype(&topk_cols_count) g_count = nullptr;
decltype(&topk_cols_verify) g_verify = nullptr;
decltype(&topk_cols_plan) g_plan = nullptr;
decltype(&topk_cols_tree) g_tree = nullptr;
decltype(&topk_cols_cache_write) g_cache_write = nullptr;
decltype(&topk_cols_cache_move) g_cache_move = nullptr;
decltype(&topk_cols_attend) g_attend = nullptr;
decltype(&topk_cols_attend_workspace) g_attend_workspace = nullptr;
decltype(&topk_cols_verify_tree) g_verify_tree = nullptr;

struct Failed {};  // a Python error is set

[[noreturn]] void fail(const char* what) {
    PyErr_SetString(PyExc_ValueError, what);
    throw Failed{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw Failed{};
    }
    return THPVariable_Unpack(o);
}

bool fits(const at::Tensor& t, int64_t numel, int index) {
    return t.layout() == at::kStrided && t.is_cuda() && t.device().index() == index && t.numel() >= numel &&
           t.is_contiguous();
}

// Values of `size` bytes as the library stores them: bfloat16, float32 or
// integer patterns (not float16, which has the size of bfloat16).
bool holds_values(const at::Tensor& t, int64_t size) {
    const at::ScalarType type = t.scalar_type();
    const bool known = type == at::kBFloat16 || type == at::kFloat || at::isIntegralType(type, /*includeBool=*/false);
    return known && t.element_size() == size;
}

// Address of a contiguous tensor of at least numel elements on GPU index (None: NULL).
template <class T>
T* need(PyObject* o, const char* name, int64_t numel, int index, at::ScalarType type = at::kInt) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || !fits(t, numel, index)) {
        PyErr_Format(PyExc_ValueError, "%s must be a contiguous torch.%s tensor of at least %lld elements on GPU %d", name,
                     type == at::kInt ? "int32" : type == at::kLong ? "int64" : "float32", (long long)numel, index);
        throw Failed{};
    }
    return static_cast<T*>(t.data_ptr());
}

int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Failed{};
    return v;
}

double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Failed{};
    return v;
}

uint64_t wrapped(PyObject* o) {  // modulo 2^64, as ctypes passes numbers
    const unsigned long long v = PyLong_AsUnsignedLongLongMask(o);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) throw Failed{};
    return v;
}

hipStream_t stream_of(PyObject* o) { return reinterpret_cast<hipStream_t>((uintptr_t)wrapped(o)); }

int gpu_of(const at::Tensor& t) { return t.is_cuda() ? (int)t.device().index() : -1; }

void expect(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) fail("wrong number of arguments");
}

// No C++ exception passes into the interpreter.
template <class F>
PyObject* guarded(const F& f) {
    try {
        return PyLong_FromLong(f());
    } catch (const Failed&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// bind(adjust, count, verify, plan, tree, cache_write, cache_move, attend, attend_workspace, verify_tree): addresses of
// the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 10);
        g_adjust = reinterpret_cast<decltype(g_adjust)>((uintptr_t)wrapped(a[0]));
        g_count = reinterpret_cast<decltype(g_count)>((uintptr_t)wrapped(a[1]));
        g_verify = reinterpret_cast<decltype(g_verify)>((uintptr_t)wrapped(a[2]));
        g_plan = reinterpret_cast<decltype(g_plan)>((uintptr_t)wrapped(a[3]));
        g_tree = reinterpret_cast<decltype(g_tree)>((uintptr_t)wrapped(a[4]));
        g_cache_write = reinterpret_cast<decltype(g_cache_write)>((uintptr_t)wrapped(a[5]));
        g_cache_move = reinterpret_cast<decltype(g_cache_move)>((uintptr_t)wrapped(a[6]));
        g_attend = reinterpret_cast<decltype(g_attend)>((uintptr_t)wrapped(a[7]));
        g_attend_workspace = reinterpret_cast<decltype(g_attend_workspace)>((uintptr_t)wrapped(a[8]));
        g_verify_tree = reinterpret_cast<decltype(g_verify_tree)>((uintptr_t)wrapped(a[9]));
        return 0;
    });
}

// adjust(stream, address of the rules, x, out, element size, elements of x, of out, GPU)
PyObject* adjust(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 8);
        const at::Tensor &x = tensor(a[2], "x"), &out = tensor(a[3], "out");
        const int64_t size = whole(a[4]);
        const int index = (int)whole(a[7]);
        if (!holds_values(x, size) || !holds_values(out, size) || !fits(x, whole(a[5]), index) ||
            !fits(out, whole(a[6]), index))
            fail("x and out must be contiguous, on the rules' GPU, and hold the matrix described by the rules");
        return g_adjust(reinterpret_cast<const topk_adjust_rules*>((uintptr_t)wrapped(a[1])), x.data_ptr(), out.data_ptr(),
                        stream_of(a[0]));
    });
}

// count(stream, V, counts, seen, ids, start, prompt_len, fresh)
PyObject* count(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 8);
        const at::Tensor &counts = tensor(a[2], "counts"), &seen = tensor(a[3], "seen"), &ids = tensor(a[4], "ids");
        if (counts.dim() != 2 || seen.dim() != 2 || seen.size(0) != counts.size(0))
            fail("counts and seen must be matrices with a row per lane");
        const int index = gpu_of(counts);
        const int64_t lanes = counts.size(0), n_ids = ids.numel();
        return g_count(whole(a[1]), lanes, n_ids ? need<int32_t>(a[4], "ids", 0, index) : nullptr, n_ids,
                       need<int32_t>(a[5], "start", lanes + 1, index), need<int32_t>(a[6], "prompt_len", lanes, index),
                       need<int32_t>(a[7], "fresh", lanes, index), need<int32_t>(a[2], "counts", 1, index),
                       counts.size(1), need<uint32_t>(a[3], "seen", 1, index), seen.size(1), stream_of(a[0]));
    });
}

// verify(stream, lanes, target_values, target_ids, col_start, drafts, draft_start, draft_values, draft_ids,
//        temperature, top_p, seed, offset, out_tokens, out_count)
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 15);
        const at::Tensor &values = tensor(a[2], "target_values"), &ids = tensor(a[3], "target_ids");
        const at::Tensor &drafts = tensor(a[5], "drafts"), &tokens = tensor(a[13], "out_tokens");
        const int index = gpu_of(values);
        topk_verify_args v = {};
        v.lanes = whole(a[1]);
        if (values.dim() != 2 || ids.sizes() != values.sizes() || tokens.dim() != 2 || tokens.size(0) < v.lanes)
            fail("target_values and target_ids must be (C, k), out_tokens a matrix with a row per lane");
        const int64_t size = values.element_size();
        if ((size != 2 && size != 4) || !holds_values(values, size) || !fits(values, 0, index))
            fail("target_values must be a contiguous GPU tensor of bf16 or fp32 (or patterns)");
        v.dtype = size == 2 ? TOPK_BF16 : TOPK_F32;
        v.C = values.size(0);
        if (values.size(1) > TOPK_MAX_K) fail("lists must have at most 64 entries");
        v.k = (int32_t)values.size(1);
        v.n_drafts = drafts.numel();
        if (a[7] == Py_None && a[8] != Py_None) fail("draft_ids without draft_values");
        if (a[7] != Py_None) {
            const at::Tensor& qv = tensor(a[7], "draft_values");
            if (qv.dim() != 2 || a[8] == Py_None || tensor(a[8], "draft_ids").sizes() != qv.sizes() ||
                !holds_values(qv, size) || !fits(qv, 0, index) || qv.size(1) > TOPK_MAX_K)
                fail("draft_values and draft_ids must be contiguous (n, kq) tensors of the target lists' types");
            if (qv.size(0) < v.n_drafts) {
                // drafts past the lists have no distribution to be judged by; split evenly, the drafts that have
                // one would be other lanes' than the rest
                if (a[6] == Py_None) fail("without draft_start, every draft needs a list");
                v.n_drafts = qv.size(0);
            }
            if (v.n_drafts) {
                v.kq = (int32_t)qv.size(1);
                v.draft_values = qv.data_ptr();
                v.draft_ids = need<int32_t>(a[8], "draft_ids", 0, index);
            }
        }
        v.col_start = need<int32_t>(a[4], "col_start", v.lanes + 1, index);
        v.target_values = values.data_ptr();
        v.target_ids = need<int32_t>(a[3], "target_ids", 1, index);
        v.draft_start = need<int32_t>(a[6], "draft_start", v.lanes + 1, index);
        v.drafts = v.n_drafts ? need<int32_t>(a[5], "drafts", 0, index) : nullptr;
        v.temperature = real(a[9]);
        v.top_p = real(a[10]);
        v.seed = wrapped(a[11]);
        v.offset = wrapped(a[12]);
        v.max_tokens = tokens.size(1);
        v.out_tokens = need<int32_t>(a[13], "out_tokens", 1, index);
        v.out_count = need<int32_t>(a[14], "out_count", v.lanes, index);
        return g_verify(&v, stream_of(a[0]));
    });
}

// plan(stream, lens, add, held, table, free_ids, free_count, block_size, capacity, then the outputs held, free_count,
//      refused, col_start, col_lane, col_pos, slots)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 16);
        const at::Tensor &lens = tensor(a[1], "lens"), &table = tensor(a[4], "table"), &free_ids = tensor(a[5], "free_ids");
        const int index = gpu_of(lens);
        topk_plan_args p = {};
        p.lanes = lens.numel();
        if (table.dim() != 2 || table.size(0) < p.lanes) fail("table must be a matrix with a row per lane");
        const int64_t block = whole(a[7]);
        p.capacity = whole(a[8]);
        if (block < 1 || block > INT32_MAX || p.capacity < 1 || p.capacity > INT32_MAX)
            fail("block_size and capacity must be positive 32-bit numbers");
        p.block_size = (int32_t)block;
        p.lens = need<int32_t>(a[1], "lens", p.lanes, index);
        p.add = need<int32_t>(a[2], "add", p.lanes, index);
        p.held = need<int32_t>(a[3], "held", p.lanes, index);
        p.table = need<int32_t>(a[4], "table", 1, index);
        p.table_ld = table.size(1);
        p.n_free_ids = free_ids.numel();
        p.free_ids = p.n_free_ids ? need<int32_t>(a[5], "free_ids", 0, index) : nullptr;
        p.free_count = need<int32_t>(a[6], "free_count", 1, index);
        p.out_held = need<int32_t>(a[9], "out held", p.lanes, index);
        p.out_free_count = need<int32_t>(a[10], "out free_count", 1, index);
        p.out_refused = need<int32_t>(a[11], "out refused", 1, index);
        p.out_col_start = need<int32_t>(a[12], "out col_start", p.lanes + 1, index);
        p.out_col_lane = need<int32_t>(a[13], "out col_lane", p.capacity, index);
        p.out_col_pos = need<int32_t>(a[14], "out col_pos", p.capacity, index);
        p.out_slots = need<int64_t>(a[15], "out slots", p.capacity, index, at::kLong);
        return g_plan(&p, stream_of(a[0]));
    });
}

// tree(stream, lanes, parents, lens, col_start, mask, positions)
PyObject* tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 7);
        const at::Tensor &parents = tensor(a[2], "parents"), &mask = tensor(a[5], "mask");
        const int index = gpu_of(parents);
        const int64_t lanes = whole(a[1]), C = parents.numel();
        if (mask.dim() != 2 || mask.size(0) < C) fail("mask must be a matrix with a row per column");
        return g_tree(lanes, C, need<int32_t>(a[4], "col_start", lanes + 1, index), need<int32_t>(a[2], "parents", 1, index),
                      need<int32_t>(a[3], "lens", lanes, index), need<uint32_t>(a[5], "mask", 1, index), mask.size(1),
                      need<int32_t>(a[6], "positions", C, index), stream_of(a[0]));
    });
}

// verify_tree(stream, lanes, target_values, target_ids, col_start, tokens, parents, uniforms, draft_values, draft_ids,
//             temperature, top_p, out_tokens, out_columns, out_count)
PyObject* verify_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 15);
        const at::Tensor &values = tensor(a[2], "target_values"), &ids = tensor(a[3], "target_ids");
        const at::Tensor &tokens = tensor(a[12], "out_tokens"), &columns = tensor(a[13], "out_columns");
        const int index = gpu_of(values);
        topk_verify_tree_args v = {};
        v.lanes = whole(a[1]);
        if (values.dim() != 2 || ids.sizes() != values.sizes()) fail("target_values and target_ids must be (C, k)");
        if (tokens.dim() != 2 || tokens.size(0) < v.lanes || columns.dim() != 2 || columns.size(0) < v.lanes ||
            columns.size(1) != tokens.size(1))
            fail("out_tokens and out_columns must be matrices of one width with a row per lane");
        const int64_t size = values.element_size();
        if ((size != 2 && size != 4) || !holds_values(values, size) || !fits(values, 0, index))
            fail("target_values must be a contiguous GPU tensor of bf16 or fp32 (or patterns)");
        v.dtype = size == 2 ? TOPK_BF16 : TOPK_F32;
        v.C = values.size(0);
        if (values.size(1) > TOPK_MAX_K) fail("lists must have at most 64 entries");
        v.k = (int32_t)values.size(1);
        if (a[8] == Py_None && a[9] != Py_None) fail("draft_ids without draft_values");
        if (a[8] != Py_None) {
            const at::Tensor& qv = tensor(a[8], "draft_values");
            if (qv.dim() != 2 || a[9] == Py_None || tensor(a[9], "draft_ids").sizes() != qv.sizes() || qv.size(0) < v.C ||
                !holds_values(qv, size) || !fits(qv, 1, index) || qv.size(1) > TOPK_MAX_K)
                fail("draft_values and draft_ids must be contiguous (C, kq) tensors of the target lists' types");
            v.kq = (int32_t)qv.size(1);
            v.draft_values = qv.data_ptr();
            v.draft_ids = need<int32_t>(a[9], "draft_ids", 0, index);
        }
        v.col_start = need<int32_t>(a[4], "col_start", v.lanes + 1, index);
        v.target_values = values.data_ptr();
        v.target_ids = need<int32_t>(a[3], "target_ids", 1, index);
        v.tokens = need<int32_t>(a[5], "tokens", v.C, index);
        v.parents = need<int32_t>(a[6], "parents", v.C, index);
        v.uniforms = need<float>(a[7], "uniforms", 2 * v.C, index, at::kFloat);
        v.temperature = real(a[10]);
        v.top_p = real(a[11]);
        v.max_tokens = tokens.size(1);
        v.out_tokens = need<int32_t>(a[12], "out_tokens", 1, index);
        v.out_columns = need<int32_t>(a[13], "out_columns", 1, index);
        v.out_count = need<int32_t>(a[14], "out_count", v.lanes, index);
        return g_verify_tree(&v, stream_of(a[0]));
    });
}

// A stride as the library takes it: none where there is one entry.
int64_t stride_of(const at::Tensor& t, int64_t dim) { return t.size(dim) == 1 ? 0 : t.stride(dim); }

// Rows (C, heads, dim) on GPU index, whose strides the library checks but for the last.
const at::Tensor& rows(PyObject* o, const char* name, int64_t heads, int64_t dim, int index) {
    const at::Tensor& t = tensor(o, name);
    if (t.layout() != at::kStrided || t.dim() != 3 || (heads > 0 && t.size(1) != heads) || t.size(2) != dim ||
        t.stride(2) != 1 || gpu_of(t) != index) {
        PyErr_Format(PyExc_ValueError, "%s must be a (columns, heads, dim) tensor of the cache's sizes on GPU %d, its last stride 1",
                     name, index);
        throw Failed{};
    }
    return t;
}

// cache_write(stream, address of the cache, GPU, k, v, slots, layer)
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 7);
        const topk_cache* c = reinterpret_cast<const topk_cache*>((uintptr_t)wrapped(a[1]));
        const int index = (int)whole(a[2]);
        const at::Tensor &k = rows(a[3], "k", c->heads, c->dim, index), &v = rows(a[4], "v", c->heads, c->dim, index);
        if ((k.scalar_type() != at::kBFloat16 && k.scalar_type() != at::kFloat) || v.scalar_type() != k.scalar_type() ||
            v.size(0) != k.size(0))
            fail("k and v must both be bfloat16 or float32, with a row per column");
        topk_cache_write_args w = {};
        w.C = k.size(0);
        w.layer = whole(a[6]);
        w.dtype = k.scalar_type() == at::kBFloat16 ? TOPK_BF16 : TOPK_F32;
        w.keys = k.data_ptr();
        w.values = v.data_ptr();
        w.key_stride = stride_of(k, 0);
        w.key_head_stride = stride_of(k, 1);
        w.value_stride = stride_of(v, 0);
        w.value_head_stride = stride_of(v, 1);
        w.slots = need<int64_t>(a[5], "slots", w.C, index, at::kLong);
        return g_cache_write(c, &w, stream_of(a[0]));
    });
}

// attend(stream, address of the cache, GPU, q, lens, table, col_start, mask, positions, window, scale, layer, out)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 13);
        const topk_cache* c = reinterpret_cast<const topk_cache*>((uintptr_t)wrapped(a[1]));
        const int index = (int)whole(a[2]);
        const at::Tensor &q = rows(a[3], "q", 0, c->dim, index), &out = rows(a[12], "out", q.size(1), c->dim, index);
        const at::Tensor &lens = tensor(a[4], "lens"), &table = tensor(a[5], "table");
        if (q.scalar_type() != at::kBFloat16 || out.scalar_type() != at::kBFloat16 || out.size(0) < q.size(0))
            fail("q and out must be bfloat16, out with a row per column");
        topk_attend_args t = {};
        t.lanes = a[6] == Py_None ? lens.numel() : tensor(a[6], "col_start").numel() - 1;
        if (table.dim() != 2 || table.size(0) < t.lanes) fail("table must be a matrix with a row per lane");
        const int64_t window = whole(a[9]);
        if (window < 0 || window > INT32_MAX) fail("window must be a 32-bit number, 0 for none");
        t.C = q.size(0);
        t.layer = whole(a[11]);
        if (q.size(1) > INT32_MAX) fail("too many heads");
        t.heads = (int32_t)q.size(1);
        t.window = (int32_t)window;
        t.scale = (float)real(a[10]);
        t.q = q.data_ptr();
        t.q_stride = stride_of(q, 0);
        t.q_head_stride = stride_of(q, 1);
        t.col_start = need<int32_t>(a[6], "col_start", t.lanes + 1, index);
        t.lens = need<int32_t>(a[4], "lens", t.lanes, index);
        t.table = need<int32_t>(a[5], "table", 1, index);
        t.table_ld = table.size(1);
        if (a[7] != Py_None) {
            const at::Tensor& mask = tensor(a[7], "mask");
            if (mask.dim() != 2 || mask.size(0) < t.C || mask.size(1) < 1) fail("mask must be a matrix with a row per column");
            t.mask = need<uint32_t>(a[7], "mask", 1, index);
            t.mask_ld = mask.size(1);
        }
        t.positions = need<int32_t>(a[8], "positions", t.C, index);
        t.out = out.data_ptr();
        t.out_stride = stride_of(out, 0);
        t.out_head_stride = stride_of(out, 1);
        if (const int bad = g_attend_workspace(c, &t, &t.workspace_bytes)) return bad;
        at::Tensor workspace;  // its memory goes back to the stream that the call is ordered on
        if (t.workspace_bytes > 0) {
            workspace = at::empty({t.workspace_bytes}, q.options().dtype(at::kByte));
            t.workspace = workspace.data_ptr();
        }
        return g_attend(c, &t, stream_of(a[0]));
    });
}

// cache_move(stream, address of the cache, GPU, lens, table, columns)
PyObject* cache_move(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 6);
        const int index = (int)whole(a[2]);
        const at::Tensor &lens = tensor(a[3], "lens"), &table = tensor(a[4], "table"), &columns = tensor(a[5], "columns");
        const int64_t lanes = lens.numel();
        if (table.dim() != 2 || table.size(0) < lanes || columns.dim() != 2 || columns.size(0) < lanes)
            fail("table and columns must be matrices with a row per lane");
        return g_cache_move(reinterpret_cast<const topk_cache*>((uintptr_t)wrapped(a[1])), lanes,
                            need<int32_t>(a[3], "lens", lanes, index), need<int32_t>(a[4], "table", 1, index), table.size(1),
                            need<int32_t>(a[5], "columns", 1, index), columns.size(1), stream_of(a[0]));
    });
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"adjust", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(adjust)), METH_FASTCALL, nullptr},
    {"count", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(count)), METH_FASTCALL, nullptr},
    {"verify", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(verify)), METH_FASTCALL, nullptr},
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(plan)), METH_FASTCALL, nullptr},
    {"tree", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(tree)), METH_FASTCALL, nullptr},
    {"verify_tree", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(verify_tree)), METH_FASTCALL, nullptr},
    {"cache_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_write)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"cache_move", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_move)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_round_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__round_binding() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", TOPK_BUILT_FOR) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
