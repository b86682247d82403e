// CPython module behind AdjustRules.apply, count_tokens, verify and plan of the
// binding: takes their tensors apart, checks them and calls the C ABI.
//
// A round's calls run kernels of 3 to 5 us; checking a dozen tensors from
// Python takes as long.  Reading them here takes a call from 7 - 9 us to 4 - 5,
// of which the runtime's launch is 2.6.  Nothing else happens here: the
// checks are the binding's (each tensor's type, device, size and contiguity),
// every other argument is checked by the library.
//
// The library's functions are bound at load time (bind), so that the binding
// keeps choosing which library is in use.
#include <torch/csrc/autograd/python_variable.h>

#include "topk_cols.h"

namespace {

decltype(&topk_cols_adjust) g_adjust = nullptr;
decltype(&topk_cols_count) g_count = nullptr;
decltype(&topk_cols_verify) g_verify = nullptr;
decltype(&topk_cols_plan) g_plan = nullptr;

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
                     type == at::kInt ? "int32" : "int64", (long long)numel, index);
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

// bind(adjust, count, verify, plan): addresses of the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&] {
        expect(n, 4);
        g_adjust = reinterpret_cast<decltype(g_adjust)>((uintptr_t)wrapped(a[0]));
        g_count = reinterpret_cast<decltype(g_count)>((uintptr_t)wrapped(a[1]));
        g_verify = reinterpret_cast<decltype(g_verify)>((uintptr_t)wrapped(a[2]));
        g_plan = reinterpret_cast<decltype(g_plan)>((uintptr_t)wrapped(a[3]));
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

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"adjust", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(adjust)), METH_FASTCALL, nullptr},
    {"count", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(count)), METH_FASTCALL, nullptr},
    {"verify", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(verify)), METH_FASTCALL, nullptr},
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(plan)), METH_FASTCALL, nullptr},
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
