// Python binding of the serving calls (paged KV cache, beam search), whose kernels
// run for a few microseconds: the tensors' types, shapes, layouts and devices are
// checked and their addresses passed on in C++, at some 1 us a call where the same
// checks in Python and ctypes take 9.  Every function takes the model's handle and
// GPU first and the CUDA stream last, and returns the C ABI's status code.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "nanochat_b200.h"

namespace {

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(PyObject* kind, const char* format, const char* a = "", long long b = 0, long long c = 0) {
    PyErr_Format(kind, format, a, b, c);
    throw Refused();
}

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kInt: return "torch.int32";
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        default: return at::toString(t);
    }
}

// The arguments of a call, taken one after another.
class Args {
public:
    Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : at_(args), end_(args + n) {
        if (n != want) refuse(PyExc_TypeError, "%s: wrong number of arguments", "serving call");
        model = static_cast<nc_model*>(pointer());
        device = integer();
    }
    long long integer() {
        const long long v = PyLong_AsLongLong(*at_++);
        if (v == -1 && PyErr_Occurred()) throw Refused();
        return v;
    }
    int i32(const char* name) {
        const long long v = integer();
        if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_ValueError, "%s is out of range", name);
        return static_cast<int>(v);
    }
    void* pointer() {  // an address, or None
        PyObject* o = *at_++;
        if (o == Py_None) return nullptr;
        void* p = PyLong_AsVoidPtr(o);
        if (!p && PyErr_Occurred()) throw Refused();
        return p;
    }
    // The next tensor (null where it is None and that is allowed).
    const at::Tensor* tensor(const char* name, bool optional = false) {
        PyObject* o = *at_++;
        if (optional && o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
        return &THPVariable_Unpack(o);
    }
    // The address of a contiguous tensor of that type (or of any) on the model's GPU.
    void* address(const at::Tensor& t, at::ScalarType type, const char* name) {
        if (type != at::ScalarType::Undefined && t.scalar_type() != type) {
            PyErr_Format(PyExc_TypeError, "%s: expected %s, got %s", name, type_name(type), type_name(t.scalar_type()));
            throw Refused();
        }
        if (t.layout() != at::kStrided || !t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
        if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be in device memory", name);
        if (t.get_device() != device) refuse(PyExc_ValueError, "%s must be on the model's cuda:%lld, not cuda:%lld", name, device, t.get_device());
        return t.data_ptr();
    }

    nc_model* model;
    long long device;

private:
    PyObject* const* at_;
    PyObject* const* end_;
};

constexpr at::ScalarType kI32 = at::kInt, kF32 = at::kFloat, kAny = at::ScalarType::Undefined;

void shape(const at::Tensor& t, std::initializer_list<int64_t> want, const char* name) {
    if (t.sizes().equals(at::IntArrayRef(want))) return;
    char text[200];
    int n = snprintf(text, sizeof text, "must be [");
    for (int64_t w : want) n += snprintf(text + n, sizeof text - n, n > 9 ? ", %lld" : "%lld", (long long)w);
    n += snprintf(text + n, sizeof text - n, "], got [");
    const int start = n;
    for (int64_t w : t.sizes())
        if (n < 150) n += snprintf(text + n, sizeof text - n, n > start ? ", %lld" : "%lld", (long long)w);
    snprintf(text + n, sizeof text - n, "]");
    PyErr_Format(PyExc_ValueError, "%s %s", name, text);
    throw Refused();
}

int i32_of(int64_t v, const char* name) {
    if (v > INT32_MAX) refuse(PyExc_ValueError, "%s is too large", name);
    return static_cast<int>(v);
}

// Calls the library without the interpreter's lock: a launch waits where the stream's queue is full,
// and the program's other threads go on meanwhile.  The arguments are addresses and sizes by then, taken
// before the lock is given up; the caller holds the tensors.
template <typename F, typename... A>
int unlocked(F* f, A... args) {
    struct Unlocked {
        PyThreadState* const state = PyEval_SaveThread();
        ~Unlocked() { PyEval_RestoreThread(state); }
    } unlocked;
    return f(args...);
}

template <typename F>
PyObject* call(F f) {
    try {
        return PyLong_FromLong(f());
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

at::ScalarType weight_type(Args& a) { return a.integer() ? at::kBFloat16 : at::kFloat; }

// page_plan(model, device, page_size, cached_len, new_len, release, block_table, free_pages, free_count, cu_rows,
//           kv_len, positions, slots, stream)
PyObject* page_plan(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    return call([&] {
        Args a(args, nargs, 14);
        const int page = a.i32("page_size");
        const at::Tensor &cached = *a.tensor("cached_len"), &fresh = *a.tensor("new_len"), *release = a.tensor("release", true);
        const at::Tensor &table = *a.tensor("block_table"), &free = *a.tensor("free_pages"), &count = *a.tensor("free_count");
        const at::Tensor &cu = *a.tensor("cu_rows"), &kv_len = *a.tensor("kv_len"), &pos = *a.tensor("positions"), &slots = *a.tensor("slots");
        const int64_t n = fresh.numel();
        shape(fresh, {n}, "new_len");
        shape(cached, {n}, "cached_len");
        shape(cu, {n + 1}, "cu_rows");
        shape(kv_len, {n}, "kv_len");
        shape(count, {1}, "free_count");
        if (table.dim() != 2 || table.size(0) != n || free.dim() != 1 || pos.dim() != 1)
            refuse(PyExc_ValueError, "block_table must be [requests, blocks], free_pages [pages], positions and slots [rows]");
        shape(slots, {pos.numel()}, "slots");
        if (release) shape(*release, {n}, "release");
        auto p = [&](const at::Tensor& t, const char* name) { return static_cast<int32_t*>(a.address(t, kI32, name)); };
        return unlocked(nc_page_plan, a.model, i32_of(n, "new_len"), page, i32_of(table.size(1), "block_table"), i32_of(free.numel(), "free_pages"),
                        i32_of(pos.numel(), "positions"), p(cached, "cached_len"), p(fresh, "new_len"),
                        release ? p(*release, "release") : nullptr, p(table, "block_table"), p(free, "free_pages"),
                        p(count, "free_count"), p(cu, "cu_rows"), p(kv_len, "kv_len"), p(pos, "positions"), p(slots, "slots"), a.pointer());
    });
}

// A planned step's arrays.
struct Step {
    int n, blocks;
    const int32_t *cu, *kv_len, *slots, *table;
    Step(Args& a, int64_t rows) {
        const at::Tensor &c = *a.tensor("cu_rows"), &k = *a.tensor("kv_len"), &s = *a.tensor("slots"), &t = *a.tensor("block_table");
        const int64_t r = k.numel();
        shape(k, {r}, "kv_len");
        shape(c, {r + 1}, "cu_rows");
        shape(s, {rows}, "slots");
        if (t.dim() != 2 || t.size(0) != r) refuse(PyExc_ValueError, "block_table must be [requests, blocks]");
        n = i32_of(r, "kv_len");
        blocks = i32_of(t.size(1), "block_table");
        cu = static_cast<int32_t*>(a.address(c, kI32, "cu_rows"));
        kv_len = static_cast<int32_t*>(a.address(k, kI32, "kv_len"));
        slots = static_cast<int32_t*>(a.address(s, kI32, "slots"));
        table = static_cast<int32_t*>(a.address(t, kI32, "block_table"));
    }
};

// paged_attention(model, device, bf16, n_head, n_kv_head, head_dim, max_new, cu_rows, kv_len, slots, block_table, qkv,
//                 k_pages, v_pages, o, workspace, stream)
PyObject* paged_attention(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    return call([&] {
        Args a(args, nargs, 17);
        const at::ScalarType type = weight_type(a);
        const int64_t h = a.integer(), nkv = a.integer(), hd = a.integer();
        const int max_new = a.i32("max_new");
        Args peek = a;  // the step's arrays are checked against qkv's rows
        for (int i = 0; i < 4; ++i) peek.tensor("cu_rows");
        const at::Tensor &qkv = *peek.tensor("qkv"), &k = *peek.tensor("k_pages"), &v = *peek.tensor("v_pages"), &o = *peek.tensor("o");
        const at::Tensor& ws = *peek.tensor("workspace");
        if (qkv.dim() != 2) refuse(PyExc_ValueError, "qkv must be [rows, (n_head + 2 n_kv_head) head_dim]");
        const int64_t rows = qkv.size(0);
        shape(qkv, {rows, (h + 2 * nkv) * hd}, "qkv");
        shape(o, {rows, h * hd}, "o");
        if (k.dim() != 4 || k.size(2) != nkv || k.size(3) != hd)
            refuse(PyExc_ValueError, "k_pages must be [pages, page_size, n_kv_head, head_dim]");
        shape(v, {k.size(0), k.size(1), nkv, hd}, "v_pages");
        const Step s(a, rows);
        return unlocked(nc_paged_attention, a.model, a.address(qkv, type, "qkv"), i32_of(rows, "qkv"), s.n, max_new, s.cu, s.kv_len, s.slots, s.table,
                        s.blocks, i32_of(k.size(1), "page_size"), i32_of(k.size(0), "k_pages"), a.address(k, type, "k_pages"),
                        a.address(v, type, "v_pages"), a.address(o, type, "o"), a.address(ws, kAny, "workspace"), ws.nbytes(),
                        peek.pointer());
    });
}

// The paged cache of a model, [n_layer, 2, pages, page_size, n_kv_head, head_dim].
void check_pages(const at::Tensor& kv, int64_t layers, int64_t nkv, int64_t hd) {
    if (kv.dim() != 6 || kv.size(0) != layers || kv.size(1) != 2 || kv.size(4) != nkv || kv.size(5) != hd)
        refuse(PyExc_ValueError, "kv_pages must be [n_layer, 2, pages, page_size, n_kv_head, head_dim]");
}

// paged_forward(model, device, bf16, n_layer, n_kv_head, head_dim, vocab, n_params, max_new, cu_rows, kv_len, slots,
//               block_table, tokens, positions, weights, kv_pages, logits, workspace, stream)
PyObject* paged_forward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    return call([&] {
        Args a(args, nargs, 20);
        const at::ScalarType type = weight_type(a);
        const int64_t layers = a.integer(), nkv = a.integer(), hd = a.integer(), vocab = a.integer(), params = a.integer();
        const int max_new = a.i32("max_new");
        Args peek = a;
        for (int i = 0; i < 4; ++i) peek.tensor("cu_rows");
        const at::Tensor &tokens = *peek.tensor("tokens"), &pos = *peek.tensor("positions"), &w = *peek.tensor("weights");
        const at::Tensor &kv = *peek.tensor("kv_pages"), &logits = *peek.tensor("logits"), &ws = *peek.tensor("workspace");
        const int64_t rows = tokens.numel();
        shape(tokens, {rows}, "tokens");
        shape(pos, {rows}, "positions");
        if (w.numel() < params) refuse(PyExc_ValueError, "weights shorter than the flat layout");
        check_pages(kv, layers, nkv, hd);
        const Step s(a, rows);
        shape(logits, {s.n, vocab}, "logits");
        return unlocked(nc_paged_forward, a.model, static_cast<int32_t*>(a.address(tokens, kI32, "tokens")), i32_of(rows, "tokens"), s.n, max_new,
                        static_cast<int32_t*>(a.address(pos, kI32, "positions")), s.cu, s.kv_len, s.slots, s.table, s.blocks,
                        i32_of(kv.size(3), "page_size"), i32_of(kv.size(2), "kv_pages"), a.address(w, type, "weights"),
                        a.address(kv, type, "kv_pages"), a.address(logits, type, "logits"), a.address(ws, kAny, "workspace"),
                        ws.nbytes(), peek.pointer());
    });
}

// beam_select(model, device, bf16, vocab, eos, logits, scores, finished, scores_out, tokens, parents, finished_out, stream)
PyObject* beam_select(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    return call([&] {
        Args a(args, nargs, 13);
        const at::ScalarType type = weight_type(a);
        const int64_t vocab = a.integer();
        const int eos = a.i32("eos");
        const at::Tensor &logits = *a.tensor("logits"), &scores = *a.tensor("scores"), *fin = a.tensor("finished", true);
        const at::Tensor &out = *a.tensor("scores_out"), &tokens = *a.tensor("tokens"), &parents = *a.tensor("parents");
        const at::Tensor* fin_out = a.tensor("finished_out", true);
        if (scores.dim() != 2) refuse(PyExc_ValueError, "scores must be [batch, beams]");
        const int64_t b = scores.size(0), k = scores.size(1);
        if (!logits.sizes().equals({b, k, vocab}) && !logits.sizes().equals({b * k, vocab}))
            refuse(PyExc_ValueError, "%s must be [batch, beams, %lld] or [batch * beams, %lld]", "logits", vocab, vocab);
        shape(out, {b, k}, "scores_out");
        shape(tokens, {b, k}, "tokens");
        shape(parents, {b, k}, "parents");
        if (!fin != !fin_out) refuse(PyExc_ValueError, "finished and finished_out go together");
        if (fin) {
            shape(*fin, {b, k}, "finished");
            shape(*fin_out, {b, k}, "finished_out");
        }
        const void* z = a.address(logits, type, "logits");
        const auto *sc = static_cast<float*>(a.address(scores, kF32, "scores"));
        auto* so = static_cast<float*>(a.address(out, kF32, "scores_out"));
        auto p = [&](const at::Tensor* t, const char* name) { return t ? static_cast<int32_t*>(a.address(*t, kI32, name)) : nullptr; };
        int32_t *f = p(fin, "finished"), *fo = p(fin_out, "finished_out"), *to = p(&tokens, "tokens"), *pa = p(&parents, "parents");
        return unlocked(nc_beam_select, a.model, z, i32_of(b, "batch"), i32_of(k, "beams"), sc, f, eos, so, to, pa, fo, a.pointer());
    });
}

// beam_reorder(model, device, bytes of a position over all layers, kv_cache, T_max, parents, start, end, stream)
PyObject* beam_reorder(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    return call([&] {
        Args a(args, nargs, 9);
        const int64_t each = a.integer();
        const at::Tensor& kv = *a.tensor("kv_cache");
        const int t_max = a.i32("T_max");
        const at::Tensor& parents = *a.tensor("parents");
        const int start = a.i32("start"), end = a.i32("end");
        if (parents.dim() != 2) refuse(PyExc_ValueError, "parents must be [batch, beams]");
        const int64_t b = parents.size(0), k = parents.size(1);
        if ((double)kv.nbytes() < (double)each * b * k * t_max)
            refuse(PyExc_ValueError, "kv_cache smaller than kv_cache_bytes(batch * beams, T_max)");
        return unlocked(nc_beam_reorder, a.model, a.address(kv, kAny, "kv_cache"), i32_of(b, "batch"), i32_of(k, "beams"), t_max,
                        static_cast<int32_t*>(a.address(parents, kI32, "parents")), start, end, a.pointer());
    });
}

// beam_reorder_paged(model, device, bf16, n_layer, n_kv_head, head_dim, kv_pages, parents, block_table, starts, ends, stream)
PyObject* beam_reorder_paged(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    return call([&] {
        Args a(args, nargs, 12);
        const at::ScalarType type = weight_type(a);
        const int64_t layers = a.integer(), nkv = a.integer(), hd = a.integer();
        const at::Tensor &kv = *a.tensor("kv_pages"), &parents = *a.tensor("parents"), &table = *a.tensor("block_table");
        const at::Tensor &starts = *a.tensor("starts"), &ends = *a.tensor("ends");
        if (parents.dim() != 2) refuse(PyExc_ValueError, "parents must be [batch, beams]");
        const int64_t b = parents.size(0), k = parents.size(1);
        check_pages(kv, layers, nkv, hd);
        if (table.dim() != 2 || table.size(0) != b * k) refuse(PyExc_ValueError, "block_table must be [batch * beams, blocks]");
        shape(starts, {b * k}, "starts");
        shape(ends, {b * k}, "ends");
        auto p = [&](const at::Tensor& t, const char* name) { return static_cast<int32_t*>(a.address(t, kI32, name)); };
        return unlocked(nc_beam_reorder_paged, a.model, a.address(kv, type, "kv_pages"), i32_of(b, "batch"), i32_of(k, "beams"),
                        i32_of(kv.size(2), "kv_pages"), i32_of(kv.size(3), "page_size"), p(parents, "parents"),
                        p(table, "block_table"), i32_of(table.size(1), "block_table"), p(starts, "starts"), p(ends, "ends"),
                        a.pointer());
    });
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(page_plan),   ENTRY(paged_attention),    ENTRY(paged_forward),         ENTRY(beam_select),
                         ENTRY(beam_reorder), ENTRY(beam_reorder_paged), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", "Checked calls of the serving entry points.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&module); }
