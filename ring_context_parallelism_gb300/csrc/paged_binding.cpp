// paged_binding.cpp -- the Python binding of the operators over paged sequences, as a
// CPython extension module (_paged.so, next to libra.so).
//
// Checks of shapes, types and devices, allocation through PyTorch and the call into
// the C ABI, as ra.py does through ctypes for the other entry points.  These calls run
// once per layer and decoded token, and a decode step's kernels take 3 to 11 us.  Host
// time per call for one sequence of 1000 keys, in Python and through ctypes -> here:
// tree_attn with its three allocations 23 -> 9 us, key_mass 9.3 -> 2.6, evict_select
// 14.6 -> 6, cache_move 7.8 -> 2.4, cache_append 7.9 -> 2.5.
//
// tree_attn and evict_select return their tensors, or the entry point's status where that
// is not RA_OK; the others return the status.  ra.py raises from it.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <string>
#include <utility>

#include "ra.h"

namespace {

// A refused argument, raised as a Python exception.
struct Refused {
    PyObject* type;
    std::string message;
};

[[noreturn]] void refuse(const char* message) { throw Refused{PyExc_ValueError, message}; }

using Maybe = const at::Tensor*;  // NULL: None

Maybe maybe_tensor(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a tensor"};
    return &THPVariable_Unpack(o);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    Maybe t = maybe_tensor(o, name);
    if (!t) throw Refused{PyExc_TypeError, std::string(name) + " must be a tensor"};
    return *t;
}

int integer(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
    if (v > INT_MAX || v < INT_MIN) throw Refused{PyExc_ValueError, std::string(name) + " is too large"};
    return static_cast<int>(v);
}

int size_of(const at::Tensor& t, int dim) {
    const int64_t n = t.size(dim);
    if (n > INT_MAX) refuse("a tensor has a dimension of more than 2^31 - 1");
    return static_cast<int>(n);
}

ra_dtype type_of(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return RA_BF16;
    if (t.scalar_type() == at::kFloat) return RA_F32;
    throw Refused{PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + " (bf16 or fp32)"};
}

void int32(Maybe t, const char* name) {
    if (t && t->scalar_type() != at::kInt) throw Refused{PyExc_ValueError, std::string(name) + " must be int32"};
}

// One CUDA device, contiguous; the device's index.
int on_one_device(std::initializer_list<Maybe> ts) {
    int dev = -1;
    for (Maybe t : ts) {
        if (!t) continue;
        if (!t->is_cuda()) refuse("tensors must be on a CUDA device");
        if (dev >= 0 && t->get_device() != dev) refuse("tensors must be on one device");
        dev = static_cast<int>(t->get_device());
        if (!t->is_contiguous()) refuse("tensors must be contiguous");
    }
    return dev;
}

template <class T = void>
T* pointer(Maybe t) {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

at::Tensor empty_on(int dev, at::IntArrayRef sizes, at::ScalarType type) {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev))));
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

struct Pool {
    int n_pages, page_size, Hkv, D;
};
Pool pool_of(const at::Tensor& k, Maybe v) {
    if (k.dim() != 4 || (v && (!v->sizes().equals(k.sizes()) || v->scalar_type() != k.scalar_type())))
        refuse("k_pages (and v_pages alike) must be [n_pages, page_size, Hkv, D]");
    return {size_of(k, 0), size_of(k, 1), size_of(k, 2), size_of(k, 3)};
}

struct Batch {
    int n_seqs, max_pages;
};
Batch batch_of(const at::Tensor& row_offsets, const at::Tensor& pages, const at::Tensor& kv_lens) {
    int32(&row_offsets, "row_offsets");
    int32(&pages, "pages");
    int32(&kv_lens, "kv_lens");
    if (pages.dim() != 2 || kv_lens.dim() != 1 || kv_lens.size(0) != pages.size(0) || row_offsets.dim() != 1 ||
        row_offsets.size(0) != pages.size(0) + 1)
        refuse("pages must be [n_seqs, max_pages], kv_lens [n_seqs], row_offsets [n_seqs + 1]");
    return {size_of(pages, 0), size_of(pages, 1)};
}

int mask_cols(Maybe mask, int R) {
    if (!mask) return 0;
    if ((mask->scalar_type() != at::kBool && mask->scalar_type() != at::kByte) || mask->dim() != 2 || mask->size(0) != R)
        refuse("tree_mask must be bool [R, mask_cols]");
    // without columns it would hide every new token, but has no memory to point at
    if (mask->size(1) == 0) refuse("tree_mask needs at least one column");
    return size_of(*mask, 1);
}

// The interpreter lock is given up while memory is allocated and kernels are launched: both
// can wait for the GPU, and what it waits for can need the lock (a host function in a stream).
class Unlocked {
  public:
    Unlocked() : state_(PyEval_SaveThread()) {}
    ~Unlocked() { PyEval_RestoreThread(state_); }
    Unlocked(const Unlocked&) = delete;
    Unlocked& operator=(const Unlocked&) = delete;

  private:
    PyThreadState* state_;
};

PyObject* status_object(ra_status st) { return PyLong_FromLong(st); }

// A new reference: `made` where this call allocated it, else the argument as it came.
PyObject* result(const at::Tensor& made, PyObject* given) {
    if (!made.defined()) return Py_NewRef(given);
    PyObject* o = THPVariable_Wrap(made);
    if (!o) throw python_error();
    return o;
}

// q_rows, row_offsets, k_pages, v_pages, pages, kv_lens, tree_mask, out, lse, workspace, want_lse
PyObject* tree_attn(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q_rows"), &offs = tensor(a[1], "row_offsets"), &k = tensor(a[2], "k_pages"),
                     &v = tensor(a[3], "v_pages"), &pages = tensor(a[4], "pages"), &lens = tensor(a[5], "kv_lens");
    Maybe mask = maybe_tensor(a[6], "tree_mask"), out = maybe_tensor(a[7], "out"), lse = maybe_tensor(a[8], "lse"),
          ws = maybe_tensor(a[9], "workspace");
    const bool want_lse = PyObject_IsTrue(a[10]) > 0;
    if (q.dim() != 3) refuse("q_rows must be [R, Hq, D]");
    const int R = size_of(q, 0), Hq = size_of(q, 1), D = size_of(q, 2);
    const Pool p = pool_of(k, &v);
    const Batch b = batch_of(offs, pages, lens);
    const int cols = mask_cols(mask, R);
    if (p.D != D || k.scalar_type() != q.scalar_type()) refuse("q_rows and the page pools disagree in D or dtype");
    const ra_dtype dt = type_of(q);
    if (out && (!out->sizes().equals(q.sizes()) || out->scalar_type() != q.scalar_type()))
        refuse("out must be shaped and typed as q_rows");
    if (lse && (lse->dim() != 2 || lse->size(0) != Hq || lse->size(1) != R || lse->scalar_type() != at::kFloat))
        refuse("lse must be fp32 [Hq, R]");
    const int dev = on_one_device({&q, &offs, &k, &v, &pages, &lens, mask, out, lse, ws});
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    at::Tensor new_out, new_lse, new_ws;
    ra_status st;
    {
        const Unlocked unlocked;
        if (!out) out = &(new_out = empty_on(dev, q.sizes(), q.scalar_type()));
        if (!lse && want_lse) lse = &(new_lse = empty_on(dev, {Hq, R}, at::kFloat));
        size_t bytes;
        if (ws) {
            bytes = static_cast<size_t>(ws->numel()) * ws->element_size();
        } else {
            bytes = ra_tree_attn_workspace_size(R, b.n_seqs, Hq, p.Hkv, D, dt);
            ws = &(new_ws = empty_on(dev, {static_cast<int64_t>(std::max<size_t>(bytes, 1))}, at::kByte));
        }
        st = ra_tree_attn_paged(pointer(&q), pointer<int>(&offs), b.n_seqs, R, pointer(&k), pointer(&v), p.n_pages,
                                p.page_size, pointer<int>(&pages), b.max_pages, pointer<int>(&lens),
                                pointer<unsigned char>(mask), cols, pointer(out), pointer<float>(lse), Hq, p.Hkv, D, dt,
                                pointer(ws), bytes, stream_of(dev));
    }
    if (st != RA_OK) return status_object(st);
    PyObject* o = result(new_out, a[7]);
    return Py_BuildValue("NN", o, result(new_lse, a[8]));
}

// q_rows, lse, row_offsets, k_pages, pages, kv_lens, mass_out, mass_in, decay, tree_mask
PyObject* key_mass(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q_rows"), &lse = tensor(a[1], "lse"), &offs = tensor(a[2], "row_offsets"),
                     &k = tensor(a[3], "k_pages"), &pages = tensor(a[4], "pages"), &lens = tensor(a[5], "kv_lens"),
                     &out = tensor(a[6], "mass_out");
    Maybe in = maybe_tensor(a[7], "mass_in"), mask = maybe_tensor(a[9], "tree_mask");
    const double decay = PyFloat_AsDouble(a[8]);
    if (decay == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
    if (q.dim() != 3) refuse("q_rows must be [R, Hq, D]");
    const int R = size_of(q, 0), Hq = size_of(q, 1), D = size_of(q, 2);
    const Pool p = pool_of(k, nullptr);
    const Batch b = batch_of(offs, pages, lens);
    const int cols = mask_cols(mask, R);
    if (p.D != D || k.scalar_type() != q.scalar_type()) refuse("q_rows and k_pages disagree in D or dtype");
    if (lse.dim() != 2 || lse.size(0) != Hq || lse.size(1) != R || lse.scalar_type() != at::kFloat)
        refuse("lse must be fp32 [Hq, R]");
    if (out.dim() != 3 || out.size(0) != b.n_seqs || out.size(1) != p.Hkv || out.scalar_type() != at::kFloat ||
        (in && (!in->sizes().equals(out.sizes()) || in->scalar_type() != at::kFloat)))
        refuse("mass_out and mass_in must be fp32 [n_seqs, Hkv, mass_cols]");
    const ra_dtype dt = type_of(q);
    const int dev = on_one_device({&q, &lse, &offs, &k, &pages, &lens, mask, in, &out});
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    const int mass_cols = size_of(out, 2);
    ra_status st;
    {
        const Unlocked unlocked;
        st = ra_key_mass_paged(pointer(&q), pointer<float>(&lse), pointer<int>(&offs), b.n_seqs, R, pointer(&k), p.n_pages,
                               p.page_size, pointer<int>(&pages), b.max_pages, pointer<int>(&lens),
                               pointer<unsigned char>(mask), cols, pointer<float>(in), pointer<float>(&out), mass_cols,
                               static_cast<float>(decay), Hq, p.Hkv, D, dt, stream_of(dev));
    }
    return status_object(st);
}

// mass, kv_lens, budget, n_first, n_recent, kept_mass
PyObject* evict_select(PyObject* const* a) {
    const at::Tensor &mass = tensor(a[0], "mass"), &lens = tensor(a[1], "kv_lens");
    const int budget = integer(a[2], "budget"), n_first = integer(a[3], "n_first"), n_recent = integer(a[4], "n_recent");
    Maybe kept = maybe_tensor(a[5], "kept_mass");
    int32(&lens, "kv_lens");
    if (mass.dim() != 3 || mass.scalar_type() != at::kFloat || lens.dim() != 1 || lens.size(0) != mass.size(0))
        refuse("mass must be fp32 [n_seqs, Hkv, mass_cols], kv_lens [n_seqs]");
    if (budget < 1) refuse("budget must be >= 1");
    if (kept && (kept->dim() != 3 || kept->size(0) != mass.size(0) || kept->size(1) != mass.size(1) ||
                 kept->scalar_type() != at::kFloat))
        refuse("kept_mass must be fp32 [n_seqs, Hkv, kept_cols]");
    if (kept && kept->size(2) == 0) refuse("kept_mass needs at least budget columns");
    const int dev = on_one_device({&mass, &lens, kept});
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    const int n_seqs = size_of(mass, 0), Hkv = size_of(mass, 1), cols = size_of(mass, 2);
    const int kept_cols = kept ? size_of(*kept, 2) : budget;
    at::Tensor positions, counts, new_kept;
    ra_status st;
    {
        const Unlocked unlocked;
        positions = empty_on(dev, {n_seqs, Hkv, budget}, at::kInt);
        counts = empty_on(dev, {n_seqs}, at::kInt);
        if (!kept) kept = &(new_kept = empty_on(dev, {n_seqs, Hkv, budget}, at::kFloat));
        st = ra_evict_select(pointer<float>(&mass), cols, pointer<int>(&lens), n_seqs, Hkv, budget, n_first, n_recent,
                             pointer<int>(&positions), pointer<int>(&counts), pointer<float>(kept), kept_cols,
                             stream_of(dev));
    }
    if (st != RA_OK) return status_object(st);
    PyObject *o = result(positions, nullptr), *c = result(counts, nullptr);
    return Py_BuildValue("NNN", o, c, result(new_kept, a[5]));
}

// k_pages, v_pages, src_pages, dst_pages, positions, counts, dst_start
PyObject* cache_move(PyObject* const* a) {
    const at::Tensor &k = tensor(a[0], "k_pages"), &v = tensor(a[1], "v_pages"), &src = tensor(a[2], "src_pages"),
                     &dst = tensor(a[3], "dst_pages"), &pos = tensor(a[4], "positions"), &counts = tensor(a[5], "counts");
    Maybe start = maybe_tensor(a[6], "dst_start");
    const Pool p = pool_of(k, &v);
    int32(&src, "src_pages");
    int32(&dst, "dst_pages");
    int32(&pos, "positions");
    int32(&counts, "counts");
    int32(start, "dst_start");
    if (src.dim() != 2 || dst.dim() != 2 || pos.dim() != 3 || counts.dim() != 1 || src.size(0) != counts.size(0) ||
        dst.size(0) != counts.size(0) || pos.size(0) != counts.size(0) || (start && !start->sizes().equals(counts.sizes())))
        refuse("page lists [n_seqs, max_pages], positions [n_seqs, heads, max_count], counts and dst_start [n_seqs]");
    const ra_dtype dt = type_of(k);
    const int dev = on_one_device({&k, &v, &src, &dst, &pos, &counts, start});
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    const int src_cols = size_of(src, 1), dst_cols = size_of(dst, 1), heads = size_of(pos, 1), max_count = size_of(pos, 2),
              n_seqs = size_of(counts, 0);
    ra_status st;
    {
        const Unlocked unlocked;
        st = ra_cache_move_paged(pointer(&k), pointer(&v), p.n_pages, p.page_size, pointer<int>(&src), src_cols,
                                 pointer<int>(&dst), dst_cols, pointer<int>(&pos), heads, max_count, pointer<int>(&counts),
                                 pointer<int>(start), n_seqs, p.Hkv, p.D, dt, stream_of(dev));
    }
    return status_object(st);
}

// k_rows, v_rows, row_offsets, k_pages, v_pages, pages, kv_lens
PyObject* cache_append(PyObject* const* a) {
    const at::Tensor &kr = tensor(a[0], "k_rows"), &vr = tensor(a[1], "v_rows"), &offs = tensor(a[2], "row_offsets"),
                     &k = tensor(a[3], "k_pages"), &v = tensor(a[4], "v_pages"), &pages = tensor(a[5], "pages"),
                     &lens = tensor(a[6], "kv_lens");
    const Pool p = pool_of(k, &v);
    const Batch b = batch_of(offs, pages, lens);
    if (kr.dim() != 3 || kr.size(1) != p.Hkv || kr.size(2) != p.D || !vr.sizes().equals(kr.sizes()) ||
        kr.scalar_type() != k.scalar_type() || vr.scalar_type() != k.scalar_type())
        refuse("k_rows and v_rows must be [R, Hkv, D] of the pools' dtype");
    const ra_dtype dt = type_of(k);
    const int dev = on_one_device({&kr, &vr, &offs, &k, &v, &pages, &lens});
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    const int R = size_of(kr, 0);
    ra_status st;
    {
        const Unlocked unlocked;
        st = ra_cache_append_paged(pointer(&kr), pointer(&vr), pointer<int>(&offs), b.n_seqs, R, pointer(&k), pointer(&v),
                                   p.n_pages, p.page_size, pointer<int>(&pages), b.max_pages, pointer<int>(&lens), p.Hkv,
                                   p.D, dt, stream_of(dev));
    }
    return status_object(st);
}

// Argument count and exceptions around one of the above.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refused& r) {
        if (r.type) PyErr_SetString(r.type, r.message.c_str());  // else Python's own error is set
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<tree_attn, 11>("tree_attn"),       method<key_mass, 10>("key_mass"),
                         method<evict_select, 6>("evict_select"), method<cache_move, 7>("cache_move"),
                         method<cache_append, 7>("cache_append"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module_def); }
