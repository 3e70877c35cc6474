// paged_binding.cpp -- the Python binding of the operators over paged sequences, and of the
// norm and rotation before them, as a CPython extension module (_paged.so, next to
// libra.so).
//
// Checks of shapes, types and devices, allocation through PyTorch and the call into
// the C ABI, as ra.py does through ctypes for the other entry points.  These calls run
// once per layer and decoded token, and a decode step's kernels take 3 to 11 us.  Host
// time per call for one sequence of 1000 keys, in Python and through ctypes -> here:
// tree_attn with its three allocations 23 -> 9 us, key_mass 9.3 -> 2.6, evict_select
// 14.6 -> 6, cache_move 7.8 -> 2.4, cache_append 7.9 -> 2.5.
//
// tree_attn, evict_select and others that allocate return their tensors, or the entry
// point's status where that is not RA_OK; the others return the status.  ra.py raises from it.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
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
    const at::Device on(at::kCUDA, static_cast<c10::DeviceIndex>(dev));
    // past the dispatcher (the norm's two outputs 5.1 -> 4.5 us of a call, its gradient's five tensors 11.5 -> 9.8), but where
    // it would fill the memory
    if (!at::globalContext().deterministicAlgorithms()) return at::detail::empty_cuda(sizes, type, on, std::nullopt);
    return at::empty(sizes, at::TensorOptions().dtype(type).device(on));
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

// The pools of an 8-bit cache.
struct Q8Pool : Pool {
    unsigned char *k_scales, *v_scales;
};
Q8Pool q8_pool_of(const at::Tensor& k, const at::Tensor& v, const at::Tensor& ks, const at::Tensor& vs) {
    const Pool p = pool_of(k, &v);
    if (k.scalar_type() != at::kFloat8_e4m3fn)
        throw Refused{PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(k.scalar_type()) + " of the pages (float8_e4m3fn)"};
    for (const at::Tensor* t : {&ks, &vs})
        if (t->scalar_type() != at::kByte || t->dim() != 3 || t->size(0) != p.n_pages || t->size(1) != p.Hkv ||
            t->size(2) != p.page_size)
            refuse("k_scales and v_scales must be uint8 [n_pages, Hkv, page_size]");
    return {p, pointer<unsigned char>(&ks), pointer<unsigned char>(&vs)};
}

// k_rows, v_rows, row_offsets, k_pages, v_pages, k_scales, v_scales, pages, kv_lens
PyObject* cache_append_q8(PyObject* const* a) {
    const at::Tensor &kr = tensor(a[0], "k_rows"), &vr = tensor(a[1], "v_rows"), &offs = tensor(a[2], "row_offsets"),
                     &k = tensor(a[3], "k_pages"), &v = tensor(a[4], "v_pages"), &ks = tensor(a[5], "k_scales"),
                     &vs = tensor(a[6], "v_scales"), &pages = tensor(a[7], "pages"), &lens = tensor(a[8], "kv_lens");
    const Q8Pool p = q8_pool_of(k, v, ks, vs);
    const Batch b = batch_of(offs, pages, lens);
    if (kr.dim() != 3 || kr.size(1) != p.Hkv || kr.size(2) != p.D || !vr.sizes().equals(kr.sizes()) ||
        vr.scalar_type() != kr.scalar_type())
        refuse("k_rows and v_rows must be [R, Hkv, D] of one dtype");
    const ra_dtype dt = type_of(kr);
    const int dev = on_one_device({&kr, &vr, &offs, &k, &v, &ks, &vs, &pages, &lens});
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    const int R = size_of(kr, 0);
    ra_status st;
    {
        const Unlocked unlocked;
        st = ra_cache_append_paged_q8(pointer(&kr), pointer(&vr), pointer<int>(&offs), b.n_seqs, R, pointer(&k), pointer(&v),
                                      p.k_scales, p.v_scales, p.n_pages, p.page_size, pointer<int>(&pages), b.max_pages,
                                      pointer<int>(&lens), p.Hkv, p.D, dt, stream_of(dev));
    }
    return status_object(st);
}

// row_offsets, n_rows, k_pages, v_pages, k_scales, v_scales, pages, kv_lens, bf16, k_rows, v_rows
PyObject* cache_read_q8(PyObject* const* a) {
    const at::Tensor &offs = tensor(a[0], "row_offsets"), &k = tensor(a[2], "k_pages"), &v = tensor(a[3], "v_pages"),
                     &ks = tensor(a[4], "k_scales"), &vs = tensor(a[5], "v_scales"), &pages = tensor(a[6], "pages"),
                     &lens = tensor(a[7], "kv_lens");
    const int R = integer(a[1], "n_rows");
    const bool bf16 = PyObject_IsTrue(a[8]) > 0;
    Maybe kr = maybe_tensor(a[9], "k_rows"), vr = maybe_tensor(a[10], "v_rows");
    if (R < 0) refuse("n_rows must be >= 0");
    const Q8Pool p = q8_pool_of(k, v, ks, vs);
    const Batch b = batch_of(offs, pages, lens);
    const at::ScalarType type = bf16 ? at::kBFloat16 : at::kFloat;
    for (Maybe t : {kr, vr})
        if (t && (t->dim() != 3 || t->size(0) != R || t->size(1) != p.Hkv || t->size(2) != p.D || t->scalar_type() != type))
            refuse("k_rows and v_rows must be [n_rows, Hkv, D] of the dtype asked for");
    const int dev = on_one_device({&offs, &k, &v, &ks, &vs, &pages, &lens, kr, vr});
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    at::Tensor new_k, new_v;
    ra_status st;
    {
        const Unlocked unlocked;
        if (!kr) kr = &(new_k = empty_on(dev, {R, p.Hkv, p.D}, type));
        if (!vr) vr = &(new_v = empty_on(dev, {R, p.Hkv, p.D}, type));
        st = ra_cache_read_paged_q8(pointer<int>(&offs), b.n_seqs, R, pointer(&k), pointer(&v), p.k_scales, p.v_scales,
                                    p.n_pages, p.page_size, pointer<int>(&pages), b.max_pages, pointer<int>(&lens), pointer(kr),
                                    pointer(vr), p.Hkv, p.D, bf16 ? RA_BF16 : RA_F32, stream_of(dev));
    }
    if (st != RA_OK) return status_object(st);
    PyObject* o = result(new_k, a[9]);
    return Py_BuildValue("NN", o, result(new_v, a[10]));
}

// q_rows, row_offsets, k_pages, v_pages, k_scales, v_scales, pages, kv_lens, tree_mask, out, lse, workspace, want_lse
PyObject* tree_attn_q8(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q_rows"), &offs = tensor(a[1], "row_offsets"), &k = tensor(a[2], "k_pages"),
                     &v = tensor(a[3], "v_pages"), &ks = tensor(a[4], "k_scales"), &vs = tensor(a[5], "v_scales"),
                     &pages = tensor(a[6], "pages"), &lens = tensor(a[7], "kv_lens");
    Maybe mask = maybe_tensor(a[8], "tree_mask"), out = maybe_tensor(a[9], "out"), lse = maybe_tensor(a[10], "lse"),
          ws = maybe_tensor(a[11], "workspace");
    const bool want_lse = PyObject_IsTrue(a[12]) > 0;
    if (q.dim() != 3) refuse("q_rows must be [R, Hq, D]");
    const int R = size_of(q, 0), Hq = size_of(q, 1), D = size_of(q, 2);
    const Q8Pool p = q8_pool_of(k, v, ks, vs);
    const Batch b = batch_of(offs, pages, lens);
    const int cols = mask_cols(mask, R);
    if (p.D != D) refuse("q_rows and the page pools disagree in D");
    const ra_dtype dt = type_of(q);
    if (out && (!out->sizes().equals(q.sizes()) || out->scalar_type() != q.scalar_type()))
        refuse("out must be shaped and typed as q_rows");
    if (lse && (lse->dim() != 2 || lse->size(0) != Hq || lse->size(1) != R || lse->scalar_type() != at::kFloat))
        refuse("lse must be fp32 [Hq, R]");
    const int dev = on_one_device({&q, &offs, &k, &v, &ks, &vs, &pages, &lens, mask, out, lse, ws});
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
            bytes = ra_tree_attn_q8_workspace_size(R, b.n_seqs, Hq, p.Hkv, D, dt);
            ws = &(new_ws = empty_on(dev, {static_cast<int64_t>(std::max<size_t>(bytes, 1))}, at::kByte));
        }
        st = ra_tree_attn_paged_q8(pointer(&q), pointer<int>(&offs), b.n_seqs, R, pointer(&k), pointer(&v), p.k_scales,
                                   p.v_scales, p.n_pages, p.page_size, pointer<int>(&pages), b.max_pages, pointer<int>(&lens),
                                   pointer<unsigned char>(mask), cols, pointer(out), pointer<float>(lse), Hq, p.Hkv, D, dt,
                                   pointer(ws), bytes, stream_of(dev));
    }
    if (st != RA_OK) return status_object(st);
    PyObject* o = result(new_out, a[9]);
    return Py_BuildValue("NN", o, result(new_lse, a[10]));
}

// Tokens [..., heads, D] whose heads lie next to each other, a fixed number of elements apart.
struct Tokens {
    int64_t n, stride;
    int heads, D;
};
Tokens tokens_of(const at::Tensor& t, const char* name) {
    const int64_t dims = t.dim();
    if (dims < 3) throw Refused{PyExc_ValueError, std::string(name) + " must be [..., heads, D]"};
    Tokens r{1, 0, size_of(t, static_cast<int>(dims) - 2), size_of(t, static_cast<int>(dims) - 1)};
    const int64_t row = static_cast<int64_t>(r.heads) * r.D;
    bool dense = (t.stride(dims - 1) == 1 || r.D == 1) && (t.stride(dims - 2) == r.D || r.heads == 1);
    r.stride = row;
    for (int64_t i = dims - 3; i >= 0; --i) {  // the leading dimensions as one
        const int64_t n = t.size(i);
        if (n != 1) {
            if (r.n == 1)
                r.stride = t.stride(i);
            else
                dense = dense && t.stride(i) == r.stride * r.n;
        }
        r.n *= n;
    }
    if (r.n > 0 && !dense)
        throw Refused{PyExc_ValueError, std::string(name) + " must have dense heads, and tokens at a fixed stride"};
    if (r.n <= 1) r.stride = row;
    return r;
}

// What the norm and its gradient share: arguments 0 to 8 are q, k, q_weight, k_weight, positions, inv_freq, sections,
// eps, interleaved.
struct NormCall {
    const at::Tensor &q, &k;
    Maybe wq, wk, positions, freq;
    Tokens tq, tk;
    int R, rot, sections[4], n_axes;
    bool interleaved;
    float eps;
    ra_dtype dt;
};
NormCall norm_call(PyObject* const* a) {
    NormCall c{tensor(a[0], "q"), tensor(a[1], "k"), maybe_tensor(a[2], "q_weight"), maybe_tensor(a[3], "k_weight"),
               maybe_tensor(a[4], "positions"), maybe_tensor(a[5], "inv_freq")};
    c.tq = tokens_of(c.q, "q");
    c.tk = tokens_of(c.k, "k");
    c.dt = type_of(c.q);
    if (c.k.scalar_type() != c.q.scalar_type() || c.k.dim() != c.q.dim() || c.tk.D != c.tq.D ||
        !c.k.sizes().slice(0, c.k.dim() - 2).equals(c.q.sizes().slice(0, c.q.dim() - 2)))
        refuse("q and k must be [..., heads, D] of the same tokens, D and dtype");
    if (c.tq.n > INT_MAX) refuse("a tensor has more than 2^31 - 1 tokens");
    c.R = static_cast<int>(c.tq.n);
    if (!c.wq != !c.wk) refuse("q_weight and k_weight must both be given, or neither");
    for (Maybe w : {c.wq, c.wk})
        if (w && (w->dim() != 1 || w->size(0) != c.tq.D || w->scalar_type() != c.q.scalar_type()))
            refuse("q_weight and k_weight must be [D] of q's dtype");
    const double eps = PyFloat_AsDouble(a[7]);
    if (eps == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
    c.eps = static_cast<float>(eps);
    c.interleaved = PyObject_IsTrue(a[8]) > 0;
    if (!c.positions != !c.freq) refuse("positions and inv_freq must both be given, or neither");
    if (!c.freq) {
        if (a[6] != Py_None) refuse("sections need positions and inv_freq");
        return c;
    }
    if (c.freq->dim() != 1 || c.freq->scalar_type() != at::kFloat) refuse("inv_freq must be fp32 [rot / 2]");
    if (c.freq->size(0) == 0 || c.freq->size(0) > c.tq.D / 2) refuse("inv_freq must have between 1 and D / 2 entries");
    c.rot = 2 * static_cast<int>(c.freq->size(0));
    int32(c.positions, "positions");
    if (a[6] == Py_None) {
        c.n_axes = 1;
        c.sections[0] = c.rot / 2;
    } else {
        if (!PyTuple_Check(a[6]) && !PyList_Check(a[6])) throw Refused{PyExc_TypeError, "sections must be a tuple or list of integers"};
        const Py_ssize_t n = PySequence_Size(a[6]);
        if (n < 1 || n > 4) refuse("sections must be of one to four axes");
        c.n_axes = static_cast<int>(n);
        for (int i = 0; i < c.n_axes; ++i) {
            PyObject* item = PySequence_GetItem(a[6], i);
            if (!item) throw Refused{nullptr, ""};
            struct Drop {
                PyObject* o;
                ~Drop() { Py_DECREF(o); }
            } drop{item};
            c.sections[i] = integer(item, "sections");
        }
    }
    // [axes, ...] with the tokens of q, or [...] for one axis
    const int64_t lead = c.q.dim() - 2;
    const auto tokens = c.q.sizes().slice(0, lead);
    const bool plain = c.n_axes == 1 && c.positions->sizes().equals(tokens);
    if (!plain && !(c.positions->dim() == lead + 1 && c.positions->size(0) == c.n_axes && c.positions->sizes().slice(1).equals(tokens)))
        refuse("positions must be int32 [axes, ...] over q's tokens ([...] for one axis)");
    return c;
}

// q and k (and what is shaped like them) may be slices; the rest is contiguous.
int norm_device(const NormCall& c, std::initializer_list<Maybe> slices, std::initializer_list<Maybe> more) {
    int dev = on_one_device({c.wq, c.wk, c.positions, c.freq});
    const int dev2 = on_one_device(more);
    if (dev < 0) dev = dev2;
    for (Maybe t : slices) {
        if (!t) continue;
        if (!t->is_cuda()) refuse("tensors must be on a CUDA device");
        if (dev < 0) dev = static_cast<int>(t->get_device());
        if (t->get_device() != dev) refuse("tensors must be on one device");
    }
    if (dev2 >= 0 && dev2 != dev) refuse("tensors must be on one device");
    return dev;
}

Tokens like(Maybe t, const at::Tensor& what, const Tokens& dense, const char* name) {
    if (!t) return {dense.n, static_cast<int64_t>(dense.heads) * dense.D, dense.heads, dense.D};
    if (!t->sizes().equals(what.sizes()) || t->scalar_type() != what.scalar_type())
        throw Refused{PyExc_ValueError, std::string(name) + " must be shaped and typed as its input"};
    return tokens_of(*t, name);
}

// ..., q_out, k_out
PyObject* qk_norm_rope(PyObject* const* a) {
    const NormCall c = norm_call(a);
    Maybe qo = maybe_tensor(a[9], "q_out"), ko = maybe_tensor(a[10], "k_out");
    const Tokens tqo = like(qo, c.q, c.tq, "q_out"), tko = like(ko, c.k, c.tk, "k_out");
    const int dev = norm_device(c, {&c.q, &c.k, qo, ko}, {});
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    at::Tensor new_q, new_k;
    ra_status st;
    {
        const Unlocked unlocked;
        if (!qo) qo = &(new_q = empty_on(dev, c.q.sizes(), c.q.scalar_type()));
        if (!ko) ko = &(new_k = empty_on(dev, c.k.sizes(), c.k.scalar_type()));
        st = ra_qk_norm_rope(pointer(&c.q), c.tq.stride, pointer(&c.k), c.tk.stride, pointer(c.wq), pointer(c.wk),
                             pointer<int>(c.positions), pointer<float>(c.freq), pointer(qo), tqo.stride, pointer(ko), tko.stride,
                             c.R, c.tq.heads, c.tk.heads, c.tq.D, c.rot, c.sections, c.n_axes, c.interleaved, c.eps, c.dt,
                             stream_of(dev));
    }
    if (st != RA_OK) return status_object(st);
    PyObject* o = result(new_q, a[9]);
    return Py_BuildValue("NN", o, result(new_k, a[10]));
}

// ..., dq_out, dk_out, dq, dk, workspace
PyObject* qk_norm_rope_bwd(PyObject* const* a) {
    const NormCall c = norm_call(a);
    const at::Tensor &gq = tensor(a[9], "dq_out"), &gk = tensor(a[10], "dk_out");
    Maybe dq = maybe_tensor(a[11], "dq"), dk = maybe_tensor(a[12], "dk"), ws = maybe_tensor(a[13], "workspace");
    if (!gq.sizes().equals(c.q.sizes()) || !gk.sizes().equals(c.k.sizes()) || gq.scalar_type() != c.q.scalar_type() ||
        gk.scalar_type() != c.q.scalar_type())
        refuse("dq_out and dk_out must be shaped and typed as q and k");
    const Tokens tdq = like(dq, c.q, c.tq, "dq"), tdk = like(dk, c.k, c.tk, "dk");
    const int dev = norm_device(c, {&c.q, &c.k, dq, dk}, {&gq, &gk, ws});
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    at::Tensor new_dq, new_dk, new_ws, dwq, dwk;
    ra_status st;
    {
        const Unlocked unlocked;
        if (!dq) dq = &(new_dq = empty_on(dev, c.q.sizes(), c.q.scalar_type()));
        if (!dk) dk = &(new_dk = empty_on(dev, c.k.sizes(), c.k.scalar_type()));
        size_t bytes = ws ? static_cast<size_t>(ws->numel()) * ws->element_size() : 0;
        if (c.wq) {
            dwq = empty_on(dev, {c.tq.D}, at::kFloat);
            dwk = empty_on(dev, {c.tq.D}, at::kFloat);
            if (!ws) {
                bytes = ra_qk_norm_rope_bwd_workspace_size(c.tq.D);
                ws = &(new_ws = empty_on(dev, {static_cast<int64_t>(std::max<size_t>(bytes, 1))}, at::kByte));
            }
        }
        st = ra_qk_norm_rope_bwd(pointer(&c.q), c.tq.stride, pointer(&c.k), c.tk.stride, pointer(c.wq), pointer(c.wk),
                                 pointer<int>(c.positions), pointer<float>(c.freq), pointer(&gq), pointer(&gk), pointer(dq),
                                 tdq.stride, pointer(dk), tdk.stride, dwq.defined() ? dwq.data_ptr<float>() : nullptr,
                                 dwk.defined() ? dwk.data_ptr<float>() : nullptr, c.R, c.tq.heads, c.tk.heads, c.tq.D, c.rot,
                                 c.sections, c.n_axes, c.interleaved, c.eps, c.dt, pointer(ws), bytes, stream_of(dev));
    }
    if (st != RA_OK) return status_object(st);
    PyObject *o = result(new_dq, a[11]), *k = result(new_dk, a[12]);
    return Py_BuildValue("NNNN", o, k, dwq.defined() ? result(dwq, nullptr) : Py_NewRef(Py_None),
                         dwk.defined() ? result(dwk, nullptr) : Py_NewRef(Py_None));
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
                         method<cache_append, 7>("cache_append"), method<cache_append_q8, 9>("cache_append_q8"),
                         method<cache_read_q8, 11>("cache_read_q8"), method<tree_attn_q8, 13>("tree_attn_q8"),
                         method<qk_norm_rope, 11>("qk_norm_rope"), method<qk_norm_rope_bwd, 14>("qk_norm_rope_bwd"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module_def); }
