// bind.cpp -- the Python binding of the paged-cache operators: argument
// marshalling only, as binding.py does it for the other entry points, but
// compiled.  These calls are made once a step or a layer and run for ten
// microseconds or less, so what the binding costs is what the user waits for:
// in Python the checks, the stream and the workspace of a call took 8 to 12 us.
//
// Every function checks the tensors (CUDA, one device, type, contiguous, size:
// ValueError), makes that device current, allocates what is not given on the
// current stream, and calls the C entry point of the same name; a status other
// than SPK_OK raises SpeckvError.  `stream` is None (the device's current
// stream) or a handle; with a handle, outputs and workspace are given.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <string>

#include "../../include/speckv.h"

namespace {

PyObject* g_error = nullptr;      // SpeckvError

struct Bad {                      // becomes a ValueError
  std::string what;
};

[[noreturn]] void bad(const char* fmt, ...) {
  char s[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(s, sizeof s, fmt, ap);
  va_end(ap);
  throw Bad{s};
}

struct Failed {};                 // a Python exception is set

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

int device_of(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda()) bad("%s must be a CUDA tensor", name);
  return t.get_device();
}

const char* type_name(at::ScalarType t) { return at::toString(t); }

// Data pointer of a contiguous tensor on CUDA device `index`; null for None.
// type Undefined: any; numel -1: any.
void* ptr(PyObject* o, const char* name, at::ScalarType type, int index, int64_t numel = -1) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda() || t.get_device() != index)
    bad("%s must be a CUDA tensor on cuda:%d, got one on %s", name, index, t.device().str().c_str());
  if (type != at::ScalarType::Undefined && t.scalar_type() != type)
    bad("%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
  if (!t.is_contiguous()) bad("%s must be contiguous", name);
  if (numel >= 0 && t.numel() != numel)
    bad("%s has %lld elements, the call needs %lld", name, static_cast<long long>(t.numel()), static_cast<long long>(numel));
  return t.data_ptr();
}

constexpr at::ScalarType kAny = at::ScalarType::Undefined, kInt = at::ScalarType::Int;

int32_t* ints(PyObject* o, const char* name, int index, int64_t numel = -1) {
  return static_cast<int32_t*>(ptr(o, name, kInt, index, numel));
}

int32_t* need_ints(PyObject* o, const char* name, int index, int64_t numel = -1) {
  if (o == Py_None) bad("%s is required", name);
  return ints(o, name, index, numel);
}

int number(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed{};
  if (v < INT32_MIN || v > INT32_MAX) bad("%s is out of range", name);
  return static_cast<int>(v);
}

int as_int(int64_t v, const char* name) {
  if (v > INT32_MAX) bad("%s is too large", name);
  return static_cast<int>(v);
}

void* stream_of(PyObject* o, int index) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw Failed{};
  return p;
}

void check(spk_status st) {
  if (st == SPK_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(st), spk_last_error());
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Failed{};
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int index) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(index))));
}

// The caller's workspace, or a temporary one of `bytes`.
struct Workspace {
  at::Tensor hold;
  void* p;
  size_t bytes;
  Workspace(PyObject* o, size_t need, int index) {
    if (o == Py_None) {
      bytes = need > 0 ? need : 256;
      hold = fresh({static_cast<int64_t>(bytes)}, at::kByte, index);
      p = hold.data_ptr();
    } else {
      p = ptr(o, "workspace", kAny, index);
      bytes = tensor(o, "workspace").nbytes();
    }
  }
};

PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// An int32 [1] result: the caller's, or a new one (returned either way).
PyObject* result_of(PyObject* o, int index) {
  return o != Py_None ? same(o) : THPVariable_Wrap(fresh({1}, kInt, index));
}

struct Held {                     // a reference that is dropped unless it is handed on
  PyObject* o;
  explicit Held(PyObject* x) : o(x) {
    if (o == nullptr) throw Failed{};
  }
  ~Held() { Py_XDECREF(o); }
  PyObject* out() {
    PyObject* x = o;
    o = nullptr;
    return x;
  }
};

// ------------------------------------------------------------------- shapes
void table_shape(spk_pages_shape& s, PyObject* refs, PyObject* table, PyObject* lens) {
  const at::Tensor& t = tensor(table, "page_table");
  if (t.dim() != 2) bad("page_table is [n_seqs, max_pages]");
  s.n_seqs = as_int(t.size(0), "n_seqs");
  s.max_pages = as_int(t.size(1), "max_pages");
  s.n_pages = as_int(tensor(refs, "page_refs").numel(), "n_pages");
  if (tensor(lens, "seq_lens").numel() != s.n_seqs)
    bad("seq_lens has %lld elements, the call needs %d", static_cast<long long>(tensor(lens, "seq_lens").numel()), s.n_seqs);
}

void pages_shape(spk_pages_shape& s, PyObject* k, PyObject* v, PyObject* refs, PyObject* table, PyObject* lens) {
  const at::Tensor &kt = tensor(k, "k_pages"), &vt = tensor(v, "v_pages");
  if (kt.dim() != 5 || kt.sizes() != vt.sizes() || kt.scalar_type() != vt.scalar_type())
    bad("k_pages and v_pages are [L, n_pages, Hkv, page_rows, d], of the same dtype");
  if (tensor(refs, "page_refs").numel() != kt.size(1))
    bad("page_refs has %lld elements, the call needs %lld", static_cast<long long>(tensor(refs, "page_refs").numel()),
        static_cast<long long>(kt.size(1)));
  table_shape(s, refs, table, lens);
  s.layers = as_int(kt.size(0), "layers");
  s.hkv = as_int(kt.size(2), "Hkv");
  s.page_rows = as_int(kt.size(3), "page_rows");
  s.head_dim = as_int(kt.size(4), "head_dim");
  s.elem_bytes = static_cast<int>(kt.element_size());
}

int length(PyObject* o, const char* name) { return as_int(tensor(o, name).numel(), name); }

int64_t lists_of(const spk_pages_shape& s, int n, int per) {
  const int64_t units = static_cast<int64_t>(n) * s.layers * s.hkv;
  if (per < 1 || units % per != 0)
    bad("units (%lld) must be a multiple of units_per_idx (%d)", static_cast<long long>(units), per);
  return units / per;
}

int columns(PyObject* idx) {
  const at::Tensor& t = tensor(idx, "idx");
  if (t.dim() < 1) bad("idx is [lists, n_idx]");
  return as_int(t.size(-1), "n_idx");
}

// ---------------------------------------------------------------- functions
#define SPK_CALL(NAME, COUNT)                                                                   \
  PyObject* NAME##_impl(PyObject* const* a);                                                    \
  PyObject* NAME(PyObject*, PyObject* const* a, Py_ssize_t n) {                                 \
    HANDLE_TH_ERRORS                                                                            \
    if (n != COUNT) {                                                                           \
      PyErr_SetString(PyExc_TypeError, #NAME " takes " #COUNT " arguments");                    \
      return nullptr;                                                                           \
    }                                                                                           \
    try {                                                                                       \
      return NAME##_impl(a);                                                                    \
    } catch (const Bad& e) {                                                                    \
      PyErr_SetString(PyExc_ValueError, e.what.c_str());                                        \
      return nullptr;                                                                           \
    } catch (const Failed&) {                                                                   \
      return nullptr;                                                                           \
    }                                                                                           \
    END_HANDLE_TH_ERRORS                                                                        \
  }                                                                                             \
  PyObject* NAME##_impl(PyObject* const* a)

// k_pages v_pages page_refs page_table seq_lens seqs n_new result workspace stream
SPK_CALL(py_kv_pages_reserve, 10) {
  const int index = device_of(a[0], "k_pages");
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  spk_pages_shape s{};
  pages_shape(s, a[0], a[1], a[2], a[3], a[4]);
  const int n = length(a[5], "seqs");
  Held result(result_of(a[7], index));
  const Workspace ws(a[8], a[8] == Py_None ? kv_pages_workspace_size(&s, n) : 0, index);
  check(kv_pages_reserve(&s, ptr(a[0], "k_pages", kAny, index), ptr(a[1], "v_pages", kAny, index),
                         need_ints(a[2], "page_refs", index), need_ints(a[3], "page_table", index),
                         need_ints(a[4], "seq_lens", index), need_ints(a[5], "seqs", index),
                         need_ints(a[6], "n_new", index, n), n, need_ints(result.o, "result", index, 1), ws.p, ws.bytes,
                         stream_of(a[9], index)));
  return result.out();
}

// k v k_pages v_pages page_refs page_table seq_lens seqs idx counts units_per_idx reserved stream
SPK_CALL(py_kv_pages_write, 13) {
  const int index = device_of(a[2], "k_pages");
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  spk_pages_shape s{};
  pages_shape(s, a[2], a[3], a[4], a[5], a[6]);
  const int n = length(a[7], "seqs");
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  if (k.dim() != 5 || k.sizes() != v.sizes() || k.size(0) != n || k.size(1) != s.layers || k.size(2) != s.hkv ||
      k.size(4) != s.head_dim)
    bad("k and v are [n, L, Hkv, n_src, d] with the pages' L, Hkv and d");
  const at::ScalarType type = tensor(a[2], "k_pages").scalar_type();
  const int n_src = as_int(k.size(3), "n_src");
  const int n_idx = a[8] == Py_None ? n_src : columns(a[8]), per = number(a[10], "units_per_idx");
  const int64_t lists = lists_of(s, n, per);
  check(kv_pages_write(&s, ptr(a[0], "k", type, index), ptr(a[1], "v", type, index), n_src,
                       ints(a[8], "idx", index, lists * n_idx), n_idx, per, ints(a[9], "counts", index, n),
                       need_ints(a[4], "page_refs", index), need_ints(a[5], "page_table", index),
                       need_ints(a[6], "seq_lens", index), need_ints(a[7], "seqs", index), n,
                       ptr(a[2], "k_pages", kAny, index), ptr(a[3], "v_pages", kAny, index),
                       ints(a[11], "reserved", index, 1), stream_of(a[12], index)));
  Py_RETURN_NONE;
}

// k_pages v_pages page_refs page_table seq_lens src dst idx units_per_idx result workspace stream
SPK_CALL(py_kv_pages_compact, 12) {
  const int index = device_of(a[0], "k_pages");
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  spk_pages_shape s{};
  pages_shape(s, a[0], a[1], a[2], a[3], a[4]);
  const int n = length(a[5], "src"), n_idx = columns(a[7]), per = number(a[8], "units_per_idx");
  const int64_t lists = lists_of(s, n, per);
  Held result(result_of(a[9], index));
  const Workspace ws(a[10], a[10] == Py_None ? kv_pages_workspace_size(&s, n) : 0, index);
  check(kv_pages_compact(&s, ptr(a[0], "k_pages", kAny, index), ptr(a[1], "v_pages", kAny, index),
                         need_ints(a[2], "page_refs", index), need_ints(a[3], "page_table", index),
                         need_ints(a[4], "seq_lens", index), need_ints(a[5], "src", index),
                         need_ints(a[6], "dst", index, n), n, need_ints(a[7], "idx", index, lists * n_idx), n_idx, per,
                         need_ints(result.o, "result", index, 1), ws.p, ws.bytes, stream_of(a[11], index)));
  return result.out();
}

// page_refs page_table seq_lens src dst page_rows n_rows result workspace stream
SPK_CALL(py_kv_pages_fork, 10) {
  const int index = device_of(a[1], "page_table");
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  spk_pages_shape s{};
  table_shape(s, a[0], a[1], a[2]);
  s.page_rows = number(a[5], "page_rows");
  const int n = length(a[3], "src");
  Held result(result_of(a[7], index));
  const Workspace ws(a[8], a[8] == Py_None ? kv_pages_workspace_size(&s, n) : 0, index);
  check(kv_pages_fork(&s, need_ints(a[0], "page_refs", index), need_ints(a[1], "page_table", index),
                      need_ints(a[2], "seq_lens", index), need_ints(a[3], "src", index), need_ints(a[4], "dst", index, n),
                      ints(a[6], "n_rows", index, n), n, need_ints(result.o, "result", index, 1), ws.p, ws.bytes,
                      stream_of(a[9], index)));
  return result.out();
}

// page_refs page_table seq_lens seqs page_rows keep_rows stream
SPK_CALL(py_kv_pages_free, 7) {
  const int index = device_of(a[1], "page_table");
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  spk_pages_shape s{};
  table_shape(s, a[0], a[1], a[2]);
  s.page_rows = number(a[4], "page_rows");
  const int n = length(a[3], "seqs");
  check(kv_pages_free(&s, need_ints(a[0], "page_refs", index), need_ints(a[1], "page_table", index),
                      need_ints(a[2], "seq_lens", index), need_ints(a[3], "seqs", index),
                      ints(a[5], "keep_rows", index, n), n, stream_of(a[6], index)));
  Py_RETURN_NONE;
}

// q k_pages v_pages page_table seq_lens k_tree v_tree mask n_live seqs out lse2 workspace scale stream
SPK_CALL(py_tree_attention, 15) {
  const int index = device_of(a[0], "q");
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  const at::Tensor &q = tensor(a[0], "q"), &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages"),
                   &table = tensor(a[3], "page_table");
  if (q.dim() != 5 || kp.dim() != 5 || table.dim() != 2)
    bad("q is [B, L, Hq, T, d], k_pages [L, n_pages, Hkv, page_rows, d], page_table [n_seqs, max_pages]");
  if (q.size(1) != kp.size(0) || q.size(4) != kp.size(4)) bad("q and k_pages disagree on layers or head_dim");
  const at::ScalarType type = q.scalar_type();
  if (type != at::kBFloat16 && type != at::kHalf) bad("q must be BFloat16 or Half, got %s", type_name(type));
  if (vp.sizes() != kp.sizes()) bad("v_pages must have k_pages' shape");
  if ((a[5] == Py_None) != (a[6] == Py_None)) bad("k_tree and v_tree are given together or not at all");
  spk_tree_shape s{};
  s.batch = as_int(q.size(0), "batch");
  s.layers = as_int(q.size(1), "layers");
  s.hq = as_int(q.size(2), "Hq");
  s.n_nodes = as_int(q.size(3), "T");
  s.head_dim = as_int(q.size(4), "head_dim");
  s.n_pages = as_int(kp.size(1), "n_pages");
  s.hkv = as_int(kp.size(2), "Hkv");
  s.page_rows = as_int(kp.size(3), "page_rows");
  s.n_seqs = as_int(table.size(0), "n_seqs");
  s.max_pages = as_int(table.size(1), "max_pages");
  s.dtype = type == at::kHalf ? SPK_FP16 : SPK_BF16;
  const double scale = PyFloat_AsDouble(a[13]);
  if (scale == -1.0 && PyErr_Occurred()) throw Failed{};
  s.scale = static_cast<float>(scale);
  const int64_t B = s.batch, T = s.n_nodes, rows = B * s.layers * s.hq * T;
  if (a[5] != Py_None) {
    const int64_t tree[5] = {B, s.layers, s.hkv, T, s.head_dim};
    if (tensor(a[5], "k_tree").sizes() != at::IntArrayRef(tree) || tensor(a[6], "v_tree").sizes() != at::IntArrayRef(tree))
      bad("k_tree and v_tree must be [%lld, %d, %d, %lld, %d]", static_cast<long long>(B), s.layers, s.hkv,
          static_cast<long long>(T), s.head_dim);
  }
  Held out(a[10] != Py_None ? same(a[10]) : THPVariable_Wrap(fresh(q.sizes(), type, index)));
  const Workspace ws(a[12], a[12] == Py_None ? tree_attention_workspace_size(&s) : 0, index);
  check(tree_attention(&s, ptr(a[0], "q", kAny, index), ptr(a[1], "k_pages", type, index), ptr(a[2], "v_pages", type, index),
                       need_ints(a[3], "page_table", index), need_ints(a[4], "seq_lens", index, s.n_seqs),
                       ints(a[9], "seqs", index, B), ptr(a[5], "k_tree", type, index), ptr(a[6], "v_tree", type, index),
                       reinterpret_cast<uint32_t*>(ints(a[7], "mask", index, B * T * ((T + 31) / 32))),
                       ints(a[8], "n_live", index, B), ptr(out.o, "out", type, index, rows * s.head_dim),
                       static_cast<float*>(ptr(a[11], "lse2", at::kFloat, index, rows)), ws.p, ws.bytes,
                       stream_of(a[14], index)));
  return out.out();
}

// parents n_live mask depth stream
SPK_CALL(py_tree_mask, 5) {
  const int index = device_of(a[0], "parents");
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  const at::Tensor& parents = tensor(a[0], "parents");
  if (parents.dim() != 2) bad("parents is [B, T]");
  const int64_t B = parents.size(0), T = parents.size(1), words = (T + 31) / 32;
  Held mask(a[2] != Py_None ? same(a[2]) : THPVariable_Wrap(fresh({B, T, words}, kInt, index)));
  Held depth(a[3] != Py_None ? same(a[3]) : THPVariable_Wrap(fresh({B, T}, kInt, index)));
  check(tree_mask(as_int(B, "B"), as_int(T, "T"), need_ints(a[0], "parents", index), ints(a[1], "n_live", index, B),
                  reinterpret_cast<uint32_t*>(need_ints(mask.o, "mask", index, B * T * words)),
                  need_ints(depth.o, "depth", index, B * T), stream_of(a[4], index)));
  return PyTuple_Pack(2, mask.o, depth.o);
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  g_error = same(cls);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}

PyMethodDef g_methods[] = {
    {"kv_pages_reserve", fast(py_kv_pages_reserve), METH_FASTCALL, nullptr},
    {"kv_pages_write", fast(py_kv_pages_write), METH_FASTCALL, nullptr},
    {"kv_pages_compact", fast(py_kv_pages_compact), METH_FASTCALL, nullptr},
    {"kv_pages_fork", fast(py_kv_pages_fork), METH_FASTCALL, nullptr},
    {"kv_pages_free", fast(py_kv_pages_free), METH_FASTCALL, nullptr},
    {"tree_attention", fast(py_tree_attention), METH_FASTCALL, nullptr},
    {"tree_mask", fast(py_tree_mask), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};
}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&g_module); }
