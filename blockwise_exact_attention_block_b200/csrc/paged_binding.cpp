// paged_binding.cpp - the paged cache's calls for Python: a CPython extension
// that checks torch tensors, allocates outputs, and calls the C ABI.
//
// A decoding step makes several of these calls for every token, each of a few
// microseconds on the GPU.  Checked and marshalled in Python with ctypes a call
// takes 10 to 20 us of the host; here it takes about a third of that.  The C
// functions are handed in as addresses, so the release and the checked library
// share this module.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <string>

#include "ra.h"

namespace {

std::string text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + ")";
}

// The tensor behind a Python argument; null (with an error set) for anything else.
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
  PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return nullptr;
}

// Checks that o is a contiguous CUDA tensor of this type and shape on `device` and
// takes its address; None gives a null address where `optional`.
bool expect(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int device, void** address,
            bool optional = false) {
  *address = nullptr;
  if (o == Py_None && optional) return true;
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  if (t->scalar_type() != type || t->sizes() != shape || !t->is_cuda() || t->get_device() != device ||
      !t->is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous %s tensor %s on cuda:%d, got %s %s on %s%s", name,
                 c10::toString(type), text(shape).c_str(), device, c10::toString(t->scalar_type()),
                 text(t->sizes()).c_str(), t->device().str().c_str(), t->is_contiguous() ? "" : ", not contiguous");
    return false;
  }
  *address = t->data_ptr();
  return true;
}

bool fail(const char* what) {
  PyErr_SetString(PyExc_ValueError, what);
  return false;
}

bool integer(PyObject* o, const char* name, int* value) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return false;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_Format(PyExc_ValueError, "%s does not fit 32 bits", name);
    return false;
  }
  *value = static_cast<int>(v);
  return true;
}

// The extents of a tensor argument as ints (the C ABI's type).
bool fits(at::IntArrayRef shape) {
  for (int64_t n : shape)
    if (n > INT32_MAX) return fail("a tensor's extent does not fit 32 bits");
  return true;
}

bool code_of(at::ScalarType t, ra_dtype* code) {
  if (t == at::kBFloat16) *code = RA_BF16;
  else if (t == at::kFloat) *code = RA_F32;
  else return fail((std::string("unsupported dtype ") + c10::toString(t)).c_str());
  return true;
}

struct Batch {
  ra_paged_cache c{};
  int device = 0;
};

bool parse_batch(PyObject* table, PyObject* lens, PyObject* news, Batch* b) {
  const at::Tensor* t = tensor(table, "page_table");
  if (!t) return false;
  if (t->dim() != 2) return fail("page_table must be [B, max_pages]");
  if (!fits(t->sizes())) return false;
  const int64_t B = t->size(0);
  b->c.B = static_cast<int>(B);
  b->c.max_pages = static_cast<int>(t->size(1));
  void *pt, *ps, *pn;
  if (!expect(table, "page_table", at::kInt, t->sizes(), b->device, &pt)) return false;
  if (!expect(lens, "seq_lens", at::kInt, {B}, b->device, &ps)) return false;
  if (!expect(news, "new_lens", at::kInt, {B}, b->device, &pn, true)) return false;
  b->c.page_table = static_cast<const int32_t*>(pt);
  b->c.seq_lens = static_cast<const int32_t*>(ps);
  b->c.new_lens = static_cast<const int32_t*>(pn);
  return true;
}

bool parse_cache(PyObject* k_pages, PyObject* v_pages, PyObject* k_scales, PyObject* v_scales, PyObject* bounds,
                 PyObject* table, PyObject* lens, PyObject* news, Batch* b) {
  const at::Tensor* k = tensor(k_pages, "k_pages");
  if (!k) return false;
  if (!k->is_cuda()) return fail("tensors must be contiguous CUDA tensors");
  const at::ScalarType type = k->scalar_type();
  if (k->dim() != 4 || (type != at::kBFloat16 && type != at::kChar && type != at::kFloat8_e4m3fn))
    return fail("k_pages must be [n_pages, Hkv, page_size, D] in bfloat16, int8 or float8_e4m3fn");
  const at::IntArrayRef s = k->sizes();
  if (!fits(s)) return false;
  b->device = k->get_device();
  b->c.dtype = type == at::kBFloat16 ? RA_BF16 : type == at::kChar ? RA_I8 : RA_E4M3;
  b->c.n_pages = static_cast<int>(s[0]);
  b->c.Hkv = static_cast<int>(s[1]);
  b->c.page_size = static_cast<int>(s[2]);
  b->c.D = static_cast<int>(s[3]);
  const bool scaled = type != at::kBFloat16;
  if (scaled != (k_scales != Py_None) || scaled != (v_scales != Py_None))
    return fail("an 8-bit cache has k_scales and v_scales, a bfloat16 one has none");
  void *ks, *vs;
  if (!expect(k_pages, "k_pages", type, s, b->device, &b->c.k_pages)) return false;
  if (!expect(v_pages, "v_pages", type, s, b->device, &b->c.v_pages)) return false;
  if (!expect(k_scales, "k_scales", at::kFloat, s.slice(0, 3), b->device, &ks, true)) return false;
  if (!expect(v_scales, "v_scales", at::kFloat, s.slice(0, 3), b->device, &vs, true)) return false;
  if (!expect(bounds, "key_bounds", at::kBFloat16, {s[0], s[1], 2, s[3]}, b->device, &b->c.key_bounds, true)) return false;
  b->c.k_scales = static_cast<float*>(ks);
  b->c.v_scales = static_cast<float*>(vs);
  return parse_batch(table, lens, news, b);
}

// Makes the device and the stream of a call current while it allocates and
// launches: a given stream (its handle as an int) owns the workspace and the new
// outputs, as if the call stood under torch.cuda.stream(); None is the device's
// current stream.
class Place {
 public:
  bool enter(PyObject* o, int device) {
    const auto index = static_cast<c10::DeviceIndex>(device);
    device_.set_index(index);
    if (o == Py_None) {
      handle = c10::cuda::getCurrentCUDAStream(index).stream();
      return true;
    }
    void* const p = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) return false;
    const c10::cuda::CUDAStream s = p ? c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), index)
                                      : c10::cuda::getDefaultCUDAStream(index);
    stream_.reset_stream(s);
    handle = p;
    return true;
  }
  void* handle = nullptr;

 private:
  c10::cuda::OptionalCUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard stream_;
};

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, int device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(device)));
}

// A given output, or a new one: a new reference to its Python object.
PyObject* output(PyObject* given, const char* name, at::IntArrayRef shape, at::ScalarType type, int device, void** address) {
  if (given != Py_None) {
    if (!expect(given, name, type, shape, device, address)) return nullptr;
    Py_INCREF(given);
    return given;
  }
  at::Tensor t = make(shape, type, device);
  *address = t.data_ptr();
  return THPVariable_Wrap(std::move(t));
}

// The element type asked for: out_dtype, or that of the given output, or `fallback`.
bool out_type(PyObject* dtype, PyObject* given, at::ScalarType fallback, at::ScalarType* type) {
  if (THPDtype_Check(dtype)) *type = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  else if (dtype != Py_None) return fail("out_dtype must be a torch.dtype");
  else if (given != Py_None && THPVariable_Check(given)) *type = THPVariable_Unpack(given).scalar_type();
  else *type = fallback;
  return true;
}

// A workspace: the given tensor's bytes, or a new one of `need`.
bool scratch(PyObject* given, size_t need, int device, at::Tensor* hold, void** address, size_t* bytes) {
  if (given == Py_None) {
    *hold = make({static_cast<int64_t>(need)}, at::kByte, device);
    *address = hold->data_ptr();
    *bytes = need;
    return true;
  }
  const at::Tensor* t = tensor(given, "workspace");
  if (!t) return false;
  if (!t->is_cuda() || t->get_device() != device || !t->is_contiguous())
    return fail("workspace must be a contiguous CUDA tensor on the cache's device");
  *address = t->data_ptr();
  *bytes = t->nbytes();
  return true;
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

template <typename Fn>
Fn function(PyObject* address) {
  return reinterpret_cast<Fn>(PyLong_AsVoidPtr(address));
}

constexpr size_t kInvalid = static_cast<size_t>(-1);

// append(fn, k, v, k_pages, v_pages, page_table, seq_lens, new_lens, k_scales, v_scales, key_bounds, stream) -> status
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Batch b;
  if (!count(n, 12) || !parse_cache(a[3], a[4], a[8], a[9], a[10], a[5], a[6], a[7], &b)) return nullptr;
  const at::Tensor* k = tensor(a[1], "k");
  if (!k) return nullptr;
  if (k->dim() != 4) return fail("k must be [B, T, Hkv, D]"), nullptr;
  const int64_t T = k->size(1);
  const int64_t shape[4] = {b.c.B, T, b.c.Hkv, b.c.D};
  Place at;
  void *pk, *pv;
  ra_dtype code;
  if (!fits(k->sizes()) || !expect(a[1], "k", k->scalar_type(), shape, b.device, &pk) ||
      !expect(a[2], "v", k->scalar_type(), shape, b.device, &pv) || !code_of(k->scalar_type(), &code) ||
      !at.enter(a[11], b.device))
    return nullptr;
  const auto fn = function<decltype(&ra_cache_append)>(a[0]);
  return PyLong_FromLong(fn(&b.c, pk, pv, code, static_cast<int>(T), at.handle));
  END_HANDLE_TH_ERRORS
}

// read(fn, k_pages, v_pages, page_table, seq_lens, T, first, k_scales, v_scales, k, v, out_dtype, stream) -> status, k, v
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Batch b;
  int T, first;
  at::ScalarType type;
  ra_dtype code;
  if (!count(n, 13) || !parse_cache(a[1], a[2], a[7], a[8], Py_None, a[3], a[4], Py_None, &b) || !integer(a[5], "T", &T) ||
      !integer(a[6], "first", &first) || !out_type(a[11], a[9] != Py_None ? a[9] : a[10], at::kBFloat16, &type) ||
      !code_of(type, &code))
    return nullptr;
  const int64_t shape[4] = {b.c.B, T > 0 ? T : 0, b.c.Hkv, b.c.D};
  Place at;
  void *pk, *pv;
  if (!at.enter(a[12], b.device)) return nullptr;
  THPObjectPtr k(output(a[9], "k", shape, type, b.device, &pk));
  if (!k) return nullptr;
  THPObjectPtr v(output(a[10], "v", shape, type, b.device, &pv));
  if (!v) return nullptr;
  const auto fn = function<decltype(&ra_cache_read)>(a[0]);
  const int status = fn(&b.c, first, T, pk, pv, code, at.handle);
  return Py_BuildValue("iNN", status, k.release(), v.release());
  END_HANDLE_TH_ERRORS
}

// decode(fn, workspace_fn, q, k_pages, v_pages, page_table, seq_lens, new_lens, k_scales, v_scales, causal, selected,
//        out, lse, out_dtype, workspace, stream) -> status, out, lse
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Batch b;
  if (!count(n, 17) || !parse_cache(a[3], a[4], a[8], a[9], Py_None, a[5], a[6], a[7], &b)) return nullptr;
  const at::Tensor* q = tensor(a[2], "q");
  if (!q) return nullptr;
  if (q->dim() != 4) return fail("q must be [B, Tq, Hq, D]"), nullptr;
  const int64_t shape[4] = {b.c.B, q->size(1), q->size(2), b.c.D};
  const at::IntArrayRef rows(shape, 3);
  const int causal = PyObject_IsTrue(a[10]);
  Place at;
  void *pq, *ps = nullptr, *po, *pl, *pw;
  ra_dtype in_code, out_code;
  at::ScalarType type;
  if (causal < 0 || !fits(q->sizes()) || !expect(a[2], "q", q->scalar_type(), shape, b.device, &pq) ||
      !code_of(q->scalar_type(), &in_code) || !out_type(a[14], a[12], at::kFloat, &type) || !code_of(type, &out_code) ||
      !at.enter(a[16], b.device))
    return nullptr;
  int n_sel = 0;
  if (a[11] != Py_None) {
    const at::Tensor* sel = tensor(a[11], "selected");
    if (!sel) return nullptr;
    if (sel->dim() != 3 || !fits(sel->sizes())) return fail("selected must be [B, Hkv, n_sel]"), nullptr;
    n_sel = static_cast<int>(sel->size(2));
    if (!expect(a[11], "selected", at::kInt, {b.c.B, b.c.Hkv, n_sel}, b.device, &ps)) return nullptr;
    // lists of no entries have no address, which the C call takes for the whole cache
    if (n_sel == 0) return Py_BuildValue("iOO", RA_ERR_INVALID_ARG, Py_None, Py_None);
  }
  const int Tq = static_cast<int>(shape[1]), Hq = static_cast<int>(shape[2]);
  at::Tensor hold;
  size_t bytes = 0;
  const size_t need = function<decltype(&ra_paged_decode_workspace)>(a[1])(b.c.B, Tq, Hq, b.c.Hkv, b.c.D);
  if (!scratch(a[15], need == kInvalid ? 0 : need, b.device, &hold, &pw, &bytes)) return nullptr;
  THPObjectPtr out(output(a[12], "out", shape, type, b.device, &po));
  if (!out) return nullptr;
  THPObjectPtr lse(output(a[13], "lse", rows, at::kFloat, b.device, &pl));
  if (!lse) return nullptr;
  const auto fn = function<decltype(&ra_paged_decode_attention)>(a[0]);
  const int status = fn(pq, in_code, &b.c, Tq, Hq, causal, static_cast<const int32_t*>(ps), n_sel, po, out_code,
                        static_cast<float*>(pl), pw, bytes, at.handle);
  return Py_BuildValue("iNN", status, out.release(), lse.release());
  END_HANDLE_TH_ERRORS
}

// select(fn, workspace_fn, q, key_bounds, page_table, seq_lens, n_sel, page_size, new_lens, selected, workspace, stream)
//   -> status, selected
PyObject* select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 12)) return nullptr;
  Batch b;
  const at::Tensor *q = tensor(a[2], "q"), *kb = tensor(a[3], "key_bounds");
  if (!q || !kb) return nullptr;
  if (!kb->is_cuda()) return fail("tensors must be contiguous CUDA tensors"), nullptr;
  if (q->dim() != 4 || kb->dim() != 4 || kb->size(2) != 2)
    return fail("q must be [B, Tq, Hq, D] and key_bounds [n_pages, Hkv, 2, D]"), nullptr;
  int n_sel;
  if (!fits(q->sizes()) || !fits(kb->sizes()) || !integer(a[6], "n_sel", &n_sel) ||
      !integer(a[7], "page_size", &b.c.page_size))
    return nullptr;
  b.device = kb->get_device();
  b.c.dtype = RA_BF16;
  b.c.n_pages = static_cast<int>(kb->size(0));
  b.c.Hkv = static_cast<int>(kb->size(1));
  b.c.D = static_cast<int>(kb->size(3));
  if (!parse_batch(a[4], a[5], a[8], &b)) return nullptr;
  const int64_t shape[4] = {b.c.B, q->size(1), q->size(2), b.c.D};
  const int64_t places[3] = {b.c.B, b.c.Hkv, n_sel > 0 ? n_sel : 0};
  Place at;
  void *pq, *ps, *pw;
  ra_dtype code;
  if (!expect(a[3], "key_bounds", at::kBFloat16, kb->sizes(), b.device, &b.c.key_bounds) ||
      !expect(a[2], "q", q->scalar_type(), shape, b.device, &pq) || !code_of(q->scalar_type(), &code) ||
      !at.enter(a[11], b.device))
    return nullptr;
  at::Tensor hold;
  size_t bytes = 0;
  const size_t need = function<decltype(&ra_page_select_workspace)>(a[1])(b.c.B, b.c.Hkv, b.c.max_pages);
  if (!scratch(a[10], need == kInvalid ? 0 : need, b.device, &hold, &pw, &bytes)) return nullptr;
  THPObjectPtr sel(output(a[9], "selected", places, at::kInt, b.device, &ps));
  if (!sel) return nullptr;
  const auto fn = function<decltype(&ra_page_select)>(a[0]);
  const int status = fn(pq, code, &b.c, static_cast<int>(shape[1]), static_cast<int>(shape[2]), n_sel,
                        static_cast<int32_t*>(ps), pw, bytes, at.handle);
  return Py_BuildValue("iN", status, sel.release());
  END_HANDLE_TH_ERRORS
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(append), ENTRY(read), ENTRY(decode), ENTRY(select), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", "Calls of the paged key-value cache.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// What the module was compiled against (build.py looks for it, and compiles it anew for another).
const char built_for[] = RA_BINDING_TAG;

PyMODINIT_FUNC PyInit__paged(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", built_for) < 0) Py_CLEAR(m);
  return m;
}
