// Argument checks and calls of the E2M1 entry points for the Python binding.
//
// The C ABI takes pointers and sizes; this module reads them from torch tensors,
// checks every tensor's type, device, shape and contiguity, and calls the
// library function whose address it is given.  In Python the same checks cost
// more than the kernels of a small decode step (14 us a call against 5 to 9 us on
// the device); here they take well under a microsecond.  It computes nothing.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

namespace {

using at::Tensor;

bool fail(PyObject* type, const char* format, const char* name) {
  PyErr_Format(type, format, name);
  return false;
}

// The tensor of an argument, or null with an error set.
const Tensor* tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s is not a tensor", name);
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

// Memory that the kernels may address: on the device, or pinned on the host (as the
// graph runner's staging and output rows are).
bool reachable(const Tensor& t, int device) {
  return t.get_device() == device || (t.device().is_cpu() && t.is_pinned());
}

// A contiguous, reachable tensor of that type and shape.
bool fits(const Tensor& t, const char* name, at::ScalarType type, int device,
          std::initializer_list<int64_t> shape) {
  if (t.scalar_type() != type)
    return fail(PyExc_TypeError, "%s has the wrong dtype for this call", name);
  if (!reachable(t, device))
    return fail(PyExc_ValueError, "%s is not on the device of the caches", name);
  if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size()))
    return fail(PyExc_ValueError, "%s has the wrong shape for this call", name);
  if (!t.is_contiguous()) return fail(PyExc_ValueError, "%s must be contiguous", name);
  return true;
}

// An argument that may be None: its pointer, or null.
bool optional(PyObject* o, const char* name, at::ScalarType type, int device,
              std::initializer_list<int64_t> shape, void** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const Tensor* t = tensor(o, name);
  if (t == nullptr || !fits(*t, name, type, device, shape)) return false;
  *p = t->data_ptr();
  return true;
}

// A pair of caches [num_blocks, num_kv_heads, 9 head_dim] on the current device.
struct Caches {
  void *k, *v;
  int device;
  int64_t blocks, heads, dim;
};
bool caches(PyObject* k, PyObject* v, int device, Caches* c) {
  const Tensor *kt = tensor(k, "k_cache"), *vt = kt ? tensor(v, "v_cache") : nullptr;
  if (vt == nullptr) return false;
  if (!kt->is_cuda() || kt->get_device() != device)
    return fail(PyExc_ValueError, "%s is not on the current CUDA device", "k_cache");
  if (kt->dim() != 3 || kt->size(2) % 9 != 0)
    return fail(PyExc_ValueError, "%s: an E2M1 cache is [num_blocks, num_kv_heads, 9 * head_dim]",
                "k_cache");
  *c = {kt->data_ptr(), vt->data_ptr(), device, kt->size(0), kt->size(1), kt->size(2) / 9};
  const int64_t page = kt->size(2);
  if (!vt->is_cuda()) return fail(PyExc_ValueError, "%s is not on a CUDA device", "v_cache");
  return fits(*kt, "k_cache", at::kByte, device, {c->blocks, c->heads, page}) &&
         fits(*vt, "v_cache", at::kByte, device, {c->blocks, c->heads, page});
}

bool integer(PyObject* o, int64_t* v) {
  *v = PyLong_AsLongLong(o);
  return *v != -1 || !PyErr_Occurred();
}
bool number(PyObject* o, float* v) {
  const double d = PyFloat_AsDouble(o);
  *v = static_cast<float>(d);
  return d != -1.0 || !PyErr_Occurred();
}
bool as_int(int64_t v) { return v >= INT32_MIN && v <= INT32_MAX; }

PyObject* guarded(PyObject* (*f)(PyObject* const*, Py_ssize_t), PyObject* const* args,
                  Py_ssize_t n) {
  try {
    return f(args, n);
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
}

// rows(function, write, k_rows, v_rows, slots, k_cache, v_cache, k_scale, v_scale,
//      error_flag, device, stream) -> status
PyObject* rows(PyObject* const* a, Py_ssize_t n) {
  if (n != 12) return PyErr_Format(PyExc_TypeError, "rows takes 12 arguments");
  int64_t fn, device, stream;
  float ks, vs;
  Caches c;
  if (!integer(a[0], &fn) || !integer(a[10], &device) || !integer(a[11], &stream) ||
      !number(a[7], &ks) || !number(a[8], &vs) ||
      !caches(a[5], a[6], static_cast<int>(device), &c))
    return nullptr;
  const Tensor* kr = tensor(a[2], "k rows");
  const Tensor* vr = kr ? tensor(a[3], "v rows") : nullptr;
  const Tensor* slots = vr ? tensor(a[4], "slot_mapping") : nullptr;
  if (slots == nullptr) return nullptr;
  const at::ScalarType type = kr->scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) {
    PyErr_SetString(PyExc_TypeError, "rows are float32 or bfloat16");
    return nullptr;
  }
  const int64_t count = slots->numel();
  void* flag;
  if (!fits(*kr, "k rows", type, c.device, {count, c.heads, c.dim}) ||
      !fits(*vr, "v rows", type, c.device, {count, c.heads, c.dim}) ||
      !fits(*slots, "slot_mapping", at::kLong, c.device, {count}) ||
      !optional(a[9], "error_flag", at::kInt, c.device, {1}, &flag))
    return nullptr;
  if (!as_int(c.heads) || !as_int(c.dim))
    return PyErr_Format(PyExc_ValueError, "the caches are too large");
  using Fn = int (*)(const void*, const void*, const void*, int64_t, const void*, const void*,
                     int64_t, int, int, int, int, float, float, void*, void*);
  const bool write = PyObject_IsTrue(a[1]);
  const void *first[2] = {kr->data_ptr(), vr->data_ptr()}, *last[2] = {c.k, c.v};
  const void** x = write ? first : last;
  const void** y = write ? last : first;
  const int status = reinterpret_cast<Fn>(fn)(
      x[0], x[1], slots->data_ptr(), count, y[0], y[1], c.blocks, 16, static_cast<int>(c.heads),
      static_cast<int>(c.dim), type == at::kBFloat16 ? 1 : 0, ks, vs, flag,
      reinterpret_cast<void*>(stream));
  return PyLong_FromLong(status);
}

// attention(function, write, k_new, v_new, slots, q, k_cache, v_cache, out,
//           query_start_loc, seq_lens, block_table, max_query_len, max_seq_len,
//           softmax_scale, k_scale, v_scale, causal, num_splits, workspace, lse_out,
//           error_flag, window, device, stream) -> status
// `write` says which of the two signatures the function has; k_new, v_new and slots
// are tensors then, and are not looked at otherwise.
PyObject* attention(PyObject* const* args, Py_ssize_t n) {
  if (n != 25) return PyErr_Format(PyExc_TypeError, "attention takes 25 arguments");
  const int write = PyObject_IsTrue(args[1]);
  if (write < 0) return nullptr;
  PyObject* const* a = args + 1;                         // (a[1], a[2], a[3]: the new rows)
  const Tensor *k = nullptr, *v = nullptr, *slots = nullptr;
  if (write) {
    k = tensor(a[1], "k_new");
    v = k ? tensor(a[2], "v_new") : nullptr;
    slots = v ? tensor(a[3], "slot_mapping") : nullptr;
    if (slots == nullptr) return nullptr;
  }
  int64_t fn, device, stream, mq, ms, splits, window;
  float scale, ks, vs;
  Caches c;
  if (!integer(args[0], &fn) || !integer(a[22], &device) || !integer(a[23], &stream) ||
      !integer(a[11], &mq) || !integer(a[12], &ms) || !integer(a[17], &splits) ||
      !integer(a[21], &window) || !number(a[13], &scale) || !number(a[14], &ks) ||
      !number(a[15], &vs) || !caches(a[5], a[6], static_cast<int>(device), &c))
    return nullptr;
  const Tensor* q = tensor(a[4], "q");
  const Tensor* out = q ? tensor(a[7], "out") : nullptr;
  const Tensor* qsl = out ? tensor(a[8], "query_start_loc") : nullptr;
  const Tensor* lens = qsl ? tensor(a[9], "seq_lens") : nullptr;
  const Tensor* table = lens ? tensor(a[10], "block_table") : nullptr;
  if (table == nullptr) return nullptr;
  if (q->dim() != 3) return PyErr_Format(PyExc_ValueError, "q is [num_tokens, Hq, head_dim]");
  if (table->dim() != 2)
    return PyErr_Format(PyExc_ValueError, "block_table is [num_seqs, max_blocks_per_seq]");
  const int64_t tokens = q->size(0), hq = q->size(1), seqs = lens->numel(), width = table->size(1);
  void *lse, *flag;
  if (!fits(*q, "q", at::kBFloat16, c.device, {tokens, hq, c.dim}) ||
      !fits(*out, "out", at::kBFloat16, c.device, {tokens, hq, c.dim}) ||
      !fits(*qsl, "query_start_loc", at::kInt, c.device, {seqs + 1}) ||
      !fits(*lens, "seq_lens", at::kInt, c.device, {seqs}) ||
      !fits(*table, "block_table", at::kInt, c.device, {seqs, width}) ||
      !optional(a[19], "lse_out", at::kFloat, c.device, {tokens, hq}, &lse) ||
      !optional(a[20], "error_flag", at::kInt, c.device, {1}, &flag))
    return nullptr;
  void* workspace = nullptr;
  size_t workspace_bytes = 0;
  if (a[18] != Py_None) {
    const Tensor* w = tensor(a[18], "workspace");
    if (w == nullptr) return nullptr;
    if (w->get_device() != c.device || !w->is_contiguous())
      return PyErr_Format(PyExc_ValueError,
                          "workspace is a contiguous tensor on the device of the caches");
    workspace = w->data_ptr();
    workspace_bytes = static_cast<size_t>(w->nbytes());
  }
  if (!as_int(c.heads) || !as_int(c.dim) || !as_int(hq) || !as_int(seqs) || !as_int(width) ||
      !as_int(mq) || !as_int(ms) || !as_int(splits) || !as_int(window))
    return PyErr_Format(PyExc_ValueError, "a size or count does not fit 32 bits");
  const int causal = PyObject_IsTrue(a[16]);
  if (causal < 0) return nullptr;
  auto i = [](int64_t v) { return static_cast<int>(v); };
  int status;
  if (!write) {
    using Fn = int (*)(const void*, const void*, const void*, void*, void*, const void*,
                       const void*, const void*, int, int, int64_t, int, int, int, int, int, int,
                       float, float, float, int, int, int, void*, size_t, void*, int64_t, void*);
    status = reinterpret_cast<Fn>(fn)(
        q->data_ptr(), c.k, c.v, out->data_ptr(), lse, qsl->data_ptr(), lens->data_ptr(),
        table->data_ptr(), i(width), i(seqs), tokens, i(mq), i(ms), i(hq), i(c.heads), i(c.dim),
        16, scale, ks, vs, causal, i(window), i(splits), workspace, workspace_bytes, flag,
        c.blocks, reinterpret_cast<void*>(stream));
  } else {
    if (!fits(*k, "k_new", at::kBFloat16, c.device, {tokens, c.heads, c.dim}) ||
        !fits(*v, "v_new", at::kBFloat16, c.device, {tokens, c.heads, c.dim}) ||
        !fits(*slots, "slot_mapping", at::kLong, c.device, {tokens}))
      return nullptr;
    using Fn = int (*)(const void*, const void*, const void*, const void*, void*, void*, void*,
                       void*, const void*, const void*, const void*, int, int, int64_t, int, int,
                       int, int, int, int, float, float, float, int, int, int, void*, size_t,
                       void*, int64_t, void*);
    status = reinterpret_cast<Fn>(fn)(
        k->data_ptr(), v->data_ptr(), slots->data_ptr(), q->data_ptr(), c.k, c.v, out->data_ptr(),
        lse, qsl->data_ptr(), lens->data_ptr(), table->data_ptr(), i(width), i(seqs), tokens,
        i(mq), i(ms), i(hq), i(c.heads), i(c.dim), 16, scale, ks, vs, causal, i(window), i(splits),
        workspace, workspace_bytes, flag, c.blocks, reinterpret_cast<void*>(stream));
  }
  return PyLong_FromLong(status);
}

PyObject* py_rows(PyObject*, PyObject* const* a, Py_ssize_t n) { return guarded(rows, a, n); }
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(attention, a, n);
}

PyMethodDef methods[] = {
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_rows)), METH_FASTCALL,
     "Check the tensors of a row call and make it; returns its status."},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_attention)),
     METH_FASTCALL, "Check the tensors of an attention call and make it; returns its status."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
