// Marshalling of the calls that a decode step makes for each layer: tensors looked at
// and a function of the library called, without an object of Python's in between.
// kv.py and rope.py look at every argument themselves and word what they refuse; here an
// argument that is not plainly right gives None, and they take the call over.  A step's
// calls are short on the GPU, 2 to 5 us, and the host has to keep ahead of them: with
// ctypes and the checks in Python append took 6.6 us of host time, now 2.4 (1.6 of them
// the launch), append_rotated 8.6, now 2.5, attention 8.0 and 3.4, a rotation 5.7 and 2.7.
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "../../include/dec.h"

namespace {

// What a cache's or a rotation's calls have in common.
struct Context {
  const void* desc;
  int device;
  int64_t heads, head_dim;  // KV heads (0: a rotation)
  void* calls[4];
};

enum Call { APPEND = 0, READ = 1, ATTENTION = 2, APPEND_ROTATED = 3, ROTATE = 0 };

const char* const kName = "tld context";

Context* context_of(PyObject* o) { return static_cast<Context*>(PyCapsule_GetPointer(o, kName)); }

// A [n, heads, head_dim] tensor with whole rows, as KVCache._rows has it.
struct Rows {
  void* at;
  int type;
  int64_t n, heads, stride;
};
bool rows_of(const Context& c, PyObject* o, int64_t heads, Rows* r) {
  if (!THPVariable_CheckExact(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || t.layout() != at::kStrided || t.dim() != 3 || !t.is_cuda() || t.get_device() != c.device) return false;
  const auto size = t.sizes(), step = t.strides();
  if (size[2] != c.head_dim || (heads >= 0 && size[1] != heads) || step[2] != 1 || (step[1] != size[2] && size[1] != 1))
    return false;
  if (t.scalar_type() == at::kFloat) r->type = DEC_IO_F32;
  else if (t.scalar_type() == at::kBFloat16) r->type = DEC_IO_BF16;
  else return false;
  r->at = t.data_ptr();
  r->n = size[0];
  r->heads = size[1];
  r->stride = size[0] > 1 ? step[0] : size[1] * size[2];
  return r->n <= INT32_MAX && r->heads <= INT32_MAX;
}

// A list of n int32 numbers, or none.
bool list_of(const Context& c, PyObject* o, int64_t n, const int32_t** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  if (!THPVariable_CheckExact(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || t.layout() != at::kStrided || t.dim() != 1 || !t.is_cuda() || t.get_device() != c.device) return false;
  if (t.scalar_type() != at::kInt || t.size(0) != n || !t.is_contiguous()) return false;
  *p = static_cast<const int32_t*>(t.data_ptr());
  return true;
}

bool int_of(PyObject* o, int* x) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  const long y = PyLong_AsLongAndOverflow(o, &over);
  if (over || y < 0 || y > INT32_MAX) return false;
  *x = (int)y;
  return true;
}

// Looks the arguments over with `look`, which fills in a call, and makes it on the current
// stream: the call's answer, or None.
template <class Look>
PyObject* make(PyObject* const* args, Py_ssize_t n, Py_ssize_t wanted, const Look& look) {
  if (n != wanted) {
    PyErr_SetString(PyExc_TypeError, "another number of arguments is wanted");
    return nullptr;
  }
  const Context* c = context_of(args[0]);
  if (!c) return nullptr;
  int rc = 0;
  try {
    if (c10::cuda::current_device() != c->device) Py_RETURN_NONE;
    auto call = look(*c);
    if (!call.ok) Py_RETURN_NONE;
    const dec_stream_t s = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c->device).stream();
    PyThreadState* held = PyEval_SaveThread();
    rc = call(s);
    PyEval_RestoreThread(held);
  } catch (const std::exception&) {  // (of the looking over: the library throws nothing)
    Py_RETURN_NONE;
  }
  return PyLong_FromLong(rc);
}

struct AppendCall {
  bool ok = false;
  const Context* c = nullptr;
  int layer = 0;
  Rows k, v;
  const int32_t *seqs = nullptr, *positions = nullptr;
  void* call = nullptr;
  int operator()(dec_stream_t s) const {
    using Fn = int (*)(const void*, int, void*, void*, int, int64_t, const int32_t*, const int32_t*, int, dec_stream_t);
    return reinterpret_cast<Fn>(call)(c->desc, layer, k.at, v.at, k.type, k.stride, seqs, positions, (int)k.n, s);
  }
};
template <class C>
bool keys_and_values(const Context& c, PyObject* const* a, C* call) {
  call->c = &c;
  return int_of(a[0], &call->layer) && rows_of(c, a[1], c.heads, &call->k) && rows_of(c, a[2], c.heads, &call->v) &&
         call->k.n == call->v.n && call->k.type == call->v.type && call->k.stride == call->v.stride &&
         list_of(c, a[3], call->k.n, &call->seqs) && list_of(c, a[4], call->k.n, &call->positions);
}

// append(context, layer, k, v, seqs, positions)
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return make(args, n, 6, [&](const Context& c) {
    AppendCall call;
    call.ok = keys_and_values(c, args + 1, &call);
    call.call = c.calls[APPEND];
    return call;
  });
}

// read(context, layer, k_out, v_out, seqs, positions)
PyObject* read(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return make(args, n, 6, [&](const Context& c) {
    AppendCall call;
    call.ok = args[4] != Py_None && keys_and_values(c, args + 1, &call);
    call.call = c.calls[READ];
    return call;
  });
}

struct RotatedCall : AppendCall {
  const void* rope = nullptr;
  Rows q{}, out{};
  int operator()(dec_stream_t s) const {
    using Fn = int (*)(const void*, int, const void*, void*, void*, int64_t, int64_t, int, void*, void*, int, int64_t,
                       const int32_t*, const int32_t*, int, dec_stream_t);
    return reinterpret_cast<Fn>(call)(c->desc, layer, rope, q.at, out.at, q.stride, out.stride, (int)q.heads, k.at, v.at,
                                      k.type, k.stride, seqs, positions, (int)k.n, s);
  }
};

// append_rotated(context, layer, k, v, seqs, positions, the rotation's context, q or None, q_out)
PyObject* append_rotated(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return make(args, n, 9, [&](const Context& c) {
    RotatedCall call;
    call.ok = keys_and_values(c, args + 1, &call);
    call.call = c.calls[APPEND_ROTATED];
    const Context* r = PyCapsule_IsValid(args[6], kName) ? context_of(args[6]) : nullptr;
    call.ok = call.ok && r && r->device == c.device;
    if (call.ok) call.rope = r->desc;
    if (call.ok && args[7] != Py_None)
      call.ok = rows_of(c, args[7], -1, &call.q) && rows_of(c, args[8], call.q.heads, &call.out) &&
                call.q.type == call.k.type && call.out.type == call.k.type && call.q.n == call.k.n && call.out.n == call.k.n;
    return call;
  });
}

struct AttentionCall {
  bool ok = false;
  const Context* c = nullptr;
  int layer = 0, window = 0, sinks = 0;
  Rows q, out;
  const int32_t* seqs = nullptr;
  float scale = 0;
  void* workspace = nullptr;
  size_t bytes = 0;
  int operator()(dec_stream_t s) const {
    using Fn = int (*)(const void*, int, void*, void*, int, int64_t, int64_t, const int32_t*, int, int, int, int, float,
                       void*, size_t, dec_stream_t);
    return reinterpret_cast<Fn>(c->calls[ATTENTION])(c->desc, layer, q.at, out.at, q.type, q.stride, out.stride, seqs,
                                                     (int)q.n, (int)q.heads, window, sinks, scale, workspace, bytes, s);
  }
};

// attention(context, layer, q, out, seqs, window, sinks, scale, workspace's address, its bytes)
PyObject* attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return make(args, n, 10, [&](const Context& c) {
    AttentionCall call;
    call.c = &c;
    call.ok = int_of(args[1], &call.layer) && rows_of(c, args[2], -1, &call.q) && rows_of(c, args[3], call.q.heads, &call.out) &&
              call.q.type == call.out.type && call.q.n == call.out.n && list_of(c, args[4], call.q.n, &call.seqs) &&
              int_of(args[5], &call.window) && int_of(args[6], &call.sinks) && PyFloat_CheckExact(args[7]) &&
              PyLong_CheckExact(args[8]) && PyLong_CheckExact(args[9]);
    if (call.ok) {
      call.scale = (float)PyFloat_AS_DOUBLE(args[7]);
      call.workspace = PyLong_AsVoidPtr(args[8]);
      call.bytes = PyLong_AsSize_t(args[9]);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        call.ok = false;
      }
    }
    return call;
  });
}

struct RotateCall {
  bool ok = false;
  const Context* c = nullptr;
  Rows x, out;
  const int32_t* positions = nullptr;
  int backward = 0;
  int operator()(dec_stream_t s) const {
    using Fn = int (*)(const void*, void*, void*, int, int64_t, int64_t, const int32_t*, int, int, int, dec_stream_t);
    return reinterpret_cast<Fn>(c->calls[ROTATE])(c->desc, x.at, out.at, x.type, x.stride, out.stride, positions, (int)x.n,
                                                  (int)x.heads, backward, s);
  }
};

// rotate(context, x, positions, out, backward)
PyObject* rotate(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return make(args, n, 5, [&](const Context& c) {
    RotateCall call;
    call.c = &c;
    call.ok = rows_of(c, args[1], -1, &call.x) && call.x.heads > 0 && list_of(c, args[2], call.x.n, &call.positions) &&
              rows_of(c, args[3], call.x.heads, &call.out) && call.x.type == call.out.type && call.x.n == call.out.n &&
              PyBool_Check(args[4]);
    call.backward = args[4] == Py_True;
    return call;
  });
}

// context(description's address, device, heads, head_dim, addresses of up to four functions)
PyObject* make_context(PyObject*, PyObject* args) {
  unsigned long long desc = 0, f[4] = {0, 0, 0, 0};
  int device = 0;
  long long heads = 0, head_dim = 0;
  if (!PyArg_ParseTuple(args, "KiLLK|KKK", &desc, &device, &heads, &head_dim, &f[0], &f[1], &f[2], &f[3])) return nullptr;
  Context* c = new (std::nothrow) Context{reinterpret_cast<const void*>(desc), device, heads, head_dim, {}};
  if (!c) return PyErr_NoMemory();
  for (int i = 0; i < 4; ++i) c->calls[i] = reinterpret_cast<void*>(f[i]);
  return PyCapsule_New(c, kName, [](PyObject* o) { delete context_of(o); });
}

#define TLD_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef kMethods[] = {{"context", make_context, METH_VARARGS, nullptr},
                          {"append", TLD_FAST(append), nullptr},
                          {"read", TLD_FAST(read), nullptr},
                          {"append_rotated", TLD_FAST(append_rotated), nullptr},
                          {"attention", TLD_FAST(attention), nullptr},
                          {"rotate", TLD_FAST(rotate), nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "tld_calls", "Marshalling of a decode step's calls.", -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit_tld_calls(void) { return PyModule_Create(&kModule); }
