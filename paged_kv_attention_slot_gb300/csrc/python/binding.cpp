// The Python calls of a decode step over selected pages (token_map, rope_store, bound_keys, select, run with blocks): checks
// of the tensors, outputs and the library's call in one step.
//
// Their kernels take 2 to 10 us on a decode step, so what a call costs on the host is what it costs.  Through ctypes and
// Python's own checks a call with its outputs took 10.6 us (token map of 256 requests), 16.8 (rotary write of 64 tokens), 4.0
// (key bounds of a step) and 13.0 (selection, 512 units); here it takes 5.0, 5.4, 3.2 and 8.1, of which the driver's launch is
// 2.4 (one GB300's host, Python 3.12).  The functions check and marshal only: everything that runs is behind the C ABI, whose
// addresses attach() receives.
//
// Conventions: a tensor argument that may be absent is None; `stream` is what the caller was given, None for torch's current
// stream, to which outputs made here belong (for another stream the caller passes outputs); `owner` is the Plan or Rotary whose
// buffers the call uses and `streams` its set of the handles that they are recorded on.  A wrong argument raises ValueError (one of
// a wrong kind TypeError), an error status of the library what `check` raises.  Memory is asked for and kernels are launched
// without the interpreter's lock: the allocator's own lock may be held by a thread that waits for it.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>

#include "pkv_attn.h"

namespace {

struct Api {
  decltype(&pkv_token_map) token_map;
  decltype(&pkv_rope_kv_store) rope_kv_store;
  decltype(&pkv_key_bounds_update) key_bounds_update;
  decltype(&pkv_block_select) block_select;
  decltype(&pkv_attn_decode_run_blocks) decode_run_blocks;
} api;
PyObject* check_status = nullptr;  // called with a status other than PKV_OK: raises

#define REQUIRE(cond, ...)                       \
  do {                                           \
    if (!(cond)) {                               \
      PyErr_Format(PyExc_ValueError, __VA_ARGS__); \
      return nullptr;                            \
    }                                            \
  } while (0)

struct Shape3 {
  int64_t a, b, c;
};

// The arguments of a call, in order; after a failure (a Python error is set) the rest are zeros.
class Args {
 public:
  Args(PyObject* const* args, Py_ssize_t given, Py_ssize_t wanted) : at_(args) {
    if (given != wanted) {
      PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", given, wanted);
      ok_ = false;
    }
  }
  bool ok() const { return ok_; }
  int64_t integer() {
    PyObject* o = next();
    if (!o) return 0;
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) ok_ = false;
    return v;
  }
  int32_t int32() {
    PyObject* o = next();
    if (!o) return 0;
    int overflow = 0;
    const int64_t v = PyLong_AsLongLongAndOverflow(o, &overflow);
    if (overflow || (v != (int32_t)v)) {
      PyErr_Format(PyExc_ValueError, "%S does not fit 32 bits", o);
      ok_ = false;
    } else if (v == -1 && PyErr_Occurred()) {
      ok_ = false;
    }
    return ok_ ? (int32_t)v : 0;
  }
  bool truth() {
    PyObject* o = next();
    const int v = o ? PyObject_IsTrue(o) : 0;
    if (v < 0) ok_ = false;
    return v > 0;
  }
  double real() {
    PyObject* o = next();
    if (!o) return 0;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) ok_ = false;
    return v;
  }
  template <typename T>
  T* pointer() {
    return reinterpret_cast<T*>(static_cast<uintptr_t>(integer()));
  }
  const at::Tensor* tensor(bool may_be_absent = false) {
    PyObject* o = next();
    if (!o || (may_be_absent && o == Py_None)) return nullptr;
    if (!THPVariable_Check(o)) {
      PyErr_SetString(PyExc_TypeError, "a torch.Tensor is wanted");
      ok_ = false;
      return nullptr;
    }
    return &THPVariable_Unpack(o);
  }
  Shape3 shape3() {
    PyObject* o = next();
    Shape3 s{};
    if (o && !(PyTuple_Check(o) && PyArg_ParseTuple(o, "LLL", &s.a, &s.b, &s.c))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "a shape of three is wanted");
      ok_ = false;
    }
    return s;
  }
  PyObject* object() { return next(); }

 private:
  PyObject* next() { return ok_ ? *at_++ : nullptr; }
  PyObject* const* at_;
  bool ok_ = true;
};

bool is(const at::Tensor& t, at::ScalarType type, int64_t device) {
  return t.scalar_type() == type && t.is_contiguous() && t.get_device() == device;
}
bool shape3(const at::Tensor& t, int64_t a, int64_t b, int64_t c) {
  return t.dim() == 3 && t.size(0) == a && t.size(1) == b && t.size(2) == c;
}
bool on_current_device(int64_t device) { return device >= 0 && device == c10::cuda::current_device(); }
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, int64_t device) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)device));
}

// The tensors of a KeyBounds, whose attributes a program may have exchanged since it was made
bool are_bounds(const at::Tensor& codes, const at::Tensor& scale) {
  if (codes.scalar_type() == at::kChar && codes.dim() == 4 && codes.size(2) == 2 && codes.is_contiguous() &&
      is(scale, at::kFloat, codes.get_device()) && scale.dim() == 2 && scale.size(0) == codes.size(1) && scale.size(1) == codes.size(3))
    return true;
  PyErr_SetString(PyExc_ValueError, "bounds.codes must be a contiguous int8 tensor [num_pages, num_kv_heads, 2, head_dim], bounds.scale a "
                                    "contiguous float32 tensor [num_kv_heads, head_dim] on its device");
  return false;
}

// The handle of the stream to launch on; false: a Python error is set.
bool handle_of(PyObject* stream, int64_t device, void*& handle) {
  if (stream == Py_None) {
    handle = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    return true;
  }
  PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
  if (!h) return false;
  handle = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  return handle || !PyErr_Occurred();
}

// The same for a call that uses an owner's buffers, which are recorded on the stream the first time it is seen.
struct OwnedStream {
  PyObject *owner, *streams, *stream;
  explicit OwnedStream(Args& a) : owner(a.object()), streams(a.object()), stream(a.object()) {}
  bool use(int64_t device, void*& handle) const {
    if (!handle_of(stream, device, handle)) return false;
    PyObject* h = PyLong_FromVoidPtr(handle);
    if (!h) return false;
    const int seen = PySet_Contains(streams, h);
    Py_DECREF(h);
    if (seen) return seen > 0;
    PyObject* r = PyObject_CallMethod(owner, "_use", "O", stream);
    Py_XDECREF(r);
    return r != nullptr;
  }
};

struct Unlocked {  // without the interpreter's lock
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// f() makes outputs and calls the library, whose status it returns
template <typename F>
bool call(F f) {
  int status;
  {
    Unlocked u;
    status = f();
  }
  if (status == PKV_OK) return true;
  PyObject* r = PyObject_CallFunction(check_status, "i", status);
  if (r) {
    Py_DECREF(r);
    PyErr_SetString(PyExc_RuntimeError, "an error status of the library raised nothing");
  }
  return false;
}
// a tensor that the caller passed (a new reference), or one made here
PyObject* result(PyObject* given, const at::Tensor& made) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(made);
}
PyObject* pair(PyObject* a, PyObject* b) {
  if (!a || !b) {
    Py_XDECREF(a);
    Py_XDECREF(b);
    return nullptr;
  }
  PyObject* t = PyTuple_New(2);
  if (!t) {
    Py_DECREF(a);
    Py_DECREF(b);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  return t;
}

// attach(check, token_map, rope_kv_store, key_bounds_update, block_select, decode_run_blocks): the library's addresses
PyObject* attach(PyObject*, PyObject* const* args, Py_ssize_t n) {
  Args a(args + 1, n - 1, 5);
  api.token_map = reinterpret_cast<decltype(api.token_map)>(a.integer());
  api.rope_kv_store = reinterpret_cast<decltype(api.rope_kv_store)>(a.integer());
  api.key_bounds_update = reinterpret_cast<decltype(api.key_bounds_update)>(a.integer());
  api.block_select = reinterpret_cast<decltype(api.block_select)>(a.integer());
  api.decode_run_blocks = reinterpret_cast<decltype(api.decode_run_blocks)>(a.integer());
  if (!a.ok()) return nullptr;
  Py_INCREF(args[0]);
  Py_XSETREF(check_status, args[0]);
  Py_RETURN_NONE;
}

// token_map(plan, owner, streams, stream, tokens, batch, workspace, offsets, positions, slots) -> (positions, slots)
PyObject* token_map(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 10);
  auto* plan = a.pointer<const pkv_plan>();
  const OwnedStream on(a);
  const int64_t tokens = a.integer(), batch = a.integer();
  const at::Tensor* workspace = a.tensor();
  const at::Tensor* offsets = a.tensor(true);
  const at::Tensor* positions = a.tensor(true);
  const at::Tensor* slots = a.tensor(true);
  if (!a.ok()) return nullptr;
  const int64_t device = workspace->get_device();
  REQUIRE(!offsets || (is(*offsets, at::kLong, device) && offsets->dim() == 1 && offsets->size(0) == batch),
          "offsets must be a contiguous int64 tensor [%lld] on the plan's device", (long long)batch);
  REQUIRE(on_current_device(device), "the plan's workspace must be on the current CUDA device");
  void* stream;
  if (!on.use(device, stream)) return nullptr;
  at::Tensor p, s;
  if (!call([&] {
        p = positions ? *positions : make({tokens}, at::kLong, device);
        s = slots ? *slots : make({tokens}, at::kLong, device);
        return api.token_map(plan, offsets ? static_cast<const int64_t*>(offsets->data_ptr()) : nullptr,
                             static_cast<int64_t*>(p.data_ptr()), static_cast<int64_t*>(s.data_ptr()), stream);
      }))
    return nullptr;
  return pair(result(args[8], p), result(args[9], s));
  END_HANDLE_TH_ERRORS
}

// rope_store(cache, device, owner, streams, stream, q, k, v, positions, slots, phase_step, rotary_head_dim, rotary_dim,
//            interleaved, amplitude, scores, q_out, k_out, return_k) -> q or (q, k)
PyObject* rope_store(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 19);
  auto* cache = a.pointer<const pkv_cache>();
  const int64_t device = a.integer();
  const OwnedStream on(a);
  const at::Tensor *q = a.tensor(), *k = a.tensor(), *v = a.tensor(), *positions = a.tensor(), *slots = a.tensor();
  const at::Tensor* step = a.tensor();
  pkv_rope_args r{};
  const int64_t rotary_head_dim = a.integer();
  r.rotary_dim = a.int32();
  r.interleaved = a.int32();
  r.amplitude = (float)a.real();
  r.scores = a.pointer<float>();
  const at::Tensor *q_out = a.tensor(true), *k_out = a.tensor(true);
  const bool return_k = a.truth() || k_out;
  if (!a.ok()) return nullptr;
  const int64_t H = cache->num_kv_heads, D = cache->head_dim;
  REQUIRE(q->dim() == 3, "q must be [T, num_qo_heads, head_dim]");
  const int64_t T = q->size(0), Hq = q->size(1);
  REQUIRE(q->size(2) == D && shape3(*k, T, H, D) && shape3(*v, T, H, D),
          "q must be [T, num_qo_heads, head_dim], k and v [T, num_kv_heads, head_dim] of the cache's geometry");
  REQUIRE(Hq <= INT32_MAX, "num_qo_heads does not fit 32 bits");
  REQUIRE(rotary_head_dim == D, "the rotary is for head_dim %lld, the cache has %lld", (long long)rotary_head_dim, (long long)D);
  for (const at::Tensor* t : {q, k, v})
    REQUIRE(t->scalar_type() == at::kBFloat16 && t->stride(2) == 1 && t->get_device() == device,
            "q, k and v must be bf16 tensors on the cache's device with a contiguous last dimension");
  for (const at::Tensor* t : {positions, slots})
    REQUIRE(is(*t, at::kLong, device) && t->dim() == 1 && t->size(0) == T,
            "positions and slot_mapping must be contiguous int64 tensors [T] on the cache's device");
  REQUIRE(step->get_device() == device, "the rotary must be on the cache's device");
  REQUIRE(is(*step, at::kLong, device) && step->dim() == 1 && step->size(0) == r.rotary_dim / 2,
          "the rotary's phase_step must be a contiguous int64 tensor [rotary_dim / 2]");
  REQUIRE((!q_out || (is(*q_out, at::kBFloat16, device) && shape3(*q_out, T, Hq, D))) &&
              (!k_out || (is(*k_out, at::kBFloat16, device) && shape3(*k_out, T, H, D))),
          "q_out and k_out must be contiguous bf16 tensors like q and k");
  REQUIRE(on_current_device(device), "the cache must be on the current CUDA device");
  r.q = q->data_ptr();
  r.k = k->data_ptr();
  r.v = v->data_ptr();
  r.positions = static_cast<const int64_t*>(positions->data_ptr());
  r.slot_mapping = static_cast<const int64_t*>(slots->data_ptr());
  r.num_tokens = T;
  r.q_stride_token = q->stride(0), r.q_stride_head = q->stride(1);
  r.k_stride_token = k->stride(0), r.k_stride_head = k->stride(1);
  r.v_stride_token = v->stride(0), r.v_stride_head = v->stride(1);
  r.phase_step = static_cast<const uint64_t*>(step->data_ptr());
  r.num_qo_heads = (int32_t)Hq;
  void* stream;
  if (!on.use(device, stream)) return nullptr;
  at::Tensor qo, ko;
  if (!call([&] {
        qo = q_out ? *q_out : make({T, Hq, D}, at::kBFloat16, device);
        r.q_out = qo.data_ptr();
        if (return_k) {
          ko = k_out ? *k_out : make({T, H, D}, at::kBFloat16, device);
          r.k_out = ko.data_ptr();
        }
        return api.rope_kv_store(&r, cache, stream);
      }))
    return nullptr;
  PyObject* first = result(args[16], qo);
  return return_k ? pair(first, result(args[17], ko)) : first;
  END_HANDLE_TH_ERRORS
}

// bound_keys(plan, owner, streams, stream, cache, device, codes, scale, all_pages)
PyObject* bound_keys(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 9);
  auto* plan = a.pointer<const pkv_plan>();
  const OwnedStream on(a);
  auto* cache = a.pointer<const pkv_cache>();
  const int64_t device = a.integer();
  const at::Tensor *codes = a.tensor(), *scale = a.tensor();
  const int32_t all_pages = a.truth();
  if (!a.ok()) return nullptr;
  if (!are_bounds(*codes, *scale)) return nullptr;
  REQUIRE(codes->size(0) == cache->num_pages && codes->size(1) == cache->num_kv_heads && codes->size(3) == cache->head_dim,
          "the bounds do not match the cache's geometry");
  REQUIRE(codes->get_device() == device, "the bounds must be on the cache's device");
  REQUIRE(on_current_device(device), "the cache must be on the current CUDA device");
  void* stream;
  if (!on.use(device, stream)) return nullptr;
  if (!call([&] {
        return api.key_bounds_update(plan, cache, static_cast<int8_t*>(codes->data_ptr()),
                                     static_cast<const float*>(scale->data_ptr()), all_pages, stream);
      }))
    return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// select(plan, owner, streams, stream, (tokens, kv_heads, num_blocks), q_heads, head_dim, q, codes, scale, num_sink, num_recent,
//        blocks) -> blocks
PyObject* block_select(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 13);
  auto* plan = a.pointer<const pkv_plan>();
  const OwnedStream on(a);
  const Shape3 shape = a.shape3();
  const auto [T, H, K] = shape;
  const int64_t Hq = a.integer(), D = a.integer();
  const at::Tensor *q = a.tensor(), *codes = a.tensor(), *scale = a.tensor();
  const int32_t num_sink = a.int32(), num_recent = a.int32();
  const at::Tensor* blocks = a.tensor(true);
  if (!a.ok()) return nullptr;
  const int64_t device = codes->get_device();
  REQUIRE(is(*q, at::kBFloat16, device) && shape3(*q, T, Hq, D),
          "q must be a contiguous bf16 tensor [%lld, %lld, %lld] on the bounds' device", (long long)T, (long long)Hq, (long long)D);
  if (!are_bounds(*codes, *scale)) return nullptr;
  REQUIRE(codes->size(1) == H && codes->size(3) == D, "the bounds do not match the plan's KV heads and head_dim");
  REQUIRE(on_current_device(device), "the bounds must be on the current CUDA device");
  REQUIRE(!blocks || (is(*blocks, at::kInt, device) && shape3(*blocks, T, H, K)),
          "blocks must be a contiguous int32 tensor [%lld, %lld, %lld] on the bounds' device", (long long)T, (long long)H, (long long)K);
  void* stream;
  if (!on.use(device, stream)) return nullptr;
  at::Tensor b;
  if (!call([&, T = T, H = H, K = K] {
        b = blocks ? *blocks : make({T, H, K}, at::kInt, device);
        return api.block_select(plan, q->data_ptr(), static_cast<const int8_t*>(codes->data_ptr()),
                                static_cast<const float*>(scale->data_ptr()), codes->size(0), num_sink, num_recent,
                                static_cast<int32_t*>(b.data_ptr()), stream);
      }))
    return nullptr;
  return result(args[12], b);
  END_HANDLE_TH_ERRORS
}

// run_blocks(plan, owner, streams, stream, cache, device, (tokens, kv_heads, num_blocks), q_heads, head_dim, q, blocks, out,
//            lse, return_lse) -> out or (out, lse)
PyObject* run_blocks(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a(args, n, 14);
  auto* plan = a.pointer<const pkv_plan>();
  const OwnedStream on(a);
  auto* cache = a.pointer<const pkv_cache>();
  const int64_t device = a.integer();
  const Shape3 shape = a.shape3();
  const auto [T, H, K] = shape;
  const int64_t Hq = a.integer(), D = a.integer();
  const at::Tensor *q = a.tensor(), *blocks = a.tensor(), *out = a.tensor(true), *lse = a.tensor(true);
  const bool return_lse = a.truth() || lse;
  if (!a.ok()) return nullptr;
  REQUIRE(is(*blocks, at::kInt, device) && shape3(*blocks, T, H, K),
          "blocks must be a contiguous int32 tensor [%lld, %lld, %lld] on the cache's device", (long long)T, (long long)H, (long long)K);
  REQUIRE(is(*q, at::kBFloat16, device) && shape3(*q, T, Hq, D),
          "q must be a contiguous bf16 tensor [%lld, %lld, %lld] on the cache's device", (long long)T, (long long)Hq, (long long)D);
  REQUIRE(!out || (is(*out, at::kBFloat16, device) && shape3(*out, T, Hq, D)),
          "out must be a contiguous bf16 tensor [%lld, %lld, %lld] on the cache's device", (long long)T, (long long)Hq, (long long)D);
  REQUIRE(!lse || (is(*lse, at::kFloat, device) && lse->dim() == 2 && lse->size(0) == T && lse->size(1) == Hq),
          "lse must be a contiguous float32 tensor [%lld, %lld] on the cache's device", (long long)T, (long long)Hq);
  REQUIRE(on_current_device(device), "the cache must be on the current CUDA device");
  void* stream;
  if (!on.use(device, stream)) return nullptr;
  at::Tensor o, l;
  if (!call([&, T = T] {
        o = out ? *out : make({T, Hq, D}, at::kBFloat16, device);
        if (return_lse) l = lse ? *lse : make({T, Hq}, at::kFloat, device);
        return api.decode_run_blocks(plan, q->data_ptr(), cache, static_cast<const int32_t*>(blocks->data_ptr()), o.data_ptr(),
                                     return_lse ? static_cast<float*>(l.data_ptr()) : nullptr, stream);
      }))
    return nullptr;
  PyObject* first = result(args[11], o);
  return return_lse ? pair(first, result(args[12], l)) : first;
  END_HANDLE_TH_ERRORS
}

#define METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("attach", attach),         METHOD("token_map", token_map), METHOD("rope_store", rope_store),
                         METHOD("bound_keys", bound_keys), METHOD("select", block_select), METHOD("run_blocks", run_blocks),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyObject* PyInit__binding() { return PyModule_Create(&module); }
