// py_grouped.cpp -- the Python binding of a serving step with grouped K/V heads.
//
// The kernels of a single-token step take 2 to 6 us; checking ten to seventeen
// tensor arguments and marshalling them through ctypes took 7 to 9 us of host
// time around them.  Here the checks read the tensors' own fields, so a call
// costs its launch.  Each function checks its arguments, takes the stream (the
// tensors' device's current one where none is given), makes that device current
// and calls the C entry point of the same name (include/pagedkv.h).  It returns
// the entry point's status, or -1 where an argument does not fit: the caller
// (grouped.py) then looks for the one to complain about.
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "pagedkv.h"

namespace {

using at::ScalarType;
constexpr int kUnfit = -1;

// The tensor of an argument; null for None and for what is no tensor.
const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool dense(const at::Tensor* t, ScalarType type, int device,
           std::initializer_list<int64_t> shape) {
  if (t == nullptr || t->scalar_type() != type || !t->is_cuda() || t->get_device() != device ||
      t->dim() != (int64_t)shape.size() || !t->is_contiguous())
    return false;
  int64_t i = 0;
  for (const int64_t n : shape)
    if (t->size(i++) != n) return false;
  return true;
}

// [T, heads, D] with a token's heads contiguous, and the distance between tokens
// in elements (any for a single token).
bool rows(const at::Tensor* t, ScalarType type, int device, int64_t T, int64_t heads, int64_t D) {
  return t != nullptr && t->scalar_type() == type && t->is_cuda() && t->get_device() == device &&
         t->dim() == 3 && t->size(0) == T && t->size(1) == heads && t->size(2) == D &&
         t->stride(2) == 1 && (t->stride(1) == D || heads == 1);
}
int64_t stride(const at::Tensor* t) {
  return t->size(0) > 1 ? t->stride(0) : t->size(1) * t->size(2);
}

// None, or one int32 on the device.
bool status_fits(PyObject* o, int device) {
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  return t != nullptr && t->scalar_type() == ScalarType::Int && t->is_cuda() &&
         t->get_device() == device && t->numel() >= 1;
}

template <typename P>
P* data(const at::Tensor* t) {
  return t == nullptr ? nullptr : static_cast<P*>(t->data_ptr());
}
int32_t* status_of(PyObject* o) { return o == Py_None ? nullptr : data<int32_t>(tensor(o)); }

bool half_type(const at::Tensor* q, pa_dtype* type) {
  if (q->scalar_type() == ScalarType::Half)
    *type = PA_F16;
  else if (q->scalar_type() == ScalarType::BFloat16)
    *type = PA_BF16;
  else
    return false;
  return true;
}

// Numbers: a Python error where they are none (or do not fit).
bool number(PyObject* o, int* x) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return false;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
    return false;
  }
  *x = (int)v;
  return true;
}
bool number(PyObject* o, float* x) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) return false;
  *x = (float)v;
  return true;
}

// The stream handle of an argument (an int), or the device's current stream.
bool stream_of(PyObject* o, int device, pa_stream_t* s) {
  if (o == Py_None) {
    *s = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    return true;
  }
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) return false;
  *s = static_cast<pa_stream_t>(p);
  return true;
}

// A C++ exception must not leave through the interpreter.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd given", want, n);
    return nullptr;
  }
  try {
    const int rc = f();
    return PyErr_Occurred() ? nullptr : PyLong_FromLong(rc);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// cached_lens, new_lens, block_tables, free_blocks, free_state, context_lens,
// q_offsets, slot_mapping, positions, free_state_out, status, block_size,
// max_tokens, stream
PyObject* step_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> int {
    const at::Tensor *c = tensor(a[0]), *nw = tensor(a[1]), *bt = tensor(a[2]),
                     *ring = tensor(a[3]), *st = tensor(a[4]), *ctx = tensor(a[5]), *off = tensor(a[6]),
                     *slot = tensor(a[7]), *pos = tensor(a[8]), *so = tensor(a[9]);
    int bs, T;
    pa_stream_t s;
    if (!number(a[11], &bs) || !number(a[12], &T)) return kUnfit;
    if (c == nullptr || !c->is_cuda() || c->dim() != 1 || bt == nullptr || bt->dim() != 2 ||
        ring == nullptr || ring->dim() != 1)
      return kUnfit;
    const int dev = c->get_device();
    const int64_t B = c->size(0), M = bt->size(1), NB = ring->size(0);
    if (B > INT32_MAX || M > INT32_MAX || NB > INT32_MAX ||
        !dense(c, ScalarType::Int, dev, {B}) || !dense(nw, ScalarType::Int, dev, {B}) ||
        !dense(bt, ScalarType::Int, dev, {B, M}) || !dense(ring, ScalarType::Int, dev, {NB}) ||
        !dense(st, ScalarType::Long, dev, {2}) || !dense(ctx, ScalarType::Int, dev, {B}) ||
        !dense(off, ScalarType::Int, dev, {B + 1}) ||
        !dense(slot, ScalarType::Long, dev, {T}) || !dense(pos, ScalarType::Int, dev, {T}) ||
        !dense(so, ScalarType::Long, dev, {2}) || !status_fits(a[10], dev) ||
        !stream_of(a[13], dev, &s))
      return kUnfit;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    return pa_step_plan(data<int32_t>(c), data<int32_t>(nw), (int)B, bs, (int)NB, (int)M, T,
                        data<int32_t>(ring), data<int64_t>(st), data<int32_t>(bt),
                        data<int32_t>(ctx), data<int32_t>(off), data<int64_t>(slot),
                        data<int32_t>(pos), data<int64_t>(so), status_of(a[10]), s);
  });
}

// q, k, v, positions, table, slot_mapping, k_cache, v_cache, q_out, k_out, status,
// interleaved, stream; v, slot_mapping and the caches None for rotation only
PyObject* rope_cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> int {
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *pos = tensor(a[3]),
                     *tab = tensor(a[4]), *slot = tensor(a[5]), *kc = tensor(a[6]),
                     *vc = tensor(a[7]), *qo = tensor(a[8]), *ko = tensor(a[9]);
    const int il = PyObject_IsTrue(a[11]);
    pa_dtype type;
    pa_stream_t s;
    if (il < 0 || q == nullptr || !q->is_cuda() || q->dim() != 3 || k == nullptr ||
        k->dim() != 3 || pos == nullptr || tab == nullptr || tab->dim() != 1 ||
        !half_type(q, &type))
      return kUnfit;
    const int dev = q->get_device();
    const ScalarType t = q->scalar_type();
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2), Hkv = k->size(1);
    const int64_t axes = pos->dim() == 2 ? pos->size(0) : 1;
    int64_t NB = 0, bs = 0;
    if (T > INT32_MAX || H > INT32_MAX || Hkv > INT32_MAX || D > INT32_MAX ||
        axes > INT32_MAX || tab->size(0) > INT32_MAX / 2)
      return kUnfit;
    const bool cache = a[6] != Py_None || a[7] != Py_None;
    if (cache) {
      if (kc == nullptr || kc->dim() != 4) return kUnfit;
      NB = kc->size(0);
      bs = kc->size(1);
      if (NB > INT32_MAX || bs > INT32_MAX || !dense(kc, t, dev, {NB, bs, Hkv, D}) ||
          !dense(vc, t, dev, {NB, bs, Hkv, D}) || !rows(v, t, dev, T, Hkv, D) ||
          !dense(slot, ScalarType::Long, dev, {T}))
        return kUnfit;
    }
    if (!rows(q, t, dev, T, H, D) || !rows(k, t, dev, T, Hkv, D) ||
        !(pos->dim() == 1 ? dense(pos, ScalarType::Int, dev, {T})
                          : dense(pos, ScalarType::Int, dev, {axes, T})) ||
        !dense(tab, ScalarType::Long, dev, {tab->size(0)}) || !rows(qo, t, dev, T, H, D) ||
        (a[9] != Py_None && !rows(ko, t, dev, T, Hkv, D)) || !status_fits(a[10], dev) ||
        !stream_of(a[12], dev, &s))
      return kUnfit;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    return pa_rope_cache_write(
        data<void>(q), data<void>(k), cache ? data<void>(v) : nullptr, data<int32_t>(pos),
        reinterpret_cast<const uint64_t*>(data<int64_t>(tab)),
        cache ? data<int64_t>(slot) : nullptr, (int)T, (int)H, (int)Hkv, (int)D,
        2 * (int)tab->size(0), (int)axes, il, type, stride(q), stride(k),
        cache ? stride(v) : 0, (int)bs, (int)NB, data<void>(qo), stride(qo),
        ko ? data<void>(ko) : nullptr, ko ? stride(ko) : 0, cache ? data<void>(kc) : nullptr,
        cache ? data<void>(vc) : nullptr, status_of(a[10]), s);
  });
}

// q, k, v, q_offsets, out, status, scale, stream
PyObject* prompt_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> int {
    const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *off = tensor(a[3]),
                     *out = tensor(a[4]);
    float scale;
    pa_dtype type;
    pa_stream_t s;
    if (!number(a[6], &scale)) return kUnfit;
    if (q == nullptr || !q->is_cuda() || q->dim() != 3 || k == nullptr || k->dim() != 3 ||
        off == nullptr || off->dim() != 1 || !half_type(q, &type))
      return kUnfit;
    const int dev = q->get_device();
    const ScalarType t = q->scalar_type();
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2), Hkv = k->size(1),
                  B = off->size(0) - 1;
    if (T > INT32_MAX || H > INT32_MAX || Hkv > INT32_MAX || D > INT32_MAX || B > INT32_MAX ||
        !rows(q, t, dev, T, H, D) || !rows(k, t, dev, T, Hkv, D) ||
        !rows(v, t, dev, T, Hkv, D) || !dense(off, ScalarType::Int, dev, {B + 1}) ||
        !dense(out, t, dev, {T, H, D}) || !status_fits(a[5], dev) || !stream_of(a[7], dev, &s))
      return kUnfit;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    return pa_prompt_attention(data<void>(q), data<void>(k), data<void>(v), data<int32_t>(off),
                               (int)B, (int)T, (int)H, (int)Hkv, (int)D, type, stride(q),
                               stride(k), stride(v), scale, data<void>(out), status_of(a[5]), s);
  });
}

// The paged cache of an attention call.
struct Cache {
  const at::Tensor *k, *v, *bt, *ctx;
  int64_t NB, bs, Hkv, M;
  bool fits(PyObject* const* a, ScalarType t, int dev, int64_t B, int64_t D) {
    k = tensor(a[0]);
    v = tensor(a[1]);
    bt = tensor(a[2]);
    ctx = tensor(a[3]);
    if (k == nullptr || k->dim() != 4 || bt == nullptr || bt->dim() != 2) return false;
    NB = k->size(0);
    bs = k->size(1);
    Hkv = k->size(2);
    M = bt->size(1);
    return NB <= INT32_MAX && bs <= INT32_MAX && Hkv <= INT32_MAX && M <= INT32_MAX &&
           dense(k, t, dev, {NB, bs, Hkv, D}) && dense(v, t, dev, {NB, bs, Hkv, D}) &&
           dense(bt, ScalarType::Int, dev, {B, M}) && dense(ctx, ScalarType::Int, dev, {B});
  }
};

// A workspace argument: a tensor, or None.
bool workspace_fits(PyObject* o, int device, void** p, size_t* bytes) {
  *p = nullptr;
  *bytes = 0;
  if (o == Py_None || o == Py_True) return true;
  const at::Tensor* t = tensor(o);
  if (t == nullptr || !t->is_cuda() || t->get_device() != device || !t->is_contiguous())
    return false;
  *p = t->data_ptr();
  *bytes = t->nbytes();
  return true;
}

// A workspace for one call, from the pool of the stream that the call runs on: one
// of another stream's pool could still be in use there, or be handed out again
// before the call is done.
at::Tensor workspace_for(size_t bytes, int device, PyObject* given, pa_stream_t s) {
  const at::TensorOptions options =
      at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)device);
  if (given == Py_None) return at::empty({(int64_t)bytes}, options);
  const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(
      static_cast<cudaStream_t>(s), (c10::DeviceIndex)device));
  return at::empty({(int64_t)bytes}, options);
}

// q, k_cache, v_cache, block_tables, context_lens, q_offsets, out, workspace (True:
// one is allocated for the call), status, max_context_len, scale, stream
PyObject* chunk_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    const at::Tensor *q = tensor(a[0]), *off = tensor(a[5]), *out = tensor(a[6]);
    int cap;
    float scale;
    pa_dtype type;
    pa_stream_t s;
    Cache c;
    void* ws;
    size_t ws_bytes;
    if (!number(a[9], &cap) || !number(a[10], &scale)) return kUnfit;
    if (q == nullptr || !q->is_cuda() || q->dim() != 3 || off == nullptr || off->dim() != 1 ||
        !half_type(q, &type))
      return kUnfit;
    const int dev = q->get_device();
    const ScalarType t = q->scalar_type();
    const int64_t T = q->size(0), H = q->size(1), D = q->size(2), B = off->size(0) - 1;
    if (T > INT32_MAX || H > INT32_MAX || D > INT32_MAX || B > INT32_MAX ||
        !rows(q, t, dev, T, H, D) || !c.fits(a + 1, t, dev, B, D) ||
        !dense(off, ScalarType::Int, dev, {B + 1}) || !dense(out, t, dev, {T, H, D}) ||
        !workspace_fits(a[7], dev, &ws, &ws_bytes) || !status_fits(a[8], dev) ||
        !stream_of(a[11], dev, &s))
      return kUnfit;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    at::Tensor own;
    if (a[7] == Py_True) {
      ws_bytes = pa_chunk_attention_workspace_size((int)B, (int)T, (int)H, (int)c.Hkv, (int)D, cap);
      if (ws_bytes > 0) {
        own = workspace_for(ws_bytes, dev, a[11], s);
        ws = own.data_ptr();
      }
    }
    return pa_chunk_attention(data<void>(q), data<void>(c.k), data<void>(c.v),
                              data<int32_t>(c.bt), data<int32_t>(c.ctx), data<int32_t>(off),
                              (int)B, (int)T, (int)H, (int)c.Hkv, (int)D, type, stride(q),
                              (int)c.bs, (int)c.NB, (int)c.M, cap, scale, data<void>(out), ws,
                              ws_bytes, status_of(a[8]), s);
  });
}

// q, k_cache, v_cache, block_tables, context_lens, out, workspace (None: one is
// allocated where the call needs it), status, max_context_len, partition_tokens,
// scale, stream
PyObject* decode_grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    const at::Tensor *q = tensor(a[0]), *out = tensor(a[5]);
    int cap, pt;
    float scale;
    pa_dtype type;
    pa_stream_t s;
    Cache c;
    void* ws;
    size_t ws_bytes;
    if (!number(a[8], &cap) || !number(a[9], &pt) || !number(a[10], &scale)) return kUnfit;
    if (q == nullptr || !q->is_cuda() || q->dim() != 3 || !half_type(q, &type)) return kUnfit;
    const int dev = q->get_device();
    const ScalarType t = q->scalar_type();
    const int64_t B = q->size(0), H = q->size(1), D = q->size(2);
    if (a[6] == Py_True || B > INT32_MAX || H > INT32_MAX || D > INT32_MAX ||
        !dense(q, t, dev, {B, H, D}) ||
        !c.fits(a + 1, t, dev, B, D) || !dense(out, t, dev, {B, H, D}) ||
        !workspace_fits(a[6], dev, &ws, &ws_bytes) || !status_fits(a[7], dev) ||
        !stream_of(a[11], dev, &s))
      return kUnfit;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    auto call = [&]() {
      return pa_decode_grouped(data<void>(q), data<void>(c.k), data<void>(c.v),
                               data<int32_t>(c.bt), data<int32_t>(c.ctx), (int)B, (int)H,
                               (int)c.Hkv, (int)D, type, (int)c.bs, (int)c.NB, (int)c.M, cap, pt,
                               scale, data<void>(out), ws, ws_bytes, status_of(a[7]), s);
    };
    const int rc = call();
    if (rc != PA_ERR_WORKSPACE || a[6] != Py_None) return rc;
    ws_bytes = pa_decode_grouped_workspace_size((int)B, (int)H, (int)c.Hkv, (int)D, (int)c.bs, cap,
                                                pt);
    const at::Tensor own = workspace_for(ws_bytes, dev, a[11], s);
    ws = own.data_ptr();
    return call();
  });
}

PyMethodDef methods[] = {
    {"step_plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(step_plan)),
     METH_FASTCALL, nullptr},
    {"rope_cache_write",
     reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_cache_write)), METH_FASTCALL,
     nullptr},
    {"prompt_attention",
     reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prompt_attention)), METH_FASTCALL,
     nullptr},
    {"chunk_attention",
     reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(chunk_attention)), METH_FASTCALL,
     nullptr},
    {"decode_grouped",
     reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode_grouped)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_grouped", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__grouped() { return PyModule_Create(&module); }
