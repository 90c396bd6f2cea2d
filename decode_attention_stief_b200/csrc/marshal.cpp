// marshal.cpp -- the short way from Python tensors to the C calls of page planning and
// shared-latent attention (CPython extension `_marshal`).
//
// A decode step makes these calls many times, and checking and converting a dozen tensors in
// Python takes longer than the launch itself (measured for stief_plan_pages: 10.8 us through
// ctypes, 2.4 us of it the launch).  Each function here checks exactly what the Python function
// of the same name checks and, if everything is as it should be, makes the C call and returns
// its status.  If anything is not -- another type, shape, device or memory layout, an argument
// it does not know -- it touches nothing and returns None, and the Python function goes its long
// way, which says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "stief.h"

namespace {

// The library's functions, whose addresses bind() gets from the loaded libstief.so.
decltype(&stief_plan_pages) fn_plan = nullptr;
decltype(&stief_append_shared_paged) fn_append = nullptr;
decltype(&stief_decode_shared_paged) fn_decode = nullptr;
decltype(&stief_expand_shared_paged) fn_expand = nullptr;
decltype(&stief_prefill_attention) fn_prefill = nullptr;

struct NotPlain {};  // some argument is not as it should be: the Python function takes over

constexpr auto kI32 = at::kInt;
constexpr auto kB16 = at::kBFloat16;

struct Call {
  int dev;
  stief_stream_t stream;
  Call() : dev(c10::cuda::current_device()) {
    stream = reinterpret_cast<stief_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
  }
  const at::Tensor& any(PyObject* o) const {
    if (!THPVariable_Check(o)) throw NotPlain{};
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != dev) throw NotPlain{};
    return t;
  }
  const at::Tensor& dense(PyObject* o, at::ScalarType type, int64_t ndim) const {
    const at::Tensor& t = any(o);
    if (t.scalar_type() != type || t.dim() != ndim || !t.is_contiguous()) throw NotPlain{};
    return t;
  }
  uint32_t* status(PyObject* o) const {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = any(o);
    if ((t.scalar_type() != at::kInt && t.scalar_type() != at::kUInt32) || t.numel() < 1) throw NotPlain{};
    return static_cast<uint32_t*>(t.data_ptr());
  }
};

void need(bool ok) {
  if (!ok) throw NotPlain{};
}
int as_int(PyObject* o) {
  need(PyLong_CheckExact(o));
  int over = 0;
  const long v = PyLong_AsLongAndOverflow(o, &over);
  need(over == 0 && v >= INT32_MIN && v <= INT32_MAX);
  return (int)v;
}
int size32(int64_t v) {
  need(v <= INT32_MAX);
  return (int)v;
}
float as_float(PyObject* o) {
  need(PyFloat_CheckExact(o));
  return (float)PyFloat_AS_DOUBLE(o);
}
template <class T>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// Runs `body` (which makes the C call) and turns its outcome into the status or None.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, const void* fn, F body) {
  if (got != want || fn == nullptr) Py_RETURN_NONE;
  try {
    return PyLong_FromLong(body());
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

#define STIEF_CALL(expr)            \
  [&] {                             \
    stief_status st_;               \
    Py_BEGIN_ALLOW_THREADS;         \
    st_ = (expr);                   \
    Py_END_ALLOW_THREADS;           \
    return (long)st_;               \
  }()

PyObject* plan_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, (const void*)fn_plan, [&] {
    const Call c;
    const at::Tensor& fresh = c.dense(a[0], kI32, 1);
    const at::Tensor& lens = c.dense(a[1], kI32, 1);
    const at::Tensor& table = c.dense(a[2], kI32, 2);
    const at::Tensor& free = c.dense(a[3], kI32, 1);
    const at::Tensor& count = c.dense(a[4], kI32, 1);
    const int64_t B = table.size(0);
    int32_t* opt[4] = {nullptr, nullptr, nullptr, nullptr};  // slots, q_start, kv_start, seq_lens_out
    int max_tokens = 0;
    for (int i = 0; i < 4; ++i) {
      if (a[5 + i] == Py_None) continue;
      const at::Tensor& t = c.dense(a[5 + i], kI32, 1);
      if (i == 0) {
        max_tokens = size32(t.size(0));
        need(max_tokens > 0);
      } else {
        need(t.size(0) == (i == 3 ? B : B + 1));
      }
      opt[i] = ptr<int32_t>(t);
    }
    const at::Tensor& left = c.dense(a[9], kI32, 1);
    const at::Tensor& ws = c.any(a[10]);
    need(ws.is_contiguous() && fresh.size(0) == B && lens.size(0) == B && count.size(0) == 1 && left.size(0) == 1);
    const int page_size = as_int(a[11]), pages = size32(free.size(0)), batch = size32(B),
              max_pages = size32(table.size(1));
    uint32_t* status = c.status(a[12]);
    return STIEF_CALL(fn_plan(ptr<int32_t>(fresh), ptr<int32_t>(lens), ptr<int32_t>(table), ptr<int32_t>(free),
                              ptr<int32_t>(count), opt[0], opt[1], opt[2], opt[3], ptr<int32_t>(left),
                              ws.data_ptr(), ws.nbytes(), batch, pages, page_size, max_pages, max_tokens, status,
                              c.stream));
  });
}

// A 2-D bf16 tensor of contiguous rows; its row stride.
const at::Tensor& rows(const Call& c, PyObject* o, int64_t* stride) {
  const at::Tensor& t = c.any(o);
  need(t.scalar_type() == kB16 && t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1));
  *stride = t.size(0) > 1 ? t.stride(0) : t.size(1);
  return t;
}

PyObject* append_shared_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, (const void*)fn_append, [&] {
    const Call c;
    int64_t sc = 0, sp = 0, dr = 0;
    const at::Tensor& lat = rows(c, a[0], &sc);
    const int64_t N = lat.size(0), r = lat.size(1);
    const uint16_t* pe = nullptr;
    if (a[1] != Py_None) {
      const at::Tensor& t = rows(c, a[1], &sp);
      need(t.size(0) == N);
      dr = t.size(1);
      if (dr > 0) pe = ptr<uint16_t>(t);
    }
    const at::Tensor& slots = c.dense(a[2], kI32, 1);
    const at::Tensor& pages = c.dense(a[3], kB16, 3);
    need(slots.size(0) == N && pages.size(2) == r + dr);
    const int n32 = size32(N), np = size32(pages.size(0)), ps = size32(pages.size(1)), r32 = size32(r), dr32 = size32(dr);
    uint32_t* status = c.status(a[4]);
    return STIEF_CALL(fn_append(ptr<uint16_t>(lat), pe, ptr<int32_t>(slots), ptr<uint16_t>(pages), n32, r32, dr32, sc,
                                sp, np, ps, status, c.stream));
  });
}

PyObject* decode_shared_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, (const void*)fn_decode, [&] {
    const Call c;
    const at::Tensor& q = c.dense(a[0], kB16, 3);
    const at::Tensor& pages = c.dense(a[1], kB16, 3);
    const at::Tensor& table = c.dense(a[2], kI32, 2);
    const at::Tensor& lens = c.dense(a[3], kI32, 1);
    const at::Tensor& out = c.dense(a[4], kB16, 3);
    const at::Tensor& ws = c.any(a[5]);
    const int64_t B = q.size(0), H = q.size(1), w = q.size(2), r = out.size(2);
    need(ws.is_contiguous() && pages.size(2) == w && r <= w && out.size(0) == B && out.size(1) == H &&
         table.size(0) == B && lens.size(0) == B);
    const int b32 = size32(B), h32 = size32(H), r32 = size32(r), dr32 = size32(w - r), np = size32(pages.size(0)),
              ps = size32(pages.size(1)), mp = size32(table.size(1)), most = as_int(a[6]);
    const float scale = as_float(a[7]);
    uint32_t* status = c.status(a[8]);
    return STIEF_CALL(fn_decode(ptr<uint16_t>(q), ptr<uint16_t>(pages), ptr<int32_t>(table), ptr<int32_t>(lens),
                                ptr<uint16_t>(out), ws.data_ptr(), ws.nbytes(), b32, h32, r32, dr32, np, ps, mp, most,
                                scale, status, c.stream));
  });
}

PyObject* expand_shared_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, (const void*)fn_expand, [&] {
    const Call c;
    const at::Tensor& pages = c.dense(a[0], kB16, 3);
    const at::Tensor& table = c.dense(a[1], kI32, 2);
    const at::Tensor& start = c.dense(a[2], kI32, 1);
    const at::Tensor& wk = c.dense(a[3], kB16, 3);
    const at::Tensor& wv = c.dense(a[4], kB16, 3);
    const at::Tensor& k = c.dense(a[5], kB16, 3);
    const at::Tensor& v = c.dense(a[6], kB16, 3);
    const int64_t H = wk.size(0), d = wk.size(1), r = wk.size(2), N = k.size(0), B = table.size(0),
                  dr = pages.size(2) - r;
    uint16_t* pe = nullptr;
    need(dr >= 0 && wv.sizes() == wk.sizes() && k.size(1) == H && k.size(2) == d && v.sizes() == k.sizes() &&
         start.size(0) == B + 1);
    if (dr > 0) {
      const at::Tensor& t = c.dense(a[7], kB16, 2);
      need(t.size(0) == N && t.size(1) == dr);
      pe = ptr<uint16_t>(t);
    }
    const int b32 = size32(B), n32 = size32(N), h32 = size32(H), d32 = size32(d), r32 = size32(r), dr32 = size32(dr),
              np = size32(pages.size(0)), ps = size32(pages.size(1)), mp = size32(table.size(1));
    uint32_t* status = c.status(a[8]);
    return STIEF_CALL(fn_expand(ptr<uint16_t>(pages), ptr<int32_t>(table), ptr<int32_t>(start), ptr<uint16_t>(wk),
                                ptr<uint16_t>(wv), ptr<uint16_t>(k), ptr<uint16_t>(v), pe, b32, n32, h32, d32, r32,
                                dr32, np, ps, mp, status, c.stream));
  });
}

PyObject* prefill_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, (const void*)fn_prefill, [&] {
    const Call c;
    const at::Tensor& q = c.dense(a[0], kB16, 3);
    const at::Tensor& k = c.dense(a[1], kB16, 3);
    const at::Tensor& v = c.dense(a[2], kB16, 3);
    const at::Tensor& qs = c.dense(a[3], kI32, 1);
    const at::Tensor& ks = c.dense(a[4], kI32, 1);
    const at::Tensor& out = c.dense(a[5], kB16, 3);
    const int64_t Nq = q.size(0), Hq = q.size(1), Nkv = k.size(0), Hkv = k.size(1), d = k.size(2), B = qs.size(0) - 1;
    int64_t dr = 0;
    const uint16_t* pe = nullptr;
    if (a[8] != Py_None) {
      const at::Tensor& t = c.dense(a[8], kB16, 2);
      need(t.size(0) == Nkv);
      dr = t.size(1);
      if (dr > 0) pe = ptr<uint16_t>(t);
    }
    need(v.sizes() == k.sizes() && q.size(2) == d + dr && out.size(0) == Nq && out.size(1) == Hq && out.size(2) == d &&
         ks.size(0) == B + 1);
    const int b32 = size32(B), hq = size32(Hq), hk = size32(Hkv), d32 = size32(d), dr32 = size32(dr), nq = size32(Nq),
              nk = size32(Nkv), most = as_int(a[6]);
    const float scale = as_float(a[7]);
    uint32_t* status = c.status(a[9]);
    return STIEF_CALL(fn_prefill(ptr<uint16_t>(q), ptr<uint16_t>(k), ptr<uint16_t>(v), pe, ptr<int32_t>(qs),
                                 ptr<int32_t>(ks), ptr<uint16_t>(out), b32, hq, hk, d32, dr32, nq, nk, most, scale,
                                 status, c.stream));
  });
}

// bind(plan, append, decode, expand, prefill): the addresses of the library's functions.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  fn_plan = reinterpret_cast<decltype(fn_plan)>(p[0]);
  fn_append = reinterpret_cast<decltype(fn_append)>(p[1]);
  fn_decode = reinterpret_cast<decltype(fn_decode)>(p[2]);
  fn_expand = reinterpret_cast<decltype(fn_expand)>(p[3]);
  fn_prefill = reinterpret_cast<decltype(fn_prefill)>(p[4]);
  Py_RETURN_NONE;
}

template <class F>
PyCFunction method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", method(bind), METH_FASTCALL, nullptr},
    {"plan_pages", method(plan_pages), METH_FASTCALL, nullptr},
    {"append_shared_paged", method(append_shared_paged), METH_FASTCALL, nullptr},
    {"decode_shared_paged", method(decode_shared_paged), METH_FASTCALL, nullptr},
    {"expand_shared_paged", method(expand_shared_paged), METH_FASTCALL, nullptr},
    {"prefill_attention", method(prefill_attention), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
