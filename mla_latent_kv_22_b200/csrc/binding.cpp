// The quick path of the Python binding for calls whose kernels are shorter than their argument
// checks: one C function per call that tests what the Python code in __init__.py tests, takes
// the workspace from torch's allocator and calls the C ABI.  Anything out of the ordinary (a
// wrong argument, another device, a non-contiguous tensor) is handed back as NotImplemented to
// the Python code, which accepts it or says what is wrong.
//
// The library is entered without the interpreter's lock, as ctypes does: it may wait for another
// thread that holds the library's.
//
// Host time per call, Python code / this (us): append 11.3 / 2.9, window decode 15.8 / 8.4
// (6.2 of it two launches and three tensor maps; 5.9 a short one, of one launch), value
// absorption 6.4 / 3.5.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/Allocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "mla.h"

namespace {

constexpr int64_t kLatent = MLA_D_LATENT, kRope = MLA_D_ROPE, kRow = MLA_D_QK, kPage = MLA_PAGE_TOKENS, kV = 128;

PyObject* not_mine() { Py_RETURN_NOTIMPLEMENTED; }

// The checks of one call; `ok` stays true while every argument fits.
struct Args {
  bool ok = true;
  c10::DeviceIndex dev = -1;  // the current device, once there is a CUDA tensor

  // The tensor behind an argument, of the type and on the current device.
  const at::Tensor* tensor(PyObject* o, at::ScalarType type) {
    if (!ok || !THPVariable_Check(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || !t.is_cuda() || t.layout() != at::kStrided) return fail();
    if (dev < 0) dev = c10::cuda::current_device();
    if (t.get_device() != dev) return fail();
    return &t;
  }
  // The address of a contiguous tensor of that shape.
  void* dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(o, type);
    if (!t || !t->is_contiguous() || !is(t->sizes(), shape)) return fail();
    return t->data_ptr();
  }
  // The address of a tensor of that shape whose last dimension is dense.
  void* rows(PyObject* o, std::initializer_list<int64_t> shape, at::IntArrayRef* strides) {
    const at::Tensor* t = tensor(o, at::kBFloat16);
    if (!t || !is(t->sizes(), shape) || t->strides().back() != 1) return fail();
    *strides = t->strides();
    return t->data_ptr();
  }
  long integer(PyObject* o) {
    int over = 0;
    const long v = PyLong_CheckExact(o) ? PyLong_AsLongAndOverflow(o, &over) : (ok = false, 0);
    if (over || v > INT32_MAX || v < INT32_MIN) ok = false;
    return v;
  }
  double real(PyObject* o) {
    if (!PyFloat_CheckExact(o)) {
      ok = false;
      return 0;
    }
    return PyFloat_AS_DOUBLE(o);
  }
  static bool is(at::IntArrayRef a, std::initializer_list<int64_t> b) { return a.equals(at::IntArrayRef(b)); }
  std::nullptr_t fail() {
    ok = false;
    return nullptr;
  }
  mla_stream_t stream() const { return reinterpret_cast<mla_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream()); }
};

// A paged or contiguous cache of B sequences.
struct Cache {
  void* kv = nullptr;
  const int32_t* table = nullptr;
  int num_pages = 0, max_blocks = 0;
  Cache(Args& a, PyObject* kv_cache, PyObject* block_table, int64_t B) {
    const at::Tensor* k = a.tensor(kv_cache, at::kBFloat16);
    if (!k || k->dim() != 3 || k->size(2) != kRow || !k->is_contiguous()) {
      a.fail();
      return;
    }
    kv = k->data_ptr();
    int64_t pages = 0, blocks = 0;
    if (block_table == Py_None) {
      if (k->size(0) != B || k->size(1) % kPage) a.fail();
      blocks = k->size(1) / kPage;
    } else {
      const at::Tensor* t = a.tensor(block_table, at::kInt);
      if (!t || t->dim() != 2 || t->size(0) != B || !t->is_contiguous() || k->size(1) != kPage) {
        a.fail();
        return;
      }
      table = static_cast<const int32_t*>(t->data_ptr());
      pages = k->size(0);
      blocks = t->size(1);
    }
    if (pages > INT32_MAX || blocks > INT32_MAX) a.fail();
    num_pages = (int)pages;
    max_blocks = (int)blocks;
  }
};

// The status of a call into the library, made without the interpreter's lock; its arguments are
// plain values by then.
template <typename Call>
PyObject* status(const Call& call) {
  mla_status_t s;
  Py_BEGIN_ALLOW_THREADS
  s = call();
  Py_END_ALLOW_THREADS
  if (s == MLA_OK) Py_RETURN_NONE;
  return PyLong_FromLong(s);
}

// q [B, H, 576] or [B, s_q, H, 576] with out and lse of the same rows, and the lengths.
struct Query {
  int64_t B = 0, SQ = 1, H = 0;
  void *q = nullptr, *out = nullptr;
  float* lse = nullptr;
  int32_t* lens = nullptr;
  Query(Args& a, PyObject* q_, PyObject* lens_, PyObject* out_, PyObject* lse_) {
    const at::Tensor* t = a.tensor(q_, at::kBFloat16);
    if (!t || t->dim() < 3 || t->dim() > 4) {
      a.fail();
      return;
    }
    B = t->size(0);
    H = t->size(t->dim() - 2);
    if (t->dim() == 4) {
      SQ = t->size(1);
      q = a.dense(q_, at::kBFloat16, {B, SQ, H, kRow});
      out = a.dense(out_, at::kBFloat16, {B, SQ, H, kLatent});
      lse = static_cast<float*>(a.dense(lse_, at::kFloat, {B, SQ, H}));
    } else {
      q = a.dense(q_, at::kBFloat16, {B, H, kRow});
      out = a.dense(out_, at::kBFloat16, {B, H, kLatent});
      lse = static_cast<float*>(a.dense(lse_, at::kFloat, {B, H}));
    }
    lens = static_cast<int32_t*>(a.dense(lens_, at::kInt, {B}));
    if (B > INT32_MAX || SQ > INT32_MAX || H > INT32_MAX) a.fail();
  }
};

// Scratch from torch's allocator, on the current stream: reused only after this call there.
at::DataPtr scratch(size_t bytes) { return c10::GetAllocator(c10::DeviceType::CUDA)->allocate(bytes); }

// (q, kv_cache, block_table, cache_seqlens, out, lse, softmax_scale, window, sinks)
PyObject* decode_window(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) return not_mine();
  Args a;
  const Query x(a, p[0], p[3], p[4], p[5]);
  const Cache c(a, p[1], p[2], x.B);
  const double scale = a.real(p[6]);
  const long window = a.integer(p[7]), sinks = a.integer(p[8]);
  if (!a.ok) return not_mine();
  const size_t bytes = mla_decode_window_workspace_size((int)x.B, (int)x.SQ, (int)x.H);
  const at::DataPtr ws = scratch(bytes);
  const mla_stream_t stream = a.stream();
  return status([&] {
    return mla_decode_window(x.q, c.kv, c.table, x.lens, x.out, x.lse, (int)x.B, (int)x.SQ, (int)x.H, c.num_pages, c.max_blocks,
                             (int)window, (int)sinks, (float)scale, ws.get(), bytes, stream);
  });
  END_HANDLE_TH_ERRORS
}

// (q, kv_cache, prefix_table, prefix_len, block_table, cache_seqlens, out, lse, softmax_scale)
PyObject* decode_shared(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) return not_mine();
  Args a;
  const Query x(a, p[0], p[5], p[6], p[7]);
  if (p[4] == Py_None) return not_mine();
  const Cache c(a, p[1], p[4], x.B);
  const at::Tensor* pt = a.tensor(p[2], at::kInt);
  const int32_t* plen = static_cast<const int32_t*>(a.dense(p[3], at::kInt, {1}));
  const double scale = a.real(p[8]);
  if (!a.ok || pt->dim() != 1 || !pt->is_contiguous() || pt->size(0) > INT32_MAX) return not_mine();
  const size_t bytes = mla_decode_shared_workspace_size((int)x.B, (int)x.SQ, (int)x.H);
  const at::DataPtr ws = scratch(bytes);
  const int32_t* const prefix = static_cast<const int32_t*>(pt->data_ptr());
  const int prefix_blocks = (int)pt->size(0);
  const mla_stream_t stream = a.stream();
  return status([&] {
    return mla_decode_shared(x.q, c.kv, prefix, plen, c.table, x.lens, x.out, x.lse, (int)x.B, (int)x.SQ, (int)x.H, c.num_pages,
                             prefix_blocks, c.max_blocks, (float)scale, ws.get(), bytes, stream);
  });
  END_HANDLE_TH_ERRORS
}

// (c_kv, k_rope, kv_cache, block_table, cache_seqlens, cos_sin, cu_tokens, q_rope, q_out, pos_offset, interleaved)
PyObject* append(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11) return not_mine();
  Args a;
  const at::Tensor *t = a.tensor(p[0], at::kBFloat16), *l = a.tensor(p[4], at::kInt), *cs = a.tensor(p[5], at::kFloat);
  if (!a.ok || t->dim() != 2 || l->dim() != 1 || cs->dim() != 2 || cs->size(1) != kRope || !cs->is_contiguous() || !l->is_contiguous())
    return not_mine();
  const int64_t N = t->size(0), B = l->size(0);
  at::IntArrayRef sc, sk, sq, so;
  void *c_kv = a.rows(p[0], {N, kLatent}, &sc), *k_rope = a.rows(p[1], {N, kRope}, &sk);
  const int32_t* cu = p[6] == Py_None ? nullptr : static_cast<int32_t*>(a.dense(p[6], at::kInt, {B + 1}));
  const int32_t* off = p[9] == Py_None ? nullptr : static_cast<int32_t*>(a.dense(p[9], at::kInt, {B}));
  int64_t H = 0;
  void *q = nullptr, *qo = nullptr;
  const int64_t none[3] = {0, 0, 0};
  sq = so = at::IntArrayRef(none, 3);
  if ((p[7] == Py_None) != (p[8] == Py_None)) return not_mine();
  if (p[7] != Py_None) {
    const at::Tensor* qt = a.tensor(p[7], at::kBFloat16);
    if (!qt || qt->dim() != 3) return not_mine();
    H = qt->size(1);
    q = a.rows(p[7], {N, H, kRope}, &sq);
    qo = a.rows(p[8], {N, H, kRope}, &so);
  }
  const Cache c(a, p[2], p[3], B);
  if (!a.ok || N > INT32_MAX || B > INT32_MAX || H > INT32_MAX || cs->size(0) > INT32_MAX || (p[10] != Py_True && p[10] != Py_False))
    return not_mine();
  const float* const cos_sin = static_cast<const float*>(cs->data_ptr());
  const int32_t* const lens = static_cast<const int32_t*>(l->data_ptr());
  const int64_t st[6] = {sc[0], sk[0], sq[0], sq[1], so[0], so[1]};
  const int max_pos = (int)cs->size(0), interleaved = p[10] == Py_True;
  const mla_stream_t stream = a.stream();
  return status([&] {
    return mla_append(c_kv, k_rope, q, qo, cos_sin, cu, lens, off, c.table, c.kv, st[0], st[1], st[2], st[3], st[4], st[5], (int)N,
                      (int)B, (int)H, c.num_pages, c.max_blocks, max_pos, interleaved, stream);
  });
  END_HANDLE_TH_ERRORS
}

// (out_latent, w_uv, out) with a bf16 latent
PyObject* absorb_o(PyObject*, PyObject* const* p, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3) return not_mine();
  Args a;
  const at::Tensor* t = a.tensor(p[0], at::kBFloat16);
  if (!t || t->dim() != 3) return not_mine();
  const int64_t B = t->size(0), H = t->size(1);
  void *x = a.dense(p[0], at::kBFloat16, {B, H, kLatent}), *w = a.dense(p[1], at::kBFloat16, {H, kLatent, kV});
  float* out = static_cast<float*>(a.dense(p[2], at::kFloat, {B, H, kV}));
  if (!a.ok || B > INT32_MAX || H > INT32_MAX) return not_mine();
  const mla_stream_t stream = a.stream();
  return status([&] { return mla_absorb_o_bf16(x, w, out, (int)B, (int)H, stream); });
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"decode_window", (PyCFunction)(void (*)(void))decode_window, METH_FASTCALL, nullptr},
    {"decode_shared", (PyCFunction)(void (*)(void))decode_shared, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"absorb_o", (PyCFunction)(void (*)(void))absorb_o, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
