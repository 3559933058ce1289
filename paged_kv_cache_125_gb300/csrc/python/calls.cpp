// The Python binding's quick way into the calls that run once per layer or
// step beside kernels of a few microseconds (shared decode, page operators).
//
// Each function takes the arguments of the Python function of the same name,
// all by position.  When every tensor is of the kind that the call takes it
// allocates what the caller left out, makes the C ABI call on the current
// stream of the tensors' device and returns the results; otherwise it returns
// None and has done nothing, and the Python function finds and names the fault.
// In Python alone the checks and the marshalling of such a call took 15 to 20
// us on a Grace core, several times the 3 to 6 us of its launches.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>
#include <initializer_list>

#include "kvpaged.h"

namespace {

PyObject* g_check;  // of the Python binding: raises the error of a return code

// The arguments of one call, checked one after the other; ok turns false at
// the first that is not what the call takes.
struct Args {
  PyObject* const* o;
  int idx = -1;  // CUDA device, that of the first tensor
  bool ok = true;

  const at::Tensor* tensor(int i, at::ScalarType type) {
    if (!ok || !THPVariable_Check(o[i])) return fail();
    const at::Tensor& t = THPVariable_Unpack(o[i]);
    if (!t.defined() || t.scalar_type() != type || !t.is_cuda() || t.layout() != at::kStrided) return fail();
    if (idx < 0) idx = t.device().index();
    if (t.device().index() != idx) return fail();
    return &t;
  }
  // A contiguous tensor of that shape (-1: any size).
  const at::Tensor* dense(int i, at::ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(i, type);
    if (!t || t->dim() != (int64_t)shape.size() || !t->is_contiguous()) return fail();
    int d = 0;
    for (int64_t n : shape) {
      if (n >= 0 && t->size(d) != n) return fail();
      ++d;
    }
    return t;
  }
  // bf16 rows [rows, heads, head_dim], heads and head_dim contiguous.
  const at::Tensor* rows(int i, int64_t n, int64_t heads, int64_t d) {
    const at::Tensor* t = tensor(i, at::kBFloat16);
    if (!t || t->dim() != 3 || t->size(0) != n || t->size(1) != heads || t->size(2) != d ||
        t->stride(2) != 1 || t->stride(1) != d)
      return fail();
    return t;
  }
  // A scratch buffer, or null where the caller gave none.
  const at::Tensor* scratch(int i) {
    if (o[i] == Py_None) return nullptr;
    const at::Tensor* t = tensor(i, at::kByte);
    if (!t || !t->is_contiguous()) return fail();
    return t;
  }
  int64_t integer(int i, int64_t lo, int64_t hi) {
    if (!ok) return 0;
    if (!PyLong_CheckExact(o[i])) {
      ok = false;
      return 0;
    }
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o[i], &overflow);
    if (overflow || v < lo || v > hi) ok = false;
    return v;
  }
  int small(int i) { return (int)integer(i, INT_MIN, INT_MAX); }
  std::nullptr_t fail() {
    ok = false;
    return nullptr;
  }
};

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int idx) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)idx)));
}

bool fits_int(int64_t n) { return n <= INT_MAX; }

kvp_stream_t stream_of(int idx) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)idx).stream(); }

template <typename T>
T* at_(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
int32_t* ints(const at::Tensor& t) { return at_<int32_t>(t); }
kvp_bf16* halves(const at::Tensor& t) { return at_<kvp_bf16>(t); }

// Makes a call of the library without the interpreter lock, which a full launch
// queue would hold up.
template <typename F>
int unlocked(F call) {
  PyThreadState* state = PyEval_SaveThread();
  const int rc = call();
  PyEval_RestoreThread(state);
  return rc;
}

// Raises the error of rc.
PyObject* failed(int rc) {
  PyObject* r = PyObject_CallFunction(g_check, "i", rc);
  if (r) {
    Py_DECREF(r);
    PyErr_SetString(PyExc_RuntimeError, "call failed");
  }
  return nullptr;
}

PyObject* given(PyObject* o) {
  Py_INCREF(o);
  return o;
}

bool argc(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return n == want;
}

// block_tables, context_lens, block_size, num_heads, num_kv_heads, num_blocks, min_shared_len, plan
PyObject* shared_plan(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!argc(n, 8)) return nullptr;
  Args a{o};
  const at::Tensor* bt = a.dense(0, at::kInt, {-1, -1});
  const at::Tensor* ctx = bt ? a.dense(1, at::kInt, {bt->size(0)}) : nullptr;
  const int bs = a.small(2), hq = a.small(3), hkv = a.small(4);
  const int64_t nb = a.integer(5, LLONG_MIN, LLONG_MAX);
  const int least = a.small(6);
  const at::Tensor* plan = a.scratch(7);
  if (!a.ok || !fits_int(bt->size(0)) || !fits_int(bt->size(1))) Py_RETURN_NONE;
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)a.idx);
  const int b = (int)bt->size(0);
  at::Tensor made;
  if (!plan) {
    const size_t bytes = attn_shared_plan_size(b, hq, hkv);
    if (!bytes) return failed(KVP_ERR_INVALID_ARG);
    made = fresh({(int64_t)bytes}, at::kByte, a.idx);
    plan = &made;
  }
  const int rc = unlocked([&] {
    return attn_shared_plan(ints(*bt), (int)bt->size(1), ints(*ctx), b, nb, bs, hq, hkv, least,
                            plan->data_ptr(), (size_t)plan->numel(), stream_of(a.idx));
  });
  if (rc) return failed(rc);
  return made.defined() ? THPVariable_Wrap(made) : given(o[7]);
  END_HANDLE_TH_ERRORS
}

// q, k, v, slot_mapping (the three None: no append), k_cache, v_cache,
// block_tables, plan, softmax_scale, workspace, out
PyObject* decode_shared(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!argc(n, 11)) return nullptr;
  Args a{o};
  const bool append = o[1] != Py_None;
  const at::Tensor* kc = a.dense(4, at::kBFloat16, {-1, -1, -1, -1});
  if (!kc) Py_RETURN_NONE;
  const int64_t nb = kc->size(0), bs = kc->size(1), hkv = kc->size(2), d = kc->size(3);
  const at::Tensor* vc = a.dense(5, at::kBFloat16, {nb, bs, hkv, d});
  const at::Tensor* q = a.tensor(0, at::kBFloat16);
  if (!q || q->dim() != 3) Py_RETURN_NONE;
  const int64_t b = q->size(0), hq = q->size(1);
  a.rows(0, b, hq, d);
  const at::Tensor* bt = a.dense(6, at::kInt, {b, -1});
  const at::Tensor *k = nullptr, *v = nullptr, *slots = nullptr;
  if (append) {
    k = a.rows(1, b, hkv, d);
    v = a.rows(2, b, hkv, d);
    slots = a.dense(3, at::kInt, {b});
  }
  const at::Tensor* plan = a.scratch(7);
  const at::Tensor* ws = a.scratch(9);
  const at::Tensor* out = o[10] == Py_None ? nullptr : a.rows(10, b, hq, d);
  if (!a.ok || !plan || !fits_int(b) || !fits_int(hq) || !fits_int(hkv) || !fits_int(bs) || !fits_int(d) ||
      !fits_int(bt->size(1)))
    Py_RETURN_NONE;
  double scale = 0;
  if (o[8] == Py_None) {
    scale = 1.0 / std::sqrt((double)d);
  } else if (PyFloat_Check(o[8])) {
    scale = PyFloat_AS_DOUBLE(o[8]);
  } else {
    Py_RETURN_NONE;
  }
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)a.idx);
  at::Tensor made_ws, made;
  if (!ws) {
    const size_t bytes = attn_decode_shared_workspace_size((int)b, (int)hq, (int)hkv, (int)d);
    if (!bytes) return failed(KVP_ERR_INVALID_ARG);
    made_ws = fresh({(int64_t)bytes}, at::kByte, a.idx);
    ws = &made_ws;
  }
  if (!out) {
    made = fresh({b, hq, d}, at::kBFloat16, a.idx);
    out = &made;
  }
  const kvp_stream_t st = stream_of(a.idx);
  const int rc = unlocked([&] {
    if (append)
      return attn_decode_shared_append(halves(*q), q->stride(0), halves(*k), halves(*v), k->stride(0),
                                       v->stride(0), ints(*slots), halves(*kc), halves(*vc), nb, (int)bs,
                                       ints(*bt), (int)bt->size(1), plan->data_ptr(), (size_t)plan->numel(),
                                       (int)b, (int)hq, (int)hkv, (int)d, (float)scale, ws->data_ptr(),
                                       (size_t)ws->numel(), halves(*out), out->stride(0), st);
    return attn_decode_shared(halves(*q), q->stride(0), halves(*kc), halves(*vc), nb, (int)bs, ints(*bt),
                              (int)bt->size(1), plan->data_ptr(), (size_t)plan->numel(), (int)b, (int)hq,
                              (int)hkv, (int)d, (float)scale, ws->data_ptr(), (size_t)ws->numel(), halves(*out),
                              out->stride(0), st);
  });
  if (rc) return failed(rc);
  return made.defined() ? THPVariable_Wrap(made) : given(o[10]);
  END_HANDLE_TH_ERRORS
}

// The page operators' pool: [..., num_blocks, block_size, heads, head_dim].
struct Pool {
  kvp_bf16* base = nullptr;
  int64_t planes = 0, stride = 0, blocks = 0, row = 0;
  int block_size = 0;
};
Pool pool_of(Args& a, int i) {
  Pool p;
  const at::Tensor* t = a.tensor(i, at::kBFloat16);
  if (!t || t->dim() < 4 || !t->is_contiguous() || t->numel() == 0 || !fits_int(t->size(-3))) {
    a.fail();
    return p;
  }
  p.base = halves(*t);
  p.blocks = t->size(-4);
  p.block_size = (int)t->size(-3);
  p.row = t->size(-2) * t->size(-1);
  p.stride = p.blocks * p.block_size * p.row;
  p.planes = t->numel() / p.stride;
  return p;
}

// N int32 outputs: the caller's (a tuple or list of them) or new ones.
template <int N>
struct Outputs {
  at::Tensor t[N];
  bool theirs = false;  // the caller's

  bool take(Args& a, PyObject* given_out, std::initializer_list<int64_t> (&shapes)[N]) {
    if (given_out == Py_None) return a.ok;
    if (!a.ok || !(PyTuple_CheckExact(given_out) || PyList_CheckExact(given_out)) ||
        PySequence_Fast_GET_SIZE(given_out) != N)
      return a.ok = false;
    PyObject** items = PySequence_Fast_ITEMS(given_out);
    Args b{items, a.idx};
    for (int i = 0; i < N; ++i) {
      const at::Tensor* x = b.dense(i, at::kInt, shapes[i]);
      if (!x) return a.ok = false;
      t[i] = *x;
    }
    return theirs = true;
  }
  void make(std::initializer_list<int64_t> (&shapes)[N], int idx) {
    if (theirs) return;
    for (int i = 0; i < N; ++i) t[i] = fresh(at::IntArrayRef(shapes[i].begin(), shapes[i].size()), at::kInt, idx);
  }
  // (Wrapping a tensor of the caller's gives the caller's own object.)
  PyObject* result() {
    PyObject* r = PyTuple_New(N);
    for (int i = 0; r && i < N; ++i) {
      PyObject* x = THPVariable_Wrap(t[i]);
      if (!x) {
        Py_CLEAR(r);
        break;
      }
      PyTuple_SET_ITEM(r, i, x);
    }
    return r;
  }
};

// The workspace of a page operator: the caller's, or a new one in `made`.
const at::Tensor* pages_workspace(const at::Tensor* theirs, at::Tensor* made, int64_t blocks, int64_t rows,
                                  int idx) {
  if (theirs) return theirs;
  const size_t bytes = kv_pages_workspace_size(blocks, (int)rows);
  if (!bytes) return nullptr;
  *made = fresh({(int64_t)bytes}, at::kByte, idx);
  return made;
}

// kv_cache, block_tables, context_lens, ref_counts, parents, workspace, out
PyObject* pages_fork(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!argc(n, 7)) return nullptr;
  Args a{o};
  const Pool p = pool_of(a, 0);
  const at::Tensor* bt = a.dense(1, at::kInt, {-1, -1});
  if (!a.ok || !fits_int(bt->size(0)) || !fits_int(bt->size(1))) Py_RETURN_NONE;
  const int64_t rows = bt->size(0), mb = bt->size(1);
  const at::Tensor* ctx = a.dense(2, at::kInt, {rows});
  const at::Tensor* counts = a.dense(3, at::kInt, {p.blocks});
  const at::Tensor* parents = a.dense(4, at::kInt, {-1});
  const at::Tensor* ws = a.scratch(5);
  if (!a.ok || !fits_int(parents->size(0))) Py_RETURN_NONE;
  const int64_t m = parents->size(0);
  std::initializer_list<int64_t> tables{m, mb}, lens{m}, blocks{p.blocks};
  std::initializer_list<int64_t> shapes[3] = {tables, lens, blocks};
  Outputs<3> out;
  if (!out.take(a, o[6], shapes)) Py_RETURN_NONE;
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)a.idx);
  out.make(shapes, a.idx);
  at::Tensor made;
  ws = pages_workspace(ws, &made, p.blocks, rows > m ? rows : m, a.idx);
  if (!ws) return failed(KVP_ERR_INVALID_ARG);
  const int rc = unlocked([&] {
    return kv_pages_fork(p.base, p.planes, p.stride, p.blocks, p.block_size, p.row, ints(*bt), (int)mb,
                         ints(*ctx), (int)rows, ints(*counts), ints(*parents), (int)m, ints(out.t[0]),
                         ints(out.t[1]), ints(out.t[2]), ws->data_ptr(), (size_t)ws->numel(),
                         stream_of(a.idx));
  });
  return rc ? failed(rc) : out.result();
  END_HANDLE_TH_ERRORS
}

// block_tables, context_lens, ref_counts, new_tokens, block_size, num_slots, workspace, out
PyObject* pages_extend(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!argc(n, 8)) return nullptr;
  Args a{o};
  const at::Tensor* bt = a.dense(0, at::kInt, {-1, -1});
  if (!a.ok || !fits_int(bt->size(0)) || !fits_int(bt->size(1))) Py_RETURN_NONE;
  const int64_t rows = bt->size(0), mb = bt->size(1);
  const at::Tensor* ctx = a.dense(1, at::kInt, {rows});
  const at::Tensor* counts = a.dense(2, at::kInt, {-1});
  const at::Tensor* add = a.dense(3, at::kInt, {rows});
  const int bs = a.small(4);
  const int64_t slots = a.integer(5, 0, INT_MAX);
  const at::Tensor* ws = a.scratch(6);
  if (!a.ok) Py_RETURN_NONE;
  const int64_t nb = counts->size(0);
  std::initializer_list<int64_t> tables{rows, mb}, lens{rows}, blocks{nb}, mapping{slots};
  std::initializer_list<int64_t> shapes[4] = {tables, lens, blocks, mapping};
  Outputs<4> out;
  if (!out.take(a, o[7], shapes)) Py_RETURN_NONE;
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)a.idx);
  out.make(shapes, a.idx);
  at::Tensor made;
  ws = pages_workspace(ws, &made, nb, rows, a.idx);
  if (!ws) return failed(KVP_ERR_INVALID_ARG);
  const int rc = unlocked([&] {
    return kv_pages_extend(ints(*bt), (int)mb, ints(*ctx), (int)rows, ints(*counts), nb, bs, ints(*add),
                           slots, ints(out.t[0]), ints(out.t[1]), ints(out.t[2]), ints(out.t[3]),
                           ws->data_ptr(), (size_t)ws->numel(), stream_of(a.idx));
  });
  return rc ? failed(rc) : out.result();
  END_HANDLE_TH_ERRORS
}

// kv_cache, block_tables, context_lens, ref_counts, workspace, out
PyObject* pages_compact(PyObject*, PyObject* const* o, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!argc(n, 6)) return nullptr;
  Args a{o};
  const Pool p = pool_of(a, 0);
  const at::Tensor* bt = a.dense(1, at::kInt, {-1, -1});
  if (!a.ok || !fits_int(bt->size(0)) || !fits_int(bt->size(1))) Py_RETURN_NONE;
  const int64_t rows = bt->size(0), mb = bt->size(1);
  const at::Tensor* ctx = a.dense(2, at::kInt, {rows});
  const at::Tensor* counts = a.dense(3, at::kInt, {p.blocks});
  const at::Tensor* ws = a.scratch(4);
  std::initializer_list<int64_t> tables{rows, mb}, blocks{p.blocks};
  std::initializer_list<int64_t> shapes[3] = {tables, blocks, blocks};
  Outputs<3> out;
  if (!a.ok || !out.take(a, o[5], shapes)) Py_RETURN_NONE;
  c10::cuda::CUDAGuard guard((c10::DeviceIndex)a.idx);
  out.make(shapes, a.idx);
  at::Tensor made;
  ws = pages_workspace(ws, &made, p.blocks, rows, a.idx);
  if (!ws) return failed(KVP_ERR_INVALID_ARG);
  const int rc = unlocked([&] {
    return kv_pages_compact(p.base, p.planes, p.stride, p.blocks, p.block_size, p.row, ints(*bt), (int)mb,
                            ints(*ctx), (int)rows, ints(*counts), ints(out.t[0]), ints(out.t[1]),
                            ints(out.t[2]), ws->data_ptr(), (size_t)ws->numel(), stream_of(a.idx));
  });
  return rc ? failed(rc) : out.result();
  END_HANDLE_TH_ERRORS
}

PyObject* set_check(PyObject*, PyObject* check) {
  Py_INCREF(check);
  Py_XSETREF(g_check, check);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef kMethods[] = {
    {"attn_shared_plan", fast(shared_plan), METH_FASTCALL, nullptr},
    {"attn_decode_shared", fast(decode_shared), METH_FASTCALL, nullptr},
    {"kv_pages_fork", fast(pages_fork), METH_FASTCALL, nullptr},
    {"kv_pages_extend", fast(pages_extend), METH_FASTCALL, nullptr},
    {"kv_pages_compact", fast(pages_compact), METH_FASTCALL, nullptr},
    {"set_check", set_check, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_kvpaged_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvpaged_calls() { return PyModule_Create(&kModule); }
