// The usual call of rotate, matvec, gemm_glu and block_norms without the interpreter's part: strided tensors of
// the expected types and shapes, all on the current device, on its current stream. Anything else - another
// stream or device, a subclass of Tensor, an argument that is to be refused - returns NotImplemented, and the
// Python function of the same name does the call or names what is wrong, so every refusal is worded in one place.
//
// Why: one token's block_norms runs 3.0 us on the device and rotate 2.9 (captured), but a call through Python's checks and
// ctypes takes 8.7 to 9.0 and 7.6 to 8.2 us. Through here the same calls take 3.9 to 4.5 and 3.8 to 4.5 us (12 processes; in
// some the host launches quicker, 3.2 and 3.1), M=4 K=5120 N=8192 matvec 5.3 against 8.5, M=7 gemm_glu 7.2 against 9.4.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "pq.h"

namespace {

// The library's entry points, as the loaded libpq.so has them, and the Python function that turns a code into an error.
struct Entries {
  decltype(&pq_rotate) rotate;
  decltype(&pq_matvec) matvec;
  decltype(&pq_gemm_glu) gemm_glu;
  decltype(&pq_block_norms) block_norms;
  decltype(&pq_packed_weight_bytes) packed_weight_bytes;
  decltype(&pq_gemm_workspace_bytes) gemm_workspace_bytes;
};
Entries pq{};
PyObject* check = nullptr;

constexpr at::ScalarType kF16 = at::kHalf, kBF16 = at::kBFloat16, kF32 = at::kFloat, kU8 = at::kByte;

// An optional tensor argument; bad: neither None nor a plain strided tensor on a GPU.
struct Arg {
  const at::Tensor* t = nullptr;
  bool bad = false;
  explicit Arg(PyObject* o) {
    if (o == Py_None) return;
    if (!THPVariable_CheckExact(o)) { bad = true; return; }
    t = &THPVariable_Unpack(o);
    bad = t->layout() != at::kStrided || !t->is_cuda();
  }
  explicit operator bool() const { return t != nullptr; }
  const at::Tensor* operator->() const { return t; }
  void* ptr() const { return t ? t->data_ptr() : nullptr; }
};

// The device of the first tensor, which has to be the current one, and every other's.
struct Device {
  int index = -1;
  bool same(const Arg& a) {
    if (a.bad) return false;
    if (!a) return true;
    const int i = a->get_device();
    if (index < 0) index = i;
    return i == index;
  }
  bool current() const { return index >= 0 && c10::hip::current_device() == index; }
  pq_stream_t stream() const { return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(index)).stream(); }
};

template <typename... A>
bool all_on(Device& d, const A&... a) { return (d.same(a) && ...) && d.current(); }

int type_code(at::ScalarType t) { return t == kF16 ? PQ_F16 : t == kBF16 ? PQ_BF16 : t == kF32 ? PQ_F32 : -1; }
bool half_type(at::ScalarType t) { return t == kF16 || t == kBF16; }

bool dense(const Arg& a, at::ScalarType t, at::IntArrayRef shape) {
  return a->scalar_type() == t && a->sizes() == shape && a->is_contiguous();
}
bool bytes(const Arg& a, size_t least) {
  return a->scalar_type() == kU8 && a->is_contiguous() && static_cast<size_t>(a->numel()) >= least;
}
// [M, K] rows with unit column stride
bool rows(const Arg& a, at::ScalarType t, int64_t M, int64_t K) {
  return a->scalar_type() == t && a->dim() == 2 && a->size(0) == M && a->size(1) == K && a->stride(1) == 1;
}
int64_t pitch(const at::Tensor& t, int64_t M, int64_t K) { return M > 1 ? t.stride(0) : K; }

bool fits(int64_t v) { return v >= 0 && v <= INT_MAX; }
bool get_int(PyObject* o, int* v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  const long n = PyLong_AsLongAndOverflow(o, &over);
  if (over || n > INT_MAX || n < INT_MIN) return false;
  *v = static_cast<int>(n);
  return true;
}
bool get_float(PyObject* o, float* v) {
  int i = 0;
  if (PyFloat_CheckExact(o)) *v = static_cast<float>(PyFloat_AS_DOUBLE(o));
  else if (get_int(o, &i)) *v = static_cast<float>(i);
  else return false;
  return true;
}
// The output's type: the given output's, else dtype, else the default; false where they contradict.
bool out_type(const Arg& out, PyObject* dtype, at::ScalarType otherwise, at::ScalarType* t) {
  *t = otherwise;
  if (dtype != Py_None) {
    if (!THPDtype_Check(dtype)) return false;
    *t = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  }
  if (out) {
    if (dtype != Py_None && out->scalar_type() != *t) return false;
    *t = out->scalar_type();
  }
  return half_type(*t);
}
// [M, >= N] rows with unit column stride
bool out_rows(const Arg& out, int64_t M, int64_t N) {
  return out->dim() == 2 && out->size(0) == M && out->size(1) >= N && out->stride(1) == 1;
}

PyObject* unusual() { Py_RETURN_NOTIMPLEMENTED; }

// The given output (a new reference), or the one made here.
PyObject* result(PyObject* given, const at::Tensor& made) {
  if (given != Py_None) {
    Py_INCREF(given);
    return given;
  }
  return THPVariable_Wrap(made);
}
// null with the error set for a code that is not PQ_OK
bool ok(const char* fn, int rc) {
  if (rc == PQ_OK) return true;
  PyObject* r = PyObject_CallFunction(check, "si", fn, rc);
  Py_XDECREF(r);
  if (r) PyErr_SetString(PyExc_RuntimeError, fn);   // check raises
  return false;
}
// Other Python threads run while a launch is queued, which waits where the queue is full.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F, typename... A>
int call(F f, A... a) {
  Unlocked u;
  return f(a...);
}

// rotate(x, rec, cs, out)
PyObject* rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) return unusual();
  const Arg x(a[0]), rec(a[1]), cs(a[2]), out(a[3]);
  Device d;
  if (!x || !rec || !cs || !all_on(d, x, rec, cs, out)) return unusual();
  const at::ScalarType t = x->scalar_type();
  if (x->dim() != 2 || x->stride(1) != 1 || !half_type(t)) return unusual();
  const int64_t M = x->size(0), K = x->size(1), P = rec->dim() == 4 ? rec->size(0) : 1;
  if (!fits(M) || !fits(K) || K == 0 || K % PQ_GROUP || P < 1 || P > PQ_MAX_PARTITIONS) return unusual();
  if (!(rec->dim() == 4 ? dense(rec, kU8, {P, PQ_LAYERS, K / 2, 8}) : dense(rec, kU8, {PQ_LAYERS, K / 2, 8})) ||
      !(cs->dim() == 2 ? dense(cs, kF16, {P, K}) : P == 1 && dense(cs, kF16, {K})))
    return unusual();
  if (out && !dense(out, t, {P, M, K})) return unusual();
  at::Tensor y;
  if (!out) y = at::empty({P, M, K}, x->options());
  void* yp = out ? out.ptr() : y.data_ptr();
  const int rc = call(pq.rotate, static_cast<const uint16_t*>(x.ptr()), pitch(*x.t, M, K), type_code(t), static_cast<int>(M), static_cast<int>(K),
                        static_cast<int>(P), rec.ptr(), static_cast<const uint16_t*>(cs.ptr()), static_cast<uint16_t*>(yp), d.stream());
  return ok("pq_rotate", rc) ? result(a[3], y) : nullptr;
  END_HANDLE_TH_ERRORS
}

// matvec(x, wpk, sz, N, pb1, pb2, out, dtype)
PyObject* matvec(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int N, pb1, pb2;
  if (n != 8 || !get_int(a[3], &N) || !get_int(a[4], &pb1) || !get_int(a[5], &pb2)) return unusual();
  const Arg x(a[0]), wpk(a[1]), sz(a[2]), out(a[6]);
  Device d;
  if (!x || !wpk || !sz || !all_on(d, x, wpk, sz, out)) return unusual();
  const at::ScalarType t = x->scalar_type();
  const int64_t dim = x->dim();
  if ((dim != 2 && dim != 3) || !half_type(t)) return unusual();
  const int64_t P = dim == 3 ? x->size(0) : 1, M = x->size(dim - 2), K = x->size(dim - 1);
  if (!fits(P) || !fits(K) || K == 0 || K % PQ_GROUP || M > 16) return unusual();
  if (dim == 3 ? !x->is_contiguous() : x->stride(1) != 1) return unusual();
  const size_t need = pq.packed_weight_bytes(static_cast<int>(K), N);
  if (need == 0 || !bytes(wpk, need) || !dense(sz, kF16, {K / PQ_GROUP, N, 2})) return unusual();
  at::ScalarType ot;
  if ((out && !out_rows(out, M, N)) || !out_type(out, a[7], t, &ot)) return unusual();
  at::Tensor y;
  if (!out) y = at::empty({M, N}, x->options().dtype(ot));
  const at::Tensor& o = out ? *out.t : y;
  const int64_t ldx = dim == 3 ? K : pitch(*x.t, M, K), ldy = pitch(o, M, N);
  const int rc = call(pq.matvec, static_cast<const uint16_t*>(x.ptr()), ldx, type_code(t), static_cast<int>(M), static_cast<int>(K),
                        static_cast<int>(P), wpk.ptr(), static_cast<const uint16_t*>(sz.ptr()), N, pb1, pb2,
                        static_cast<uint16_t*>(o.data_ptr()), ldy, type_code(ot), d.stream());
  return ok("pq_matvec", rc) ? result(a[6], y) : nullptr;
  END_HANDLE_TH_ERRORS
}

// gemm_glu(A, ASG, RS, wpk, sz, F, act, out, dtype, workspace, prepared)
PyObject* gemm_glu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int F, act;
  if (n != 11 || !get_int(a[5], &F) || !get_int(a[6], &act) || !PyBool_Check(a[10])) return unusual();
  const Arg A(a[0]), asg(a[1]), rs(a[2]), wpk(a[3]), sz(a[4]), out(a[7]), ws(a[9]);
  const bool prepared = a[10] == Py_True;
  Device d;
  if (!A || !asg || !rs || !wpk || !sz || !all_on(d, A, asg, rs, wpk, sz, out, ws) || A->dim() != 3) return unusual();
  const int64_t P = A->size(0), M = A->size(1), K = A->size(2), G = K / PQ_GROUP;
  if (!fits(P) || !fits(M) || !fits(K) || K == 0 || K % PQ_GROUP || F <= 0 || F % 16 || F > INT_MAX / 2) return unusual();
  const size_t need = pq.packed_weight_bytes(static_cast<int>(K), 2 * F);
  if (need == 0 || !dense(A, kU8, {P, M, K}) || !dense(asg, kF32, {P, M, G}) || !dense(rs, kF32, {P, M, G}) || !bytes(wpk, need) ||
      !dense(sz, kF16, {G, 2 * static_cast<int64_t>(F), 2}))
    return unusual();
  const size_t wsb = pq.gemm_workspace_bytes(static_cast<int>(M), 2 * F, static_cast<int>(K));
  if (ws ? !bytes(ws, wsb) : prepared && wsb) return unusual();
  at::ScalarType ot;
  if ((out && !out_rows(out, M, F)) || !out_type(out, a[8], kF16, &ot)) return unusual();
  at::Tensor h, made;
  if (!out) h = at::empty({M, F}, A->options().dtype(ot));
  if (!ws && wsb) made = at::empty({static_cast<int64_t>(wsb)}, A->options());
  const at::Tensor& o = out ? *out.t : h;
  void* wsp = ws ? ws.ptr() : wsb ? made.data_ptr() : nullptr;
  const size_t wsn = ws ? static_cast<size_t>(ws->numel()) : wsb;
  const int64_t ldh = pitch(o, M, F);
  const int rc = call(pq.gemm_glu, static_cast<const uint8_t*>(A.ptr()), static_cast<const float*>(asg.ptr()), static_cast<const float*>(rs.ptr()),
                          static_cast<int>(M), static_cast<int>(K), static_cast<int>(P), wpk.ptr(), static_cast<const uint16_t*>(sz.ptr()), F,
                          act, static_cast<uint16_t*>(o.data_ptr()), ldh, type_code(ot), wsp, wsn, prepared ? 1 : 0, d.stream());
  return ok("pq_gemm_glu", rc) ? result(a[7], h) : nullptr;
  END_HANDLE_TH_ERRORS
}

// block_norms(x, residual, w_post, gate, w_pre, eps, scale, res_scale, gate_act, gemma, residual_out, out)
PyObject* block_norms(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  float eps, scale, res_scale;
  int act;
  if (n != 12 || !get_float(a[5], &eps) || !get_float(a[6], &scale) || !get_float(a[7], &res_scale) || !get_int(a[8], &act) ||
      !PyBool_Check(a[9]))
    return unusual();
  const Arg x(a[0]), res(a[1]), w_post(a[2]), gate(a[3]), w_pre(a[4]), ro(a[10]), out(a[11]);
  Device d;
  if (!x || !res || !all_on(d, x, res, w_post, gate, w_pre, ro, out) || x->dim() != 2 || (out && !w_pre)) return unusual();
  const int64_t M = x->size(0), K = x->size(1);
  const at::ScalarType xt = x->scalar_type(), rt = res->scalar_type();
  const at::ScalarType wt = w_pre ? w_pre->scalar_type() : w_post ? w_post->scalar_type() : kF16;
  if (!fits(M) || !fits(K) || !half_type(xt) || type_code(rt) < 0 || !half_type(wt)) return unusual();
  if (!rows(x, xt, M, K) || !rows(res, rt, M, K) || (w_post && !dense(w_post, wt, {K})) || (w_pre && !dense(w_pre, wt, {K})) ||
      (ro && !rows(ro, rt, M, K)) || (out && !rows(out, wt, M, K)))
    return unusual();
  int64_t ldg = 0, gcols = K;
  if (gate) {
    if (gate->dim() == 1) {
      if (!dense(gate, xt, {K})) return unusual();
    } else if (gate->dim() == 2 && gate->size(1) == 1 && gate->size(0) == M && gate->scalar_type() == xt) {
      gcols = 1;
      ldg = pitch(*gate.t, M, 1);
    } else {
      if (!rows(gate, xt, M, K)) return unusual();
      ldg = pitch(*gate.t, M, K);
    }
  }
  at::Tensor h, hs;
  if (!ro) h = at::empty({M, K}, res->options());
  if (!out && w_pre) hs = at::empty({M, K}, w_pre->options());
  const at::Tensor& o = ro ? *ro.t : h;
  const at::Tensor* s = out ? out.t : w_pre ? &hs : nullptr;
  const int64_t ldo = pitch(o, M, K), lds = s ? pitch(*s, M, K) : K;
  const int rc = call(pq.block_norms, x.ptr(), pitch(*x.t, M, K), type_code(xt), res.ptr(), pitch(*res.t, M, K), type_code(rt), w_post.ptr(),
                             gate.ptr(), ldg, static_cast<int>(gcols), act, w_pre.ptr(), eps, scale, res_scale, a[9] == Py_True ? 1 : 0,
                             static_cast<int>(M), static_cast<int>(K), o.data_ptr(), ldo, s ? s->data_ptr() : nullptr, lds, type_code(wt),
                             d.stream());
  if (!ok("pq_block_norms", rc)) return nullptr;
  PyObject* first = result(a[10], h);
  PyObject* second = nullptr;
  if (first) {
    if (s) second = result(a[11], hs);
    else { Py_INCREF(Py_None); second = Py_None; }
  }
  PyObject* pair = first && second ? PyTuple_Pack(2, first, second) : nullptr;
  Py_XDECREF(first);
  Py_XDECREF(second);
  return pair;
  END_HANDLE_TH_ERRORS
}

// bind(check, abi_version, rotate, matvec, gemm_glu, block_norms, packed_weight_bytes, gemm_workspace_bytes): addresses, of a
// library of this ABI version. The signatures are the ones that pq.h had when this file was compiled, so another version raises.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long f[6];
  PyObject* c;
  int version;
  if (!PyArg_ParseTuple(args, "OiKKKKKK", &c, &version, f, f + 1, f + 2, f + 3, f + 4, f + 5)) return nullptr;
  if (version != PQ_ABI_VERSION) {
    PyErr_Format(PyExc_ImportError, "compiled for ABI version %d of the library, which has %d", PQ_ABI_VERSION, version);
    return nullptr;
  }
  Py_INCREF(c);
  Py_XDECREF(check);
  check = c;
  pq.rotate = reinterpret_cast<decltype(pq.rotate)>(f[0]);
  pq.matvec = reinterpret_cast<decltype(pq.matvec)>(f[1]);
  pq.gemm_glu = reinterpret_cast<decltype(pq.gemm_glu)>(f[2]);
  pq.block_norms = reinterpret_cast<decltype(pq.block_norms)>(f[3]);
  pq.packed_weight_bytes = reinterpret_cast<decltype(pq.packed_weight_bytes)>(f[4]);
  pq.gemm_workspace_bytes = reinterpret_cast<decltype(pq.gemm_workspace_bytes)>(f[5]);
  Py_RETURN_NONE;
}

#define PQ_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         {"rotate", PQ_FAST(rotate), nullptr},
                         {"matvec", PQ_FAST(matvec), nullptr},
                         {"gemm_glu", PQ_FAST(gemm_glu), nullptr},
                         {"block_norms", PQ_FAST(block_norms), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
