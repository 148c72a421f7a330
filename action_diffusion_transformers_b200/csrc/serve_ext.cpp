// serve_ext.cpp - the serving calls for Python callers: reads torch tensors
// directly (no per-argument Python work), checks the layouts that the C ABI
// cannot see, makes the tensors' device current and calls libsage.so on the
// given stream or that device's current one.  Each function returns the call's
// sage_status; a layout it does not take raises ValueError or TypeError before
// anything is launched.  (The same checks written in Python took 11-16 us a
// call, four times what the launch itself takes.)
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <string>
#include <vector>

#include "sage.h"

namespace {

struct Refused {};   // a Python exception is set

[[noreturn]] void refuse(PyObject* kind, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(kind, fmt, ap);
  va_end(ap);
  throw Refused{};
}

std::string shape_of(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor (got %s)", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

int dtype_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return SAGE_BF16;
    case at::kHalf: return SAGE_FP16;
    case at::kFloat: return SAGE_FP32;
    default: refuse(PyExc_TypeError, "%s: dtype %s is not bfloat16, float16 or float32", name, c10::toString(t.scalar_type()));
  }
}
void same_dtype(const at::Tensor& a, const at::Tensor& b, const char* name) {
  if (a.scalar_type() != b.scalar_type())
    refuse(PyExc_TypeError, "%s: %s beside %s", name, c10::toString(b.scalar_type()), c10::toString(a.scalar_type()));
}

// Token stride of rows [T, H, D] whose heads are contiguous (0: one row at most).
int64_t row_stride(const at::Tensor& t, const char* name, int64_t T, int64_t H, int64_t D) {
  if (t.dim() != 3 || t.size(0) != T || t.size(1) != H || t.size(2) != D)
    refuse(PyExc_ValueError, "%s must be [%lld, %lld, %lld] (got %s)", name, (long long)T, (long long)H, (long long)D,
           shape_of(t).c_str());
  if (t.numel() && ((D > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != D)))
    refuse(PyExc_ValueError, "%s: the heads of a token must be contiguous (strides %lld, %lld, %lld)", name,
           (long long)t.stride(0), (long long)t.stride(1), (long long)t.stride(2));
  if (T > 1 && t.stride(0) == 0) refuse(PyExc_ValueError, "%s: its tokens share one row (stride 0)", name);
  return T > 1 ? t.stride(0) : 0;
}

int int_of(int64_t x, const char* name) {
  if (x < 0 || x > 0x7FFFFFFF) refuse(PyExc_ValueError, "%s is too large (%lld)", name, (long long)x);
  return static_cast<int>(x);
}

void three_dims(const at::Tensor& t, const char* name) {
  if (t.dim() != 3) refuse(PyExc_ValueError, "%s must be [T, H, D] (got %s)", name, shape_of(t).c_str());
}

void vector_of(const at::Tensor& t, const char* name, int64_t n, at::ScalarType dt) {
  if (t.scalar_type() != dt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(PyExc_ValueError, "%s must be a contiguous %s tensor [%lld] (got %s %s)", name, c10::toString(dt),
           (long long)n, c10::toString(t.scalar_type()), shape_of(t).c_str());
}

void lse_of(const at::Tensor& t, int64_t a, int64_t b) {
  if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != a || t.size(1) != b || !t.is_contiguous())
    refuse(PyExc_ValueError, "lse must be contiguous float32 [%lld, %lld] (got %s %s)", (long long)a, (long long)b,
           c10::toString(t.scalar_type()), shape_of(t).c_str());
}

sage_kv_cache cache_of(PyObject* const* args, const at::Tensor** first) {
  const at::Tensor &kc = tensor(args[0], "k_codes"), &ks = tensor(args[1], "k_scale"), &vc = tensor(args[2], "v_codes"),
                   &vs = tensor(args[3], "v_scale");
  sage_kv_cache c;
  const at::ScalarType ct = kc.scalar_type();
  if (ct == at::kChar) c.format = SAGE_KV_INT8;
  else if (ct == at::kFloat8_e4m3fn || ct == at::kByte) c.format = SAGE_KV_E4M3;
  else refuse(PyExc_TypeError, "codes must be int8, float8_e4m3fn or uint8 (got %s)", c10::toString(ct));
  if (vc.scalar_type() != ct)
    refuse(PyExc_TypeError, "k_codes are %s, v_codes %s", c10::toString(ct), c10::toString(vc.scalar_type()));
  if (ks.scalar_type() != at::kFloat || vs.scalar_type() != at::kFloat)
    refuse(PyExc_TypeError, "scales must be float32");
  bool ok = kc.dim() == 4 && vc.sizes() == kc.sizes() && ks.dim() == 3 && vs.sizes() == ks.sizes();
  for (int i = 0; ok && i < 3; ++i) ok = ks.size(i) == kc.size(i);
  if (!ok)
    refuse(PyExc_ValueError, "codes must be [pages, Hk, page_size, D] and scales [pages, Hk, page_size] (got %s, %s, %s, %s)",
           shape_of(kc).c_str(), shape_of(vc).c_str(), shape_of(ks).c_str(), shape_of(vs).c_str());
  if (!kc.is_contiguous() || !ks.is_contiguous() || !vc.is_contiguous() || !vs.is_contiguous())
    refuse(PyExc_ValueError, "the cache must be contiguous");
  c.k_codes = kc.data_ptr();
  c.k_scale = static_cast<float*>(ks.data_ptr());
  c.v_codes = vc.data_ptr();
  c.v_scale = static_cast<float*>(vs.data_ptr());
  c.num_pages = int_of(kc.size(0), "pages");
  c.Hk = int_of(kc.size(1), "Hk");
  c.page_size = int_of(kc.size(2), "page_size");
  c.D = int_of(kc.size(3), "D");
  *first = &kc;
  return c;
}

// The tensors' one CUDA device, made current while the call launches.
class OnDevice {
 public:
  OnDevice(PyObject* const* args, std::initializer_list<int> tensors, PyObject* stream) {
    c10::Device dev(c10::kCPU);
    bool first = true;
    for (const int i : tensors) {
      if (args[i] == Py_None) continue;
      if (!THPVariable_Check(args[i])) refuse(PyExc_TypeError, "a tensor is wanted (got %s)", Py_TYPE(args[i])->tp_name);
      const c10::Device d = THPVariable_Unpack(args[i]).device();
      if (first) {
        if (!d.is_cuda()) refuse(PyExc_ValueError, "tensors must be on a CUDA device (got %s)", d.str().c_str());
        dev = d;
        first = false;
      } else if (d != dev) {
        refuse(PyExc_ValueError, "tensors on %s and %s", dev.str().c_str(), d.str().c_str());
      }
    }
    before_ = c10::cuda::current_device();
    mine_ = dev.index();
    if (stream == Py_None) {
      stream_ = c10::cuda::getCurrentCUDAStream(mine_).stream();
    } else {
      PyObject* num = PyLong_Check(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
      if (!num) throw Refused{};
      stream_ = static_cast<cudaStream_t>(PyLong_AsVoidPtr(num));
      Py_DECREF(num);
      if (PyErr_Occurred()) throw Refused{};
    }
    if (mine_ != before_) c10::cuda::set_device(mine_);
  }
  ~OnDevice() {
    if (mine_ != before_) c10::cuda::set_device(before_);
  }
  sage_stream_t stream() const { return reinterpret_cast<sage_stream_t>(stream_); }

 private:
  c10::DeviceIndex before_ = 0, mine_ = 0;
  cudaStream_t stream_ = nullptr;
};

template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
  try {
    if (got != want) refuse(PyExc_TypeError, "%zd arguments, %zd wanted", got, want);
    return PyLong_FromLong(f());
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused{};
  return x;
}
int truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Refused{};
  return x;
}

// q, k, positions, plan address, q_out, k_out, transpose, stream
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const auto* plan = static_cast<const sage_rope_plan*>(PyLong_AsVoidPtr(a[3]));
    if (PyErr_Occurred()) throw Refused{};
    sage_rows rows[2] = {};
    const char* names[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
    int64_t T = 0, D = 0;
    int dt = 0;
    const at::Tensor* first = nullptr;
    for (int w = 0; w < 2; ++w) {
      if (a[w] == Py_None) {
        if (a[4 + w] != Py_None) refuse(PyExc_TypeError, "%s without %s, which must be a tensor", names[w][1], names[w][0]);
        continue;
      }
      const at::Tensor &x = tensor(a[w], names[w][0]), &y = tensor(a[4 + w], names[w][1]);
      three_dims(x, names[w][0]);
      if (!first) {
        first = &x;
        T = x.size(0);
        D = x.size(2);
        dt = dtype_of(x, names[w][0]);
      }
      same_dtype(*first, x, names[w][0]);
      same_dtype(*first, y, names[w][1]);
      const int64_t H = x.size(1);
      rows[w].in_stride = row_stride(x, names[w][0], T, H, D);
      rows[w].out_stride = row_stride(y, names[w][1], T, H, D);
      rows[w].in = x.data_ptr();
      rows[w].out = y.data_ptr();
      rows[w].H = int_of(H, "H");
    }
    if (!first) refuse(PyExc_ValueError, "q or k must be given");
    const at::Tensor& pos = tensor(a[2], "positions");
    const int64_t axes = plan->n_axes;
    if (pos.scalar_type() != at::kLong || !pos.is_contiguous() || pos.dim() < 1 || pos.size(-1) != T ||
        !((pos.dim() == 1 && axes == 1) || (pos.dim() == 2 && pos.size(0) == axes)))
      refuse(PyExc_ValueError, "positions must be contiguous int64 [%lld] for one axis or [%lld, %lld] (got %s %s)",
             (long long)T, (long long)axes, (long long)T, c10::toString(pos.scalar_type()), shape_of(pos).c_str());
    const int tr = truth(a[6]);
    OnDevice on(a, {0, 1, 2, 4, 5}, a[7]);
    return sage_rope(rows[0], rows[1], int_of(T, "T"), int_of(D, "D"), dt, static_cast<const int64_t*>(pos.data_ptr()),
                     plan, tr, on.stream());
  });
}

// k, v, slots, k_codes, k_scale, v_codes, v_scale, stream
template <bool kWrite>
PyObject* py_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const at::Tensor* codes;
    const sage_kv_cache c = cache_of(a + 3, &codes);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots");
    three_dims(k, "k");
    const int64_t T = k.size(0);
    const int64_t ks = row_stride(k, "k", T, c.Hk, c.D), vs = row_stride(v, "v", T, c.Hk, c.D);
    const int dt = dtype_of(k, "k");
    same_dtype(k, v, "v");
    vector_of(slots, "slots", T, at::kLong);
    OnDevice on(a, {0, 1, 2, 3, 4, 5, 6}, a[7]);
    const auto* s = static_cast<const int64_t*>(slots.data_ptr());
    if (kWrite) return sage_kv_write(k.data_ptr(), v.data_ptr(), int_of(T, "T"), ks, vs, dt, s, c, on.stream());
    return sage_kv_read(c, s, int_of(T, "T"), k.data_ptr(), v.data_ptr(), ks, vs, dt, on.stream());
  });
}

// Offsets of packed sequences from a list, a tuple or a CPU tensor.
void offsets(PyObject* o, const char* name, int64_t total, std::vector<int32_t>& out) {
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.device().is_cpu()) refuse(PyExc_ValueError, "%s must be on the host (a list or a CPU tensor)", name);
    if (t.dim() != 1 || (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong))
      refuse(PyExc_ValueError, "%s must be int32 or int64, one-dimensional", name);
    out.resize(t.size(0));
    for (int64_t i = 0; i < t.size(0); ++i)
      out[i] = t.scalar_type() == at::kInt
                   ? static_cast<const int32_t*>(t.data_ptr())[i * t.stride(0)]
                   : static_cast<int32_t>(int_of(static_cast<const int64_t*>(t.data_ptr())[i * t.stride(0)], name));
  } else {
    PyObject* seq = PySequence_Fast(o, "offsets must be a list, a tuple or a CPU tensor");
    if (!seq) throw Refused{};
    const Py_ssize_t m = PySequence_Fast_GET_SIZE(seq);
    out.resize(m);
    bool ok = true;
    for (Py_ssize_t i = 0; ok && i < m; ++i) {
      const long long x = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
      ok = !PyErr_Occurred();
      if (ok && (x < 0 || x > 0x7FFFFFFF)) {
        PyErr_Format(PyExc_ValueError, "%s[%zd] = %lld is out of range", name, i, x);
        ok = false;
      }
      if (ok) out[i] = static_cast<int32_t>(x);
    }
    Py_DECREF(seq);
    if (!ok) throw Refused{};
  }
  if (out.empty() || out.back() != total)
    refuse(PyExc_ValueError, "%s must end at the %lld packed rows (got %d)", name, (long long)total,
           out.empty() ? -1 : out.back());
}

// q, k, v, cu_q, cu_k, out, lse, causal, sm_scale, stream
PyObject* py_prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"), &out = tensor(a[5], "out");
    three_dims(q, "q");
    three_dims(k, "k");
    const int64_t Tq = q.size(0), Hq = q.size(1), D = q.size(2), Tk = k.size(0), Hk = k.size(1);
    sage_prompt p;
    p.dtype = dtype_of(q, "q");
    same_dtype(q, k, "k");
    same_dtype(q, v, "v");
    same_dtype(q, out, "out");
    p.q_stride = row_stride(q, "q", Tq, Hq, D);
    p.k_stride = row_stride(k, "k", Tk, Hk, D);
    p.v_stride = row_stride(v, "v", Tk, Hk, D);
    p.out_stride = row_stride(out, "out", Tq, Hq, D);
    p.Hq = int_of(Hq, "Hq");
    p.Hk = int_of(Hk, "Hk");
    p.D = int_of(D, "D");
    std::vector<int32_t> cq, ck;
    offsets(a[3], "cu_q", Tq, cq);
    offsets(a[4] == Py_None ? a[3] : a[4], "cu_k", Tk, ck);
    if (cq.size() != ck.size())
      refuse(PyExc_ValueError, "cu_q and cu_k name %zd and %zd sequences", cq.size() - 1, ck.size() - 1);
    p.n_seq = static_cast<int>(cq.size()) - 1;
    p.cu_q = cq.data();
    p.cu_k = ck.data();
    float* lse = nullptr;
    if (a[6] != Py_None) {
      const at::Tensor& t = tensor(a[6], "lse");
      lse_of(t, Hq, Tq);
      lse = static_cast<float*>(t.data_ptr());
    }
    p.causal = truth(a[7]);
    p.sm_scale = static_cast<float>(number(a[8]));
    OnDevice on(a, {0, 1, 2, 5, 6}, a[9]);
    return sage_attn_prompt(q.data_ptr(), k.data_ptr(), v.data_ptr(), &p, out.data_ptr(), lse, on.stream());
  });
}

// q, k_codes, k_scale, v_codes, v_scale, page_table, lens, out, workspace, max_len, lse, sm_scale, stream
PyObject* py_token(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const at::Tensor* codes;
    const sage_kv_cache c = cache_of(a + 1, &codes);
    const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[5], "page_table"), &lens = tensor(a[6], "lens"),
                     &out = tensor(a[7], "out");
    three_dims(q, "q");
    const int64_t B = q.size(0), Hq = q.size(1);
    sage_token p;
    p.dtype = dtype_of(q, "q");
    same_dtype(q, out, "out");
    p.q_stride = row_stride(q, "q", B, Hq, c.D);
    p.out_stride = row_stride(out, "out", B, Hq, c.D);
    p.B = int_of(B, "B");
    p.Hq = int_of(Hq, "Hq");
    if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != B ||
        (table.size(1) > 1 && table.stride(1) != 1) || (B > 1 && table.size(1) > 0 && table.stride(0) < table.size(1)))
      refuse(PyExc_ValueError, "page_table must be int32 [%lld, pages] with contiguous rows (got %s %s)", (long long)B,
             c10::toString(table.scalar_type()), shape_of(table).c_str());
    vector_of(lens, "lens", B, at::kInt);
    const int64_t named = table.size(1) * c.page_size;
    int64_t longest = named;
    if (a[9] != Py_None) {
      longest = PyLong_AsLongLong(a[9]);
      if (PyErr_Occurred()) throw Refused{};
      if (longest < 0 || longest > named)
        refuse(PyExc_ValueError, "max_len %lld must be 0 .. %lld, what the page table can name", (long long)longest,
               (long long)named);
    }
    p.max_len = int_of(longest, "max_len");
    p.page_table = static_cast<const int32_t*>(table.data_ptr());
    p.table_stride = B > 1 ? table.stride(0) : table.size(1);
    p.lens = static_cast<const int32_t*>(lens.data_ptr());
    p.sm_scale = static_cast<float>(number(a[11]));
    float* lse = nullptr;
    if (a[10] != Py_None) {
      const at::Tensor& t = tensor(a[10], "lse");
      lse_of(t, B, Hq);
      lse = static_cast<float*>(t.data_ptr());
    }
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[8] != Py_None) {
      const at::Tensor& t = tensor(a[8], "workspace");
      if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
      ws = t.data_ptr();
      ws_bytes = t.nbytes();
    }
    OnDevice on(a, {0, 1, 2, 3, 4, 5, 6, 7, 8, 10}, a[12]);
    return sage_attn_token(q.data_ptr(), &p, c, out.data_ptr(), lse, ws, ws_bytes, on.stream());
  });
}

PyMethodDef kMethods[] = {
    {"rope", reinterpret_cast<PyCFunction>(py_rope), METH_FASTCALL, nullptr},
    {"kv_write", reinterpret_cast<PyCFunction>(py_kv<true>), METH_FASTCALL, nullptr},
    {"kv_read", reinterpret_cast<PyCFunction>(py_kv<false>), METH_FASTCALL, nullptr},
    {"attn_prompt", reinterpret_cast<PyCFunction>(py_prompt), METH_FASTCALL, nullptr},
    {"attn_token", reinterpret_cast<PyCFunction>(py_token), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_serve_ext", "Serving calls of libsage.so on torch tensors.  Built for " SAGE_BUILT_FOR, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve_ext(void) { return PyModule_Create(&kModule); }
