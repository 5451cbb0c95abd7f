// The operators around the recurrent layer on torch tensors: a Python module
// that checks the tensors, allocates the outputs and calls the C entry points
// (include/kda.h) on the current stream.  Compiled because such a call on one
// token takes the GPU less time than Python needs to look at its arguments:
// the same steps in Python with ctypes took 12 to 26 us of host time.
//
// The C library is loaded by path (select), so that the module serves the
// normal and the bounds-checked build.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <map>
#include <string>

#include "kda.h"

namespace {

// ---- the library
struct Library {
  decltype(&kda_add_rms_norm) add_rms_norm;
  decltype(&kda_matmul_fp8) matmul_fp8;
  decltype(&kda_short_conv_fwd) short_conv_fwd;
  decltype(&kda_short_conv_step) short_conv_step;
  decltype(&kda_ssm_scan_fwd) ssm_scan_fwd;
  decltype(&kda_ssm_scan_step) ssm_scan_step;
  decltype(&kda_attention_fwd) attention_fwd;
  decltype(&kda_kv4_write) kv4_write;
  decltype(&kda_kv4_read) kv4_read;
  decltype(&kda_kv4_attention) kv4_attention;
  decltype(&kda_last_error_message) last_error_message;
};
std::map<std::string, Library> g_libraries;
const Library* g_lib = nullptr;
PyObject* g_error = nullptr;  // KdaError(status, message)

struct Refused {
  int status;
  std::string message;
};
[[noreturn]] void refuse(const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  throw Refused{KDA_ERR_INVALID_ARGUMENT, buf};
}

PyObject* raise(const Refused& r) {
  PyObject* args = Py_BuildValue("(is)", r.status, r.message.c_str());
  if (args) {
    PyErr_SetObject(g_error, args);
    Py_DECREF(args);
  }
  return nullptr;
}

// A call: refusals become KdaError, torch's own errors their Python forms.
template <typename F>
PyObject* call(Py_ssize_t given, Py_ssize_t wanted, F f) {
  HANDLE_TH_ERRORS
  if (given != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", wanted, given);
    return nullptr;
  }
  try {
    if (!g_lib) refuse("no library is selected");
    return f();
  } catch (const Refused& r) {
    return raise(r);
  }
  END_HANDLE_TH_ERRORS
}

void check(kda_status st) {
  if (st != KDA_OK) throw Refused{st, g_lib->last_error_message()};
}

// ---- arguments
using Tensor = at::Tensor;
const Tensor kNone;

const Tensor& tensor(PyObject* o, const char* name, bool optional = false) {
  if (optional && o == Py_None) return kNone;
  if (!THPVariable_Check(o)) refuse("%s must be a tensor%s", name, optional ? " or None" : "");
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}
void same_shape(const Tensor& t, at::IntArrayRef shape, const char* name) {
  if (t.sizes() != shape)
    refuse("%s must have the shape %s, got %s", name, shape_of(shape).c_str(), shape_of(t.sizes()).c_str());
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "bfloat16";
    case at::kFloat: return "float32";
    case at::kInt: return "int32";
    case at::kFloat8_e4m3fn: return "float8_e4m3fn";
    default: return c10::toString(t);
  }
}
kda_dtype code_of(at::ScalarType t, const char* name) {
  if (t == at::kBFloat16) return KDA_BF16;
  if (t == at::kFloat) return KDA_F32;
  refuse("%s must be bfloat16 or float32, got %s", name, type_name(t));
}
// Of that type, on x's GPU (the library runs on one GPU and cannot tell whose a pointer is).
void of_type(const Tensor& t, at::ScalarType type, const char* name, const Tensor& x) {
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
  if (t.get_device() != x.get_device())
    refuse("%s is on cuda:%d, expected cuda:%d", name, (int)t.get_device(), (int)x.get_device());
  if (t.scalar_type() != type)
    refuse("%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
}

// Rows with a unit last stride, one stride apart over all leading dimensions.
// A single row stands its `width` from a next one (by default the last dimension).
struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
};
Rows rows(void* p, at::IntArrayRef shape, at::IntArrayRef stride, const char* name, int64_t width = 0) {
  const int64_t d = shape.size();
  if (d < 2) refuse("%s must have at least 2 dimensions", name);
  if (stride[d - 1] != 1 && shape[d - 1] > 1) refuse("%s: the last dimension must be contiguous", name);
  const int64_t alone = std::max<int64_t>({width, shape[d - 1], 1});
  int64_t ld = alone, n = 1;  // the rows of the dimensions looked at, and their distance
  bool refused = false;
  for (int64_t k = d - 2; k >= 0; --k) {
    if (shape[k] == 0) return Rows{p, alone};  // no rows
    if (shape[k] == 1) continue;               // its stride says nothing
    if (n == 1) ld = stride[k];
    else refused = refused || stride[k] != ld * n;
    n *= shape[k];
  }
  if (refused) refuse("%s: the leading dimensions must be one row stride apart", name);
  return Rows{p, ld};
}
Rows rows(const Tensor& t, at::ScalarType type, const char* name, const Tensor& x) {
  if (!t.defined()) return Rows{};
  of_type(t, type, name, x);
  return rows(t.data_ptr(), t.sizes(), t.strides(), name);
}
// A contiguous tensor of that shape, or none.
void* dense(const Tensor& t, at::IntArrayRef shape, at::ScalarType type, const char* name,
            const Tensor& x) {
  if (!t.defined()) return nullptr;
  of_type(t, type, name, x);
  if (!t.is_contiguous()) refuse("%s must be contiguous", name);
  same_shape(t, shape, name);
  return t.data_ptr();
}

// The output given, its shape checked, or a new one.
Tensor output(PyObject* given, at::IntArrayRef shape, at::ScalarType type, const Tensor& like,
              const char* name) {
  const Tensor& t = tensor(given, name, true);
  if (!t.defined()) return at::empty(shape, like.options().dtype(type));
  same_shape(t, shape, name);
  return t;
}

// For the time of a library call x's GPU is the current one; its current stream.
struct Launch {
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit Launch(const Tensor& x)
      : guard(x.device()), stream(c10::cuda::getCurrentCUDAStream(x.get_device()).stream()) {}
};

int64_t row_count(const Tensor& t) {
  int64_t n = 1;
  for (int64_t k = 0; k + 1 < t.dim(); ++k) n *= t.size(k);
  return n;
}
std::vector<int64_t> with_last(const Tensor& t, int64_t last) {
  std::vector<int64_t> s = t.sizes().vec();
  s.back() = last;
  return s;
}
const Tensor& matrix(const Tensor& t, const char* name) {
  if (t.dim() < 2) refuse("%s must have at least 2 dimensions", name);
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
  return t;
}
int32_t narrow(int64_t v, const char* name) {
  if (v < 0 || v > INT32_MAX)
    refuse("%s=%lld is %s", name, (long long)v, v < 0 ? "negative" : "too large");
  return static_cast<int32_t>(v);
}

// (tokens, sequences, cu_seqlens) of packed [T, dim] or uniform [B, T_b, dim] x.
struct Sequences {
  int64_t tokens;
  int32_t count;
  const int32_t* cu;
};
Sequences sequences(const Tensor& x, PyObject* cu_o, PyObject* n_o) {
  const Tensor& cu = tensor(cu_o, "cu_seqlens", true);
  Sequences s{row_count(x), 0, nullptr};
  if (cu.defined()) {
    if (cu.dim() != 1 || cu.size(0) < 1) refuse("cu_seqlens must be a vector of n_seqs + 1 elements");
    s.cu = static_cast<const int32_t*>(dense(cu, cu.sizes(), at::kInt, "cu_seqlens", x));
    s.count = narrow(cu.size(0) - 1, "n_seqs");
  } else {
    s.count = narrow(n_o != Py_None ? integer(n_o) : x.dim() > 2 ? x.size(0) : 1, "n_seqs");
  }
  return s;
}

// ---- the operators
// x, weight, residual, eps, y, y_scale, h, quant
PyObject* add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 8, [&]() -> PyObject* {
    const Tensor& x = matrix(tensor(a[0], "x"), "x");
    const Tensor& weight = tensor(a[1], "weight");
    const Tensor& residual = tensor(a[2], "residual", true);
    const bool quant = a[7] == Py_True;
    const at::ScalarType type = x.scalar_type();
    const kda_dtype code = code_of(type, "x"), w_code = code_of(weight.scalar_type(), "weight");
    const int64_t dim = x.sizes().back(), groups = (dim + 127) / 128;
    const Rows xr = rows(x, type, "x", x);
    const void* wp = dense(weight, {dim}, weight.scalar_type(), "weight", x);
    if (residual.defined()) same_shape(residual, x.sizes(), "residual");
    const Rows rr = rows(residual, type, "residual", x);
    Tensor h, y, scale;
    if (residual.defined() || a[6] != Py_None) h = output(a[6], x.sizes(), type, x, "h");
    const Rows hr = rows(h, type, "h", x);
    const at::ScalarType y_type = quant ? at::kFloat8_e4m3fn : type;
    if (quant && a[4] == Py_None) {  // rows at multiples of 16 bytes, as matmul_fp8 reads them
      std::vector<int64_t> stride(x.dim(), 1);
      stride[x.dim() - 2] = (dim + 15) / 16 * 16;
      for (int64_t k = x.dim() - 3; k >= 0; --k) stride[k] = stride[k + 1] * x.size(k + 1);
      y = at::empty_strided(x.sizes(), stride, x.options().dtype(y_type));
    } else {
      y = output(a[4], x.sizes(), y_type, x, "y");
    }
    if (quant) scale = output(a[5], with_last(x, groups), at::kFloat, x, "y_scale");
    const Rows yr = rows(y, y_type, "y", x), sr = rows(scale, at::kFloat, "y_scale", x);
    const Launch on(x);
    check(g_lib->add_rms_norm(xr.p, xr.ld, rr.p, rr.ld, wp, hr.p, hr.ld, yr.p, yr.ld,
                              static_cast<float*>(sr.p), sr.ld, row_count(x), narrow(dim, "dim"),
                              static_cast<float>(real(a[3])), code, w_code, quant ? KDA_E4M3 : code,
                              on.stream));
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    auto item = [](const Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); };
    PyTuple_SET_ITEM(r, 0, item(y));
    PyTuple_SET_ITEM(r, 1, item(scale));
    PyTuple_SET_ITEM(r, 2, item(h));
    return r;
  });
}

// a, a_scale, b, b_scale, out, whether a new out is float32
PyObject* matmul_fp8(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call(n, 6, [&]() -> PyObject* {
    const Tensor& a = matrix(tensor(v[0], "a"), "a");
    const Tensor& b = matrix(tensor(v[2], "b"), "b");
    const Tensor& a_scale = matrix(tensor(v[1], "a_scale"), "a_scale");
    const Tensor& b_scale = matrix(tensor(v[3], "b_scale"), "b_scale");
    const int64_t K = a.sizes().back(), N = b.size(0), M = row_count(a), blocks = (K + 127) / 128;
    if (b.dim() != 2 || b.size(1) != K)
      refuse("a has %lld columns and b has the shape %s", (long long)K, shape_of(b.sizes()).c_str());
    same_shape(a_scale, with_last(a, blocks), "a_scale");
    same_shape(b_scale, {(N + 127) / 128, blocks}, "b_scale");
    const Rows ar = rows(a, at::kFloat8_e4m3fn, "a", a), br = rows(b, at::kFloat8_e4m3fn, "b", a);
    const Rows as = rows(a_scale, at::kFloat, "a_scale", a), bs = rows(b_scale, at::kFloat, "b_scale", a);
    const Tensor out = output(v[4], with_last(a, N), v[5] == Py_True ? at::kFloat : at::kBFloat16, a, "out");
    const kda_dtype code = code_of(out.scalar_type(), "out");
    const Rows o = rows(out, out.scalar_type(), "out", a);
    const Launch on(a);
    check(g_lib->matmul_fp8(ar.p, ar.ld, static_cast<float*>(as.p), as.ld, br.p, br.ld,
                            static_cast<float*>(bs.p), bs.ld, o.p, o.ld, narrow(M, "M"), narrow(N, "N"),
                            narrow(K, "K"), code, on.stream));
    return THPVariable_Wrap(out);
  });
}

// What the convolution's two calls share.
struct Conv {
  const Tensor& x;
  const Tensor& weight;
  at::ScalarType type;
  kda_dtype code, w_code;
  int64_t dim;
  int32_t width;
  Rows xr;
  const void *wp, *bp;

  Conv(PyObject* x_o, PyObject* w_o, PyObject* b_o)
      : x(matrix(tensor(x_o, "x"), "x")), weight(tensor(w_o, "weight")) {
    type = x.scalar_type();
    code = code_of(type, "x");
    w_code = code_of(weight.scalar_type(), "weight");
    dim = x.sizes().back();
    if (weight.dim() != 2 || weight.size(0) != dim)
      refuse("weight must have the shape (%lld, width), got %s", (long long)dim,
             shape_of(weight.sizes()).c_str());
    width = narrow(weight.size(1), "width");
    if (width == 0) refuse("weight has a width of 0");
    xr = rows(x, type, "x", x);
    wp = dense(weight, weight.sizes(), weight.scalar_type(), "weight", x);
    bp = dense(tensor(b_o, "bias", true), {dim}, weight.scalar_type(), "bias", x);
  }
};

// x, weight, bias, conv_state, cu_seqlens, n_seqs, silu, want_state, y, state_out
PyObject* short_conv_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 10, [&]() -> PyObject* {
    const Conv c(a[0], a[1], a[2]);
    const Sequences s = sequences(c.x, a[4], a[5]);
    const int64_t shape[3] = {s.count, c.width - 1, c.dim};
    const void* in = dense(tensor(a[3], "conv_state", true), shape, c.type, "conv_state", c.x);
    const Tensor y = output(a[8], c.x.sizes(), c.type, c.x, "y");
    const Rows yr = rows(y, c.type, "y", c.x);
    Tensor state;
    if (a[7] == Py_True || a[9] != Py_None) state = output(a[9], shape, c.type, c.x, "state_out");
    void* to = dense(state, shape, c.type, "state_out", c.x);
    const Launch on(c.x);
    check(g_lib->short_conv_fwd(c.xr.p, c.xr.ld, c.wp, c.bp, in, to, s.cu, yr.p, yr.ld, s.tokens,
                                s.count, narrow(c.dim, "dim"), c.width, a[6] == Py_True, c.code,
                                c.w_code, on.stream));
    return Py_BuildValue("(NN)", THPVariable_Wrap(y),
                         state.defined() ? THPVariable_Wrap(state) : Py_NewRef(Py_None));
  });
}

// x, weight, conv_state, bias, silu, y
PyObject* short_conv_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 6, [&]() -> PyObject* {
    const Conv c(a[0], a[1], a[3]);
    if (c.x.dim() != 2) refuse("x must have 2 dimensions, got %s", shape_of(c.x.sizes()).c_str());
    const int64_t shape[3] = {c.x.size(0), c.width - 1, c.dim};
    void* state = dense(tensor(a[2], "conv_state"), shape, c.type, "conv_state", c.x);
    const Tensor y = output(a[5], c.x.sizes(), c.type, c.x, "y");
    const Rows yr = rows(y, c.type, "y", c.x);
    const Launch on(c.x);
    check(g_lib->short_conv_step(c.xr.p, c.xr.ld, c.wp, c.bp, state, yr.p, yr.ld,
                                 narrow(c.x.size(0), "n_seqs"), narrow(c.dim, "dim"), c.width,
                                 a[4] == Py_True, c.code, c.w_code, on.stream));
    return THPVariable_Wrap(y);
  });
}

// What the scan's two calls share.  B and C are [..., groups, state], a token's
// values dense.
struct Ssm {
  const Tensor& x;
  at::ScalarType type;
  kda_dtype code;
  int64_t dim, groups, state;
  Rows xr, dtr, zr, br, cr;
  const float *A, *D, *bias;

  Rows groups_of(const Tensor& t, const char* name) const {
    const int64_t d = t.dim();
    if (d != x.dim() + 1 || t.sizes().slice(0, d - 2) != x.sizes().slice(0, d - 2))
      refuse("%s must have x's leading dimensions and (groups, state), got %s", name,
             shape_of(t.sizes()).c_str());
    if (t.size(-2) > 1 && t.stride(-2) != t.size(-1)) refuse("%s: the groups of a token must be dense", name);
    if (t.size(-2) == 0) refuse("%s has no groups", name);
    of_type(t, type, name, x);
    // a token's first group stands for its row (a view by select took 2 us)
    at::DimVector shape(t.sizes()), stride(t.strides());
    shape.erase(shape.end() - 2);
    stride.erase(stride.end() - 2);
    return rows(t.data_ptr(), shape, stride, name, t.size(-2) * t.size(-1));
  }

  Ssm(PyObject* x_o, PyObject* dt_o, PyObject* A_o, PyObject* B_o, PyObject* C_o, PyObject* D_o,
      PyObject* z_o, PyObject* bias_o)
      : x(matrix(tensor(x_o, "x"), "x")) {
    const Tensor &dt = tensor(dt_o, "dt"), &z = tensor(z_o, "z", true);
    const Tensor &B = tensor(B_o, "B"), &C = tensor(C_o, "C");
    type = x.scalar_type();
    code = code_of(type, "x");
    dim = x.sizes().back();
    xr = rows(x, type, "x", x);
    same_shape(dt, x.sizes(), "dt");
    dtr = rows(dt, type, "dt", x);
    if (z.defined()) same_shape(z, x.sizes(), "z");
    zr = rows(z, type, "z", x);
    br = groups_of(B, "B");
    same_shape(C, B.sizes(), "C");
    cr = groups_of(C, "C");
    groups = B.size(-2);
    state = B.size(-1);
    A = static_cast<float*>(dense(tensor(A_o, "A"), {dim, state}, at::kFloat, "A", x));
    D = static_cast<float*>(dense(tensor(D_o, "D", true), {dim}, at::kFloat, "D", x));
    bias = static_cast<float*>(dense(tensor(bias_o, "dt_bias", true), {dim}, at::kFloat, "dt_bias", x));
  }
};

// x, dt, A, B, C, D, z, dt_bias, h0, cu_seqlens, n_seqs, softplus, want_state, y, h_final
PyObject* ssm_scan_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 15, [&]() -> PyObject* {
    const Ssm m(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7]);
    const Sequences s = sequences(m.x, a[9], a[10]);
    const int64_t shape[3] = {s.count, m.dim, m.state};
    const float* h0 = static_cast<float*>(dense(tensor(a[8], "h0", true), shape, at::kFloat, "h0", m.x));
    const Tensor y = output(a[13], m.x.sizes(), m.type, m.x, "y");
    const Rows yr = rows(y, m.type, "y", m.x);
    Tensor h;
    if (a[12] == Py_True || a[14] != Py_None) h = output(a[14], shape, at::kFloat, m.x, "h_final");
    float* to = static_cast<float*>(dense(h, shape, at::kFloat, "h_final", m.x));
    const Launch on(m.x);
    check(g_lib->ssm_scan_fwd(m.xr.p, m.xr.ld, m.dtr.p, m.dtr.ld, m.A, m.br.p, m.br.ld, m.cr.p, m.cr.ld,
                              m.D, m.zr.p, m.zr.ld, m.bias, h0, s.cu, yr.p, yr.ld, to, s.tokens, s.count, narrow(m.dim, "dim"), narrow(m.state, "state"),
                              narrow(m.groups, "groups"), a[11] == Py_True, m.code, on.stream));
    return Py_BuildValue("(NN)", THPVariable_Wrap(y),
                         h.defined() ? THPVariable_Wrap(h) : Py_NewRef(Py_None));
  });
}

// x, dt, A, B, C, h, D, z, dt_bias, softplus, y
PyObject* ssm_scan_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&]() -> PyObject* {
    const Ssm m(a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8]);
    if (m.x.dim() != 2) refuse("x must have 2 dimensions, got %s", shape_of(m.x.sizes()).c_str());
    const int64_t shape[3] = {m.x.size(0), m.dim, m.state};
    float* h = static_cast<float*>(dense(tensor(a[5], "h"), shape, at::kFloat, "h", m.x));
    const Tensor y = output(a[10], m.x.sizes(), m.type, m.x, "y");
    const Rows yr = rows(y, m.type, "y", m.x);
    const Launch on(m.x);
    check(g_lib->ssm_scan_step(m.xr.p, m.xr.ld, m.dtr.p, m.dtr.ld, m.A, m.br.p, m.br.ld, m.cr.p, m.cr.ld,
                               m.D, m.zr.p, m.zr.ld, m.bias, h, yr.p, yr.ld,
                               narrow(m.x.size(0), "n_seqs"), narrow(m.dim, "dim"),
                               narrow(m.state, "state"), narrow(m.groups, "groups"), a[9] == Py_True,
                               m.code, on.stream));
    return THPVariable_Wrap(y);
  });
}

// ---- full attention
// Tokens of heads: [..., heads, d], a token's values dense.
struct Heads {
  void* p = nullptr;
  int64_t ld = 0, tokens = 1, heads = 0, d = 0;
};
Heads heads_of(const Tensor& t, const char* name, const Tensor& x) {
  const int64_t n = t.dim();
  if (n < 3) refuse("%s must have at least 3 dimensions, got %s", name, shape_of(t.sizes()).c_str());
  if (n > 4) refuse("%s must have 3 or 4 dimensions, got %s", name, shape_of(t.sizes()).c_str());
  of_type(t, at::kBFloat16, name, x);
  Heads h;
  h.heads = t.size(n - 2);
  h.d = t.size(n - 1);
  if ((h.d > 1 && t.stride(n - 1) != 1) || (h.heads > 1 && t.stride(n - 2) != h.d))
    refuse("%s: the heads of a token must be dense", name);
  for (int64_t k = 0; k + 2 < n; ++k) h.tokens *= t.size(k);
  // a token's first head stands for its row
  at::DimVector shape(t.sizes()), stride(t.strides());
  shape.erase(shape.end() - 2);
  stride.erase(stride.end() - 2);
  const Rows r = rows(t.data_ptr(), shape, stride, name, h.heads * h.d);
  h.p = r.p;
  h.ld = r.ld;
  return h;
}
// Without cu_seqlens: a uniform batch [B, T_b, heads, d] has as many sequences as the call.
void of_batch(const Tensor& t, const char* name, int64_t seqs) {
  if (t.dim() > 3 && t.size(0) != seqs)
    refuse("%s has %lld sequences, expected %lld", name, (long long)t.size(0), (long long)seqs);
}
const Tensor& on_gpu(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
  return t;
}

float scale_of(PyObject* o, int64_t d) {
  return o == Py_None ? 1.0f / std::sqrt(static_cast<float>(d)) : static_cast<float>(real(o));
}

// The output given or, if wanted, a new one for the sums' logarithms.
Tensor lse_of(PyObject* given, bool want, const Tensor& q) {
  if (!want && given == Py_None) return Tensor();
  return output(given, q.sizes().slice(0, q.dim() - 1), at::kFloat, q, "lse");
}
PyObject* pair(const Tensor& a, const Tensor& b) {
  return Py_BuildValue("(NN)", THPVariable_Wrap(a), b.defined() ? THPVariable_Wrap(b) : Py_NewRef(Py_None));
}

// q, k, v, cu_seqlens_q, cu_seqlens_k, n_seqs, causal, scale, want_lse, out, lse
PyObject* attention_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 11, [&]() -> PyObject* {
    const Tensor& q = on_gpu(tensor(a[0], "q"), "q");
    const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const Heads qh = heads_of(q, "q", q), kh = heads_of(k, "k", q), vh = heads_of(v, "v", q);
    if (k.dim() != q.dim() || kh.d != qh.d)
      refuse("k must have q's dimensions and head size, got %s", shape_of(k.sizes()).c_str());
    same_shape(v, k.sizes(), "v");
    if (q.dim() > 3 && k.size(0) != q.size(0))
      refuse("q has %lld sequences, k %lld", (long long)q.size(0), (long long)k.size(0));
    const Tensor& cq = tensor(a[3], "cu_seqlens_q", true);
    const Tensor& ck = tensor(a[4], "cu_seqlens_k", true);
    if (ck.defined() && !cq.defined()) refuse("cu_seqlens_k is given but cu_seqlens_q is not");
    int32_t seqs;
    const int32_t *cqp = nullptr, *ckp = nullptr;
    if (cq.defined()) {
      if (cq.dim() != 1 || cq.size(0) < 1) refuse("cu_seqlens_q must be a vector of n_seqs + 1 elements");
      seqs = narrow(cq.size(0) - 1, "n_seqs");
      cqp = static_cast<const int32_t*>(dense(cq, cq.sizes(), at::kInt, "cu_seqlens_q", q));
      ckp = static_cast<const int32_t*>(dense(ck, cq.sizes(), at::kInt, "cu_seqlens_k", q));
    } else {
      seqs = narrow(a[5] != Py_None ? integer(a[5]) : q.dim() > 3 ? q.size(0) : 1, "n_seqs");
      of_batch(q, "q", seqs);
    }
    const Tensor out = output(a[9], q.sizes(), at::kBFloat16, q, "out");
    const Heads oh = heads_of(out, "out", q);
    const Tensor lse = lse_of(a[10], a[8] == Py_True, q);
    float* lp = static_cast<float*>(dense(lse, q.sizes().slice(0, q.dim() - 1), at::kFloat, "lse", q));
    const Launch on(q);
    check(g_lib->attention_fwd(qh.p, qh.ld, kh.p, kh.ld, vh.p, vh.ld, cqp, ckp, oh.p, oh.ld, lp, qh.tokens,
                               kh.tokens, seqs, narrow(qh.heads, "heads"), narrow(kh.heads, "kv_heads"),
                               narrow(qh.d, "d"), scale_of(a[7], qh.d), a[6] == Py_True, on.stream));
    return pair(out, lse);
  });
}

// (k_codes, k_scales, v_codes, v_scales) and the block table
struct Pages {
  kda_kv4_cache cache;
  const int32_t* table;
  int64_t ld, seqs;
  int32_t width;

  Pages(PyObject* o, PyObject* table_o, const Tensor& x) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4)
      refuse("cache must be the tuple (k_codes, k_scales, v_codes, v_scales)");
    static const char* const names[4] = {"k_codes", "k_scales", "v_codes", "v_scales"};
    void* p[4];
    const Tensor& codes = tensor(PyTuple_GET_ITEM(o, 0), "k_codes");
    if (codes.dim() != 4)
      refuse("k_codes must have the shape (pages, heads, page_size, d / 2), got %s",
             shape_of(codes.sizes()).c_str());
    at::DimVector shape(codes.sizes());
    const int64_t d = 2 * shape[3];
    for (int i = 0; i < 4; ++i) {
      shape[3] = i % 2 ? d / 32 : d / 2;
      p[i] = dense(tensor(PyTuple_GET_ITEM(o, i), names[i]), shape, i % 2 ? at::kBFloat16 : at::kByte,
                   names[i], x);
    }
    cache = kda_kv4_cache{p[0], p[1], p[2], p[3], narrow(shape[0], "n_pages"), narrow(shape[2], "page_size"),
                          narrow(shape[1], "kv_heads"), narrow(d, "d")};
    const Tensor& t = tensor(table_o, "block_table");
    if (t.dim() != 2) refuse("block_table must have 2 dimensions, got %s", shape_of(t.sizes()).c_str());
    const Rows r = rows(t, at::kInt, "block_table", x);
    table = static_cast<const int32_t*>(r.p);
    ld = r.ld;
    seqs = t.size(0);
    width = narrow(t.size(1), "max_pages");
  }
};

// The spans of both: start, cu_seqlens, n_seqs of tokens [T, heads, d] or [B, T_b, heads, d].
struct Span {
  const int32_t *start, *cu = nullptr;
  int32_t count;

  Span(PyObject* start_o, PyObject* cu_o, PyObject* n_o, const Pages& pages, const Tensor& x) {
    const Tensor& c = tensor(cu_o, "cu_seqlens", true);
    if (c.defined()) {
      if (c.dim() != 1 || c.size(0) < 1) refuse("cu_seqlens must be a vector of n_seqs + 1 elements");
      cu = static_cast<const int32_t*>(dense(c, c.sizes(), at::kInt, "cu_seqlens", x));
      count = narrow(c.size(0) - 1, "n_seqs");
    } else {
      count = narrow(n_o != Py_None ? integer(n_o) : pages.seqs, "n_seqs");
    }
    if (pages.seqs != count)
      refuse("block_table has %lld rows for %d sequences", (long long)pages.seqs, count);
    const Tensor& s = tensor(start_o, "start", true);
    start = static_cast<const int32_t*>(dense(s, {count}, at::kInt, "start", x));
  }
};

void of_cache(const Heads& h, const Pages& p, const char* name) {
  if (h.heads != p.cache.n_kv_heads || h.d != p.cache.d)
    refuse("%s has %lld heads of %lld, the cache %d of %d", name, (long long)h.heads, (long long)h.d,
           p.cache.n_kv_heads, p.cache.d);
}

// k, v, cache, block_table, start, cu_seqlens, n_seqs
PyObject* kv4_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 7, [&]() -> PyObject* {
    const Tensor& k = on_gpu(tensor(a[0], "k"), "k");
    const Tensor& v = tensor(a[1], "v");
    const Heads kh = heads_of(k, "k", k), vh = heads_of(v, "v", k);
    same_shape(v, k.sizes(), "v");
    const Pages p(a[2], a[3], k);
    of_cache(kh, p, "k");
    const Span s(a[4], a[5], a[6], p, k);
    if (!s.cu) of_batch(k, "k", s.count);
    const Launch on(k);
    check(g_lib->kv4_write(kh.p, kh.ld, vh.p, vh.ld, &p.cache, p.table, p.ld, p.width, s.start, s.cu,
                           kh.tokens, s.count, on.stream));
    Py_RETURN_NONE;
  });
}

// cache, block_table, total_tokens, start, cu_seqlens, n_seqs, k, v
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 8, [&]() -> PyObject* {
    const Tensor& table = on_gpu(tensor(a[1], "block_table"), "block_table");
    const Pages p(a[0], a[1], table);
    const Span s(a[3], a[4], a[5], p, table);
    const int64_t tokens = integer(a[2]);
    if (tokens < 0) refuse("total_tokens=%lld is negative", (long long)tokens);
    const int64_t shape[3] = {tokens, p.cache.n_kv_heads, p.cache.d};
    Tensor made[2];
    Heads h[2];
    for (int i = 0; i < 2; ++i) {
      const char* name = i ? "v" : "k";
      const Tensor& t = tensor(a[6 + i], name, true);
      made[i] = t.defined() ? t : at::empty(shape, table.options().dtype(at::kBFloat16));
      h[i] = heads_of(made[i], name, table);
      of_cache(h[i], p, name);
      if (h[i].tokens != tokens)
        refuse("%s has %lld tokens, expected %lld", name, (long long)h[i].tokens, (long long)tokens);
      if (!s.cu) of_batch(made[i], name, s.count);
    }
    const Launch on(table);
    check(g_lib->kv4_read(h[0].p, h[0].ld, h[1].p, h[1].ld, &p.cache, p.table, p.ld, p.width, s.start, s.cu,
                          tokens, s.count, on.stream));
    return pair(made[0], made[1]);
  });
}

// q, cache, block_table, seq_lens, scale, want_lse, out, lse
PyObject* kv4_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call(n, 8, [&]() -> PyObject* {
    const Tensor& q = on_gpu(tensor(a[0], "q"), "q");
    const Heads qh = heads_of(q, "q", q);
    const Pages p(a[1], a[2], q);
    if (qh.d != p.cache.d) refuse("q has heads of %lld, the cache of %d", (long long)qh.d, p.cache.d);
    const int32_t seqs = narrow(q.size(0), "n_seqs");
    if (p.seqs != seqs) refuse("block_table has %lld rows for %d sequences", (long long)p.seqs, seqs);
    const int32_t* lens = static_cast<const int32_t*>(dense(tensor(a[3], "seq_lens"), {seqs}, at::kInt, "seq_lens", q));
    const Tensor out = output(a[6], q.sizes(), at::kBFloat16, q, "out");
    const Heads oh = heads_of(out, "out", q);
    const Tensor lse = lse_of(a[7], a[5] == Py_True, q);
    float* lp = static_cast<float*>(dense(lse, q.sizes().slice(0, q.dim() - 1), at::kFloat, "lse", q));
    const Launch on(q);
    check(g_lib->kv4_attention(qh.p, qh.ld, &p.cache, p.table, p.ld, p.width, lens, oh.p, oh.ld, lp, seqs,
                               q.dim() == 4 ? narrow(q.size(1), "n_tokens") : 1, narrow(qh.heads, "heads"),
                               scale_of(a[4], qh.d), on.stream));
    return pair(out, lse);
  });
}

// path, KdaError: the calls go to the library at that path from now on.
PyObject* select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* path = n == 2 ? PyUnicode_AsUTF8(a[0]) : nullptr;
  if (!path) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "select(path, error class)");
    return nullptr;
  }
  Py_XSETREF(g_error, Py_NewRef(a[1]));
  auto it = g_libraries.find(path);
  if (it == g_libraries.end()) {
    void* lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!lib) {
      PyErr_SetString(PyExc_OSError, dlerror());
      return nullptr;
    }
    Library l;
    auto find = [&](auto& f, const char* name) {
      f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(lib, name));
      return f != nullptr;
    };
    if (!find(l.add_rms_norm, "kda_add_rms_norm") || !find(l.matmul_fp8, "kda_matmul_fp8") ||
        !find(l.short_conv_fwd, "kda_short_conv_fwd") || !find(l.short_conv_step, "kda_short_conv_step") ||
        !find(l.ssm_scan_fwd, "kda_ssm_scan_fwd") || !find(l.ssm_scan_step, "kda_ssm_scan_step") ||
        !find(l.attention_fwd, "kda_attention_fwd") || !find(l.kv4_write, "kda_kv4_write") ||
        !find(l.kv4_read, "kda_kv4_read") || !find(l.kv4_attention, "kda_kv4_attention") ||
        !find(l.last_error_message, "kda_last_error_message")) {
      PyErr_Format(PyExc_OSError, "%s lacks an entry point", path);
      return nullptr;
    }
    it = g_libraries.emplace(path, l).first;
  }
  g_lib = &it->second;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define KDA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {KDA_METHOD(select),         KDA_METHOD(add_rms_norm),
                           KDA_METHOD(matmul_fp8),     KDA_METHOD(short_conv_fwd),
                           KDA_METHOD(short_conv_step), KDA_METHOD(ssm_scan_fwd),
                           KDA_METHOD(ssm_scan_step),  KDA_METHOD(attention_fwd),
                           KDA_METHOD(kv4_write),      KDA_METHOD(kv4_read),
                           KDA_METHOD(kv4_attention),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "kda_torch", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit_kda_torch() { return PyModule_Create(&g_module); }
