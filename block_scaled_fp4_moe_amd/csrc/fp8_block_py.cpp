// Python entry of the block-scaled FP8 operators (module _fp8_block): argument
// checks, output allocation and the call of the C ABI in include/fp8block.h.
//
// In C++ because a decode step's kernels take 3 to 8 us: the same checks in Python
// with ctypes took 7 us of a call, here they take about 1.
//
// Every function takes positional arguments (None for an absent tensor) and
// the raw stream last; fp8_block.py holds the signatures users see.  A refused
// argument raises ValueError, a status of the library the error class that
// set_error_class received.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <stdexcept>

#include "fp4moe.h"
#include "fp8block.h"

namespace {

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PythonError {};                     // the Python error is set already

PyObject* g_error_class = nullptr;

template <class... Args>
[[noreturn]] void refuse(const Args&... args) {
  std::ostringstream s;
  (s << ... << args);
  throw Refused(s.str());
}

bool is_codes(at::ScalarType t) { return t == at::kByte || t == at::kFloat8_e4m3fn; }

int dtype_code(at::ScalarType t) {
  return t == at::kBFloat16 ? FP8BLOCK_BF16 : t == at::kHalf ? FP8BLOCK_F16 : t == at::kFloat ? FP8BLOCK_F32 : -1;
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, ": a tensor is wanted");
  return THPVariable_Unpack(o);
}

[[noreturn]] void bad(const at::Tensor& t, const char* name, const char* wanted) {
  refuse(name, ": ", t.sizes(), " ", t.scalar_type(), " on ", t.device(), " with strides ",
         t.strides(), "; wanted ", wanted);
}

// Row stride of a matrix; of a single row, whose stride means nothing (torch keeps any
// number there), the row's length.
int64_t ld(const at::Tensor& t) { return t.size(-2) > 1 ? t.stride(-2) : t.size(-1); }

bool rows_contiguous(const at::Tensor& t) { return t.size(-1) <= 1 || t.stride(-1) == 1; }

// A matrix with contiguous rows on the current GPU, at most 2^31-1 either way.
void leading(const at::Tensor& t, const char* name) {
  if (t.dim() != 2 || !rows_contiguous(t)) bad(t, name, "a matrix with contiguous rows");
  const c10::Device d = t.device();
  if (d.type() != at::kCUDA ||
      d.index() != c10::impl::VirtualGuardImpl(at::kCUDA).getDevice().index())
    refuse(name, " is on ", d, ", not on the current GPU");
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) bad(t, name, "fewer than 2^31 rows and columns");
}


void same_matrix(const at::Tensor& t, const char* name, const at::Tensor& x) {
  if (t.sizes() != x.sizes() || t.scalar_type() != x.scalar_type() || t.device() != x.device() ||
      !rows_contiguous(t))
    bad(t, name, "x's shape, type and device, rows contiguous");
}

void scales_matrix(const at::Tensor& t, const char* name, int64_t rows, int64_t blocks,
                   const at::Tensor& x) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != blocks || t.scalar_type() != at::kFloat ||
      t.device() != x.device() || t.stride(0) < 0 || t.stride(1) < 0)
    refuse(name, ": ", t.sizes(), " ", t.scalar_type(), " on ", t.device(), "; wanted float32 [", rows,
           ", ", blocks, "] on ", x.device());
}

void index_tensor(const at::Tensor& t, const char* name, int64_t least, const at::Tensor& x) {
  if (t.scalar_type() != at::kInt || t.numel() < least || t.device() != x.device() || !t.is_contiguous())
    refuse(name, ": ", t.sizes(), " ", t.scalar_type(), " on ", t.device(),
           "; wanted a contiguous int32 tensor of at least ", least, " on ", x.device());
}

void* stream_of(PyObject* o) {
  void* s = PyLong_AsVoidPtr(o);
  if (!s && PyErr_Occurred()) throw PythonError();
  return s;
}

int64_t number(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}

int int32(PyObject* o, const char* name) {
  const int64_t v = number(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(name, "=", v);
  return (int)v;
}

void check(int status) {
  if (status == FP4MOE_OK) return;
  PyObject* e = g_error_class ? PyObject_CallFunction(g_error_class, "is", status, fp4moe_last_error()) : nullptr;
  if (e) {
    PyErr_SetObject(g_error_class, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, fp4moe_last_error());
  }
  throw PythonError();
}

// codes [M, K] and scales [M, ceil(K/128)]: the caller's or new ones (the scales of
// one block side by side).
void quantized_out(PyObject* codes_o, PyObject* scales_o, int64_t M, int64_t K, const at::Tensor& x,
                   at::Tensor& codes, at::Tensor& scales) {
  const int64_t blocks = (K + 127) / 128;
  if (codes_o == Py_None) {
    codes = at::empty_strided({M, K}, {K, 1}, x.options().dtype(at::kByte));
  } else {
    codes = tensor(codes_o, "codes");
    if (codes.dim() != 2 || codes.size(0) != M || codes.size(1) != K || !is_codes(codes.scalar_type()) ||
        codes.device() != x.device() || !rows_contiguous(codes))
      bad(codes, "codes", "a uint8 or float8_e4m3fn matrix of the result's shape, rows contiguous");
  }
  if (scales_o == Py_None) {
    scales = at::empty_strided({M, blocks}, {1, M}, x.options().dtype(at::kFloat));
  } else {
    scales = tensor(scales_o, "scales");
    scales_matrix(scales, "scales", M, blocks, x);
  }
}

PyObject* wrap(const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw PythonError();
  return o;
}

// A tensor that goes back to Python: the caller's own object where it was given.
PyObject* give(PyObject* given, const at::Tensor& t) {
  if (given == Py_None) return wrap(t);
  Py_INCREF(given);
  return given;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(want, " arguments are wanted, got ", n);
}

// x, weight, eps, residual, residual_out, y, codes (False: neither codes nor scales),
// scales, stream
PyObject* norm(PyObject* const* a, Py_ssize_t n) {
  count(n, 9);
  const at::Tensor& x = tensor(a[0], "x");
  const int dt = dtype_code(x.scalar_type());
  if (dt < 0) bad(x, "x", "bfloat16, float16 or float32");
  leading(x, "x");
  const int64_t M = x.size(0), K = x.size(1);
  const at::Tensor& w = tensor(a[1], "weight");
  if (w.dim() != 1 || w.size(0) != K || w.scalar_type() != x.scalar_type() || w.device() != x.device() ||
      !rows_contiguous(w))
    bad(w, "weight", "a contiguous vector of x's columns, type and device");
  const double eps = PyFloat_AsDouble(a[2]);
  if (eps == -1.0 && PyErr_Occurred()) throw PythonError();
  fp8block_norm_args p{};
  p.dtype = dt, p.M = (int)M, p.K = (int)K, p.eps = (float)eps;
  p.x = x.data_ptr(), p.ldx = ld(x), p.weight = w.data_ptr();
  at::Tensor res_out, codes, scales;
  if (a[3] != Py_None) {
    const at::Tensor& r = tensor(a[3], "residual");
    same_matrix(r, "residual", x);
    p.residual = r.data_ptr(), p.ldr = ld(r);
    if (a[4] == Py_None) res_out = at::empty_strided({M, K}, {K, 1}, x.options());
  }
  if (a[4] != Py_None) {
    res_out = tensor(a[4], "residual_out");
    same_matrix(res_out, "residual_out", x);
  }
  if (res_out.defined()) p.residual_out = res_out.data_ptr(), p.ldro = ld(res_out);
  if (a[5] != Py_None) {
    const at::Tensor& y = tensor(a[5], "y");
    same_matrix(y, "y", x);
    p.y_out = y.data_ptr(), p.ldy = ld(y);
  }
  if (a[6] != Py_False) {
    quantized_out(a[6], a[7], M, K, x, codes, scales);
    p.codes = static_cast<uint8_t*>(codes.data_ptr()), p.ldc = ld(codes);
    p.scales = static_cast<float*>(scales.data_ptr());
    p.scale_row = scales.stride(0), p.scale_blk = scales.stride(1);
  }
  check(rms_norm_fp8(&p, stream_of(a[8])));
  PyObject* out = PyTuple_New(3);
  if (!out) throw PythonError();
  auto put = [&](int at, PyObject* given, const at::Tensor& t) {
    if (!t.defined()) Py_INCREF(Py_None);
    PyTuple_SET_ITEM(out, at, t.defined() ? give(given, t) : Py_None);
  };
  put(0, a[6], codes);
  put(1, a[7], scales);
  put(2, a[4], res_out);
  return out;
}

// gate_up, row_count, codes, scales, stream
PyObject* swiglu(PyObject* const* a, Py_ssize_t n) {
  count(n, 5);
  const at::Tensor& g = tensor(a[0], "gate_up");
  const int dt = dtype_code(g.scalar_type());
  if (dt < 0) bad(g, "gate_up", "bfloat16, float16 or float32");
  leading(g, "gate_up");
  const int64_t M = g.size(0), I = g.size(1) / 2;
  if (I < 1 || g.size(1) != 2 * I) bad(g, "gate_up", "[M, 2I]");
  const int32_t* rows = nullptr;
  if (a[1] != Py_None) {
    const at::Tensor& r = tensor(a[1], "row_count");
    index_tensor(r, "row_count", 1, g);
    rows = static_cast<const int32_t*>(r.data_ptr());
  }
  at::Tensor codes, scales;
  quantized_out(a[2], a[3], M, I, g, codes, scales);
  check(swiglu_fp8(dt, g.data_ptr(), (int)M, (int)I, ld(g), rows, static_cast<uint8_t*>(codes.data_ptr()),
                   ld(codes), static_cast<float*>(scales.data_ptr()), scales.stride(0),
                   scales.stride(1), stream_of(a[4])));
  PyObject* out = PyTuple_New(2);
  if (!out) throw PythonError();
  PyTuple_SET_ITEM(out, 0, give(a[2], codes));
  PyTuple_SET_ITEM(out, 1, give(a[3], scales));
  return out;
}

// Operands and result of both products: a, a_scale, w, w_scale, out, out_dtype (0 or 1).
at::Tensor operands(PyObject* const* a, int w_dims, int64_t rows, fp8block_gemm_args& g) {
  const at::Tensor& x = tensor(a[0], "a");
  if (!is_codes(x.scalar_type())) bad(x, "a", "uint8 or float8_e4m3fn codes");
  leading(x, "a");
  const int64_t K = x.size(1), blocks = (K + 127) / 128;
  const at::Tensor& sa = tensor(a[1], "a_scale");
  scales_matrix(sa, "a_scale", x.size(0), blocks, x);
  const at::Tensor& w = tensor(a[2], "w");
  if (w.dim() != w_dims || !is_codes(w.scalar_type()) || w.device() != x.device() || w.size(-1) != K ||
      w.size(-2) < 1 || w.size(-2) > INT32_MAX || !rows_contiguous(w))
    bad(w, "w", w_dims == 2 ? "codes [N, K] with a's K, rows contiguous"
                            : "codes [experts, N, K] with a's K, rows contiguous");
  const int64_t N = w.size(-2);
  const at::Tensor& sw = tensor(a[3], "w_scale");
  if (sw.dim() != w_dims || sw.scalar_type() != at::kFloat || sw.device() != x.device() ||
      sw.size(-1) != blocks || sw.size(-2) != (N + 127) / 128 || !rows_contiguous(sw) ||
      (w_dims == 3 && sw.size(0) != w.size(0)))
    bad(sw, "w_scale", "float32 [(experts,) ceil(N/128), ceil(K/128)], rows contiguous");
  at::Tensor out;
  if (a[4] == Py_None) {
    out = at::empty_strided({rows, N}, {N, 1},
                            x.options().dtype(number(a[5]) == FP8BLOCK_F16 ? at::kHalf : at::kBFloat16));
  } else {
    out = tensor(a[4], "out");
    if (out.dim() != 2 || out.size(0) != rows || out.size(1) != N || out.device() != x.device() ||
        (out.scalar_type() != at::kBFloat16 && out.scalar_type() != at::kHalf) || !rows_contiguous(out))
      bad(out, "out", "a bfloat16 or float16 matrix of the result's shape, rows contiguous");
  }
  g.M = (int)rows, g.N = (int)N, g.K = (int)K, g.a_rows = (int)x.size(0);
  g.a = static_cast<const uint8_t*>(x.data_ptr()), g.lda = ld(x);
  g.a_scale = static_cast<const float*>(sa.data_ptr()), g.as_row = sa.stride(0), g.as_blk = sa.stride(1);
  g.w = static_cast<const uint8_t*>(w.data_ptr()), g.ldw = ld(w);
  g.w_scale = static_cast<const float*>(sw.data_ptr()), g.ld_ws = ld(sw);
  g.out_dtype = dtype_code(out.scalar_type()), g.out = out.data_ptr(), g.ldo = ld(out);
  return out;
}

// a, a_scale, w, w_scale, out, out_dtype, stream
PyObject* linear(PyObject* const* a, Py_ssize_t n) {
  count(n, 7);
  fp8block_gemm_args g{};
  const at::Tensor& x = tensor(a[0], "a");
  const at::Tensor out = operands(a, 2, x.dim() ? x.size(0) : 0, g);
  check(fp8_block_linear(&g, stream_of(a[6])));
  return give(a[4], out);
}

// a, a_scale, w, w_scale, out, out_dtype, expert_offsets, sorted_pairs, tiles, n_tiles,
// max_tiles, block_m, a_row_gather, gather_div, stream
PyObject* grouped(PyObject* const* a, Py_ssize_t n) {
  count(n, 15);
  fp8block_gemm_args g{};
  const at::Tensor& pairs = tensor(a[7], "sorted_pairs");
  const int64_t rows = pairs.numel();
  if (rows > INT32_MAX) bad(pairs, "sorted_pairs", "fewer than 2^31 entries");
  const at::Tensor out = operands(a, 3, rows, g);
  const at::Tensor& x = tensor(a[0], "a");
  const at::Tensor& w = tensor(a[2], "w");
  const at::Tensor& sw = tensor(a[3], "w_scale");
  g.max_tiles = int32(a[10], "max_tiles"), g.block_m = int32(a[11], "block_m");
  g.gather_div = int32(a[13], "gather_div");
  const at::Tensor& offsets = tensor(a[6], "expert_offsets");
  const at::Tensor& tiles = tensor(a[8], "tiles");
  const at::Tensor& n_tiles = tensor(a[9], "n_tiles");
  index_tensor(offsets, "expert_offsets", w.size(0) + 1, x);
  index_tensor(tiles, "tiles", 2 * (int64_t)g.max_tiles, x);
  index_tensor(n_tiles, "n_tiles", 1, x);
  if (a[12] != Py_None) {
    const at::Tensor& gather = tensor(a[12], "a_row_gather");
    index_tensor(gather, "a_row_gather", rows, x);
    g.a_row_gather = static_cast<const int32_t*>(gather.data_ptr());
  } else if (x.size(0) < rows) {
    refuse("a has ", x.size(0), " rows for ", rows);
  }
  if (w.size(0) > INT32_MAX) bad(w, "w", "fewer than 2^31 experts");
  g.n_experts = (int)w.size(0);
  if (g.n_experts > 1) g.w_expert = w.stride(0), g.ws_expert = sw.stride(0);
  g.expert_offsets = static_cast<const int32_t*>(offsets.data_ptr());
  g.tiles = static_cast<const int32_t*>(tiles.data_ptr());
  g.n_tiles = static_cast<const int32_t*>(n_tiles.data_ptr());
  check(fp8_block_grouped_gemm(&g, stream_of(a[14])));
  return give(a[4], out);
}

// No C++ exception leaves a Python entry.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return F(args, n);
  } catch (const PythonError&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception&) {
    // as torch does for its own calls: torch.OutOfMemoryError where an output does not fit
    torch::translate_exception_to_python(std::current_exception());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* set_error_class(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error_class);
  g_error_class = cls;
  Py_RETURN_NONE;
}

#define FASTCALL(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(entry<f>)), METH_FASTCALL
PyMethodDef methods[] = {
    {"rms_norm_fp8", FASTCALL(norm), nullptr},
    {"swiglu_fp8", FASTCALL(swiglu), nullptr},
    {"fp8_block_linear", FASTCALL(linear), nullptr},
    {"fp8_block_grouped_gemm", FASTCALL(grouped), nullptr},
    {"set_error_class", set_error_class, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8_block", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8_block() { return PyModule_Create(&module); }
