// Native half of the binding for the calls that run once a decode step (ga_page_plan,
// ga_qk_prologue_axes, ga_kv_quantize_q4, ga_kv_dequantize_q4, ga_attn_verify_q4): the checks of
// their torch tensors, the outputs that the caller did not give, and the call of the C ABI, in one
// step. In Python the same checks and calls took 18 to 25 microseconds of host time, longer than
// the kernels of a small step; here 4 to 9 (12 for the attention on one host).
//
// Every function returns (status, outputs); a tensor that does not belong raises ValueError. Only
// torch's own types are used here; every step of the computation is in libga_attn.so.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/Exception.h>

#include <initializer_list>
#include <sstream>
#include <string>

#include "../../include/ga_attn.h"

namespace {

using at::Tensor;
constexpr auto kBf16 = at::kBFloat16;
constexpr auto kI32 = at::kInt;
constexpr auto kU8 = at::kByte;
constexpr int64_t kHeadsQ = GA_N_Q_HEADS, kHeadsKv = GA_N_KV_HEADS, kDim = GA_HEAD_DIM,
                  kPairs = GA_ROPE_DIMS / 2;

[[noreturn]] void value_error(const std::string& what) { C10_THROW_ERROR(ValueError, what); }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) value_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// The tensors of one call: all on the current device.
struct Call {
  int dev;
  Call(const Tensor& t, const char* name) : dev(t.is_cuda() ? c10::cuda::current_device() : -1) {
    if (dev < 0 || t.get_device() != dev)
      value_error(std::string(name) + " must be a tensor on the current CUDA device");
  }
  [[noreturn]] void refuse(const Tensor& t, const char* name, at::ScalarType type,
                           std::initializer_list<int64_t> shape) const {
    std::ostringstream s;
    s << name << " must be a contiguous " << type << " tensor " << at::IntArrayRef(shape)
      << " on CUDA device " << dev << ", not " << t.scalar_type() << " " << t.sizes() << " on "
      << t.device() << (t.is_contiguous() ? "" : ", not contiguous");
    value_error(s.str());
  }
  // The address of a contiguous tensor of that type and shape; of an empty one, a stand-in that
  // is aligned and never read.
  template <typename T = void>
  T* at(const Tensor& t, const char* name, at::ScalarType type,
        std::initializer_list<int64_t> shape) const {
    if (t.scalar_type() != type || t.sizes() != at::IntArrayRef(shape) || !t.is_cuda() ||
        t.get_device() != dev || !t.is_contiguous())
      refuse(t, name, type, shape);
    void* p = t.data_ptr();
    return static_cast<T*>(p ? p : reinterpret_cast<void*>(256));
  }
  template <typename T = void>
  T* at(PyObject* o, const char* name, at::ScalarType type,
        std::initializer_list<int64_t> shape) const {
    return at<T>(tensor(o, name), name, type, shape);
  }
  // The tensor the caller gave, or a new one.
  Tensor output(PyObject* o, const char* name, at::ScalarType type,
                std::initializer_list<int64_t> shape) const {
    if (o != Py_None) return tensor(o, name);
    return at::empty(at::IntArrayRef(shape),
                     at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)dev)));
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

struct Pools {
  uint8_t *kc, *ks, *vc, *vs;
  int n_pages, page_size;
  Pools(const Call& c, PyObject* const* a) {
    const Tensor& t = tensor(a[0], "k_codes");
    if (t.dim() != 4) value_error("k_codes must be [n_pages, 2, page_size, 128]");
    const int64_t n = t.size(0), page = t.size(2);
    if (n > INT32_MAX || page > INT32_MAX) value_error("k_codes is too large");
    kc = c.at<uint8_t>(t, "k_codes", kU8, {n, kHeadsKv, page, GA_Q4_ROW_BYTES});
    ks = c.at<uint8_t>(a[1], "k_scales", kU8, {n, kHeadsKv, page, GA_Q4_SCALE_BYTES});
    vc = c.at<uint8_t>(a[2], "v_codes", kU8, {n, kHeadsKv, page, GA_Q4_ROW_BYTES});
    vs = c.at<uint8_t>(a[3], "v_scales", kU8, {n, kHeadsKv, page, GA_Q4_SCALE_BYTES});
    n_pages = (int)n;
    page_size = (int)page;
  }
};

int to_int(PyObject* o, const char* name) {
  int overflow = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (overflow || v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " is out of range");
  return (int)v;
}
int extent(int64_t n, const char* name) {
  if (n > INT32_MAX) value_error(std::string(name) + " has too many rows");
  return (int)n;
}

// The C call, its arguments formed before, with the interpreter free for other threads.
template <typename F, typename... A>
int without_gil(F call, A... args) {
  py::gil_scoped_release free;
  return call(args...);
}

PyObject* result(int status, std::initializer_list<Tensor> outputs) {
  PyObject* r = PyTuple_New(1 + (Py_ssize_t)outputs.size());
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
  Py_ssize_t i = 1;
  for (const Tensor& t : outputs) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

void expect(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) value_error("wrong number of arguments");
}

// (seq_len, new_len, page_table, held, free_pages, free_count, page_size, max_tokens, pos_delta,
//  held_out, free_count_out, row_start, slot_map, positions, info)
PyObject* page_plan(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  expect(n_args, 15);
  const Tensor& len = tensor(a[0], "seq_len");
  const Call c(len, "seq_len");
  if (len.dim() != 1) value_error("seq_len must be [n_seq]");
  const int64_t n = len.size(0);
  const Tensor &table = tensor(a[2], "page_table"), &pages = tensor(a[4], "free_pages");
  if (table.dim() != 2 || pages.dim() != 1)
    value_error("page_table must be [n_seq, max_pages] and free_pages [n_free]");
  const int64_t width = table.size(1), n_free = pages.size(0);
  const int page_size = to_int(a[6], "page_size"), max_tokens = to_int(a[7], "max_tokens");
  if (max_tokens < 0) value_error("max_tokens must not be negative");
  const Tensor row_start = c.output(a[11], "row_start", kI32, {n + 1}),
               slots = c.output(a[12], "slot_map", kI32, {max_tokens}),
               positions = c.output(a[13], "positions", kI32, {max_tokens}),
               info = c.output(a[14], "info", kI32, {4});
  int* held = c.at<int>(a[3], "held", kI32, {n});
  int* count = c.at<int>(a[5], "free_count", kI32, {1});
  const int st = without_gil(
      ga_page_plan,
      c.at<int>(len, "seq_len", kI32, {n}), c.at<int>(a[1], "new_len", kI32, {n}), extent(n, "seq_len"),
      page_size, c.at<int>(table, "page_table", kI32, {n, width}), extent(width, "page_table"), held,
      a[9] == Py_None ? held : c.at<int>(a[9], "held_out", kI32, {n}),
      c.at<int>(pages, "free_pages", kI32, {n_free}), extent(n_free, "free_pages"), count,
      a[10] == Py_None ? count : c.at<int>(a[10], "free_count_out", kI32, {1}),
      a[8] == Py_None ? nullptr : c.at<int>(a[8], "pos_delta", kI32, {n}), max_tokens,
      c.at<int>(row_start, "row_start", kI32, {n + 1}), c.at<int>(slots, "slot_map", kI32, {max_tokens}),
      c.at<int>(positions, "positions", kI32, {max_tokens}), c.at<int>(info, "info", kI32, {4}),
      c.stream());
  return result(st, {row_start, slots, positions, info});
  END_HANDLE_TH_ERRORS
}

// (k_raw, w_k, qg, w_q, positions, pair_axis, cos_tab, sin_tab, k_prep, q_prep)
PyObject* qk_prologue_axes(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  expect(n_args, 10);
  const bool has_k = a[0] != Py_None, has_q = a[2] != Py_None;
  if (!has_k && !has_q) value_error("k_raw or qg must be given");
  if ((!has_k && (a[1] != Py_None || a[8] != Py_None)) || (!has_q && (a[3] != Py_None || a[9] != Py_None)))
    value_error("w_k and k_prep come with k_raw, w_q and q_prep with qg");
  const char* first = has_k ? "k_raw" : "qg";
  const Tensor& some = tensor(has_k ? a[0] : a[2], first);
  const Call c(some, first);
  if (some.dim() != 3) value_error("k_raw must be [n_tok, 2, 256] and qg [n_tok, 24, 512]");
  const int64_t n = some.size(0);
  const uint16_t *k = nullptr, *wk = nullptr, *q = nullptr, *wq = nullptr;
  uint16_t *kp = nullptr, *qp = nullptr;
  Tensor k_prep, q_prep;
  if (has_k) {
    k = c.at<uint16_t>(a[0], "k_raw", kBf16, {n, kHeadsKv, kDim});
    wk = c.at<uint16_t>(a[1], "w_k", kBf16, {kDim});
    k_prep = c.output(a[8], "k_prep", kBf16, {n, kHeadsKv, kDim});
    kp = c.at<uint16_t>(k_prep, "k_prep", kBf16, {n, kHeadsKv, kDim});
  }
  if (has_q) {
    q = c.at<uint16_t>(a[2], "qg", kBf16, {n, kHeadsQ, 2 * kDim});
    wq = c.at<uint16_t>(a[3], "w_q", kBf16, {kDim});
    q_prep = c.output(a[9], "q_prep", kBf16, {n, kHeadsQ, kDim});
    qp = c.at<uint16_t>(q_prep, "q_prep", kBf16, {n, kHeadsQ, kDim});
  }
  const Tensor& pos = tensor(a[4], "positions");
  const int64_t dims = pos.dim(), n_axes = dims == 2 ? pos.size(0) : 1, cols = dims ? pos.size(-1) : 0;
  if (dims < 1 || dims > 2 || n_axes < 1 || pos.scalar_type() != kI32 || !pos.is_cuda() ||
      pos.get_device() != c.dev || cols < n || (cols > 1 && pos.stride(-1) != 1))
    value_error("positions must be int32 [n_tok] or [n_axes, >= n_tok] with unit column "
                          "stride, on the current CUDA device");
  uint8_t axes[kPairs] = {};
  if (a[5] != Py_None) {
    THPObjectPtr seq(PySequence_Fast(a[5], "pair_axis must be 32 axis numbers"));
    if (!seq) throw python_error();
    if (PySequence_Fast_GET_SIZE(seq.get()) != kPairs)
      value_error("pair_axis must be 32 axis numbers");
    for (int64_t i = 0; i < kPairs; ++i) {
      const int v = to_int(PySequence_Fast_GET_ITEM(seq.get(), i), "pair_axis");
      if (v < 0 || v > 255) value_error("pair_axis must be 32 axis numbers");
      axes[i] = (uint8_t)v;
    }
  }
  const Tensor& cos = tensor(a[6], "cos_tab");
  if (cos.dim() != 2) value_error("cos_tab must be [table_rows, 32]");
  const int64_t rows = cos.size(0);
  const void* p = pos.data_ptr();
  const int st = without_gil(
      ga_qk_prologue_axes,
      k, wk, kp, q, wq, qp, extent(n, first), static_cast<const int*>(p ? p : reinterpret_cast<void*>(256)),
      n_axes > 1 ? pos.stride(0) : cols, extent(n_axes, "positions"), axes,
      c.at<uint16_t>(cos, "cos_tab", kBf16, {rows, kPairs}),
      c.at<uint16_t>(a[7], "sin_tab", kBf16, {rows, kPairs}), extent(rows, "cos_tab"), c.stream());
  return result(st, {k_prep, q_prep});
  END_HANDLE_TH_ERRORS
}

// bf16 rows [n_tok, 2, 256], heads and dims dense; the token stride may be larger.
const uint16_t* kv_rows(const Call& c, PyObject* o, const char* name, int64_t n, int64_t& ld) {
  const Tensor& x = tensor(o, name);
  if (x.scalar_type() != kBf16 || x.sizes() != at::IntArrayRef({n, kHeadsKv, kDim}) || !x.is_cuda() ||
      x.get_device() != c.dev || x.stride(2) != 1 || x.stride(1) != kDim)
    value_error(std::string(name) + " must be bfloat16 [n_tok, 2, 256] with dense heads and "
                          "dims on the current CUDA device, k and v of the same tokens");
  ld = n > 1 ? x.stride(0) : kHeadsKv * kDim;
  void* p = x.data_ptr();
  return static_cast<const uint16_t*>(p ? p : reinterpret_cast<void*>(256));
}

// (k, v, k_codes, k_scales, v_codes, v_scales, slots)
PyObject* kv_quantize_q4(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  expect(n_args, 7);
  const Tensor& k = tensor(a[0], "k");
  const Call c(k, "k");
  if (k.dim() != 3) value_error("k must be [n_tok, 2, 256]");
  const int64_t n = k.size(0);
  const Pools p(c, a + 2);
  int64_t ld_k, ld_v;
  const uint16_t *k_at = kv_rows(c, a[0], "k", n, ld_k), *v_at = kv_rows(c, a[1], "v", n, ld_v);
  const int st = without_gil(
      ga_kv_quantize_q4, k_at, ld_k, v_at, ld_v, n,
                                   a[6] == Py_None ? nullptr : c.at<int>(a[6], "slots", kI32, {n}),
                                   p.kc, p.ks, p.vc, p.vs, p.n_pages, p.page_size, c.stream());
  return result(st, {});
  END_HANDLE_TH_ERRORS
}

// (k_codes, k_scales, v_codes, v_scales, slots, n_tok, k_out, v_out)
PyObject* kv_dequantize_q4(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  expect(n_args, 8);
  const Call c(tensor(a[0], "k_codes"), "k_codes");
  const Pools p(c, a);
  int64_t n = (int64_t)p.n_pages * p.page_size;
  const int* slots = nullptr;
  if (a[4] != Py_None) {
    const Tensor& s = tensor(a[4], "slots");
    if (s.dim() != 1) value_error("slots must be [n_tok]");
    n = s.size(0);
    slots = c.at<int>(s, "slots", kI32, {n});
    if (a[5] != Py_None && to_int(a[5], "n_tok") != n) value_error("slots must be [n_tok]");
  } else if (a[5] != Py_None) {
    n = to_int(a[5], "n_tok");
    if (n < 0) value_error("n_tok must not be negative");
  }
  const Tensor k_out = c.output(a[6], "k_out", kBf16, {n, kHeadsKv, kDim}),
               v_out = c.output(a[7], "v_out", kBf16, {n, kHeadsKv, kDim});
  const int st = without_gil(
      ga_kv_dequantize_q4, p.kc, p.ks, p.vc, p.vs, p.n_pages, p.page_size, slots, n,
                                     c.at<uint16_t>(k_out, "k_out", kBf16, {n, kHeadsKv, kDim}),
                                     c.at<uint16_t>(v_out, "v_out", kBf16, {n, kHeadsKv, kDim}),
                                     c.stream());
  return result(st, {k_out, v_out});
  END_HANDLE_TH_ERRORS
}

// (q_prep, qg, k_codes, k_scales, v_codes, v_scales, page_table, seq_len, out, workspace)
PyObject* attn_verify_q4(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  HANDLE_TH_ERRORS
  expect(n_args, 10);
  const Tensor& q = tensor(a[0], "q_prep");
  const Call c(q, "q_prep");
  if (q.dim() != 4) value_error("q_prep must be [n_seq, rows, 24, 256]");
  const int64_t n = q.size(0), rows = q.size(1);
  const Pools p(c, a + 2);
  const Tensor& table = tensor(a[6], "page_table");
  if (table.dim() != 2) value_error("page_table must be [n_seq, max_pages]");
  const int64_t width = table.size(1);
  const Tensor out = c.output(a[8], "out", kBf16, {n, rows, kHeadsQ * kDim});
  const Tensor ws = c.output(a[9], "workspace", kU8, {(int64_t)ga_verify_q4_workspace_bytes()});
  if (!ws.is_cuda() || ws.get_device() != c.dev || !ws.is_contiguous())
    value_error("workspace must be a contiguous tensor on the current CUDA device");
  const int st = without_gil(
      ga_attn_verify_q4,
      c.at<uint16_t>(q, "q_prep", kBf16, {n, rows, kHeadsQ, kDim}),
      c.at<uint16_t>(a[1], "qg", kBf16, {n, rows, kHeadsQ, 2 * kDim}), p.kc, p.ks, p.vc, p.vs, p.n_pages,
      p.page_size, c.at<int>(table, "page_table", kI32, {n, width}), extent(width, "page_table"),
      c.at<int>(a[7], "seq_len", kI32, {n}), extent(n, "q_prep"), extent(rows, "q_prep"),
      c.at<uint16_t>(out, "out", kBf16, {n, rows, kHeadsQ * kDim}), ws.data_ptr(), ws.nbytes(),
      c.stream());
  return result(st, {out});
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"page_plan", (PyCFunction)(void*)page_plan, METH_FASTCALL, nullptr},
    {"qk_prologue_axes", (PyCFunction)(void*)qk_prologue_axes, METH_FASTCALL, nullptr},
    {"kv_quantize_q4", (PyCFunction)(void*)kv_quantize_q4, METH_FASTCALL, nullptr},
    {"kv_dequantize_q4", (PyCFunction)(void*)kv_dequantize_q4, METH_FASTCALL, nullptr},
    {"attn_verify_q4", (PyCFunction)(void*)attn_verify_q4, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&kModule); }
