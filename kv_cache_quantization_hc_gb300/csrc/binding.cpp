// Python binding of the serving calls: torch tensors to the C ABI of
// include/hc.h, checked and marshalled in C++.
//
// A decoding step makes these calls once per layer with little work in each:
// marshalling 20 arguments through ctypes took 25 to 35 us a call on the
// GPU's host core, more than the kernels of a small step, and takes 3 to 5
// here.  The functions below take their arguments by position, in the order
// of their wrappers in serve.py.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <stdexcept>
#include <string>

#include "hc.h"

namespace {

// A Python exception already set, or one to set from a message.
struct PythonError {};
struct BadArgument : std::runtime_error {
  using std::runtime_error::runtime_error;
};

const char* type_name(at::ScalarType s) { return c10::toString(s); }

// The tensors of a call, all on one GPU: the kernel that the call launches
// there dereferences them all.
struct Tensors {
  const at::Tensor* first = nullptr;

  const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw BadArgument(std::string(name) + " must be a torch tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) throw BadArgument(std::string(name) + " must be a CUDA tensor");
    if (!first) first = &t;
    if (t.device() != first->device())
      throw BadArgument(std::string(name) + " is on " + t.device().str() + ", other tensors of the call on " +
                        first->device().str());
    return t;
  }
  // None: null
  const at::Tensor* given(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

  // A contiguous tensor of `dtype` with at least `numel` elements.
  const at::Tensor& buffer(PyObject* o, const char* name, at::ScalarType dtype, int64_t numel = 0) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != dtype)
      throw BadArgument(std::string(name) + " must be " + type_name(dtype) + ", not " + type_name(t.scalar_type()));
    if (!t.is_contiguous()) throw BadArgument(std::string(name) + " must be contiguous");
    if (t.numel() < numel)
      throw BadArgument(std::string(name) + " has " + std::to_string(t.numel()) + " elements; the call addresses " +
                        std::to_string(numel));
    return t;
  }
};

template <typename T>
T* data(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

int dtype_of(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return HC_F32;
    case at::kHalf: return HC_F16;
    case at::kBFloat16: return HC_BF16;
    default:
      throw BadArgument(std::string(name) + " must be float32, float16 or bfloat16, not " +
                        type_name(t.scalar_type()));
  }
}

// hc_rows of [n, heads, d] (-1: any) with adjacent channels.
hc_rows rows(const at::Tensor& t, const char* name, int64_t n, int64_t heads, int64_t d,
             at::ScalarType dtype) {
  if (t.dim() != 3 || (n >= 0 && t.size(0) != n) || (heads >= 0 && t.size(1) != heads) || (d >= 0 && t.size(2) != d))
    throw BadArgument(std::string(name) + " must be [n_tokens" + (n >= 0 ? "=" + std::to_string(n) : "") + ", heads" +
                      (heads >= 0 ? "=" + std::to_string(heads) : "") + ", channels" +
                      (d >= 0 ? "=" + std::to_string(d) : "") + "], not " + c10::str(t.sizes()));
  if (t.scalar_type() != dtype)
    throw BadArgument(std::string(name) + " must be " + type_name(dtype) + ", not " + type_name(t.scalar_type()));
  if (t.numel() == 0) return hc_rows{t.data_ptr(), 0, 0};  // whose strides may be anything
  if (t.stride(2) != 1 && t.size(2) != 1) throw BadArgument(std::string("the channels of ") + name + " must be adjacent");
  return hc_rows{t.data_ptr(), t.stride(0), t.stride(1)};
}

int32_t i32(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) throw BadArgument(std::string(name) + " does not fit 32 bits");
  return static_cast<int32_t>(v);
}
int32_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return i32(v, name);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v != 0;
}
bool none(PyObject* o) { return o == Py_None; }

// The tensors' device made current for the call, and the stream: None for
// torch's current one, an integer cudaStream_t, or a torch.cuda.Stream.  What
// the call allocates, it allocates on that stream: a block of another stream
// may still be in use by work queued there.
struct Where {
  c10::cuda::CUDAGuard guard;
  cudaStream_t stream;
  c10::cuda::OptionalCUDAStreamGuard on_stream;
  Where(const at::Tensor& t, PyObject* s) : guard(t.device()) {
    if (none(s)) {
      stream = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
      return;
    }
    PyObject* handle = PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttrString(s, "cuda_stream");
    if (!handle) throw PythonError{};
    stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
    Py_DECREF(handle);
    if (PyErr_Occurred()) throw PythonError{};
    if (stream == cudaStreamPerThread) return;  // see empty
    // cudaStreamLegacy is another name of the default stream
    on_stream.reset_stream(c10::cuda::getStreamFromExternal(stream == cudaStreamLegacy ? nullptr : stream,
                                                            t.device().index()));
  }
};

at::Tensor empty(at::IntArrayRef size, at::ScalarType dtype, const at::Tensor& like, const Where& w) {
  // one handle for as many streams as there are host threads: the allocator cannot tell them apart
  if (w.stream == cudaStreamPerThread) throw BadArgument("on cudaStreamPerThread the output tensors have to be given");
  return at::Tensor(at::detail::empty_cuda(size, dtype, like.device(), std::nullopt));
}

hc_int4_cache cache_desc(const at::Tensor& codes, const at::Tensor& scales) {
  if (codes.dim() != 5 || scales.dim() != 5 || codes.size(1) != 2 || codes.size(0) != scales.size(0) ||
      scales.size(1) != 2 || codes.size(2) != scales.size(2) || codes.size(3) != scales.size(3))
    throw BadArgument("codes must be [num_slots, 2, H, B, d/2] and scales [num_slots, 2, H, B, d/group]");
  const int64_t d = 2 * codes.size(4), groups = scales.size(4);
  if (groups < 1 || d % groups)
    throw BadArgument("scales hold " + std::to_string(groups) + " groups per row of " + std::to_string(d) + " channels");
  if (scales.scalar_type() != at::kHalf && scales.scalar_type() != at::kFloat)
    throw BadArgument(std::string("scales must be float16 or float32, not ") + type_name(scales.scalar_type()));
  if (!scales.is_contiguous()) throw BadArgument("scales must be contiguous");
  return hc_int4_cache{i32(codes.size(2), "H"),         i32(d, "d"),
                       i32(codes.size(3), "B"),         i32(codes.size(0), "num_slots"),
                       i32(d / groups, "group"),        dtype_of(scales, "scales")};
}

// One layer's pages [num_slots, B, H, d], each slot's rows adjacent.
hc_paged_desc pages_desc(const at::Tensor& k, const at::Tensor& v) {
  if (k.dim() != 4 || v.sizes() != k.sizes()) throw BadArgument("k_pages and v_pages must both be [num_slots, B, H, d]");
  if (v.scalar_type() != k.scalar_type())
    throw BadArgument(std::string("v_pages must be ") + type_name(k.scalar_type()) + ", not " + type_name(v.scalar_type()));
  const int64_t S = k.size(0), B = k.size(1), H = k.size(2), d = k.size(3);
  for (const at::Tensor* t : {&k, &v})
    if ((d > 1 && t->stride(3) != 1) || (H > 1 && t->stride(2) != d) || (B > 1 && t->stride(1) != H * d))
      throw BadArgument("each slot of k_pages and v_pages must be a contiguous [B, H, d] block");
  if (S > 1 && v.stride(0) != k.stride(0)) throw BadArgument("k_pages and v_pages must have the same strides");
  return hc_paged_desc{1, i32(H, "H"), i32(d, "d"), i32(B, "B"), i32(S, "num_slots"), dtype_of(k, "k_pages"),
                       S > 1 ? k.stride(0) : B * H * d, 0};
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}

// Block tables [n_req, width], each row adjacent.
int64_t table_stride(const at::Tensor& t, int64_t n_req) {
  if (t.dim() != 2 || t.size(0) != n_req || t.scalar_type() != at::kInt || (t.size(1) > 1 && t.stride(1) != 1))
    throw BadArgument("block_tables must be int32 [" + std::to_string(n_req) + ", width], each row adjacent");
  return n_req > 1 ? t.stride(0) : t.size(1);
}

hc_rope_axes_desc rope_desc(Tensors& in, PyObject* positions, PyObject* table, PyObject* pair_axis, PyObject* pairing,
                            bool inverse, int64_t n) {
  hc_rope_axes_desc r;
  std::memset(&r, 0, sizeof r);
  const at::Tensor& pos = in.tensor(positions, "positions");
  const bool flat = pos.dim() == 1;
  if (pos.scalar_type() != at::kInt || (!flat && pos.dim() != 2) || pos.size(-1) != n || (n > 1 && pos.stride(-1) != 1))
    throw BadArgument("positions must be int32 [n_axes, " + std::to_string(n) + "], each axis adjacent");
  r.positions = data<int32_t>(pos);
  r.n_axes = flat ? 1 : i32(pos.size(0), "n_axes");
  r.position_stride = r.n_axes > 1 ? pos.stride(0) : 0;
  PyObject* seq = PySequence_Fast(pair_axis, "pair_axis must be a sequence");
  if (!seq) throw PythonError{};
  const Py_ssize_t half = PySequence_Fast_GET_SIZE(seq);
  bool ok = half >= 1 && half <= 128;
  for (Py_ssize_t i = 0; ok && i < half; ++i) {
    const long a = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
    ok = a >= 0 && a < r.n_axes;
    r.pair_axis[i] = static_cast<uint8_t>(a);
  }
  Py_DECREF(seq);
  if (PyErr_Occurred()) throw PythonError{};
  if (!ok) throw BadArgument("pair_axis holds the axis (below " + std::to_string(r.n_axes) + ") of each of 1 to 128 pairs");
  const at::Tensor& tab = in.buffer(table, "table", at::kFloat);
  if (tab.dim() != 3 || tab.size(1) != half || tab.size(2) != 2)
    throw BadArgument("table must be [n_positions, " + std::to_string(half) + ", 2]");
  r.table = data<float>(tab);
  r.n_positions = i32(tab.size(0), "n_positions");
  r.rot_dim = static_cast<int32_t>(2 * half);
  const char* name = PyUnicode_Check(pairing) ? PyUnicode_AsUTF8(pairing) : nullptr;
  if (PyErr_Occurred()) throw PythonError{};
  if (name && !std::strcmp(name, "half_split"))
    r.pairing = HC_PAIR_HALF_SPLIT;
  else if (name && !std::strcmp(name, "interleaved"))
    r.pairing = HC_PAIR_INTERLEAVED;
  else
    throw BadArgument("pairing must be 'half_split' or 'interleaved'");
  r.inverse = inverse;
  return r;
}

// A status other than HC_OK becomes hc.HCError.
void check(const char* fn, int status) {
  if (status == HC_OK) return;
  PyObject* m = PyImport_ImportModule("kv_cache_quantization_hc_gb300.hc");
  if (m) {
    PyObject* r = PyObject_CallMethod(m, "_check", "si", fn, status);
    Py_XDECREF(r);
    Py_DECREF(m);
  }
  if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s returned %s", fn, hc_status_string(status));
  throw PythonError{};
}

PyTypeObject* step_tables_type = nullptr;

PyObject* build_block_tables(PyObject* const* a) {
  // cached_lens, new_lens, free_slots, block_tables, block_size, n_tokens, err, out, stream
  Tensors in;
  const at::Tensor& cached = in.buffer(a[0], "cached_lens", at::kInt);
  const int64_t n_req = cached.numel();
  const at::Tensor& fresh = in.buffer(a[1], "new_lens", at::kInt);
  if (fresh.numel() != n_req) throw BadArgument("new_lens must hold as many requests as cached_lens");
  const at::Tensor& free_slots = in.buffer(a[2], "free_slots", at::kInt);
  const at::Tensor& table = in.tensor(a[3], "block_tables");
  const int64_t stride = table_stride(table, n_req);
  const int32_t n_tokens = integer(a[5], "n_tokens");
  if (n_tokens < 0) throw BadArgument("n_tokens must not be negative");
  const at::Tensor& err = in.buffer(a[6], "err", at::kInt, 1);
  const int64_t sizes[6] = {n_req + 1, n_req, n_tokens, n_tokens, n_tokens, 1};
  static const char* const names[6] = {"q_starts", "kv_lens", "token_req", "token_pos", "token_rows", "n_taken"};
  const bool makes = none(a[7]);
  if (!makes && Py_TYPE(a[7]) != step_tables_type) throw BadArgument("out must be a StepTables");
  auto output = [&](PyObject* step, int i) {
    return in.buffer(PyStructSequence_GetItem(step, i), names[i], i == 4 ? at::kLong : at::kInt, sizes[i]).data_ptr();
  };
  for (int i = 0; !makes && i < 6; ++i) output(a[7], i);
  const Where w(cached, a[8]);
  PyObject* result = makes ? PyStructSequence_New(step_tables_type) : Py_NewRef(a[7]);
  if (!result) throw PythonError{};
  try {
    for (int i = 0; makes && i < 6; ++i) {
      PyObject* t = THPVariable_Wrap(empty({sizes[i]}, i == 4 ? at::kLong : at::kInt, cached, w));
      if (!t) throw PythonError{};
      PyStructSequence_SetItem(result, i, t);
    }
    void* p[6];
    for (int i = 0; i < 6; ++i) p[i] = output(result, i);
    check("hc_build_block_tables",
          hc_build_block_tables(data<int32_t>(cached), data<int32_t>(fresh), i32(n_req, "n_req"),
                                integer(a[4], "block_size"), data<int32_t>(free_slots),
                                i32(free_slots.numel(), "n_free"), data<int32_t>(table), stride,
                                i32(table.size(1), "width"), n_tokens, static_cast<int32_t*>(p[0]),
                                static_cast<int32_t*>(p[1]), static_cast<int32_t*>(p[2]),
                                static_cast<int32_t*>(p[3]), static_cast<int64_t*>(p[4]),
                                static_cast<int32_t*>(p[5]), data<int32_t>(err), w.stream));
  } catch (...) {
    Py_DECREF(result);
    throw;
  }
  return result;
}

PyObject* rope_axes(PyObject* const* a) {
  // x, positions, table, pair_axis, err, pairing, inverse, out, stream
  Tensors in;
  const at::Tensor& x = in.tensor(a[0], "x");
  const int dtype = dtype_of(x, "x");
  const hc_rows xr = rows(x, "x", -1, -1, -1, x.scalar_type());
  const int64_t n = x.size(0), heads = x.size(1), d = x.size(2);
  const hc_rope_axes_desc rope = rope_desc(in, a[1], a[2], a[3], a[5], truth(a[6]), n);
  const at::Tensor& err = in.buffer(a[4], "err", at::kInt, 1);
  const at::Tensor* out = in.given(a[7], "out");
  const Where w(x, a[8]);
  const at::Tensor y = out ? *out : empty({n, heads, d}, x.scalar_type(), x, w);
  const hc_rows yr = rows(y, "out", n, heads, d, x.scalar_type());
  check("hc_rope_axes", hc_rope_axes(&xr, &yr, dtype, i32(n, "n_tokens"), i32(heads, "n_heads"), i32(d, "d"), &rope,
                                     data<int32_t>(err), w.stream));
  return none(a[7]) ? THPVariable_Wrap(y) : Py_NewRef(a[7]);
}

PyObject* append_int4(PyObject* const* a) {
  // q, k, v, token_rows, codes, scales, positions, table, pair_axis, err, pairing, q_out, stream, wire_scales
  Tensors in;
  const at::Tensor& codes = in.buffer(a[4], "codes", at::kByte);
  const at::Tensor& scales = in.tensor(a[5], "scales");
  const hc_int4_cache cache = cache_desc(codes, scales);
  const at::Tensor& k = in.tensor(a[1], "k");
  const int dtype = dtype_of(k, "k");
  const at::ScalarType st = k.scalar_type();
  const hc_rows kr = rows(k, "k", -1, cache.n_kv_heads, cache.d_head, st);
  const int64_t n = k.size(0);
  const hc_rows vr = rows(in.tensor(a[2], "v"), "v", n, cache.n_kv_heads, cache.d_head, st);
  const at::Tensor& token_rows = in.buffer(a[3], "token_rows", at::kLong, n);
  const at::Tensor& err = in.buffer(a[9], "err", at::kInt, 1);
  hc_rope_axes_desc rope;
  const bool turns = !none(a[7]);
  if (turns) rope = rope_desc(in, a[6], a[7], a[8], a[10], false, n);
  const at::Tensor* q = in.given(a[0], "q");
  const at::Tensor* q_out = q ? in.given(a[11], "q_out") : nullptr;
  const Where w(k, a[12]);
  hc_rows qr{}, qo{};
  int64_t heads = 0;
  at::Tensor out;
  const bool has_q = q != nullptr;
  if (has_q) {
    qr = rows(*q, "q", n, -1, cache.d_head, st);
    heads = q->size(1);
    out = q_out ? *q_out : empty({n, heads, cache.d_head}, st, k, w);
    qo = rows(out, "q_out", n, heads, cache.d_head, st);
  }
  const bool wire = truth(a[13]);
  const auto append = wire ? hc_append_int4_wire : hc_append_int4;
  check(wire ? "hc_append_int4_wire" : "hc_append_int4",
        append(has_q ? &qr : nullptr, &kr, &vr, dtype, i32(n, "n_tokens"), i32(heads, "heads"), turns ? &rope : nullptr,
               data<int64_t>(token_rows), &cache, data<uint8_t>(codes), scales.data_ptr(), has_q ? &qo : nullptr,
               data<int32_t>(err), w.stream));
  if (!has_q) Py_RETURN_NONE;
  return none(a[11]) ? THPVariable_Wrap(out) : Py_NewRef(a[11]);
}

PyObject* attend_int4(PyObject* const* a) {
  // q, codes, scales, block_tables, q_starts, kv_lens, max_new, workspace, err, causal, window, softmax_scale,
  // out, lse, return_lse, stream
  Tensors in;
  const at::Tensor& codes = in.buffer(a[1], "codes", at::kByte);
  const at::Tensor& scales = in.tensor(a[2], "scales");
  const hc_int4_cache cache = cache_desc(codes, scales);
  const at::Tensor& q = in.tensor(a[0], "q");
  const int dtype = dtype_of(q, "q");
  const hc_rows qr = rows(q, "q", -1, -1, cache.d_head, q.scalar_type());
  const int64_t n = q.size(0), heads = q.size(1);
  const at::Tensor& kv = in.buffer(a[5], "kv_lens", at::kInt);
  const int64_t n_req = kv.numel();
  const at::Tensor& table = in.tensor(a[3], "block_tables");
  const int64_t stride = table_stride(table, n_req);
  const at::Tensor& starts = in.buffer(a[4], "q_starts", at::kInt, n_req + 1);
  const at::Tensor& workspace = in.buffer(a[7], "workspace", at::kByte);
  const at::Tensor& err = in.buffer(a[8], "err", at::kInt, 1);
  double scale = 1.0 / std::sqrt(static_cast<double>(cache.d_head));
  if (!none(a[11])) {
    scale = PyFloat_AsDouble(a[11]);
    if (scale == -1.0 && PyErr_Occurred()) throw PythonError{};
  }
  const at::Tensor* out_given = in.given(a[12], "out");
  const at::Tensor* lse_given = none(a[13]) ? nullptr : &in.buffer(a[13], "lse", at::kFloat, n * heads);
  const Where w(q, a[15]);
  const at::Tensor y = out_given ? *out_given : empty({n, heads, cache.d_head}, q.scalar_type(), q, w);
  const hc_rows yr = rows(y, "out", n, heads, cache.d_head, q.scalar_type());
  const bool with_lse = truth(a[14]);
  at::Tensor lse;
  if (lse_given)
    lse = *lse_given;
  else if (with_lse)
    lse = empty({n, heads}, at::kFloat, q, w);
  check("hc_attend_int4",
        hc_attend_int4(&qr, &yr, lse.defined() ? data<float>(lse) : nullptr, dtype, i32(n, "n_tokens"),
                       i32(heads, "heads"), &cache, data<uint8_t>(codes), scales.data_ptr(), data<int32_t>(table),
                       stride, i32(table.size(1), "width"), data<int32_t>(starts), data<int32_t>(kv),
                       i32(n_req, "n_req"), integer(a[6], "max_new"), truth(a[9]), integer(a[10], "window"),
                       static_cast<float>(scale), workspace.data_ptr(), workspace.numel(), data<int32_t>(err),
                       w.stream));
  PyObject* out = none(a[12]) ? THPVariable_Wrap(y) : Py_NewRef(a[12]);
  if (!with_lse) return out;
  PyObject* l = none(a[13]) ? THPVariable_Wrap(lse) : Py_NewRef(a[13]);
  PyObject* both = out && l ? PyTuple_Pack(2, out, l) : nullptr;
  Py_XDECREF(out);
  Py_XDECREF(l);
  return both;
}

PyObject* append_paged(PyObject* const* a) {
  // q, k, v, token_rows, k_pages, v_pages, positions, table, pair_axis, err, pairing, q_out, stream
  Tensors in;
  const at::Tensor& k_pages = in.tensor(a[4], "k_pages");
  const at::Tensor& v_pages = in.tensor(a[5], "v_pages");
  const hc_paged_desc desc = pages_desc(k_pages, v_pages);
  const at::ScalarType st = k_pages.scalar_type();
  const at::Tensor& k = in.tensor(a[1], "k");
  const hc_rows kr = rows(k, "k", -1, desc.n_kv_heads, desc.d_head, st);
  const int64_t n = k.size(0);
  const hc_rows vr = rows(in.tensor(a[2], "v"), "v", n, desc.n_kv_heads, desc.d_head, st);
  const at::Tensor& token_rows = in.buffer(a[3], "token_rows", at::kLong, n);
  const at::Tensor& err = in.buffer(a[9], "err", at::kInt, 1);
  hc_rope_axes_desc rope;
  const bool turns = !none(a[7]);
  if (turns) rope = rope_desc(in, a[6], a[7], a[8], a[10], false, n);
  const at::Tensor* q = in.given(a[0], "q");
  const at::Tensor* q_out = q ? in.given(a[11], "q_out") : nullptr;
  const Where w(k, a[12]);
  hc_rows qr{}, qo{};
  int64_t heads = 0;
  at::Tensor out;
  if (q) {
    qr = rows(*q, "q", n, -1, desc.d_head, st);
    heads = q->size(1);
    out = q_out ? *q_out : empty({n, heads, desc.d_head}, st, k, w);
    qo = rows(out, "q_out", n, heads, desc.d_head, st);
  }
  check("hc_append_paged",
        hc_append_paged(q ? &qr : nullptr, &kr, &vr, i32(n, "n_tokens"), i32(heads, "heads"), turns ? &rope : nullptr,
                        data<int64_t>(token_rows), &desc, k_pages.data_ptr(), v_pages.data_ptr(), q ? &qo : nullptr,
                        data<int32_t>(err), w.stream));
  if (!q) Py_RETURN_NONE;
  return none(a[11]) ? THPVariable_Wrap(out) : Py_NewRef(a[11]);
}

PyObject* attend_paged(PyObject* const* a) {
  // q, k_pages, v_pages, block_tables, q_starts, kv_lens, max_new, workspace, err, causal, window, softmax_scale,
  // softcap, slopes, positions, prefix_lens, out, lse, return_lse, stream
  Tensors in;
  const at::Tensor& k_pages = in.tensor(a[1], "k_pages");
  const at::Tensor& v_pages = in.tensor(a[2], "v_pages");
  const hc_paged_desc desc = pages_desc(k_pages, v_pages);
  if (desc.dtype == HC_F32) throw BadArgument("attend_paged takes pages of float16 or bfloat16, not of Float as append_paged does");
  const at::Tensor& q = in.tensor(a[0], "q");
  const hc_rows qr = rows(q, "q", -1, -1, desc.d_head, k_pages.scalar_type());
  const int64_t n = q.size(0), heads = q.size(1);
  const at::Tensor& kv = in.buffer(a[5], "kv_lens", at::kInt);
  const int64_t n_req = kv.numel();
  const at::Tensor& table = in.tensor(a[3], "block_tables");
  const int64_t stride = table_stride(table, n_req);
  const at::Tensor& starts = in.buffer(a[4], "q_starts", at::kInt, n_req + 1);
  const at::Tensor& workspace = in.buffer(a[7], "workspace", at::kByte);
  const at::Tensor& err = in.buffer(a[8], "err", at::kInt, 1);
  hc_attend_scores scores;
  std::memset(&scores, 0, sizeof scores);
  scores.causal = truth(a[9]);
  scores.window = integer(a[10], "window");
  scores.softmax_scale = static_cast<float>(none(a[11]) ? 1.0 / std::sqrt(static_cast<double>(desc.d_head)) : number(a[11]));
  scores.softcap = static_cast<float>(number(a[12]));
  if (!none(a[13])) scores.slopes = data<float>(in.buffer(a[13], "slopes", at::kFloat, heads));
  if (!none(a[14])) scores.positions = data<int32_t>(in.buffer(a[14], "positions", at::kInt, n));
  if (!none(a[15])) scores.prefix_lens = data<int32_t>(in.buffer(a[15], "prefix_lens", at::kInt, n_req));
  const at::Tensor* out_given = in.given(a[16], "out");
  const at::Tensor* lse_given = none(a[17]) ? nullptr : &in.buffer(a[17], "lse", at::kFloat, n * heads);
  const Where w(q, a[19]);
  const at::Tensor y = out_given ? *out_given : empty({n, heads, desc.d_head}, q.scalar_type(), q, w);
  const hc_rows yr = rows(y, "out", n, heads, desc.d_head, q.scalar_type());
  const bool with_lse = truth(a[18]);
  at::Tensor lse;
  if (lse_given)
    lse = *lse_given;
  else if (with_lse)
    lse = empty({n, heads}, at::kFloat, q, w);
  check("hc_attend_paged",
        hc_attend_paged(&qr, &yr, lse.defined() ? data<float>(lse) : nullptr, i32(n, "n_tokens"), i32(heads, "heads"),
                        &desc, k_pages.data_ptr(), v_pages.data_ptr(), data<int32_t>(table), stride,
                        i32(table.size(1), "width"), data<int32_t>(starts), data<int32_t>(kv), i32(n_req, "n_req"),
                        integer(a[6], "max_new"), &scores, workspace.data_ptr(), workspace.numel(), data<int32_t>(err),
                        w.stream));
  PyObject* out = none(a[16]) ? THPVariable_Wrap(y) : Py_NewRef(a[16]);
  if (!with_lse) return out;
  PyObject* l = none(a[17]) ? THPVariable_Wrap(lse) : Py_NewRef(a[17]);
  PyObject* both = out && l ? PyTuple_Pack(2, out, l) : nullptr;
  Py_XDECREF(out);
  Py_XDECREF(l);
  return both;
}

PyObject* merge_attention(PyObject* const* a) {
  // out_a, lse_a, out_b, lse_b, out, lse, stream
  Tensors in;
  const at::Tensor& x = in.tensor(a[0], "out_a");
  const int dtype = dtype_of(x, "out_a");
  const hc_rows xr = rows(x, "out_a", -1, -1, -1, x.scalar_type());
  const int64_t n = x.size(0), heads = x.size(1), d = x.size(2);
  const at::Tensor& lse_a = in.buffer(a[1], "lse_a", at::kFloat, n * heads);
  const hc_rows yr = rows(in.tensor(a[2], "out_b"), "out_b", n, heads, d, x.scalar_type());
  const at::Tensor& lse_b = in.buffer(a[3], "lse_b", at::kFloat, n * heads);
  const at::Tensor* out_given = in.given(a[4], "out");
  const at::Tensor* lse_given = none(a[5]) ? nullptr : &in.buffer(a[5], "lse", at::kFloat, n * heads);
  const Where w(x, a[6]);
  const at::Tensor out = out_given ? *out_given : empty({n, heads, d}, x.scalar_type(), x, w);
  const hc_rows zr = rows(out, "out", n, heads, d, x.scalar_type());
  const at::Tensor lse = lse_given ? *lse_given : empty({n, heads}, at::kFloat, x, w);
  check("hc_merge_attention",
        hc_merge_attention(&xr, data<float>(lse_a), &yr, data<float>(lse_b), &zr, data<float>(lse), dtype,
                           i32(n, "n_tokens"), i32(heads, "heads"), i32(d, "d"), w.stream));
  PyObject* o = none(a[4]) ? THPVariable_Wrap(out) : Py_NewRef(a[4]);
  PyObject* l = none(a[5]) ? THPVariable_Wrap(lse) : Py_NewRef(a[5]);
  PyObject* both = o && l ? PyTuple_Pack(2, o, l) : nullptr;
  Py_XDECREF(o);
  Py_XDECREF(l);
  return both;
}

// No C++ exception leaves a call.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PythonError&) {
  } catch (const BadArgument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown error");
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<build_block_tables, 9>("build_block_tables"), method<rope_axes, 9>("rope_axes"),
                         method<append_int4, 14>("append_int4"), method<attend_int4, 16>("attend_int4"),
                         method<append_paged, 13>("append_paged"), method<attend_paged, 20>("attend_paged"),
                         method<merge_attention, 7>("merge_attention"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve", "Native binding of the serving calls (see serve.py).", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

PyStructSequence_Field step_fields[] = {{"q_starts", "int32 [n_req + 1]: first new token of each request"},
                                        {"kv_lens", "int32 [n_req]: cached and new tokens"},
                                        {"token_req", "int32 [n_tokens]: request of each new token"},
                                        {"token_pos", "int32 [n_tokens]: its position"},
                                        {"token_rows", "int64 [n_tokens]: its cache row"},
                                        {"n_taken", "int32 [1]: free slots that were taken"},
                                        {nullptr, nullptr}};
PyStructSequence_Desc step_desc = {"kv_cache_quantization_hc_gb300.serve.StepTables",
                                   "Addressing of one step, as hc_build_block_tables defines it.", step_fields, 6};

}  // namespace

PyMODINIT_FUNC PyInit__serve(void) {
  PyObject* m = PyModule_Create(&module);
  if (!m) return nullptr;
  step_tables_type = PyStructSequence_NewType(&step_desc);
  if (!step_tables_type || PyModule_AddObjectRef(m, "StepTables", reinterpret_cast<PyObject*>(step_tables_type)) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
