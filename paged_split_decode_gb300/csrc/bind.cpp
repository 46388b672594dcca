// bind.cpp -- argument checks and marshalling of the calls that run beside
// kernels of a few microseconds (decode_paged_diff, build_block_tables,
// release_blocks, rms_norm), as a CPython extension over libpdecode's C ABI:
// tensors become device pointers, the current stream becomes the launch stream,
// a status other than PD_OK becomes an exception. No computation happens here.
//
// Why compiled: a call checks up to twelve tensors (device, type, layout, size).
// Through the interpreter and ctypes that took 8.7 us for build_block_tables on
// the GPU's host, more than twice its kernel (3.2 us).
//
// The functions take their arguments by position, in the order of the Python
// functions that wrap them (binding.py, which documents them); None stands for
// an argument left out.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <ATen/ops/zeros_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <map>
#include <string>
#include <tuple>

#include "pdecode.h"

namespace {

using at::ScalarType;
using at::Tensor;

// libpdecode's entry points, handed over by init()
decltype(&::decode_paged_diff) f_diff;
decltype(&::pd_diff_workspace_bytes) f_diff_ws;
decltype(&::build_block_tables) f_build;
decltype(&::release_blocks) f_release;
decltype(&::rms_norm) f_norm;
decltype(&::pd_status_str) f_status;
PyObject* g_error = nullptr;      // DecodeError
PyObject* g_workspace = nullptr;  // callable(need, device index, stream handle) -> tensor

struct PyFail {};  // a Python error is set

[[noreturn]] void fail(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw PyFail{};
}
[[noreturn]] void type_error(const std::string& text) { fail(PyExc_TypeError, text); }
[[noreturn]] void value_error(const std::string& text) { fail(PyExc_ValueError, text); }

// An optional tensor argument.
const Tensor* tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name) {
  const Tensor* t = tensor_or_none(o, name);
  if (!t) type_error(std::string(name) + " must be a tensor");
  return *t;
}
int32_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyFail{};
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " is out of range");
  return static_cast<int32_t>(v);
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyFail{};
  return v;
}
int32_t extent(int64_t v, const char* name) {
  if (v > INT32_MAX) value_error(std::string(name) + " is too large");
  return static_cast<int32_t>(v);
}

int gpu_of(const Tensor& t, const char* name) {
  if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
  return t.get_device();
}

// Device pointer of a contiguous tensor on GPU `index` (null for none), of type
// a or b.
template <class T = void>
T* pointer(const Tensor* t, const char* name, int index, ScalarType a, ScalarType b) {
  if (!t) return nullptr;
  if (!t->is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
  if (t->get_device() != index)
    value_error(std::string(name) + " is on " + t->device().str() + ", expected cuda:" + std::to_string(index));
  const ScalarType s = t->scalar_type();
  if (s != a && s != b)
    type_error(std::string(name) + " has dtype " + c10::toString(s) + ", expected " + c10::toString(a));
  if (!t->is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return static_cast<T*>(t->data_ptr());
}
template <class T = void>
T* pointer(const Tensor* t, const char* name, int index, ScalarType a) {
  return pointer<T>(t, name, index, a, a);
}
int32_t* ints(const Tensor* t, const char* name, int index) { return pointer<int32_t>(t, name, index, at::kInt); }
uint32_t* flag_of(const Tensor* t, int index) {
  return pointer<uint32_t>(t, "error_flag", index, at::kInt, at::kUInt32);
}

// The launch stream, and the device made current for the call: an explicit
// handle, or the device's current stream. Outputs made for an explicit stream
// are allocated in its order.
struct Launch {
  int index;
  cudaStream_t stream;
  bool given;
  c10::cuda::OptionalCUDAGuard device;

  Launch(int idx, PyObject* handle) : index(idx), given(handle != Py_None) {
    if (given) {
      stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
      if (PyErr_Occurred()) throw PyFail{};
    } else {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(idx)).stream();
    }
    if (c10::cuda::current_device() != idx) device.set_index(static_cast<c10::DeviceIndex>(idx));
  }
  // Runs `make` with allocations ordered by the launch stream.
  template <class F>
  Tensor alloc(F make) const {
    if (!given) return make();
    c10::cuda::CUDAStreamGuard guard(
        c10::cuda::getStreamFromExternal(stream, static_cast<c10::DeviceIndex>(index)));
    return make();
  }
};

void check(pd_status st, const char* what) {
  if (st != PD_OK)
    fail(g_error, std::string(what) + ": " + f_status(st) + " (status " + std::to_string(static_cast<int>(st)) + ")");
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* same(PyObject* o) { return Py_NewRef(o); }

// Arguments of a call: a fixed count, by position.
struct Args {
  PyObject* const* a;
  Args(PyObject* const* args, Py_ssize_t n, Py_ssize_t want) : a(args) {
    if (n != want) type_error("wrong number of arguments");
  }
  PyObject* operator[](int i) const { return a[i]; }
};

template <class F>
PyObject* guarded(F body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const PyFail&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
pd_dims table_dims(const Tensor& table, const Tensor& free_blocks, PyObject* block_size) {
  pd_dims d{};
  d.B = extent(table.size(0), "block_table");
  d.Hq = d.Hkv = d.D = 1;
  d.block_size = integer(block_size, "block_size");
  d.num_blocks = extent(free_blocks.numel(), "free_blocks");
  d.max_blocks_per_seq = extent(table.size(1), "block_table");
  d.k_scale = d.v_scale = 1.f;
  return d;
}

// context_lens, query_lens, block_table, free_blocks, free_count, block_size,
// num_tokens, seq_lens, query_start_loc, slot_mapping, positions,
// free_count_out, error_flag, stream
PyObject* build_tables(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 14);
    const Tensor &ctx = tensor(a[0], "context_lens"), &query = tensor(a[1], "query_lens"),
                 &table = tensor(a[2], "block_table"), &free_blocks = tensor(a[3], "free_blocks"),
                 &count = tensor(a[4], "free_count");
    const Tensor *seq = tensor_or_none(a[7], "seq_lens"), *start = tensor_or_none(a[8], "query_start_loc"),
                 *slots = tensor_or_none(a[9], "slot_mapping"), *pos = tensor_or_none(a[10], "positions"),
                 *count_out = tensor_or_none(a[11], "free_count_out"), *flag = tensor_or_none(a[12], "error_flag");
    if (table.dim() != 2) value_error("block_table must be [B, max_blocks]");
    const int64_t B = table.size(0);
    if (ctx.numel() != B || query.numel() != B) value_error("context_lens and query_lens must be [B]");
    if (!slots && a[6] == Py_None) value_error("give num_tokens or a slot_mapping");
    const int32_t T = a[6] == Py_None ? extent(slots->numel(), "slot_mapping") : integer(a[6], "num_tokens");
    if (T < 0) value_error("num_tokens must not be negative");
    if (slots && slots->numel() != T) value_error("slot_mapping must be [num_tokens]");
    if (pos && pos->numel() != T) value_error("positions must be [num_tokens]");
    if (!count_out) count_out = &count;
    if (count.numel() != 1 || count_out->numel() != 1) value_error("free_count must be [1]");
    if (seq && seq->numel() != B) value_error("seq_lens must be [B]");
    if (start && start->numel() != B + 1) value_error("query_start_loc must be [B+1]");
    const pd_dims d = table_dims(table, free_blocks, a[5]);
    const int index = gpu_of(table, "block_table");
    const Launch at_stream(index, a[13]);
    Tensor made[4];
    const auto i32 = table.options().dtype(at::kInt);
    auto provide = [&](const Tensor*& t, Tensor& slot, int64_t size, const at::TensorOptions& o) {
      if (t) return;
      slot = at_stream.alloc([&] { return at::empty({size}, o); });
      t = &slot;
    };
    provide(seq, made[0], B, i32);
    provide(start, made[1], B + 1, i32);
    provide(slots, made[2], T, table.options().dtype(at::kLong));
    provide(pos, made[3], T, i32);
    int32_t *pc = ints(&ctx, "context_lens", index), *pq = ints(&query, "query_lens", index),
            *pt = ints(&table, "block_table", index), *pf = ints(&free_blocks, "free_blocks", index),
            *pn = ints(&count, "free_count", index), *po = ints(count_out, "free_count_out", index),
            *ps = ints(seq, "seq_lens", index), *pstart = ints(start, "query_start_loc", index),
            *pp = ints(pos, "positions", index);
    int64_t* pslot = pointer<int64_t>(slots, "slot_mapping", index, at::kLong);
    uint32_t* pflag = flag_of(flag, index);
    pd_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = f_build(pc, pq, T, pt, pf, pn, po, ps, pstart, pslot, pp, &d, pflag, at_stream.stream);
    Py_END_ALLOW_THREADS;
    check(st, "build_block_tables");
    PyObject* out = PyTuple_New(4);
    if (!out) return nullptr;
    for (int i = 0; i < 4; ++i) PyTuple_SET_ITEM(out, i, made[i].defined() ? wrap(made[i]) : same(a[7 + i]));
    return out;
  });
}

// block_table, seq_lens, released, free_blocks, free_count, block_size,
// seq_lens_out, free_count_out, error_flag, stream
PyObject* release(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 10);
    const Tensor &table = tensor(a[0], "block_table"), &seq = tensor(a[1], "seq_lens"),
                 &released = tensor(a[2], "released"), &free_blocks = tensor(a[3], "free_blocks"),
                 &count = tensor(a[4], "free_count");
    const Tensor *seq_out = tensor_or_none(a[6], "seq_lens_out"), *count_out = tensor_or_none(a[7], "free_count_out"),
                 *flag = tensor_or_none(a[8], "error_flag");
    if (table.dim() != 2) value_error("block_table must be [B, max_blocks]");
    const int64_t B = table.size(0);
    if (seq.numel() != B || released.numel() != B) value_error("seq_lens and released must be [B]");
    if (!count_out) count_out = &count;
    if (count.numel() != 1 || count_out->numel() != 1) value_error("free_count must be [1]");
    if (seq_out && seq_out->numel() != B) value_error("seq_lens_out must be [B]");
    const pd_dims d = table_dims(table, free_blocks, a[5]);
    const int index = gpu_of(table, "block_table");
    const Launch at_stream(index, a[9]);
    int32_t *pt = ints(&table, "block_table", index), *ps = ints(&seq, "seq_lens", index),
            *pf = ints(&free_blocks, "free_blocks", index), *pn = ints(&count, "free_count", index),
            *po = ints(count_out, "free_count_out", index), *pso = ints(seq_out ? seq_out : &seq, "seq_lens_out", index);
    uint8_t* pr = pointer<uint8_t>(&released, "released", index, at::kBool, at::kByte);
    uint32_t* pflag = flag_of(flag, index);
    pd_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = f_release(pt, ps, pr, pf, pn, po, pso, &d, pflag, at_stream.stream);
    Py_END_ALLOW_THREADS;
    check(st, "release_blocks");
    return same(seq_out ? a[6] : a[1]);
  });
}

// x, weight, eps, residual, residual_out, gain, norm_size, out_dtype,
// scale_size, out, out_scale, stream
PyObject* norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 12);
    const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
    const Tensor *res = tensor_or_none(a[3], "residual"), *res_out = tensor_or_none(a[4], "residual_out"),
                 *out = tensor_or_none(a[9], "out"), *scale = tensor_or_none(a[10], "out_scale");
    const ScalarType xt = x.scalar_type();
    if (xt != at::kHalf && xt != at::kBFloat16)
      type_error(std::string("x has dtype ") + c10::toString(xt) + ", expected Half or BFloat16");
    if (x.dim() < 1 || x.size(-1) < 1) value_error("x must be [..., N] with N >= 1");
    pd_norm_dims d{};
    d.N = extent(x.size(-1), "x");
    d.rows = x.numel() / d.N;
    d.norm_size = a[6] == Py_None ? d.N : integer(a[6], "norm_size");
    d.scale_size = a[8] == Py_None ? d.N : integer(a[8], "scale_size");
    ScalarType ot = xt;
    if (a[7] != Py_None) {
      if (!THPDtype_Check(a[7])) type_error("out_dtype must be a torch.dtype");
      ot = reinterpret_cast<THPDtype*>(a[7])->scalar_type;
    } else if (out) {
      ot = out->scalar_type();
    }
    if (ot == xt) d.out_kind = PD_NORM_SAME;
    else if (ot == at::kFloat8_e4m3fn) d.out_kind = PD_NORM_E4M3;
    else if (ot == at::kChar) d.out_kind = PD_NORM_INT8;
    else type_error(std::string("unsupported output dtype ") + c10::toString(ot));
    const bool codes = d.out_kind != PD_NORM_SAME;
    if (d.norm_size < 1 || d.scale_size < 1 || d.N % d.norm_size || d.N % d.scale_size)
      value_error("norm_size and scale_size must divide N");
    if (weight.numel() != d.norm_size) value_error("weight must be [norm_size]");
    if (res && res->sizes() != x.sizes()) value_error("residual must have x's shape");
    if (res && !res_out) res_out = res;
    if (res_out && res_out->sizes() != x.sizes()) value_error("residual_out must have x's shape");
    if (out && (out->sizes() != x.sizes() || out->scalar_type() != ot))
      value_error("out must have x's shape and the output dtype");
    if (scale && (!codes || scale->numel() != d.rows * (d.N / d.scale_size)))
      value_error("out_scale is [..., N / scale_size], for 8-bit outputs only");
    const int index = gpu_of(x, "x");
    const Launch at_stream(index, a[11]);
    Tensor made_out, made_scale;
    if (!out) {
      made_out = at_stream.alloc([&] { return at::empty(x.sizes(), x.options().dtype(ot)); });
      out = &made_out;
    }
    if (codes && !scale) {
      auto shape = x.sizes().vec();
      shape.back() = d.N / d.scale_size;
      made_scale = at_stream.alloc([&] { return at::empty(shape, x.options().dtype(at::kFloat)); });
      scale = &made_scale;
    }
    d.x_bf16 = xt == at::kBFloat16;
    d.weight_f32 = weight.scalar_type() == at::kFloat;
    void *px = pointer(&x, "x", index, xt), *pr = pointer(res, "residual", index, xt),
         *pw = pointer(&weight, "weight", index, xt, at::kFloat), *pro = pointer(res_out, "residual_out", index, xt),
         *po = pointer(out, "out", index, ot);
    float* ps = pointer<float>(scale, "out_scale", index, at::kFloat);
    const float eps = static_cast<float>(real(a[2])), gain = static_cast<float>(real(a[5]));
    pd_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = f_norm(px, pr, pw, eps, gain, pro, po, ps, &d, at_stream.stream);
    Py_END_ALLOW_THREADS;
    check(st, "rms_norm");
    PyObject* o = made_out.defined() ? wrap(made_out) : same(a[9]);
    if (!codes) return o;
    PyObject* s = made_scale.defined() ? wrap(made_scale) : same(a[10]);
    PyObject* both = PyTuple_New(2);
    if (!both) return nullptr;
    PyTuple_SET_ITEM(both, 0, o);
    PyTuple_SET_ITEM(both, 1, s);
    return both;
  });
}

// q, k_cache, v_cache, block_table, seq_lens, lam, scale, window, qlen,
// num_splits, out, query_start_loc, norm_weight, norm_eps, norm_gain, k_scale,
// v_scale, workspace, error_flag, stream
PyObject* diff(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 20);
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache"),
                 &table = tensor(a[3], "block_table"), &seq = tensor(a[4], "seq_lens"), &lam = tensor(a[5], "lam");
    const Tensor *out = tensor_or_none(a[10], "out"), *start = tensor_or_none(a[11], "query_start_loc"),
                 *weight = tensor_or_none(a[12], "norm_weight"), *ws = tensor_or_none(a[17], "workspace"),
                 *flag = tensor_or_none(a[18], "error_flag");
    const ScalarType qt = q.scalar_type(), kt = k.scalar_type();
    pd_dims d{};
    if (kt == at::kHalf) d.kv_dtype = PD_KV_F16;
    else if (kt == at::kBFloat16) d.kv_dtype = PD_KV_BF16;
    else if (kt == at::kByte || kt == at::kFloat8_e4m3fn)
      d.kv_dtype = qt == at::kBFloat16 ? PD_KV_FP8_E4M3_BF16 : PD_KV_FP8_E4M3;
    else if (kt == at::kChar) d.kv_dtype = qt == at::kBFloat16 ? PD_KV_INT8_BF16 : PD_KV_INT8;
    else type_error(std::string("unsupported KV cache dtype ") + c10::toString(kt));
    const ScalarType io = d.kv_dtype >= PD_KV_BF16 ? at::kBFloat16 : at::kHalf;
    if (q.dim() != 3 || k.dim() != 4 || table.dim() != 2)
      value_error("q must be [T, Hq, D], the caches [num_blocks, block_size, Hkv, D], block_table [B, max_blocks]");
    if (v.sizes() != k.sizes() || v.scalar_type() != kt) value_error("v_cache must match k_cache in shape and dtype");
    const int64_t T = q.size(0), B = table.size(0);
    const int32_t qlen = integer(a[8], "qlen"), splits = integer(a[9], "num_splits");
    if (q.size(2) != k.size(3) || seq.numel() != B) value_error("q must be [T, Hq, D] with the caches' D; seq_lens [B]");
    if (!start && T != B * qlen) value_error("q must be [B*qlen, Hq, D] with B = rows of block_table");
    if (start && start->numel() != B + 1) value_error("query_start_loc must be [B+1]");
    if (lam.numel() != q.size(1)) value_error("lam must be [Hq]");
    if (weight && weight->numel() != q.size(2)) value_error("norm_weight must be [D]");
    if (out && out->sizes() != q.sizes()) value_error("out must have q's shape");
    d.B = extent(B, "block_table");
    d.Hq = extent(q.size(1), "q");
    d.Hkv = extent(k.size(2), "k_cache");
    d.D = extent(q.size(2), "q");
    d.block_size = extent(k.size(1), "k_cache");
    d.num_blocks = extent(k.size(0), "k_cache");
    d.max_blocks_per_seq = extent(table.size(1), "block_table");
    d.k_scale = static_cast<float>(real(a[15]));
    d.v_scale = static_cast<float>(real(a[16]));
    const int32_t total = extent(T, "q");
    const int index = gpu_of(q, "q");
    const Launch at_stream(index, a[19]);
    Tensor made;
    if (!out) {  // rows outside every sequence's range are zero in a new output
      made = at_stream.alloc([&] { return start ? at::zeros_like(q) : at::empty_like(q); });
      out = &made;
    }
    Tensor ws_made;
    if (!ws) {
      // kept by the shapes that the plan depends on
      using Key = std::tuple<int, int, int, int, int, int, int, int, int, int, int>;
      static std::map<Key, size_t> sizes;
      const Key key{index, d.B, d.Hq, d.Hkv, d.D, d.block_size, d.num_blocks, d.max_blocks_per_seq, d.kv_dtype, qlen,
                    splits};
      auto it = sizes.find(key);
      if (it == sizes.end()) {
        if (sizes.size() >= 4096) sizes.clear();
        it = sizes.emplace(key, f_diff_ws(&d, qlen, splits, 0)).first;
      }
      if (it->second > 0) {
        PyObject* o = PyObject_CallFunction(g_workspace, "niO", static_cast<Py_ssize_t>(it->second), index, a[19]);
        if (!o) throw PyFail{};
        if (THPVariable_Check(o)) ws_made = THPVariable_Unpack(o);
        Py_DECREF(o);
        if (!ws_made.defined()) type_error("workspace must be a tensor");
        ws = &ws_made;
      }
    }
    void *pq = pointer(&q, "q", index, io), *pk = pointer(&k, "k_cache", index, kt),
         *pv = pointer(&v, "v_cache", index, kt), *po = pointer(out, "out", index, io),
         *pw = pointer(weight, "norm_weight", index, io, at::kFloat),
         *pws = ws ? pointer(ws, "workspace", index, ws->scalar_type()) : nullptr;
    int32_t *pt = ints(&table, "block_table", index), *ps = ints(&seq, "seq_lens", index),
            *pstart = ints(start, "query_start_loc", index);
    float* pl = pointer<float>(&lam, "lam", index, at::kFloat);
    uint32_t* pflag = flag_of(flag, index);
    const float scale = static_cast<float>(real(a[6])), eps = static_cast<float>(real(a[13])),
                gain = static_cast<float>(real(a[14]));
    const int32_t window = integer(a[7], "window");
    const size_t ws_bytes = ws ? ws->nbytes() : 0;
    const int f32 = weight && weight->scalar_type() == at::kFloat;
    pd_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = f_diff(pq, pk, pv, pt, ps, pstart, total, pl, scale, window, qlen, splits, pw, f32, eps, gain, po, &d, pws,
                ws_bytes, pflag, at_stream.stream);
    Py_END_ALLOW_THREADS;
    check(st, "decode_paged_diff");
    return made.defined() ? wrap(made) : same(a[10]);
  });
}

// init(addresses of decode_paged_diff, pd_diff_workspace_bytes,
// build_block_tables, release_blocks, rms_norm, pd_status_str; the error class;
// the workspace callable)
PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 8);
    void* p[6];
    for (int i = 0; i < 6; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (!p[i]) {
        if (!PyErr_Occurred()) value_error("a null entry point");
        throw PyFail{};
      }
    }
    f_diff = reinterpret_cast<decltype(f_diff)>(p[0]);
    f_diff_ws = reinterpret_cast<decltype(f_diff_ws)>(p[1]);
    f_build = reinterpret_cast<decltype(f_build)>(p[2]);
    f_release = reinterpret_cast<decltype(f_release)>(p[3]);
    f_norm = reinterpret_cast<decltype(f_norm)>(p[4]);
    f_status = reinterpret_cast<decltype(f_status)>(p[5]);
    Py_XSETREF(g_error, Py_NewRef(a[6]));
    Py_XSETREF(g_workspace, Py_NewRef(a[7]));
    Py_RETURN_NONE;
  });
}

PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(init)), METH_FASTCALL, nullptr},
    {"decode_paged_diff", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(diff)), METH_FASTCALL, nullptr},
    {"build_block_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(build_tables)), METH_FASTCALL, nullptr},
    {"release_blocks", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(release)), METH_FASTCALL, nullptr},
    {"rms_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(norm)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Argument marshalling over libpdecode.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
