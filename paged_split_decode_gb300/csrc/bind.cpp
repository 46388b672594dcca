// bind.cpp -- argument checks and marshalling of the calls that run beside
// kernels of a few microseconds (decode_paged_diff, decode_paged_scored,
// write_kv_cache_fp4, evict_kv_cache, build_block_tables, release_blocks,
// rms_norm), as a CPython extension over libpdecode's C ABI:
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
decltype(&::decode_paged_scored) f_scored;
decltype(&::pd_scored_workspace_bytes) f_scored_ws;
decltype(&::write_kv_cache_fp4) f_write4;
decltype(&::evict_kv_cache) f_evict;
decltype(&::pd_evict_workspace_bytes) f_evict_ws;
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

// The caches of a call: their kind, and the sizes that follow from them. 4-bit caches are uint8
// tensors of codes with block scales beside them, heads before keys.
struct Caches {
  const Tensor &k, &v;
  const Tensor *k_scale, *v_scale;
  ScalarType type;

  Caches(const Tensor& k_, const Tensor& v_, const Tensor* ks, const Tensor* vs) : k(k_), v(v_), k_scale(ks), v_scale(vs) {
    type = k.scalar_type();
    if (k.dim() != 4) value_error("the caches must be [num_blocks, block_size, Hkv, D], 4-bit ones [num_blocks, Hkv, block_size, D/2]");
    if (v.sizes() != k.sizes() || v.scalar_type() != type) value_error("v_cache must match k_cache in shape and dtype");
    if ((k_scale != nullptr) != (v_scale != nullptr)) value_error("give both k_block_scale and v_block_scale, or neither");
    if (!k_scale) return;
    if (type != at::kByte) type_error("4-bit caches (those with block scales) must be uint8");
    for (const Tensor* s : {k_scale, v_scale})
      if (s->dim() != 4 || s->size(0) != k.size(0) || s->size(1) != k.size(1) || s->size(2) != k.size(2) ||
          s->size(3) * 8 != k.size(3))
        value_error("block scales must be [num_blocks, Hkv, block_size, D/16]");
  }
  bool fp4() const { return k_scale != nullptr; }
  // q (or new tokens) of type qt
  int32_t kind(ScalarType qt) const {
    const bool bf = qt == at::kBFloat16;
    if (fp4()) return bf ? PD_KV_FP4_BF16 : PD_KV_FP4;
    if (type == at::kHalf) return PD_KV_F16;
    if (type == at::kBFloat16) return PD_KV_BF16;
    if (type == at::kByte || type == at::kFloat8_e4m3fn) return bf ? PD_KV_FP8_E4M3_BF16 : PD_KV_FP8_E4M3;
    if (type == at::kChar) return bf ? PD_KV_INT8_BF16 : PD_KV_INT8;
    type_error(std::string("unsupported KV cache dtype ") + c10::toString(type));
  }
  void fill(pd_dims& d) const {
    d.num_blocks = extent(k.size(0), "k_cache");
    d.Hkv = extent(k.size(fp4() ? 1 : 2), "k_cache");
    d.block_size = extent(k.size(fp4() ? 2 : 1), "k_cache");
    d.D = extent(k.size(3) * (fp4() ? 2 : 1), "k_cache");
  }
  void check_weights(const Tensor* w, const char* name) const {
    if (w && (w->dim() != 3 || w->size(0) != k.size(0) || w->size(1) != k.size(fp4() ? 1 : 2) ||
              w->size(2) != k.size(fp4() ? 2 : 1)))
      value_error(std::string(name) + " must be [num_blocks, Hkv, block_size]");
  }
  void* scale_ptr(const Tensor* s, const char* name, int index) const {
    return pointer(s, name, index, at::kFloat8_e4m3fn, at::kByte);
  }
};

// The workspace that a call brought none of, from binding.py.
Tensor own_workspace(size_t need, int index, PyObject* stream) {
  PyObject* o = PyObject_CallFunction(g_workspace, "niO", static_cast<Py_ssize_t>(need), index, stream);
  if (!o) throw PyFail{};
  Tensor t;
  if (THPVariable_Check(o)) t = THPVariable_Unpack(o);
  Py_DECREF(o);
  if (!t.defined()) type_error("workspace must be a tensor");
  return t;
}

// q, k_cache, v_cache, block_table, seq_lens, scale, window, qlen, num_splits, out, query_start_loc,
// score_cap, alibi_slopes, prefix_lens, k_block_scale, v_block_scale, k_scale, v_scale, lse, key_weights,
// key_weights_out, workspace, error_flag, stream
PyObject* scored(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 24);
    const Tensor &q = tensor(a[0], "q"), &table = tensor(a[3], "block_table"), &seq = tensor(a[4], "seq_lens");
    const Caches c(tensor(a[1], "k_cache"), tensor(a[2], "v_cache"), tensor_or_none(a[14], "k_block_scale"),
                   tensor_or_none(a[15], "v_block_scale"));
    const Tensor *out = tensor_or_none(a[9], "out"), *start = tensor_or_none(a[10], "query_start_loc"),
                 *slopes = tensor_or_none(a[12], "alibi_slopes"), *prefix = tensor_or_none(a[13], "prefix_lens"),
                 *lse = tensor_or_none(a[18], "lse"), *weights = tensor_or_none(a[19], "key_weights"),
                 *weights_out = tensor_or_none(a[20], "key_weights_out"), *ws = tensor_or_none(a[21], "workspace"),
                 *flag = tensor_or_none(a[22], "error_flag");
    pd_dims d{};
    d.kv_dtype = c.kind(q.scalar_type());
    const ScalarType io = d.kv_dtype == PD_KV_BF16 || d.kv_dtype == PD_KV_FP8_E4M3_BF16 ||
                                  d.kv_dtype == PD_KV_INT8_BF16 || d.kv_dtype == PD_KV_FP4_BF16
                              ? at::kBFloat16
                              : at::kHalf;
    c.fill(d);
    if (q.dim() != 3 || table.dim() != 2) value_error("q must be [T, Hq, D], block_table [B, max_blocks]");
    const int64_t T = q.size(0), B = table.size(0);
    const int32_t qlen = integer(a[7], "qlen"), splits = integer(a[8], "num_splits");
    if (q.size(2) != d.D || seq.numel() != B) value_error("q must be [T, Hq, D] with the caches' D; seq_lens [B]");
    if (!start && T != B * qlen) value_error("q must be [B*qlen, Hq, D] with B = rows of block_table");
    if (start && start->numel() != B + 1) value_error("query_start_loc must be [B+1]");
    if (slopes && slopes->numel() != q.size(1)) value_error("alibi_slopes must be [Hq]");
    if (prefix && prefix->numel() != B) value_error("prefix_lens must be [B]");
    if (lse && lse->numel() != T * q.size(1)) value_error("lse must be [T, Hq]");
    if (out && out->sizes() != q.sizes()) value_error("out must have q's shape");
    if (weights_out && !weights) value_error("key_weights_out needs key_weights");
    if (!weights_out) weights_out = weights;
    c.check_weights(weights, "key_weights");
    c.check_weights(weights_out, "key_weights_out");
    d.B = extent(B, "block_table");
    d.Hq = extent(q.size(1), "q");
    d.max_blocks_per_seq = extent(table.size(1), "block_table");
    d.k_scale = static_cast<float>(real(a[16]));
    d.v_scale = static_cast<float>(real(a[17]));
    const int32_t total = extent(T, "q");
    const int index = gpu_of(q, "q");
    const Launch at_stream(index, a[23]);
    Tensor made;
    if (!out) {  // rows outside every sequence's range are zero in a new output
      made = at_stream.alloc([&] { return start ? at::zeros_like(q) : at::empty_like(q); });
      out = &made;
    }
    Tensor ws_made;
    if (!ws) {
      // kept by the shapes that the plan depends on
      using Key = std::tuple<int, int, int, int, int, int, int, int, int, int, int, bool>;
      static std::map<Key, size_t> sizes;
      const Key key{index, d.B, d.Hq, d.Hkv, d.D, d.block_size, d.num_blocks, d.max_blocks_per_seq, d.kv_dtype, qlen,
                    splits, weights != nullptr};
      auto it = sizes.find(key);
      if (it == sizes.end()) {
        if (sizes.size() >= 4096) sizes.clear();
        it = sizes.emplace(key, f_scored_ws(&d, qlen, splits, weights != nullptr, 0)).first;
      }
      if (it->second > 0) {
        ws_made = own_workspace(it->second, index, a[23]);
        ws = &ws_made;
      }
    }
    void *pq = pointer(&q, "q", index, io), *pk = pointer(&c.k, "k_cache", index, c.type),
         *pv = pointer(&c.v, "v_cache", index, c.type), *po = pointer(out, "out", index, io),
         *pws = ws ? pointer(ws, "workspace", index, ws->scalar_type()) : nullptr;
    int32_t *pt = ints(&table, "block_table", index), *ps = ints(&seq, "seq_lens", index),
            *pstart = ints(start, "query_start_loc", index);
    pd_score s{};
    s.cap = static_cast<float>(real(a[11]));
    s.alibi_slopes = pointer<float>(slopes, "alibi_slopes", index, at::kFloat);
    s.prefix_lens = ints(prefix, "prefix_lens", index);
    s.k_block_scale = c.scale_ptr(c.k_scale, "k_block_scale", index);
    s.v_block_scale = c.scale_ptr(c.v_scale, "v_block_scale", index);
    s.lse = pointer<float>(lse, "lse", index, at::kFloat);
    s.key_weights = pointer<float>(weights, "key_weights", index, at::kFloat);
    s.key_weights_out = pointer<float>(weights_out, "key_weights_out", index, at::kFloat);
    uint32_t* pflag = flag_of(flag, index);
    const float scale = static_cast<float>(real(a[5]));
    const int32_t window = integer(a[6], "window");
    const size_t ws_bytes = ws ? ws->nbytes() : 0;
    pd_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = f_scored(pq, pk, pv, pt, ps, pstart, total, scale, window, qlen, splits, &s, po, &d, pws, ws_bytes, pflag,
                  at_stream.stream);
    Py_END_ALLOW_THREADS;
    check(st, "decode_paged_scored");
    return made.defined() ? wrap(made) : same(a[9]);
  });
}

// k_new, v_new, slot_mapping, k_cache, v_cache, k_block_scale, v_block_scale, k_scale, v_scale, error_flag, stream
PyObject* write_fp4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 11);
    const Tensor &k = tensor(a[0], "k_new"), &v = tensor(a[1], "v_new"), &slots = tensor(a[2], "slot_mapping");
    const Caches c(tensor(a[3], "k_cache"), tensor(a[4], "v_cache"), &tensor(a[5], "k_block_scale"),
                   &tensor(a[6], "v_block_scale"));
    const Tensor* flag = tensor_or_none(a[9], "error_flag");
    const ScalarType xt = k.scalar_type();
    if (xt != at::kHalf && xt != at::kBFloat16)
      type_error(std::string("k_new has dtype ") + c10::toString(xt) + ", expected Half or BFloat16");
    pd_dims d{};
    c.fill(d);
    d.Hq = d.Hkv;
    d.kv_dtype = c.kind(xt);
    if (k.dim() != 3 || k.size(0) != slots.numel() || k.size(1) != d.Hkv || k.size(2) != d.D || v.sizes() != k.sizes())
      value_error("k_new/v_new must be [T, Hkv, D] with T = len(slot_mapping)");
    d.k_scale = static_cast<float>(real(a[7]));
    d.v_scale = static_cast<float>(real(a[8]));
    const int32_t T = extent(slots.numel(), "slot_mapping");
    const int index = gpu_of(c.k, "k_cache");
    const Launch at_stream(index, a[10]);
    void *pkn = pointer(&k, "k_new", index, xt), *pvn = pointer(&v, "v_new", index, xt),
         *pk = pointer(&c.k, "k_cache", index, at::kByte), *pv = pointer(&c.v, "v_cache", index, at::kByte),
         *pks = c.scale_ptr(c.k_scale, "k_block_scale", index), *pvs = c.scale_ptr(c.v_scale, "v_block_scale", index);
    int64_t* pslot = pointer<int64_t>(&slots, "slot_mapping", index, at::kLong);
    uint32_t* pflag = flag_of(flag, index);
    pd_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = f_write4(pkn, pvn, pslot, T, pk, pv, pks, pvs, &d, pflag, at_stream.stream);
    Py_END_ALLOW_THREADS;
    check(st, "write_kv_cache_fp4");
    Py_RETURN_NONE;
  });
}

// k_cache, v_cache, key_weights, block_table, seq_lens, keep, trigger, first, recent, block_table_out, seq_lens_out,
// k_block_scale, v_block_scale, free_blocks, free_count, workspace, error_flag, stream
PyObject* evict(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args a(args, n, 18);
    const Caches c(tensor(a[0], "k_cache"), tensor(a[1], "v_cache"), tensor_or_none(a[11], "k_block_scale"),
                   tensor_or_none(a[12], "v_block_scale"));
    const Tensor &weights = tensor(a[2], "key_weights"), &table = tensor(a[3], "block_table"),
                 &seq = tensor(a[4], "seq_lens");
    const Tensor *table_out = tensor_or_none(a[9], "block_table_out"), *seq_out = tensor_or_none(a[10], "seq_lens_out"),
                 *free_blocks = tensor_or_none(a[13], "free_blocks"), *count = tensor_or_none(a[14], "free_count"),
                 *ws = tensor_or_none(a[15], "workspace"), *flag = tensor_or_none(a[16], "error_flag");
    pd_dims d{};
    c.fill(d);
    d.Hq = d.Hkv;
    d.kv_dtype = c.kind(at::kHalf);
    c.check_weights(&weights, "key_weights");
    if (table.dim() != 2) value_error("block_table must be [B, max_blocks]");
    if (table_out && (table_out->dim() != 2 || table_out->size(0) != table.size(0)))
      value_error("block_table_out must be [B, max_blocks_out]");
    if (seq.numel() != table.size(0)) value_error("seq_lens must be [B]");
    if (seq_out && seq_out->numel() != table.size(0)) value_error("seq_lens_out must be [B]");
    if (free_blocks && free_blocks->numel() != d.num_blocks) value_error("free_blocks must be [num_blocks]");
    if (count && count->numel() != 1) value_error("free_count must be [1]");
    if (!seq_out) seq_out = &seq;
    d.B = extent(table.size(0), "block_table");
    d.max_blocks_per_seq = extent(table.size(1), "block_table");
    pd_eviction e{};
    e.keep = integer(a[5], "keep");
    e.trigger = a[6] == Py_None ? e.keep : integer(a[6], "trigger");
    e.first = integer(a[7], "first");
    e.recent = integer(a[8], "recent");
    const int index = gpu_of(c.k, "k_cache");
    const Launch at_stream(index, a[17]);
    Tensor ws_made;
    if (!ws) {
      const size_t need = f_evict_ws(&d, &e);
      if (need > 0) {
        ws_made = own_workspace(need, index, a[17]);
        ws = &ws_made;
      }
    }
    void *pk = pointer(&c.k, "k_cache", index, c.type), *pv = pointer(&c.v, "v_cache", index, c.type),
         *pks = c.scale_ptr(c.k_scale, "k_block_scale", index), *pvs = c.scale_ptr(c.v_scale, "v_block_scale", index),
         *pws = ws ? pointer(ws, "workspace", index, ws->scalar_type()) : nullptr;
    float* pw = pointer<float>(&weights, "key_weights", index, at::kFloat);
    int32_t *pt = ints(&table, "block_table", index), *pto = ints(table_out, "block_table_out", index),
            *ps = ints(&seq, "seq_lens", index), *pso = ints(seq_out, "seq_lens_out", index),
            *pf = ints(free_blocks, "free_blocks", index), *pn = ints(count, "free_count", index);
    uint32_t* pflag = flag_of(flag, index);
    const int32_t cols = table_out ? extent(table_out->size(1), "block_table_out") : 0;
    const size_t ws_bytes = ws ? ws->nbytes() : 0;
    pd_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = f_evict(pk, pv, pks, pvs, pw, pt, ps, &e, pto, cols, pso, pf, pn, &d, pws, ws_bytes, pflag, at_stream.stream);
    Py_END_ALLOW_THREADS;
    check(st, "evict_kv_cache");
    return same(a[10] == Py_None ? a[4] : a[10]);
  });
}

// init(addresses of decode_paged_diff, pd_diff_workspace_bytes,
// build_block_tables, release_blocks, rms_norm, pd_status_str, decode_paged_scored,
// pd_scored_workspace_bytes, write_kv_cache_fp4, evict_kv_cache, pd_evict_workspace_bytes;
// the error class; the workspace callable)
PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    constexpr int kEntries = 11;
    Args a(args, n, kEntries + 2);
    void* p[kEntries];
    for (int i = 0; i < kEntries; ++i) {
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
    f_scored = reinterpret_cast<decltype(f_scored)>(p[6]);
    f_scored_ws = reinterpret_cast<decltype(f_scored_ws)>(p[7]);
    f_write4 = reinterpret_cast<decltype(f_write4)>(p[8]);
    f_evict = reinterpret_cast<decltype(f_evict)>(p[9]);
    f_evict_ws = reinterpret_cast<decltype(f_evict_ws)>(p[10]);
    Py_XSETREF(g_error, Py_NewRef(a[kEntries]));
    Py_XSETREF(g_workspace, Py_NewRef(a[kEntries + 1]));
    Py_RETURN_NONE;
  });
}

PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(init)), METH_FASTCALL, nullptr},
    {"decode_paged_diff", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(diff)), METH_FASTCALL, nullptr},
    {"build_block_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(build_tables)), METH_FASTCALL, nullptr},
    {"release_blocks", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(release)), METH_FASTCALL, nullptr},
    {"rms_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(norm)), METH_FASTCALL, nullptr},
    {"decode_paged_scored", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(scored)), METH_FASTCALL, nullptr},
    {"write_kv_cache_fp4", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(write_fp4)), METH_FASTCALL, nullptr},
    {"evict_kv_cache", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(evict)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Argument marshalling over libpdecode.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
