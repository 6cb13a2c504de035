// Compiled half of the Python binding, for the calls around the 4-bit cache and
// multi-axis rotary positions: it checks the tensors, allocates outputs,
// and calls the C ABI (include/exattn.h) on the tensors' device and stream.
//
// A serving step makes these calls with a handful of tokens, where the kernels take
// a few microseconds; marshalling the same call through ctypes takes about 20
// (attribute look-ups and 20 converted arguments), through here 5.  Arguments
// come positionally from the functions of exattn.py, which document them.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <array>
#include <cmath>
#include <cstdarg>
#include <optional>

#include "../../include/exattn.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // exattn.ExattnError

[[noreturn]] void fail(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw python_error();
}

const Tensor& tensor(PyObject* o, const char* name, int64_t ndim, at::ScalarType type) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
  const Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != type) fail(PyExc_TypeError, "%s must be torch.%s, got %s", name,
                                    type == at::kBFloat16 ? "bfloat16" : type == at::kInt ? "int32"
                                    : type == at::kFloat ? "float32" : "uint8", c10::toString(t.scalar_type()));
  if (t.dim() != ndim) fail(PyExc_ValueError, "%s must have %lld dimensions, got %lld", name,
                            static_cast<long long>(ndim), static_cast<long long>(t.dim()));
  return t;
}

// A tensor of the call: on `device`, of the given shape (-1: any).
void check(const Tensor& t, const char* name, c10::Device device, at::IntArrayRef shape, bool contiguous) {
  if (t.device() != device) fail(PyExc_ValueError, "%s must live on %s, is on %s", name, device.str().c_str(),
                                 t.device().str().c_str());
  for (size_t i = 0; i < shape.size(); ++i)
    if (shape[i] >= 0 && t.size(i) != shape[i])
      fail(PyExc_ValueError, "%s: size of dimension %d must be %lld, got %lld", name, static_cast<int>(i),
           static_cast<long long>(shape[i]), static_cast<long long>(t.size(i)));
  if (contiguous ? !t.is_contiguous() : t.stride(-1) != 1)
    fail(PyExc_ValueError, contiguous ? "%s must be contiguous" : "the last dimension of %s must be contiguous", name);
}

c10::Device cuda_device(const Tensor& t, const char* name) {
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must live on a CUDA device", name);
  return t.device();
}

int narrow(int64_t v, const char* name) {
  if (v > 0x7FFFFFFF) fail(PyExc_ValueError, "%s is too large", name);
  return static_cast<int>(v);
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// Pairs of each axis.
struct Sections {
  int size[8];
  int count;
  explicit Sections(PyObject* o) {
    PyObject* seq = PySequence_Fast(o, "sections must be a sequence of integers");
    if (seq == nullptr) throw python_error();
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    count = n > 8 ? 8 : static_cast<int>(n);  // more than the library's four are refused there
    for (int i = 0; i < count; ++i) {
      const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
      if (v == -1 && PyErr_Occurred()) {
        Py_DECREF(seq);
        throw python_error();
      }
      size[i] = v < -1 || v > 0x7FFFFFFF ? -1 : static_cast<int>(v);
    }
    Py_DECREF(seq);
  }
};

// Where a call runs: the tensors' device, and the given stream or that device's current
// one.  While it exists they are the current device and stream, so that what the call
// allocates belongs to the stream that uses it: out of the caller's current stream's
// memory it could be a block whose last use there is still to come.
struct Target {
  c10::Device device;
  c10::cuda::CUDAGuard guard;
  c10::cuda::CUDAStream callers;  // the caller's current stream
  cudaStream_t handle;
  c10::cuda::OptionalCUDAStreamGuard on;

  Target(c10::Device d, PyObject* stream)
      : device(d), guard(d), callers(c10::cuda::getCurrentCUDAStream(d.index())), handle(callers.stream()) {
    if (stream == Py_None) return;
    PyObject* raw = PyObject_GetAttrString(stream, "cuda_stream");
    if (raw == nullptr) throw python_error();
    handle = static_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
    Py_DECREF(raw);
    if (handle == nullptr && PyErr_Occurred()) throw python_error();
    if (handle != callers.stream()) on.reset_stream(c10::cuda::getStreamFromExternal(handle, d.index()));
  }

  // A new contiguous tensor, straight from the CUDA allocator (through the
  // operators' dispatcher it takes half a microsecond more).
  Tensor fresh(at::IntArrayRef shape, at::ScalarType type) const {
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
  }

  // The output `o`, or a new contiguous tensor where it is None.  The caller will go on
  // with that on its own stream: the allocator is told, for when it is dropped.
  Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, bool contiguous) const {
    if (o == Py_None) {
      const Tensor t = fresh(shape, type);
      if (handle != callers.stream() && t.numel() > 0)
        c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), callers);
      return t;
    }
    const Tensor& t = tensor(o, name, static_cast<int64_t>(shape.size()), type);
    check(t, name, device, shape, contiguous);
    return t;
  }

  // Runs call(stream), without the interpreter's lock.
  template <typename Call>
  void launch(const char* name, Call call) const {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call(static_cast<void*>(handle));
    Py_END_ALLOW_THREADS
    if (rc != EXATTN_OK) {
      PyObject* e = PyObject_CallFunction(g_error, "si", name, rc);
      if (e != nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
      }
      throw python_error();
    }
  }
};

void need_args(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) fail(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
}

const int32_t* ints(const Tensor& t) { return static_cast<const int32_t*>(t.const_data_ptr()); }

PyObject* pair(const Tensor& a, const Tensor& b) {
  return Py_BuildValue("NN", THPVariable_Wrap(a), b.defined() ? THPVariable_Wrap(b) : Py_NewRef(Py_None));
}

// (q, k, positions, sections, base, per_axis, inverse, q_out, k_out, stream)
PyObject* rope_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 10);
  const Tensor& q = tensor(a[0], "q", 4, at::kBFloat16);
  const Tensor& k = tensor(a[1], "k", 4, at::kBFloat16);
  const c10::Device device = cuda_device(q, "q");
  const int64_t B = q.size(0), Hq = q.size(1), N = q.size(2), d = q.size(3), Hkv = k.size(1);
  check(q, "q", device, {}, false);
  check(k, "k", device, {B, -1, N, d}, false);
  const Sections sections(a[3]);
  if (!THPVariable_Check(a[2])) fail(PyExc_TypeError, "positions must be a torch.Tensor");
  const bool batched = THPVariable_Unpack(a[2]).dim() == 3;
  const Tensor& pos = tensor(a[2], "positions", batched ? 3 : 2, at::kInt);
  if (pos.device() != device || pos.size(0) != sections.count || pos.size(-1) != N || (batched && pos.size(1) != B))
    fail(PyExc_ValueError, "positions must be [%d, %lld, %lld] or [%d, %lld] on the tensors' device", sections.count,
         static_cast<long long>(B), static_cast<long long>(N), sections.count, static_cast<long long>(N));
  const Target on(device, a[9]);
  const Tensor qo = on.output(a[7], "q_out", q.sizes(), at::kBFloat16, false);
  const Tensor ko = on.output(a[8], "k_out", k.sizes(), at::kBFloat16, false);
  const int64_t strides[15] = {q.stride(0),  q.stride(1),  q.stride(2),  k.stride(0),  k.stride(1),
                               k.stride(2),  qo.stride(0), qo.stride(1), qo.stride(2), ko.stride(0),
                               ko.stride(1), ko.stride(2), pos.stride(0), batched ? pos.stride(1) : 0, pos.stride(-1)};
  const float base = static_cast<float>(number(a[4]));
  const int per_axis = truth(a[5]), inverse = truth(a[6]);
  const int iB = narrow(B, "B"), iHq = narrow(Hq, "Hq"), iHkv = narrow(Hkv, "Hkv"), iN = narrow(N, "N"),
            id = narrow(d, "d");
  on.launch("attn_rope_axes", [&](void* s) {
    return attn_rope_axes(q.const_data_ptr(), k.const_data_ptr(), qo.data_ptr(), ko.data_ptr(), ints(pos), strides,
                          sections.size, sections.count, iB, iHq, iHkv, iN, id, base, per_axis, inverse, s);
  });
  return pair(qo, ko);
  END_HANDLE_TH_ERRORS
}

// The cache and block table that the 4-bit calls share.
struct Cache {
  const Tensor& t;
  c10::Device device;
  int num_blocks, Hkv, d;
  explicit Cache(PyObject* o) : t(tensor(o, "kv_cache", 3, at::kByte)), device(cuda_device(t, "kv_cache")) {
    if (t.size(2) % 18 != 0 || !t.is_contiguous())
      fail(PyExc_ValueError, "kv_cache must be contiguous [num_blocks, Hkv, 18 d], got [%lld, %lld, %lld]",
           static_cast<long long>(t.size(0)), static_cast<long long>(t.size(1)), static_cast<long long>(t.size(2)));
    num_blocks = narrow(t.size(0), "num_blocks");
    Hkv = narrow(t.size(1), "Hkv");
    d = narrow(t.size(2) / 18, "d");
  }
};

// A contiguous int32 tensor.
const Tensor& indexes(PyObject* o, const char* name, c10::Device device, at::IntArrayRef shape) {
  const Tensor& t = tensor(o, name, static_cast<int64_t>(shape.size()), at::kInt);
  check(t, name, device, shape, true);
  return t;
}

// (q, k, v, seq_ids, slots, positions, block_table, kv_cache, sections, base, per_axis, k_scale, v_scale, q_out, stream)
PyObject* rope_cache_write_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 15);
  const Cache c(a[7]);
  const Tensor& q = tensor(a[0], "q", 3, at::kBFloat16);
  const Tensor& k = tensor(a[1], "k", 3, at::kBFloat16);
  const Tensor& v = tensor(a[2], "v", 3, at::kBFloat16);
  const int64_t T = q.size(0), Hq = q.size(1);
  check(q, "q", c.device, {T, Hq, c.d}, false);
  check(k, "k", c.device, {T, c.Hkv, c.d}, false);
  check(v, "v", c.device, {T, c.Hkv, c.d}, false);
  const Sections sections(a[8]);
  const Tensor& seq_ids = indexes(a[3], "seq_ids", c.device, {T});
  const Tensor& slots = indexes(a[4], "slots", c.device, {T});
  const Tensor& positions = indexes(a[5], "positions", c.device, {sections.count, T});
  const Tensor& table = indexes(a[6], "block_table", c.device, {-1, -1});
  const Target on(c.device, a[14]);
  const Tensor qo = on.output(a[13], "q_out", q.sizes(), at::kBFloat16, false);
  const int64_t strides[9] = {q.stride(0), q.stride(1),  k.stride(0),  k.stride(1), v.stride(0),
                              v.stride(1), qo.stride(0), qo.stride(1), T};
  const float base = static_cast<float>(number(a[9])), k_scale = static_cast<float>(number(a[11])),
              v_scale = static_cast<float>(number(a[12]));
  const int per_axis = truth(a[10]);
  const int iT = narrow(T, "num_tokens"), iHq = narrow(Hq, "Hq"), S = narrow(table.size(0), "num_seqs"),
            mb = narrow(table.size(1), "max_blocks_per_seq");
  on.launch("attn_rope_cache_write_fp4", [&](void* s) {
    return attn_rope_cache_write_fp4(q.const_data_ptr(), k.const_data_ptr(), v.const_data_ptr(), qo.data_ptr(),
                                     ints(seq_ids), ints(slots), ints(positions), ints(table), c.t.data_ptr(), strides,
                                     sections.size, sections.count, iT, iHq, c.Hkv, c.d, S, c.num_blocks, mb, base,
                                     per_axis, k_scale, v_scale, s);
  });
  return THPVariable_Wrap(qo);
  END_HANDLE_TH_ERRORS
}

// (kv_cache, seq_ids, slots, block_table, k_scale, v_scale, k_out, v_out, stream)
PyObject* cache_read_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 9);
  const Cache c(a[0]);
  const Tensor& seq_ids = indexes(a[1], "seq_ids", c.device, {-1});
  const int64_t T = seq_ids.size(0);
  const Tensor& slots = indexes(a[2], "slots", c.device, {T});
  const Tensor& table = indexes(a[3], "block_table", c.device, {-1, -1});
  const std::array<int64_t, 3> shape = {T, c.Hkv, c.d};
  const Target on(c.device, a[8]);
  const Tensor ko = on.output(a[6], "k_out", shape, at::kBFloat16, false);
  const Tensor vo = on.output(a[7], "v_out", shape, at::kBFloat16, false);
  const int64_t strides[4] = {ko.stride(0), ko.stride(1), vo.stride(0), vo.stride(1)};
  const float k_scale = static_cast<float>(number(a[4])), v_scale = static_cast<float>(number(a[5]));
  const int iT = narrow(T, "num_tokens"), S = narrow(table.size(0), "num_seqs"),
            mb = narrow(table.size(1), "max_blocks_per_seq");
  on.launch("attn_cache_read_fp4", [&](void* s) {
    return attn_cache_read_fp4(c.t.const_data_ptr(), ints(seq_ids), ints(slots), ints(table), ko.data_ptr(),
                               vo.data_ptr(), strides, iT, c.Hkv, c.d, S, c.num_blocks, mb, k_scale, v_scale, s);
  });
  return pair(ko, vo);
  END_HANDLE_TH_ERRORS
}

// (q, kv_cache, block_table, ctx_lens, scale, k_scale, v_scale, out, lse, workspace, return_lse, stream)
PyObject* decode_paged_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need_args(n, 12);
  const Cache c(a[1]);
  const Tensor& q = tensor(a[0], "q", 3, at::kBFloat16);
  const int64_t S = q.size(0), Hq = q.size(1);
  check(q, "q", c.device, {S, Hq, c.d}, true);
  const Tensor& table = indexes(a[2], "block_table", c.device, {S, -1});
  const Tensor& ctx_lens = indexes(a[3], "ctx_lens", c.device, {S});
  const float scale = static_cast<float>(a[4] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.d)) : number(a[4]));
  const float k_scale = static_cast<float>(number(a[5])), v_scale = static_cast<float>(number(a[6]));
  const Target on(c.device, a[11]);
  const Tensor out = on.output(a[7], "out", q.sizes(), at::kBFloat16, true);
  Tensor lse;
  if (a[8] != Py_None || truth(a[10])) lse = on.output(a[8], "lse", {S, Hq}, at::kFloat, true);
  const int iS = narrow(S, "num_seqs"), iHq = narrow(Hq, "Hq"), mb = narrow(table.size(1), "max_blocks_per_seq");
  Tensor workspace;
  size_t bytes = 0;
  if (a[9] == Py_None) {
    bytes = attn_decode_fp4_workspace_bytes(iS, iHq, c.Hkv, c.d, mb);
    if (bytes > 0) workspace = on.fresh({static_cast<int64_t>(bytes)}, at::kByte);
  } else {
    if (!THPVariable_Check(a[9])) fail(PyExc_TypeError, "workspace must be a torch.Tensor");
    workspace = THPVariable_Unpack(a[9]);
    if (workspace.device() != c.device || !workspace.is_contiguous())
      fail(PyExc_ValueError, "workspace must be contiguous on the tensors' device");
    bytes = static_cast<size_t>(workspace.numel()) * workspace.element_size();
  }
  on.launch("attn_decode_paged_fp4", [&](void* s) {
    return attn_decode_paged_fp4(q.const_data_ptr(), c.t.const_data_ptr(), ints(table), ints(ctx_lens), out.data_ptr(),
                                 lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, iS, iHq, c.Hkv, c.d,
                                 c.num_blocks, mb, scale, k_scale, v_scale,
                                 workspace.defined() ? workspace.data_ptr() : nullptr, bytes, s);
  });
  return pair(out, lse);
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_XSETREF(g_error, Py_NewRef(type));
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"rope_axes", reinterpret_cast<PyCFunction>(rope_axes), METH_FASTCALL, nullptr},
    {"rope_cache_write_fp4", reinterpret_cast<PyCFunction>(rope_cache_write_fp4), METH_FASTCALL, nullptr},
    {"cache_read_fp4", reinterpret_cast<PyCFunction>(cache_read_fp4), METH_FASTCALL, nullptr},
    {"decode_paged_fp4", reinterpret_cast<PyCFunction>(decode_paged_fp4), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
