// Python binding of the calls on the paged store whose work takes the device
// a few microseconds: one pass over the tensors in C++, outputs and launch
// from there (in Python the checks, allocations and argument conversion of a
// plan took 18 us of the host, here 8.6, and 6.4 with one allocation for
// its four outputs).  Everything runs on the current stream
// of the tensors' device; a failing status of the C ABI is returned as an
// int.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/sdk.h"

namespace {

const char* const kTypeNames[] = {"torch.int32", "torch.int64", "torch.bfloat16", "torch.float32",
                                  "torch.uint8"};
enum Type { kI32, kI64, kBF16, kF32, kU8 };
constexpr at::ScalarType kTypes[] = {at::kInt, at::kLong, at::kBFloat16, at::kFloat, at::kByte};

// The arguments of one call, all on the device of the first tensor.
class Call {
 public:
  explicit Call(PyObject* const* args) : args_(args) {}

  const at::Tensor& tensor(int i, const char* name, Type type, int64_t dims = -1) {
    PyObject* o = args_[i];
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a CUDA tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_VALUE(t.scalar_type() == kTypes[type], name, " has dtype ", t.dtype().name(),
                      ", expected ", kTypeNames[type]);
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
    if (!guard_.current_device().has_value()) guard_.set_device(t.device());
    TORCH_CHECK_VALUE(t.device() == *guard_.current_device(), name, " is on ", t.device(),
                      ", the other tensors on ", *guard_.current_device());
    TORCH_CHECK_VALUE(dims < 0 || t.dim() == dims, name, " has ", t.dim(), " dimensions, expected ",
                      dims);
    return t;
  }
  bool given(int i) const { return args_[i] != Py_None; }
  // a given output, or a new one
  at::Tensor output(int i, const char* name, Type type, at::IntArrayRef shape) {
    if (!given(i)) return at::empty(shape, options(type));
    const at::Tensor& t = tensor(i, name, type);
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
    return t;
  }
  // Outputs that lie in one new buffer: added in turn (0 bytes where the
  // caller gives the tensor), then cut from it.
  int64_t add(int i, Type type, int64_t n) {
    const int64_t at = bytes_;
    if (!given(i)) bytes_ += (n * (int64_t)c10::elementSize(kTypes[type]) + 15) / 16 * 16;
    return at;
  }
  at::Tensor piece(int i, const char* name, Type type, int64_t n, int64_t at) {
    if (given(i)) return output(i, name, type, {n});
    if (!buffer_.defined()) buffer_ = at::empty({bytes_}, options(kU8));
    at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
        c10::Storage(buffer_.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
        c10::scalarTypeToTypeMeta(kTypes[type]));
    t.unsafeGetTensorImpl()->set_storage_offset(at / (int64_t)c10::elementSize(kTypes[type]));
    t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
    return t;
  }
  // a given workspace, or a new one of `bytes`
  at::Tensor workspace(int i, size_t bytes) {
    if (given(i)) return tensor(i, "workspace", kU8);
    at::Tensor ws = at::empty({(int64_t)std::max<size_t>(bytes, 256)}, options(kU8));
    status = sdk_workspace_init(ws.data_ptr(), (size_t)ws.numel(), stream());
    return ws;
  }
  int64_t integer(int i, const char* name) {
    const long long v = PyLong_AsLongLong(args_[i]);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
  }
  int32_t int32(int i, const char* name) {
    const int64_t v = integer(i, name);
    TORCH_CHECK_VALUE(v == (int32_t)v, name, " = ", v, " does not fit 32 bits");
    return (int32_t)v;
  }
  sdk_stream_t stream() const {
    return reinterpret_cast<sdk_stream_t>(
        c10::cuda::getCurrentCUDAStream(guard_.current_device()->index()).stream());
  }
  int status = SDK_OK;

 private:
  at::TensorOptions options(Type type) const {
    return at::TensorOptions().dtype(kTypes[type]).device(*guard_.current_device());
  }
  PyObject* const* args_;
  int64_t bytes_ = 0;
  at::Tensor buffer_;
  c10::cuda::OptionalCUDAGuard guard_;
};

int32_t narrow(int64_t v, const char* what) {
  TORCH_CHECK_VALUE(v == (int32_t)v, what, " ", v, " does not fit 32 bits");
  return (int32_t)v;
}

void check_pages(const at::Tensor& pages) {
  TORCH_CHECK_VALUE(pages.dim() == 5 && pages.size(3) == 2 && pages.size(4) == SDK_K_ATOMS,
                    "pages must be [n_pages, Hkv, page_size, 2, 16]");
}

void check_count(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}

// lens, n_new, free_pages, n_free, block_table, page_size, max_new, n_pages,
// slot_map, cu_new, new_lens, n_free_out, workspace, and whether n_free itself
// holds the new count afterwards (a copy: the plan's CTAs read n_free until
// they end)
PyObject* block_tables(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count(n, 14);
  Call c(args);
  const at::Tensor& lens = c.tensor(0, "lens", kI32, 1);
  const at::Tensor& n_new = c.tensor(1, "n_new", kI32, 1);
  const at::Tensor& stack = c.tensor(2, "free_pages", kI32, 1);
  const at::Tensor& n_free = c.tensor(3, "n_free", kI32);
  const at::Tensor& table = c.tensor(4, "block_table", kI32, 2);
  const int64_t B = lens.size(0), max_new = c.integer(6, "max_new");
  TORCH_CHECK_VALUE(n_new.size(0) == B && table.size(0) == B && n_free.numel() == 1,
                    "lens and n_new are [B], block_table is [B, max_pages], n_free [1]");
  TORCH_CHECK_VALUE(max_new >= 0, "max_new is negative");
  const int64_t n_pages = c.given(7) ? c.integer(7, "n_pages") : stack.size(0);
  TORCH_CHECK_VALUE(max_new <= 0x7FFFFFFF, "max_new ", max_new, " does not fit 32 bits");
  const int64_t at_slots = c.add(8, kI64, max_new), at_cu = c.add(9, kI32, B + 1),
                at_lens = c.add(10, kI32, B), at_left = c.add(11, kI32, 1);
  const at::Tensor slots = c.piece(8, "slot_map", kI64, max_new, at_slots);
  const at::Tensor cu = c.piece(9, "cu_new", kI32, B + 1, at_cu);
  const at::Tensor new_lens = c.piece(10, "new_lens", kI32, B, at_lens);
  const at::Tensor left = c.piece(11, "n_free_out", kI32, 1, at_left);
  const at::Tensor ws = c.workspace(12, sdk_block_tables_workspace_bytes(narrow(B, "B")));
  if (c.status == SDK_OK)
    c.status = sdk_block_tables(
        (const int32_t*)lens.data_ptr(), (const int32_t*)n_new.data_ptr(), narrow(B, "B"),
        (const int32_t*)stack.data_ptr(), narrow(stack.size(0), "stack of"),
        (const int32_t*)n_free.data_ptr(), narrow(n_pages, "n_pages"), c.int32(5, "page_size"),
        (int32_t*)table.data_ptr(), narrow(table.size(1), "max_pages"), max_new,
        (int64_t*)slots.data_ptr(), (int32_t*)cu.data_ptr(), (int32_t*)new_lens.data_ptr(),
        (int32_t*)left.data_ptr(), ws.data_ptr(), (size_t)ws.numel(), c.stream());
  if (c.status == SDK_OK && args[13] == Py_True &&
      cudaMemcpyAsync(n_free.data_ptr(), left.data_ptr(), 4, cudaMemcpyDeviceToDevice,
                      reinterpret_cast<cudaStream_t>(c.stream())) != cudaSuccess)
    c.status = SDK_ERR_CUDA;
  if (c.status != SDK_OK) return PyLong_FromLong(c.status);
  PyObject* r = PyTuple_New(5);
  Py_INCREF(args[4]);
  PyTuple_SET_ITEM(r, 0, args[4]);
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(slots));
  PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(cu));
  PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(new_lens));
  PyTuple_SET_ITEM(r, 4, THPVariable_Wrap(left));
  return r;
  END_HANDLE_TH_ERRORS
}

// pages, codes_k, codes_v, slot_map, workspace
PyObject* paged_store(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count(n, 5);
  Call c(args);
  const at::Tensor& pages = c.tensor(0, "pages", kI32);
  check_pages(pages);
  const at::Tensor& k = c.tensor(1, "codes_k", kI32);
  const at::Tensor& v = c.tensor(2, "codes_v", kI32);
  const at::Tensor& slots = c.tensor(3, "slot_map", kI64);
  const int64_t n_tok = slots.numel(), words = n_tok * pages.size(1) * SDK_K_ATOMS;
  TORCH_CHECK_VALUE(k.numel() == words && v.numel() == words && k.dim() > 0 && v.dim() > 0 &&
                        k.size(-1) == SDK_K_ATOMS && v.size(-1) == SDK_K_ATOMS,
                    "codes_k and codes_v must hold 16 words of ", pages.size(1), " heads for ", n_tok,
                    " tokens");
  const at::Tensor ws = c.workspace(4, sdk_paged_store_workspace_bytes());
  if (c.status == SDK_OK)
    c.status = sdk_paged_store((const uint32_t*)k.data_ptr(), (const uint32_t*)v.data_ptr(), n_tok,
                               narrow(pages.size(1), "Hkv"), (const int64_t*)slots.data_ptr(),
                               (uint32_t*)pages.data_ptr(), narrow(pages.size(0), "n_pages"),
                               narrow(pages.size(2), "page_size"), ws.data_ptr(),
                               (size_t)ws.numel(), c.stream());
  if (c.status != SDK_OK) return PyLong_FromLong(c.status);
  Py_INCREF(args[0]);
  return args[0];
  END_HANDLE_TH_ERRORS
}

// q, dict_k, dict_v, pages, block_table, lens, cu_q, max_q, max_len,
// total_len, causal, window, scale, out, lse, workspace
PyObject* chunk_attn(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  check_count(n, 16);
  Call c(args);
  const at::Tensor& q = c.tensor(0, "q", kBF16, 3);
  const at::Tensor& dk = c.tensor(1, "dict_k", kBF16, 2);
  const at::Tensor& dv = c.tensor(2, "dict_v", kBF16, 2);
  const at::Tensor& pages = c.tensor(3, "pages", kI32);
  check_pages(pages);
  const at::Tensor& table = c.tensor(4, "block_table", kI32, 2);
  const at::Tensor& lens = c.tensor(5, "lens", kI32, 1);
  const at::Tensor& cu = c.tensor(6, "cu_q", kI32, 1);
  const int64_t n_tok = q.size(0), B = lens.size(0), d = q.size(2);
  TORCH_CHECK_VALUE(dk.size(1) == d && dv.sizes() == dk.sizes(), "dict_k and dict_v are [n_atoms, ",
                    d, "]");
  TORCH_CHECK_VALUE(table.size(0) == B && cu.size(0) == B + 1,
                    "lens is [B], block_table [B, max_pages], cu_q [B + 1]");
  const double scale =
      c.given(12) ? PyFloat_AsDouble(args[12]) : 1.0 / std::sqrt((double)std::max<int64_t>(d, 1));
  if (PyErr_Occurred()) throw python_error();
  const int causal = PyObject_IsTrue(args[10]);
  if (causal < 0) throw python_error();
  const int32_t Hq = narrow(q.size(1), "Hq"), Hkv = narrow(pages.size(1), "Hkv"),
                n_atoms = narrow(dk.size(0), "n_atoms"), max_q = c.int32(7, "max_q"),
                max_len = c.int32(8, "max_len");
  const int64_t total = c.integer(9, "total_len");
  const at::Tensor out = c.output(13, "out", kBF16, q.sizes());
  float* lse = nullptr;
  if (c.given(14)) lse = (float*)c.output(14, "lse", kF32, {n_tok, q.size(1)}).data_ptr();
  const at::Tensor ws =
      c.workspace(15, c.given(15) ? 0
                                  : sdk_chunk_attn_workspace_bytes(narrow(B, "B"), n_tok, Hq, Hkv,
                                                                   narrow(d, "head_dim"), n_atoms,
                                                                   max_q, max_len, total));
  if (c.status == SDK_OK)
    c.status = sdk_chunk_attn(
        q.data_ptr(), n_tok, narrow(B, "B"), Hq, Hkv, narrow(d, "head_dim"), dk.data_ptr(),
        dv.data_ptr(), n_atoms, (const uint32_t*)pages.data_ptr(), narrow(pages.size(0), "n_pages"),
        narrow(pages.size(2), "page_size"), (const int32_t*)table.data_ptr(),
        narrow(table.size(1), "max_pages"), (const int32_t*)lens.data_ptr(),
        (const int32_t*)cu.data_ptr(), max_q, max_len, total, c.int32(11, "window"),
        causal ? SDK_CHUNK_CAUSAL : 0, (float)scale, out.data_ptr(), lse, ws.data_ptr(),
        (size_t)ws.numel(), c.stream());
  if (c.status != SDK_OK) return PyLong_FromLong(c.status);
  if (!c.given(13)) return THPVariable_Wrap(out);
  Py_INCREF(args[13]);
  return args[13];
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"block_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(block_tables)),
     METH_FASTCALL, nullptr},
    {"paged_store", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_store)),
     METH_FASTCALL, nullptr},
    {"chunk_attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(chunk_attn)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
