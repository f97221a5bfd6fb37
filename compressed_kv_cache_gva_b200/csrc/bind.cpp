// Python binding of the paged serving calls (argument marshalling only).
//
// These calls take ten to twenty small tensors and run for a few microseconds on the
// GPU, so checking and unpacking the arguments in Python (about half a microsecond a
// tensor, 18 us a call in all) would cost more than the work.  This module reads the
// tensors directly and calls the C ABI of libgva.so.  A wrong tensor raises ValueError;
// otherwise the status of the call is returned.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/gva.h"

namespace {

struct Wrong {};   // a Python exception is set

[[noreturn]] void wrong(const char* name, const char* why) {
  PyErr_Format(PyExc_ValueError, "%s: %s", name, why);
  throw Wrong{};
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Wrong{};
  return v;
}

int int32_arg(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) wrong(name, "does not fit 32 bits");
  return (int)v;
}

struct Args {
  PyObject* const* o;
  int dev;

  const at::Tensor& tensor(int i, const char* name) const {
    if (!THPVariable_Check(o[i])) wrong(name, "must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o[i]);
    if (!t.is_cuda() || t.get_device() != dev) wrong(name, "must live on the current CUDA device");
    return t;
  }
  // a dense tensor of this type and shape
  template <class T = void>
  T* dense(int i, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    const at::Tensor& t = tensor(i, name);
    if (t.scalar_type() != type) wrong(name, "has another type than expected");
    if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size())) wrong(name, "has another shape than expected");
    if (!t.is_contiguous()) wrong(name, "must be contiguous");
    return static_cast<T*>(t.data_ptr());
  }
  int32_t* words(int i, const char* name, int64_t n) const { return dense<int32_t>(i, name, at::kInt, {n}); }
  int32_t* words_or_null(int i, const char* name, int64_t n) const {
    return o[i] == Py_None ? nullptr : words(i, name, n);
  }
  // a [rows, >= cols] matrix of dense, possibly strided rows
  const at::Tensor& matrix(int i, const char* name, int64_t rows, int64_t cols) const {
    const at::Tensor& t = tensor(i, name);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) < cols) wrong(name, "has another shape than expected");
    if ((t.size(1) > 1 && t.stride(1) != 1) || (t.size(0) > 1 && t.stride(0) < t.size(1)))
      wrong(name, "rows must be dense and must not overlap");
    return t;
  }
  void* stream(int i) const {
    if (o[i] != Py_None) return reinterpret_cast<void*>((uintptr_t)integer(o[i]));
    return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  }
};

int64_t row_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

template <class F>
PyObject* call(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f(Args{args, (int)c10::cuda::current_device()}));
  } catch (const Wrong&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* plan_pages(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 17, [](const Args& a) {
    const int page = int32_arg(a.o[0], "page_size"), pages = int32_arg(a.o[1], "num_pages");
    const at::Tensor& kept = a.tensor(2, "kept_len");
    const at::Tensor& slot = a.tensor(13, "slot");
    if (kept.dim() != 1) wrong("kept_len", "must have one dimension");
    if (slot.dim() != 1) wrong("slot", "must have one dimension");
    const int64_t B = kept.size(0), room = slot.size(0);
    if (B > INT32_MAX || room > INT32_MAX) wrong("kept_len, slot", "too long");
    const at::Tensor& table = a.matrix(9, "block_table", B, 1);
    if (table.scalar_type() != at::kInt) wrong("block_table", "must be int32");
    if (table.size(1) > INT32_MAX) wrong("block_table", "too wide");
    return gva_plan_pages((int)B, page, pages, (int)table.size(1), row_stride(table), (int)room,
                          a.words(2, "kept_len", B), a.words(3, "n_new", B), a.words(4, "held_in", B),
                          a.words(5, "held_out", B), a.words(6, "free_pages", pages),
                          a.words(7, "free_count_in", 1), a.words(8, "free_count_out", 1),
                          table.data_ptr<int32_t>(), a.words(10, "q_start", B + 1), a.words(11, "seq_len", B),
                          a.words(12, "n_granted", B), a.words(13, "slot", room), a.words(14, "pos", room),
                          a.words_or_null(15, "err_flag", 1), a.stream(16));
  });
}

PyObject* paged_attention(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 14, [](const Args& a) {
    Py_buffer view;
    if (PyObject_GetBuffer(a.o[0], &view, PyBUF_SIMPLE)) throw Wrong{};
    gva_shape_t sh;
    const bool whole = view.len == (Py_ssize_t)sizeof(sh);
    if (whole) memcpy(&sh, view.buf, sizeof(sh));
    PyBuffer_Release(&view);
    if (!whole) wrong("shape", "is no gva shape");
    const auto type = [](int code) { return code == GVA_F32 ? at::kFloat : at::kBFloat16; };
    const int page = int32_arg(a.o[1], "page_size");
    const at::Tensor& q = a.tensor(2, "q_abs");
    const at::Tensor& V = a.tensor(3, "V_cache");
    if (q.dim() != 3 || V.dim() != 3) wrong("q_abs, V_cache", "must have three dimensions");
    const int64_t rows = q.size(0), slots = V.size(0);
    if (rows > INT32_MAX) wrong("q_abs", "too many rows");
    const at::Tensor& table = a.matrix(5, "block_table", sh.B, 1);
    if (table.scalar_type() != at::kInt) wrong("block_table", "must be int32");
    if (table.size(1) > INT32_MAX) wrong("block_table", "too wide");
    const at::Tensor& ws = a.tensor(12, "workspace");
    if (!ws.is_contiguous()) wrong("workspace", "must be contiguous");
    return gva_paged_attention(
        &sh, page, a.dense<float>(2, "q_abs", at::kFloat, {rows, sh.H, (int64_t)sh.d_h + sh.d_r}),
        a.dense(3, "V_cache", type(sh.cache_dtype), {slots, sh.G, sh.d_h}),
        sh.d_r == 0 ? nullptr : a.dense(4, "kr_cache", type(sh.cache_dtype), {slots, sh.d_r}), slots,
        table.data_ptr<int32_t>(), (int)table.size(1), row_stride(table),
        a.words(6, "q_start", (int64_t)sh.B + 1), a.words(7, "seq_len", sh.B), (int)rows,
        int32_arg(a.o[8], "max_query_len"), integer(a.o[9]),
        a.dense(10, "out", type(sh.out_dtype), {rows, sh.H, sh.d_h}),
        a.o[11] == Py_None ? nullptr : a.dense<float>(11, "lse", at::kFloat, {rows, sh.H}), ws.data_ptr(),
        ws.nbytes(), a.stream(13));
  });
}

PyObject* verify_draft(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return call(args, n, 13, [](const Args& a) {
    const int vocab = int32_arg(a.o[0], "vocab");
    const at::Tensor& tokens = a.tensor(1, "tokens");
    const at::Tensor& us = a.tensor(6, "u_sample");
    if (tokens.dim() != 1 || us.dim() != 1) wrong("tokens, u_sample", "must have one dimension");
    const int64_t N = tokens.size(0), B = us.size(0);
    if (N > INT32_MAX || B > INT32_MAX) wrong("tokens, u_sample", "too long");
    const at::Tensor& target = a.matrix(3, "target_probs", N, vocab);
    const at::ScalarType type = target.scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) wrong("target_probs", "must be float32 or bfloat16");
    const void* draft = nullptr;
    int64_t draft_stride = 0;
    if (a.o[4] != Py_None) {
      const at::Tensor& d = a.matrix(4, "draft_probs", N, vocab);
      if (d.scalar_type() != type) wrong("draft_probs", "must have target_probs' type");
      draft = d.data_ptr();
      draft_stride = row_stride(d);
    }
    return gva_verify_draft((int)B, vocab, (int)N, a.words(1, "tokens", N), a.words(2, "q_start", B + 1),
                            type == at::kFloat ? GVA_F32 : GVA_BF16, target.data_ptr(), row_stride(target),
                            draft, draft_stride, a.dense<float>(5, "u_accept", at::kFloat, {N}),
                            a.dense<float>(6, "u_sample", at::kFloat, {B}), a.words(7, "out_tokens", N),
                            a.words(8, "n_accepted", B), a.words_or_null(9, "seq_len", B),
                            a.words_or_null(10, "kept_len", B), a.words_or_null(11, "err_flag", 1),
                            a.stream(12));
  });
}

#define GVA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GVA_METHOD(plan_pages), GVA_METHOD(paged_attention), GVA_METHOD(verify_draft),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&module); }
