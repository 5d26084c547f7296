// hybridcall.cpp -- the usual calls of the operators of hybrid stacks from Python,
// marshalled in C++, as blockcall.cpp does for the layer operators: each function
// returns the result, or the (negative) return code of the C ABI, or None where the
// tensors are not the usual ones, which hybrid.py then goes over itself.
#include "callutil.h"

#include <algorithm>
#include <cmath>
#include <utility>

namespace {

// the C ABI of libreplayssm.so, as addresses handed over by bind()
struct Abi {
  decltype(&rsm_causal_conv) conv;
  decltype(&rsm_causal_conv_step) conv_step;
  decltype(&rsm_rotary_append) rotary;
  decltype(&rsm_paged_attention) attention;
  decltype(&rsm_paged_attention_workspace) attention_workspace;
  decltype(&rsm_copy_pages) copy;
} abi;

// weight [C, W], bias [C] or nothing, fp32
bool taps(const Tensor& w, const Tensor* bias, int64_t C) {
  return w.scalar_type() == at::kFloat && w.dim() == 2 && w.size(0) == C && w.is_contiguous() && (bias == nullptr || vector(*bias, C, at::kFloat));
}

template <typename P>
void fill_conv(P& p, const Tensor& x, const Tensor& w, const Tensor* bias, int code) {
  p.x = x.data_ptr(), p.weight = w.const_data_ptr<float>(), p.bias = static_cast<const float*>(ptr(bias));
  p.channels = static_cast<int32_t>(x.size(-1)), p.width = static_cast<int32_t>(w.size(1)), p.input_dtype = code;
}

template <typename P>
bool fill_cache(P& p, const Tensor& cache, const Tensor& x) {
  if (cache.scalar_type() != x.scalar_type() || cache.dim() != 3 || cache.size(2) != x.size(-1) || !cache.is_contiguous() ||
      !fits(cache.size(0)) || !fits(cache.size(1)))
    return false;
  p.cache = cache.data_ptr(), p.cache_slot_stride = cache.stride(0);
  p.num_slots = static_cast<int32_t>(cache.size(0)), p.cache_rows = static_cast<int32_t>(cache.size(1));
  return true;
}

// conv(x, weight, cu_seqlens, bias, cache, slots, positions, silu, pad_slot_id)
PyObject* conv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 9) return none();
    const Tensor* t[7];
    for (int i = 0; i < 7; ++i) {
      t[i] = tensor(a[i]);
      if (t[i] == nullptr && !(i >= 3 && a[i] == Py_None)) return none();
    }
    const Tensor &x = *t[0], &w = *t[1], &cu = *t[2];
    const int dev = device_of(t), code = input_code(x);
    if (dev < 0 || code < 0 || x.dim() != 2 || x.size(1) < 1 || !fits(x.size(1)) || x.stride(1) != 1 || !taps(w, t[3], x.size(1))) return none();
    const int64_t seqs = cu.dim() == 1 ? cu.size(0) - 1 : -1;
    if (!fits(seqs) || !vector(cu, seqs + 1, at::kInt) || (t[4] == nullptr) != (t[5] == nullptr) || (t[6] != nullptr && t[4] == nullptr))
      return none();
    rsm_causal_conv_args p{};
    if (!int32(a[8], &p.pad_slot_id)) return none();
    p.silu = PyObject_IsTrue(a[7]);
    if (p.silu < 0) throw 0;
    if (t[4] != nullptr) {
      if (!fill_cache(p, *t[4], x) || !vector(*t[5], seqs, at::kInt) || (t[6] != nullptr && !vector(*t[6], seqs, at::kInt))) return none();
      p.slots = t[5]->const_data_ptr<int32_t>(), p.positions = static_cast<const int32_t*>(ptr(t[6]));
    }
    const Tensor out = like(x);
    fill_conv(p, x, w, t[3], code);
    p.cu_seqlens = cu.const_data_ptr<int32_t>(), p.num_seqs = static_cast<int32_t>(seqs);
    p.tokens = x.size(0), p.x_stride = x.stride(0), p.out_stride = x.size(1), p.out = out.data_ptr();
    const int rc = abi.conv(&p, c10::cuda::getCurrentCUDAStream(dev).stream());
    return rc != 0 ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
  });
}

// conv_step(x, weight, cache, slots, positions, bias, silu, pad_slot_id)
PyObject* conv_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 8) return none();
    const Tensor* t[6];
    for (int i = 0; i < 6; ++i) {
      t[i] = tensor(a[i]);
      if (t[i] == nullptr && !(i == 5 && a[i] == Py_None)) return none();
    }
    const Tensor &x = *t[0], &w = *t[1];
    const int dev = device_of(t), code = input_code(x), k = static_cast<int>(x.dim()) - 1;
    if (dev < 0 || code < 0 || (k != 1 && k != 2) || x.size(k) < 1 || !fits(x.size(k)) || x.stride(k) != 1 || !fits(x.size(0)) ||
        !fits(x.size(1)) || !taps(w, t[5], x.size(k)))
      return none();
    rsm_causal_conv_step_args p{};
    if (!fill_cache(p, *t[2], x) || !vector(*t[3], x.size(0), at::kInt) || !vector(*t[4], x.size(0), at::kInt) || !int32(a[7], &p.pad_slot_id))
      return none();
    p.silu = PyObject_IsTrue(a[6]);
    if (p.silu < 0) throw 0;
    const Tensor out = like(x);
    fill_conv(p, x, w, t[5], code);
    p.slots = t[3]->const_data_ptr<int32_t>(), p.positions = t[4]->const_data_ptr<int32_t>(), p.out = out.data_ptr();
    p.batch = static_cast<int32_t>(x.size(0)), p.window = k == 2 ? static_cast<int32_t>(x.size(1)) : 1;
    p.x_batch_stride = x.stride(0), p.x_stride = k == 2 ? x.stride(1) : 0;
    const int rc = abi.conv_step(&p, c10::cuda::getCurrentCUDAStream(dev).stream());
    return rc != 0 ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
  });
}

// No two rows of pages [pages, page_size, heads, dim] share memory, whatever their order.
bool apart(const Tensor& t, int64_t need) {
  std::pair<int64_t, int64_t> d[3];
  for (int i = 0; i < 3; ++i) d[i] = {t.stride(i), t.size(i)};
  std::sort(d, d + 3);
  for (const auto& [stride, n] : d) {
    if (n < 2) continue;
    if (stride < need) return false;
    need = stride * n;
  }
  return true;
}

// The pages of `b` requests for heads of x's type and size `dim`.
bool fill_pages(rsm_pages& g, const Tensor& k, const Tensor& v, const Tensor& table, const Tensor& lengths, const Tensor& x, int64_t b) {
  const int64_t dim = x.size(-1);
  if (k.scalar_type() != x.scalar_type() || v.scalar_type() != x.scalar_type() || k.dim() != 4 || v.sizes() != k.sizes() || k.size(3) != dim ||
      k.stride(3) != 1 || v.stride(3) != 1 || !fits(k.size(0)) || !fits(k.size(1)) || !fits(k.size(2)))
    return false;
  if (!apart(k, dim) || !apart(v, dim)) return false;
  if (table.scalar_type() != at::kInt || table.dim() != 2 || table.size(0) != b || !fits(b) || !fits(table.size(1)) ||
      (table.size(1) > 1 && table.stride(1) != 1) || !vector(lengths, b, at::kInt))
    return false;
  g.k = k.data_ptr(), g.v = v.data_ptr();
  g.page_table = table.const_data_ptr<int32_t>(), g.lengths = lengths.const_data_ptr<int32_t>();
  g.k_page_stride = k.stride(0), g.k_row_stride = k.stride(1), g.k_head_stride = k.stride(2);
  g.v_page_stride = v.stride(0), g.v_row_stride = v.stride(1), g.v_head_stride = v.stride(2);
  g.table_stride = table.stride(0);
  g.requests = static_cast<int32_t>(b), g.table_width = static_cast<int32_t>(table.size(1));
  g.num_pages = static_cast<int32_t>(k.size(0)), g.page_size = static_cast<int32_t>(k.size(1));
  return true;
}

// [lead.., heads, dim] with contiguous heads
bool heads(const Tensor& t, int k) {
  return t.dim() == k + 2 && fits(t.size(k)) && fits(t.size(k + 1)) && t.stride(k + 1) == 1 && t.stride(k) == t.size(k + 1);
}

// rotary(q, k, v, inv_freq, k_cache, v_cache, page_table, lengths, cu_seqlens or None, interleaved, amplitude)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 11) return none();
    const Tensor* t[9];
    for (int i = 0; i < 9; ++i) {
      t[i] = tensor(a[i]);
      if (t[i] == nullptr && !(i == 8 && a[i] == Py_None)) return none();
    }
    const Tensor &q = *t[0], &k = *t[1], &v = *t[2], &f = *t[3];
    const int dev = device_of(t), code = input_code(q), lead = static_cast<int>(q.dim()) - 2;
    if (dev < 0 || code < 0 || lead < 1 || lead > (t[8] == nullptr ? 2 : 1) || !heads(q, lead) || !heads(k, lead) || !heads(v, lead) ||
        k.sizes() != v.sizes() || k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type() || k.size(-1) != q.size(-1) ||
        t[4]->dim() != 4 || t[4]->size(2) != k.size(-2))
      return none();
    for (int i = 0; i < lead; ++i)
      if (q.size(i) != k.size(i) || !fits(q.size(i))) return none();
    if (f.dim() != 1 || !vector(f, f.size(0), at::kFloat) || 2 * f.size(0) > q.size(-1)) return none();
    rsm_rotary_append_args p{};
    int64_t b = q.size(0);
    if (t[8] != nullptr) {
      b = t[8]->dim() == 1 ? t[8]->size(0) - 1 : -1;
      if (b < 0 || !vector(*t[8], b + 1, at::kInt)) return none();
      p.cu_seqlens = t[8]->const_data_ptr<int32_t>();
      p.tokens = q.size(0);
      p.q_stride = q.stride(0), p.k_stride = k.stride(0), p.v_stride = v.stride(0);
    } else {
      p.window = lead == 2 ? static_cast<int32_t>(q.size(1)) : 1;
      p.q_batch_stride = q.stride(0), p.k_batch_stride = k.stride(0), p.v_batch_stride = v.stride(0);
      if (lead == 2) p.q_stride = q.stride(1), p.k_stride = k.stride(1), p.v_stride = v.stride(1);
    }
    if (!fill_pages(p.pages, *t[4], *t[5], *t[6], *t[7], q, b)) return none();
    p.interleaved = PyObject_IsTrue(a[9]);
    p.amplitude = static_cast<float>(PyFloat_AsDouble(a[10]));
    if (PyErr_Occurred()) throw 0;
    const Tensor out = like(q);
    p.q = q.data_ptr(), p.k = k.data_ptr(), p.v = v.data_ptr(), p.inv_freq = f.const_data_ptr<float>(), p.q_out = out.data_ptr();
    p.num_heads = static_cast<int32_t>(q.size(-2)), p.num_kv_heads = static_cast<int32_t>(k.size(-2)), p.dim = static_cast<int32_t>(q.size(-1));
    p.rotary_dim = static_cast<int32_t>(2 * f.size(0)), p.input_dtype = code;
    p.out_stride = q.size(-2) * q.size(-1), p.out_batch_stride = p.out_stride * p.window;
    const int rc = abi.rotary(&p, c10::cuda::getCurrentCUDAStream(dev).stream());
    return rc != 0 ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
  });
}

// attention(q, k_cache, v_cache, page_table, lengths, scale or None)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6) return none();
    const Tensor* t[5];
    for (int i = 0; i < 5; ++i) {
      t[i] = tensor(a[i]);
      if (t[i] == nullptr) return none();
    }
    const Tensor& q = *t[0];
    const int dev = device_of(t), code = input_code(q), lead = static_cast<int>(q.dim()) - 2;
    rsm_paged_attention_args p{};
    if (dev < 0 || code < 0 || (lead != 1 && lead != 2) || !heads(q, lead) || q.size(-1) < 1 || !fits(q.size(0)) || !fits(q.size(1)) ||
        !fill_pages(p.pages, *t[1], *t[2], *t[3], *t[4], q, q.size(0)))
      return none();
    p.scale = a[5] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(q.size(-1)))) : static_cast<float>(PyFloat_AsDouble(a[5]));
    if (PyErr_Occurred()) throw 0;
    p.window = lead == 2 ? static_cast<int32_t>(q.size(1)) : 1;
    p.q_batch_stride = q.stride(0), p.q_stride = lead == 2 ? q.stride(1) : 0;
    p.num_heads = static_cast<int32_t>(q.size(-2)), p.num_kv_heads = static_cast<int32_t>(t[1]->size(2));
    p.dim = static_cast<int32_t>(q.size(-1)), p.input_dtype = code;
    p.q = q.data_ptr();
    const int64_t bytes = abi.attention_workspace(&p);
    if (bytes < 0) return PyLong_FromLongLong(bytes);
    const Tensor out = like(q);
    Tensor workspace;
    if (bytes > 0) {
      workspace = at::empty({bytes}, q.options().dtype(at::kByte));
      p.workspace = workspace.data_ptr(), p.workspace_bytes = bytes;
    }
    p.out = out.data_ptr();
    const int rc = abi.attention(&p, c10::cuda::getCurrentCUDAStream(dev).stream());
    return rc != 0 ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
  });
}

// copy(page_ptrs, page_strides, src_pages, dst_pages, dtype code, page_elements, num_pages): 0, a return code or None
PyObject* copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 7) return none();
    const Tensor* t[4];
    for (int i = 0; i < 4; ++i) {
      t[i] = tensor(a[i]);
      if (t[i] == nullptr || t[i]->dim() != 1 || !fits(t[i]->size(0))) return none();
    }
    const int dev = device_of(t);
    rsm_copy_pages_args p{};
    if (dev < 0 || !vector(*t[0], t[0]->size(0), at::kLong) || !vector(*t[1], t[0]->size(0), at::kLong) ||
        !vector(*t[2], t[2]->size(0), at::kInt) || !vector(*t[3], t[2]->size(0), at::kInt) || !int32(a[4], &p.dtype) || !int32(a[6], &p.num_pages))
      return none();
    p.page_elements = PyLong_AsLongLong(a[5]);
    if (PyErr_Occurred()) throw 0;
    p.page_ptrs = t[0]->const_data_ptr<int64_t>(), p.page_strides = t[1]->const_data_ptr<int64_t>();
    p.src_pages = t[2]->const_data_ptr<int32_t>(), p.dst_pages = t[3]->const_data_ptr<int32_t>();
    p.num_pools = static_cast<int32_t>(t[0]->size(0)), p.num_pairs = static_cast<int32_t>(t[2]->size(0));
    return PyLong_FromLong(abi.copy(&p, c10::cuda::getCurrentCUDAStream(dev).stream()));
  });
}

// bind(six addresses of the C ABI, in Abi's order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* at[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "six addresses are needed");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (at[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is NULL");
      return nullptr;
    }
  }
  abi.conv = reinterpret_cast<decltype(abi.conv)>(at[0]);
  abi.conv_step = reinterpret_cast<decltype(abi.conv_step)>(at[1]);
  abi.rotary = reinterpret_cast<decltype(abi.rotary)>(at[2]);
  abi.attention = reinterpret_cast<decltype(abi.attention)>(at[3]);
  abi.attention_workspace = reinterpret_cast<decltype(abi.attention_workspace)>(at[4]);
  abi.copy = reinterpret_cast<decltype(abi.copy)>(at[5]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {FAST(bind), FAST(conv), FAST(conv_step), FAST(rotary), FAST(attention), FAST(copy), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hybridcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hybridcall() { return PyModule_Create(&module); }
