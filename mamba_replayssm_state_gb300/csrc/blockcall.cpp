// blockcall.cpp -- the layer operators' usual calls from Python, marshalled in
// C++: a decoding batch makes several of them a layer, and in Python their checks
// cost more than their kernels.
//
// Each function takes the call's tensors, and returns the result, or the (negative)
// return code of the C ABI, or None where the tensors are not the usual ones (another
// type, shape, stride or device than the kernels take as they are, or anything
// wrong): block.py then goes over them itself and names what is wrong or lets it
// pass.  So nothing here raises, and nothing is accepted that block.py refuses.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/replayssm_block.h"

namespace {

// the C ABI of libreplayssm.so, as addresses handed over by bind()
struct Abi {
  decltype(&rsm_ssm_prefill) prefill;
  decltype(&rsm_ssm_prefill_workspace) prefill_workspace;
  decltype(&rsm_ssm_step) step;
  decltype(&rsm_replayssm_decode) decode;
  decltype(&rsm_add_rms_norm) add_norm;
  decltype(&rsm_gated_rms_norm) gated_norm;
} abi;

using Tensor = at::Tensor;

PyObject* none() { Py_RETURN_NONE; }

// The tensor, or nullptr for anything else.
const Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// All tensors on the current device, and none wants a gradient (nullptr: not given); its index, or -1.
template <int N>
int device_of(const Tensor* const (&ts)[N]) {
  const int d = c10::cuda::current_device();
  const bool grad = c10::GradMode::is_enabled();
  for (const Tensor* t : ts)
    if (t != nullptr && !(t->is_cuda() && t->get_device() == d && !(grad && t->requires_grad()))) return -1;
  return d;
}

int input_code(const Tensor& t) {
  const auto s = t.scalar_type();
  return s == at::kBFloat16 ? RSM_BF16 : s == at::kFloat ? RSM_F32 : -1;
}

int state_code(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return RSM_F32;
    case at::kBFloat16: return RSM_BF16;
    case at::kHalf: return RSM_F16;
    case at::kChar: return RSM_I8;
    case at::kFloat8_e4m3fn: return RSM_FP8_E4M3;
    default: return -1;
  }
}

// contiguous [n] of a type
bool vector(const Tensor& t, int64_t n, at::ScalarType type) {
  return t.scalar_type() == type && t.dim() == 1 && t.size(0) == n && (n <= 1 || t.stride(0) == 1);
}

bool is(const Tensor& t, at::IntArrayRef sizes, at::ScalarType type) {
  return t.scalar_type() == type && t.sizes() == sizes && t.is_contiguous();
}

bool fits(int64_t v) { return v >= 0 && v <= 0x7FFFFFFF; }

// a Python integer of 32 bits
bool int32(PyObject* o, int32_t* v) {
  const long long n = PyLong_AsLongLong(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  *v = static_cast<int32_t>(n);
  return *v == n;
}

// x [lead.., H, dim], dt [lead.., H], A [H], B and C [lead.., G, N], D [H] or
// nothing, with `k` leading dimensions and contiguous inner ones.
struct Tokens {
  int code, H, G, dim, N;
  bool read(const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& B, const Tensor& C, const Tensor* D, int k) {
    code = input_code(x);
    if (code < 0 || x.dim() != k + 2 || B.dim() != k + 2 || dt.dim() != k + 1 || B.sizes() != C.sizes()) return false;
    if (B.scalar_type() != x.scalar_type() || C.scalar_type() != x.scalar_type() || dt.scalar_type() != at::kFloat) return false;
    for (int i = 0; i < k; ++i)
      if (B.size(i) != x.size(i) || dt.size(i) != x.size(i)) return false;
    const int64_t h = x.size(k), d = x.size(k + 1), g = B.size(k), n = B.size(k + 1);
    if (!fits(h) || !fits(d) || !fits(g) || !fits(n)) return false;
    H = static_cast<int>(h), dim = static_cast<int>(d), G = static_cast<int>(g), N = static_cast<int>(n);
    return dt.size(k) == h && dt.stride(k) == 1 && vector(A, h, at::kFloat) && (D == nullptr || vector(*D, h, at::kFloat)) &&
           x.stride(k + 1) == 1 && x.stride(k) == d && B.stride(k + 1) == 1 && B.stride(k) == n && C.stride(k + 1) == 1 &&
           C.stride(k) == n;
  }
};

// a pool [slots, H, dim, N] with contiguous slots, laid out without gaps
bool pool(const Tensor& t, const Tokens& k) {
  return t.dim() == 4 && t.is_contiguous() && t.size(1) == k.H && t.size(2) == k.dim && t.size(3) == k.N && fits(t.size(0));
}

void* ptr(const Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

Tensor like(const Tensor& x) { return at::empty(x.sizes(), x.options()); }

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {  // block.py meets the same, and says so
    PyErr_Clear();
    return none();
  }
}

// prefill(x, dt, A, B, C, cu_seqlens, state, initial_slots, final_slots, D, pad_slot_id)
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 11) return none();
    const Tensor *x = tensor(a[0]), *dt = tensor(a[1]), *A = tensor(a[2]), *B = tensor(a[3]), *C = tensor(a[4]), *cu = tensor(a[5]),
                 *state = tensor(a[6]), *initial = tensor(a[7]), *final_ = tensor(a[8]), *D = tensor(a[9]);
    if (!x || !dt || !A || !B || !C || !cu || (!state && a[6] != Py_None) || (!initial && a[7] != Py_None) ||
        (!final_ && a[8] != Py_None) || (!D && a[9] != Py_None))
      return none();
    const Tensor* const all[] = {x, dt, A, B, C, cu, state, initial, final_, D};
    const int dev = device_of(all);
    Tokens k;
    if (dev < 0 || !k.read(*x, *dt, *A, *B, *C, D, 1)) return none();
    const int64_t seqs = cu->dim() == 1 ? cu->size(0) - 1 : -1;
    if (!fits(seqs) || !vector(*cu, seqs + 1, at::kInt)) return none();
    if ((initial && !vector(*initial, seqs, at::kInt)) || (final_ && !vector(*final_, seqs, at::kInt))) return none();
    rsm_ssm_prefill_args p{};
    p.state_dtype = RSM_F32;
    if (state) {
      p.state_dtype = state_code(*state);
      if (p.state_dtype < 0 || !pool(*state, k)) return none();
      p.state = state->data_ptr();
      p.state_slot_stride = state->stride(0);
      p.num_slots = static_cast<int32_t>(state->size(0));
    } else if (initial || final_) {
      return none();
    }
    int32_t pad;
    if (!int32(a[10], &pad)) return none();
    const Tensor out = like(*x);
    p.x = x->data_ptr(), p.B = B->data_ptr(), p.C = C->data_ptr();
    p.dt = dt->const_data_ptr<float>(), p.A = A->const_data_ptr<float>(), p.D = static_cast<const float*>(ptr(D));
    p.cu_seqlens = cu->const_data_ptr<int32_t>();
    p.initial_slots = static_cast<const int32_t*>(ptr(initial)), p.final_slots = static_cast<const int32_t*>(ptr(final_));
    p.out = out.data_ptr();
    p.tokens = x->size(0);
    p.x_stride = x->stride(0), p.B_stride = B->stride(0), p.C_stride = C->stride(0), p.dt_stride = dt->stride(0);
    p.out_stride = static_cast<int64_t>(k.H) * k.dim;
    p.num_seqs = static_cast<int32_t>(seqs), p.num_heads = k.H, p.num_groups = k.G, p.dim = k.dim, p.dstate = k.N;
    p.input_dtype = k.code, p.pad_slot_id = pad;
    const int64_t bytes = abi.prefill_workspace(&p);
    if (bytes < 0) return PyLong_FromLongLong(bytes);
    Tensor workspace;
    if (bytes > 0) {
      workspace = at::empty({bytes}, x->options().dtype(at::kByte));
      p.workspace = workspace.data_ptr();
      p.workspace_bytes = bytes;
    }
    const int rc = abi.prefill(&p, c10::cuda::getCurrentCUDAStream(dev).stream());
    return rc != 0 ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
  });
}

// What a step and a ring decode share; x [batch, window, H, dim], or without the window.
template <typename P>
bool batch(P& p, Tokens& k, const Tensor& x, const Tensor& dt, const Tensor& A, const Tensor& B, const Tensor& C, const Tensor* D) {
  const int lead = static_cast<int>(x.dim()) - 2;
  if ((lead != 1 && lead != 2) || !k.read(x, dt, A, B, C, D, lead) || !fits(x.size(0)) || (lead == 2 && !fits(x.size(1)))) return false;
  p.x = x.data_ptr(), p.B = B.data_ptr(), p.C = C.data_ptr();
  p.dt = dt.const_data_ptr<float>(), p.A = A.const_data_ptr<float>(), p.D = static_cast<const float*>(ptr(D));
  p.x_batch_stride = x.stride(0), p.B_batch_stride = B.stride(0), p.C_batch_stride = C.stride(0), p.dt_batch_stride = dt.stride(0);
  if (lead == 2) p.x_stride = x.stride(1), p.B_stride = B.stride(1), p.C_stride = C.stride(1), p.dt_stride = dt.stride(1);
  p.batch = static_cast<int32_t>(x.size(0)), p.window = lead == 2 ? static_cast<int32_t>(x.size(1)) : 1;
  p.num_heads = k.H, p.num_groups = k.G, p.dim = k.dim, p.dstate = k.N, p.input_dtype = k.code;
  return true;
}

// step(state, slots, x, dt, A, B, C, dst_slots, D, pad_slot_id)
PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 10) return none();
    const Tensor *state = tensor(a[0]), *slots = tensor(a[1]), *x = tensor(a[2]), *dt = tensor(a[3]), *A = tensor(a[4]),
                 *B = tensor(a[5]), *C = tensor(a[6]), *dst = tensor(a[7]), *D = tensor(a[8]);
    if (!state || !slots || !x || !dt || !A || !B || !C || (!dst && a[7] != Py_None) || (!D && a[8] != Py_None)) return none();
    const Tensor* const all[] = {state, slots, x, dt, A, B, C, dst, D};
    const int dev = device_of(all);
    rsm_ssm_step_args p{};
    Tokens k;
    if (dev < 0 || !batch(p, k, *x, *dt, *A, *B, *C, D)) return none();
    p.state_dtype = state_code(*state);
    if (p.state_dtype < 0 || !pool(*state, k) || !vector(*slots, p.batch, at::kInt) || (dst && !vector(*dst, p.batch, at::kInt)))
      return none();
    int32_t pad;
    if (!int32(a[9], &pad)) return none();
    const Tensor out = like(*x);
    p.state = state->data_ptr(), p.src_slots = slots->const_data_ptr<int32_t>(), p.dst_slots = static_cast<const int32_t*>(ptr(dst));
    p.out = out.data_ptr();
    p.state_slot_stride = state->stride(0), p.num_slots = static_cast<int32_t>(state->size(0));
    p.pad_slot_id = pad;
    const int rc = abi.step(&p, c10::cuda::getCurrentCUDAStream(dev).stream());
    return rc != 0 ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
  });
}

// decode(state, slots, x_cache, B_cache, dt_cache, ring_start, ring_len, x, dt, A, B, C, state_scale, D, pad_slot_id)
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 15) return none();
    const Tensor* t[14];
    for (int i = 0; i < 14; ++i) {
      t[i] = tensor(a[i]);
      if (t[i] == nullptr && !(i >= 12 && a[i] == Py_None)) return none();
    }
    const Tensor &state = *t[0], &xc = *t[2], &Bc = *t[3], &dtc = *t[4], &x = *t[7];
    const int dev = device_of(t);
    rsm_replayssm_decode_args p{};
    Tokens k;
    if (dev < 0 || !batch(p, k, x, *t[8], *t[9], *t[10], *t[11], t[13])) return none();
    p.state_dtype = state_code(state);
    if (p.state_dtype < 0 || !pool(state, k) || xc.dim() != 4 || !fits(xc.size(1))) return none();
    const int64_t S = state.size(0), R = xc.size(1);
    if (!is(xc, {S, R, k.H, k.dim}, x.scalar_type()) || !is(Bc, {S, R, k.G, k.N}, x.scalar_type()) || !is(dtc, {S, R, k.H}, at::kFloat))
      return none();
    for (int i : {1, 5, 6})
      if (!vector(*t[i], p.batch, at::kInt)) return none();
    if (t[12] != nullptr && !is(*t[12], {S, k.H, k.dim}, at::kFloat)) return none();
    int32_t pad;
    if (!int32(a[14], &pad)) return none();
    const Tensor out = like(x);
    p.state = state.data_ptr(), p.state_scale = static_cast<const float*>(ptr(t[12]));
    p.x_cache = xc.data_ptr(), p.B_cache = Bc.data_ptr(), p.dt_cache = dtc.data_ptr<float>();
    p.slots = t[1]->const_data_ptr<int32_t>(), p.ring_start = t[5]->const_data_ptr<int32_t>(), p.ring_len = t[6]->const_data_ptr<int32_t>();
    p.out = out.data_ptr();
    p.state_slot_stride = state.stride(0), p.scale_slot_stride = t[12] == nullptr ? 0 : t[12]->stride(0);
    p.x_cache_slot_stride = xc.stride(0), p.B_cache_slot_stride = Bc.stride(0), p.dt_cache_slot_stride = dtc.stride(0);
    p.num_slots = static_cast<int32_t>(S), p.ring_buffer_len = static_cast<int32_t>(R), p.pad_slot_id = pad;
    const int rc = abi.decode(&p, c10::cuda::getCurrentCUDAStream(dev).stream());
    return rc != 0 ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
  });
}

// Rows of a tensor: contiguous, or two-dimensional with contiguous columns; their stride, or -1.
int64_t row_stride(const Tensor& t) {
  if (t.is_contiguous()) return t.size(-1);
  return t.dim() == 2 && t.stride(1) == 1 ? t.stride(0) : -1;
}

// add_norm(x, residual, weight, residual_scale, eps)
PyObject* add_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5) return none();
    const Tensor *x = tensor(a[0]), *r = tensor(a[1]), *w = tensor(a[2]);
    if (!x || !r || !w) return none();
    const Tensor* const all[] = {x, r, w};
    const int dev = device_of(all), code = input_code(*x), rcode = input_code(*r);
    if (dev < 0 || code < 0 || rcode < 0 || x->dim() < 1 || x->size(-1) < 1 || !fits(x->size(-1)) || x->sizes() != r->sizes() ||
        !vector(*w, x->size(-1), at::kFloat))
      return none();
    rsm_add_rms_norm_args p{};
    p.dim = static_cast<int32_t>(x->size(-1));
    p.x_stride = row_stride(*x), p.residual_stride = row_stride(*r);
    if (p.x_stride < 0 || p.residual_stride < 0) return none();
    p.residual_scale = static_cast<float>(PyFloat_AsDouble(a[3])), p.eps = static_cast<float>(PyFloat_AsDouble(a[4]));
    if (PyErr_Occurred()) throw 0;
    const Tensor out = like(*x), rout = like(*r);
    p.x = x->data_ptr(), p.residual = r->data_ptr(), p.weight = w->const_data_ptr<float>();
    p.out = out.data_ptr(), p.residual_out = rout.data_ptr();
    p.rows = x->numel() / p.dim, p.out_stride = p.residual_out_stride = p.dim;
    p.input_dtype = code, p.residual_dtype = rcode;
    const int rc = abi.add_norm(&p, c10::cuda::getCurrentCUDAStream(dev).stream());
    if (rc != 0) return PyLong_FromLong(rc);
    PyObject* first = THPVariable_Wrap(out);
    PyObject* second = THPVariable_Wrap(rout);
    PyObject* both = PyTuple_Pack(2, first, second);
    Py_XDECREF(first);
    Py_XDECREF(second);
    return both;
  });
}

// gated_norm(x, z, weight, group_size or None, eps, norm_before_gate)
PyObject* gated_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 6) return none();
    const Tensor *x = tensor(a[0]), *z = tensor(a[1]), *w = tensor(a[2]);
    if (!x || !z || !w) return none();
    const Tensor* const all[] = {x, z, w};
    const int dev = device_of(all), code = input_code(*x);
    if (dev < 0 || code < 0 || x->dim() < 1 || x->size(-1) < 1 || !fits(x->size(-1)) || x->sizes() != z->sizes() ||
        x->scalar_type() != z->scalar_type() || !vector(*w, x->size(-1), at::kFloat))
      return none();
    rsm_gated_rms_norm_args p{};
    p.dim = static_cast<int32_t>(x->size(-1));
    p.group_size = p.dim;
    if (a[3] != Py_None && !int32(a[3], &p.group_size)) return none();
    p.eps = static_cast<float>(PyFloat_AsDouble(a[4]));
    p.norm_before_gate = PyObject_IsTrue(a[5]);
    if (PyErr_Occurred()) throw 0;
    p.x_stride = row_stride(*x), p.z_stride = row_stride(*z);
    if (p.x_stride < 0 || p.z_stride < 0) return none();
    const Tensor out = like(*x);
    p.x = x->data_ptr(), p.z = z->data_ptr(), p.weight = w->const_data_ptr<float>(), p.out = out.data_ptr();
    p.rows = x->numel() / p.dim, p.out_stride = p.dim, p.input_dtype = code;
    const int rc = abi.gated_norm(&p, c10::cuda::getCurrentCUDAStream(dev).stream());
    return rc != 0 ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
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
  abi.prefill = reinterpret_cast<decltype(abi.prefill)>(at[0]);
  abi.prefill_workspace = reinterpret_cast<decltype(abi.prefill_workspace)>(at[1]);
  abi.step = reinterpret_cast<decltype(abi.step)>(at[2]);
  abi.decode = reinterpret_cast<decltype(abi.decode)>(at[3]);
  abi.add_norm = reinterpret_cast<decltype(abi.add_norm)>(at[4]);
  abi.gated_norm = reinterpret_cast<decltype(abi.gated_norm)>(at[5]);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(prefill), FAST(step), FAST(decode), FAST(add_norm), FAST(gated_norm), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_blockcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__blockcall() { return PyModule_Create(&module); }
