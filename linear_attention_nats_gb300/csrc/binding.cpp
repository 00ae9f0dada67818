// binding.cpp - the torch-facing side of the operators around the layers
// (norm + rotation, paged cache, layer norm, linear attention with a decay): checks of the tensors, allocation of the
// outputs, the stream, and the call into libnats' C ABI.
//
// A small call's time is its host's: in Python these checks took two to three
// times as long as the launch they guard (a batch's append of one token each
// 10.4 us a call, of which the kernel 4.8; now 3.8, the kernel's).  Nothing is computed here; the functions of libnats
// are given by address when the module is set up, so that the one library that
// the package has loaded is the one that is called.
#include <Python.h>

#include <ATen/MemoryOverlap.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <optional>
#include <vector>

#include "../../include/nats.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

struct Functions {
  decltype(&nats_qk_norm_rope) rope;
  decltype(&nats_qk_norm_rope_bwd) rope_bwd;
  decltype(&nats_qk_norm_rope_bwd_workspace_size) rope_bwd_ws;
  decltype(&nats_paged_append) append;
  decltype(&nats_paged_decode) decode;
  decltype(&nats_paged_decode_workspace_size) decode_ws;
  decltype(&nats_paged_evict) evict;
  decltype(&nats_paged_evict_workspace_size) evict_ws;
  decltype(&nats_layer_norm) norm;
  decltype(&nats_layer_norm_bwd) norm_bwd;
  decltype(&nats_layer_norm_bwd_workspace_size) norm_bwd_ws;
  decltype(&nats_decay_attn) decay;
  decltype(&nats_decay_attn_workspace_size) decay_ws;
  decltype(&nats_decay_attn_bwd) decay_bwd;
  decltype(&nats_decay_attn_bwd_workspace_size) decay_bwd_ws;
  decltype(&nats_decay_attn_step) decay_step;
} fn;
PyObject* nats_error = nullptr;

// ------------------------------------------------------------------ checks

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

int code_of(const Tensor& t, const char* name) {
  const ScalarType s = t.scalar_type();
  TORCH_CHECK_TYPE(s == at::kBFloat16 || s == at::kFloat, name, " must be bfloat16 or float32, got ", s);
  return s == at::kBFloat16 ? NATS_BF16 : NATS_F32;
}

int device_of(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
  return t.device().index();
}

void check(const Tensor& t, const char* name, ScalarType s, int dev) {
  TORCH_CHECK_TYPE(t.scalar_type() == s, name, " must be ", s, ", got ", t.scalar_type());
  TORCH_CHECK_VALUE(t.is_cuda() && t.device().index() == dev, name, " is on ", t.device(), ", not on cuda:", dev);
}
void check_shape(const Tensor& t, const char* name, IntArrayRef shape) {
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", got ", t.sizes());
}

// A contiguous argument's address (NULL for None).
void* contiguous(PyObject* o, const char* name, ScalarType s, int dev) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, name);
  check(t, name, s, dev);
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
  return t.data_ptr();
}
void* contiguous(PyObject* o, const char* name, ScalarType s, IntArrayRef shape, int dev) {
  if (o == Py_None) return nullptr;
  void* p = contiguous(o, name, s, dev);
  check_shape(THPVariable_Unpack(o), name, shape);
  return p;
}

// A [B, H, L, d] operand with any strides but the last.
struct Heads {
  void* p = nullptr;
  nats_strides st = {0, 0, 0};
};
Heads heads(const Tensor& t, const char* name, ScalarType s, IntArrayRef shape, int dev) {
  check(t, name, s, dev);
  check_shape(t, name, shape);
  const IntArrayRef st = t.strides();
  TORCH_CHECK_VALUE(st[3] == 1 || t.numel() == 0, name, ": the entries of a row must be contiguous (last stride 1, got ",
                    st[3], ")");
  return Heads{t.data_ptr(), {st[0], st[1], st[2]}};
}
// The same for an output, which must not be an expanded tensor.
Heads heads_out(const Tensor& t, const char* name, ScalarType s, IntArrayRef shape, int dev) {
  const Heads h = heads(t, name, s, shape, dev);
  for (int i = 0; i < 3; ++i)
    TORCH_CHECK_VALUE(t.strides()[i] != 0 || t.sizes()[i] <= 1, name,
                      " is written and must not be an expanded tensor");
  return h;
}

// An output that must not share memory with another argument: overlaps that torch can tell (tensors without gaps), and
// tensors that start at one address.  `same`: the argument itself (of the same shape), at the same strides, is allowed.
void apart(const Tensor& out, const char* name, const Tensor& t, const char* other, bool same = false) {
  if (out.numel() == 0 || t.numel() == 0) return;
  const bool one = out.data_ptr() == t.data_ptr();
  if (same && one) {
    bool alike = true;
    for (int64_t i = 0; i < out.dim(); ++i) alike = alike && (out.size(i) <= 1 || out.stride(i) == t.stride(i));
    if (alike) return;
  }
  const auto s = at::get_overlap_status(out, t);
  TORCH_CHECK_VALUE(!one && s != at::MemOverlapStatus::Full && s != at::MemOverlapStatus::Partial, name,
                    " must not share memory with ", other, same ? " other than as the same tensor" : "");
}

struct Rotation {
  int rot = 0;
  const double* inv_freq = nullptr;
  const int64_t* pos = nullptr;
  int64_t pos_b = 0;
};
Rotation rotation(PyObject* inv_freq, PyObject* positions, int64_t B, int64_t L, int dev) {
  Rotation r;
  if (inv_freq != Py_None) {
    const Tensor& t = tensor(inv_freq, "inv_freq");
    TORCH_CHECK_VALUE(t.dim() == 1, "inv_freq must have shape (rot / 2,), got ", t.sizes());
    TORCH_CHECK_VALUE(t.size(0) < (1 << 20), "inv_freq is too long");
    r.inv_freq = (const double*)contiguous(inv_freq, "inv_freq", at::kDouble, dev);
    r.rot = 2 * (int)t.size(0);
  }
  if (positions != Py_None) {
    const Tensor& t = tensor(positions, "positions");
    check(t, "positions", at::kLong, dev);
    if (t.dim() == 2)
      check_shape(t, "positions", {B, L});
    else
      check_shape(t, "positions", {L});
    TORCH_CHECK_VALUE(L <= 1 || t.stride(-1) == 1, "positions of a sequence must be contiguous");
    r.pos = (const int64_t*)t.data_ptr();
    r.pos_b = t.dim() == 2 ? t.stride(0) : 0;
  }
  return r;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
int64_t integer(PyObject* o, const char* name, int64_t lo, int64_t hi) {
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  TORCH_CHECK_VALUE(!over && v >= lo && v <= hi, name, " is out of range");
  return v;
}
int32_t int32(PyObject* o, const char* name) { return (int32_t)integer(o, name, INT32_MIN, INT32_MAX); }
int32_t extent(int64_t v, const char* name) {
  TORCH_CHECK_VALUE(v <= INT32_MAX, name, " is out of range");
  return (int32_t)v;
}

// ---------------------------------------------------------------- the call

at::TensorOptions on(ScalarType s, int dev) {
  return at::TensorOptions().dtype(s).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
}

// The device and stream of one call.  What it allocates comes from that
// stream's own memory, where work still to run on the current stream has no
// part, and is marked as used on the current stream, where the caller will
// read and free it.  What it is given is marked as used on the call's stream
// (uses), so that the caller may free it before the call has run.
struct Call {
  int dev;
  c10::cuda::CUDAStream cur;
  std::optional<c10::cuda::CUDAGuard> device;
  std::optional<c10::cuda::CUDAStreamGuard> other;
  nats_stream_t stream;

  Call(int device_index, PyObject* s)
      : dev(device_index), cur(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device_index)) {
    stream = (nats_stream_t)cur.stream();
    if (s != Py_None) {
      const auto get = [&](const char* name) {
        PyObject* v = PyObject_GetAttrString(s, name);
        if (!v) throw python_error();
        const long long x = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (x == -1 && PyErr_Occurred()) throw python_error();
        return x;
      };
      const long long index = get("device_index");
      TORCH_CHECK_VALUE(index == dev, "the stream is on cuda:", index, ", the tensors on cuda:", dev);
      const c10::cuda::CUDAStream given(
          c10::cuda::CUDAStream::UNCHECKED,
          c10::Stream(c10::Stream::UNSAFE, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev), get("stream_id")));
      if (given != cur) {
        other.emplace(given);
        stream = (nats_stream_t)given.stream();
      }
    }
    if (!other && c10::cuda::current_device() != dev) device.emplace((c10::DeviceIndex)dev);
  }
  template <class... O>
  void uses(O*... args) const {
    if (!other) return;
    for (PyObject* o : {args...})
      if (o != Py_None) THPVariable_Unpack(o).record_stream(other->current_stream());
  }
  Tensor made(const Tensor& t) const {
    if (other) t.record_stream(cur);
    return t;
  }
  Tensor empty(IntArrayRef shape, ScalarType s) const { return made(at::empty(shape, on(s, dev))); }
  Tensor zeros(IntArrayRef shape, ScalarType s) const { return made(at::zeros(shape, on(s, dev))); }
  // the caller's workspace, or a new one of `size` bytes
  Tensor workspace(PyObject* o, size_t size) const {
    if (o == Py_None) return at::empty({(int64_t)size}, on(at::kByte, dev));
    contiguous(o, "workspace", at::kByte, dev);
    return THPVariable_Unpack(o);
  }
};

struct Refused {};  // the Python error is set
void done(nats_status s, const char* where) {
  if (s == NATS_OK) return;
  PyObject* e = PyObject_CallFunction(nats_error, "is", (int)s, where);
  if (e) {
    PyErr_SetObject(nats_error, e);
    Py_DECREF(e);
  }
  throw Refused();
}

PyObject* ref(PyObject* o) {
  Py_INCREF(o);
  return o;
}
PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* t = a && b ? PyTuple_New(2) : nullptr;
  if (!t) {
    Py_XDECREF(a);
    Py_XDECREF(b);
    throw python_error();
  }
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  return t;
}

// A dict of results in the making.
struct Dict {
  PyObject* d = PyDict_New();
  Dict() {
    if (!d) throw python_error();
  }
  ~Dict() { Py_XDECREF(d); }
  Dict(const Dict&) = delete;
  void put(const char* name, PyObject* o) {
    const int bad = o ? PyDict_SetItemString(d, name, o) : -1;
    Py_XDECREF(o);
    if (bad) throw python_error();
  }
  PyObject* give() {
    PyObject* r = d;
    d = nullptr;
    return r;
  }
};

#define NATS_BEGIN(count)                                                       \
  HANDLE_TH_ERRORS                                                              \
  try {                                                                         \
    if (n != (count)) {                                                         \
      PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", count, n); \
      return nullptr;                                                           \
    }
#define NATS_END             \
  }                          \
  catch (const Refused&) {   \
    return nullptr;          \
  }                          \
  END_HANDLE_TH_ERRORS

void check_pair(const Tensor& q, const Tensor& k) {
  TORCH_CHECK_VALUE(q.dim() == 4 && k.dim() == 4, "q and k must be [B, H, L, d]");
  TORCH_CHECK_VALUE(q.size(0) == k.size(0) && q.size(2) == k.size(2) && q.size(3) == k.size(3), "q ", q.sizes(),
                    " and k ", k.sizes(), " differ in more than their heads");
}

// q, k, w_q, w_k, inv_freq, positions, pos0, interleaved, norm, eps, out_q, out_k, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NATS_BEGIN(13)
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  check_pair(q, k);
  const int dev = device_of(q, "q"), code = code_of(q, "q");
  const ScalarType s = q.scalar_type();
  const Heads hq = heads(q, "q", s, q.sizes(), dev), hk = heads(k, "k", s, k.sizes(), dev);
  const int64_t d = q.size(3);
  const float* wq = (const float*)contiguous(a[2], "w_q", at::kFloat, {d}, dev);
  const float* wk = (const float*)contiguous(a[3], "w_k", at::kFloat, {d}, dev);
  const Rotation r = rotation(a[4], a[5], q.size(0), q.size(2), dev);
  const Call call(dev, a[12]);
  Tensor oq, ok;
  Heads hoq, hok;
  if (a[10] == Py_None) oq = call.empty(q.sizes(), s);
  if (a[11] == Py_None) ok = call.empty(k.sizes(), s);
  hoq = heads_out(a[10] == Py_None ? oq : tensor(a[10], "out_q"), "out_q", s, q.sizes(), dev);
  hok = heads_out(a[11] == Py_None ? ok : tensor(a[11], "out_k"), "out_k", s, k.sizes(), dev);
  const nats_rope_dims dm = {extent(q.size(0), "B"), extent(q.size(2), "L"), extent(q.size(1), "Hq"),
                             extent(k.size(1), "Hk"), extent(d, "d"), r.rot, truth(a[7]), truth(a[8]), code,
                             (float)real(a[9])};
  const int64_t pos0 = integer(a[6], "pos0", -(1ll << 62), 1ll << 62);
  done(fn.rope(&dm, hq.p, &hq.st, hk.p, &hk.st, wq, wk, r.inv_freq, r.pos, r.pos_b, pos0, hoq.p, &hoq.st, hok.p,
               &hok.st, call.stream),
       "nats_qk_norm_rope");
  call.uses(a[0], a[1], a[2], a[3], a[4], a[5], a[10], a[11]);
  return pair(a[10] == Py_None ? THPVariable_Wrap(oq) : ref(a[10]), a[11] == Py_None ? THPVariable_Wrap(ok) : ref(a[11]));
  NATS_END
}

// dq_out, dk_out, q, k, w_q, w_k, inv_freq, positions, pos0, interleaved, norm, eps, dq, dk, weight_grads, workspace, stream
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NATS_BEGIN(17)
  const Tensor &gq = tensor(a[0], "dq_out"), &gk = tensor(a[1], "dk_out"), &q = tensor(a[2], "q"),
               &k = tensor(a[3], "k");
  check_pair(q, k);
  const int dev = device_of(q, "q"), code = code_of(q, "q"), gcode = code_of(gq, "dq_out");
  const ScalarType s = q.scalar_type();
  const Heads hq = heads(q, "q", s, q.sizes(), dev), hk = heads(k, "k", s, k.sizes(), dev);
  const Heads hgq = heads(gq, "dq_out", gq.scalar_type(), q.sizes(), dev);
  const Heads hgk = heads(gk, "dk_out", gq.scalar_type(), k.sizes(), dev);
  const int64_t d = q.size(3);
  const float* wq = (const float*)contiguous(a[4], "w_q", at::kFloat, {d}, dev);
  const float* wk = (const float*)contiguous(a[5], "w_k", at::kFloat, {d}, dev);
  const Rotation r = rotation(a[6], a[7], q.size(0), q.size(2), dev);
  const Call call(dev, a[16]);
  const ScalarType xs = a[12] != Py_None ? tensor(a[12], "dq").scalar_type()
                        : a[13] != Py_None ? tensor(a[13], "dk").scalar_type() : s;
  const Tensor dq = a[12] == Py_None ? call.empty(q.sizes(), xs) : tensor(a[12], "dq");
  const Tensor dk = a[13] == Py_None ? call.empty(k.sizes(), xs) : tensor(a[13], "dk");
  const int xcode = code_of(dq, "dq");
  const Heads hdq = heads_out(dq, "dq", xs, q.sizes(), dev), hdk = heads_out(dk, "dk", xs, k.sizes(), dev);
  const nats_rope_dims dm = {extent(q.size(0), "B"), extent(q.size(2), "L"), extent(q.size(1), "Hq"),
                             extent(k.size(1), "Hk"), extent(d, "d"), r.rot, truth(a[9]), truth(a[10]), code,
                             (float)real(a[11])};
  const int64_t pos0 = integer(a[8], "pos0", -(1ll << 62), 1ll << 62);
  Tensor dwq, dwk, ws;
  const bool dw = truth(a[14]) && dm.norm;
  if (dw) {
    dwq = call.empty({d}, at::kFloat), dwk = call.empty({d}, at::kFloat);
    ws = call.workspace(a[15], fn.rope_bwd_ws(&dm));
  }
  done(fn.rope_bwd(&dm, gcode, xcode, hgq.p, &hgq.st, hgk.p, &hgk.st, hq.p, &hq.st, hk.p, &hk.st, wq, wk, r.inv_freq,
                   r.pos, r.pos_b, pos0, hdq.p, &hdq.st, hdk.p, &hdk.st, dw ? (float*)dwq.data_ptr() : nullptr,
                   dw ? (float*)dwk.data_ptr() : nullptr, dw ? ws.data_ptr() : nullptr,
                   dw ? (size_t)ws.numel() : 0, call.stream),
       "nats_qk_norm_rope_bwd");
  call.uses(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[12], a[13], dw ? a[15] : Py_None);
  Dict res;
  res.put("dq", a[12] == Py_None ? THPVariable_Wrap(dq) : ref(a[12]));
  res.put("dk", a[13] == Py_None ? THPVariable_Wrap(dk) : ref(a[13]));
  if (dw) {
    res.put("dw_q", THPVariable_Wrap(dwq));
    res.put("dw_k", THPVariable_Wrap(dwk));
  }
  return res.give();
  NATS_END
}

const nats_paged_cache* cache_at(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p) throw python_error();
  return (const nats_paged_cache*)p;
}
ScalarType type_of(const nats_paged_cache* c) { return c->dtype == NATS_BF16 ? at::kBFloat16 : at::kFloat; }

// cache, device, k, v, start, n_new, q, out_q, norm, w_q, w_k, inv_freq, positions, interleaved, eps, stream
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NATS_BEGIN(16)
  const nats_paged_cache* c = cache_at(a[0]);
  const int dev = int32(a[1], "device");
  const ScalarType s = type_of(c);
  const Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
  TORCH_CHECK_VALUE(k.dim() == 4 && k.size(0) == c->B && k.size(1) == c->Hk && k.size(3) == c->d, "k must be [", c->B, ", ",
                    c->Hk, ", T, ", c->d, "], got ", k.sizes());
  const int64_t B = c->B, T = k.size(2), d = c->d;
  const Heads hk = heads(k, "k", s, k.sizes(), dev), hv = heads(v, "v", s, k.sizes(), dev);
  const int32_t* start = (const int32_t*)contiguous(a[4], "start", at::kInt, {B}, dev);
  const int32_t* n_new = (const int32_t*)contiguous(a[5], "n_new", at::kInt, {B}, dev);
  const float* wq = (const float*)contiguous(a[9], "w_q", at::kFloat, {d}, dev);
  const float* wk = (const float*)contiguous(a[10], "w_k", at::kFloat, {d}, dev);
  const Rotation r = rotation(a[11], a[12], B, T, dev);
  const Call call(dev, a[15]);
  Heads hq, hoq;
  Tensor oq;
  int64_t Hq = 0;
  const bool has_q = a[6] != Py_None;
  if (has_q) {
    const Tensor& q = tensor(a[6], "q");
    TORCH_CHECK_VALUE(q.dim() == 4 && q.size(0) == B && q.size(2) == T && q.size(3) == d, "q must be [", B, ", Hq, ", T,
                      ", ", d, "], got ", q.sizes());
    Hq = q.size(1);
    hq = heads(q, "q", s, q.sizes(), dev);
    if (a[7] == Py_None)
      oq = a[5] == Py_None ? call.empty(q.sizes(), s) : call.zeros(q.sizes(), s);
    else
      oq = tensor(a[7], "out_q");
    hoq = heads_out(oq, "out_q", s, q.sizes(), dev);
  }
  const nats_rope_dims dm = {(int32_t)B, extent(T, "T"), extent(Hq, "Hq"), c->Hk, (int32_t)d, r.rot, truth(a[13]),
                             truth(a[8]), c->dtype, (float)real(a[14])};
  done(fn.append(c, &dm, hq.p, &hq.st, hk.p, &hk.st, hv.p, &hv.st, wq, wk, r.inv_freq, start, n_new, r.pos, r.pos_b,
                 hoq.p, &hoq.st, call.stream),
       "nats_paged_append");
  call.uses(a[2], a[3], a[4], a[5], a[6], has_q ? a[7] : Py_None, a[9], a[10], a[11], a[12]);
  if (!has_q) Py_RETURN_NONE;
  return a[7] == Py_None ? THPVariable_Wrap(oq) : ref(a[7]);
  NATS_END
}

// cache, device, q, scale, accumulate, return_lse, out, workspace, stream
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NATS_BEGIN(9)
  const nats_paged_cache* c = cache_at(a[0]);
  const int dev = int32(a[1], "device");
  const ScalarType s = type_of(c);
  const Tensor& q = tensor(a[2], "q");
  TORCH_CHECK_VALUE(q.dim() == 3 && q.size(0) == c->B && q.size(2) == c->d, "q must be [", c->B, ", Hq, ", c->d, "], got ",
                    q.sizes());
  check(q, "q", s, dev);
  TORCH_CHECK_VALUE(q.stride(2) == 1 || q.numel() == 0, "q: the entries of a row must be contiguous");
  const double given = real(a[3]);
  const float scale = (float)given;
  // (0 asks for 1 / sqrt(d): a smaller scale than fp32 has must not become one)
  TORCH_CHECK_VALUE(scale != 0.f || given == 0.0, "scale is out of range");
  const int accumulate = truth(a[4]);
  const bool has_lse = truth(a[5]);
  const int32_t Hq = extent(q.size(1), "Hq");
  const Call call(dev, a[8]);
  Tensor out, lse;
  if (a[6] == Py_None)
    out = call.empty(q.sizes(), s);
  else
    contiguous(a[6], "out", s, q.sizes(), dev), out = THPVariable_Unpack(a[6]);
  if (has_lse) lse = call.empty({q.size(0), q.size(1)}, at::kFloat);
  const Tensor ws = call.workspace(a[7], a[7] == Py_None ? fn.decode_ws(c, Hq, accumulate) : 0);
  done(fn.decode(c, Hq, scale, q.data_ptr(), q.stride(0), q.stride(1), out.data_ptr(),
                 has_lse ? (float*)lse.data_ptr() : nullptr, accumulate, ws.data_ptr(), (size_t)ws.numel(), call.stream),
       "nats_paged_decode");
  call.uses(a[2], a[6], a[7]);
  PyObject* o = a[6] == Py_None ? THPVariable_Wrap(out) : ref(a[6]);
  return has_lse ? pair(o, THPVariable_Wrap(lse)) : o;
  NATS_END
}

// cache, device, out_table, budget, recent, sinks, lens_out, return_keep, workspace, stream
PyObject* paged_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NATS_BEGIN(10)
  const nats_paged_cache* c = cache_at(a[0]);
  const int dev = int32(a[1], "device");
  const Tensor& table = tensor(a[2], "out_table");
  TORCH_CHECK_VALUE(table.dim() == 2 && table.size(0) == c->B, "out_table must be [", c->B, ", pages], got ",
                    table.sizes());
  const int32_t* pt = (const int32_t*)contiguous(a[2], "out_table", at::kInt, dev);
  const int32_t budget = int32(a[3], "budget"), recent = int32(a[4], "recent"), sinks = int32(a[5], "sinks");
  const bool has_keep = truth(a[7]);
  const Call call(dev, a[9]);
  Tensor lens, keep;
  if (a[6] == Py_None)
    lens = call.empty({c->B}, at::kInt);
  else
    contiguous(a[6], "lens_out", at::kInt, {c->B}, dev), lens = THPVariable_Unpack(a[6]);
  if (has_keep) keep = call.empty({c->B, c->Hk, budget > 0 ? budget : 0}, at::kInt);
  const Tensor ws = call.workspace(a[8], a[8] == Py_None ? fn.evict_ws(c, budget) : 0);
  done(fn.evict(c, pt, extent(table.size(1), "out_table"), budget, recent, sinks, (int32_t*)lens.data_ptr(),
                has_keep ? (int32_t*)keep.data_ptr() : nullptr, ws.data_ptr(), (size_t)ws.numel(), call.stream),
       "nats_paged_evict");
  call.uses(a[2], a[6], a[8]);
  PyObject* l = a[6] == Py_None ? THPVariable_Wrap(lens) : ref(a[6]);
  return has_keep ? pair(THPVariable_Wrap(keep), l) : l;
  NATS_END
}

// The leading dimensions of tensors of one shape, brought to three: those that
// follow one another in memory in all of them are one.
template <int N>
struct Lead {
  int64_t size[3] = {1, 1, 1};
  nats_strides st[N];
  bool empty = false;

  Lead(const Tensor* const (&t)[N], const char* name) {
    std::vector<int64_t> n;
    std::vector<std::array<int64_t, N>> s;
    const int64_t dims = t[0]->dim() - 1;
    for (int64_t i = 0; i < dims; ++i) {
      const int64_t e = t[0]->size(i);
      if (e == 0) empty = true;
      if (e == 1) continue;
      std::array<int64_t, N> x;
      bool joins = !n.empty();
      for (int j = 0; j < N; ++j) {
        x[j] = t[j]->stride(i);
        joins = joins && s.back()[j] == x[j] * e;
      }
      if (joins) {
        n.back() *= e, s.back() = x;
      } else {
        n.push_back(e), s.push_back(x);
      }
    }
    if (empty) n.clear(), s.clear();
    TORCH_CHECK_VALUE(n.size() <= 3, name, " has more than three leading dimensions that do not follow one another in memory");
    for (int j = 0; j < N; ++j) {
      int64_t* p[3] = {&st[j].b, &st[j].h, &st[j].t};
      for (size_t i = 0; i < 3; ++i) *p[i] = 0;
      for (size_t i = 0; i < n.size(); ++i) *p[3 - n.size() + i] = s[i][j];
    }
    for (size_t i = 0; i < n.size(); ++i) size[3 - n.size() + i] = n[i];
    if (empty) size[2] = 0;
  }
};

const Tensor& rows(const Tensor& t, const char* name, ScalarType s, IntArrayRef shape, int dev, bool out) {
  check(t, name, s, dev);
  check_shape(t, name, shape);
  TORCH_CHECK_VALUE(t.stride(-1) == 1 || t.size(-1) <= 1 || t.numel() == 0, name,
                    ": the entries of a row must be contiguous (last stride 1, got ", t.stride(-1), ")");
  if (out)
    for (int64_t i = 0; i < t.dim(); ++i)
      TORCH_CHECK_VALUE(t.stride(i) != 0 || t.size(i) <= 1, name, " is written and must not be an expanded tensor");
  return t;
}

// x, weight, bias, eps, out, stream
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NATS_BEGIN(6)
  const Tensor& x = tensor(a[0], "x");
  TORCH_CHECK_VALUE(x.dim() >= 1, "x must have at least one dimension");
  const int dev = device_of(x, "x"), code = code_of(x, "x");
  const ScalarType s = x.scalar_type();
  const int64_t D = x.size(-1);
  rows(x, "x", s, x.sizes(), dev, false);
  const float* w = (const float*)contiguous(a[1], "weight", at::kFloat, {D}, dev);
  const float* b = (const float*)contiguous(a[2], "bias", at::kFloat, {D}, dev);
  const Call call(dev, a[5]);
  const Tensor out = a[4] == Py_None ? call.empty(x.sizes(), s) : tensor(a[4], "out");
  rows(out, "out", s, x.sizes(), dev, true);
  if (a[4] != Py_None) apart(out, "out", x, "x", true);
  const Tensor* const both[2] = {&x, &out};
  const Lead<2> l(both, "x");
  const nats_norm_dims dm = {extent(l.size[0], "x"), extent(l.size[1], "x"), extent(l.size[2], "x"), extent(D, "x"), code,
                             (float)real(a[3])};
  done(fn.norm(&dm, x.data_ptr(), &l.st[0], w, b, out.data_ptr(), &l.st[1], call.stream), "nats_layer_norm");
  call.uses(a[0], a[1], a[2], a[4]);
  return a[4] == Py_None ? THPVariable_Wrap(out) : ref(a[4]);
  NATS_END
}

// dout, x, weight, eps, dx, weight_grads, workspace, stream
PyObject* layer_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NATS_BEGIN(8)
  const Tensor &u = tensor(a[0], "dout"), &x = tensor(a[1], "x");
  TORCH_CHECK_VALUE(x.dim() >= 1, "x must have at least one dimension");
  const int dev = device_of(x, "x"), code = code_of(x, "x");
  const ScalarType s = x.scalar_type();
  const int64_t D = x.size(-1);
  rows(x, "x", s, x.sizes(), dev, false);
  rows(u, "dout", s, x.sizes(), dev, false);
  const float* w = (const float*)contiguous(a[2], "weight", at::kFloat, {D}, dev);
  const Call call(dev, a[7]);
  const Tensor dx = a[4] == Py_None ? call.empty(x.sizes(), s) : tensor(a[4], "dx");
  rows(dx, "dx", s, x.sizes(), dev, true);
  if (a[4] != Py_None) {
    apart(dx, "dx", u, "dout", true);
    apart(dx, "dx", x, "x", true);
  }
  const Tensor* const all[3] = {&u, &x, &dx};
  const Lead<3> l(all, "x");
  const nats_norm_dims dm = {extent(l.size[0], "x"), extent(l.size[1], "x"), extent(l.size[2], "x"), extent(D, "x"), code,
                             (float)real(a[3])};
  const bool sums = truth(a[5]);
  Tensor dw, db, ws;
  if (sums) {
    dw = call.empty({D}, at::kFloat), db = call.empty({D}, at::kFloat);
    ws = call.workspace(a[6], a[6] == Py_None ? fn.norm_bwd_ws(&dm) : 0);
  }
  done(fn.norm_bwd(&dm, u.data_ptr(), &l.st[0], x.data_ptr(), &l.st[1], w, dx.data_ptr(), &l.st[2],
                   sums ? (float*)dw.data_ptr() : nullptr, sums ? (float*)db.data_ptr() : nullptr,
                   sums ? ws.data_ptr() : nullptr, sums ? (size_t)ws.numel() : 0, call.stream),
       "nats_layer_norm_bwd");
  call.uses(a[0], a[1], a[2], a[4], sums ? a[6] : Py_None);
  Dict res;
  res.put("dx", a[4] == Py_None ? THPVariable_Wrap(dx) : ref(a[4]));
  if (sums) {
    res.put("dw", THPVariable_Wrap(dw));
    res.put("db", THPVariable_Wrap(db));
  }
  return res.give();
  NATS_END
}

float scale_of(PyObject* o) {
  const double given = real(o);
  const float scale = (float)given;
  // (0 asks for 1 / sqrt(d): a smaller scale than fp32 has must not become one)
  TORCH_CHECK_VALUE(scale != 0.f || given == 0.0, "scale is out of range");
  return scale;
}

nats_decay_dims decay_dims(const Tensor& q, int code, PyObject* scale) {
  TORCH_CHECK_VALUE(q.dim() == 4, "q must be [B, H, L, d], got ", q.sizes());
  return {extent(q.size(0), "B"), extent(q.size(1), "H"), extent(q.size(2), "L"), extent(q.size(3), "d"), code,
          scale_of(scale)};
}

// q, k, v, log_decay, scale, lens, state, return_state, state_out, out, workspace, stream
PyObject* decay_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NATS_BEGIN(12)
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  tensor(a[3], "log_decay");
  const int dev = device_of(q, "q"), code = code_of(q, "q");
  const ScalarType s = q.scalar_type();
  const nats_decay_dims dm = decay_dims(q, code, a[4]);
  const int64_t B = dm.B, H = dm.H, d = dm.d;
  const Heads hq = heads(q, "q", s, q.sizes(), dev), hk = heads(k, "k", s, q.sizes(), dev),
              hv = heads(v, "v", s, q.sizes(), dev);
  const float* gp = (const float*)contiguous(a[3], "log_decay", at::kFloat, {H}, dev);
  const int32_t* lens = (const int32_t*)contiguous(a[5], "lens", at::kInt, {B}, dev);
  const float* s_in = (const float*)contiguous(a[6], "state", at::kFloat, {B, H, d, d}, dev);
  const bool has_out = a[8] != Py_None, has_state = has_out || truth(a[7]);
  const Call call(dev, a[11]);
  Tensor so;
  if (has_out)
    contiguous(a[8], "state_out", at::kFloat, {B, H, d, d}, dev), so = THPVariable_Unpack(a[8]);
  else if (has_state)
    so = call.empty({B, H, d, d}, at::kFloat);
  const Tensor out = a[9] == Py_None ? call.empty(q.sizes(), s) : tensor(a[9], "out");
  const Heads ho = heads_out(out, "out", s, q.sizes(), dev);
  if (a[9] != Py_None) {
    apart(out, "out", q, "q");
    apart(out, "out", k, "k");
    apart(out, "out", v, "v");
  }
  if (has_out && s_in) apart(so, "state_out", THPVariable_Unpack(a[6]), "state", true);
  const Tensor ws = call.workspace(a[10], a[10] == Py_None ? fn.decay_ws(&dm) : 0);
  done(fn.decay(&dm, hq.p, &hq.st, hk.p, &hk.st, hv.p, &hv.st, gp, lens, s_in, ho.p, &ho.st,
                has_state ? (float*)so.data_ptr() : nullptr, ws.data_ptr(), (size_t)ws.numel(), call.stream),
       "nats_decay_attn");
  call.uses(a[0], a[1], a[2], a[3], a[5], a[6], a[8], a[9], a[10]);
  PyObject* o = a[9] == Py_None ? THPVariable_Wrap(out) : ref(a[9]);
  return has_state ? pair(o, has_out ? ref(a[8]) : THPVariable_Wrap(so)) : o;
  NATS_END
}

// dout, q, k, v, log_decay, scale, lens, state, dstate_out, state_grad, dq, dk, dv, workspace, stream
PyObject* decay_attn_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NATS_BEGIN(15)
  const Tensor &u = tensor(a[0], "dout"), &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
  tensor(a[4], "log_decay");
  const int dev = device_of(q, "q"), code = code_of(q, "q");
  const ScalarType s = q.scalar_type();
  const nats_decay_dims dm = decay_dims(q, code, a[5]);
  const int64_t B = dm.B, H = dm.H, d = dm.d;
  const Heads hu = heads(u, "dout", s, q.sizes(), dev), hq = heads(q, "q", s, q.sizes(), dev),
              hk = heads(k, "k", s, q.sizes(), dev), hv = heads(v, "v", s, q.sizes(), dev);
  const float* gp = (const float*)contiguous(a[4], "log_decay", at::kFloat, {H}, dev);
  const int32_t* lens = (const int32_t*)contiguous(a[6], "lens", at::kInt, {B}, dev);
  const float* s_in = (const float*)contiguous(a[7], "state", at::kFloat, {B, H, d, d}, dev);
  const float* ds_out = (const float*)contiguous(a[8], "dstate_out", at::kFloat, {B, H, d, d}, dev);
  const bool has_state = truth(a[9]);
  const Call call(dev, a[14]);
  Tensor ds, grads[3];
  Heads hg[3];
  const char* const names[3] = {"dq", "dk", "dv"};
  if (has_state) ds = call.empty({B, H, d, d}, at::kFloat);
  for (int i = 0; i < 3; ++i) {
    grads[i] = a[10 + i] == Py_None ? call.empty(q.sizes(), s) : tensor(a[10 + i], names[i]);
    hg[i] = heads_out(grads[i], names[i], s, q.sizes(), dev);
    if (a[10 + i] == Py_None) continue;
    apart(grads[i], names[i], u, "dout");
    apart(grads[i], names[i], q, "q");
    apart(grads[i], names[i], k, "k");
    apart(grads[i], names[i], v, "v");
    for (int j = 0; j < i; ++j) apart(grads[i], names[i], grads[j], names[j]);
  }
  const Tensor ws = call.workspace(a[13], a[13] == Py_None ? fn.decay_bwd_ws(&dm) : 0);
  done(fn.decay_bwd(&dm, hu.p, &hu.st, hq.p, &hq.st, hk.p, &hk.st, hv.p, &hv.st, gp, lens, s_in, ds_out, hg[0].p,
                    &hg[0].st, hg[1].p, &hg[1].st, hg[2].p, &hg[2].st, has_state ? (float*)ds.data_ptr() : nullptr,
                    ws.data_ptr(), (size_t)ws.numel(), call.stream),
       "nats_decay_attn_bwd");
  call.uses(a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8], a[10], a[11], a[12], a[13]);
  Dict res;
  for (int i = 0; i < 3; ++i) res.put(names[i], a[10 + i] == Py_None ? THPVariable_Wrap(grads[i]) : ref(a[10 + i]));
  if (has_state) res.put("dstate", THPVariable_Wrap(ds));
  return res.give();
  NATS_END
}

// A [B, H, d] operand of single tokens.
Heads token(const Tensor& t, const char* name, ScalarType s, IntArrayRef shape, int dev, bool out) {
  rows(t, name, s, shape, dev, out);
  return Heads{t.data_ptr(), {t.stride(0), t.stride(1), 0}};
}

// q, k, v, log_decay, state, scale, out, stream
PyObject* decay_attn_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NATS_BEGIN(8)
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  tensor(a[3], "log_decay");
  tensor(a[4], "state");
  TORCH_CHECK_VALUE(q.dim() == 3, "q must be [B, H, d], got ", q.sizes());
  const int dev = device_of(q, "q"), code = code_of(q, "q");
  const ScalarType s = q.scalar_type();
  const int64_t B = q.size(0), H = q.size(1), d = q.size(2);
  const Heads hq = token(q, "q", s, q.sizes(), dev, false), hk = token(k, "k", s, q.sizes(), dev, false),
              hv = token(v, "v", s, q.sizes(), dev, false);
  const float* gp = (const float*)contiguous(a[3], "log_decay", at::kFloat, {H}, dev);
  float* S = (float*)contiguous(a[4], "state", at::kFloat, {B, H, d, d}, dev);
  const nats_decay_dims dm = {extent(B, "B"), extent(H, "H"), 1, extent(d, "d"), code, scale_of(a[5])};
  const Call call(dev, a[7]);
  const Tensor out = a[6] == Py_None ? call.empty(q.sizes(), s) : tensor(a[6], "out");
  const Heads ho = token(out, "out", s, q.sizes(), dev, true);
  if (a[6] != Py_None) {
    apart(out, "out", q, "q");
    apart(out, "out", k, "k");
    apart(out, "out", v, "v");
  }
  done(fn.decay_step(&dm, hq.p, &hq.st, hk.p, &hk.st, hv.p, &hv.st, gp, S, ho.p, &ho.st, call.stream),
       "nats_decay_attn_step");
  call.uses(a[0], a[1], a[2], a[3], a[4], a[6]);
  return a[6] == Py_None ? THPVariable_Wrap(out) : ref(a[6]);
  NATS_END
}

// setup(address of function by name, the error class)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  NATS_BEGIN(2)
  const auto get = [&](const char* name) {
    PyObject* v = PyMapping_GetItemString(a[0], name);
    if (!v) throw python_error();
    void* p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (!p && PyErr_Occurred()) throw python_error();
    return p;
  };
  fn.rope = (decltype(fn.rope))get("nats_qk_norm_rope");
  fn.rope_bwd = (decltype(fn.rope_bwd))get("nats_qk_norm_rope_bwd");
  fn.rope_bwd_ws = (decltype(fn.rope_bwd_ws))get("nats_qk_norm_rope_bwd_workspace_size");
  fn.append = (decltype(fn.append))get("nats_paged_append");
  fn.decode = (decltype(fn.decode))get("nats_paged_decode");
  fn.decode_ws = (decltype(fn.decode_ws))get("nats_paged_decode_workspace_size");
  fn.evict = (decltype(fn.evict))get("nats_paged_evict");
  fn.evict_ws = (decltype(fn.evict_ws))get("nats_paged_evict_workspace_size");
  fn.norm = (decltype(fn.norm))get("nats_layer_norm");
  fn.norm_bwd = (decltype(fn.norm_bwd))get("nats_layer_norm_bwd");
  fn.norm_bwd_ws = (decltype(fn.norm_bwd_ws))get("nats_layer_norm_bwd_workspace_size");
  fn.decay = (decltype(fn.decay))get("nats_decay_attn");
  fn.decay_ws = (decltype(fn.decay_ws))get("nats_decay_attn_workspace_size");
  fn.decay_bwd = (decltype(fn.decay_bwd))get("nats_decay_attn_bwd");
  fn.decay_bwd_ws = (decltype(fn.decay_bwd_ws))get("nats_decay_attn_bwd_workspace_size");
  fn.decay_step = (decltype(fn.decay_step))get("nats_decay_attn_step");
  nats_error = ref(a[1]);
  Py_RETURN_NONE;
  NATS_END
}

#define NATS_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {NATS_METHOD(setup),        NATS_METHOD(qk_norm_rope),   NATS_METHOD(qk_norm_rope_bwd),
                         NATS_METHOD(paged_append), NATS_METHOD(paged_decode),   NATS_METHOD(paged_evict),
                         NATS_METHOD(layer_norm),   NATS_METHOD(layer_norm_bwd), NATS_METHOD(decay_attn),
                         NATS_METHOD(decay_attn_bwd), NATS_METHOD(decay_attn_step), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operators", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__operators(void) { return PyModule_Create(&module); }
