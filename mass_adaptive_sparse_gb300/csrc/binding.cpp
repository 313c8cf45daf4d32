// Python binding of the serving entry points (8-bit cache, decode over it,
// decode behind a shared prefix): checks of the torch tensors, output and
// workspace allocation, and the call into libmala.so.
//
// A serving step's calls are short (5 to 10 us of GPU time on small batches), and the
// same marshalling written in Python takes 18 to 25 us of host time.  No step of
// the computation is here: the library's functions come in as addresses from the
// ctypes binding, so that both use the one library it has loaded.
#include <Python.h>

#include <ATen/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <sstream>
#include <string>

#include "mala.h"
#include "shared_plan.h"

namespace {

decltype(&mala_cache_write) f_cache_write = nullptr;
decltype(&mala_cache_read) f_cache_read = nullptr;
decltype(&mala_decode_quant) f_decode_quant = nullptr;
decltype(&mala_decode_quant_workspace_size) f_decode_quant_ws = nullptr;
decltype(&mala_decode_shared) f_decode_shared = nullptr;
decltype(&mala_decode_shared_workspace_size) f_decode_shared_ws = nullptr;

struct Refused {                          // becomes a ValueError
  std::string what;
};

using Shape = at::IntArrayRef;

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

[[noreturn]] void refuse(const char* name, const at::Tensor& t, const char* types, Shape shape) {
  std::ostringstream s;
  s << name << " must be " << types << " " << shape << ", got " << t.scalar_type() << " " << t.sizes();
  throw Refused{s.str()};
}

void want(const char* name, const at::Tensor& t, at::ScalarType type, Shape shape) {
  if (t.scalar_type() != type || t.sizes() != shape) refuse(name, t, c10::toString(type), shape);
}

void want_float(const char* name, const at::Tensor& t, Shape shape) {
  if ((t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat) || t.sizes() != shape)
    refuse(name, t, "BFloat16 or Float", shape);
}

void want_codes(const char* name, const at::Tensor& t, Shape shape) {
  if ((t.scalar_type() != at::kFloat8_e4m3fn && t.scalar_type() != at::kByte) || t.sizes() != shape)
    refuse(name, t, "Float8_e4m3fn or Byte", shape);
}

// The device and stream of a call.  Every tensor is a contiguous CUDA tensor of the current device: the library
// launches there.
struct Place {
  int dev = -1;

  void* at(const at::Tensor& t) {
    if (!t.is_cuda() || !t.is_contiguous()) throw Refused{"tensors must be contiguous CUDA tensors"};
    if (dev < 0) dev = c10::cuda::current_device();
    if (t.get_device() != dev) {
      std::ostringstream s;
      s << "tensor on " << t.device() << ", but the current device is cuda:" << dev;
      throw Refused{s.str()};
    }
    return t.data_ptr();
  }
  at::Tensor empty(Shape shape, at::ScalarType type) const {
    return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<at::DeviceIndex>(dev)), std::nullopt));
  }
  // `stream`: None (the current one) or a cudaStream_t as a number
  void* stream(PyObject* o) const {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<at::DeviceIndex>(dev)).stream();
    void* s = PyLong_AsVoidPtr(o);
    if (s == nullptr && PyErr_Occurred()) throw python_error();
    return s;
  }
  int sms() const {
    static std::atomic<int> cache[64] = {};
    if (dev < 0 || dev >= 64) return 1;
    int n = cache[dev].load(std::memory_order_relaxed);
    if (n == 0) {
      if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
      cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
  }
};

int64_t integer(PyObject* o) {
  const int64_t x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return x;
}

float scale_of(PyObject* o, int64_t D) { return static_cast<float>(o == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : number(o)); }

int as_int(const char* name, int64_t x) {
  if (x < INT32_MIN || x > INT32_MAX) throw Refused{std::string(name) + " does not fit a 32-bit int"};
  return static_cast<int>(x);
}

mala_dtype dtype_of(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? MALA_BF16 : MALA_FP32; }

at::ScalarType type_of(int64_t code) { return code == MALA_BF16 ? at::kBFloat16 : at::kFloat; }

const int32_t* int32s(Place& p, const char* name, PyObject* o, int64_t n) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(name, o);
  want(name, t, at::kInt, {n});
  return static_cast<const int32_t*>(p.at(t));
}

struct Cache {
  const at::Tensor &kc, &ke, &vc, &ve;
  int64_t B, N, H, D;

  explicit Cache(PyObject* const* a)
      : kc(tensor("k_codes", a[0])), ke(tensor("k_exps", a[1])), vc(tensor("v_codes", a[2])), ve(tensor("v_exps", a[3])) {
    if (kc.dim() != 4) throw Refused{"cache codes must be [B, N, Hkv, D]"};
    B = kc.size(0); N = kc.size(1); H = kc.size(2); D = kc.size(3);
    want_codes("k_codes", kc, {B, N, H, D});
    want_codes("v_codes", vc, {B, N, H, D});
    want("k_exps", ke, at::kByte, {B, H, N});
    want("v_exps", ve, at::kByte, {B, H, N});
  }
};

// The call itself, without the interpreter's lock (a full launch queue makes it wait).
template <typename F>
mala_status released(F&& call) {
  PyThreadState* state = PyEval_SaveThread();
  const mala_status s = call();
  PyEval_RestoreThread(state);
  return s;
}

PyObject* result(mala_status s, const at::Tensor& a, const at::Tensor& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = x ? THPVariable_Wrap(b) : nullptr;
  PyObject* out = y ? Py_BuildValue("(iNN)", static_cast<int>(s), x, y) : nullptr;
  if (!y) Py_XDECREF(x);
  return out;
}

// (k, v, k_codes, k_exps, v_codes, v_exps, starts, new_lens, stream) -> status
PyObject* cache_write(PyObject* const* a) {
  const Cache c(a + 2);
  const at::Tensor &k = tensor("k", a[0]), &v = tensor("v", a[1]);
  const int64_t T = k.dim() == 4 ? k.size(1) : -1;
  want_float("k", k, {c.B, T, c.H, c.D});
  want("v", v, k.scalar_type(), {c.B, T, c.H, c.D});
  Place p;
  const int32_t *starts = int32s(p, "starts", a[6], c.B), *lens = int32s(p, "new_lens", a[7], c.B);
  void *pk = p.at(k), *pv = p.at(v), *kc = p.at(c.kc), *ke = p.at(c.ke), *vc = p.at(c.vc), *ve = p.at(c.ve);
  void* stream = p.stream(a[8]);
  const int B = as_int("B", c.B), t = as_int("T", T), N = as_int("N", c.N), H = as_int("Hkv", c.H), D = as_int("D", c.D);
  return PyLong_FromLong(released([&] {
    return f_cache_write(pk, pv, kc, static_cast<uint8_t*>(ke), vc, static_cast<uint8_t*>(ve), starts, lens, B, t, N, H, D,
                         dtype_of(k), stream);
  }));
}

// (k_codes, k_exps, v_codes, v_exps, k, v, T, dtype, starts, lens, zero_rest, stream) -> status, k, v; k = None:
// new [B, T, Hkv, D] tensors of the dtype code (negative: bf16); else k and v are such tensors (a negative T or dtype:
// of any)
PyObject* cache_read(PyObject* const* a) {
  const Cache c(a);
  const bool given = a[4] != Py_None;
  int64_t T = integer(a[6]);
  const int64_t code = integer(a[7]);
  at::Tensor k, v;
  if (given) {
    k = tensor("k", a[4]);
    v = tensor("v", a[5]);
    if (T < 0) T = k.dim() == 4 ? k.size(1) : -1;
    if (code < 0) want_float("k", k, {c.B, T, c.H, c.D});
    else want("k", k, type_of(code), {c.B, T, c.H, c.D});
    want("v", v, k.scalar_type(), {c.B, T, c.H, c.D});
  } else if (T < 0) {
    throw Refused{"k must be a tensor"};
  }
  Place p;
  void *kc = p.at(c.kc), *ke = p.at(c.ke), *vc = p.at(c.vc), *ve = p.at(c.ve);
  if (!given) {
    k = p.empty({c.B, T, c.H, c.D}, code < 0 ? at::kBFloat16 : type_of(code));
    v = p.empty({c.B, T, c.H, c.D}, k.scalar_type());
  }
  const int32_t *starts = int32s(p, "starts", a[8], c.B), *lens = int32s(p, "lens", a[9], c.B);
  void *pk = p.at(k), *pv = p.at(v), *stream = p.stream(a[11]);
  const int rest = as_int("zero_rest", integer(a[10]));
  const int B = as_int("B", c.B), t = as_int("T", T), N = as_int("N", c.N), H = as_int("Hkv", c.H), D = as_int("D", c.D);
  const mala_status s = released([&] {
    return f_cache_read(kc, static_cast<uint8_t*>(ke), vc, static_cast<uint8_t*>(ve), pk, pv, starts, lens, B, t, N, H, D,
                        dtype_of(k), rest, stream);
  });
  return result(s, k, v);
}

// Splits that bring the CTAs of a call to about `ctas`, at most one a tile.
int64_t splits_for(int64_t ctas, int64_t per_split, int64_t tiles) {
  return std::max<int64_t>(1, std::min<int64_t>({256, tiles, (ctas + per_split - 1) / per_split}));
}

// The dtype code of a call that makes no outputs of its own: None is refused for them.
constexpr int64_t kGivenOutputs = -2;

// Given output, or a new one of a dtype code (-1: q's type).
at::Tensor output(Place& p, const char* name, PyObject* o, Shape shape, int64_t code, const at::Tensor& q) {
  if (o == Py_None && code != kGivenOutputs) return p.empty(shape, code < 0 ? q.scalar_type() : type_of(code));
  const at::Tensor& t = tensor(name, o);
  want_float(name, t, shape);
  return t;
}

at::Tensor logs(Place& p, PyObject* o, Shape shape, int64_t code) {
  if (o == Py_None && code != kGivenOutputs) return p.empty(shape, at::kFloat);
  const at::Tensor& t = tensor("lse", o);
  want("lse", t, at::kFloat, shape);
  return t;
}

// The workspace of a call: a tensor, or memory of torch's allocator on the call's stream until the call is issued.
struct Scratch {
  void* at;
  size_t bytes;
  bool own;

  Scratch(Place& p, PyObject* o, size_t need, void* stream) : bytes(need), own(o == Py_None) {
    if (own) {
      bytes = std::max<size_t>(need, 256);
      at = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, static_cast<cudaStream_t>(stream));
    } else {
      const at::Tensor& t = tensor("workspace", o);
      at = p.at(t);
      bytes = t.nbytes();
    }
  }
  Scratch(const Scratch&) = delete;
  ~Scratch() {
    if (own) c10::cuda::CUDACachingAllocator::raw_delete(at);
  }
};

// The number of splits of a decode over a cache [B, N, Hkv, D] that is not given one.
int64_t quant_splits(const Place& p, const at::Tensor& q, const at::Tensor& k_codes, double tau) {
  const int64_t D = k_codes.size(3), tiles = (k_codes.size(1) + 127) / 128;
  const int64_t rows = std::max<int64_t>(1, k_codes.size(0) * k_codes.size(2));
  if (!(tau > 0)) return splits_for(mala::stream_ctas(static_cast<int>(D)) * p.sms(), rows, tiles);
  // Whole waves of the CTAs that the GPU holds, of about 32 tiles a CTA: each is one KV head's, and the CTAs of a
  // row of heads drift apart over a long split (128K x 8 sequences: 337 us with 32 splits, 368 with five)
  const int64_t slots = mala::skip_ctas(static_cast<int>(D), q.scalar_type() == at::kFloat) * static_cast<int64_t>(p.sms());
  const int64_t waves = std::max<int64_t>(1, std::llround(static_cast<double>(rows * tiles) / (32.0 * slots)));
  return std::max<int64_t>(1, std::min<int64_t>({256, tiles, slots * waves / rows}));
}

// (q, k_codes, tau) -> the number of splits that decode_quant takes by itself
PyObject* decode_quant_splits(PyObject* const* a) {
  const at::Tensor &q = tensor("q", a[0]), &kc = tensor("k_codes", a[1]);
  if (kc.dim() != 4) throw Refused{"cache codes must be [B, N, Hkv, D]"};
  Place p;
  p.at(kc);
  return PyLong_FromLongLong(quant_splits(p, q, kc, number(a[2])));
}

// (q, k_codes, k_exps, v_codes, v_exps, o, lse, workspace, cache_lens, counts, mask, block, num_splits, tau, scale,
// out dtype, stream) -> status, o, lse; None: a new output (unless the dtype is kGivenOutputs) or workspace, num_splits that
// fill the GPU, 1 / sqrt(D)
PyObject* decode_quant(PyObject* const* a) {
  const Cache c(a + 1);
  const at::Tensor& q = tensor("q", a[0]);
  const int64_t Hq = q.dim() == 3 ? q.size(1) : -1;
  want_float("q", q, {c.B, Hq, c.D});
  Place p;
  const int32_t* lens = int32s(p, "cache_lens", a[8], c.B);
  void *pq = p.at(q), *kc = p.at(c.kc), *ke = p.at(c.ke), *vc = p.at(c.vc), *ve = p.at(c.ve);
  const int64_t block = integer(a[11]);
  const double tau = number(a[13]);
  const int64_t splits = a[12] != Py_None ? integer(a[12]) : quant_splits(p, q, c.kc, tau);
  void *counts = nullptr, *mask = nullptr;
  if (a[9] != Py_None) {
    const at::Tensor& t = tensor("retained_counts", a[9]);
    want("retained_counts", t, at::kInt, {c.B, c.H, splits});
    counts = p.at(t);
  }
  if (a[10] != Py_None) {
    const at::Tensor& t = tensor("tile_mask", a[10]);
    want("tile_mask", t, at::kByte, {c.B, c.H, block > 0 ? (c.N + block - 1) / block : 0});
    mask = p.at(t);
  }
  const at::Tensor o = output(p, "o", a[5], {c.B, Hq, c.D}, integer(a[15]), q), lse = logs(p, a[6], {c.B, Hq}, integer(a[15]));
  const int B = as_int("B", c.B), N = as_int("N", c.N), hq = as_int("Hq", Hq), H = as_int("Hkv", c.H), D = as_int("D", c.D);
  const int blk = as_int("block", block), sp = as_int("num_splits", splits);
  void *po = p.at(o), *pl = p.at(lse), *stream = p.stream(a[16]);
  const Scratch ws(p, a[7], f_decode_quant_ws(B, hq, D, sp), stream);
  const float scale = scale_of(a[14], c.D);
  const mala_status s = released([&] {
    return f_decode_quant(pq, kc, static_cast<uint8_t*>(ke), vc, static_cast<uint8_t*>(ve), po, static_cast<float*>(pl), lens, B,
                          N, hq, H, D, dtype_of(q), dtype_of(o), blk, sp, static_cast<float>(tau), scale, ws.at, ws.bytes,
                          static_cast<int32_t*>(counts), static_cast<uint8_t*>(mask), stream);
  });
  return result(s, o, lse);
}

// (q, k_prefix, v_prefix, k_cache, v_cache, o, lse, workspace, suffix_lens, prefix_splits, suffix_splits, scale,
// out dtype, stream) -> status, o, lse; None as for decode_quant, and no caches
PyObject* decode_shared(PyObject* const* a) {
  const at::Tensor &q = tensor("q", a[0]), &kp = tensor("k_prefix", a[1]), &vp = tensor("v_prefix", a[2]);
  if (q.dim() != 3 || kp.dim() != 3) throw Refused{"q must be [B, Hq, D] and k_prefix [P, Hkv, D]"};
  const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), P = kp.size(0), H = kp.size(1);
  want_float("q", q, {B, Hq, D});
  want("k_prefix", kp, q.scalar_type(), {P, H, D});
  want("v_prefix", vp, q.scalar_type(), {P, H, D});
  if ((a[3] == Py_None) != (a[4] == Py_None)) throw Refused{"k_cache and v_cache go together"};
  int64_t N = 0;
  Place p;
  void *pkc = nullptr, *pvc = nullptr;
  if (a[3] != Py_None) {
    const at::Tensor &kc = tensor("k_cache", a[3]), &vc = tensor("v_cache", a[4]);
    N = kc.dim() == 4 ? kc.size(1) : -1;
    want("k_cache", kc, q.scalar_type(), {B, N, H, D});
    want("v_cache", vc, q.scalar_type(), {B, N, H, D});
    if (N > 0) { pkc = p.at(kc); pvc = p.at(vc); }
  }
  const int32_t* lens = int32s(p, "suffix_lens", a[8], B);
  void *pq = p.at(q), *pkp = p.at(kp), *pvp = p.at(vp);
  // sizes the plan can reckon with; the library refuses the others
  const bool sized = B > 0 && B <= 65535 && H > 0 && Hq >= H && Hq % H == 0 && Hq / H <= 128 && P > 0 && P <= INT32_MAX && N <= INT32_MAX;
  const int64_t ps = a[9] != Py_None ? integer(a[9])
                     : !sized        ? 1
                                     : mala::SharedPlan(p.sms(), static_cast<int>(B), static_cast<int>(P), static_cast<int>(N), lens != nullptr,
                                                        static_cast<int>(Hq), static_cast<int>(H)).best_splits();
  const int64_t ss = a[10] != Py_None ? integer(a[10]) : !sized ? 1 : splits_for(mala::stream_ctas(static_cast<int>(D)) * p.sms(), B * H, std::max<int64_t>(1, (N + 63) / 64));
  const at::Tensor o = output(p, "o", a[5], {B, Hq, D}, integer(a[12]), q), lse = logs(p, a[6], {B, Hq}, integer(a[12]));
  const int b = as_int("B", B), pl = as_int("P", P), n = as_int("N", N), hq = as_int("Hq", Hq), h = as_int("Hkv", H), d = as_int("D", D);
  const int psi = as_int("prefix_splits", ps), ssi = as_int("suffix_splits", ss);
  void *po = p.at(o), *plse = p.at(lse), *stream = p.stream(a[13]);
  const Scratch ws(p, a[7], f_decode_shared_ws(b, hq, d, psi, ssi), stream);
  const float scale = scale_of(a[11], D);
  const mala_status s = released([&] {
    return f_decode_shared(pq, pkp, pvp, pkc, pvc, po, static_cast<float*>(plse), lens, b, pl, n, hq, h, d, dtype_of(q),
                           dtype_of(o), psi, ssi, scale, ws.at, ws.bytes, stream);
  });
  return result(s, o, lse);
}

template <PyObject* (*fn)(PyObject* const*), int count>
PyObject* method(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != count) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", count, n);
    return nullptr;
  }
  if (f_cache_write == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "the library's functions are not bound");
    return nullptr;
  }
  try {
    return fn(args);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind(addresses): mala_cache_write, mala_cache_read, mala_decode_quant, mala_decode_quant_workspace_size,
// mala_decode_shared, mala_decode_shared_workspace_size of the loaded library
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "six addresses expected");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  f_cache_write = reinterpret_cast<decltype(f_cache_write)>(p[0]);
  f_cache_read = reinterpret_cast<decltype(f_cache_read)>(p[1]);
  f_decode_quant = reinterpret_cast<decltype(f_decode_quant)>(p[2]);
  f_decode_quant_ws = reinterpret_cast<decltype(f_decode_quant_ws)>(p[3]);
  f_decode_shared = reinterpret_cast<decltype(f_decode_shared)>(p[4]);
  f_decode_shared_ws = reinterpret_cast<decltype(f_decode_shared_ws)>(p[5]);
  Py_RETURN_NONE;
}

#define MALA_METHOD(name, count) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&method<name, count>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    MALA_METHOD(cache_write, 9),
    MALA_METHOD(cache_read, 12),
    MALA_METHOD(decode_quant, 17),
    MALA_METHOD(decode_quant_splits, 3),
    MALA_METHOD(decode_shared, 14),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
