// C ABI of libmala.so (declarations and contracts in include/mala.h):
// argument validation, workspace layout, kernel selection, device status word.

#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/mala.h"
#include "mala_internal.h"
#include "shared_plan.h"

namespace {

using namespace mala;

// Set by kernels whose bounded waits expire; read and cleared by mala_device_status.
__device__ int g_device_status = 0;

std::atomic<uint64_t> g_launches{0};
std::atomic<int> g_inject_next{0};         // one-shot failure-detection test hook
thread_local int g_last_cuda_error = 0;   // cudaError_t of this thread's last MALA_ERR_CUDA

constexpr int kMaxDevices = 64;

// Device address of a __device__ symbol on the current device, looked up once
// per device and cached (the host-side name is only a stand-in).  Concurrent
// first calls from several host threads store the same address; the slots
// are atomic, so that is well defined.
template <typename T, typename Sym>
T* symbol_address(std::atomic<T*> (&cache)[kMaxDevices], const Sym& sym) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  T* p = cache[dev].load(std::memory_order_relaxed);
  if (p == nullptr) {
    void* addr = nullptr;
    if (cudaGetSymbolAddress(&addr, sym) != cudaSuccess) return nullptr;
    p = static_cast<T*>(addr);
    cache[dev].store(p, std::memory_order_relaxed);
  }
  return p;
}

int* status_word() {
  static std::atomic<int*> cache[kMaxDevices] = {};
  return symbol_address(cache, g_device_status);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_dtype(int d) { return d == MALA_BF16 || d == MALA_FP32; }
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

mala_status finish(cudaError_t e, int launches) {
  g_launches.fetch_add(static_cast<uint64_t>(launches), std::memory_order_relaxed);
  if (e != cudaSuccess) g_last_cuda_error = static_cast<int>(e);
  return e == cudaSuccess ? MALA_OK : MALA_ERR_CUDA;
}

// Common shape checks of the prefill calls.
mala_status check_prefill(int batch, int seqlen_q, int seqlen_k, int heads_q, int heads_kv,
                          int head_dim, int in_dt, int out_dt, int causal, int block_q,
                          int block_k, float tau, float scale) {
  if (batch < 1 || seqlen_q < 1 || seqlen_k < 1 || heads_q < 1 || heads_kv < 1) return MALA_ERR_INVALID_ARG;
  if (batch > 65535 || heads_q > 65535 || heads_q % heads_kv != 0) return MALA_ERR_INVALID_ARG;
  if (!ok_dtype(in_dt) || !ok_dtype(out_dt)) return MALA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return MALA_ERR_INVALID_ARG;
  if (causal == 1 && seqlen_q != seqlen_k) return MALA_ERR_INVALID_ARG;
  if (!(tau >= 0.f) || !std::isfinite(tau)) return MALA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return MALA_ERR_INVALID_ARG;
  if (block_q < 1 || block_k < 1) return MALA_ERR_INVALID_ARG;
  if (head_dim < 1) return MALA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MALA_ERR_UNSUPPORTED;
  if (block_q != block_k || (block_q != 64 && block_q != 128)) return MALA_ERR_UNSUPPORTED;
  // the kernels number their CTAs (batch x heads x tile rows or columns) with 32-bit ints
  const int64_t tiles = (static_cast<int64_t>(seqlen_q > seqlen_k ? seqlen_q : seqlen_k) + block_q - 1) / block_q;
  if (static_cast<int64_t>(batch) * heads_q * tiles > INT32_MAX) return MALA_ERR_UNSUPPORTED;
  return MALA_OK;
}

struct BwdLayout {
  size_t delta = 0, dq_acc = 0, scratch = 0, total = 0;
};

// Scratch of mala_decode_noalloc: the per-split (m, l, u) records, at most
// kNoAllocDecodeFloats floats (4 MiB).  Every device that loads the library
// holds one copy until the process exits.
constexpr size_t kNoAllocDecodeFloats = size_t(1) << 20;
__device__ __align__(256) float g_decode_scratch[kNoAllocDecodeFloats];

// Device address of g_decode_scratch on the current device, looked up once per
// device (the host-side name is only a stand-in, not a device address).
float* decode_scratch() {
  static std::atomic<float*> cache[kMaxDevices] = {};
  return symbol_address(cache, g_decode_scratch);
}

// Workspace: D [B, Hq, Lq] fp32 | dQ accumulator fp32 (bf16 gradients only) |
// fp16 operand copies (tensor-core path: bf16 inputs, head_dim 128).
BwdLayout bwd_layout(int batch, int seqlen_q, int seqlen_k, int heads_q, int heads_kv, int head_dim,
                     int in_dt, int grad_dt) {
  BwdLayout w;
  const size_t rows = static_cast<size_t>(batch) * seqlen_q * heads_q;
  w.delta = 0;
  size_t off = round256(rows * sizeof(float));
  w.dq_acc = off;
  if (grad_dt == MALA_BF16) off += round256(rows * head_dim * sizeof(float));
  w.scratch = off;
  if (in_dt == MALA_BF16 && head_dim == 128)
    off += round256(bwd_tc_scratch_bytes(batch, seqlen_q, seqlen_k, heads_q, heads_kv, head_dim));
  w.total = off;
  return w;
}

// Argument checks shared by the decode entry points (workspace excepted).
mala_status check_decode(const void* q, const void* k_cache, const void* v_cache, const void* o,
                         const float* lse, int batch, int cache_len, int heads_q, int heads_kv,
                         int head_dim, int in_dtype, int out_dtype, int block_k, int num_splits,
                         float tau, float softmax_scale) {
  const void* ptrs[] = {q, k_cache, v_cache, o, lse};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MALA_ERR_INVALID_ARG;
  if (batch < 1 || cache_len < 1 || heads_q < 1 || heads_kv < 1 || heads_q % heads_kv != 0)
    return MALA_ERR_INVALID_ARG;
  if (batch > 65535 || heads_kv > 65535) return MALA_ERR_INVALID_ARG;
  if (!ok_dtype(in_dtype) || !ok_dtype(out_dtype)) return MALA_ERR_INVALID_ARG;
  if (!(tau >= 0.f) || !std::isfinite(tau)) return MALA_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale)) return MALA_ERR_INVALID_ARG;
  if (num_splits < 1 || num_splits > 256 || block_k < 1 || head_dim < 1) return MALA_ERR_INVALID_ARG;
  const int g = heads_q / heads_kv;
  if (g != 1 && g != 2 && g != 4 && g != 8) return MALA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return MALA_ERR_UNSUPPORTED;
  if (block_k != 64 && block_k != 128) return MALA_ERR_UNSUPPORTED;
  return MALA_OK;
}

// Split kernel (tensor-core or CUDA-core) then the exact merge.
mala_status run_decode(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                       const int32_t* cache_lens, int batch, int cache_len, int heads_q, int heads_kv,
                       int head_dim, int in_dtype, int out_dtype, int block_k, int num_splits, float tau,
                       float softmax_scale, float* partial, int32_t* retained_counts, uint8_t* tile_mask,
                       int* status, void* stream, int per_head = 0) {
  DecArgs a{};
  a.q = q; a.k = k_cache; a.v = v_cache; a.o = o; a.lse = lse;
  a.B = batch; a.N = cache_len; a.Hq = heads_q; a.Hkv = heads_kv; a.D = head_dim;
  a.lens = cache_lens;
  a.in_dt = in_dtype; a.out_dt = out_dtype; a.blk = block_k; a.splits = num_splits;
  a.tau = tau; a.log2_tau = tau > 0.f ? std::log2(tau) : 0.f;
  a.scale_log2 = softmax_scale * kLog2e;
  a.partial = partial;
  a.per_head = per_head;
  a.counts = retained_counts; a.mask = tile_mask; a.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int launches = 0;
  cudaError_t e = decode_mma_supported(a) ? launch_decode_mma(a, s, &launches) : launch_decode_simt(a, s, &launches);
  if (e == cudaSuccess) e = launch_decode_merge(a, s, &launches);
  return finish(e, launches);
}

bool workspace_ok(const void* workspace, size_t workspace_bytes, size_t need) {
  return workspace && (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0 && workspace_bytes >= need;
}

// Forward of B sequences of Lq / Lk rows (cu == null) or of a packed batch
// (cu != null, Lq = Lk = total rows, each sequence at most Lmax long).
mala_status run_fwd(const void* q, const void* k, const void* v, void* o, float* lse, const int32_t* cu,
                    int batch, int seqlen_q, int seqlen_k, int lmax, int heads_q, int heads_kv, int head_dim,
                    int in_dtype, int out_dtype, int causal, int block_q, int block_k, float tau,
                    float softmax_scale, int32_t* retained_counts, uint8_t* tile_mask, void* stream,
                    const uint8_t* force = nullptr) {
  if (!q || !k || !v || !o || !lse) return MALA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return MALA_ERR_INVALID_ARG;
  mala_status st = check_prefill(batch, seqlen_q, seqlen_k, heads_q, heads_kv, head_dim, in_dtype,
                                 out_dtype, causal, block_q, block_k, tau, softmax_scale);
  if (st != MALA_OK) return st;
  int* status = status_word();
  if (!status) return MALA_ERR_CUDA;
  FwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.o = o; a.lse = lse;
  a.B = batch; a.Lq = seqlen_q; a.Lk = seqlen_k; a.Hq = heads_q; a.Hkv = heads_kv; a.D = head_dim;
  a.cu = cu; a.Lmax = lmax;
  a.in_dt = in_dtype; a.out_dt = out_dtype; a.causal = causal; a.blk = block_q;
  a.tau = tau; a.log2_tau = tau > 0.f ? std::log2(tau) : 0.f;
  a.scale_log2 = softmax_scale * kLog2e;
  a.counts = retained_counts; a.mask = tile_mask; a.status = status;
  a.force = force;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int launches = 0;
  // forced decisions run on the CUDA-core kernel (an evaluation path)
  const bool tc = force == nullptr && fwd_tc_supported(a);
  if (tc) a.inject = g_inject_next.exchange(0);
  cudaError_t e = tc ? launch_fwd_tc(a, s, &launches) : launch_fwd_simt(a, s, &launches);
  return finish(e, launches);
}

// Host-side checks of a packed batch (the bounds themselves are checked on the device).
bool check_packed(const int32_t* cu, int batch, int total, int lmax) {
  return cu && (reinterpret_cast<uintptr_t>(cu) & 3u) == 0 && batch >= 1 && total >= 1 && lmax >= 1 &&
         lmax <= total;
}

// Backward of B sequences of Lq / Lk rows (cu == null) or of a packed batch
// (cu != null, Lq = Lk = total rows, each sequence at most Lmax long).
mala_status run_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                    void* dq, void* dk, void* dv, const int32_t* cu, int batch, int seqlen_q, int seqlen_k,
                    int lmax, int heads_q, int heads_kv, int head_dim, int in_dtype, int grad_dtype, int causal,
                    int block_q, int block_k, float tau, float softmax_scale, void* workspace,
                    size_t workspace_bytes, int32_t* retained_counts, uint8_t* tile_mask, void* stream) {
  const void* ptrs[] = {q, k, v, o, dout, lse, dq, dk, dv};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MALA_ERR_INVALID_ARG;
  mala_status st = check_prefill(batch, seqlen_q, seqlen_k, heads_q, heads_kv, head_dim, in_dtype,
                                 grad_dtype, causal, block_q, block_k, tau, softmax_scale);
  if (st != MALA_OK) return st;
  // a packed batch is laid out as one run of seqlen_q = seqlen_k = total rows
  const BwdLayout w = bwd_layout(cu ? 1 : batch, seqlen_q, seqlen_k, heads_q, heads_kv, head_dim, in_dtype,
                                 grad_dtype);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < w.total)
    return MALA_ERR_WORKSPACE;
  int* status = status_word();
  if (!status) return MALA_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  BwdArgs a{};
  a.q = q; a.k = k; a.v = v; a.o = o; a.dout = dout; a.lse = lse; a.dq = dq; a.dk = dk; a.dv = dv;
  a.B = batch; a.Lq = seqlen_q; a.Lk = seqlen_k; a.Hq = heads_q; a.Hkv = heads_kv; a.D = head_dim;
  a.cu = cu; a.Lmax = lmax;
  a.in_dt = in_dtype; a.grad_dt = grad_dtype; a.causal = causal; a.blk = block_q;
  a.tau = tau; a.log2_tau = tau > 0.f ? std::log2(tau) : 0.f;
  a.scale_log2 = softmax_scale * kLog2e; a.scale = softmax_scale;
  a.delta = reinterpret_cast<float*>(ws + w.delta);
  a.dq_acc = grad_dtype == MALA_FP32 ? static_cast<float*>(dq) : reinterpret_cast<float*>(ws + w.dq_acc);
  a.scratch = ws + w.scratch;
  a.counts = retained_counts; a.mask = tile_mask; a.status = status;
  const bool tc = bwd_tc_supported(a);
  if (!tc && bwd_simt_smem(in_dtype, head_dim, block_q) > 227u * 1024u) return MALA_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int launches = 0;
  cudaError_t e = cudaSuccess;
  if (tc) {
    e = launch_bwd_tc(a, s, &launches);
  } else {
    e = launch_bwd_preprocess(a, s, &launches);
    if (e == cudaSuccess) e = launch_bwd_simt(a, s, &launches);
  }
  if (e == cudaSuccess && grad_dtype == MALA_BF16) e = launch_dq_convert(a, s, &launches);
  return finish(e, launches);
}

constexpr int kMaxRows = INT32_MAX - 1024;     // the serving kernels round row numbers up to whole tiles in 32 bits

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }   // null included

mala_status run_cache(const void* k, const void* v, const void* k_codes, const uint8_t* k_exps, const void* v_codes,
                      const uint8_t* v_exps, const int32_t* starts, const int32_t* lens, int batch, int len,
                      int cache_len, int heads_kv, int head_dim, int dtype, int zero_rest, void* stream,
                      cudaError_t (*launch)(const CacheArgs&, cudaStream_t, int*)) {
  const void* ptrs[] = {k, v, k_codes, v_codes};
  for (const void* p : ptrs)
    if (!p || !aligned16(p)) return MALA_ERR_INVALID_ARG;
  if (!k_exps || !v_exps) return MALA_ERR_INVALID_ARG;       // bytes: any alignment
  if (!aligned4(starts) || !aligned4(lens)) return MALA_ERR_INVALID_ARG;
  if (batch < 1 || batch > 65535 || len < 1 || cache_len < 1 || heads_kv < 1 || heads_kv > 32767 || head_dim < 1)
    return MALA_ERR_INVALID_ARG;
  if (!ok_dtype(dtype) || (zero_rest != 0 && zero_rest != 1)) return MALA_ERR_INVALID_ARG;
  // without starts or lens every span is known here
  if (!starts && !lens && len > cache_len) return MALA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MALA_ERR_UNSUPPORTED;
  // a span's (token, head) rows are numbered with 32-bit ints
  if (static_cast<int64_t>(len) * heads_kv > INT32_MAX - 65536) return MALA_ERR_UNSUPPORTED;
  int* status = status_word();
  if (!status) return MALA_ERR_CUDA;
  CacheArgs a{};
  a.k = const_cast<void*>(k); a.v = const_cast<void*>(v);
  a.k_codes = static_cast<uint8_t*>(const_cast<void*>(k_codes)); a.k_exps = const_cast<uint8_t*>(k_exps);
  a.v_codes = static_cast<uint8_t*>(const_cast<void*>(v_codes)); a.v_exps = const_cast<uint8_t*>(v_exps);
  a.starts = starts; a.lens = lens;
  a.B = batch; a.T = len; a.N = cache_len; a.Hkv = heads_kv; a.D = head_dim; a.dt = dtype;
  a.zero_rest = zero_rest;
  a.status = status;
  int launches = 0;
  const cudaError_t e = launch(a, static_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

}  // namespace

extern "C" {

const char* mala_status_string(mala_status status) {
  switch (status) {
    case MALA_OK: return "MALA_OK";
    case MALA_ERR_INVALID_ARG: return "MALA_ERR_INVALID_ARG";
    case MALA_ERR_UNSUPPORTED: return "MALA_ERR_UNSUPPORTED";
    case MALA_ERR_WORKSPACE: return "MALA_ERR_WORKSPACE";
    case MALA_ERR_CUDA: return "MALA_ERR_CUDA";
    case MALA_ERR_TIMEOUT: return "MALA_ERR_TIMEOUT";
  }
  return "MALA_ERR_UNKNOWN";
}

mala_status mala_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                     int batch, int seqlen_q, int seqlen_k, int heads_q, int heads_kv,
                     int head_dim, mala_dtype in_dtype, mala_dtype out_dtype, int causal,
                     int block_q, int block_k, float tau, float softmax_scale,
                     int32_t* retained_counts, uint8_t* tile_mask, void* stream) {
  return run_fwd(q, k, v, o, lse, nullptr, batch, seqlen_q, seqlen_k, seqlen_q, heads_q, heads_kv, head_dim,
                 in_dtype, out_dtype, causal, block_q, block_k, tau, softmax_scale, retained_counts, tile_mask,
                 stream);
}

mala_status mala_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                            const int32_t* cu_seqlens, int batch, int total_tokens, int max_seqlen,
                            int heads_q, int heads_kv, int head_dim, mala_dtype in_dtype,
                            mala_dtype out_dtype, int causal, int block_q, int block_k, float tau,
                            float softmax_scale, int32_t* retained_counts, uint8_t* tile_mask,
                            void* stream) {
  if (!check_packed(cu_seqlens, batch, total_tokens, max_seqlen)) return MALA_ERR_INVALID_ARG;
  return run_fwd(q, k, v, o, lse, cu_seqlens, batch, total_tokens, total_tokens, max_seqlen, heads_q, heads_kv,
                 head_dim, in_dtype, out_dtype, causal, block_q, block_k, tau, softmax_scale, retained_counts,
                 tile_mask, stream);
}

mala_status mala_fwd_forced(const void* q, const void* k, const void* v, void* o, float* lse,
                            int batch, int seqlen_q, int seqlen_k, int heads_q, int heads_kv,
                            int head_dim, mala_dtype in_dtype, mala_dtype out_dtype, int causal,
                            int block_q, int block_k, float softmax_scale, const uint8_t* tile_keep,
                            int32_t* retained_counts, uint8_t* tile_mask, void* stream) {
  if (!tile_keep) return MALA_ERR_INVALID_ARG;
  return run_fwd(q, k, v, o, lse, nullptr, batch, seqlen_q, seqlen_k, seqlen_q, heads_q, heads_kv, head_dim,
                 in_dtype, out_dtype, causal, block_q, block_k, 0.f, softmax_scale, retained_counts, tile_mask,
                 stream, tile_keep);
}

mala_status mala_region_mass(const void* q, const void* k, const float* lse, float* region_mass,
                             int batch, int seqlen_q, int seqlen_k, int heads_q, int heads_kv,
                             int head_dim, mala_dtype in_dtype, int causal, int block_q, int block_k,
                             float softmax_scale, void* stream) {
  if (!q || !k || !lse || !region_mass) return MALA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(region_mass) & 3u))
    return MALA_ERR_INVALID_ARG;
  mala_status st = check_prefill(batch, seqlen_q, seqlen_k, heads_q, heads_kv, head_dim, in_dtype, in_dtype,
                                 causal, block_q, block_k, 0.f, softmax_scale);
  if (st != MALA_OK) return st;
  FwdArgs a{};
  a.q = q; a.k = k; a.lse = const_cast<float*>(lse); a.region_mass = region_mass;
  a.B = batch; a.Lq = seqlen_q; a.Lk = seqlen_k; a.Hq = heads_q; a.Hkv = heads_kv; a.D = head_dim;
  a.Lmax = seqlen_q;
  a.in_dt = in_dtype; a.out_dt = in_dtype; a.causal = causal; a.blk = block_q;
  a.scale_log2 = softmax_scale * kLog2e;
  int launches = 0;
  cudaError_t e = launch_region_mass(a, static_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

size_t mala_bwd_workspace_size(int batch, int seqlen_q, int seqlen_k, int heads_q, int heads_kv,
                               int head_dim, mala_dtype in_dtype, mala_dtype grad_dtype) {
  if (batch < 1 || seqlen_q < 1 || seqlen_k < 1 || heads_q < 1 || heads_kv < 1 || head_dim < 1) return 0;
  return bwd_layout(batch, seqlen_q, seqlen_k, heads_q, heads_kv, head_dim, in_dtype, grad_dtype).total;
}

mala_status mala_bwd(const void* q, const void* k, const void* v, const void* o,
                     const void* dout, const float* lse, void* dq, void* dk, void* dv,
                     int batch, int seqlen_q, int seqlen_k, int heads_q, int heads_kv,
                     int head_dim, mala_dtype in_dtype, mala_dtype grad_dtype, int causal,
                     int block_q, int block_k, float tau, float softmax_scale,
                     void* workspace, size_t workspace_bytes,
                     int32_t* retained_counts, uint8_t* tile_mask, void* stream) {
  return run_bwd(q, k, v, o, dout, lse, dq, dk, dv, nullptr, batch, seqlen_q, seqlen_k, seqlen_q, heads_q,
                 heads_kv, head_dim, in_dtype, grad_dtype, causal, block_q, block_k, tau, softmax_scale,
                 workspace, workspace_bytes, retained_counts, tile_mask, stream);
}

size_t mala_bwd_varlen_workspace_size(int total_tokens, int heads_q, int heads_kv, int head_dim,
                                      mala_dtype in_dtype, mala_dtype grad_dtype) {
  return mala_bwd_workspace_size(1, total_tokens, total_tokens, heads_q, heads_kv, head_dim, in_dtype, grad_dtype);
}

mala_status mala_bwd_varlen(const void* q, const void* k, const void* v, const void* o,
                            const void* dout, const float* lse, void* dq, void* dk, void* dv,
                            const int32_t* cu_seqlens, int batch, int total_tokens, int max_seqlen,
                            int heads_q, int heads_kv, int head_dim, mala_dtype in_dtype,
                            mala_dtype grad_dtype, int causal, int block_q, int block_k, float tau,
                            float softmax_scale, void* workspace, size_t workspace_bytes,
                            int32_t* retained_counts, uint8_t* tile_mask, void* stream) {
  if (!check_packed(cu_seqlens, batch, total_tokens, max_seqlen)) return MALA_ERR_INVALID_ARG;
  return run_bwd(q, k, v, o, dout, lse, dq, dk, dv, cu_seqlens, batch, total_tokens, total_tokens, max_seqlen,
                 heads_q, heads_kv, head_dim, in_dtype, grad_dtype, causal, block_q, block_k, tau, softmax_scale,
                 workspace, workspace_bytes, retained_counts, tile_mask, stream);
}

size_t mala_decode_workspace_size(int batch, int heads_q, int head_dim, int num_splits) {
  if (batch < 1 || heads_q < 1 || head_dim < 1 || num_splits < 1) return 0;
  return round256(static_cast<size_t>(num_splits) * batch * heads_q * (head_dim + 4) * sizeof(float));
}

mala_status mala_decode(const void* q, const void* k_cache, const void* v_cache, void* o,
                        float* lse, int batch, int cache_len, int heads_q, int heads_kv,
                        int head_dim, mala_dtype in_dtype, mala_dtype out_dtype, int block_k,
                        int num_splits, float tau, float softmax_scale,
                        void* workspace, size_t workspace_bytes,
                        int32_t* retained_counts, uint8_t* tile_mask, void* stream) {
  const mala_status c = check_decode(q, k_cache, v_cache, o, lse, batch, cache_len, heads_q, heads_kv, head_dim,
                                     in_dtype, out_dtype, block_k, num_splits, tau, softmax_scale);
  if (c != MALA_OK) return c;
  if (!workspace_ok(workspace, workspace_bytes, mala_decode_workspace_size(batch, heads_q, head_dim, num_splits)))
    return MALA_ERR_WORKSPACE;
  int* status = status_word();
  if (!status) return MALA_ERR_CUDA;
  return run_decode(q, k_cache, v_cache, o, lse, nullptr, batch, cache_len, heads_q, heads_kv, head_dim, in_dtype,
                    out_dtype, block_k, num_splits, tau, softmax_scale, static_cast<float*>(workspace),
                    retained_counts, tile_mask, status, stream);
}

mala_status mala_decode_per_head(const void* q, const void* k_cache, const void* v_cache, void* o,
                                 float* lse, int batch, int cache_len, int heads_q, int heads_kv,
                                 int head_dim, mala_dtype in_dtype, mala_dtype out_dtype, int block_k,
                                 int num_splits, float tau, float softmax_scale,
                                 void* workspace, size_t workspace_bytes,
                                 int32_t* retained_counts, uint8_t* tile_mask, void* stream) {
  const mala_status c = check_decode(q, k_cache, v_cache, o, lse, batch, cache_len, heads_q, heads_kv, head_dim,
                                     in_dtype, out_dtype, block_k, num_splits, tau, softmax_scale);
  if (c != MALA_OK) return c;
  if (!workspace_ok(workspace, workspace_bytes, mala_decode_workspace_size(batch, heads_q, head_dim, num_splits)))
    return MALA_ERR_WORKSPACE;
  int* status = status_word();
  if (!status) return MALA_ERR_CUDA;
  return run_decode(q, k_cache, v_cache, o, lse, nullptr, batch, cache_len, heads_q, heads_kv, head_dim, in_dtype,
                    out_dtype, block_k, num_splits, tau, softmax_scale, static_cast<float*>(workspace),
                    retained_counts, tile_mask, status, stream, /*per_head=*/1);
}

mala_status mala_decode_varlen(const void* q, const void* k_cache, const void* v_cache, void* o,
                               float* lse, const int32_t* cache_lens, int batch, int max_cache_len,
                               int heads_q, int heads_kv, int head_dim, mala_dtype in_dtype,
                               mala_dtype out_dtype, int block_k, int num_splits, float tau,
                               float softmax_scale, void* workspace, size_t workspace_bytes,
                               int32_t* retained_counts, uint8_t* tile_mask, void* stream) {
  if (!cache_lens || (reinterpret_cast<uintptr_t>(cache_lens) & 3u) != 0) return MALA_ERR_INVALID_ARG;
  const mala_status c = check_decode(q, k_cache, v_cache, o, lse, batch, max_cache_len, heads_q, heads_kv,
                                     head_dim, in_dtype, out_dtype, block_k, num_splits, tau, softmax_scale);
  if (c != MALA_OK) return c;
  if (!workspace_ok(workspace, workspace_bytes, mala_decode_workspace_size(batch, heads_q, head_dim, num_splits)))
    return MALA_ERR_WORKSPACE;
  int* status = status_word();
  if (!status) return MALA_ERR_CUDA;
  return run_decode(q, k_cache, v_cache, o, lse, cache_lens, batch, max_cache_len, heads_q, heads_kv, head_dim,
                    in_dtype, out_dtype, block_k, num_splits, tau, softmax_scale, static_cast<float*>(workspace),
                    retained_counts, tile_mask, status, stream);
}

mala_status mala_decode_noalloc(const void* q, const void* k_cache, const void* v_cache, void* o,
                                float* lse, int batch, int cache_len, int heads_q, int heads_kv,
                                int head_dim, mala_dtype in_dtype, mala_dtype out_dtype, int block_k,
                                int num_splits, float tau, float softmax_scale,
                                int32_t* retained_counts, uint8_t* tile_mask, void* stream) {
  const mala_status c = check_decode(q, k_cache, v_cache, o, lse, batch, cache_len, heads_q, heads_kv, head_dim,
                                     in_dtype, out_dtype, block_k, num_splits, tau, softmax_scale);
  if (c != MALA_OK) return c;
  const size_t need = static_cast<size_t>(num_splits) * batch * heads_q * (head_dim + 4);
  if (need > kNoAllocDecodeFloats) return MALA_ERR_WORKSPACE;
  float* scratch = decode_scratch();
  int* status = status_word();
  if (!scratch || !status) return MALA_ERR_CUDA;
  return run_decode(q, k_cache, v_cache, o, lse, nullptr, batch, cache_len, heads_q, heads_kv, head_dim, in_dtype,
                    out_dtype, block_k, num_splits, tau, softmax_scale, scratch, retained_counts, tile_mask,
                    status, stream);
}

mala_status mala_cache_write(const void* k, const void* v, void* k_codes, uint8_t* k_exps, void* v_codes,
                             uint8_t* v_exps, const int32_t* starts, const int32_t* new_lens, int batch, int new_len,
                             int cache_len, int heads_kv, int head_dim, mala_dtype in_dtype, void* stream) {
  return run_cache(k, v, k_codes, k_exps, v_codes, v_exps, starts, new_lens, batch, new_len, cache_len, heads_kv,
                   head_dim, in_dtype, 0, stream, launch_cache_write);
}

mala_status mala_cache_read(const void* k_codes, const uint8_t* k_exps, const void* v_codes, const uint8_t* v_exps,
                            void* k, void* v, const int32_t* starts, const int32_t* lens, int batch, int len,
                            int cache_len, int heads_kv, int head_dim, mala_dtype out_dtype, int zero_rest,
                            void* stream) {
  return run_cache(k, v, k_codes, k_exps, v_codes, v_exps, starts, lens, batch, len, cache_len, heads_kv, head_dim,
                   out_dtype, zero_rest, stream, launch_cache_read);
}

// Dense: at most four workers a split and sequence, and one record more a sequence for the cuts inside a worker.
size_t mala_decode_quant_workspace_size(int batch, int heads_q, int head_dim, int num_splits) {
  if (num_splits < 1 || num_splits > 256) return 0;
  return mala_decode_workspace_size(batch, heads_q, head_dim, 4 * num_splits + 1);
}

mala_status mala_decode_quant(const void* q, const void* k_codes, const uint8_t* k_exps, const void* v_codes,
                              const uint8_t* v_exps, void* o, float* lse, const int32_t* cache_lens, int batch,
                              int cache_len, int heads_q, int heads_kv, int head_dim, mala_dtype q_dtype,
                              mala_dtype out_dtype, int block_k, int num_splits, float tau, float softmax_scale,
                              void* workspace, size_t workspace_bytes, int32_t* retained_counts, uint8_t* tile_mask,
                              void* stream) {
  const mala_status c = check_decode(q, k_codes, v_codes, o, lse, batch, cache_len, heads_q, heads_kv, head_dim,
                                     q_dtype, out_dtype, block_k, num_splits, tau, softmax_scale);
  if (c != MALA_OK) return c;
  if (!k_exps || !v_exps || !aligned4(cache_lens)) return MALA_ERR_INVALID_ARG;      // exponents: any alignment
  if (block_k != 128 || cache_len > kMaxRows) return MALA_ERR_UNSUPPORTED;
  if (!workspace_ok(workspace, workspace_bytes, mala_decode_quant_workspace_size(batch, heads_q, head_dim, num_splits)))
    return MALA_ERR_WORKSPACE;
  // the dense pass numbers its CTAs with 32-bit ints
  if (static_cast<int64_t>(num_splits) * batch * heads_kv > INT32_MAX) return MALA_ERR_UNSUPPORTED;
  int* status = status_word();
  if (!status) return MALA_ERR_CUDA;
  StreamArgs a{};
  a.q = q; a.o = o; a.lse = lse;
  a.k = k_codes; a.v = v_codes; a.k_exps = k_exps; a.v_exps = v_exps;
  a.lens = cache_lens;
  a.B = batch; a.N = cache_len; a.Hq = heads_q; a.Hkv = heads_kv; a.D = head_dim;
  a.q_dt = q_dtype; a.out_dt = out_dtype; a.splits = num_splits; a.min_len = 1;
  a.log2_tau = tau > 0.f ? std::log2(tau) : 0.f;
  a.scale_log2 = softmax_scale * kLog2e;
  a.partial = static_cast<float*>(workspace);
  a.counts = retained_counts; a.mask = tile_mask; a.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int launches = 0;
  cudaError_t e;
  if (tau > 0.f) {
    a.records = num_splits;
    e = launch_decode_quant(a, s, &launches);
  } else {
    a.spread = a.partial;
    stream_divide(a, 0);
    e = launch_stream(a, s, &launches);
  }
  if (e == cudaSuccess) e = launch_stream_merge(a, s, &launches);
  return finish(e, launches);
}

size_t mala_decode_shared_workspace_size(int batch, int heads_q, int head_dim, int prefix_splits,
                                         int suffix_splits) {
  if (prefix_splits < 1 || prefix_splits > 256 || suffix_splits < 1 || suffix_splits > 256) return 0;
  return mala_decode_workspace_size(batch, heads_q, head_dim, prefix_splits + 4 * suffix_splits + 1);
}

mala_status mala_decode_shared(const void* q, const void* k_prefix, const void* v_prefix, const void* k_cache,
                               const void* v_cache, void* o, float* lse, const int32_t* suffix_lens, int batch,
                               int prefix_len, int max_suffix_len, int heads_q, int heads_kv, int head_dim,
                               mala_dtype in_dtype, mala_dtype out_dtype, int prefix_splits, int suffix_splits,
                               float softmax_scale, void* workspace, size_t workspace_bytes, void* stream) {
  const mala_status c = check_decode(q, k_prefix, v_prefix, o, lse, batch, prefix_len, heads_q, heads_kv, head_dim,
                                     in_dtype, out_dtype, 128, prefix_splits, 0.f, softmax_scale);
  if (c != MALA_OK) return c;
  if (max_suffix_len < 0 || suffix_splits < 1 || suffix_splits > 256 || !aligned4(suffix_lens))
    return MALA_ERR_INVALID_ARG;
  if (max_suffix_len > 0 && (!k_cache || !v_cache)) return MALA_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return MALA_ERR_INVALID_ARG;
  if (in_dtype != MALA_BF16 || prefix_len > kMaxRows || max_suffix_len > kMaxRows) return MALA_ERR_UNSUPPORTED;
  // the kernels number their CTAs with 32-bit ints
  if ((static_cast<int64_t>(prefix_blocks(batch, heads_q, heads_kv)) + 1) / 2 * heads_kv * prefix_splits > INT32_MAX ||
      static_cast<int64_t>(batch) * heads_kv * suffix_splits > INT32_MAX)
    return MALA_ERR_UNSUPPORTED;
  if (!workspace_ok(workspace, workspace_bytes,
                    mala_decode_shared_workspace_size(batch, heads_q, head_dim, prefix_splits, suffix_splits)))
    return MALA_ERR_WORKSPACE;
  int* status = status_word();
  if (!status) return MALA_ERR_CUDA;
  StreamArgs a{};
  a.q = q; a.o = o; a.lse = lse;
  a.B = batch; a.Hq = heads_q; a.Hkv = heads_kv; a.D = head_dim;
  a.q_dt = in_dtype; a.out_dt = out_dtype;
  a.scale_log2 = softmax_scale * kLog2e;
  a.partial = static_cast<float*>(workspace);
  a.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int launches = 0;
  a.records = prefix_splits;
  a.k = k_prefix; a.v = v_prefix; a.N = prefix_len; a.splits = prefix_splits;
  cudaError_t e = launch_prefix_tc(a, s, &launches);
  a.N = max_suffix_len; a.lens = suffix_lens;
  if (e == cudaSuccess && max_suffix_len > 0) {
    a.k = k_cache; a.v = v_cache; a.splits = suffix_splits; a.after_prefix = 1;
    a.spread = a.partial + static_cast<size_t>(a.records) * batch * heads_q * (head_dim + 4);
    // Where the SMs that the prefix pass leaves can be done with the suffix pass by its end, it is cut for them alone
    // (32 x (8192 + 512): 20.7 us, cut for all SMs 25.5); else for all SMs, and its later CTAs follow the prefix's.
    const SharedPlan plan(sm_count(), batch, prefix_len, max_suffix_len, suffix_lens != nullptr, heads_q, heads_kv);
    stream_divide(a, static_cast<int>(plan.beside(prefix_splits)));
    e = launch_stream(a, s, &launches);
  }
  if (e == cudaSuccess) e = launch_stream_merge(a, s, &launches);
  return finish(e, launches);
}

size_t mala_decode_noalloc_max_floats(void) { return kNoAllocDecodeFloats; }

mala_status mala_device_status(void* stream, int* device_code) {
  if (!device_code) return MALA_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return MALA_ERR_CUDA;
  int word = 0;
  if (cudaMemcpyFromSymbol(&word, g_device_status, sizeof(int)) != cudaSuccess) return MALA_ERR_CUDA;
  const int zero = 0;
  if (word != 0 && cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int)) != cudaSuccess) return MALA_ERR_CUDA;
  *device_code = word;
  if (word & kStatusWaitTimeout) return MALA_ERR_TIMEOUT;
  return word == 0 ? MALA_OK : MALA_ERR_INVALID_ARG;
}

uint64_t mala_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

void mala_test_drop_next_load(void) { g_inject_next.store(1); }

int mala_last_cuda_error(void) { return g_last_cuda_error; }

const char* mala_cuda_error_string(int code) { return cudaGetErrorString(static_cast<cudaError_t>(code)); }

}  // extern "C"
