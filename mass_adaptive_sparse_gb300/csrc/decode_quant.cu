// MALA split-KV decode over the 8-bit cache (tau > 0; dense passes:
// decode_stream.cu).
//
// mala_decode's rule on what the cache stands for ("MassAlloc Attention: Let
// Attention Allocate Its Own Compute", §2.2 Eq. (3), App. A.1): a split starts
// from its own empty (m, l), visits its 128-key tiles newest to oldest, scores
// each, and skips a tile whose largest score, for every query head of the KV
// head's group, stays below m + log l + log(tau / L).  A skipped tile loads no V.
//
// Bound: HBM, D + 2 bytes a key and KV head (the value's exponent comes with the
// key's), D more in a kept tile.  8 sequences of 128K keys at tau = 1, 28
// splits, every tile kept: 324 us, 6.7 TB/s (dense on that machine: 314).
//
// One CTA of four warps per (KV head, split, sequence), a warp owns 32 keys of
// every tile.  One barrier a tile exchanges the warps' maxima and sums; every
// warp then takes the decision for itself.  The P V product of a kept tile is
// held back by one kept tile, so that its V, loaded at the decision, lands
// behind the next tile's scores.
#include "shared_plan.h"
#include "stream_common.cuh"

namespace mala {
namespace {

using namespace stream;

template <int D, bool kWide>
__global__ void __launch_bounds__(32 * kWarps, skip_ctas(D, kWide))
decode_quant_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const StreamArgs a) {
  using L = Layout<D, true>;
  constexpr int S = L::kStages, kTile = kWarps * L::kKeys;
  static_assert(S >= 2, "a V stage to land while the previous one is read");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_k[S], full_v[S];
  __shared__ int abort_flag;
  __shared__ float xmax[2][kWarps][8], xl[2][kWarps][8], xm[kWarps][8], xsum[kWarps][8];

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, gq = lane >> 2, cq = lane & 3;
  const int hk = blockIdx.x, sp = blockIdx.y, b = blockIdx.z, G = a.Hq / a.Hkv;
  grid_wait();                           // what ran before on the stream is complete; then the merge may start, which
  grid_launch_dependents();              // reads the lengths at once
  Running<D, true, kWide> run;
  const auto raw_q = run.q.fetch(a, b, hk);      // ahead of the ring's loads, or it queues behind them
  run.reset();
  const int n = stream_len(a, b);        // 0 for a rejected length
  const int T = (n + kTile - 1) / kTile, Tmax = (a.N + kTile - 1) / kTile;
  const int per = (T + a.splits - 1) / a.splits;
  const int t0 = min(T, sp * per), t1 = min(T, t0 + per), rounds = t1 - t0;

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sk = base, sv = base + S * L::kStageBytes;    // stages of a whole tile: the warps' sub-tiles in turn
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&full_k[i]), 1);
      mbar_init(smem_u32(&full_v[i]), 1);
    }
    abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&mk);
    prefetch_tensormap(&mv);
  }
  __syncthreads();
  volatile int* abortp = &abort_flag;

  auto issue_k = [&](int i) {
    load_step<D, true>(&mk, sk + (i % S) * L::kStageBytes, smem_u32(&full_k[i % S]), hk, (t1 - 1 - i) * kTile, b, n, a);
  };
  if (tid == 0)
    for (int i = 0; i < min(rounds, S); ++i) issue_k(i);
  int k_issued = min(rounds, S);

  // Exponent bytes of this warp's keys, one key a lane, a round ahead of their use.  Nothing but the loads may stand
  // here: any arithmetic on them would wait for them a round early.
  uint32_t ke_next = 0, ve_next = 0;
  auto key_of = [&](int i) { return (t1 - 1 - i) * kTile + warp * L::kKeys; };   // this warp's first key in round i
  auto load_exps = [&](int i) {
    const int key = key_of(i) + lane;
    ke_next = ve_next = 0;
    if (i < rounds && key < n) {
      const size_t at = (static_cast<size_t>(b) * a.Hkv + hk) * a.N + key;
      ke_next = a.k_exps[at];
      ve_next = a.v_exps[at];
    }
  };
  load_exps(0);
  run.q.set(a, raw_q);

  const int g = lane & 7;                // the head this lane decides
  const float thr = a.log2_tau - log2f(static_cast<float>(n));
  float m_g = -INFINITY;                 // its reference (the same in every warp)
  int kept = 0;
  bool ok = true;
  // the previous kept tile's weights, whose product waits for its V
  typename Running<D, true, kWide>::Weights pend;
  bool waiting = false;
  int pend_key = 0;
  auto finish_pending = [&](int v) {     // v: the kept tile's number
    if (!waiting) return;
    ok = mbar_wait(smem_u32(&full_v[v % S]), (v / S) & 1, abortp, a.status) && ok;
    if (__all_sync(kFull, ok)) run.values(sv + v % S * L::kStageBytes + warp * L::kSub, pend_key, n, pend);
    waiting = false;
  };

  // After a timed-out wait the loop runs on (waits then fail at once), so the CTA's barriers always stay matched.
  for (int i = 0; i < rounds; ++i) {
    const int s = i % S, key0 = key_of(i), j = t1 - 1 - i;
    const uint32_t ke = ke_next, ve = ve_next;
    load_exps(i + 1);
    float acc[2][4];
    ok = mbar_wait(smem_u32(&full_k[s]), (i / S) & 1, abortp, a.status) && ok;
    if (__all_sync(kFull, ok)) {
      run.scores(sk + s * L::kStageBytes + warp * L::kSub, ke, key0, n, acc);
    } else {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][e] = -INFINITY;
    }
    float x0, x1;
    run.largest(acc, x0, x1);
    x0 = head_max(x0);
    x1 = head_max(x1);
    const float ls0 = head_sum(run.l0), ls1 = head_sum(run.l1);
    if (gq == 0) {
      xmax[i & 1][warp][2 * cq] = x0; xmax[i & 1][warp][2 * cq + 1] = x1;
      xl[i & 1][warp][2 * cq] = ls0; xl[i & 1][warp][2 * cq + 1] = ls1;
    }
    __syncthreads();                     // also: this round's K is read, and the V of the kept tile before the last
    if (tid == 0 && i + S < rounds) issue_k(i + S);
    k_issued = min(rounds, i + S + 1);
    float tm = xmax[i & 1][0][g], lt = xl[i & 1][0][g];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) { tm = max_nan(tm, xmax[i & 1][w][g]); lt += xl[i & 1][w][g]; }
    // Eq. (3) for head g; the group keeps a tile that one of its heads keeps.  A NaN score keeps its tile: the answer is NaN
    const bool keep = __any_sync(kFull, g < G && (lt == 0.f || !(tm - m_g - lg2(lt) < thr)));
    if (a.mask != nullptr && tid == 0) a.mask[(static_cast<size_t>(b) * a.Hkv + hk) * Tmax + j] = keep ? 1 : 0;
    if (!keep) continue;
    if (tid == 0)
      load_step<D, true>(&mv, sv + kept % S * L::kStageBytes, smem_u32(&full_v[kept % S]), hk, j * kTile, b, n, a);
    finish_pending(kept - 1);
    ++kept;
    if (tm > m_g + kSlack) m_g = tm;
    run.move(__shfl_sync(kFull, m_g, 2 * cq), __shfl_sync(kFull, m_g, 2 * cq + 1));
    run.weights(acc, ve, pend);
    waiting = true;
    pend_key = key0;
  }
  finish_pending(kept - 1);
  if (a.counts != nullptr && tid == 0) a.counts[(static_cast<size_t>(b) * a.Hkv + hk) * a.splits + sp] = kept;

  // loads that were issued and not waited for (a wait that expired) land before the CTA can finish
  if (tid == 0 && !ok) {
    for (int i = max(0, k_issued - S); i < k_issued; ++i) mbar_drain(smem_u32(&full_k[i % S]), (i / S) & 1, a.status);
    for (int i = max(0, kept - S); i < kept; ++i) mbar_drain(smem_u32(&full_v[i % S]), (i / S) & 1, a.status);
  }

  // join the warps (one reference m for all): l added up, u rescaled from z to m and added up
  const float l0 = head_sum(run.l0), l1 = head_sum(run.l1);
  if (gq == 0) {
    xm[warp][2 * cq] = run.m0; xm[warp][2 * cq + 1] = run.m1;
    xsum[warp][2 * cq] = l0; xsum[warp][2 * cq + 1] = l1;
  }
  __syncthreads();                       // every ring is idle too: its memory takes the warps' O
  run.join_o();
  const float f0 = run.z0 == -INFINITY ? 0.f : ex2(run.z0 - kLift - run.m0);
  const float f1 = run.z1 == -INFINITY ? 0.f : ex2(run.z1 - kLift - run.m1);
  constexpr int kPitch = D + 4;          // spreads the heads' rows over the banks
  float* su = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)));   // [warp][8 heads][D]
#pragma unroll
  for (int t = 0; t < D / 16; ++t) {
    const int d = (D / 8) * gq + 2 * t;  // the dimensions O^T's rows gq and gq + 8 of tile t stand for: d, d + 1
    float* h0 = su + (warp * 8 + 2 * cq) * kPitch + d;
    *reinterpret_cast<float2*>(h0) = make_float2(run.o[t][0] * f0, run.o[t][2] * f0);
    *reinterpret_cast<float2*>(h0 + kPitch) = make_float2(run.o[t][1] * f1, run.o[t][3] * f1);
  }
  __syncthreads();
  if (*abortp) return;
  const size_t all = static_cast<size_t>(a.records) * a.B * a.Hq * (D + 4);
  for (int i = tid; i < G * D; i += 32 * kWarps) {
    const int h = i / D, d = i % D;
    const size_t rec = ((static_cast<size_t>(sp) * a.B + b) * a.Hq + hk * G + h) * (D + 4);
    if (!dbg_idx(rec + 4 + d, all, a.status)) continue;
    float u = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) { u += su[(w * 8 + h) * kPitch + d]; l += xsum[w][h]; }
    a.partial[rec + 4 + d] = u;
    if (d == 0) *reinterpret_cast<float4*>(a.partial + rec) = make_float4(xm[0][h], l, l, 0.f);
  }
}

template <int D, bool kWide>
cudaError_t quant_go(const StreamArgs& a, cudaStream_t s) {
  using L = Layout<D, true>;
  CUtensorMap mk, mv;
  if (!stream_maps<D, true>(a, &mk, &mv)) return cudaErrorInvalidValue;
  auto kern = decode_quant_kernel<D, kWide>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(kern, L::kSmem, allowed);
  if (e != cudaSuccess) return e;
  return launch_early(kern, dim3(a.Hkv, a.splits, a.B), 32 * kWarps, L::kSmem, s, mk, mv, a);
}

}  // namespace

cudaError_t launch_decode_quant(const StreamArgs& args, cudaStream_t s, int* launches) {
  ++*launches;
  StreamArgs a = args;
  a.heads_cta = 1;
  if (a.q_dt == kBF16) return a.D == 64 ? quant_go<64, false>(a, s) : quant_go<128, false>(a, s);
  return a.D == 64 ? quant_go<64, true>(a, s) : quant_go<128, true>(a, s);
}

}  // namespace mala
