// Dense split-KV decode: over the 8-bit cache (tau = 0), and over the sequences'
// own bf16 rows behind a shared prefix (the prefix itself: prefix_tc.cu).
//
// o = softmax(scale q K^T) V by the (m, l, u) identity: a part's running
// maximum m, l = sum 2^(s - m) and u = sum 2^(s - m) v leave as one record per
// (part, query head), and a sequence's records are merged exactly ("Why exact
// attention does not need a quadratic matrix", Method/Mechanism).
//
// Bound: HBM.  A key and its value are read once for the G <= 8 query heads of
// their KV head: 4 D G flops over 4 D bytes of bf16 (G flops a byte) or 2 (D + 1)
// of the 8-bit cache (about 2 G).
//
// Every tile is kept, so the work can be cut anywhere.  The sequences' keys, in
// units of a sub-tile (32 keys of e4m3, 16 of bf16), are laid end to end and
// cut into Z <= W equal parts: worker z of a KV head takes units z W / Z up to
// (z + 1) W / Z of the W, however long or short the sequences in it are.  (A cut per
// sequence leaves the longest sequence's parts running alone: 3 sequences of 6.7K
// to 20K keys, 64 / 8 heads, took 26.6 us with it and take 23.1.)  Part of sequence b in worker z is
// record z + b, a number that no other pair has, since both grow along the line.
//
// A worker is a CTA of four warps that takes up to four neighbouring KV heads, a
// warp or more each: their rows lie side by side in memory, and one TMA box
// brings the same keys of all of them.  (With one head a CTA, the CTAs of a row
// drift apart and its DRAM pages are opened again for each: 5.7 TB/s with 8 KV
// heads where 1 KV head gave 7.0.)  8 sequences of 128K keys, 32 / 8 heads: 304 to
// 314 us by machine, 7.1 to 6.9 TB/s.  The warps share the stages of the ring but
// never wait for one another: the last to have read a stage loads it again.
#include <algorithm>

#include "shared_plan.h"
#include "stream_common.cuh"

namespace mala {
namespace {

using namespace stream;

// CTAs an SM.  Two streams of 64 KB in flight fill the memory with 128-byte rows;
// a third only scatters the DRAM's pages (128K x 8 sequences: 305 us with two, 341
// with three).  Rows of 64 bytes have twice the instructions a byte.
template <int D> constexpr int kCtas = stream_ctas(D);

// Keys of sequence b that count: its length, 0 if that is outside [min_len, N] (the merge reports it).
__device__ __forceinline__ int keys_of(const StreamArgs& a, int b) {
  if (a.lens == nullptr) return a.N;
  const int n = a.lens[b];
  return n < a.min_len || n > a.N ? 0 : n;
}

__device__ __forceinline__ uint32_t units_in(const StreamArgs& a, int n) {
  return (static_cast<uint32_t>(n) + a.unit - 1) / a.unit;
}
__device__ __forceinline__ uint32_t units_of(const StreamArgs& a, int b) { return units_in(a, keys_of(a, b)); }

// A place on the line of units: unit u of sequence b, which has `units` and n keys.
struct Place {
  int b, u, units, n;
  __device__ __forceinline__ void next(const StreamArgs& a) {
    if (++u < units) return;
    u = 0;
    do {
      ++b;
      n = b < a.B ? keys_of(a, b) : 0;
      units = (n + a.unit - 1) / a.unit;
    } while (units == 0 && b < a.B);
  }
};

// n / d, in 32 bits where both fit (several times faster).
__device__ __forceinline__ uint64_t quotient(uint64_t n, uint64_t d) {
  return ((n | d) >> 32) == 0 ? static_cast<uint32_t>(n) / static_cast<uint32_t>(d) : n / d;
}

// Counts an event in shared memory: what came before it is seen by whoever counts after it.
__device__ __forceinline__ int count_up(int* counter) {
  int before;
  asm volatile("atom.acq_rel.cta.shared::cta.add.s32 %0, [%1], 1;" : "=r"(before) : "r"(smem_u32(counter)) : "memory");
  return before;
}

// Worker z's first unit and how many it has (called by a whole warp).
__device__ __forceinline__ Place worker_span(const StreamArgs& a, int z, int& count) {
  const int lane = threadIdx.x % 32;
  uint64_t W = 0;
  int n0 = 0;                             // keys of sequence `lane`, of the first 32
  if (a.lens == nullptr) {
    W = static_cast<uint64_t>(units_of(a, 0)) * a.B;
  } else {
    for (int c = 0; c < a.B; c += 32) {
      const int n = c + lane < a.B ? keys_of(a, c + lane) : 0;
      if (c == 0) n0 = n;
      W += __reduce_add_sync(kFull, units_in(a, n));
    }
  }
  const uint64_t Z = min(static_cast<uint64_t>(a.workers), W);
  Place p{0, 0, 1, 0};
  count = 0;
  if (static_cast<uint64_t>(z) >= Z) return p;
  const uint64_t u0 = quotient(W * z, Z);
  count = static_cast<int>(quotient(W * (z + 1), Z) - u0);
  if (a.lens == nullptr) {
    p.units = units_of(a, 0);
    p.b = static_cast<int>(quotient(u0, p.units));
    p.u = static_cast<int>(u0) - p.b * p.units;
    p.n = a.N;
    return p;
  }
  uint64_t before = 0;
  for (int c = 0; c < a.B; c += 32) {
    const int n = c == 0 ? n0 : c + lane < a.B ? keys_of(a, c + lane) : 0;
    const uint32_t x = units_in(a, n);
    uint32_t sum = x;                     // inclusive over the 32 sequences
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(kFull, sum, off);
      if (lane >= off) sum += y;
    }
    const uint32_t past = __ballot_sync(kFull, before + sum > u0);
    if (past != 0) {
      const int i = __ffs(past) - 1;
      p.b = c + i;
      p.units = static_cast<int>(__shfl_sync(kFull, x, i));
      p.u = static_cast<int>(u0 - before) - static_cast<int>(__shfl_sync(kFull, sum - x, i));
      p.n = __shfl_sync(kFull, n, i);
      return p;
    }
    before += __shfl_sync(kFull, sum, 31);
  }
  return p;
}

template <int D, bool kQuant, bool kWide>
__global__ void __launch_bounds__(32 * kWarps, kCtas<D>)
decode_stream_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const StreamArgs a) {
  using L = Layout<D, kQuant>;
  using Run = Running<D, kQuant, kWide>;
  constexpr int S = L::kStages;
  static_assert(S >= 2, "exponents are loaded two units ahead, within the ring");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_k[S], full_v[S];
  __shared__ int read_k[S], read_v[S], abort_flag;      // warps that have read a stage, all uses counted
  __shared__ int loads_k[S], loads_v[S];                // loads issued into it
  __shared__ float jm[kWarps][8], jl[2][kWarps][8];
  __shared__ __align__(16) float ju[kWarps / 2][8][D + 4];

  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, gq = lane >> 2, cq = lane & 3;
  const int G = a.Hq / a.Hkv;
  // the CTA's heads, the warps of one head, and this warp's place
  const int HW = a.heads_cta, QW = kWarps / HW, part = warp % QW;
  const int groups = a.Hkv / HW, hk0 = static_cast<int>(blockIdx.x) % groups * HW, z = blockIdx.x / groups;
  const int hk = hk0 + warp / QW;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sk = base, sv = base + S * L::kStageBytes;
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&full_k[i]), 1);
      mbar_init(smem_u32(&full_v[i]), 1);
      read_k[i] = read_v[i] = loads_k[i] = loads_v[i] = 0;
    }
    abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&mk);
    prefetch_tensormap(&mv);
  }
  volatile int* abortp = &abort_flag;
  // What ran before on the stream is complete.  Behind a prefix it is already: the prefix pass lets this one start once
  // it has waited for that itself.  Only then may the merge start, which reads the lengths at once.
  if (!a.after_prefix) grid_wait();
  grid_launch_dependents();

  int count = 0;
  Place at = worker_span(a, z, count);

  if (kQuant && (a.counts != nullptr || a.mask != nullptr)) {
    // every tile is kept: the counts of the splits that mala_decode would make, and the mask
    const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + tid, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    const int Tmax = (a.N + 127) / 128;
    for (int64_t i = first; a.counts != nullptr && i < static_cast<int64_t>(a.B) * a.Hkv * a.splits; i += step) {
      const int T = (keys_of(a, static_cast<int>(i / a.splits / a.Hkv)) + 127) / 128, per = (T + a.splits - 1) / a.splits;
      const int t0 = min(T, static_cast<int>(i % a.splits) * per);
      a.counts[i] = min(T, t0 + per) - t0;
    }
    for (int64_t i = first; a.mask != nullptr && i < static_cast<int64_t>(a.B) * a.Hkv * Tmax; i += step)
      if (static_cast<int>(i % Tmax) < (keys_of(a, static_cast<int>(i / Tmax / a.Hkv)) + 127) / 128) a.mask[i] = 1;
  }

  if (count > 0) {
    Run run;
    const auto raw_q = run.q.fetch(a, at.b, hk);   // ahead of the ring's loads, or it queues behind them
    run.reset();
    __syncthreads();                     // the barriers are set up
    auto issue_k = [&](int i, const Place& p) {
      ++loads_k[i % S];                  // one stage's loads follow one another
      load_step<D, kQuant>(&mk, sk + i % S * L::kStageBytes, smem_u32(&full_k[i % S]), hk0, p.u * a.unit, p.b, p.n, a);
    };
    auto issue_v = [&](int i, const Place& p) {
      ++loads_v[i % S];
      load_step<D, kQuant>(&mv, sv + i % S * L::kStageBytes, smem_u32(&full_v[i % S]), hk0, p.u * a.unit, p.b, p.n, a);
    };
    // A stage is loaded again by whichever warp is the last to have read it: no warp waits for another.
    auto last_reader = [&](int* counter) {
      __syncwarp();
      return lane == 0 && (count_up(counter) & (kWarps - 1)) == kWarps - 1;
    };
    auto key_of = [&](const Place& p) { return p.u * a.unit + part * L::kKeys; };     // this warp's first key of a unit
    // Exponent bytes of a unit's keys, one key a lane.  Nothing but the loads may stand here: any arithmetic on them
    // would wait for them on the spot (as a packed pair they cost the 128K batch-8 decode 403 instead of 356 us).
    auto load_exps = [&](const Place& p, uint32_t& ke, uint32_t& ve) {
      ke = ve = 0;
      if constexpr (kQuant) {
        const int key = key_of(p) + lane;
        if (key < p.n) {
          const size_t e = (static_cast<size_t>(p.b) * a.Hkv + hk) * a.N + key;
          ke = a.k_exps[e];
          ve = a.v_exps[e];
        }
      }
    };
    Place ahead = at;                    // next unit to load
    uint32_t ke = 0, ve = 0, ke1 = 0, ve1 = 0;      // of this unit and the next
    load_exps(at, ke, ve);
    Place at_exps = at;
    for (int i = 0; i < min(count, S); ++i) {
      if (tid == 0) {
        issue_k(i, ahead);
        issue_v(i, ahead);
      }
      if (i + 1 < count) ahead.next(a);
      if (i == 0 && count > 1) {
        at_exps = ahead;
        load_exps(at_exps, ke1, ve1);
      }
    }
    run.q.set(a, raw_q);
    bool ok = true;

    // After a timed-out wait the loop runs on (waits then fail at once), so that the CTA's barriers stay matched and
    // every stage is still counted as read.
    for (int i = 0; i < count; ++i) {
      const int s = i % S, key0 = key_of(at);
      const bool more = i + S < count;
      ok = mbar_wait(smem_u32(&full_k[s]), (i / S) & 1, abortp, a.status) && ok;
      float acc[Run::kMT][4];
      run.scores(sk + s * L::kStageBytes + warp * L::kPiece, ke, key0, at.n, acc);
      if (last_reader(&read_k[s]) && more && !*abortp) issue_k(i + S, ahead);
      run.grow(acc);
      typename Run::Weights w;
      run.weights(acc, ve, w);
      ke = ke1;
      ve = ve1;
      if (i + 2 < count) {
        at_exps.next(a);
        load_exps(at_exps, ke1, ve1);
      }
      ok = mbar_wait(smem_u32(&full_v[s]), (i / S) & 1, abortp, a.status) && ok;
      run.values(sv + s * L::kStageBytes + warp * L::kPiece, key0, at.n, w);
      if (last_reader(&read_v[s]) && more && !*abortp) issue_v(i + S, ahead);
      if (i + S + 1 < count) ahead.next(a);
      // the sequence's last unit, or the worker's: its record
      const int b = at.b;
      if (i + 1 < count) at.next(a);
      if (i + 1 < count && at.b == b) continue;

      run.join_o();
      float l0 = head_sum(run.l0), l1 = head_sum(run.l1);
      float r0 = kQuant ? l0 : head_sum(run.r0), r1 = kQuant ? l1 : head_sum(run.r1);
      // one head's warps agree on a reference
      float t0 = run.m0, t1 = run.m1;
      if (QW > 1) {
        if (gq == 0) { jm[warp][2 * cq] = t0; jm[warp][2 * cq + 1] = t1; }
        __syncthreads();
        for (int w2 = warp - part; w2 < warp - part + QW; ++w2) {
          t0 = fmaxf(t0, jm[w2][2 * cq]);
          t1 = fmaxf(t1, jm[w2][2 * cq + 1]);
        }
      }
      const float tr0 = t0 == -INFINITY ? 0.f : t0, tr1 = t1 == -INFINITY ? 0.f : t1;
      const float e0 = ex2(run.m0 - tr0), e1 = ex2(run.m1 - tr1);
      l0 *= e0; l1 *= e1; r0 *= e0; r1 *= e1;
      const float f0 = !kQuant ? e0 : run.z0 == -INFINITY ? 0.f : ex2(run.z0 - kLift - tr0);
      const float f1 = !kQuant ? e1 : run.z1 == -INFINITY ? 0.f : ex2(run.z1 - kLift - tr1);
      float* rec0 = a.spread + (static_cast<size_t>(z + b) * a.Hq + hk * G) * (D + 4);
      const bool in = dbg_idx((static_cast<size_t>(z + b) * a.Hq + hk * G + G) * (D + 4) - 1,
                              static_cast<size_t>(a.workers + a.B) * a.Hq * (D + 4), a.status);
      if (QW == 1) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (2 * cq + e >= G || !in) continue;
          float* out = rec0 + (2 * cq + e) * (D + 4);
          const float f = e ? f1 : f0;
          if (gq == 0) *reinterpret_cast<float4*>(out) = make_float4(e ? t1 : t0, e ? l1 : l0, e ? r1 : r0, 0.f);
          if constexpr (kQuant) {
            // O^T's rows gq and gq + 8 of tile t stand for the dimensions (D / 8) gq + 2t and + 1
#pragma unroll
            for (int t = 0; t < D / 16; t += 2)
              *reinterpret_cast<float4*>(out + 4 + (D / 8) * gq + 2 * t) =
                  make_float4(run.o[t][e] * f, run.o[t][2 + e] * f, run.o[t + 1][e] * f, run.o[t + 1][2 + e] * f);
          } else {
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
              out[4 + 16 * t + gq] = run.o[t][e] * f;
              out[4 + 16 * t + gq + 8] = run.o[t][2 + e] * f;
            }
          }
        }
      } else {
        // the parts add into one copy, one after the other (in a fixed order)
        float (*u)[D + 4] = ju[warp / QW];
        if (gq == 0) {
          jl[0][warp][2 * cq] = l0; jl[0][warp][2 * cq + 1] = l1;
          jl[1][warp][2 * cq] = r0; jl[1][warp][2 * cq + 1] = r1;
        }
        for (int turn = 0; turn < QW; ++turn) {
          if (part == turn) {
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int d = kQuant ? (D / 8) * gq + 2 * t + (e >> 1) : 16 * t + gq + 8 * (e >> 1);
                float* x = &u[2 * cq + (e & 1)][d];
                *x = (turn == 0 ? 0.f : *x) + run.o[t][e] * ((e & 1) ? f1 : f0);
              }
          }
          __syncthreads();
        }
        for (int x = part * 32 + lane; x < G * D && in; x += QW * 32) rec0[x / D * (D + 4) + 4 + x % D] = u[x / D][x % D];
        if (part == 0 && lane < G && in) {
          float m = -INFINITY, l = 0.f, lr = 0.f;
          for (int w2 = warp; w2 < warp + QW; ++w2) { m = fmaxf(m, jm[w2][lane]); l += jl[0][w2][lane]; lr += jl[1][w2][lane]; }
          *reinterpret_cast<float4*>(rec0 + lane * (D + 4)) = make_float4(m, l, lr, 0.f);
        }
        __syncthreads();                 // the copies are free again
      }
      if (i + 1 < count) {
        run.q.set(a, run.q.fetch(a, at.b, hk));
        run.reset();
      }
    }
    // after an abort: loads that nothing waited for land before the CTA can finish
    __syncthreads();
    if (tid == 0 && *abortp)
      for (int i = 0; i < S; ++i) {
        if (loads_k[i] > 0) mbar_drain(smem_u32(&full_k[i]), (loads_k[i] - 1) & 1, a.status);
        if (loads_v[i] > 0) mbar_drain(smem_u32(&full_v[i]), (loads_v[i] - 1) & 1, a.status);
      }
  }
  // Behind a prefix: the last CTA waits for it, so that this grid's end, which is all that the merge waits for, means
  // the prefix's too.  The others leave, and make room for one another while the prefix still runs.
  if (a.after_prefix && blockIdx.x == gridDim.x - 1) grid_wait();
}

__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}

// Exact merge of all records of a (sequence, query head): a.records that every
// (sequence, head) has, then the workers' that hold part of the sequence.  A record
// with l = 0 holds no key and its u is not used.  l = NaN (NaN scores) makes the
// output NaN; so does a sequence without any key, or with a rejected length.
//
// Bound: latency.  kRow warps share a row; each merges its records as it goes,
// kBatch at a time, headers and u requested together, and the warps' (m, l, u) are
// merged last.  Up to 16 records a row take two warps (a step's 15 records a row:
// 25.1 us, with one 26.4, with eight 32.0), or one where the rows would not all
// fit at once otherwise (4096 rows: 135.8, with two 138.0); 52 take eight (23.8,
// with four 26.4).
template <typename Tout, int D, int kRow>
__global__ void __launch_bounds__(32 * (kRow < 4 ? 4 : kRow), kRow <= 2 ? 7 : kRow < 16 ? 2 : 1) stream_merge_kernel(const StreamArgs a) {
  grid_launch_dependents();
  constexpr int kCtaWarps = kRow < 4 ? 4 : kRow, kLanes = D / 4, kSide = 32 / kLanes, kBatch = kRow <= 2 ? 4 : 8;
  __shared__ float4 ums[kCtaWarps][32];
  __shared__ float hds[kCtaWarps][3];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, part = lane % kLanes;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kCtaWarps / kRow) + warp / kRow;
  const bool exists = row < static_cast<int64_t>(a.B) * a.Hq;
  const int b = exists ? static_cast<int>(row / a.Hq) : 0, h = exists ? static_cast<int>(row % a.Hq) : 0;
  bool bad = false;
  int spread = 0;                            // workers' records of this sequence, from id0 on
  size_t id0 = 0;
  if (a.lens != nullptr) {
    const int n = a.lens[b];
    bad = n < a.min_len || n > a.N;
    if (bad && exists && h == 0 && lane == 0) atomicOr(a.status, kStatusBadLength);
  }
  if (a.workers > 0) {
    uint64_t before = 0, W = 0;
    const uint32_t mine = units_of(a, b);
    if (a.lens == nullptr) {
      before = static_cast<uint64_t>(mine) * b;
      W = static_cast<uint64_t>(mine) * a.B;
    } else {
      for (int c = 0; c < a.B; c += 32) {
        const uint32_t x = c + lane < a.B ? units_of(a, c + lane) : 0;
        W += __reduce_add_sync(kFull, x);
        before += __reduce_add_sync(kFull, c + lane < b ? x : 0);
      }
    }
    if (mine > 0) {
      // unit u is worker floor(((u + 1) Z - 1) / W)'s
      const uint64_t Z = min(static_cast<uint64_t>(a.workers), W);
      const uint64_t z0 = quotient((before + 1) * Z - 1, W), z1 = quotient((before + mine) * Z - 1, W);
      spread = static_cast<int>(z1 - z0) + 1;
      id0 = static_cast<size_t>(z0) + b;
    }
  }
  grid_wait();
  const int records = a.records + spread;
  const float* first = a.partial + (static_cast<size_t>(b) * a.Hq + h) * (D + 4);
  const float* second = a.spread + (id0 * a.Hq + h) * (D + 4);
  const size_t step1 = static_cast<size_t>(a.B) * a.Hq * (D + 4), step2 = static_cast<size_t>(a.Hq) * (D + 4);
  float m = -INFINITY, l = 0.f, lr = 0.f;
  float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = (warp % kRow) * kSide + lane / kLanes; s0 < records; s0 += kBatch * kRow * kSide) {
    float4 hd[kBatch], x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = s0 + i * kRow * kSide;
      const float* p = s < a.records ? first + s * step1 : second + (s - a.records) * step2;
      hd[i] = s < records ? *reinterpret_cast<const float4*>(p) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      x[i] = s < records ? *reinterpret_cast<const float4*>(p + 4 + 4 * part) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (!(hd[i].y == 0.f)) top = fmaxf(top, hd[i].x);
    const float old = l == 0.f ? 0.f : exp2f(m - top);
    l *= old; lr *= old;
    u.x *= old; u.y *= old; u.z *= old; u.w *= old;
    m = top;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (hd[i].y == 0.f) continue;
      const float w = exp2f(hd[i].x - top);
      l += w * hd[i].y;
      lr += w * hd[i].z;
      u.x += w * x[i].x; u.y += w * x[i].y; u.z += w * x[i].z; u.w += w * x[i].w;
    }
  }
  auto join = [&](float m2, float l2, float lr2, float4 u2) {
    if (l2 == 0.f) return;
    const float top = fmaxf(m, m2), f = l == 0.f ? 0.f : exp2f(m - top), f2 = exp2f(m2 - top);
    l = l * f + l2 * f2;
    lr = lr * f + lr2 * f2;
    u.x = u.x * f + u2.x * f2; u.y = u.y * f + u2.y * f2; u.z = u.z * f + u2.z * f2; u.w = u.w * f + u2.w * f2;
    m = top;
  };
  if constexpr (kSide == 2) {
    const float m2 = __shfl_xor_sync(kFull, m, 16), l2 = __shfl_xor_sync(kFull, l, 16), lr2 = __shfl_xor_sync(kFull, lr, 16);
    const float4 u2 = make_float4(__shfl_xor_sync(kFull, u.x, 16), __shfl_xor_sync(kFull, u.y, 16),
                                  __shfl_xor_sync(kFull, u.z, 16), __shfl_xor_sync(kFull, u.w, 16));
    join(m2, l2, lr2, u2);                   // the lower half's lanes hold the row now
  }
  if constexpr (kRow > 1) {
    ums[warp][lane] = u;
    if (lane == 0) { hds[warp][0] = m; hds[warp][1] = l; hds[warp][2] = lr; }
    __syncthreads();
    if (warp % kRow != 0) return;
#pragma unroll
    for (int w = 1; w < kRow; ++w) join(hds[warp + w][0], hds[warp + w][1], hds[warp + w][2], ums[warp + w][lane]);
  }
  if (!exists) return;
  const bool any = !bad && !(l == 0.f);
  if (lane < kLanes) {
    const float inv = any ? 1.f / lr : NAN;
    store4(static_cast<Tout*>(a.o) + row * D + 4 * part, make_float4(u.x * inv, u.y * inv, u.z * inv, u.w * inv));
  }
  if (lane == 0) a.lse[row] = any ? (m + log2f(l)) * kLn2 : NAN;
}

template <int D, bool kQuant, bool kWide>
cudaError_t stream_go(const StreamArgs& a, cudaStream_t s) {
  using L = Layout<D, kQuant>;
  CUtensorMap mk, mv;
  if (!stream_maps<D, kQuant>(a, &mk, &mv)) return cudaErrorInvalidValue;
  auto kern = decode_stream_kernel<D, kQuant, kWide>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(kern, L::kSmem, allowed);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.workers) * (a.Hkv / a.heads_cta));
  return launch_early(kern, grid, 32 * kWarps, L::kSmem, s, mk, mv, a);
}

template <int D>
cudaError_t stream_pick(const StreamArgs& a, cudaStream_t s) {
  if (!a.k_exps) return stream_go<D, false, false>(a, s);
  return a.q_dt == kBF16 ? stream_go<D, true, false>(a, s) : stream_go<D, true, true>(a, s);
}

template <typename Tout, int D>
cudaError_t merge_pick(const StreamArgs& a, int64_t mean, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq;
  const auto grid = [&](int per) { return dim3(static_cast<unsigned>((rows + per - 1) / per)); };
  if (mean <= 16 && rows > 2 * 7 * sm_count()) return launch_early(stream_merge_kernel<Tout, D, 1>, grid(4), 128, 0, s, a);
  if (mean <= 16) return launch_early(stream_merge_kernel<Tout, D, 2>, grid(2), 128, 0, s, a);
  if (mean <= 48) return launch_early(stream_merge_kernel<Tout, D, 4>, grid(1), 128, 0, s, a);
  if (rows > sm_count()) return launch_early(stream_merge_kernel<Tout, D, 8>, grid(1), 256, 0, s, a);
  return launch_early(stream_merge_kernel<Tout, D, 16>, grid(1), 512, 0, s, a);
}

}  // namespace

void stream_divide(StreamArgs& a, int one_wave_on) {
  a.heads_cta = a.Hkv % 4 == 0 ? 4 : a.Hkv % 2 == 0 ? 2 : 1;
  a.unit = (a.k_exps ? Layout<64, true>::kKeys : Layout<64, false>::kKeys) * kWarps / a.heads_cta;
  // splits CTAs a sequence and KV head, and at most one a unit
  const int64_t groups = a.Hkv / a.heads_cta, units = static_cast<int64_t>(a.B) * ((a.N + a.unit - 1) / a.unit);
  int64_t z = std::min<int64_t>(static_cast<int64_t>(a.heads_cta) * a.splits * a.B, std::max<int64_t>(units, 1));
  // whole waves of CTAs, where there is more than one
  const int64_t wave = static_cast<int64_t>(one_wave_on > 0 ? one_wave_on : sm_count()) * stream_ctas(a.D);
  if (z * groups > wave) z = std::max<int64_t>(1, (one_wave_on > 0 ? wave : z * groups / wave * wave) / groups);
  a.workers = static_cast<int>(z);
}

cudaError_t launch_stream(const StreamArgs& a, cudaStream_t s, int* launches) {
  ++*launches;
  return a.D == 64 ? stream_pick<64>(a, s) : stream_pick<128>(a, s);
}

cudaError_t launch_stream_merge(const StreamArgs& a, cudaStream_t s, int* launches) {
  ++*launches;
  // records of an average row
  const int64_t mean = a.records + (a.workers + a.B - 1) / a.B + (a.workers > 0);
  if (a.out_dt == kBF16) return a.D == 64 ? merge_pick<__nv_bfloat16, 64>(a, mean, s) : merge_pick<__nv_bfloat16, 128>(a, mean, s);
  return a.D == 64 ? merge_pick<float, 64>(a, mean, s) : merge_pick<float, 128>(a, mean, s);
}

}  // namespace mala
