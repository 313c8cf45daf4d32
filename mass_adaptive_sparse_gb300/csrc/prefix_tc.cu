// Decode queries against a prefix that the whole batch shares, on the
// 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
// A prefix row's K and V are the same for every sequence, so the B G query rows
// of a KV head form one matrix: S = Q K^T, P = 2^(scale S - m), O += P V over the
// prefix's 128-key tiles, and (m, l, O) leave as the records of a split that
// the merge joins with each sequence's own part ("Why exact attention does
// not need a quadratic matrix", Method/Mechanism).  Every tile is kept.
//
// Bound: the prefix is read once for all rows, B G flops a byte: HBM up to
// about 200 rows a KV head, the tensor pipe beyond.  A 64K prefix, 8 KV heads: 47 us
// for 4 rows a KV head (5.7 TB/s), 54 for 128; 121 for 512 (1138 TFLOP/s), where a
// step of two tiles takes 1.97 us and its four single-CTA MMAs 1.87 of them.
//
// One CTA per (split, KV head, pair of query blocks).  A query block is 128
// rows: the G heads of 128 / G sequences, loaded by one TMA box.  The CTA runs two
// streams ("slots") that alternate on the tensor pipe, so that one's softmax
// covers the other's MMAs.  With a pair of query blocks the slots are the two
// blocks and share each K and V tile.  A last block without a partner gives
// both slots the same rows: they take the tiles in turn and join their (m, l, O)
// at the end, so that a batch of up to 128 rows a KV head, too, keeps the pipe
// and the loads going.
//   warps 0, 3  sequencers, one thread a slot: O += P V of a step, then the
//               next step's S, in turns passed by a token barrier
//   warp 1      V tiles by TMA, warp 2 Q and K tiles
//   warps 4-7   softmax of slot 0, warps 8-11 of slot 1: a thread owns a row
// TMEM: S of the slots in columns 0-127 and 128-255, O in 256.. and 384..; P (bf16)
// is written over the consumed S.  l sums P exactly (lse); the bf16-rounded P
// that enters P V is summed apart and normalises O.  The running maximum moves
// only past 2^8 growth.
#include <cuda_bf16.h>

#include "mala_internal.h"
#include "tc_common.cuh"

namespace mala {
namespace {

using namespace tc;

constexpr int kBlk = 128;               // query rows of a block, keys of a tile
constexpr int kThreads = 384;
constexpr uint32_t kColO = 256;
constexpr float kSlack = 8.0f;

template <int D>
struct Layout {
  static constexpr int kHalf = kBlk * 128;             // one 64-column TMA box
  static constexpr int kTile = kHalf * (D / 64);
  // a lone block has one Q tile and its place for one more K stage: each slot then owns every other stage of
  // both (even) rings, and so waits for every phase of the stages that it reads
  static constexpr int kNK = 3;
  static constexpr int kNV = D == 128 ? 2 : 4;
  static constexpr int kSmem = kTile * (2 + kNK + kNV) + 1024;
};

template <int NK, int NV>
struct Bars {
  uint64_t q_full;
  uint64_t k_full[NK + 1], k_empty[NK + 1];
  uint64_t v_full[NV], v_empty[NV];
  uint64_t s_full[2];     // Q K^T of the slot complete (so is its previous P V)
  uint64_t p_ready[2];    // P is in TMEM (one arrival per warp)
  uint64_t o_done[2];     // every MMA of the slot complete
  uint64_t tok[2];        // [slot]: the other slot's sequencer has taken its turn
  uint64_t fin[2];        // every MMA of a sequencer complete (its own wait before exit)
};

// Scores of columns past `last` become -inf.
__device__ __forceinline__ void mask_tail(uint32_t* sr, int last) {
#pragma unroll
  for (int c = 0; c < 64; ++c)
    if (c > last) sr[c] = 0xff800000u;
}

// 64 raw scores -> 32 bf16 pairs of P = 2^(S * scale - m) in sr[0..31]; `acc`
// sums P exactly, r0 / r1 the pairs' halves as rounded.
__device__ __forceinline__ void exponents(uint32_t* sr, uint64_t scale2, uint64_t neg_m2, uint64_t& acc, float& r0,
                                          float& r1) {
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    float e0, e1;
    f2_split(fma2(f2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), scale2, neg_m2), e0, e1);
    const float p0 = ex2(e0), p1 = ex2(e1);
    const uint32_t w = pack_bf16(p0, p1);
    acc = add2(acc, f2(p0, p1));
    add_bf16x2(r0, r1, w);
    sr[c] = w;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prefix_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv, const StreamArgs a) {
  using L = Layout<D>;
  constexpr int NV = L::kNV, kHalves = D / 64;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) Bars<L::kNK, NV> bars;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_flag;
  __shared__ float joint[3][kBlk];       // a lone block: slot 1's m, l and l of the rounded P

  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int G = a.Hq / a.Hkv, seqs = kBlk / G;             // sequences of a query block
  const int nblk = (a.B + seqs - 1) / seqs, npairs = (nblk + 1) / 2;
  // pairs of one (split, KV head) start side by side: they read the same tiles
  const int cta = static_cast<int>(blockIdx.x);
  const int pair = cta % npairs, hk = cta / npairs % a.Hkv, sp = cta / npairs / a.Hkv;
  const bool alone = 2 * pair + 1 >= nblk;                 // both slots on one block, tiles in turn
  const int NK = alone ? L::kNK + 1 : L::kNK;
  const uint32_t sQ = base, sK = base + (alone ? 1 : 2) * L::kTile, sV = base + (2 + L::kNK) * L::kTile;
  const int T = (a.N + kBlk - 1) / kBlk;
  const int t0 = static_cast<int>(static_cast<int64_t>(T) * sp / a.splits);
  const int ntiles = static_cast<int>(static_cast<int64_t>(T) * (sp + 1) / a.splits) - t0;
  // slot s takes steps u = 0 .. steps[s] - 1, on the CTA's tile (alone ? 2u + s : u)
  const int steps0 = alone ? (ntiles + 1) / 2 : ntiles, steps1 = alone ? ntiles / 2 : ntiles;
  const bool solo = steps1 == 0;

  // one 128-row tile of a prefix row matrix
  auto load_tile = [&](const CUtensorMap* m, uint32_t dst, uint32_t bar, int t) {
    const int row = (t0 + t) * kBlk;
    mbar_expect_tx(bar, L::kTile);
    if (!dbg_box(64 * (kHalves - 1), hk, row, 0, D, a.Hkv, 0, a.N, a.N, 1, a.status)) return;
#pragma unroll
    for (int i = 0; i < kHalves; ++i) tma_load_4d(dst + i * L::kHalf, m, bar, 64 * i, hk, row, 0);
  };

  // The loading threads set up their own barriers and fill their rings before the CTA meets: the first tiles are on
  // their way while TMEM is allocated.
  const int readers = alone ? 1 : 2;                       // slots that read a tile
  if (warp == 2 && lane == 0) {
    mbar_init(smem_u32(&bars.q_full), 1);
    for (int i = 0; i < NK; ++i) { mbar_init(smem_u32(&bars.k_full[i]), 1); mbar_init(smem_u32(&bars.k_empty[i]), readers); }
    fence_barrier_init();
    prefetch_tensormap(&mq);
    prefetch_tensormap(&mk);
    grid_wait();
    if (ntiles > 0) {
      const uint32_t qf = smem_u32(&bars.q_full);
      mbar_expect_tx(qf, (alone ? 1 : 2) * L::kTile);
      for (int s = 0; s < (alone ? 1 : 2); ++s) {
        const int seq = (2 * pair + s) * seqs;
        if (!dbg_ok(seq < a.B, a.status)) continue;
#pragma unroll
        for (int i = 0; i < kHalves; ++i) tma_load_4d(sQ + s * L::kTile + i * L::kHalf, &mq, qf, 64 * i, hk * G, seq, 0);
      }
    }
    for (int t = 0; t < min(NK, ntiles); ++t) load_tile(&mk, sK + t * L::kTile, smem_u32(&bars.k_full[t]), t);
  } else if (warp == 1 && lane == 0) {
    for (int i = 0; i < NV; ++i) { mbar_init(smem_u32(&bars.v_full[i]), 1); mbar_init(smem_u32(&bars.v_empty[i]), readers); }
    fence_barrier_init();
    prefetch_tensormap(&mv);
    grid_wait();
    for (int t = 0; t < min(NV, ntiles); ++t) load_tile(&mv, sV + t * L::kTile, smem_u32(&bars.v_full[t]), t);
  } else if (tid == 0) {
    abort_flag = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&bars.s_full[s]), 1);
      mbar_init(smem_u32(&bars.p_ready[s]), 4);
      mbar_init(smem_u32(&bars.o_done[s]), 1);
      mbar_init(smem_u32(&bars.tok[s]), 1);
      mbar_init(smem_u32(&bars.fin[s]), 1);
    }
    fence_barrier_init();
  }
  if (warp == 3) tmem_alloc<512>(smem_u32(&tmem_sh));
  // What ran before on the stream is complete; then the suffix pass may start, which needs nothing of this one.
  grid_wait();
  grid_launch_dependents();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = tmem_sh;
  volatile int* abortp = &abort_flag;

  if (warp == 2) {
    // ---------------- the K ring's further tiles ----------------
    if (lane == 0 && ntiles > 0) {
      int issued = min(NK, ntiles);
      for (int t = issued; t < ntiles; ++t, ++issued) {
        if (!mbar_wait(smem_u32(&bars.k_empty[t % NK]), (t / NK - 1) & 1, abortp, a.status)) break;
        load_tile(&mk, sK + (t % NK) * L::kTile, smem_u32(&bars.k_full[t % NK]), t);
      }
      // every issued load lands before the CTA can finish
      mbar_drain(smem_u32(&bars.q_full), 0, a.status);
      for (int t = max(0, issued - NK); t < issued; ++t) mbar_drain(smem_u32(&bars.k_full[t % NK]), (t / NK) & 1, a.status);
    }
  } else if (warp == 1) {
    // ---------------- the V ring's further tiles ----------------
    if (lane == 0 && ntiles > 0) {
      int issued = min(NV, ntiles);
      for (int t = issued; t < ntiles; ++t, ++issued) {
        if (!mbar_wait(smem_u32(&bars.v_empty[t % NV]), (t / NV - 1) & 1, abortp, a.status)) break;
        load_tile(&mv, sV + (t % NV) * L::kTile, smem_u32(&bars.v_full[t % NV]), t);
      }
      for (int t = max(0, issued - NV); t < issued; ++t) mbar_drain(smem_u32(&bars.v_full[t % NV]), (t / NV) & 1, a.status);
    }
  } else if (warp == 0 || warp == 3) {
    // ---------------- sequencers ----------------
    const int s = warp == 0 ? 0 : 1, steps = s == 0 ? steps0 : steps1;
    if (lane == 0 && steps > 0) {
      constexpr uint32_t idesc_qk = idesc_f16(1, 0, 0, kBlk, kBlk);
      constexpr uint32_t idesc_pv = idesc_f16(1, 0, 1, kBlk, D);
      const uint64_t dq = desc_kmajor_sw128(sQ + (alone ? 0 : s) * L::kTile);
      const uint32_t d_s = tmem + s * 128, d_o = tmem + kColO + s * 128;
      int turn = 0;
      // slot 0 takes the first turn; a turn waits for the other slot's last one (slot 1 never has more turns)
      auto take_turn = [&]() -> bool {
        const int k = s == 0 ? turn - 1 : turn;
        return solo || k < 0 || mbar_wait(smem_u32(&bars.tok[s]), k & 1, abortp, a.status);
      };
      auto pass_turn = [&]() {
        if (!solo) mbar_arrive(smem_u32(&bars.tok[1 - s]));
        ++turn;
      };
      auto tile = [&](int u) { return alone ? 2 * u + s : u; };
      auto wait_k = [&](int u) {
        const int t = tile(u);
        return mbar_wait(smem_u32(&bars.k_full[t % NK]), (t / NK) & 1, abortp, a.status);
      };
      auto issue_qk = [&](int u) {
        const uint64_t dk = desc_kmajor_sw128(sK + (tile(u) % NK) * L::kTile);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k / 4) * L::kHalf + (k % 4) * 32) >> 4;
          mma_ss(d_s, dq + off, dk + off, idesc_qk, k > 0);
        }
        mma_commit(smem_u32(&bars.s_full[s]));
      };
      bool ok = mbar_wait(smem_u32(&bars.q_full), 0, abortp, a.status) && wait_k(0) && take_turn();
      if (ok) {
        fence_after_sync();
        issue_qk(0);
        pass_turn();
        mma_commit(smem_u32(&bars.k_empty[tile(0) % NK]));
      }
      for (int u = 0; ok && u < steps; ++u) {
        const bool more = u + 1 < steps;
        const int vt = tile(u);
        // all that the turn needs, gathered before it is taken, in the order it becomes ready
        ok = !more || wait_k(u + 1);
        ok = ok && mbar_wait(smem_u32(&bars.v_full[vt % NV]), (vt / NV) & 1, abortp, a.status);
        ok = ok && mbar_wait(smem_u32(&bars.p_ready[s]), u & 1, abortp, a.status);
        ok = ok && take_turn();
        if (!ok) break;
        fence_after_sync();
        // P of keys 0-63 in columns 0-31 of S, keys 64-127 in 64-95
        const uint64_t dv = desc_mnmajor_sw128(sV + (vt % NV) * L::kTile, L::kHalf, 1024);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ts(d_o, d_s + (k / 4) * 64 + (k % 4) * 8, dv + ((k * 2048) >> 4), idesc_pv, (u > 0 || k > 0) ? 1u : 0u);
        if (more) issue_qk(u + 1);
        else mma_commit(smem_u32(&bars.o_done[s]));
        pass_turn();
        mma_commit(smem_u32(&bars.v_empty[vt % NV]));
        if (more) mma_commit(smem_u32(&bars.k_empty[tile(u + 1) % NK]));
      }
      // all MMAs of this thread complete before TMEM is released
      mma_commit(smem_u32(&bars.fin[s]));
      mbar_drain(smem_u32(&bars.fin[s]), 0, a.status);
    }
  } else {
    // ---------------- softmax: thread r of slot s owns query row r ----------------
    const int s = (warp >> 2) - 1, r = tid & 127, wr = warp & 3;
    const int steps = s == 0 ? steps0 : steps1;
    const int seq0 = (alone ? 2 * pair : 2 * pair + s) * seqs;
    const bool work = seq0 + (32 * wr) / G < a.B;          // some row of this warp exists
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(wr * 32) << 16);
    const uint32_t colS = s * 128, colO = kColO + s * 128;
    float m = -INFINITY, l = 0.f, lr = 0.f;
    bool ok = true;
    // After a timed-out wait the loop runs on (waits then fail at once): the lanes of a warp may see the end of a wait
    // differently, and the loads from tensor memory take all of them.
    for (int u = 0; u < steps; ++u) {
      ok = mbar_wait(smem_u32(&bars.s_full[s]), u & 1, abortp, a.status) && ok;
      fence_after_sync();
      if (work) {
        const int last = a.N - 1 - (t0 + (alone ? 2 * u + s : u)) * kBlk;      // last column with a key
        uint32_t sr[64];
        float mx[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = -INFINITY;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          tmem_ld64_sync(lane_addr + colS + 64 * hf, sr);
          if (last < kBlk - 1) mask_tail(sr, last - 64 * hf);
#pragma unroll
          for (int c = 0; c < 64; c += 2)
            mx[(c >> 1) & 7] = max3(mx[(c >> 1) & 7], __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
        }
        const float mt = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * a.scale_log2;
        float alpha = 1.f;
        if (mt > m + kSlack) {
          alpha = ex2(m - mt);
          m = mt;
        }
        const float mref = m == -INFINITY ? 0.f : m;
        const uint64_t scale2 = f2(a.scale_log2, a.scale_log2), neg_m2 = f2(-mref, -mref);
        uint64_t acc = f2(0.f, 0.f);
        float r0 = 0.f, r1 = 0.f;
        // P of keys 64-127 goes over the (consumed) scores of keys 64-95, P of keys 0-63 over keys 0-31
        exponents(sr, scale2, neg_m2, acc, r0, r1);
        tmem_st32(lane_addr + colS + 64, sr);
        tmem_ld64_sync(lane_addr + colS, sr);
        if (last < kBlk - 1) mask_tail(sr, last);
        exponents(sr, scale2, neg_m2, acc, r0, r1);
        float s0, s1;
        f2_split(acc, s0, s1);
        // O rescaled where the reference moved; the slot's previous P V is complete: it was issued
        // before the Q K^T whose completion s_full reported
        if (u > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32_sync(lane_addr + colO + c * 32, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(lane_addr + colO + c * 32, o);
          }
        }
        tmem_st32(lane_addr + colS, sr);
        tmem_st_wait();
        l = l * alpha + (s0 + s1);
        lr = lr * alpha + (r0 + r1);
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.p_ready[s]));
    }
    if (steps > 0) {
      ok = mbar_wait(smem_u32(&bars.o_done[s]), 0, abortp, a.status) && ok;
      fence_after_sync();
    }
    const bool fine = __all_sync(0xffffffffu, ok && !*abortp);
    // A lone block's slots join: slot 1 leaves its O in the K stages that only it read (its own are 1 and 3), four
    // columns of all rows after another, and slot 0 adds it to its own.
    const bool joins = alone && !solo;
    auto left = [&](int c4) {            // columns 4 c4 .. of this thread's row
      return reinterpret_cast<float4*>(smem_raw + (sK + (c4 < D / 8 ? 1 : 3) * L::kTile - smem_u32(smem_raw))) +
             (c4 % (D / 8)) * kBlk + r;
    };
    float f0 = 1.f, f1 = 0.f;
    if (joins) {
      if (s == 1 && work) {
        fence_proxy_async_smem();
        joint[0][r] = m; joint[1][r] = l; joint[2][r] = lr;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32_sync(lane_addr + colO + c * 32, reinterpret_cast<uint32_t*>(o));
#pragma unroll
          for (int e = 0; e < 8; ++e) *left(8 * c + e) = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      named_sync(1, 256);
      if (s == 0) {
        const float m1 = joint[0][r], top = fmaxf(m, m1), ref = top == -INFINITY ? 0.f : top;
        f0 = ex2(m - ref);
        f1 = ex2(m1 - ref);
        l = l * f0 + joint[1][r] * f1;
        lr = lr * f0 + joint[2][r] * f1;
        m = top;
      }
    }
    // records: (m, l, l of the rounded P, 0, O) of each row; a buffer that only this slot's products read (its
    // query block, or its first V stage) turns the row-wise read-out into whole row segments (rows 20 floats apart)
    if (fine && work && !(alone && s == 1)) {
      fence_proxy_async_smem();
      const size_t all = static_cast<size_t>(a.records) * a.B * a.Hq * (D + 4);
      auto record = [&](int row) {
        return ((static_cast<size_t>(sp) * a.B + seq0 + row / G) * a.Hq + hk * G + row % G) * (D + 4);
      };
      if (seq0 + r / G < a.B && dbg_idx(record(r) + 3, all, a.status))
        *reinterpret_cast<float4*>(a.partial + record(r)) = make_float4(m, l, lr, 0.f);
      if (steps > 0) {
        float* tp = reinterpret_cast<float*>(smem_raw + ((alone ? sV : sQ) + s * L::kTile - smem_u32(smem_raw))) +
                    wr * (32 * 20);
        float* out[4];                     // this lane's place in rows lane / 4 + 8k of the warp's, or null
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = 32 * wr + 8 * k + lane / 4;
          const size_t at = record(row) + 4 + 4 * (lane % 4);
          out[k] = seq0 + row / G < a.B && dbg_idx(at + D - 13, all, a.status) ? a.partial + at : nullptr;
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32_sync(lane_addr + colO + c * 32, reinterpret_cast<uint32_t*>(o));
          if (joins) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 x = *left(8 * c + e);
              o[4 * e] = o[4 * e] * f0 + x.x * f1;
              o[4 * e + 1] = o[4 * e + 1] * f0 + x.y * f1;
              o[4 * e + 2] = o[4 * e + 2] * f0 + x.z * f1;
              o[4 * e + 3] = o[4 * e + 3] * f0 + x.w * f1;
            }
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<float4*>(tp + lane * 20 + 4 * e) =
                  make_float4(o[16 * hf + 4 * e], o[16 * hf + 4 * e + 1], o[16 * hf + 4 * e + 2], o[16 * hf + 4 * e + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 x = *reinterpret_cast<const float4*>(tp + (8 * k + lane / 4) * 20 + 4 * (lane % 4));
              if (out[k]) *reinterpret_cast<float4*>(out[k] + 32 * c + 16 * hf) = x;
            }
            __syncwarp();
          }
        }
      }
    }
    fence_before_sync();
  }

  __syncthreads();
  if (warp == 3) {
    fence_after_sync();
    tmem_dealloc<512>(tmem);
  }
}

template <int D>
cudaError_t prefix_go(const StreamArgs& a, cudaStream_t s) {
  using L = Layout<D>;
  const int G = a.Hq / a.Hkv, seqs = kBlk / G, pairs = (prefix_blocks(a.B, a.Hq, a.Hkv) + 1) / 2;
  CUtensorMap mq, mk, mv;
  if (!encode_query_map(&mq, a.q, a.B, a.Hq, D, G, seqs) || !encode_bshd_map(&mk, a.k, 1, a.N, a.Hkv, D, kBlk) ||
      !encode_bshd_map(&mv, a.v, 1, a.N, a.Hkv, D, kBlk))
    return cudaErrorInvalidValue;
  auto kern = prefix_tc_kernel<D>;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(kern, L::kSmem, allowed);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(pairs) * a.Hkv * a.splits);
  // Short CTAs gain by starting early (one tile each: a step of 9.3 us takes 7.5), long ones lose (57 tiles: 136.3 us
  // become 140.5).
  if ((a.N + kBlk - 1) / kBlk <= 16 * a.splits) return launch_early(kern, grid, kThreads, L::kSmem, s, mq, mk, mv, a);
  kern<<<grid, kThreads, L::kSmem, s>>>(mq, mk, mv, a);
  return cudaGetLastError();
}

}  // namespace

int prefix_blocks(int B, int Hq, int Hkv) {
  const int seqs = kBlk / (Hq / Hkv);
  return (B + seqs - 1) / seqs;
}

cudaError_t launch_prefix_tc(const StreamArgs& a, cudaStream_t s, int* launches) {
  ++*launches;
  return a.D == 64 ? prefix_go<64>(a, s) : prefix_go<128>(a, s);
}

}  // namespace mala
