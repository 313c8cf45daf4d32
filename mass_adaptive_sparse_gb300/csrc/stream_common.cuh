// Warp-level pieces of the decode streams (decode_stream.cu: dense passes,
// decode_quant.cu: the skip rule): one warp, one KV head's G <= 8 queries, a
// sub-tile of keys in shared memory.
//
// Keys are the M side of both products' mma.sync m16n8k16, the heads the N
// side:
//   S^T = K q^T.  e4m3: a lane's A fragment is 16 consecutive codes of a key
//     row.  The sum over d does not care for order, so fragment slots take d in
//     the order in which one 16-byte load brings them, and q is laid out to
//     match.  bf16: ldmatrix.
//   O^T += V^T P^T.  A is V transposed.  e4m3: a lane loads 16 consecutive d of the
//     four keys of its fragment and pairs keys with byte permutes; d is
//     permuted in O^T's rows and put right when O leaves.  bf16: ldmatrix.trans.
//     P^T comes from S^T's accumulator by movmatrix.
// e4m3 codes widen exactly to fp16.  q enters as fp16 after a power-of-two
// scaling of each head's row (exact but for elements 2^-24 below the row's
// largest); fp32 queries enter as a sum of two fp16 numbers (22 bits, for
// elements down to 2^-12 of the row's largest; 2^-34 of that below).
// The key's scale multiplies its score.  The value's scale goes into the
// exponent: w = 2^(s + e_v - z) with a running reference z of its own, one a
// head.  The largest w so far is at least 2^kLift, near fp16's top, so that w has
// fp16's 11 bits down to 2^-28 of it, and is off by at most 2^-39 of it below
// that.  fp32 queries take w as hi + lo / kLoScale, two fp16 numbers whose
// products gather in accumulators of their own (as a plain lo, the rest of w
// would go under fp16's smallest step, 2^-24, while hi still has all its bits):
// 22 bits down to 2^-28 of the largest w, 2^-50 of it below.  So what is left out is
// small beside a head's largest p 2^e_v: in a channel where the rows of that size hold
// zeros, rows more than 2^28 times smaller keep fewer bits than these.
// l sums the unrounded p in fp32, and normalises o; bf16 weights, of 8 bits,
// are summed as rounded for that too.
// p's reference moves only when it would grow by more than 2^8, z by more than 2.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mala_internal.h"
#include "tc_common.cuh"

namespace mala {
namespace stream {

using namespace tc;

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;               // warps of a CTA
constexpr float kSlack = 8.0f;          // p's reference moves past 2^8 growth
constexpr float kSlackW = 1.0f;         // w's past 2
constexpr float kLift = 14.0f;          // w <= 2^(kSlackW + kLift) < fp16's largest
constexpr float kLoScale = 2048.0f;     // what hi leaves of w, at most 2^-11 of it, times this fits where w does

template <int D, bool kQuant>
struct Layout {
  static constexpr int kKeys = kQuant ? 32 : 16;              // keys of a sub-tile
  static constexpr int kSub = kKeys * (kQuant ? D : 2 * D);   // bytes of a sub-tile's K (or V)
  static constexpr int kHalves = !kQuant && D == 128 ? 2 : 1; // 64-column boxes of a row
  static constexpr int kPiece = kSub / kHalves;               // bytes of a sub-tile that lie together
  static constexpr int kRowBytes = kPiece / kKeys;
  static constexpr int kStageBytes = kWarps * kSub;           // the CTA's K (or V) of one step: [half][warp][key]
  static constexpr int kHalfStep = kWarps * kPiece;           // from a sub-tile's first half to its second
  static constexpr int kStages = D == 64 ? 3 : 2;             // 12 or 16 KB of K and V in flight a warp
  static constexpr int kSmem = kStages * 2 * kStageBytes + 1024;
};

// Two e4m3 codes -> two fp16 numbers, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t r;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo; }" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t two) {
  uint32_t r;
  asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi; }" : "=r"(r) : "r"(two));
  return r;
}

template <bool kF16>
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void lds4(uint32_t addr, uint32_t* r) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void lds2(uint32_t addr, uint32_t* r) {
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void sts4_zero(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" :: "r"(addr), "r"(0) : "memory");
}

__device__ __forceinline__ float max_nan(float x, float y) { // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float head_max(float x) {         // over the eight lanes that share a head; NaN if one is
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) x = max_nan(x, __shfl_xor_sync(kFull, x, off));
  return x;
}
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) x += __shfl_xor_sync(kFull, x, off);
  return x;
}

// The queries of one KV head's group as B fragments, and the factors that turn
// a raw product with this lane's heads 2cq, 2cq + 1 into log2 units.
template <int D, bool kQuant, bool kWide>
struct Queries {
  static constexpr int kSteps = D / 16;
  uint32_t hi[kSteps][2];
  uint32_t lo[kWide ? kSteps : 1][2];
  float f0, f1;

  // A lane's share of its head's row as it lies in memory: requested early, turned into operands later.
  static constexpr int kRaw = kWide ? D / 4 : D / 8;
  struct Raw { uint32_t w[kRaw]; };

  __device__ __forceinline__ static Raw fetch(const StreamArgs& a, int b, int hk) {
    const int lane = threadIdx.x % 32, gq = lane >> 2, cq = lane & 3, G = a.Hq / a.Hkv;
    const size_t row = (static_cast<size_t>(b) * a.Hq + hk * G + (gq < G ? gq : 0)) * D;
    Raw r;
    if constexpr (!kQuant) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) + row);
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        r.w[2 * k] = q[(16 * k + 2 * cq) / 2];
        r.w[2 * k + 1] = q[(16 * k + 8 + 2 * cq) / 2];
      }
    } else {
      // d = (D / 4) cq + i: the 16-byte pieces that a lane's key loads bring
      const char* q = static_cast<const char*>(a.q) + (row + (D / 4) * cq) * (kWide ? 4 : 2);
#pragma unroll
      for (int i = 0; i < kRaw / 4; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(q)[i];
        r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
      }
    }
    return r;
  }

  __device__ __forceinline__ void set(const StreamArgs& a, const Raw& r) {
    const int lane = threadIdx.x % 32, gq = lane >> 2, cq = lane & 3, G = a.Hq / a.Hkv;
    if constexpr (!kQuant) {
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        hi[k][0] = gq < G ? r.w[2 * k] : 0u;
        hi[k][1] = gq < G ? r.w[2 * k + 1] : 0u;
      }
      f0 = f1 = a.scale_log2;
    } else {
      float x[D / 4];
#pragma unroll
      for (int i = 0; i < kRaw; ++i) {
        if constexpr (kWide) {
          x[i] = __uint_as_float(r.w[i]);
        } else {
          x[2 * i] = __uint_as_float(r.w[i] << 16);
          x[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
        }
      }
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) {
        if (gq >= G) x[i] = 0.f;
        most = max(most, __float_as_uint(x[i]) & 0x7fffffffu);
      }
      most = max(most, __shfl_xor_sync(kFull, most, 1));
      most = max(most, __shfl_xor_sync(kFull, most, 2));
      // the row's largest element goes to [2^9, 2^10)
      const uint32_t ex = min(max(most >> 23, 10u), 254u);
      const float up = __uint_as_float((263u - ex) << 23);
      const float f = __uint_as_float((ex - 9u) << 23) * a.scale_log2;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float y0 = x[4 * k + 2 * e] * up, y1 = x[4 * k + 2 * e + 1] * up;
          hi[k][e] = pack_f16(y0, y1);
          if constexpr (kWide) {
            const __half2 h = *reinterpret_cast<const __half2*>(&hi[k][e]);
            lo[k][e] = pack_f16(y0 - __low2float(h), y1 - __high2float(h));
          }
        }
      }
      f0 = __shfl_sync(kFull, f, 8 * cq);
      f1 = __shfl_sync(kFull, f, 8 * cq + 4);
    }
  }
};

// A warp's running softmax over the sub-tiles it is given.
template <int D, bool kQuant, bool kWide>
struct Running {
  using L = Layout<D, kQuant>;
  static constexpr int kMT = L::kKeys / 16, kOT = D / 16;
  struct Weights {                        // of a sub-tile, as B fragments
    uint32_t hi[kMT][2], lo[kWide ? kMT : 1][2];
  };

  Queries<D, kQuant, kWide> q;
  float o[kOT][4];
  float olo[kWide ? kOT : 1][4];          // the lo weights' products, kLoScale times too large
  // of this lane's heads 2cq, 2cq + 1: reference and sum of p, reference of w, and (bf16) sum of the rounded p
  float m0, m1, l0, l1, z0, z1, r0, r1;

  __device__ __forceinline__ void reset() {
    m0 = m1 = z0 = z1 = -INFINITY;
    l0 = l1 = r0 = r1 = 0.f;
#pragma unroll
    for (int t = 0; t < kOT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[t][e] = 0.f;
        if constexpr (kWide) olo[t][e] = 0.f;
      }
  }
  __device__ __forceinline__ void scale_o(float f0, float f1) {
#pragma unroll
    for (int t = 0; t < kOT; ++t) {
      o[t][0] *= f0; o[t][1] *= f1; o[t][2] *= f0; o[t][3] *= f1;
      if constexpr (kWide) { olo[t][0] *= f0; olo[t][1] *= f1; olo[t][2] *= f0; olo[t][3] *= f1; }
    }
  }
  // o whole: before a record is made of it.
  __device__ __forceinline__ void join_o() {
    if constexpr (kWide) {
#pragma unroll
      for (int t = 0; t < kOT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] += olo[t][e] * (1.f / kLoScale);
    }
  }

  // Scores of a sub-tile in log2 units, -inf from key n on: acc[mt] = keys 16mt + {gq, gq + 8} x heads {2cq, 2cq + 1}.
  // `ke`: lane i's exponent byte is key i's.
  __device__ __forceinline__ void scores(uint32_t kb, uint32_t ke, int key0, int n, float (&acc)[kMT][4]) const {
    const int lane = threadIdx.x % 32, gq = lane >> 2, cq = lane & 3;
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[mt][e] = 0.f;
      if constexpr (kQuant) {
        uint32_t ra[D / 16], rb[D / 16];                 // rows gq and gq + 8: D / 64 pieces of 16 codes
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const int chunk = D == 128 ? ((2 * cq + i) ^ gq) : (cq ^ (gq >> 1));
          const uint32_t at = kb + (16 * mt + gq) * D + (chunk << 4);
          lds4(at, ra + 4 * i);
          lds4(at + 8 * D, rb + 4 * i);
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t a0 = e4m3x2_f16x2(ra[k]), a2 = e4m3x2_f16x2_hi(ra[k]);
          const uint32_t a1 = e4m3x2_f16x2(rb[k]), a3 = e4m3x2_f16x2_hi(rb[k]);
          mma16816<true>(acc[mt], a0, a1, a2, a3, q.hi[k][0], q.hi[k][1]);
          if constexpr (kWide) mma16816<true>(acc[mt], a0, a1, a2, a3, q.lo[k][0], q.lo[k][1]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int key = (lane & 7) + 8 * ((lane >> 3) & 1), dc = 2 * k + (lane >> 4);
          uint32_t r[4];
          ldsm4(kb + (dc >> 3) * L::kHalfStep + key * 128 + (((dc & 7) ^ (key & 7)) << 4), r);
          mma16816<false>(acc[mt], r[0], r[1], r[2], r[3], q.hi[k][0], q.hi[k][1]);
        }
      }
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const int r = 16 * mt + gq + 8 * hr;
        float ks = 1.f;
        if constexpr (kQuant) ks = __uint_as_float(__shfl_sync(kFull, ke, r) << 23);
        const bool valid = key0 + r < n;
        acc[mt][2 * hr] = valid ? acc[mt][2 * hr] * (ks * q.f0) : -INFINITY;
        acc[mt][2 * hr + 1] = valid ? acc[mt][2 * hr + 1] * (ks * q.f1) : -INFINITY;
      }
    }
  }

  // This lane's share of the sub-tile's largest scores; NaN where one is.
  __device__ __forceinline__ static void largest(const float (&acc)[kMT][4], float& x0, float& x1) {
    x0 = x1 = -INFINITY;
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      x0 = max_nan(x0, max_nan(acc[mt][0], acc[mt][2]));
      x1 = max_nan(x1, max_nan(acc[mt][1], acc[mt][3]));
    }
  }

  // Move p's reference where the scores outgrew it (a NaN does not; it reaches l by its p).
  __device__ __forceinline__ void grow(const float (&acc)[kMT][4]) {
    float x0, x1;
    largest(acc, x0, x1);
    if (!__any_sync(kFull, x0 > m0 + kSlack || x1 > m1 + kSlack)) return;
    x0 = head_max(x0);
    x1 = head_max(x1);
    move(x0 > m0 + kSlack ? x0 : m0, x1 > m1 + kSlack ? x1 : m1);
  }
  __device__ __forceinline__ void move(float n0, float n1) {
    const float f0 = n0 == m0 ? 1.f : ex2(m0 - n0), f1 = n1 == m1 ? 1.f : ex2(m1 - n1);
    l0 *= f0; l1 *= f1; r0 *= f0; r1 *= f1;
    if constexpr (!kQuant) scale_o(f0, f1);
    m0 = n0;
    m1 = n1;
  }

  // p summed into l, and the weights.  `vexp`: lane i's exponent byte is key i's.
  __device__ __forceinline__ void weights(const float (&acc)[kMT][4], uint32_t vexp, Weights& w) {
    const int gq = threadIdx.x % 32 >> 2;
    const float mr0 = m0 == -INFINITY ? 0.f : m0, mr1 = m1 == -INFINITY ? 0.f : m1;
    float ve[kMT][2];
    if constexpr (kQuant) {
      float zx0 = -INFINITY, zx1 = -INFINITY;
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          ve[mt][hr] = static_cast<float>(static_cast<int>(__shfl_sync(kFull, vexp, 16 * mt + gq + 8 * hr))) - 127.f;
          zx0 = fmaxf(zx0, acc[mt][2 * hr] + ve[mt][hr]);
          zx1 = fmaxf(zx1, acc[mt][2 * hr + 1] + ve[mt][hr]);
        }
      if (__any_sync(kFull, zx0 > z0 + kSlackW || zx1 > z1 + kSlackW)) {
        zx0 = head_max(zx0);
        zx1 = head_max(zx1);
        const float n0 = zx0 > z0 + kSlackW ? zx0 : z0, n1 = zx1 > z1 + kSlackW ? zx1 : z1;
        scale_o(n0 == z0 ? 1.f : ex2(z0 - n0), n1 == z1 ? 1.f : ex2(z1 - n1));
        z0 = n0;
        z1 = n1;
      }
    }
    const float zr0 = (z0 == -INFINITY ? 0.f : z0) - kLift, zr1 = (z1 == -INFINITY ? 0.f : z1) - kLift;
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const float s0 = acc[mt][2 * hr], s1 = acc[mt][2 * hr + 1];
        const float p0 = ex2(s0 - mr0), p1 = ex2(s1 - mr1);
        l0 += p0;
        l1 += p1;
        if constexpr (kQuant) {
          const float w0 = ex2((s0 + ve[mt][hr]) - zr0), w1 = ex2((s1 + ve[mt][hr]) - zr1);
          const uint32_t h = pack_f16(w0, w1);
          w.hi[mt][hr] = movmatrix(h);
          if constexpr (kWide) {
            const __half2 hh = *reinterpret_cast<const __half2*>(&h);
            w.lo[mt][hr] = movmatrix(pack_f16((w0 - __low2float(hh)) * kLoScale, (w1 - __high2float(hh)) * kLoScale));
          }
        } else {
          const uint32_t h = pack_bf16(p0, p1);
          r0 += __uint_as_float(h << 16);
          r1 += __uint_as_float(h & 0xffff0000u);
          w.hi[mt][hr] = movmatrix(h);
        }
      }
  }

  // O^T += V^T P^T
  __device__ __forceinline__ void values(uint32_t vb, int key0, int n, const Weights& w) {
    const int lane = threadIdx.x % 32, gq = lane >> 2, cq = lane & 3;
    if (key0 + L::kKeys > n) {
      // rows behind the last key hold anything, and 0 * NaN is not 0
      for (int i = lane; i < L::kSub / 16; i += 32) {
        const int half = i * 16 / L::kPiece, at = i * 16 % L::kPiece;
        if (key0 + at / L::kRowBytes >= n) sts4_zero(vb + half * L::kHalfStep + at);
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
      if constexpr (kQuant) {
        // this lane's keys 2cq, 2cq + 1, 2cq + 8, 2cq + 9 of the 16, d = (D / 8) gq ..
        uint32_t v[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * cq + (i & 1) + 8 * (i >> 1);
          const uint32_t row = vb + (16 * mt + r) * D;
          if constexpr (D == 128) lds4(row + ((gq ^ (r & 7)) << 4), v[i]);
          else lds2(row + (((gq >> 1) ^ ((r >> 1) & 3)) << 4) + (gq & 1) * 8, v[i]);
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t x = __byte_perm(v[0][i], v[1][i], 0x5140), y = __byte_perm(v[0][i], v[1][i], 0x7362);
          const uint32_t x2 = __byte_perm(v[2][i], v[3][i], 0x5140), y2 = __byte_perm(v[2][i], v[3][i], 0x7362);
          uint32_t a0 = e4m3x2_f16x2(x), a1 = e4m3x2_f16x2_hi(x), a2 = e4m3x2_f16x2(x2), a3 = e4m3x2_f16x2_hi(x2);
          mma16816<true>(o[2 * i], a0, a1, a2, a3, w.hi[mt][0], w.hi[mt][1]);
          if constexpr (kWide) mma16816<true>(olo[2 * i], a0, a1, a2, a3, w.lo[mt][0], w.lo[mt][1]);
          a0 = e4m3x2_f16x2(y); a1 = e4m3x2_f16x2_hi(y); a2 = e4m3x2_f16x2(y2); a3 = e4m3x2_f16x2_hi(y2);
          mma16816<true>(o[2 * i + 1], a0, a1, a2, a3, w.hi[mt][0], w.hi[mt][1]);
          if constexpr (kWide) mma16816<true>(olo[2 * i + 1], a0, a1, a2, a3, w.lo[mt][0], w.lo[mt][1]);
        }
      } else {
#pragma unroll
        for (int t = 0; t < kOT; ++t) {
          const int key = (lane & 7) + 8 * (lane >> 4), dc = 2 * t + ((lane >> 3) & 1);
          uint32_t r[4];
          ldsm4_t(vb + (dc >> 3) * L::kHalfStep + key * 128 + (((dc & 7) ^ (key & 7)) << 4), r);
          mma16816<false>(o[t], r[0], r[1], r[2], r[3], w.hi[mt][0], w.hi[mt][1]);
        }
      }
    }
  }
};

// A step's K (or V) for the CTA's warps by TMA: rows row .. of `heads` neighbouring KV heads of sequence b, one box
// (of 64 columns each) that fills [head][key].
template <int D, bool kQuant>
__device__ __forceinline__ void load_step(const CUtensorMap* m, uint32_t dst, uint32_t bar, int hk, int row, int b,
                                          int n, const StreamArgs& a) {
  using L = Layout<D, kQuant>;
  mbar_expect_tx(bar, L::kStageBytes);
  if (!dbg_box(0, hk + a.heads_cta - 1, row, b, D, a.Hkv, 0, n, a.N, a.B, a.status)) return;
#pragma unroll
  for (int i = 0; i < L::kHalves; ++i) tma_load_4d(dst + i * L::kHalfStep, m, bar, 64 * i, row, hk, b);
}

// Tensor maps of a pass's K and V for steps of `heads_cta` heads, kWarps sub-tiles in all.  A pass without rows (N = 0)
// loads nothing: any address will do for its maps.
template <int D, bool kQuant>
bool stream_maps(const StreamArgs& a, CUtensorMap* mk, CUtensorMap* mv) {
  using L = Layout<D, kQuant>;
  const int N = a.N > 0 ? a.N : 1, keys = L::kKeys * kWarps / a.heads_cta;
  return encode_cache_map(mk, a.N > 0 ? a.k : a.q, a.B, N, a.Hkv, D, keys, a.heads_cta, kQuant) &&
         encode_cache_map(mv, a.N > 0 ? a.v : a.q, a.B, N, a.Hkv, D, keys, a.heads_cta, kQuant);
}

}  // namespace stream
}  // namespace mala
