// How many CTAs of the decode kernels an SM holds, and how a shared decode divides the SMs between its prefix pass and its
// suffix pass (host code; the library and the Python binding use the same).
//
// The prefix pass holds an SM a CTA; the suffix pass starts on the SMs it leaves
// and goes on where its CTAs end.  The times below, in us, were fitted to device
// times of batches of 4 to 128 over prefixes of 2K to 64K rows (D = 128, 32 / 8
// heads and fewer; for D = 64 they are too long by the same factor on both sides).
// They only choose how work is cut: the answer is exact for any cut.  Against
// splits in proportion to the rows: 20 x 2048 12.4 -> 10.2 us, 64 x (32K + 64)
// 66 -> 56.5, 8 x (16K + 64) with two KV heads, D = 64, 13.0 -> 9.8; over
// nine batches measured with up to seven splits each, the chosen one took at most
// 9% more than the best.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace mala {

// CTAs an SM of the dense stream (decode_stream.cu) and of the skip-rule kernel (decode_quant.cu): their launch bounds,
// and what default numbers of splits fill.  The reasons stand at the kernels.
constexpr int stream_ctas(int D) { return D == 64 ? 4 : 2; }
constexpr int skip_ctas(int D, bool fp32_queries) { return D == 64 ? 4 : fp32_queries ? 2 : 3; }

struct SharedPlan {
  int64_t sms, batch, prefix_len, heads_kv, groups, heads_cta, rows_kv, pairs, tiles;
  double suffix_rows;                 // of a sequence, on average

  // lens: the lengths are on the device: half of max_suffix_len on average is assumed
  SharedPlan(int sm, int B, int P, int max_suffix, bool lens, int Hq, int Hkv)
      : sms(sm), batch(B), prefix_len(P), heads_kv(Hkv) {
    heads_cta = Hkv % 4 == 0 ? 4 : Hkv % 2 == 0 ? 2 : 1;
    groups = Hkv / heads_cta;
    const int64_t G = Hq / Hkv, blocks = (B + 128 / G - 1) / (128 / G);
    rows_kv = B * G;
    pairs = (blocks + 1) / 2;
    tiles = (static_cast<int64_t>(P) + 127) / 128;
    suffix_rows = lens ? 0.5 * max_suffix : max_suffix;
  }
  int64_t prefix_ctas(int64_t splits) const { return pairs * heads_kv * splits; }
  // A CTA's first scores and its records take 6; a step of its two slots 2.3 (one tile each of a lone block) or 1.97 (one
  // tile of a pair of blocks).
  double prefix_us(int64_t splits) const {
    const int64_t t = (tiles + splits - 1) / splits;
    return 6.0 + (rows_kv <= 128 ? 2.3 * static_cast<double>((t + 1) / 2) : 1.97 * static_cast<double>(t));
  }
  // Two CTAs an SM, each 2.5 a sequence and 1 a unit of 64 key rows; 5 to start.
  double suffix_us(int64_t on) const {
    if (suffix_rows <= 0) return 0.0;
    return 5.0 + batch * groups * (2.5 + suffix_rows * heads_cta / 64.0) / (2.0 * on);
  }
  // SMs that the prefix pass leaves, if the suffix pass is done on them by its end; else 0.
  int64_t beside(int64_t splits) const {
    const int64_t left = sms - prefix_ctas(splits);
    return left > 0 && suffix_us(left) <= prefix_us(splits) + 2.0 ? left : 0;
  }
  // Splits of the least time; each CTA more adds to the first loads' burst and, by its rows, to the merge.
  int64_t best_splits() const {
    int64_t best = 1;
    double least = INFINITY;
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>({256, tiles, sms / prefix_ctas(1)}));
    for (int64_t s = 1; s <= most; ++s) {
      const double us = prefix_us(s) + (rows_kv <= 128 ? 0.0375 : 0.075) * prefix_ctas(s) + (beside(s) > 0 ? 0.0 : suffix_us(sms));
      if (us < least) { least = us; best = s; }
    }
    return best;
  }
};

}  // namespace mala
