// How many CTAs of a prompt attention call share an item (host code, no CUDA).
#pragma once

#include <math.h>
#include <stdint.h>

namespace exl3 {

constexpr int kSplitSeqs = 128;  // sequences of a launch whose items are shared

// What takes least, in units of a pair of tiles (1.4 us), if the sequences are of one length;
// how long each is lies on the device, and sequences without rows count as well. An item costs 2.8 units
// besides its own, sharing it 3.2 more (4.5 by four). `clusters`: those of 2 and of 4 CTAs that the
// device runs at once. Measured (us, one / two / four CTAs an item, D = 128): 8192 tokens of one
// head (32 items) 97 / 57 / 38; 4096 of 5 heads on one (82) 54 / 37 / 50; 2984 of 4 (48) 41 / 29
// / 32; 1024 of 4 (16) 18.6 / 18.3 / 17.4; 512 of 4 (8) 12.9 / 15.0 / 15.4; 1024 of 40 on 8
// (168) 21 / 40 / 64.
inline int prompt_ranks(int n_seqs, int64_t rows, int causal, int64_t items, int num_sms, const int *clusters) {
  if (n_seqs > kSplitSeqs) return 1;
  const float longest = (float)rows / (float)n_seqs / 128;
  auto units = [&](int ranks, int at_once, float more) {
    if (at_once < 1) return INFINITY;
    float rounds = (float)items / (float)at_once, share = longest / ranks;
    if (rounds < 1.0f) rounds = 1.0f;
    if (causal) return fmaxf(share, rounds * share * 0.5f) + rounds * (2.8f + more);  // half as long on average, dealt evenly
    return ceilf(rounds) * (share + 2.8f + more);
  };
  const float one = units(1, num_sms, 0.f), two = units(2, clusters[0], 3.2f);
  const float four = items <= clusters[1] ? units(4, clusters[1], 4.5f) : INFINITY;
  return four < one && four < two ? 4 : two < one ? 2 : 1;
}

}  // namespace exl3
