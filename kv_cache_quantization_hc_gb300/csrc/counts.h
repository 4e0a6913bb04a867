// Two counts in one 64-bit word (tokens in the low half, blocks in the high
// one), added so that a sum past 2^31 - 1 stays there: no carry into the other
// half, and no index made from one is negative.  min(a + b, M) of counts is
// associative, so sums may be taken in any grouping.
#pragma once

#include <stdint.h>

#include "fastdiv.h"

namespace hc {

constexpr uint32_t kMostCount = 0x7fffffffu;

HC_HD uint64_t counts(uint32_t tokens, uint32_t blocks) { return (static_cast<uint64_t>(blocks) << 32) | tokens; }
HC_HD uint32_t tokens_of(uint64_t c) { return static_cast<uint32_t>(c); }
HC_HD uint32_t blocks_of(uint64_t c) { return static_cast<uint32_t>(c >> 32); }
// Each half at most kMostCount, so their plain sum fits 32 bits.
HC_HD uint64_t add_counts(uint64_t a, uint64_t b) {
  const uint64_t s = a + b;
  const uint32_t t = tokens_of(s), k = blocks_of(s);
  return counts(t < kMostCount ? t : kMostCount, k < kMostCount ? k : kMostCount);
}

}  // namespace hc
