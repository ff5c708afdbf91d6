// decay_share.h -- how the CTAs of decay attention's pass on the tensor cores share its
// work, for the launch and the kernel alike; plain C++, so that the host can go through it.
//
// An item is a segment of a head and a group of value channels, and takes up to `chunks`
// chunks.  Where there are more items than CTAs can be resident, the CTAs of a pass get
// equal runs of its items' chunks, one after another, so that the last round is as full as
// the others (384 items in 2.6 rounds of 152 for 3).  An item that two CTAs share is begun
// by the first, before all else, and ended by the second, after all else, which takes the
// state over through memory; it is there by then, as no CTA has less than an item's chunks.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define DELTA_HOST_DEVICE __host__ __device__
#else
#define DELTA_HOST_DEVICE
#endif

namespace delta {
namespace decay {

constexpr int kParts = 24;  // parts of a CTA at most: the kernel keeps a table

// Chunks from .. to of an item, in the order of the pass
struct Run {
  uint32_t item;
  int from, to;
};
// the k-th part of CTA `cta` of the `ctas` that share a pass's items
DELTA_HOST_DEVICE inline bool shared_part(uint32_t items, uint32_t chunks, uint32_t cta, uint32_t ctas, int k, Run &r) {
  const uint64_t units = (uint64_t)items * chunks;
  const uint64_t u0 = units * cta / ctas, u1 = units * (cta + 1) / ctas;
  const uint32_t first = (uint32_t)(u0 / chunks), last = (uint32_t)((u1 - 1) / chunks);
  const int count = (int)(last - first) + 1;
  if (k >= count) return false;
  r.item = k == 0 ? last : k == count - 1 ? first : first + (uint32_t)k;
  r.from = r.item == first ? (int)(u0 - (uint64_t)first * chunks) : 0;
  r.to = r.item == last ? (int)(u1 - (uint64_t)last * chunks) : (int)chunks;
  return true;
}

// CTAs of each of a call's passes, one an SM
DELTA_HOST_DEVICE inline int64_t shared_ctas(int passes, int64_t sms) { return sms / passes; }

// Whether CTAs share `items`, those of all passes: where that fills the last round.  Many
// rounds need it not.  A run of r items' chunks touches up to r + 1 of them, r rounded up,
// and no CTA may have more parts than its table has places, or less than one item.
inline bool share_items(int64_t items, int passes, int64_t sms) {
  const int64_t ctas = shared_ctas(passes, sms), each = items / passes;
  return items > sms && items <= (kParts - 4) * sms && each >= ctas && each <= (kParts - 2) * ctas &&
         (items + sms - 1) / sms * sms * 20 > items * 21;
}

}  // namespace decay
}  // namespace delta
