// Sorted rows of a grouped product, held to what the caller's tensors contain: the group offsets are on the
// device, so the host can check neither them nor the rows they name.
#pragma once

#include <stdint.h>

#include "device_common.h"

namespace moe {

constexpr int kMaxRowGroups = 1024;

struct GroupRows {
  const int32_t* offs;  // group_offsets + first_group, n_groups + 1 entries
  int n_groups;
  int tail_first;       // first group (relative) of the f32 tail output; n_groups if none
  // row counts, below 2^31 (an offset and a count add up in 32 bits)
  uint32_t m_total;
  uint32_t sorted_rows;
  uint32_t out_rows;
  uint32_t tail_rows;
};

inline uint32_t row_count(int64_t n) { return (uint32_t)(n < INT32_MAX ? n : INT32_MAX); }  // no offset is larger

// The sorted row from which nothing is read or written: the first one that the caller did not vouch for.  Where the
// groups before the tail hold more rows than out does, that is the first row past out, and the tail is empty.
__device__ __forceinline__ int rows_end(const GroupRows& r) {
  const uint32_t first = r.offs[0], tail = r.offs[r.tail_first];
  const uint32_t room = tail - first > r.out_rows ? first + r.out_rows : tail + r.tail_rows;
  return (int)min(min(first + r.m_total, r.sorted_rows), room);
}

}  // namespace moe
