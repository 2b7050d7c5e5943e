// How moe_tables divides its choices among workgroups.  Host arithmetic alone,
// so that the bounds it has to keep are tested without a device.
#pragma once

#include <stdint.h>

namespace w4a16 {

constexpr int kTableThreads = 1024;
// Choices up to which one launch makes the tables; beyond, each workgroup's
// counts of the E experts lie one after another in `order`, which has n entries.
constexpr int kTablesOneLaunch = 16384;

inline int table_groups(int n, int chunk) { return n > 0 ? (n + chunk - 1) / chunk : 1; }

// Choices of a workgroup: a multiple of the threads, as few as leave at most
// 256 workgroups and, of several launches, no more counts than `order` holds.
// The last workgroup may have a single choice, so that every full one has E of
// them is not enough: 16385 choices of 1024 experts in chunks of 1024 would be
// 17 x 1024 counts in 16385 entries.
inline int table_chunk(int n, int E) {
  int chunk = kTableThreads;
  while (table_groups(n, chunk) > 256 ||
         (n > kTablesOneLaunch && (int64_t)table_groups(n, chunk) * E > n))
    chunk *= 2;
  return chunk;
}

}  // namespace w4a16
