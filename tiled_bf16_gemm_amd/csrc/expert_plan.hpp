// How many workgroups sort the slots (expert_sort.hip).  Host arithmetic only.
#pragma once
#include <stdint.h>

namespace tbg {

struct SortPlan {
  bool small;      // one workgroup and one launch, no workspace
  int parts;       // workgroups
  int64_t part;    // slots each
  int64_t bytes;   // workspace: a count for every part and expert
};

constexpr int64_t kSmallSlots = 4096;

inline SortPlan plan_expert_sort(int64_t slots, int64_t groups) {
  SortPlan s{true, 1, slots, 0};
  // one workgroup holds four slots a thread, and has fewer waves the more experts there are
  int64_t waves = 16;
  while (waves > 1 && waves * groups > 8192) waves /= 2;
  if (slots <= waves * 256 && slots <= kSmallSlots) return s;
  s.small = false;
  const int64_t step = 2048, most = 256;
  int64_t steps = (slots + step - 1) / step;
  const int64_t each = (steps + most - 1) / most;
  s.part = each * step;
  s.parts = (int)((slots + s.part - 1) / s.part);
  s.bytes = (s.parts * groups * 4 + 255) / 256 * 256;
  return s;
}

}  // namespace tbg
