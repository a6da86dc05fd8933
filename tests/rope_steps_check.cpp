// Reads "rot_dim base kind factor orig_max_pos beta_fast beta_slow" lines and
// prints each one's steps.
#include <cstdio>

#include "rope_steps.h"

int main() {
  int rot, kind, orig;
  double base, factor, fast, slow;
  while (std::scanf("%d %la %d %la %d %la %la", &rot, &base, &kind, &factor, &orig, &fast, &slow) == 7) {
    uint64_t steps[128];
    dsa::rope_steps(rot, base, {static_cast<dsa::RopeScaling::Kind>(kind), factor, orig, fast, slow}, steps);
    for (int i = 0; i < rot / 2; ++i) std::printf("%llu ", (unsigned long long)steps[i]);
    std::printf("\n");
  }
  return 0;
}
