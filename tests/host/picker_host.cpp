// Host build of the row kernels' rule (sample_rule.hpp).  For
// tests/test_picker_rule_host.py: reads lines "rows V any_list" from stdin and
// writes "threads pieces-of-the-row pieces-that-fit" for each.
#include <cstdio>

#include "sample_rule.hpp"

int main() {
  long long rows = 0, V = 0;
  int any = 0;
  while (std::scanf("%lld %lld %d", &rows, &V, &any) == 3) {
    const int t = flce::picker_threads(rows, V, any != 0);
    std::printf("%d %lld %d\n", t, (V + flce::kPiece - 1) / flce::kPiece, flce::picker_pieces(t));
  }
  return 0;
}
