// Host check of views_meet (csrc/byte_views.h). Reads pairs of views, each "base row step0
// ext0 step1 ext1 step2 ext2", from stdin and prints 1 (they meet) or 0 for each pair.
#include <cstdio>

#include "../../sparse_window_attention_b200/csrc/byte_views.h"

static bool read(basa::ByteView *v) {
  unsigned long long base;
  long long x[7];
  if (std::scanf("%llu %lld %lld %lld %lld %lld %lld %lld", &base, &x[0], &x[1], &x[2], &x[3], &x[4], &x[5], &x[6]) != 8)
    return false;
  *v = {uintptr_t(base), x[0], {x[1], x[3], x[5]}, {x[2], x[4], x[6]}};
  return true;
}

int main() {
  basa::ByteView a, b;
  while (read(&a) && read(&b)) std::printf("%d\n", int(basa::views_meet(a, b)));
  return 0;
}
