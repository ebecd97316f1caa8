// Host program: whatever an item's note of its parts holds, either it is refused or every slot that the
// joining kernel reads for it lies inside the workspace.
#include <cstdio>
#include <cstdint>
#include <initializer_list>

#include "paged.h"

int main() {
  uint64_t x = 88172645463325252ull;
  auto next = [&]() { return x ^= x << 13, x ^= x >> 7, x ^= x << 17, x; };
  long long known = 0, refused = 0;
  for (int i = 0; i < 4000000; ++i) {
    const int ctas = 1 + (int)(next() % fa::kPagedMaxCtas);
    // small numbers around the limits, large ones, and repeated bytes as in a filled workspace
    auto any = [&]() -> int {
      const uint64_t r = next();
      if (r % 4 == 0) return (int)(uint32_t)next();
      if (r % 4 == 1) return (int)(0x01010101u * (uint32_t)(next() & 255));
      return (int)(next() % 200) - 25;
    };
    const int first = any(), last = any();
    if (!fa::parts_known(first, last, ctas)) {
      ++refused;
      if (first >= 0 && last >= first && last < ctas) return std::printf("refused %d %d\n", first, last), 1;
      continue;
    }
    ++known;
    const int B = 1 + (int)(next() % 9), H_kv = 1 + (int)(next() % 5), T = 1 + (int)(next() % 300);
    const int H = H_kv * (1 + (int)(next() % 4)), d = 64 << (next() % 3);
    const fa::PagedWs w = fa::paged_ws_layout(B, H, H_kv, T, d);
    const long long base = w.packed ? w.own_items : 0;
    for (int part : {first, last})
      for (int begins : {0, 1})
        if (base + 2ll * part + begins >= w.own_slots) return std::printf("slot of part %d\n", part), 1;
  }
  if (known < 1000 || refused < 1000) return std::printf("too few cases\n"), 1;
  std::printf("ok %lld known, %lld refused\n", known, refused);
  return 0;
}
