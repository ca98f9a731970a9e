// Host run of dt::cache_row against the paged layout's definition (no GPU work).
#include <cstdio>
#include <vector>

#include "dt_cache.cuh"

int main() {
  int bad = 0;
  for (int page : {16, 32, 64, 128}) {
    const int batch = 3, width = 5, pages = 4, Hkv = 3;
    // good pages, the pool's end, negative, far outside
    std::vector<int32_t> table = {0, 3, 2, 1, 0, 4, -1, 2, 2147483647, -2147483647 - 1, 3, 3, 3, 3, 3};
    dt_cache c = {};
    c.table = table.data(); c.pages = pages; c.page = page; c.Hkv = Hkv; c.dh = 64;
    c.table_width = width; c.batch = batch;
    const dt::CacheView v = dt::cache_view(c);
    auto check = [&](int b, int64_t index, int hk) {
      int64_t want = -1;
      if (index >= 0 && index / page < width) {
        const int64_t p = table[b * width + index / page];
        if (p >= 0 && p < pages) want = (p * Hkv + hk) * page + index % page;
      }
      const int64_t got = dt::cache_row(v, b, index, hk);
      if (got != want || got >= static_cast<int64_t>(pages) * Hkv * page) {
        std::printf("page %d b %d index %lld hk %d: %lld, not %lld\n", page, b,
                    static_cast<long long>(index), hk, static_cast<long long>(got),
                    static_cast<long long>(want));
        ++bad;
      }
    };
    for (int b = 0; b < batch; ++b)
      for (int hk = 0; hk < Hkv; ++hk) {
        for (int64_t i = -3; i < static_cast<int64_t>(width + 2) * page; ++i) check(b, i, hk);
        for (int64_t i : {int64_t{1} << 31, (int64_t{1} << 31) - 1, int64_t{1} << 40, -(int64_t{1} << 33)})
          check(b, i, hk);
      }
  }
  return bad != 0;
}
