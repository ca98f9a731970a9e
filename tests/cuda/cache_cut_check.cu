// Host run of dt::head_at (no GPU work): places below, at and above 2^32 of requests whose
// heads are shorter and longer than 2^32, multiples of it among them.
#include <cstdio>

#include "dt_cache_attn.cuh"

int main() {
  int bad = 0;
  const int64_t big = int64_t{1} << 32;
  for (int64_t per : {int64_t{1}, int64_t{3}, int64_t{5000}, (int64_t{1} << 31) - 1, int64_t{1} << 31, big - 1, big,
                      big + 1, 2 * big, 3 * big + 7, int64_t{1} << 40})
    for (int64_t at : {int64_t{0}, int64_t{1}, int64_t{4999}, (int64_t{1} << 31) - 1, int64_t{1} << 31, big - 1, big,
                       big + 1, 2 * big - 1, per - 1, per, 7 * per, 8 * per - 1}) {
      if (at < 0 || at / per > 4095) continue;      // heads of a request, at most
      if (dt::head_at(at, per) != at / per) {
        std::printf("place %lld of heads of %lld: %d\n", static_cast<long long>(at), static_cast<long long>(per),
                    dt::head_at(at, per));
        ++bad;
      }
    }
  return bad != 0;
}
