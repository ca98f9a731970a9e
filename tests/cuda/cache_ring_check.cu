// Host run of dt::StepRing against a model of its barriers (no GPU work): every step taken,
// and every step left in flight by a wait that was given up, is waited for at the place and
// parity of its own phase, and nothing stays in flight.
#include <cstdio>
#include <deque>
#include <vector>

#include "dt_cache_attn.cuh"

int main() {
  int bad = 0;
  for (uint32_t places : {2u, 3u, 4u})
    for (int steps = 0; steps <= 13; ++steps)
      for (int gives_up = 0; gives_up <= steps; ++gives_up) {   // at this step; steps: never
        dt::StepRing r = {0u, 0u, 0u};
        std::vector<uint32_t> phase(places, 0);                  // of a place's next step
        std::deque<std::pair<uint32_t, uint32_t>> flight;        // place, parity
        auto issue = [&] {
          flight.push_back({r.in, phase[r.in]++ & 1u});
          r.issued(places);
        };
        auto wait = [&] {
          if (flight.empty() || flight.front() != std::make_pair(r.out, r.parity)) ++bad;
          if (!flight.empty()) flight.pop_front();
          r.taken(places);
        };
        int k = 0;
        for (; k < steps && k < static_cast<int>(places); ++k) issue();
        int s = 0;
        for (; s < steps && s != gives_up; ++s) {
          wait();
          if (k < steps) { issue(); ++k; }
        }
        for (int left = dt::StepRing::flying(s, steps, places); left > 0; --left) wait();
        if (!flight.empty()) ++bad;
      }
  if (bad) std::printf("%d waits of another step's phase, or steps left in flight\n", bad);
  return bad != 0;
}
