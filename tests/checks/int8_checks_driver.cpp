// The argument checks of the scored router and the 8-bit integer entry points
// (swiglu_checks.hpp) on extreme sizes, as checks_driver.cpp does for the other
// operators: a byte count that passes 64 bits ends the program.
#include <stdio.h>

#include <vector>

#include "swiglu_checks.hpp"

namespace swiglu {
// stand-ins of the kernels' files, as large as theirs
long long route_workspace_bytes(long long T, long long E, long long k) { return T * k > 512 ? 4 * E : 0; }
long long grouped_threads(bool, long long R, long long, long long, int) { return R; }
long long norm_threads(long long T, long long) { return T; }
long long int8_quantize_threads(long long rows, long long) { return rows * 1024; }
bool int8_launchable(const Int8Call& c, int) {
  return ((c.R + 31) / 32 + c.E) * ((c.C() + 31) / 32) < (1LL << 60);
}
}  // namespace swiglu

using namespace swiglu;

static const void* at(int i) { return (const void*)((uintptr_t)(i + 1) << 48); }

// calls f(sizes) for each size at each value; how many f accepted
template <typename F>
static int sweep(const char* name, std::vector<long long> usual, F f) {
  const long long values[] = {INT64_MIN, -1, 0, 1, 2, 8, 16, 64, 1024, 1LL << 20, 1LL << 23, 1LL << 27,
                              (1LL << 30) - 64, 1LL << 30, (1LL << 31) - 64, (1LL << 31) - 1, 1LL << 31,
                              1LL << 40, 1LL << 46, 1LL << 58, 1LL << 61, 1LL << 62, INT64_MAX - 63, INT64_MAX};
  int accepted = 0;
  for (size_t i = 0; i < usual.size(); ++i)
    for (long long v : values)
      for (int all = 0; all < 2; ++all) {
        std::vector<long long> s = all ? std::vector<long long>(usual.size(), v) : usual;
        if (all) s[i] = usual[i];
        else s[i] = v;
        accepted += f(s) == checks::kOk;
      }
  printf("%s: %d accepted\n", name, accepted);
  fflush(stdout);
  return accepted;
}

int main() {
  bool noop;
  for (int groups : {1, 8, 64})
    sweep("route_score", {100, 64, 6}, [&](const std::vector<long long>& s) {
      const int c = checks::route(at(0), at(1), at(2), at(3), at(4), at(5), 1LL << 40, s[0], s[1], s[2], 1);
      const RouteScore r{(const float*)at(6), 1, 1.0f, groups, 1, 2};
      return c != checks::kOk ? c : checks::route_score(r, at(1), at(2), at(3), at(4), at(5), s[0], s[1], s[2], 1);
    });
  sweep("quantize_int8", {10, 64}, [&](const std::vector<long long>& s) {
    return checks::quantize_int8(at(0), at(1), at(2), s[0], s[1], &noop);
  });
  sweep("pack_int8", {4, 40, 64}, [&](const std::vector<long long>& s) {
    return checks::pack_int8(at(0), at(1), s[0], s[1], s[2], &noop);
  });
  for (bool gated : {false, true})
    for (bool grouped : {false, true})
      sweep("int8_product", {10, 20, 64, 64, 8, 2}, [&](const std::vector<long long>& s) {
        const Int8Call c{gated, grouped, (const uint8_t*)at(0), (const float*)at(1), (const int32_t*)at(2),
                         (const int32_t*)at(3), (const uint8_t*)at(4), (const float*)at(5), (uint16_t*)at(6),
                         s[0], s[1], s[2], s[3], s[4], s[5], 256};
        return checks::int8_product(c, -1, &noop);
      });
  printf("done\n");
  return 0;
}
