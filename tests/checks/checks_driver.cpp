// The argument checks of the mixture-of-experts and MXFP4 entry points
// (swiglu_checks.hpp) on extreme sizes, built with the undefined-behaviour
// sanitizer: a byte count that passes 64 bits ends the program.  Every size
// takes every value below with the others at ordinary ones, and with all others
// at the same value.
#include <stdio.h>

#include <vector>

#include "swiglu_checks.hpp"

namespace swiglu {
// stand-ins of the kernels' files, as large as theirs
long long route_workspace_bytes(long long T, long long E, long long k) { return T * k > 512 ? 4 * E : 0; }
long long grouped_threads(bool up, long long R, long long N, long long E, int) {
  return (R / 16 + E) * ((up ? 2 : 1) * N / 64 + 1) * 512;
}
long long norm_threads(long long T, long long) { return T * 1024; }
}  // namespace swiglu

using namespace swiglu;

static const void* at(int i) { return (const void*)((uintptr_t)(i + 1) << 48); }

// calls f(sizes) for each size at each value; how many f accepted
template <typename F>
static int sweep(const char* name, std::vector<long long> usual, F f) {
  const long long values[] = {INT64_MIN, -1, 0, 1, 2, 8, 32, 64, 1024, 1LL << 20, 1LL << 23, 1LL << 27,
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
  sweep("route", {100, 64, 6}, [&](const std::vector<long long>& s) {
    return checks::route(at(0), at(1), at(2), at(3), at(4), at(5), 1LL << 40, s[0], s[1], s[2], 1);
  });
  for (bool up : {false, true})
    sweep("grouped", {10, 20, 64, 40, 8, 2}, [&](const std::vector<long long>& s) {
      return checks::grouped(up, at(0), at(1), at(2), at(3), at(4), s[0], s[1], s[2], s[3], s[4], s[5], -1, &noop);
    });
  for (int dtype : {0, 1})
    sweep("combine_norm", {10, 64, 2, 64}, [&](const std::vector<long long>& s) {
      NormCall c{at(0), (const float*)at(1), (const int32_t*)at(2), at(3), at(4), at(5), at(6), at(7),
                 (void*)at(8), (void*)at(9), s[0], s[1], s[2], 1.0f, 1e-6f, s[3], dtype == 1};
      return checks::combine_norm(c, dtype, &noop);
    });
  for (bool back : {false, true})
    sweep("convert_mxfp4", {10, 64}, [&](const std::vector<long long>& s) {
      return checks::convert_mxfp4(at(0), at(1), at(2), s[0], s[1], back, &noop);
    });
  sweep("forward_mxfp4", {10, 64, 64}, [&](const std::vector<long long>& s) {
    Fp4Call c{(const uint8_t*)at(0), (const uint8_t*)at(1), (const uint8_t*)at(2), (const uint8_t*)at(3),
              (uint16_t*)at(4), s[0], s[1], s[2], 256};
    return checks::forward_mxfp4(c, &noop);
  });
  printf("done\n");
  return 0;
}
