// Host stand-in for swiglu_ops_device.hpp, beside that of swiglu_device.hpp: what
// the grouped products and the MXFP4 kernels use of it.  The threads of a
// workgroup run one after another, so nothing is exchanged between lanes: the
// search for a workgroup's expert is written out for one thread (the same
// units, in the same order), maxima over lanes and swapped halves leave a
// lane's own value, and the 4-bit conversions give no values.
#pragma once

#include <tuple>
#include <type_traits>

#include "swiglu_device.hpp"

inline uint32_t max(uint32_t a, uint32_t b) { return a > b ? a : b; }
#define __builtin_amdgcn_update_dpp(old, v, ctrl, rows, banks, bound) (v)

namespace swiglu {

constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E;

inline void swap_halves(uint32_t&, uint32_t&) {}

// ---- which expert a workgroup works on -----------------------------------------
struct GroupUnit {
  int expert, first, rows, local;
};
struct GroupRange {
  int begin, end;
};
// f(expert, first row, rows) for every expert's span: offsets held to [0, R] and
// to the largest one before
template <typename F>
inline void for_spans(const int32_t* offsets, int E, int R, F f) {
  int reach = 0;
  for (int e = 0; e < E; ++e) {
    const int from = min(max((int)offsets[e], 0), R), to = min(max((int)offsets[e + 1], 0), R);
    const int lo = max(from, reach), n = max(to - lo, 0);
    reach = lo + n;
    f(e, lo, n);
  }
}
template <int BM, int PARTS>
inline int group_work(int n) {
  const int left = (n % BM + BM / PARTS - 1) / (BM / PARTS);
  return n / BM * (2 * PARTS + 3) + (left > 0 ? 2 * left + 3 : 0);
}
template <int BM, int PARTS>
inline GroupRange group_range(const int32_t* offsets, int E, int R, int ntn, int x) {
  long long work = 0;
  for_spans(offsets, E, R, [&](int, int, int n) { work += group_work<BM, PARTS>(n); });
  work *= ntn;
  const long long at[2] = {work * x / 8, work * (x + 1) / 8};
  int cut[2] = {-1, -1}, units = 0;
  long long before = 0;
  for_spans(offsets, E, R, [&](int, int, int n) {
    const long long p = (long long)group_work<BM, PARTS>(n) * ntn;
    const int t = (n + BM - 1) / BM * ntn;
    for (int i = 0; i < 2; ++i)
      if (cut[i] < 0 && before + p > at[i]) cut[i] = units + (int)((at[i] - before) * t / p);
    before += p;
    units += t;
  });
  return GroupRange{cut[0] >= 0 ? cut[0] : units, cut[1] >= 0 ? cut[1] : units};
}
template <int BM>
inline GroupUnit group_unit(const int32_t* offsets, int E, int R, int ntn, int t) {
  GroupUnit u{0, 0, 0, 0};
  int before = 0;
  for_spans(offsets, E, R, [&](int e, int lo, int n) {
    const int units = (n + BM - 1) / BM * ntn;
    if (t >= before && t < before + units) u = GroupUnit{e, lo, n, t - before};
    before += units;
  });
  return u;
}

// ---- MXFP4 ------------------------------------------------------------------------
template <int SEL0, int SEL1>
inline f32x16 mfma32_f4(const u32x4& a, const u32x4& b, const f32x16& c, uint32_t sa, uint32_t sb) {
  static_assert(SEL0 >= 0 && SEL0 < 4 && SEL1 >= 0 && SEL1 < 4, "byte select");
  emu_use(&a, 16), emu_use(&b, 16), emu_use(&sa, 4), emu_use(&sb, 4);
  return c;
}
inline uint32_t e2m1_codes(const u32x4& v, float) { return v[0] ^ v[1] ^ v[2] ^ v[3]; }
inline u32x4 e2m1_values(uint32_t c, float) { return u32x4{c, c, c, c}; }
inline float e8m0_scale(int e) { return ldexpf(1.0f, e - 127); }

// ---- launches ---------------------------------------------------------------------
template <typename... P, typename... Args>
static hipError_t launch_op(void (*k)(P...), dim3 grid, dim3 block, hipStream_t, Args... args) {
  static_assert(sizeof...(P) == sizeof...(Args), "kernel argument count");
  emu_launch(k, grid, block, static_cast<std::decay_t<P>>(args)...);
  return hipSuccess;
}

}  // namespace swiglu
