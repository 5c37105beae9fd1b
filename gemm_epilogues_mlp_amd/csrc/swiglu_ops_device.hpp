// swiglu_ops_device.hpp -- device building blocks of the mixture-of-experts and
// MXFP4 operators: cross-lane sums and scans, the search for a workgroup's
// expert, the 4-bit matrix instruction and the 4-bit conversions.
#pragma once

#include <tuple>
#include <type_traits>

#include "swiglu_device.hpp"

namespace swiglu {

// ---- cross-lane ---------------------------------------------------------------
// DPP controls (64-lane waves, rows of 16): a permutation inside quads, the
// mirrored half row and row (together an exchange over distances 1, 2, 4 and
// 8), shifts inside a row, and the broadcasts of lanes 15 and 31.
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppMirror = 0x140;

template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  const int x = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, false));
}

// Maximum and sum over aligned groups of G lanes (G = 4, 16, 32 or 64); every
// lane of the group receives the same bits (the order of the additions is the
// same tree for all of them, as addition commutes).
template <int G>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, dpp_f<kDppXor1>(v));
  v = fmaxf(v, dpp_f<kDppXor2>(v));
  if (G >= 8) v = fmaxf(v, dpp_f<kDppHalfMirror>(v));
  if (G >= 16) v = fmaxf(v, dpp_f<kDppMirror>(v));
  if (G >= 32) v = fmaxf(v, __shfl_xor(v, 16));
  if (G >= 64) v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  auto dpp = [](auto ctrl, uint32_t x) __attribute__((always_inline)) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, decltype(ctrl)::value, 0xf, 0xf, false);
  };
  v = max(v, dpp(std::integral_constant<int, kDppXor1>{}, v));
  v = max(v, dpp(std::integral_constant<int, kDppXor2>{}, v));
  if (G >= 8) v = max(v, dpp(std::integral_constant<int, kDppHalfMirror>{}, v));
  if (G >= 16) v = max(v, dpp(std::integral_constant<int, kDppMirror>{}, v));
  if (G >= 32) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
  if (G >= 64) v = max(v, (uint32_t)__shfl_xor((int)v, 32));
  return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  v += dpp_f<kDppXor1>(v);
  v += dpp_f<kDppXor2>(v);
  if (G >= 8) v += dpp_f<kDppHalfMirror>(v);
  if (G >= 16) v += dpp_f<kDppMirror>(v);
  if (G >= 32) v += __shfl_xor(v, 16);
  if (G >= 64) v += __shfl_xor(v, 32);
  return v;
}

// Lanes 32-63 of a change places with lanes 0-31 of b.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// Inclusive sum of the lanes up to and with this one, over a whole wave.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31
  return v;
}

// Inclusive maximum of the lanes up to and with this one, of v >= 0.
__device__ __forceinline__ int wave_scan_max(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));
  return v;
}

// ---- which expert a workgroup works on -----------------------------------------
// Sorted rows [offsets[e], offsets[e + 1]) belong to expert e.  Each expert's
// rows are cut into tiles of BM, the last one of as many parts (BM / PARTS
// rows) as it needs.  A unit is one tile with one of ntn column tiles; an
// expert's units follow one another, and the units of all experts in turn are
// cut into eight ranges of equal work, one for each XCD, so that the units that
// share weights and rows of A share an L2.  The work of a tile of p parts counts
// as 2 p + 3: a quarter of the rows still takes all of the weights (measured at
// PARTS = 4: 0.44 of a whole tile's time where this has 5 / 11).  (Dealing the short
// tiles out behind all whole ones balances as well, but they then read every
// expert's weights a second time: 1053 against 960 us for 32760 rows, 32
// experts, 3584 x 4736 weights each.)
// Whatever the tensor says, an offset is held to [0, R] and counts as the largest
// one before it where it is below that: no row index leaves the sorted range, and
// the spans never overlap, so there are never more than R rows in all.
struct GroupUnit {
  int expert, first, rows;  // the expert, its first sorted row, its rows
  int local;                // unit number within the expert
};
struct GroupRange {
  int begin, end;  // units of this XCD
};
// this lane's span, of expert c + lane; `reach` is where the spans before c end
// and becomes where those of this wave do
__device__ __forceinline__ void group_span(const int32_t* offsets, int c, int E, int R, int& reach,
                                           int& lo, int& n) {
  const int e = c + (int)(threadIdx.x & 63);
  int from = 0, to = 0;
  if (e < E) {
    from = min(max(offsets[e], 0), R);
    to = min(max(offsets[e + 1], 0), R);
  }
  lo = max(wave_scan_max(from), reach);
  n = max(to - lo, 0);
  reach = __builtin_amdgcn_readlane(lo + n, 63);
}
template <int BM, int PARTS>
__device__ __forceinline__ int group_work(int n) {
  const int left = (n % BM + BM / PARTS - 1) / (BM / PARTS);
  return n / BM * (2 * PARTS + 3) + (left > 0 ? 2 * left + 3 : 0);
}
template <int BM, int PARTS>
__device__ __forceinline__ GroupRange group_range(const int32_t* __restrict__ offsets, int E,
                                                  int R, int ntn, int x) {
  int lo, n, sum = 0, reach = 0;
  for (int c = 0; c < E; c += 64) {
    group_span(offsets, c, E, R, reach, lo, n);
    sum += __builtin_amdgcn_readlane(wave_scan(group_work<BM, PARTS>(n)), 63);
  }
  // where an eighth of the work ends: the expert it falls into, and of its
  // units the share that its work before that point has in its whole
  const long long work = (long long)sum * ntn;
  const long long at[2] = {work * x / 8, work * (x + 1) / 8};
  int cut[2] = {-1, -1}, before_p = 0, before_t = 0;
  reach = 0;
  for (int c = 0; c < E; c += 64) {
    if (E > 64) group_span(offsets, c, E, R, reach, lo, n);
    const int p = group_work<BM, PARTS>(n), t = (n + BM - 1) / BM;
    const int ip = wave_scan(p), it = wave_scan(t);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const unsigned long long past = __ballot((long long)(before_p + ip) * ntn > at[i]);
      if (cut[i] >= 0 || !past) continue;
      const int src = __ffsll(past) - 1;
      const int sp = __builtin_amdgcn_readlane(p, src), st = __builtin_amdgcn_readlane(t, src);
      const long long in = at[i] - (long long)(before_p + __builtin_amdgcn_readlane(ip, src) - sp) * ntn;
      cut[i] = (before_t + __builtin_amdgcn_readlane(it, src) - st) * ntn +
               (int)(in * st / sp);
    }
    before_p += __builtin_amdgcn_readlane(ip, 63);
    before_t += __builtin_amdgcn_readlane(it, 63);
  }
  // the end of the work lies in no expert
  return GroupRange{cut[0] >= 0 ? cut[0] : before_t * ntn, cut[1] >= 0 ? cut[1] : before_t * ntn};
}
// the expert of unit t, which is one of the units
template <int BM>
__device__ __forceinline__ GroupUnit group_unit(const int32_t* __restrict__ offsets, int E, int R,
                                                int ntn, int t) {
  GroupUnit u{0, 0, 0, 0};
  int before = 0, reach = 0;
  for (int c = 0; c < E; c += 64) {
    int lo, n;
    group_span(offsets, c, E, R, reach, lo, n);
    const int tiles = (n + BM - 1) / BM, incl = wave_scan(tiles);
    const unsigned long long past = __ballot((before + incl) * ntn > t);
    if (past) {
      const int src = __ffsll(past) - 1;
      u.expert = c + src;
      u.first = __builtin_amdgcn_readlane(lo, src);
      u.rows = __builtin_amdgcn_readlane(n, src);
      u.local = t - (before + __builtin_amdgcn_readlane(incl - tiles, src)) * ntn;
      break;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return u;
}

// ---- MXFP4 ------------------------------------------------------------------------
// v_mfma_scale_f32_32x32x64_f8f6f4 with both sources E2M1 (format 4): lane l
// holds row or column l % 32 and the 32 consecutive k of half l / 32 in 16
// bytes (low nibble first), and passes that block's E8M0 scale byte (byte SEL
// of its scale register).  The output layout is that of the bf16 32x32x16.
template <int SEL0, int SEL1>
__device__ __forceinline__ f32x16 mfma32_f4(const u32x4& a, const u32x4& b, const f32x16& c,
                                            uint32_t sa, uint32_t sb) {
  const u32x4 z{0, 0, 0, 0};  // the instruction reads four registers a source
  const i32x8 x = __builtin_bit_cast(i32x8, __builtin_shufflevector(a, z, 0, 1, 2, 3, 4, 5, 6, 7));
  const i32x8 y = __builtin_bit_cast(i32x8, __builtin_shufflevector(b, z, 0, 1, 2, 3, 4, 5, 6, 7));
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, SEL0, (int)sa, SEL1,
                                                          (int)sb);
}
// Eight bf16 (four dwords) times 2^-s (scale = 2^s as fp32) to E2M1, nearest
// even and saturating at 6; first value in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1_codes(const u32x4& v, float scale) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const uint32_t d0 = v[0], d1 = v[1], d2 = v[2], d3 = v[3];
  uint32_t o = 0;
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, d0), scale, 0);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, d1), scale, 1);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, d2), scale, 2);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, d3), scale, 3);
  return o;
}
// Eight E2M1 codes times scale (2^s as fp32) to bf16, four dwords.
__device__ __forceinline__ u32x4 e2m1_values(uint32_t c, float scale) {
  const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
  const auto v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
  const auto v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
  const auto v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
  return u32x4{__builtin_bit_cast(uint32_t, v0), __builtin_bit_cast(uint32_t, v1),
               __builtin_bit_cast(uint32_t, v2), __builtin_bit_cast(uint32_t, v3)};
}
// 2^(e - 127) as fp32 for an E8M0 byte e < 255 (e = 0 is a subnormal there)
__device__ __forceinline__ float e8m0_scale(int e) {
  return __builtin_bit_cast(float, e > 0 ? (uint32_t)e << 23 : 1u << 22);
}

// ---- launches ---------------------------------------------------------------------
// Judged by hipLaunchKernel's own return value, as every launch of the library.
template <typename... P, typename... Args>
static hipError_t launch_op(void (*k)(P...), dim3 grid, dim3 block, hipStream_t stream,
                            Args... args) {
  static_assert(sizeof...(P) == sizeof...(Args), "kernel argument count");
  std::tuple<std::decay_t<P>...> vals(static_cast<std::decay_t<P>>(args)...);
  return std::apply(
      [&](auto&... v) {
        void* argv[] = {static_cast<void*>(&v)...};
        return hipLaunchKernel(reinterpret_cast<const void*>(k), grid, block, argv, 0, stream);
      },
      vals);
}

}  // namespace swiglu
