// swiglu_ops_device.hpp -- device building blocks of the mixture-of-experts and
// MXFP4 operators: cross-lane sums and scans, the search for a workgroup's
// expert, the 4-bit matrix instruction and the 4-bit conversions.
#pragma once

#include <tuple>

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
__device__ __forceinline__ float group_sum(float v) {
  v += dpp_f<kDppXor1>(v);
  v += dpp_f<kDppXor2>(v);
  if (G >= 8) v += dpp_f<kDppHalfMirror>(v);
  if (G >= 16) v += dpp_f<kDppMirror>(v);
  if (G >= 32) v += __shfl_xor(v, 16);
  if (G >= 64) v += __shfl_xor(v, 32);
  return v;
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

// ---- which expert a workgroup works on -----------------------------------------
// Sorted rows [offsets[e], offsets[e + 1]) belong to expert e.  Each expert's
// rows are cut into tiles of BM; a unit is one such tile with one of ntn column
// tiles, and an expert's units follow one another.  The number of units is known on the device only:
// the grid is an upper bound, workgroup b takes unit `t` (the units in
// contiguous ranges over the 8 XCDs, as in xcd_remap) and one past the last
// ends at once.  Offsets are held to [0, R] and non-decreasing whatever the
// tensor says, so no row index leaves the sorted range.
struct GroupUnit {
  int expert, first, rows;  // the expert, its first sorted row, its rows
  int local;                // unit number within the expert
};
__device__ __forceinline__ void group_span(const int32_t* offsets, int e, int E, int R, int& lo,
                                           int& n) {
  lo = n = 0;
  if (e < E) {
    lo = min(max(offsets[e], 0), R);
    n = max(min(offsets[e + 1], R) - lo, 0);
  }
}
template <int BM>
__device__ __forceinline__ bool group_find(const int32_t* __restrict__ offsets, int E, int R,
                                           int ntn, int b, GroupUnit& u) {
  const int lane = threadIdx.x & 63;
  int lo, n;
  group_span(offsets, lane, E, R, lo, n);
  int incl = wave_scan((n + BM - 1) / BM);
  int total = __builtin_amdgcn_readlane(incl, 63);
  for (int c = 64; c < E; c += 64) {
    int l2, n2;
    group_span(offsets, c + lane, E, R, l2, n2);
    total += __builtin_amdgcn_readlane(wave_scan((n2 + BM - 1) / BM), 63);
  }
  total *= ntn;
  const int q = total / 8, r = total % 8, x = b % 8, i = b / 8;
  if (i >= q + (x < r ? 1 : 0)) return false;
  const int t = x * q + min(x, r) + i;
  // the first lane whose inclusive count passes t owns it
  int before = 0;
  for (int c = 0;;) {
    const unsigned long long past = __ballot((before + incl) * ntn > t);
    if (past) {
      const int src = __ffsll(past) - 1;
      const int tiles = (n + BM - 1) / BM;
      u.expert = c + src;
      u.first = __builtin_amdgcn_readlane(lo, src);
      u.rows = __builtin_amdgcn_readlane(n, src);
      u.local = t - (before + __builtin_amdgcn_readlane(incl - tiles, src)) * ntn;
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
    c += 64;
    if (c >= E) return false;
    group_span(offsets, c + lane, E, R, lo, n);
    incl = wave_scan((n + BM - 1) / BM);
  }
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
// value of an E2M1 code as fp32: magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  const uint32_t e = (code >> 1) & 3u, m = code & 1u;
  const float a = e ? __builtin_bit_cast(float, ((e + 126u) << 23) | (m << 22)) : 0.5f * (float)m;
  return (code & 8u) ? -a : a;
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
