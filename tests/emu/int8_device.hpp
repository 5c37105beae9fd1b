// Host stand-ins behind those of swiglu_ops_device.hpp: what the 8-bit integer
// kernels use beyond the other operators.  The sums mean nothing here, as the
// bf16 ones do not; the operands are handed to emu_use so that their reads stay.
#pragma once

#include "swiglu_ops_device.hpp"

namespace swiglu {

typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
inline i32x16 mfma32_i8(const u32x4& a, const u32x4& b, const i32x16& c) {
  emu_use(&a, 16), emu_use(&b, 16);
  return c;
}
inline i32x4 mfma16_i8(const u32x4& a, const u32x4& b, const i32x4& c) {
  emu_use(&a, 16), emu_use(&b, 16);
  return c;
}
// a lane's own value (the threads run one after another)
template <int G>
inline uint32_t group_max(uint32_t v) {
  return v;
}
// lane = threadIdx.x % 64 moves 4 bytes from base + voffset (zeros past the
// resource) to LDS offset lds_wave_base + 4 lane
inline void lds_dma16_wait(uint32_t lds_wave_base, uint32_t voffset, i32x4 rsrc) {
  lds_dma16(lds_wave_base, voffset, rsrc);
}
inline void lds_dma4_wait(uint32_t lds_wave_base, uint32_t voffset, i32x4 rsrc) {
  const uint32_t dst = lds_wave_base + 4u * (threadIdx.x & 63u);
  emu_check_lds(dst, 4, "lds_dma4_wait destination");
  emu_race_dma(dst, 4);
  uint8_t* d = emu_lds_base() + dst;
  const uint32_t bound = (uint32_t)rsrc[2];
  if (voffset >= bound) {
    emu_zero(d, 4);
    return;
  }
  if (voffset + 4u > bound) emu_check_global(nullptr, 0, "lds_dma4_wait read straddles the resource bound");
  const uint8_t* base =
      (const uint8_t*)(uintptr_t)(((uint64_t)(uint32_t)rsrc[1] << 32) | (uint32_t)rsrc[0]);
  emu_check_global(base + voffset, 4, "lds_dma4_wait source");
  emu_copy(d, base + voffset, 4);
}

// the spans' table written out for one thread, and the search in it
struct GroupTable {
  int *lo, *n, *upto;
};
template <int BM>
inline void group_table(const int32_t* offsets, int E, int R, const GroupTable& table) {
  if (threadIdx.x != 0) return;
  int tiles = 0;
  for_spans(offsets, E, R, [&](int e, int lo, int n) {
    tiles += (n + BM - 1) / BM;
    table.lo[e] = lo;
    table.n[e] = n;
    table.upto[e] = tiles;
  });
}
inline int group_find(const GroupTable& table, int E, int t, int from) {
  int e = from & ~63;
  while (e < E - 1 && table.upto[e] <= t) ++e;
  return e;
}

}  // namespace swiglu
