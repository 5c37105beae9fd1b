// swiglu_int8.hip -- 8-bit integers: quantisation of bf16 rows, weights into fragment
// order, and gated and plain products of such rows with such weights, for one
// weight set or grouped by expert.
//
// Codes are symmetric with one fp32 scale a row (a token of the activations, an
// output channel of the weights), so a product is exact in 32-bit integers and
//   p[m, c] = (SQ[m] sum_k Q[m, k] W[c, k]) SW[c],
// three roundings in all: the sum to fp32 and two products.
// Weights are stored in the order the 32x32x32 matrix instructions take them (rows
// in blocks of 32, K in groups of 128, G = ceil(K / 128)):
//   P[(((b G + g) 4 + s) 2 + h) 512 + 16 i + j] = W8[32 b + i][128 g + 32 s + 16 h + j]
// padded with zeros, so lane i + 32 h finds its 16 bytes next to its neighbours'
// (1 KB a load). Activations stay row-major, as a gather by row wants them; what is
// read past a row's end meets zeros of the weights.
#include "swiglu_internal.h"
#include "swiglu_ops_device.hpp"

#include <algorithm>
#include <cmath>
#include <type_traits>
#include <utility>

namespace swiglu {

enum Int8Op { I8_GATED = 0, I8_PLAIN = 1 };

// The tensors of a product, as its kernels take them.
struct Int8Args {
  const uint8_t* A;        // [TA, K]
  const float* SA;         // [TA]
  const int32_t* rows;     // grouped: [R] slot of each sorted row
  const int32_t* offsets;  // grouped: [E + 1]
  const uint8_t* W;        // E fragment-ordered matrices of C rows
  const float* SW;         // [E, C]
  uint16_t* Y;             // [R, N]
  int TA, R, N, K, E, k;   // not grouped: R = TA
  int C;                   // 2N (gated) or N (plain)
};

// Two fp32 to bf16, nearest even, by one instruction.
__device__ __forceinline__ uint32_t two_bf16(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// Row of A of sorted row `pos`, -1 if the slot names no row of A.
template <int OP>
__device__ __forceinline__ int int8_a_row(const Int8Args& g, int pos) {
  if (OP == I8_PLAIN) return pos;
  const int slot = g.rows[pos];
  return slot >= 0 && slot / g.k < g.TA ? slot / g.k : -1;
}

// ============================================================================
// Quantisation
// ============================================================================
// The nearest integer to 127 x / a, the even one at a tie: c = 127 x is exact (15
// bits), t = c r with r the rounded 1 / a is within two steps of the quotient, and one
// step of Newton with the exact remainder c - t a makes a quotient that is a half
// exactly that half (all other quotients of two 8-bit significands times 127 are
// 2^-17 or more away from one, relative). Adding 1.5 2^23 rounds to an integer that
// then stands in the low bits.
__device__ __forceinline__ uint32_t int8_code(float c, float a, float r) {
  float t = c * r;
  t = __builtin_fmaf(__builtin_fmaf(-t, a, c), r, t);
  return __builtin_bit_cast(uint32_t, t + 12582912.0f);
}

// One row by W waves of a workgroup of 4 or more waves, a thread holding CH chunks of 8
// values from the load of the maximum to the store of the codes, so X is read once.  Bound
// by memory: 8192 x 18944 in 75 to 84 us (78: 6.0 TB/s of bf16 in and codes out); 16 x 3584 in 2.6, a launch.
template <int W, int CH>
__global__ __launch_bounds__(64 * (W < 4 ? 4 : W)) void quantize_int8_kernel(
    const uint16_t* __restrict__ X, uint8_t* __restrict__ Q, float* __restrict__ S, int rows, int K) {
  constexpr int kThreads = 64 * (W < 4 ? 4 : W), T = 64 * W, RPW = kThreads / T;
  __shared__ __attribute__((aligned(16))) uint32_t top[W];
  const int tid = threadIdx.x % T;
  const int row = blockIdx.x * RPW + threadIdx.x / T;
  if (RPW > 1 && row >= rows) return;  // whole waves, and no barrier below
  const uint16_t* x = X + (size_t)row * K;
  u32x4 v[CH];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * T + tid) * 8;
    v[c] = k < K ? load16_stream(x + k) : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int d = 0; d < 4; ++d) m = max(m, max(v[c][d] & 0x7fffu, (v[c][d] >> 16) & 0x7fffu));
  m = group_max<64>(m);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) m = max(m, top[w]);
  }
  // bf16 bits of the largest magnitude: from 0x7f80 on an infinity or a NaN. Very
  // large and very small rows are moved by a power of two, where the steps of
  // int8_code neither overflow nor lose bits.
  const bool bad = m >= 0x7f80u;
  const float a = bf16_to_float((uint16_t)m);
  const float move = a < 0x1p-60f ? 0x1p80f : (a > 0x1p60f ? 0x1p-80f : 1.0f);
  const float am = a * move, r = bad || m == 0 ? 0.0f : 1.0f / am;
  const float by = 127.0f * move;
  if (tid == 0) S[row] = bad ? __builtin_nanf("") : a / 127.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int k = (c * T + tid) * 8;
    if (k >= K) break;
    uint32_t q[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      q[2 * d] = int8_code(bf16_to_float((uint16_t)v[c][d]) * by, am, r);
      q[2 * d + 1] = int8_code(__builtin_bit_cast(float, v[c][d] & 0xffff0000u) * by, am, r);
    }
    u32x2 o;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const uint32_t lo = __builtin_amdgcn_perm(q[4 * d + 1], q[4 * d], 0x0c0c0400u);
      const uint32_t hi = __builtin_amdgcn_perm(q[4 * d + 3], q[4 * d + 2], 0x04000c0cu);
      o[d] = bad ? 0u : lo | hi;
    }
    *reinterpret_cast<u32x2*>(Q + (size_t)row * K + k) = o;
  }
}

// Any K: the row is read twice, by one workgroup.
__global__ __launch_bounds__(1024) void quantize_int8_long_kernel(const uint16_t* __restrict__ X,
                                                                  uint8_t* __restrict__ Q,
                                                                  float* __restrict__ S, int K) {
  __shared__ __attribute__((aligned(16))) uint32_t top[16];
  const int row = blockIdx.x;
  const uint16_t* x = X + (size_t)row * K;
  uint32_t m = 0;
  for (int k = threadIdx.x * 8; k < K; k += 8192) {
    const u32x4 v = load16(x + k);
#pragma unroll
    for (int d = 0; d < 4; ++d) m = max(m, max(v[d] & 0x7fffu, (v[d] >> 16) & 0x7fffu));
  }
  m = group_max<64>(m);
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 16; ++w) m = max(m, top[w]);
  const bool bad = m >= 0x7f80u;
  const float a = bf16_to_float((uint16_t)m);
  const float move = a < 0x1p-60f ? 0x1p80f : (a > 0x1p60f ? 0x1p-80f : 1.0f);
  const float am = a * move, r = bad || m == 0 ? 0.0f : 1.0f / am;
  const float by = 127.0f * move;
  if (threadIdx.x == 0) S[row] = bad ? __builtin_nanf("") : a / 127.0f;
  for (int k = threadIdx.x * 8; k < K; k += 8192) {
    const u32x4 v = load16(x + k);
    u32x2 o{0, 0};
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t lo = int8_code(bf16_to_float((uint16_t)v[d]) * by, am, r) & 0xffu;
      const uint32_t hi = int8_code(__builtin_bit_cast(float, v[d] & 0xffff0000u) * by, am, r) & 0xffu;
      o[d / 2] |= (lo | hi << 8) << (16 * (d & 1));
    }
    *reinterpret_cast<u32x2*>(Q + (size_t)row * K + k) = bad ? u32x2{0, 0} : o;
  }
}

// ============================================================================
// Weights into fragment order
// ============================================================================
// A thread copies one run of 16 bytes at a time; once per weight set.
__global__ __launch_bounds__(256) void pack_int8_kernel(const uint8_t* __restrict__ W8,
                                                        uint8_t* __restrict__ P, int rows, int K,
                                                        long long chunks) {
  const int G = (K + 127) / 128, B = (rows + 31) / 32;
  for (long long c = (long long)blockIdx.x * 256 + threadIdx.x; c < chunks;
       c += (long long)gridDim.x * 256) {
    const int i = (int)(c & 31), h = (int)(c >> 5 & 1), s = (int)(c >> 6 & 3);
    const long long bg = c >> 8;
    const int g = (int)(bg % G);
    const long long eb = bg / G;
    const int b = (int)(eb % B);
    const int row = 32 * b + i, k = 128 * g + 32 * s + 16 * h;
    const u32x4 v = row < rows && k < K
                        ? load16(W8 + ((size_t)(eb / B) * rows + row) * K + k)
                        : u32x4{0, 0, 0, 0};
    *reinterpret_cast<u32x4*>(P + (size_t)c * 16) = v;
  }
}

// ============================================================================
// Many rows: LDS-tiled
// ============================================================================
// A tile is BM rows of A against BNW weight rows, as D = W A^T on
// v_mfma_i32_32x32x32_i8.  K runs in the stored groups of 128 as two stages of 64
// k each, in a ring of two groups in LDS: 2 KB of every block of 32 weight rows, copied
// as they are (a fragment is one 16-byte read a lane at 16 x lane), and 64-byte
// pieces of the rows of A, whose 16-byte chunks are swizzled so that the lanes read
// together spread over the banks.
//
// One workgroup stays on a CU and walks over tiles, the ring running on from one
// to the next: a tile's last two groups already load the next one's first, and the
// output goes to memory straight from registers, so that LDS stays the ring's.  What the
// next tile needs beside that arrives by the same direct loads: its scales and, by
// expert, the slots of its rows, early in this tile, from which come the row
// addresses of its loads.  None of these loads is waited for by itself: the ring's own waits
// let the newest 2 LOADS of a wave be in flight, and more loads in between only make them
// reach further.
//
// From card to card 8192 x 18944 x 3584 gated takes 896 to 1024 us and 8192 x 3584 x 18944 plain 439
// to 471 (2.2 to 2.5 POP/s; a library product of 8192^3 reaches 2.05 here): 72 % of the cycles in the
// matrix pipes at 1.46 GHz and 65 % at 1.73, whatever clock power leaves (a card that takes 1013 and
// 471 us); no bank conflicts.  LDS moves all of
// its 128 bytes a clock while the pipes run (96 read, 32 written); four waves of 128 x 128
// each read a third less but leave one wave a SIMD: 958 against 913 us.  By expert, 32760
// rows on 32: 514 to 566 us (3584 x 4736) and 280 to 313 (2368 x 3584), where partial tiles, the
// stores (12 % of the plain one without them) and the last round weigh more.
template <int BM, int BNW, int WGM, int WGN>
struct Int8Tile {
  static constexpr int kWaves = WGM * WGN, kThreads = 64 * kWaves;
  static constexpr int NA = BM / 32, NW = BNW / 32;  // blocks of 32 of the tile
  static constexpr int FA = NA / WGM, FW = NW / WGN;  // and of a wave
  static_assert(FA >= 1 && FW >= 1 && FA * WGM == NA && FW * WGN == NW, "wave tile");
  static constexpr int A_BYTES = NA * 2048, STAGE = (NA + NW) * 2048, GROUP = 2 * STAGE;
  static constexpr int A_LOADS = 2 * NA / kWaves, W_LOADS = 2 * NW / kWaves;  // 1 KB loads of a wave
  static constexpr int LOADS = A_LOADS + W_LOADS;
  static_assert(2 * NA % kWaves == 0 && 2 * NW % kWaves == 0, "every wave loads as much");
  static_assert(2 * LOADS <= 63, "vmcnt range");
  // behind the ring, by parity of the tile: scales of its rows of A and of W, slots of its rows
  static constexpr int SA_OFF = 2 * GROUP, SW_OFF = SA_OFF + 8 * BM, ROW_OFF = SW_OFF + 8 * BNW;
  static constexpr int TABLE_OFF = ROW_OFF + 8 * BM;  // by expert
  static constexpr int lds_bytes(bool grouped) {
    return grouped ? TABLE_OFF + 12 * (int)kMaxExperts : ROW_OFF;
  }
  static_assert(lds_bytes(true) <= 160 * 1024, "LDS");
  static constexpr int kPerCu = lds_bytes(true) <= 80 * 1024 ? 2 : 1;
  // 64-byte rows: chunk c of row r is stored at c ^ swz(r)
  __host__ __device__ static constexpr int swz(int row) {
    return (((row >> 2) & 1) << 1) | (((row >> 1) ^ (row >> 3)) & 1);
  }
  // groups run for a tile: the last two load for the next one and neither is the first; by
  // expert the next tile's slots, asked for in the first, come before the loads that they address
  static constexpr int kMinGroups = 3, kMinGroupsGrouped = 4;
};

template <int OP, bool GROUPED, int BM, int BNW, int WGM, int WGN, int PARTS>
__global__ __launch_bounds__(64 * WGM * WGN) void int8_tile_kernel(Int8Args a, int ntn, int group_m) {
  using C = Int8Tile<BM, BNW, WGM, WGN>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::lds_bytes(GROUPED)];
  const int lane = threadIdx.x & 63;
  const int wave_u = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wm = wave_u / WGN, wn = wave_u % WGN;
  const int K = a.K, G = (K + 127) / 128;
  const int Gp = max(G, GROUPED ? C::kMinGroupsGrouped : C::kMinGroups);
  const int nblk = (a.C + 31) / 32;
  const uint32_t wbytes = (uint32_t)nblk * (uint32_t)G * 4096u;  // of one matrix

  // workgroup b runs on XCD b % 8; each XCD owns a contiguous range of tiles, which
  // its workgroups take in turn
  const int x = blockIdx.x % 8, nwg = gridDim.x;
  const int stride = nwg / 8 + (x < nwg % 8 ? 1 : 0);
  const GroupTable table{reinterpret_cast<int*>(smem + C::TABLE_OFF),
                         reinterpret_cast<int*>(smem + C::TABLE_OFF) + kMaxExperts,
                         reinterpret_cast<int*>(smem + C::TABLE_OFF) + 2 * kMaxExperts};
  int first, end;
  const int ntm = (a.R + BM - 1) / BM;
  if constexpr (GROUPED) {
    group_table<BM>(a.offsets, a.E, a.R, table);
    const GroupRange range = group_range<BM, PARTS>(a.offsets, a.E, a.R, ntn, x);
    first = range.begin;
    end = range.end;
    __syncthreads();
  } else {
    const int ntiles = ntm * ntn;
    first = x * (ntiles / 8) + min(x, ntiles % 8);
    end = first + ntiles / 8 + (x < ntiles % 8 ? 1 : 0);
  }
  first += (int)blockIdx.x / 8;
  if (first >= end) return;

  const i32x4 rsA = make_rsrc(a.A, (uint32_t)a.TA * (uint32_t)K);
  const i32x4 rsSA = make_rsrc(a.SA, K > 0 ? (uint32_t)a.TA * 4u : 0u);
  const uint32_t lds0 = lds_addr(smem);

  // A tile: rows [pos0, pos0 + rows) against weight rows from tn BNW on; none past the
  // last one.
  struct Tile {
    int expert, pos0, rows, tn;
  };
  auto uniform = [](int v) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane(v); };
  auto locate = [&](int t, int from) __attribute__((always_inline)) {
    Tile o{from, 0, 0, 0};
    if (t < end) {
      int local = t, row0 = 0, n = a.R, high_all = ntm;
      int band_rows = group_m;
      if constexpr (GROUPED) {
        o.expert = uniform(group_find(table, a.E, t / ntn, from));
        row0 = uniform(table.lo[o.expert]);
        n = uniform(table.n[o.expert]);
        high_all = (n + BM - 1) / BM;
        local = t - uniform(table.upto[o.expert] - high_all) * ntn;
      }
      // bands of tile rows, column after column
      const int band = local / (band_rows * ntn), in = local % (band_rows * ntn);
      const int high = min(high_all - band * band_rows, band_rows);
      const int tm = band * band_rows + in % high;
      o.tn = uniform(in / high);
      o.pos0 = uniform(row0 + tm * BM);
      o.rows = uniform(min(n - tm * BM, BM));
    }
    return o;
  };

  // ---- loads --------------------------------------------------------------------------
  // Load q of a wave is 1 KB of a stage, A's before W's: 16 rows of A, or half a stage of one
  // block of 32 weight rows.  What lies past a tensor comes as zeros; k past K is
  // zero in W, whatever A has there.
  const int a_row = lane >> 2;  // of the load's 16
  uint32_t off[C::LOADS], a_next[C::A_LOADS];
  auto a_chunk = [&](int row) __attribute__((always_inline)) {
    return (uint32_t)(((lane & 3) ^ C::swz(row)) * 16);
  };
  // offset of the lane's row of A in load q, by the tile's slots
  auto a_offset = [&](const Tile& o, int par, int q) __attribute__((always_inline)) {
    const int r = (q * C::kWaves + wave_u) * 16 + a_row;
    int row = r < o.rows ? o.pos0 + r : -1;
    if constexpr (GROUPED && OP == I8_GATED) {
      const int slot = reinterpret_cast<const int*>(smem + C::ROW_OFF + par * 4 * BM)[r];
      row = r < o.rows && slot >= 0 && slot / a.k < a.TA ? slot / a.k : -1;
    }
    return row >= 0 ? (uint32_t)row * (uint32_t)K + a_chunk(r) : kOutOfRange;
  };
#pragma unroll
  for (int q = C::A_LOADS; q < C::LOADS; ++q) {
    const int c = (q - C::A_LOADS) * C::kWaves + wave_u;
    off[q] = (uint32_t)(c >> 1) * (uint32_t)G * 4096u + (uint32_t)(c & 1) * 1024u + (uint32_t)lane * 16u;
  }
  auto weights = [&](const Tile& o) __attribute__((always_inline)) {
    return make_rsrc(a.W + (size_t)o.expert * wbytes, wbytes);
  };
  // load q of stage HALF of group g of a tile into ring slot `slot`
  auto dma = [&](const Tile& o, const i32x4& rsW, const uint32_t* rows, int g, int slot, int half,
                 int q) __attribute__((always_inline)) {
    const bool in = g < G && o.rows > 0;
    const uint32_t base = lds0 + slot * C::GROUP + half * C::STAGE;
    if (q < C::A_LOADS) {
      lds_dma16_wait(base + (q * C::kWaves + wave_u) * 1024,
                in ? rows[q] + (uint32_t)(g * 128 + half * 64) : kOutOfRange, rsA);
    } else {
      const uint32_t at = (uint32_t)(o.tn * C::NW) * (uint32_t)G * 4096u + (uint32_t)g * 4096u +
                          (uint32_t)half * 2048u;
      lds_dma16_wait(base + C::A_BYTES + ((q - C::A_LOADS) * C::kWaves + wave_u) * 1024,
                off[q] + (in ? at : kOutOfRange), rsW);
    }
  };
  // the slots of a tile's rows, 64 a load
  auto load_slots = [&](const Tile& o, int par) __attribute__((always_inline)) {
    if constexpr (GROUPED) {
      const i32x4 rs = make_rsrc(a.rows + o.pos0, (uint32_t)o.rows * 4u);
#pragma unroll
      for (int c0 = 0; c0 < BM / 64; c0 += C::kWaves) {
        const int c = c0 + wave_u;
        if (c < BM / 64) lds_dma4_wait(lds0 + C::ROW_OFF + par * 4 * BM + c * 256, (uint32_t)(c * 64 + lane) * 4u, rs);
      }
    }
  };
  // its scales, 64 a load
  auto load_scales = [&](const Tile& o, int par) __attribute__((always_inline)) {
    const i32x4 rsSW = make_rsrc(a.SW + (size_t)o.expert * a.C, K > 0 ? (uint32_t)a.C * 4u : 0u);
#pragma unroll
    for (int c0 = 0; c0 < (BM + BNW) / 64; c0 += C::kWaves) {
      const int c = c0 + wave_u;
      if (c < BM / 64) {
        const int r = c * 64 + lane;
        int row = r < o.rows ? o.pos0 + r : -1;
        if constexpr (GROUPED && OP == I8_GATED) {
          const int slot = reinterpret_cast<const int*>(smem + C::ROW_OFF + par * 4 * BM)[r];
          row = r < o.rows && slot >= 0 && slot / a.k < a.TA ? slot / a.k : -1;
        }
        lds_dma4_wait(lds0 + C::SA_OFF + par * 4 * BM + c * 256, row >= 0 ? (uint32_t)row * 4u : kOutOfRange, rsSA);
      } else if (c < (BM + BNW) / 64) {
        const int r = (c - BM / 64) * 64;
        lds_dma4_wait(lds0 + C::SW_OFF + par * 4 * BNW + r * 4, (uint32_t)(o.tn * BNW + r + lane) * 4u, rsSW);
      }
    }
  };

  // ---- fragments ------------------------------------------------------------------------
  // A wave's blocks of rows are those j WGM + wm, so a short tile leaves every wave about as many.
  u32x4 af[2][C::FA], wf[2][C::FW];
  const int fr = lane & 31, fh = lane >> 5;
  uint32_t fa = (uint32_t)(wm * 2048 + fr * 64), fw = (uint32_t)(C::A_BYTES + wn * C::FW * 2048 + lane * 16);
  const uint32_t fc[2] = {(uint32_t)((fh ^ C::swz(fr)) * 16), (uint32_t)(((2 + fh) ^ C::swz(fr)) * 16)};
  auto frag = [&](uint32_t ba, uint32_t bw, int half, int sub, int r) __attribute__((always_inline)) {
    const int at = half * C::STAGE;
    if (r < C::FW)
      wf[sub][r] = *reinterpret_cast<const u32x4*>(smem + bw + (at + r * 2048 + sub * 1024));
    else
      af[sub][r - C::FW] =
          *reinterpret_cast<const u32x4*>(smem + (ba + fc[sub]) + (at + (r - C::FW) * WGM * 2048));
  };
  i32x16 acc[C::FW][C::FA];

  Tile cur = locate(first, 0), nxt = cur;
  i32x4 w_cur = weights(cur), w_nxt = w_cur;
  int par = 0;

  // Sub-step B (32 k) of a group.  The even ones read the other sub-step of their stage;
  // the odd ones wait for the next stage, and behind the barrier (every wave has read this stage)
  // read the next one's first fragments and load the stage of the group after next in this one's
  // place.  LIVE: the wave's blocks of rows that the tile has; KIND: the tile's first group, whose
  // first sums start from zero, one in between, and the last two.
  constexpr int kFirst = 0, kMiddle = 1, kBeforeLast = 2, kLast = 3;
  auto step = [&](auto b_c, auto live_c, auto kind_c, const Tile& o, const i32x4& rsW,
                  const uint32_t* rows, int lg, int slot) __attribute__((always_inline)) {
    constexpr int B = decltype(b_c)::value, SUB = B & 1, HALF = B >> 1, LIVE = decltype(live_c)::value;
    constexpr int KIND = decltype(kind_c)::value;
    constexpr bool LAST = KIND == kLast && B == 3;  // the next stage is the next tile's
    constexpr int NMF = C::FW * LIVE, NFRAG = C::FW + (LAST ? C::FA : LIVE);
    if constexpr (SUB == 1) {
      wait_vmcnt<2 * C::LOADS>();
      __syncthreads();
      if constexpr (B == 1) {
        if (GROUPED && KIND == kFirst && nxt.rows > 0) load_slots(nxt, par ^ 1);
        if (KIND == kBeforeLast && nxt.rows > 0) load_scales(nxt, par ^ 1);
      }
    }
    const int turn = HALF == 1 && SUB == 1 ? (slot ? -C::GROUP : C::GROUP) : 0;
    const uint32_t na = fa + turn, nw = fw + turn;
    auto one = [&](auto q_c) __attribute__((always_inline)) {
      constexpr int Q = decltype(q_c)::value, i = Q / LIVE, j = Q % LIVE;
      acc[i][j] = mfma32_i8(wf[SUB][i], af[SUB][j], KIND == kFirst && B == 0 ? i32x16{} : acc[i][j]);
#pragma unroll
      for (int r = Q * NFRAG / NMF; r < (Q + 1) * NFRAG / NMF; ++r)
        frag(na, nw, SUB == 0 ? HALF : HALF ^ 1, SUB ^ 1, r);
      if constexpr (SUB == 1) {
#pragma unroll
        for (int q = Q * C::LOADS / NMF; q < (Q + 1) * C::LOADS / NMF; ++q)
          dma(o, rsW, rows, lg, slot, HALF, q);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    [&]<int... Q>(std::integer_sequence<int, Q...>) __attribute__((always_inline)) {
      (one(std::integral_constant<int, Q>{}), ...);
    }(std::make_integer_sequence<int, NMF>{});
  };

  // ---- the first tile's slots and scales, its first two groups, the first fragments ------
  if constexpr (GROUPED) {
    load_slots(cur, 0);
    wait_vmcnt<0>();
    __syncthreads();
  }
  load_scales(cur, 0);
#pragma unroll
  for (int q = 0; q < C::A_LOADS; ++q) off[q] = a_offset(cur, 0, q);
#pragma unroll
  for (int st = 0; st < 4; ++st)
#pragma unroll
    for (int q = 0; q < C::LOADS; ++q) dma(cur, w_cur, off, st / 2, st / 2, st % 2, q);
  wait_vmcnt<3 * C::LOADS>();
  __syncthreads();
#pragma unroll
  for (int r = 0; r < C::FW + C::FA; ++r) frag(fa, fw, 0, 0, r);

  int slot = 0;
  for (int t = first; t < end; t += stride) {
    nxt = locate(t + stride, cur.expert);
    w_nxt = GROUPED ? weights(nxt) : w_cur;
    const int blocks = (cur.rows + 31) / 32;
    const int live = (blocks - wm + WGM - 1) / WGM;
    auto tile = [&](auto live_c) __attribute__((always_inline)) {
      constexpr int LIVE = decltype(live_c)::value;
      auto group = [&](auto kind_c, const Tile& o, const i32x4& rsW, const uint32_t* rows,
                       int lg) __attribute__((always_inline)) {
        step(std::integral_constant<int, 0>{}, live_c, kind_c, o, rsW, rows, lg, slot);
        step(std::integral_constant<int, 1>{}, live_c, kind_c, o, rsW, rows, lg, slot);
        step(std::integral_constant<int, 2>{}, live_c, kind_c, o, rsW, rows, lg, slot);
        step(std::integral_constant<int, 3>{}, live_c, kind_c, o, rsW, rows, lg, slot);
        const int turn = slot ? -C::GROUP : C::GROUP;
        fa += turn;
        fw += turn;
        slot ^= 1;
      };
      group(std::integral_constant<int, kFirst>{}, cur, w_cur, off, 2);
      for (int g = 1; g < Gp - 2; ++g) group(std::integral_constant<int, kMiddle>{}, cur, w_cur, off, g + 2);
      // the groups to load are the next tile's
#pragma unroll
      for (int q = 0; q < C::A_LOADS; ++q) a_next[q] = a_offset(nxt, par ^ 1, q);
      group(std::integral_constant<int, kBeforeLast>{}, nxt, w_nxt, a_next, 0);
      group(std::integral_constant<int, kLast>{}, nxt, w_nxt, a_next, 1);
      // Scales, SiLU(Gate) Up, stores, for each LIVE by itself (joined before, the sums would be
      // moved).  Registers 4 q .. 4 q + 3 are weight rows 8 q + 4 h + 0 .. 3 (h = lane / 32); the
      // exchanges give a lane 8 output columns next to each other.
      const float* sa = reinterpret_cast<const float*>(smem + C::SA_OFF + par * 4 * BM);
      const uint8_t* sw = smem + C::SW_OFF + par * 4 * BNW;
      const int* slots = reinterpret_cast<const int*>(smem + C::ROW_OFF + par * 4 * BM);
#pragma unroll
      for (int j = 0; j < LIVE; ++j) {
        const int r = (j * WGM + wm) * 32 + fr;
        const float s = sa[r];
        int row = cur.pos0 + r;
        if constexpr (GROUPED && OP == I8_PLAIN) row = slots[r];
        const bool there = r < cur.rows && row >= 0 && row < a.R;
        uint16_t* y = a.Y + (size_t)(there ? row : 0) * a.N;
#pragma unroll
        for (int i = 0; i < C::FW; ++i) {
          const i32x16& d = acc[i][j];
          float p[16];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 c = *reinterpret_cast<const f32x4*>(sw + ((wn * C::FW + i) * 32 + 8 * q + 4 * fh) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) p[4 * q + e] = (float)d[4 * q + e] * s * c[e];
          }
          if constexpr (OP == I8_GATED) {
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              o[q] = two_bf16(silu(p[4 * q]) * p[4 * q + 1], silu(p[4 * q + 2]) * p[4 * q + 3]);
            swap_halves(o[0], o[2]);
            swap_halves(o[1], o[3]);
            const int col = (cur.tn * C::NW + wn * C::FW + i) * 16 + 8 * fh;
            if (there && col < a.N) *reinterpret_cast<u32x4*>(y + col) = u32x4{o[0], o[2], o[1], o[3]};
          } else {
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = two_bf16(p[4 * q + 2 * e], p[4 * q + 2 * e + 1]);
              swap_halves(o[0], o[2]);
              swap_halves(o[1], o[3]);
              const int col = (cur.tn * C::NW + wn * C::FW + i) * 32 + 8 * (q + fh);
              if (there && col < a.N) *reinterpret_cast<u32x4*>(y + col) = u32x4{o[0], o[1], o[2], o[3]};
            }
          }
        }
      }
    };
    if (C::FA >= 4 && live >= 4) {
      if constexpr (C::FA >= 4) tile(std::integral_constant<int, 4>{});
    } else if (C::FA >= 3 && live >= 3) {
      if constexpr (C::FA >= 3) tile(std::integral_constant<int, 3>{});
    } else if (C::FA >= 2 && live >= 2) {
      if constexpr (C::FA >= 2) tile(std::integral_constant<int, 2>{});
    } else {
      tile(std::integral_constant<int, 1>{});  // also a wave without rows: it loads and waits with the others
    }
    cur = nxt;
    w_cur = w_nxt;
#pragma unroll
    for (int q = 0; q < C::A_LOADS; ++q) off[q] = a_next[q];
    par ^= 1;
  }
  // the zero loads issued past the last tile still write LDS
  wait_vmcnt<0>();
}

// ============================================================================
// Few rows: weight streaming
// ============================================================================
// A workgroup takes NB half blocks of 16 weight rows and MT times 16 rows of A, as D = W A^T on
// v_mfma_i32_16x16x64_i8 (a Gate / Up pair is two adjacent registers of a lane; rows of
// A come in 64-byte pieces).  Its NW waves take every NW-th group of 128 k, D groups in
// flight while one is multiplied.  The waves' sums are added in LDS: integers, so their order
// does not matter.  16 x 18944 x 3584 gated in 23.7 us (5.8 TB/s), 32 rows on 64 experts, 1536 x
// 3584, in 28.4 (6.2); 16 x 3584 x 18944 plain in 17.0 (4.0) among others of its kind and 18 to 20 by
// itself in a trace, where the 224 pieces each take in as many bytes of A as of W.  (32x32x32 instructions, whose 32 rows of A come in 32-byte pieces: 26.6,
// 36.3 and 28.4.)
template <int OP, bool GROUPED, int MT, int NB, int NW, int D>
__global__ __launch_bounds__(64 * NW) void int8_stream_kernel(Int8Args g, int nblk) {
  constexpr int BM = 16 * MT;
  __shared__ __attribute__((aligned(16))) i32x4 red[NW > 1 ? NW * MT * NB * 64 : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, quarter = lane >> 4;
  const int K = g.K, G = (K + 127) / 128, B = (g.C + 31) / 32;
  int blk, pos0, nrows, expert = 0;
  if constexpr (GROUPED) {
    const GroupRange range = group_range<BM, 1>(g.offsets, g.E, g.R, nblk, blockIdx.x % 8);
    const int t = range.begin + (int)blockIdx.x / 8;
    if (t >= range.end) return;
    const GroupUnit u = group_unit<BM>(g.offsets, g.E, g.R, nblk, t);
    blk = u.local % nblk;
    pos0 = u.first + u.local / nblk * BM;
    nrows = min(u.first + u.rows - pos0, BM);
    expert = u.expert;
  } else {
    blk = xcd_remap(blockIdx.x, gridDim.x);
    pos0 = blockIdx.y * BM;
    nrows = min(g.R - pos0, BM);
  }
  const uint8_t* wp[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {  // a half block past the last repeats it; never stored
    const int half = min(blk * NB + b, 2 * B - 1);
    wp[b] = g.W + ((size_t)expert * B + (half >> 1)) * G * 4096 +
            ((quarter >> 1) * 1024 + (quarter & 1) * 512 + (half & 1) * 256 + l16 * 16);
  }
  // rows past the span repeat the last one and are never stored
  const uint8_t* ap[MT];
  int ar[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int pos = pos0 + min(16 * j + l16, nrows - 1);
    ar[j] = GROUPED ? int8_a_row<OP>(g, pos) : pos;
    ap[j] = g.A + (size_t)max(ar[j], 0) * K + 16 * quarter;
  }
  i32x4 acc[MT][NB];
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[j][b] = i32x4{0, 0, 0, 0};

  u32x4 w[D + 1][NB][2], a[D + 1][MT][2];
  auto load = [&](auto p_c, int gi) __attribute__((always_inline)) {
    constexpr int P = decltype(p_c)::value;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int s = 0; s < 2; ++s) w[P][b][s] = load16_stream(wp[b] + (size_t)gi * 4096 + s * 2048);
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int k = gi * 128 + s * 64;
        a[P][j][s] = k + 16 * quarter < K && ar[j] >= 0 ? load16(ap[j] + k) : u32x4{0, 0, 0, 0};
      }
  };
  // round P of D + 1: this wave's group gi, and the load of the one D rounds on in the
  // registers that the round before has used
  auto round = [&](auto p_c, int gi) __attribute__((always_inline)) {
    constexpr int P = decltype(p_c)::value;
    if (gi >= G) return;
    if (gi + D * NW < G) load(std::integral_constant<int, (P + D) % (D + 1)>{}, gi + D * NW);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[j][b] = mfma16_i8(w[P][b][s], a[P][j][s], acc[j][b]);
  };
  [&]<int... P>(std::integer_sequence<int, P...>) __attribute__((always_inline)) {
    ((wave + P * NW < G ? (load(std::integral_constant<int, P>{}, wave + P * NW), 0) : 0), ...);
  }(std::make_integer_sequence<int, D>{});
  for (int gi = wave; gi < G; gi += (D + 1) * NW)
    [&]<int... P>(std::integer_sequence<int, P...>) __attribute__((always_inline)) {
      (round(std::integral_constant<int, P>{}, gi + P * NW), ...);
    }(std::make_integer_sequence<int, D + 1>{});

  // register r: weight row 16 half + 4 quarter + r of A's row lane % 16
  auto store = [&](int j, int b, const i32x4& v) __attribute__((always_inline)) {
    const int row = 16 * j + l16, c = (blk * NB + b) * 16 + 4 * quarter;
    if (row >= nrows || c >= g.C) return;
    const float sa = K > 0 && ar[j] >= 0 ? g.SA[ar[j]] : 0.0f;
    f32x4 sw{0, 0, 0, 0};
    if (K > 0) sw = __builtin_bit_cast(f32x4, load16(g.SW + (size_t)expert * g.C + c));
    float p[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) p[x] = (float)v[x] * sa * sw[x];
    const int out = GROUPED && OP == I8_PLAIN ? g.rows[pos0 + row] : pos0 + row;
    if (out < 0 || out >= g.R) return;
    uint16_t* y = g.Y + (size_t)out * g.N;
    if constexpr (OP == I8_GATED)
      *reinterpret_cast<uint32_t*>(y + c / 2) = two_bf16(silu(p[0]) * p[1], silu(p[2]) * p[3]);
    else
      *reinterpret_cast<u32x2*>(y + c) = u32x2{two_bf16(p[0], p[1]), two_bf16(p[2], p[3])};
  };
  if constexpr (NW == 1) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b) store(j, b, acc[j][b]);
  } else {
    constexpr int NQ = MT * NB;
#pragma unroll
    for (int x = 0; x < NQ; ++x) red[(wave * NQ + x) * 64 + lane] = acc[x / NB][x % NB];
    __syncthreads();
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
      if (x % NW != wave) continue;
      i32x4 v = red[x * 64 + lane];
#pragma unroll
      for (int o = 1; o < NW; ++o) v += red[(o * NQ + x) * 64 + lane];
      store(x / NB, x % NB, v);
    }
  }
}

// ============================================================================
// Launches
// ============================================================================
// At most this many tiles of bm rows, whatever the spans: one partial tile for
// each expert that has rows.
static long long int8_row_tiles(const Int8Call& c, long long bm) {
  if (!c.grouped) return (c.R + bm - 1) / bm;
  const long long some = std::min(c.R, c.E);
  return std::min(c.R, (c.R + some * (bm - 1)) / bm);
}
template <int OP, bool GROUPED, int MT, int NB, int NW, int D>
static hipError_t launch_int8_stream(const Int8Call& c, const Int8Args& g, hipStream_t stream) {
  const long long nblk = (c.C() + 16 * NB - 1) / (16 * NB), tiles = int8_row_tiles(c, 16 * MT);
  // all units weigh the same, so no XCD has more than an eighth of them, rounded up
  const long long x = GROUPED ? (tiles * nblk + 7) / 8 * 8 : nblk, y = GROUPED ? 1 : tiles;
  if (x > 0x7fffffffLL || y > 65535) return hipErrorInvalidValue;
  return launch_op(int8_stream_kernel<OP, GROUPED, MT, NB, NW, D>, dim3((unsigned)x, (unsigned)y),
                   dim3(64 * NW), stream, g, (int)nblk);
}

template <int BM, int BNW, int WGM, int WGN>
static long long int8_tile_grid(const Int8Call& c) {
  using T = Int8Tile<BM, BNW, WGM, WGN>;
  const long long tiles = int8_row_tiles(c, BM) * ((c.C() + BNW - 1) / BNW);
  // eight at least: each XCD's range of tiles needs a workgroup there.  By expert an eighth of
  // the work may be more than an eighth of the tiles, hence all that the device holds.
  const long long most = std::max<long long>((long long)c.cu_count * T::kPerCu, 8);
  return std::min(c.grouped ? (2 * tiles + 7) / 8 * 8 : tiles, most);
}
template <int OP, bool GROUPED, int BM, int BNW, int WGM, int WGN, int PARTS>
static hipError_t launch_int8_tile(const Int8Call& c, const Int8Args& g, hipStream_t stream) {
  const long long ntn = (c.C() + BNW - 1) / BNW;
  const int group_m = GROUPED ? 8 : 4;
  return launch_op(int8_tile_kernel<OP, GROUPED, BM, BNW, WGM, WGN, PARTS>,
                   dim3((unsigned)int8_tile_grid<BM, BNW, WGM, WGN>(c)), dim3(64 * WGM * WGN), stream,
                   g, (int)ntn, group_m);
}

// The kernel variants: rows of A and weight rows of a workgroup's piece, workgroups a CU of
// the tiled ones (0: streaming), and what the choice between them goes by: microseconds of a
// launch and of a piece beside its loads, bytes a microsecond that a CU takes in with this
// kernel (both operands, from HBM or an L2) and that all of them take of the weights.
// Fitted to 90 calls of 1 to 21264 rows, dense and on 4 to 96 experts (each timed in
// every variant): the choice is 1.6 % off the fastest in the mean, 30 % once (223 rows on 8
// experts, 1200 x 1712: 10.5 us for the 64 x 128 tile, 8.1 streaming), 19 % at 764 x 728 x 6736
// (26.7 and 22.4) and 14 to 20 % at 64 x 18944 x 3584 gated (38.9 to 41.1 us for the 64 x 128 tile,
// 34.1 for the 128 x 256 one).
struct Int8Plan {
  int bm, bn, per_cu;
  double launch, piece, cu_rate, weight_rate;
};
constexpr Int8Plan kInt8Plans[kInt8Variants] = {
    {16, 16, 0, 3.8, 1.1, 47700, 6.6e6},  {16, 32, 0, 3.4, 0.9, 47800, 6.4e6},
    {32, 32, 0, 3.3, 0.8, 36800, 4.8e6},  {64, 64, 0, 3.3, 0.2, 31700, 3.2e6},
    {64, 128, 2, 3.1, 0.4, 59000, 4.6e6}, {128, 128, 2, 4.0, 0.1, 55100, 3.9e6},
    {128, 256, 1, 2.7, 0.3, 44900, 3.9e6}, {256, 256, 1, 2.1, 1.8, 38500, 5.9e6},
};
// Rows of an expert that has any, in the mean (the counts are on the device), and the pieces.
static long long int8_mean(const Int8Call& c, long long* some) {
  *some = c.grouped ? std::min(c.R, c.E) : 1;
  return (c.R + *some - 1) / *some;
}
static long long int8_pieces(const Int8Call& c, const Int8Plan& p) {
  long long some;
  const long long mean = int8_mean(c, &some);
  return some * ((mean + p.bm - 1) / p.bm) * ((c.C() + p.bn - 1) / p.bn);
}
// Waves along K of a streaming workgroup: enough of them for the device (8, 4 and 2 waves at
// 16 x 18944 x 3584 plain: 16.8, 20.1, 32.8 us; 32 rows on 64 experts, 3584 x 1536 gated: 45.3,
// 30.4, 29.2).
static int int8_waves(const Int8Call& c, const Int8Plan& p) {
  const long long n = int8_pieces(c, p);
  return n >= 1024 ? 2 : (n >= 256 ? 4 : 8);
}
static double int8_cost(const Int8Call& c, const Int8Plan& p) {
  long long some;
  const long long mean = int8_mean(c, &some), tall = (mean + p.bm - 1) / p.bm;
  const double cus = std::max(c.cu_count, 1);
  long long rows = (mean + tall - 1) / tall, groups = (c.K + 127) / 128;
  const double n = (double)int8_pieces(c, p);
  double t;
  if (p.per_cu == 0) {
    t = std::max(n / cus, 1.0) * (double)((rows + p.bn) * groups * 128) / p.cu_rate + p.piece;
  } else {
    rows = (rows + 31) / 32 * 32;
    groups = std::max(groups, c.grouped ? 4LL : 3LL);
    const double rounds = std::ceil(n / (cus * p.per_cu));
    const double here = std::min<double>(p.per_cu, std::ceil(n / (cus * rounds)));
    t = rounds * ((double)((rows + p.bn) * groups * 128) * here / p.cu_rate + p.piece);
  }
  return p.launch + std::max(t, (double)(some * c.C()) * (double)c.K / p.weight_rate);
}
// Threads of a launch along x, and its workgroups along y; the tiled ones' grids are small, but
// their tile numbers are 32 bits wide.
static bool int8_fits(const Int8Call& c, int variant) {
  const Int8Plan& p = kInt8Plans[variant];
  const __int128 pieces = (__int128)int8_row_tiles(c, p.bm) * ((c.C() + p.bn - 1) / p.bn);
  if (p.per_cu) return pieces <= 0x7fffffffLL - 4096;
  if (!c.grouped && int8_row_tiles(c, p.bm) > 65535) return false;
  return (c.grouped ? pieces + 7 : (__int128)((c.C() + p.bn - 1) / p.bn)) * 512 < ((__int128)1 << 32);
}
static int int8_variant(const Int8Call& c) {
  int best = kInt8Variants - 1;
  double least = 0;
  for (int v = kInt8Variants - 1; v >= 0; --v) {
    if (!int8_fits(c, v)) continue;
    const double t = int8_cost(c, kInt8Plans[v]);
    if (least == 0 || t < least) best = v, least = t;
  }
  return best;
}
bool int8_launchable(const Int8Call& c, int variant) {
  return int8_fits(c, variant < 0 ? int8_variant(c) : variant);
}

template <int OP, bool GROUPED, int MT, int NB>
static hipError_t launch_int8_waves(const Int8Call& c, const Int8Args& g, const Int8Plan& p,
                                    hipStream_t stream) {
  switch (int8_waves(c, p)) {
    case 2: return launch_int8_stream<OP, GROUPED, MT, NB, 2, 2>(c, g, stream);
    case 4: return launch_int8_stream<OP, GROUPED, MT, NB, 4, 2>(c, g, stream);
    default: return launch_int8_stream<OP, GROUPED, MT, NB, 8, 2>(c, g, stream);
  }
}
template <int OP, bool GROUPED>
static hipError_t launch_int8_as(const Int8Call& c, int variant, hipStream_t stream) {
  const Int8Args g{c.A,        c.SA,     c.rows,   c.offsets, c.W,      c.SW,     c.Y,       (int)c.TA,
                   (int)c.R,   (int)c.N, (int)c.K, (int)c.E,  (int)c.k, (int)c.C()};
  const Int8Plan& p = kInt8Plans[variant];
  switch (variant) {
    case 0: return launch_int8_waves<OP, GROUPED, 1, 1>(c, g, p, stream);
    case 1: return launch_int8_waves<OP, GROUPED, 1, 2>(c, g, p, stream);
    case 2: return launch_int8_waves<OP, GROUPED, 2, 2>(c, g, p, stream);
    case 3: return launch_int8_stream<OP, GROUPED, 4, 4, 8, 1>(c, g, stream);
    case 4: return launch_int8_tile<OP, GROUPED, 64, 128, 2, 2, 1>(c, g, stream);
    case 5: return launch_int8_tile<OP, GROUPED, 128, 128, 2, 2, 2>(c, g, stream);
    case 6: return launch_int8_tile<OP, GROUPED, 128, 256, 2, 4, 2>(c, g, stream);
    default: return launch_int8_tile<OP, GROUPED, 256, 256, 2, 4, 4>(c, g, stream);
  }
}

hipError_t launch_int8(const Int8Call& c, int variant, hipStream_t stream) {
  if (variant < 0) variant = int8_variant(c);
  if (c.grouped)
    return c.gated ? launch_int8_as<I8_GATED, true>(c, variant, stream)
                   : launch_int8_as<I8_PLAIN, true>(c, variant, stream);
  return c.gated ? launch_int8_as<I8_GATED, false>(c, variant, stream)
                 : launch_int8_as<I8_PLAIN, false>(c, variant, stream);
}

// Waves of a row.
static int quantize_waves(long long K) {
  return K <= 1024 ? 1 : K <= 8192 ? 4 : K <= 16384 ? 8 : 16;
}
long long int8_quantize_threads(long long rows, long long K) {
  return quantize_waves(K) == 1 ? (rows + 3) / 4 * 256 : rows * 64 * quantize_waves(K);
}

template <int W, int CH>
static hipError_t launch_quantize_as(const uint16_t* X, uint8_t* Q, float* S, int rows, int K,
                                     hipStream_t stream) {
  constexpr int threads = 64 * (W < 4 ? 4 : W), per = threads / (64 * W);
  return launch_op(quantize_int8_kernel<W, CH>, dim3((unsigned)((rows + per - 1) / per)),
                   dim3(threads), stream, X, Q, S, rows, K);
}
hipError_t launch_quantize_int8(const uint16_t* X, uint8_t* Q, float* S, int rows, int K,
                                hipStream_t stream) {
  if (K <= 512) return launch_quantize_as<1, 1>(X, Q, S, rows, K, stream);
  if (K <= 1024) return launch_quantize_as<1, 2>(X, Q, S, rows, K, stream);
  if (K <= 2048) return launch_quantize_as<4, 1>(X, Q, S, rows, K, stream);
  if (K <= 4096) return launch_quantize_as<4, 2>(X, Q, S, rows, K, stream);
  if (K <= 8192) return launch_quantize_as<4, 4>(X, Q, S, rows, K, stream);
  if (K <= 16384) return launch_quantize_as<8, 4>(X, Q, S, rows, K, stream);
  if (K <= 32768) return launch_quantize_as<16, 4>(X, Q, S, rows, K, stream);
  return launch_op(quantize_int8_long_kernel, dim3((unsigned)rows), dim3(1024), stream, X, Q, S, K);
}

hipError_t launch_pack_int8(const uint8_t* W8, uint8_t* P, long long E, int rows, int K,
                            hipStream_t stream) {
  const long long chunks = E * int8_packed_bytes(rows, K) / 16;
  const long long blocks = std::min<long long>((chunks + 255) / 256, 1 << 16);
  return launch_op(pack_int8_kernel, dim3((unsigned)blocks), dim3(256), stream, W8, P, rows, K,
                   chunks);
}

}  // namespace swiglu
