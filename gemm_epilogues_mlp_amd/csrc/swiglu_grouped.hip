// swiglu_grouped.hip -- products grouped by expert for a mixture-of-experts MLP.
//
// The router sorts the T k (token, choice) slots by expert: sorted row i, in
// expert e's span [offsets[e], offsets[e + 1]), is slot rows[i] of token
// rows[i] / k.  With W_e the weights of expert e:
//   up    Y[i]       = SiLU(a G_e) (.) (a U_e),  a = A[rows[i] / k]
//                      (G_e, U_e the even and odd columns of W_e [K, 2N])
//   down  Y[rows[i]] = A[i] W_e                  (W_e [K, N])
// bf16 in, fp32 accumulation, one rounding to bf16 at the end.  The gather of
// A and the scatter of Y happen inside the products (the loads take per-lane
// row addresses, the stores per-row ones), so neither tensor is copied.
//
// Two kernels.  grouped_stream_kernel, for few rows an expert: the weights
// bound it (2 bytes a weight, 2 operations a row), so it reads them once,
// straight into registers, and does whatever rows there are on the side.
// grouped_tile_kernel, for many: LDS tiles fed by direct loads, bound by the
// matrix instructions.
#include "swiglu_internal.h"
#include "swiglu_ops_device.hpp"

#include <algorithm>
#include <type_traits>
#include <utility>

namespace swiglu {

enum GroupOp { GROUP_UP = 0, GROUP_DOWN = 1 };

// The tensors of a grouped product, as both kernels take them.
struct GroupArgs {
  const uint16_t* A;        // up: [TA, K], gathered; down: [R, K], sorted
  const int32_t* rows;      // [R] slot of each sorted row
  const int32_t* offsets;   // [E + 1]
  const uint16_t* W;        // [E, K, ldw]
  uint16_t* Y;              // [R, N]
  int TA, R, N, K, E, k;    // TA: rows of A
  int ldw;                  // 2N (up) or N (down)
};

// Row of A of sorted row `pos`, -1 if the slot names no row of A.
template <int OP>
__device__ __forceinline__ int group_a_row(const GroupArgs& g, int pos) {
  if (OP == GROUP_DOWN) return pos;
  const int slot = g.rows[pos];
  return slot >= 0 && slot / g.k < g.TA ? slot / g.k : -1;
}

// ============================================================================
// Many rows an expert: LDS-tiled
// ============================================================================
// One workgroup computes BM sorted rows of one expert against BNW of its weight
// columns, as D^T = W^T A^T on v_mfma_f32_32x32x16_bf16 (so that a Gate / Up
// pair is two adjacent registers of a lane).  K steps of BK = 32 go from HBM
// straight into a ring of STAGES LDS buffers, STAGES - 1 steps ahead of the
// matrix instructions, with one barrier a step; weight fragments are read with
// the transposing LDS read, activation fragments with 16-byte reads, both from
// XOR-swizzled chunks that spread the lanes served together over the banks (3 to
// 4 % of the LDS-active cycles still conflict, by the counters).
// With KG = 2 a step is 64 k, 32 of them for each of two groups of waves, whose
// sums are added in LDS at the end: twice the waves for a small tile.
// Rows past the span, columns past the matrix and k past K arrive as zeros (a
// buffer load past the resource returns 0).  32760 rows, 32 experts: 3584 x 4736 in
// 997 to 1160 us from card to card (0.96 to 1.12 PFLOP/s), bound by the matrix pipes
// and the power they draw (67 % of the cycles in the pipes at 1.35 GHz in a run of
// 1236 us under the counters); 2368 x 3584 in 527 to 624 us, where the fill of each
// tile's ring and the last round weigh more (53 % at 1.74 GHz in a run of 590 us).
template <int OP, int BM, int BNW, int STAGES, int WGM, int WGN, int KG = 1>
struct GroupTile {
  static constexpr int BK = 32 * KG;
  static constexpr int kThreads = 64 * WGM * WGN * KG;
  static constexpr int BNY = OP == GROUP_UP ? BNW / 2 : BNW;
  static constexpr int WTM = BM / WGM, WTW = BNW / WGN;  // a wave's rows and columns
  static constexpr int FA = WTM / 32, FW = WTW / 32;
  static_assert(FA >= 1 && FW >= 1 && WTM % 32 == 0 && WTW % 32 == 0, "wave tile");
  static constexpr int ACH = BK / 8, WCH = BNW / 8;  // 16-byte chunks of a row
  static constexpr int A_BYTES = BM * BK * 2, W_BYTES = BK * BNW * 2;
  static constexpr int STAGE_BYTES = A_BYTES + W_BYTES;
  static constexpr int A_CHUNKS = BM * ACH;
  static constexpr int A_LOADS = (A_CHUNKS + kThreads - 1) / kThreads, W_LOADS = BK * WCH / kThreads;
  static_assert(A_CHUNKS % 64 == 0 && BK * WCH % kThreads == 0, "a wave's chunks are whole");
  static constexpr int LOADS = A_LOADS + W_LOADS;
  static constexpr int LH = LOADS / 2;
  static_assert(LH >= 1 && LOADS * (STAGES - 2) + LH <= 63, "vmcnt range");
  static constexpr int YLD = BNY + 8;  // padded row of the output staging tile
  // a wave without chunks of A in a load fetches zeros into a slot of its own,
  // so that every wave has the same number of loads in flight
  static constexpr bool NEED_JUNK = A_CHUNKS % kThreads != 0;
  static constexpr int JUNK = STAGES * STAGE_BYTES;
  static constexpr int RING = JUNK + (NEED_JUNK ? 1024 : 0);
  static constexpr int Y_BYTES = BM * YLD * 2;
  // behind it, the sums of the wave groups on other k
  static constexpr int RED_BYTES = (KG - 1) * BM * BNW * 4;
  static constexpr int END = Y_BYTES + RED_BYTES;
  static constexpr int LDS_BYTES = RING > END ? RING : END;
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
  // chunk c of row r is stored at c ^ swz(r): 64-byte rows of A; weight rows
  // that are an odd multiple of 128 bytes alternate halves of 256 by themselves
  __host__ __device__ static constexpr int a_swz(int row) {
    if (ACH == 8) return (row >> 1) & 7;  // 128-byte rows: eight pairs of them
    return (((row >> 2) & 1) << 1) | (((row >> 1) ^ (row >> 3)) & 1);
  }
  __host__ __device__ static constexpr int w_swz(int row) {
    if ((WCH / 8) % 2 == 1) return (row & 3) << 1;
    return ((0x6530 >> (4 * (row & 3))) & 0xf) << 1;
  }
  static_assert(WCH % 8 == 0, "the weight swizzle permutes aligned groups of 8 chunks");
};

// Rows [pos0, pos0 + nrows) (nrows <= BM) of expert `e` against weight columns
// [tn BNW, (tn + 1) BNW).
template <int OP, int BM, int BNW, int STAGES, int WGM, int WGN, int KG = 1>
__device__ __forceinline__ void grouped_tile(const GroupArgs& g, int e, int pos0, int nrows,
                                             int tn, uint8_t* smem) {
  using C = GroupTile<OP, BM, BNW, STAGES, WGM, WGN, KG>;
  constexpr int BK = C::BK;
  // a copy of the thread index that the compiler cannot see through: else it
  // keeps the offsets of every tile height in registers around the loop over
  // units, and spills
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, wave = tid >> 6;
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);
  const int kg = wave / (WGM * WGN);  // which 32 k of a step
  const int wm = wave / WGN % WGM, wn = wave % WGN;
  const int K = g.K, ldw = g.ldw;
  const int wc0 = tn * BNW;
  const int nk = (K + BK - 1) / BK;

  // ---- loads of one K step: the per-thread parts do not change with k ----------
  const i32x4 rsA = make_rsrc(g.A, (uint32_t)((size_t)g.TA * K * 2));
  const i32x4 rsW = make_rsrc(g.W + (size_t)e * K * ldw, (uint32_t)((size_t)K * ldw * 2));
  const uint32_t lds0 = lds_addr(smem);
  uint32_t a_off[C::A_LOADS];
  int a_k[C::A_LOADS];  // k of the chunk within the step, huge if there is no row
#pragma unroll
  for (int i = 0; i < C::A_LOADS; ++i) {
    const int p = tid + C::kThreads * i;
    const int row = p / C::ACH, c = (p % C::ACH) ^ C::a_swz(row);
    const int ar = row < min(nrows, BM) ? group_a_row<OP>(g, pos0 + row) : -1;
    a_off[i] = ar >= 0 ? ((uint32_t)ar * (uint32_t)K + c * 8) * 2u : 0u;
    a_k[i] = ar >= 0 ? c * 8 : 0x3fffffff;
  }
  uint32_t w_off[C::W_LOADS];
#pragma unroll
  for (int i = 0; i < C::W_LOADS; ++i) {
    const int p = tid + C::kThreads * i;
    const int row = p / C::WCH, c = (p % C::WCH) ^ C::w_swz(row);
    w_off[i] = wc0 + c * 8 < ldw ? (uint32_t)(row * ldw + wc0 + c * 8) * 2u : kOutOfRange;
  }
  // load q (activations first) of K step `it` into stage ST; a step past the
  // end reads past the tensors, which gives zeros
  auto dma = [&](int it, auto st_c, int q) __attribute__((always_inline)) {
    constexpr int ST = decltype(st_c)::value;
    const int k0 = it < nk ? it * BK : K;
    const uint32_t sbase = lds0 + ST * C::STAGE_BYTES;
    if (q < C::A_LOADS) {
      const int p0 = C::kThreads * q + 64 * wave_u;  // this wave's first chunk
      const bool own = p0 < C::A_CHUNKS;
      const uint32_t off = k0 + a_k[q] < K ? a_off[q] + (uint32_t)k0 * 2u : kOutOfRange;
      lds_dma16(own ? sbase + p0 * 16 : lds0 + C::JUNK, off, rsA);
    } else {
      const int i = q - C::A_LOADS;
      lds_dma16(sbase + C::A_BYTES + (C::kThreads * i + 64 * wave_u) * 16,
                w_off[i] + (uint32_t)k0 * (uint32_t)ldw * 2u, rsW);
    }
  };

  // ---- fragments --------------------------------------------------------------------
  const int g16 = lane >> 4, s16 = lane & 15;
  const int w_row = 32 * kg + 8 * (g16 >> 1) + (s16 >> 2);
  const int w_col = wn * C::WTW + 16 * (g16 & 1) + 4 * (s16 & 3);
  const int a_row = wm * C::WTM + (lane & 31);
  const int a_chk = 4 * kg + (lane >> 5);
  constexpr int NFRAG = 2 * C::FW + C::FA;
  u32x4 wf[2][C::FW], af[2][C::FA];
  auto frag = [&](auto st_c, int sub, int fb, int r) __attribute__((always_inline)) {
    constexpr int ST = decltype(st_c)::value;
    const uint8_t* st = smem + ST * C::STAGE_BYTES;
    const int kk = sub * 16;
    if (r < 2 * C::FW) {
      const int fw = r >> 1, h = r & 1;
      const int col = w_col + fw * 32, row = kk + w_row + 4 * h;
      const u32x2 v = lds_read_tr16(st + C::A_BYTES + row * (BNW * 2) +
                                    ((col >> 3) ^ C::w_swz(row)) * 16 + ((col >> 2) & 1) * 8);
      wf[fb][fw][2 * h] = v[0];
      wf[fb][fw][2 * h + 1] = v[1];
    } else {
      const int fa = r - 2 * C::FW;
      const int row = a_row + fa * 32;
      af[fb][fa] = *reinterpret_cast<const u32x4*>(st + row * (BK * 2) +
                                                   ((kk / 8 + a_chk) ^ C::a_swz(row)) * 16);
    }
  };

  f32x16 acc[C::FW][C::FA];
#pragma unroll
  for (int i = 0; i < C::FW; ++i)
#pragma unroll
    for (int j = 0; j < C::FA; ++j) acc[i][j] = f32x16{};

  // One K step on stage ST, two sub-steps of 16 k.  The reads of the next
  // sub-step ride on the first half of the matrix instructions, the loads on
  // the second: sub-step 0 finishes step it + STAGES - 1, and behind the
  // barrier (every wave is done with stage ST) sub-step 1 begins it + STAGES.
  constexpr int NMF = C::FW * C::FA;
  constexpr int HALF = NMF / 2 > 0 ? NMF / 2 : 1;
  constexpr int DSLOTS = NMF - HALF > 0 ? NMF - HALF : 1;
  constexpr int DBEGIN = NMF - DSLOTS;
  auto kstep = [&](int it, auto st_c) __attribute__((always_inline)) {
    constexpr int ST = decltype(st_c)::value;
    using Next = std::integral_constant<int, (ST + 1) % STAGES>;
    using Prev = std::integral_constant<int, (ST + STAGES - 1) % STAGES>;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      if (sub == 1) {
        wait_vmcnt<(STAGES - 2) * C::LOADS>();
        __syncthreads();
      }
      const int nd = sub == 0 ? C::LOADS - C::LH : C::LH;
#pragma unroll
      for (int q = 0; q < NMF; ++q) {
        const int i = q / C::FA, j = q % C::FA;
        acc[i][j] = mfma32(wf[sub][i], af[sub][j], acc[i][j]);
        if (q < HALF) {
#pragma unroll
          for (int x = q * NFRAG / HALF; x < (q + 1) * NFRAG / HALF; ++x) {
            if (sub == 1) frag(Next{}, 0, 0, x);
            else frag(st_c, 1, 1, x);
          }
        }
        if (q >= DBEGIN) {
#pragma unroll
          for (int x = (q - DBEGIN) * nd / DSLOTS; x < (q - DBEGIN + 1) * nd / DSLOTS; ++x) {
            if (sub == 0) dma(it + STAGES - 1, Prev{}, C::LH + x);
            else dma(it + STAGES, st_c, x);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // ---- prologue: steps 0 .. STAGES - 2 and the first half of STAGES - 1 -------------
  auto fill = [&](int it, auto st_c, int q1) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < C::LOADS; ++q)
      if (q < q1) dma(it, st_c, q);
  };
  [&]<int... S>(std::integer_sequence<int, S...>) __attribute__((always_inline)) {
    (fill(S, std::integral_constant<int, S>{}, C::LOADS), ...);
  }(std::make_integer_sequence<int, STAGES - 1>{});
  fill(STAGES - 1, std::integral_constant<int, STAGES - 1>{}, C::LH);
  wait_vmcnt<(STAGES - 2) * C::LOADS + C::LH>();
  __syncthreads();
#pragma unroll
  for (int r = 0; r < NFRAG; ++r) frag(std::integral_constant<int, 0>{}, 0, 0, r);

  // ---- main loop, the stage ring unrolled ---------------------------------------------
  int it = 0;
  for (; it + STAGES <= nk; it += STAGES)
    [&]<int... S>(std::integer_sequence<int, S...>) __attribute__((always_inline)) {
      (kstep(it + S, std::integral_constant<int, S>{}), ...);
    }(std::make_integer_sequence<int, STAGES>{});
  [&]<int... S>(std::integer_sequence<int, S...>) __attribute__((always_inline)) {
    ((it + S < nk ? (kstep(it + S, std::integral_constant<int, S>{}), 0) : 0), ...);
  }(std::make_integer_sequence<int, STAGES - 1>{});

  // ---- epilogue: bf16 tile through LDS, then 16-byte row stores ---------------------
  wait_vmcnt<0>();
  __syncthreads();
  uint16_t* ys = reinterpret_cast<uint16_t*>(smem);  // [BM][YLD]
  if constexpr (KG > 1) {
    // the groups' sums are added in their order
    f32x4* red = reinterpret_cast<f32x4*>(smem + C::Y_BYTES);
    constexpr int NQ = C::FW * C::FA * 4, WAVES = WGM * WGN;
    const int w = wave % WAVES;
    if (kg > 0) {
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
        const f32x16& d = acc[x / 4 / C::FA][x / 4 % C::FA];
        const int r = x % 4 * 4;
        red[(((kg - 1) * WAVES + w) * NQ + x) * 64 + lane] = f32x4{d[r], d[r + 1], d[r + 2], d[r + 3]};
      }
    }
    __syncthreads();
    if (kg == 0) {
#pragma unroll
      for (int x = 0; x < NQ; ++x) {
        f32x16& d = acc[x / 4 / C::FA][x / 4 % C::FA];
        const int r = x % 4 * 4;
#pragma unroll
        for (int o = 0; o < KG - 1; ++o) {
          const f32x4 v = red[((o * WAVES + w) * NQ + x) * 64 + lane];
#pragma unroll
          for (int q = 0; q < 4; ++q) d[r + q] += v[q];
        }
      }
    }
  }
  const int h32 = lane >> 5;
#pragma unroll
  for (int i = 0; i < C::FW; ++i)
#pragma unroll
    for (int j = 0; j < C::FA; ++j) {
      if (KG > 1 && kg > 0) continue;
      const f32x16& d = acc[i][j];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // registers 4q .. 4q + 3: weight columns wcl .. wcl + 3 of this lane's row
        const int wcl = wn * C::WTW + i * 32 + 8 * q + 4 * h32;
        uint16_t* y = ys + (a_row + j * 32) * C::YLD;
        if constexpr (OP == GROUP_UP)
          *reinterpret_cast<uint32_t*>(y + wcl / 2) =
              pack_bf16x2(silu(d[4 * q]) * d[4 * q + 1], silu(d[4 * q + 2]) * d[4 * q + 3]);
        else
          *reinterpret_cast<u32x2*>(y + wcl) = u32x2{pack_bf16x2(d[4 * q], d[4 * q + 1]),
                                                     pack_bf16x2(d[4 * q + 2], d[4 * q + 3])};
      }
    }
  __syncthreads();
  constexpr int YCH = C::BNY / 8;
  const int y0 = tn * C::BNY;
  for (int p = tid; p < BM * YCH; p += C::kThreads) {
    const int row = p / YCH, cq = p % YCH, gc = y0 + cq * 8;
    if (row >= nrows || gc >= g.N) continue;
    const int out = OP == GROUP_UP ? pos0 + row : g.rows[pos0 + row];
    if (out < 0 || out >= g.R) continue;
    *reinterpret_cast<u32x4*>(g.Y + (size_t)out * g.N + gc) =
        *reinterpret_cast<const u32x4*>(ys + row * C::YLD + cq * 8);
  }
}

// Within an expert the tiles go in bands of up to 8 row tiles, column after
// column, so that the workgroups of an XCD share weight columns and rows of A
// in its L2.  Workgroup b runs on XCD b % 8 and takes units of that XCD's range
// in turn: how many there are is known on the device only, and with short
// tiles an eighth of the work may be more than an eighth of the units.  The
// last tile of an expert runs at the height that its rows need (fewer matrix
// instructions).
template <int OP, int BM, int BNW, int STAGES, int WGM, int WGN, int PARTS, int PWGM, int PWGN,
          int KG>
__global__ __launch_bounds__(64 * WGM * WGN * KG) void grouped_tile_kernel(GroupArgs g, int ntn) {
  constexpr int P = BM / PARTS;  // rows of a part
  constexpr int LDS = GroupTile<OP, BM, BNW, STAGES, WGM, WGN, KG>::LDS_BYTES + (PARTS > 1 ? 1024 : 0);
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS];
  const GroupRange range = group_range<BM, PARTS>(g.offsets, g.E, g.R, ntn, blockIdx.x % 8);
  const int nwg = ((int)gridDim.x + 7 - (int)(blockIdx.x % 8)) / 8;  // of this XCD
  for (int t = range.begin + (int)blockIdx.x / 8; t < range.end; t += nwg) {
    const GroupUnit u = group_unit<BM>(g.offsets, g.E, g.R, ntn, t);
    const int ntm = (u.rows + BM - 1) / BM;
    constexpr int kBand = 8;
    const int band = u.local / (kBand * ntn), in = u.local % (kBand * ntn);
    const int high = min(ntm - band * kBand, kBand);
    const int tm = band * kBand + in % high, tn = in / high;
    const int pos0 = u.first + tm * BM, rows = min(u.rows - tm * BM, BM);
    const int parts = (rows + P - 1) / P;
    auto part = [&](auto n_c) __attribute__((always_inline)) {
      constexpr int ROWS = decltype(n_c)::value * P;
      // short tiles: the waves side by side where two rows of them do not fit
      constexpr int WM = ROWS / 32 >= PWGM && ROWS % (32 * PWGM) == 0 ? PWGM : 1;
      constexpr int WN = PWGM * PWGN / WM;
      static_assert(GroupTile<OP, ROWS, BNW, STAGES, WM, WN, KG>::LDS_BYTES <= LDS, "LDS");
      grouped_tile<OP, ROWS, BNW, STAGES, WM, WN, KG>(g, u.expert, pos0, rows, tn, smem);
    };
    if (parts == PARTS) {
      grouped_tile<OP, BM, BNW, STAGES, WGM, WGN, KG>(g, u.expert, pos0, rows, tn, smem);
    } else if (PARTS >= 4 && parts == 3) {
      if constexpr (PARTS >= 4) part(std::integral_constant<int, 3>{});
    } else if (PARTS >= 4 && parts == 2) {
      if constexpr (PARTS >= 4) part(std::integral_constant<int, 2>{});
    } else {
      if constexpr (PARTS >= 2) part(std::integral_constant<int, 1>{});
    }
    __syncthreads();  // the next unit's loads overwrite this one's rows of Y in LDS
  }
}

// ============================================================================
// Few rows an expert: weight streaming
// ============================================================================
// One workgroup takes up to 16 rows of one expert and a slab of 128 of its
// weight columns; its NW waves take every NW-th step of 32 k.  A lane loads an
// 8 (k) x 8 (column) block of weights into registers, transposes it there and
// feeds eight v_mfma_f32_16x16x32_bf16; other waves' loads are in flight
// meanwhile.  The waves' fp32 sums are added in LDS in wave order, so the result
// does not depend on timing; up applies SiLU after that.  32 rows on 64 experts,
// 1536 x 3584: 59.8 us, 5.9 TB/s of weights.
constexpr int kStreamRows = 16;
template <int OP, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(4)))
void grouped_stream_kernel(GroupArgs g, int nslab) {
  __shared__ __attribute__((aligned(16))) f32x4 red[NW * 8 * 64];
  const int x = blockIdx.x % 8;
  const GroupRange range = group_range<kStreamRows, 1>(g.offsets, g.E, g.R, nslab, x);
  const int t = range.begin + (int)blockIdx.x / 8;
  if (t >= range.end) return;
  const GroupUnit u = group_unit<kStreamRows>(g.offsets, g.E, g.R, nslab, t);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int slab = u.local % nslab, pos0 = u.first + u.local / nslab * kStreamRows;
  const int nrows = min(u.first + u.rows - pos0, kStreamRows);
  const int K = g.K, ldw = g.ldw;
  const uint16_t* W = g.W + (size_t)u.expert * K * ldw;
  const int c0 = slab * 128 + (lane & 15) * 8;
  const bool cin = c0 < ldw;  // ldw % 8 == 0: eight columns are in range together

  // this lane's row of A; rows past the span repeat the last one (an output row
  // depends on its own row of A alone, and those are never stored)
  const int ar = group_a_row<OP>(g, pos0 + min(lane & 15, nrows - 1));
  const bool ain = ar >= 0;
  const uint16_t* ap = g.A + (size_t)max(ar, 0) * K;
  f32x4 acc[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = f32x4{};

  const int nsteps = (K + 31) / 32;
  for (int s = wave; s < nsteps; s += NW) {
    const int k = s * 32 + (lane >> 4) * 8;
    const bool kin = k < K;  // K % 8 == 0: eight k are in range together
    u32x4 w[8], col[8];
    const uint16_t* p = W + (size_t)k * ldw + c0;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      w[r] = kin && cin ? load16_stream(p + (size_t)r * ldw) : u32x4{0, 0, 0, 0};
    const u32x4 a = kin && ain ? load16(ap + k) : u32x4{0, 0, 0, 0};
    transpose8x8(w, col);
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = mfma16(a, col[c], acc[c]);
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) red[(wave * 8 + c) * 64 + lane] = acc[c];
  __syncthreads();
  if (wave > 0) return;

  // register r of a lane is row 4 (lane / 16) + r, accumulator c column c0 + c
  f32x4 v[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    v[c] = red[c * 64 + lane];
    for (int w = 1; w < NW; ++w) v[c] += red[(w * 8 + c) * 64 + lane];
  }
  if (!cin) return;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = (lane >> 4) * 4 + r;
    if (row >= nrows) continue;
    const int out = OP == GROUP_UP ? pos0 + row : g.rows[pos0 + row];
    if (out < 0 || out >= g.R) continue;
    uint16_t* y = g.Y + (size_t)out * g.N;
    if constexpr (OP == GROUP_UP) {
      float s[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] = silu(v[2 * q][r]) * v[2 * q + 1][r];
      *reinterpret_cast<u32x2*>(y + c0 / 2) = u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
    } else {
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(v[2 * q][r], v[2 * q + 1][r]);
      *reinterpret_cast<u32x4*>(y + c0) = o;
    }
  }
}

// ============================================================================
// Launches
// ============================================================================
// At most this many tiles of bm rows, whatever the spans: one partial tile for
// each expert that has rows.
static long long max_row_tiles(long long R, long long E, long long bm) {
  const long long some = std::min(R, E);
  return std::min(R, (R + some * (bm - 1)) / bm);
}

// Workgroups of the tile kernel.  Every XCD's range needs workgroups there.  With
// short tiles an eighth of the work can be up to 2.2 eighths of the units, so up
// to some rounds of workgroups there are twice as many as units; beyond that the
// loop takes what is left over.  Measured (us, twice as many / as many; K = 1536):
// tiles of 128 x 128, 8 experts of 513 rows and 60 of one, 400 units 39.4 / 48.5,
// 800 67.3 / 67.5; tiles of 256 x 256, 16 experts of 257 and 16 of one, 288 units
// 66.3 / 78.7; 8 of 1025 and 40 of one, 320 units 63.0 / 69.8, 640 119.1 / 110.7.
// Evenly filled experts are level (658 units 121.1 / 120.0; 1092 174.1 / 170.0).
static long long tile_grid(long long R, long long E, long long ldw, int bm, int bnw, int parts) {
  const long long units = max_row_tiles(R, E, bm) * ((ldw + bnw - 1) / bnw);
  return (units * (parts > 1 && units < 1024 ? 2 : 1) + 7) / 8 * 8;
}
// Of the streaming kernel: one a unit.  All units weigh the same, so no XCD has
// more than an eighth of them, rounded up.
static long long stream_grid(long long R, long long E, long long ldw) {
  return (max_row_tiles(R, E, kStreamRows) * ((ldw + 127) / 128) + 7) / 8 * 8;
}

template <int OP, int BM, int BNW, int STAGES, int WGM, int WGN, int PARTS, int PWGM, int PWGN,
          int KG = 1>
static hipError_t launch_tile(const GroupArgs& g, hipStream_t stream) {
  static_assert(WGM * WGN == PWGM * PWGN && (PARTS == 1 || PARTS == 2 || PARTS == 4), "one workgroup");
  const long long ntn = (g.ldw + BNW - 1) / BNW;
  const long long grid = tile_grid(g.R, g.E, g.ldw, BM, BNW, PARTS);
  if (grid > 0x7fffffffLL) return hipErrorInvalidValue;
  return launch_op(grouped_tile_kernel<OP, BM, BNW, STAGES, WGM, WGN, PARTS, PWGM, PWGN, KG>,
                   dim3((unsigned)grid), dim3(64 * WGM * WGN * KG), stream, g, (int)ntn);
}
template <int OP, int NW>
static hipError_t launch_stream(const GroupArgs& g, hipStream_t stream) {
  const long long nslab = (g.ldw + 127) / 128, grid = stream_grid(g.R, g.E, g.ldw);
  if (grid > 0x7fffffffLL) return hipErrorInvalidValue;
  return launch_op(grouped_stream_kernel<OP, NW>, dim3((unsigned)grid), dim3(64 * NW),
                   stream, g, (int)nslab);
}

template <int OP>
static hipError_t launch_grouped_op(const GroupArgs& g, int variant, hipStream_t stream) {
  switch (variant) {
    case 0: return launch_stream<OP, 8>(g, stream);
    case 1: return launch_tile<OP, 64, 128, 4, 2, 2, 1, 2, 2>(g, stream);
    case 2: return launch_tile<OP, 128, 128, 4, 2, 2, 2, 2, 2>(g, stream);
    case 4: return launch_tile<OP, 64, 64, 4, 2, 1, 1, 2, 1, 2>(g, stream);
    default: return launch_tile<OP, 256, 256, 4, 4, 2, 4, 2, 4>(g, stream);
  }
}

// The counts are on the device; the mean rows of an expert decide, and whether
// there is a workgroup for every CU.  Measured at many units (us, 2048 x 2816 weights, 32
// experts, variants 0 / 1 / 3): mean 8: 61 / 70 / 75, 24: 114 / 72 / 78, 64: 244
// / 93 / 80.  With few units the wide tiles stream better (8 experts, 3584 x
// 4736, mean 8, 0 / 3: 57 / 52).  Where even those leave CUs idle the bytes that
// one CU can take in bound the call (about 50 a ns measured, however many loads
// are in flight), so the tiles get smaller until there are about as many as CUs:
// variants 1 / 2 / 4 take 44.9 / 35.8 / 43.4 us with 168 tiles of 128 x 128 (4
// experts, 3416 x 816, mean 644), 24.9 / 31.7 / 27.9 with 112 of them (3584 x
// 1792, mean 250), and 22.7 / 29.4 / 14.7 with 84 of 64 x 128 (3584 x 896, mean
// 150).  One row an expert (a single token), weights from HBM, variants 0 / 2 / 3 / 4,
// the rule's choice in brackets: 1536 x 3584, 4 experts 14.6 / 17.4 / 22.2 / [13.4], 8
// experts 18.5 / [19.7] / 24.4 / 22.8, 24 experts [48.7] / 56.6 / 60.6 / 58.1; 1792 x
// 1536, 8 experts 15.9 / 19.0 / 24.8 / [14.1], 16 experts 19.0 / [21.6] / 27.3 / 24.6;
// 3584 x 4736, 4 experts 27.0 / [38.7] / 45.8 / 33.6, 8 experts 55.6 / 54.8 / [50.1] /
// 58.2.  So with so few rows and fewer than 128 wide tiles streaming is up to 30 %
// faster than variant 2 that the rule takes, and between 128 and 200 of them than
// variant 3 (32 rows on 16 of 64 experts, 1792 x 1536: 19.3 / 21.6 / [27.4] / 24.8).
static int grouped_variant(long long R, long long E, long long ldw) {
  const long long some = std::min(R, E), mean = (R + E - 1) / E;
  auto units = [&](long long bm, long long bnw) {
    return some * ((mean + bm - 1) / bm) * ((ldw + bnw - 1) / bnw);
  };
  const long long wide = units(256, 256);
  if (wide < 128) return units(64, 128) <= 128 ? 4 : (units(128, 128) <= 128 ? 1 : 2);
  if (wide >= 200 && mean <= 10) return 0;
  if (wide >= 200 && mean <= 28) return 1;
  return 3;
}

// Threads of the launch that launch_grouped_op makes.
long long grouped_threads(bool up, long long R, long long N, long long E, int variant) {
  const long long ldw = up ? 2 * N : N;
  if (variant < 0) variant = grouped_variant(R, E, ldw);
  switch (variant) {
    case 0: return stream_grid(R, E, ldw) * 512;
    case 1: return tile_grid(R, E, ldw, 64, 128, 1) * 256;
    case 2: return tile_grid(R, E, ldw, 128, 128, 2) * 256;
    case 4: return tile_grid(R, E, ldw, 64, 64, 1) * 256;
    default: return tile_grid(R, E, ldw, 256, 256, 4) * 512;
  }
}

hipError_t launch_grouped(bool up, const uint16_t* A, const int32_t* rows, const int32_t* offsets,
                          const uint16_t* W, uint16_t* Y, int TA, int R, int N, int K, int E,
                          int k, int variant, hipStream_t stream) {
  const GroupArgs g{A, rows, offsets, W, Y, TA, R, N, K, E, k, up ? 2 * N : N};
  if (variant < 0) variant = grouped_variant(R, E, g.ldw);
  return up ? launch_grouped_op<GROUP_UP>(g, variant, stream)
            : launch_grouped_op<GROUP_DOWN>(g, variant, stream);
}

}  // namespace swiglu
