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
// XOR-swizzled chunks so that the lanes served together hit distinct banks.
// Rows past the span, columns past the matrix and k past K arrive as zeros (a
// buffer load past the resource returns 0).
template <int OP, int BM, int BNW, int STAGES, int WGM, int WGN>
struct GroupTile {
  static constexpr int BK = 32;
  static constexpr int kThreads = 64 * WGM * WGN;
  static constexpr int BNY = OP == GROUP_UP ? BNW / 2 : BNW;
  static constexpr int WTM = BM / WGM, WTW = BNW / WGN;  // a wave's rows and columns
  static constexpr int FA = WTM / 32, FW = WTW / 32;
  static_assert(FA >= 1 && FW >= 1 && WTM % 32 == 0 && WTW % 32 == 0, "wave tile");
  static constexpr int ACH = BK / 8, WCH = BNW / 8;  // 16-byte chunks of a row
  static constexpr int A_BYTES = BM * BK * 2, W_BYTES = BK * BNW * 2;
  static constexpr int STAGE_BYTES = A_BYTES + W_BYTES;
  static constexpr int A_LOADS = BM * ACH / kThreads, W_LOADS = BK * WCH / kThreads;
  static_assert(BM * ACH % kThreads == 0 && BK * WCH % kThreads == 0, "whole loads");
  static constexpr int LOADS = A_LOADS + W_LOADS;
  static constexpr int LH = LOADS / 2;
  static_assert(LH >= 1 && LOADS * (STAGES - 2) + LH <= 63, "vmcnt range");
  static constexpr int YLD = BNY + 8;  // padded row of the output staging tile
  static constexpr int RING = STAGES * STAGE_BYTES;
  static constexpr int Y_BYTES = BM * YLD * 2;
  static constexpr int LDS_BYTES = RING > Y_BYTES ? RING : Y_BYTES;
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
  // chunk c of row r is stored at c ^ swz(r): 64-byte rows of A; weight rows
  // that are an odd multiple of 128 bytes alternate halves of 256 by themselves
  __host__ __device__ static constexpr int a_swz(int row) {
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
template <int OP, int BM, int BNW, int STAGES, int WGM, int WGN>
__device__ __forceinline__ void grouped_tile(const GroupArgs& g, int e, int pos0, int nrows,
                                             int tn, uint8_t* smem) {
  using C = GroupTile<OP, BM, BNW, STAGES, WGM, WGN>;
  constexpr int BK = C::BK;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);
  const int wm = wave / WGN, wn = wave % WGN;
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
    const int ar = row < nrows ? group_a_row<OP>(g, pos0 + row) : -1;
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
      const uint32_t off = k0 + a_k[q] < K ? a_off[q] + (uint32_t)k0 * 2u : kOutOfRange;
      lds_dma16(sbase + (C::kThreads * q + 64 * wave_u) * 16, off, rsA);
    } else {
      const int i = q - C::A_LOADS;
      lds_dma16(sbase + C::A_BYTES + (C::kThreads * i + 64 * wave_u) * 16,
                w_off[i] + (uint32_t)k0 * (uint32_t)ldw * 2u, rsW);
    }
  };

  // ---- fragments --------------------------------------------------------------------
  const int g16 = lane >> 4, s16 = lane & 15;
  const int w_row = 8 * (g16 >> 1) + (s16 >> 2);
  const int w_col = wn * C::WTW + 16 * (g16 & 1) + 4 * (s16 & 3);
  const int a_row = wm * C::WTM + (lane & 31);
  const int a_chk = lane >> 5;
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
  const int h32 = lane >> 5;
#pragma unroll
  for (int i = 0; i < C::FW; ++i)
#pragma unroll
    for (int j = 0; j < C::FA; ++j) {
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

// Units are ordered expert by expert, within one in bands of up to 8 row tiles,
// column after column, so that the workgroups of an XCD share weight columns
// and rows of A in its L2.  An expert's last tile runs at half the height when
// its rows fit (half the matrix instructions); HWGM = 0: no such form.
template <int OP, int BM, int BNW, int STAGES, int WGM, int WGN, int HWGM, int HWGN>
__global__ __launch_bounds__(64 * WGM * WGN) void grouped_tile_kernel(GroupArgs g, int ntn) {
  using C = GroupTile<OP, BM, BNW, STAGES, WGM, WGN>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS_BYTES];
  GroupUnit u;
  if (!group_find<BM>(g.offsets, g.E, g.R, ntn, blockIdx.x, u)) return;
  const int ntm = (u.rows + BM - 1) / BM;
  constexpr int kBand = 8;
  const int band = u.local / (kBand * ntn), in = u.local % (kBand * ntn);
  const int high = min(ntm - band * kBand, kBand);
  const int tm = band * kBand + in % high, tn = in / high;
  const int nrows = u.rows - tm * BM;
  if constexpr (HWGM > 0) {
    using H = GroupTile<OP, BM / 2, BNW, STAGES, HWGM, HWGN>;
    static_assert(C::kThreads == H::kThreads && H::LDS_BYTES <= C::LDS_BYTES, "one workgroup");
    if (nrows <= BM / 2) {
      grouped_tile<OP, BM / 2, BNW, STAGES, HWGM, HWGN>(g, u.expert, u.first + tm * BM, nrows, tn,
                                                        smem);
      return;
    }
  }
  grouped_tile<OP, BM, BNW, STAGES, WGM, WGN>(g, u.expert, u.first + tm * BM, min(nrows, BM), tn,
                                              smem);
}

// ============================================================================
// Few rows an expert: weight streaming
// ============================================================================
// One workgroup takes up to 16 MT rows of one expert and a slab of 128 of its
// weight columns; its NW waves take every NW-th step of 32 k.  A lane loads an
// 8 (k) x 8 (column) block of weights into registers, transposes it there and
// feeds eight v_mfma_f32_16x16x32_bf16 per 16 rows; other waves' loads are in
// flight meanwhile.  The waves' fp32 sums are added in LDS in wave order, so
// the result does not depend on timing; up applies SiLU after that.
template <int OP, int MT, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(MT == 1 ? 4 : 2)))
void grouped_stream_kernel(GroupArgs g, int nslab) {
  __shared__ __attribute__((aligned(16))) f32x4 red[NW * MT * 8 * 64];
  GroupUnit u;
  if (!group_find<16 * MT>(g.offsets, g.E, g.R, nslab, blockIdx.x, u)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int slab = u.local % nslab, pos0 = u.first + u.local / nslab * (16 * MT);
  const int nrows = min(u.first + u.rows - pos0, 16 * MT);
  const int K = g.K, ldw = g.ldw;
  const uint16_t* W = g.W + (size_t)u.expert * K * ldw;
  const int c0 = slab * 128 + (lane & 15) * 8;
  const bool cin = c0 < ldw;  // ldw % 8 == 0: eight columns are in range together

  // this lane's row of A in each block of 16; rows past the span repeat the
  // last one (an output row depends on its own row of A alone, and those are
  // never stored)
  const uint16_t* ap[MT];
  bool ain[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int ar = group_a_row<OP>(g, pos0 + min(mt * 16 + (lane & 15), nrows - 1));
    ain[mt] = ar >= 0;
    ap[mt] = g.A + (size_t)max(ar, 0) * K;
  }
  f32x4 acc[MT][8];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[mt][c] = f32x4{};

  const int nsteps = (K + 31) / 32;
  for (int s = wave; s < nsteps; s += NW) {
    const int k = s * 32 + (lane >> 4) * 8;
    const bool kin = k < K;  // K % 8 == 0: eight k are in range together
    u32x4 w[8], a[MT], col[8];
    const uint16_t* p = W + (size_t)k * ldw + c0;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      w[r] = kin && cin ? load16_stream(p + (size_t)r * ldw) : u32x4{0, 0, 0, 0};
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      a[mt] = kin && ain[mt] ? load16(ap[mt] + k) : u32x4{0, 0, 0, 0};
    transpose8x8(w, col);
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[mt][c] = mfma16(a[mt], col[c], acc[mt][c]);
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int c = 0; c < 8; ++c) red[((wave * MT + mt) * 8 + c) * 64 + lane] = acc[mt][c];
  __syncthreads();

  // register r of a lane is row 4 (lane / 16) + r, accumulator c column c0 + c
  for (int mt = wave; mt < MT; mt += NW) {
    f32x4 v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      v[c] = red[(mt * 8 + c) * 64 + lane];
      for (int w = 1; w < NW; ++w) v[c] += red[((w * MT + mt) * 8 + c) * 64 + lane];
    }
    if (!cin) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = mt * 16 + (lane >> 4) * 4 + r;
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

template <int OP, int BM, int BNW, int STAGES, int WGM, int WGN, int HWGM, int HWGN>
static hipError_t launch_tile(const GroupArgs& g, hipStream_t stream) {
  using C = GroupTile<OP, BM, BNW, STAGES, WGM, WGN>;
  const long long ntn = (g.ldw + BNW - 1) / BNW;
  const long long units = max_row_tiles(g.R, g.E, BM) * ntn;
  if (units > 0x7fffffffLL) return hipErrorInvalidValue;
  return launch_op(grouped_tile_kernel<OP, BM, BNW, STAGES, WGM, WGN, HWGM, HWGN>,
                   dim3((unsigned)units), dim3(C::kThreads), stream, g, (int)ntn);
}
template <int OP, int MT, int NW>
static hipError_t launch_stream(const GroupArgs& g, hipStream_t stream) {
  const long long nslab = (g.ldw + 127) / 128;
  const long long units = max_row_tiles(g.R, g.E, 16 * MT) * nslab;
  if (units > 0x7fffffffLL) return hipErrorInvalidValue;
  return launch_op(grouped_stream_kernel<OP, MT, NW>, dim3((unsigned)units), dim3(64 * NW),
                   stream, g, (int)nslab);
}

template <int OP>
static hipError_t launch_grouped_op(const GroupArgs& g, int variant, hipStream_t stream) {
  switch (variant) {
    case 0: return launch_stream<OP, 1, 8>(g, stream);
    case 1: return launch_stream<OP, 2, 8>(g, stream);
    case 2: return launch_tile<OP, 64, 128, 4, 2, 2, 0, 0>(g, stream);
    case 3: return launch_tile<OP, 128, 128, 4, 2, 2, 2, 2>(g, stream);
    default: return launch_tile<OP, 256, 256, 4, 4, 2, 2, 4>(g, stream);
  }
}

// Rows an expert on average decide; the counts themselves are on the device.
static int grouped_variant(long long R, long long E) {
  const long long mean = (R + E - 1) / E;
  if (mean <= 8) return 0;
  if (mean <= 24) return 1;
  if (mean <= 64) return 2;
  if (mean <= 160) return 3;
  return 4;
}

hipError_t launch_grouped(bool up, const uint16_t* A, const int32_t* rows, const int32_t* offsets,
                          const uint16_t* W, uint16_t* Y, int TA, int R, int N, int K, int E,
                          int k, int variant, hipStream_t stream) {
  const GroupArgs g{A, rows, offsets, W, Y, TA, R, N, K, E, k, up ? 2 * N : N};
  if (variant < 0) variant = grouped_variant(R, E);
  return up ? launch_grouped_op<GROUP_UP>(g, variant, stream)
            : launch_grouped_op<GROUP_DOWN>(g, variant, stream);
}

}  // namespace swiglu
