// swiglu_fp4.hip -- MXFP4: quantisation of bf16 rows to 4-bit blocks and back, and
// the gated MLP Y = SiLU(A G) (.) (A U) on MXFP4 activations and weights.
//
// Format (OCP Microscaling, E2M1 elements): 32 consecutive k of a row share an
// E8M0 byte e; element code c stands for 2^(e - 127) value(c), value one of 0,
// .5, 1, 1.5, 2, 3, 4, 6 with a sign.  Both tensors of a product are stored in
// the order its 32x32x64 matrix instructions take them (rows in blocks of 32,
// K in groups of 256 as 4 steps of 64 k, G = ceil(K / 256) groups):
//   Q[(((rb G + g) 4 + s) 2 + h) 512 + 16 i + b]  =  codes of row 32 rb + i,
//       k = 256 g + 64 s + 32 h + 2 b (low nibble) and + 1 (high nibble)
//   S[((rb G + g) 2 + h) 128 + 4 i + s]  =  the block's E8M0 byte
// padded to whole blocks with code 0 at scale 2^0.  Lane i + 32 h then finds its
// 16 bytes of a step contiguous with its neighbours' (1 KB a load) and the
// scales of four steps in one dword, for activations and weights alike.
#include "swiglu_internal.h"
#include "swiglu_ops_device.hpp"

#include <algorithm>
#include <type_traits>
#include <utility>

namespace swiglu {

// ============================================================================
// Quantisation
// ============================================================================
// A wave takes 8 rows of a block of 32 and one group of 256 k: a load
// instruction covers 8 rows x 64 k (whole 128-byte lines), four lanes share a
// block of 32, so its maximum is two lane exchanges and its 16 bytes of codes
// one run; 8 rows' runs are 128 contiguous bytes.  The lane keeps the scale
// bytes of the four steps as the dword that the format wants.  Bound by memory.
//   shared exponent = floor(log2 max |x|) - 2 (2: E2M1's largest binade),
//   clamped to [-127, 127]; elements x 2^-shared to nearest even, saturating
//   at 6.  An infinity counts as 2^128.  A block that holds a NaN has no codes
//   for it: its scale byte is 255, the format's NaN.
__global__ __launch_bounds__(256) void quantize_fp4_kernel(const uint16_t* __restrict__ X,
                                                           uint8_t* __restrict__ Q,
                                                           uint8_t* __restrict__ S, int rows,
                                                           int K, int groups, int nw) {
  const int lane = threadIdx.x & 63;
  const int w = blockIdx.x * 4 + (threadIdx.x >> 6);  // (row block, group, 8 rows of 4)
  if (w >= nw) return;
  const int r8 = w & 3, rg = w >> 2;
  const int g = rg % groups, rb = rg / groups;
  const int i = 8 * r8 + (lane >> 3);  // row of the block
  const int h = (lane >> 2) & 1, q = lane & 3;
  const int row = 32 * rb + i;
  u32x4 v[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int k = 256 * g + 64 * s + 32 * h;
    v[s] = row < rows && k < K ? load16_stream(X + (size_t)row * K + k + 8 * q) : u32x4{0, 0, 0, 0};
  }
  uint32_t scales = 0;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    // the largest magnitude as bf16 bits: above 0x7f80 it is a NaN
    uint32_t m = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) m = max(m, max(v[s][d] & 0x7fffu, (v[s][d] >> 16) & 0x7fffu));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppXor1, 0xf, 0xf, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppXor2, 0xf, 0xf, false));
    const bool pad = row >= rows || 256 * g + 64 * s + 32 * h >= K;
    const int e = max((int)(m >> 7) - 2, 0);  // biased: floor(log2) + 127 - 2
    const uint32_t byte = pad ? 127u : (m > 0x7f80u ? 255u : (uint32_t)e);
    scales |= byte << (8 * s);
    // 2^(e - 127) as fp32; e = 0 is a subnormal there
    const float scale = __builtin_bit_cast(float, e > 0 ? (uint32_t)e << 23 : 1u << 22);
    const uint32_t codes = e2m1_codes(v[s], scale);
    *reinterpret_cast<uint32_t*>(Q + ((((size_t)rg * 4 + s) * 2 + h) * 512 + 16 * i + 4 * q)) = codes;
  }
  if (q == 0) *reinterpret_cast<uint32_t*>(S + (((size_t)rg * 2 + h) * 128 + 4 * i)) = scales;
}

// The values of the codes, rounded once to bf16 (exact but where 2^128 is
// passed, which gives infinity).
__global__ __launch_bounds__(256) void dequantize_fp4_kernel(const uint8_t* __restrict__ Q,
                                                             const uint8_t* __restrict__ S,
                                                             uint16_t* __restrict__ X, int rows,
                                                             int K, int groups, int nw) {
  const int lane = threadIdx.x & 63;
  const int w = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (w >= nw) return;
  const int r8 = w & 3, rg = w >> 2;
  const int g = rg % groups, rb = rg / groups;
  const int i = 8 * r8 + (lane >> 3);
  const int h = (lane >> 2) & 1, q = lane & 3;
  const int row = 32 * rb + i;
  if (row >= rows) return;
  const uint32_t scales = *reinterpret_cast<const uint32_t*>(S + (((size_t)rg * 2 + h) * 128 + 4 * i));
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int k = 256 * g + 64 * s + 32 * h;
    if (k >= K) break;
    const uint32_t c =
        *reinterpret_cast<const uint32_t*>(Q + ((((size_t)rg * 4 + s) * 2 + h) * 512 + 16 * i + 4 * q));
    const int e = (int)((scales >> (8 * s)) & 0xffu);
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      f[j] = e == 255 ? __builtin_nanf("") : __builtin_ldexpf(e2m1_value(c >> (4 * j)), e - 127);
    *reinterpret_cast<u32x4*>(X + (size_t)row * K + k + 8 * q) =
        u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
              pack_bf16x2(f[6], f[7])};
  }
}

// ============================================================================
// The product, LDS-tiled
// ============================================================================
// One workgroup: BM rows of A against BNW rows of W (Gate and Up rows
// alternate, so a pair is two adjacent registers of a lane), as D = W A^T on
// v_mfma_scale_f32_32x32x64_f8f6f4, which multiplies 4-bit sources at four
// times the bf16 rate and applies the block scales itself.  A stage is 128 k:
// 2 KB of every block of 32 rows, contiguous in HBM and copied as it is into a
// ring of STAGES LDS stages; a fragment is one 16-byte read a lane at 16 x
// lane, without bank conflicts and with no address arithmetic.  The scales of
// a group of 256 k (two stages) come with its first stage into a ring of
// their own.
template <int BM, int BNW, int STAGES, int WGM, int WGN>
struct F4Tile {
  static constexpr int kWaves = WGM * WGN, kThreads = 64 * kWaves;
  static constexpr int BNY = BNW / 2;
  static constexpr int FA = BM / WGM / 32, FW = BNW / WGN / 32;  // blocks of 32 a wave
  static_assert(FA >= 1 && FW >= 1 && FA * WGM * 32 == BM && FW * WGN * 32 == BNW, "wave tile");
  static constexpr int NA = BM / 32, NW = BNW / 32, NB = NA + NW;  // blocks of 32 of the tile
  static constexpr int STAGE_BYTES = NB * 2048;
  static_assert(2 * NB % kWaves == 0, "every wave loads as much");
  static constexpr int LOADS = 2 * NB / kWaves;  // 1 KB loads of a wave and stage
  static constexpr int A_LOADS = 2 * NA / kWaves;
  static_assert(2 * NA % kWaves == 0 && NA % 4 == 0, "a load is of one tensor");
  static constexpr int SC_SLOT = NB * 256;       // scale bytes of a group
  static constexpr int SC_LOADS = (SC_SLOT / 1024 + kWaves - 1) / kWaves;
  static_assert(SC_SLOT % 1024 == 0, "whole loads of scales");
  static_assert(STAGES % 2 == 0 && STAGES >= 4, "whole groups of two stages");
  // scale slots: a group's dwords are in registers before its first product, so
  // its slot is free for the group that the ring brings next
  static constexpr int GROUPS = STAGES / 2;
  static constexpr int SC_OFF = STAGES * STAGE_BYTES;
  static constexpr int JUNK = SC_OFF + GROUPS * SC_SLOT;  // for waves without scales to load
  static constexpr int YLD = BNY + 8;
  static constexpr int Y_BYTES = BM * YLD * 2;
  static constexpr int RING_END = JUNK + 1024;
  static constexpr int LDS_BYTES = RING_END > Y_BYTES ? RING_END : Y_BYTES;
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
  // loads of a stage: the first of a group brings the group's scales
  __host__ __device__ static constexpr int loads(int pos) { return LOADS + (pos % 2 == 0 ? SC_LOADS : 0); }
  // still in flight when the stage after position `pos` has to have landed,
  // with the stages up to pos + STAGES - 1 issued
  __host__ __device__ static constexpr int in_flight(int pos) {
    int n = 0;
    for (int d = 2; d < STAGES; ++d) n += loads(pos + d);
    return n;
  }
  static_assert((STAGES - 1) * (LOADS + SC_LOADS) <= 63, "vmcnt range");
};

template <int BM, int BNW, int STAGES, int WGM, int WGN>
__global__ __launch_bounds__(64 * WGM * WGN) void fp4_tile_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ SA, const uint8_t* __restrict__ W,
    const uint8_t* __restrict__ SW, uint16_t* __restrict__ Y, int M, int N, int K, int group_m) {
  using C = F4Tile<BM, BNW, STAGES, WGM, WGN>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS_BYTES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);
  const int wm = wave_u / WGN, wn = wave_u % WGN;
  const int ntm = (M + BM - 1) / BM, ntn = (N + C::BNY - 1) / C::BNY;
  // bands of group_m tile rows, column after column, contiguous on an XCD
  const int t = xcd_remap(blockIdx.x, gridDim.x);
  const int band = t / (group_m * ntn), in = t % (group_m * ntn);
  const int high = min(ntm - band * group_m, group_m);
  const int tm = band * group_m + in % high, tn = in / high;

  const int G = (K + 255) / 256;   // groups stored
  const int nk = (K + 127) / 128;  // stages
  const int nra = (M + 31) / 32, nrw = (2 * N + 31) / 32;
  const i32x4 rsA = make_rsrc(A, (uint32_t)nra * (uint32_t)G * 4096u);
  const i32x4 rsW = make_rsrc(W, (uint32_t)nrw * (uint32_t)G * 4096u);
  const i32x4 rsSA = make_rsrc(SA, (uint32_t)nra * (uint32_t)G * 256u);
  const i32x4 rsSW = make_rsrc(SW, (uint32_t)nrw * (uint32_t)G * 256u);
  const uint32_t lds0 = lds_addr(smem);

  // Load q of stage `it` into ring position ST: 1 KB (half a stage of one
  // block of 32 rows), A's blocks before W's.  Blocks past a tensor lie past
  // its buffer and give zeros; stages past K are loaded but never multiplied.
  uint32_t off[C::LOADS];
#pragma unroll
  for (int q = 0; q < C::LOADS; ++q) {
    const int c = q * C::kWaves + wave_u, blk = c >> 1;
    const int rb = q < C::A_LOADS ? tm * C::NA + blk : tn * C::NW + blk - C::NA;
    off[q] = (uint32_t)rb * (uint32_t)G * 4096u + (uint32_t)(c & 1) * 1024u + (uint32_t)lane * 16u;
  }
  // scales: load q is of four blocks of 32 rows, of one tensor
  uint32_t sc_off[C::SC_LOADS], sc_dst[C::SC_LOADS];
  i32x4 rsS[C::SC_LOADS];
#pragma unroll
  for (int q = 0; q < C::SC_LOADS; ++q) {
    const int c = q * C::kWaves + wave_u, blk = 4 * c + (lane >> 4);
    const bool a = 4 * c < C::NA, own = c * 1024 < C::SC_SLOT;
    const int rb = a ? tm * C::NA + blk : tn * C::NW + blk - C::NA;
    sc_off[q] = own ? (uint32_t)rb * (uint32_t)G * 256u + (uint32_t)(lane & 15) * 16u : kOutOfRange;
    sc_dst[q] = own ? C::SC_OFF + c * 1024 : C::JUNK;
#pragma unroll
    for (int i = 0; i < 4; ++i) rsS[q][i] = a ? rsSA[i] : rsSW[i];
  }
  auto dma = [&](int it, auto st_c, int q) __attribute__((always_inline)) {
    constexpr int ST = decltype(st_c)::value;
    if (q < C::LOADS) {
      lds_dma16(lds0 + ST * C::STAGE_BYTES + (q * C::kWaves + wave_u) * 1024,
                off[q] + (uint32_t)it * 2048u, q < C::A_LOADS ? rsA : rsW);
    } else {
      const int x = q - C::LOADS;
      const uint32_t slot = sc_dst[x] == C::JUNK ? 0u : (uint32_t)((it >> 1) % C::GROUPS) * C::SC_SLOT;
      lds_dma16(lds0 + sc_dst[x] + slot, sc_off[x] + (uint32_t)(it >> 1) * 256u, rsS[x]);
    }
  };

  u32x4 af[2][C::FA], wf[2][C::FW];
  uint32_t sa[2][C::FA], sw[2][C::FW];  // scale dwords of the group, by group parity
  auto frag = [&](auto st_c, int sub, int r) __attribute__((always_inline)) {
    constexpr int ST = decltype(st_c)::value;
    const uint8_t* st = smem + ST * C::STAGE_BYTES + sub * 1024 + lane * 16;
    if (r < C::FA)
      af[sub][r] = *reinterpret_cast<const u32x4*>(st + (wm * C::FA + r) * 2048);
    else
      wf[sub][r - C::FA] =
          *reinterpret_cast<const u32x4*>(st + (C::NA + wn * C::FW + r - C::FA) * 2048);
  };
  // lane i + 32 h: the dword at [block][h][i]
  auto scales = [&](int group, int p) __attribute__((always_inline)) {
    const uint8_t* s = smem + C::SC_OFF + group % C::GROUPS * C::SC_SLOT + lane * 4;
#pragma unroll
    for (int j = 0; j < C::FA; ++j)
      sa[p][j] = *reinterpret_cast<const uint32_t*>(s + (wm * C::FA + j) * 256);
#pragma unroll
    for (int i = 0; i < C::FW; ++i)
      sw[p][i] = *reinterpret_cast<const uint32_t*>(s + (C::NA + wn * C::FW + i) * 256);
  };

  f32x16 acc[C::FW][C::FA];
#pragma unroll
  for (int i = 0; i < C::FW; ++i)
#pragma unroll
    for (int j = 0; j < C::FA; ++j) acc[i][j] = f32x16{};

  // Stage `it` at position POS of the unrolled loop (ring position POS %
  // STAGES).  Sub-step 0 reads the fragments of sub-step 1; behind the barrier
  // (the next stage has landed, every wave has read this one) sub-step 1 reads
  // the next stage's first fragments and loads stage it + STAGES in this one's
  // place.
  constexpr int NMF = C::FW * C::FA, NFRAG = C::FW + C::FA;
  auto kstep = [&](int it, auto pos_c) __attribute__((always_inline)) {
    constexpr int POS = decltype(pos_c)::value;
    constexpr int ST = POS % STAGES, GP = (POS / 2) & 1;
    using Cur = std::integral_constant<int, ST>;
    using Next = std::integral_constant<int, (ST + 1) % STAGES>;
    auto half = [&](auto sub_c) __attribute__((always_inline)) {
      constexpr int SUB = decltype(sub_c)::value;
      constexpr int B = (POS % 2) * 2 + SUB;  // step of the group: the scale byte
      if constexpr (SUB == 1) {
        wait_vmcnt<C::in_flight(POS)>();
        __syncthreads();
        if constexpr (POS % 2 == 1) scales((it + 1) >> 1, GP ^ 1);
      }
      constexpr int TL = C::loads(POS + STAGES);
      auto slot = [&](auto q_c) __attribute__((always_inline)) {
        constexpr int Q = decltype(q_c)::value;
        constexpr int i = Q / C::FA, j = Q % C::FA;
        acc[i][j] = mfma32_f4<B, B>(wf[SUB][i], af[SUB][j], acc[i][j], sw[GP][i], sa[GP][j]);
#pragma unroll
        for (int x = Q * NFRAG / NMF; x < (Q + 1) * NFRAG / NMF; ++x) {
          if constexpr (SUB == 0) frag(Cur{}, 1, x);
          else frag(Next{}, 0, x);
        }
        if constexpr (SUB == 1) {
#pragma unroll
          for (int x = Q * TL / NMF; x < (Q + 1) * TL / NMF; ++x) dma(it + STAGES, Cur{}, x);
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      [&]<int... Q>(std::integer_sequence<int, Q...>) __attribute__((always_inline)) {
        (slot(std::integral_constant<int, Q>{}), ...);
      }(std::make_integer_sequence<int, NMF>{});
    };
    half(std::integral_constant<int, 0>{});
    half(std::integral_constant<int, 1>{});
  };

  // ---- prologue: all stages of the ring in flight, the first one's fragments ------
  auto fill = [&](auto st_c) __attribute__((always_inline)) {
    constexpr int S = decltype(st_c)::value;
#pragma unroll
    for (int q = 0; q < C::loads(S); ++q) dma(S, st_c, q);
  };
  [&]<int... S>(std::integer_sequence<int, S...>) __attribute__((always_inline)) {
    (fill(std::integral_constant<int, S>{}), ...);
  }(std::make_integer_sequence<int, STAGES>{});
  wait_vmcnt<C::in_flight(2 * STAGES - 1) + C::loads(STAGES - 1)>();
  __syncthreads();
  scales(0, 0);
#pragma unroll
  for (int r = 0; r < NFRAG; ++r) frag(std::integral_constant<int, 0>{}, 0, r);

  // ---- main loop: unrolled over two rings of stages (the parity of the groups) -----
  constexpr int UNR = STAGES % 4 == 0 ? STAGES : 2 * STAGES;
  int it = 0;
  for (; it + UNR <= nk; it += UNR)
    [&]<int... S>(std::integer_sequence<int, S...>) __attribute__((always_inline)) {
      (kstep(it + S, std::integral_constant<int, S>{}), ...);
    }(std::make_integer_sequence<int, UNR>{});
  [&]<int... S>(std::integer_sequence<int, S...>) __attribute__((always_inline)) {
    ((it + S < nk ? (kstep(it + S, std::integral_constant<int, S>{}), 0) : 0), ...);
  }(std::make_integer_sequence<int, UNR - 1>{});

  // ---- epilogue: SiLU(Gate) Up, bf16 tile through LDS, 16-byte row stores ----------
  wait_vmcnt<0>();
  __syncthreads();
  int etid = threadIdx.x;
  asm volatile("" : "+v"(etid));
  const int el = etid & 63;
  uint16_t* ys = reinterpret_cast<uint16_t*>(smem);
#pragma unroll
  for (int i = 0; i < C::FW; ++i)
#pragma unroll
    for (int j = 0; j < C::FA; ++j) {
      const f32x16& d = acc[i][j];
      uint16_t* y = ys + ((wm * C::FA + j) * 32 + (el & 31)) * C::YLD +
                    ((wn * C::FW + i) * 32 + 4 * (el >> 5)) / 2;
#pragma unroll
      for (int q = 0; q < 4; ++q)  // W rows + 8 q + 0 .. 3: Gate, Up, Gate, Up
        *reinterpret_cast<uint32_t*>(y + 4 * q) =
            pack_bf16x2(silu(d[4 * q]) * d[4 * q + 1], silu(d[4 * q + 2]) * d[4 * q + 3]);
    }
  __syncthreads();
  constexpr int YCH = C::BNY / 8;
  for (int p = tid; p < BM * YCH; p += C::kThreads) {
    const int row = p / YCH, cq = p % YCH;
    const int gr = tm * BM + row, gc = tn * C::BNY + cq * 8;
    if (gr < M && gc < N)
      *reinterpret_cast<u32x4*>(Y + (size_t)gr * N + gc) =
          *reinterpret_cast<const u32x4*>(ys + row * C::YLD + cq * 8);
  }
}

// ============================================================================
// The product for few rows: weight streaming
// ============================================================================
// A workgroup takes one block of 32 rows of W and MT blocks of 32 rows of A;
// its NW waves take every NW-th group of 256 k, all of a group's loads (4 KB of
// codes and 256 bytes of scales for each block) issued before its
// first product.  The waves' fp32 sums are added in LDS in wave order, then
// SiLU.  The weights are read once for every 32 MT rows.
template <int MT, int NW>
__global__ __launch_bounds__(64 * NW) void fp4_stream_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ SA, const uint8_t* __restrict__ W,
    const uint8_t* __restrict__ SW, uint16_t* __restrict__ Y, int M, int N, int K) {
  __shared__ __attribute__((aligned(16))) f32x4 red[NW * MT * 4 * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int G = (K + 255) / 256, nra = (M + 31) / 32;
  const int rb = xcd_remap(blockIdx.x, gridDim.x), m0 = blockIdx.y * MT;
  f32x16 acc[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) acc[j] = f32x16{};
  for (int g = wave; g < G; g += NW) {
    u32x4 w[4], a[MT][4];
    uint32_t sa[MT];
    const size_t wb = (size_t)rb * G + g;
    const uint32_t sw = *reinterpret_cast<const uint32_t*>(SW + wb * 256 + lane * 4);
#pragma unroll
    for (int s = 0; s < 4; ++s) w[s] = load16_stream(W + wb * 4096 + s * 1024 + lane * 16);
#pragma unroll
    for (int j = 0; j < MT; ++j) {  // a block past the last repeats it; never stored
      const size_t ab = (size_t)min(m0 + j, nra - 1) * G + g;
      sa[j] = *reinterpret_cast<const uint32_t*>(SA + ab * 256 + lane * 4);
#pragma unroll
      for (int s = 0; s < 4; ++s) a[j][s] = load16(A + ab * 4096 + s * 1024 + lane * 16);
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      acc[j] = mfma32_f4<0, 0>(w[0], a[j][0], acc[j], sw, sa[j]);
      acc[j] = mfma32_f4<1, 1>(w[1], a[j][1], acc[j], sw, sa[j]);
      acc[j] = mfma32_f4<2, 2>(w[2], a[j][2], acc[j], sw, sa[j]);
      acc[j] = mfma32_f4<3, 3>(w[3], a[j][3], acc[j], sw, sa[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      red[((wave * MT + j) * 4 + q) * 64 + lane] =
          f32x4{acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]};
  __syncthreads();
  // quarter q of a lane: W rows 32 rb + 8 q + 4 (lane / 32) + 0 .. 3, that is
  // output columns 16 rb + 4 q + 2 (lane / 32) and + 1 of A's row lane % 32
  for (int x = wave; x < MT * 4; x += NW) {
    f32x4 v = red[x * 64 + lane];
    for (int w = 1; w < NW; ++w) v += red[(w * MT * 4 + x) * 64 + lane];
    const int row = (m0 + x / 4) * 32 + (lane & 31);
    const int col = 16 * rb + 4 * (x % 4) + 2 * (lane >> 5);
    if (row < M && col < N)
      *reinterpret_cast<uint32_t*>(Y + (size_t)row * N + col) =
          pack_bf16x2(silu(v[0]) * v[1], silu(v[2]) * v[3]);
  }
}

// ============================================================================
// Launches
// ============================================================================
template <int BM, int BNW, int STAGES, int WGM, int WGN>
static hipError_t launch_f4_tile(const Fp4Call& c, hipStream_t stream) {
  using C = F4Tile<BM, BNW, STAGES, WGM, WGN>;
  const long long ntm = (c.M + BM - 1) / BM, ntn = (c.N + C::BNY - 1) / C::BNY;
  if (ntm * ntn > 0x7fffffffLL) return hipErrorInvalidValue;
  const int group_m = (int)std::min(ntm, 4LL);
  return launch_op(fp4_tile_kernel<BM, BNW, STAGES, WGM, WGN>, dim3((unsigned)(ntm * ntn)),
                   dim3(C::kThreads), stream, c.A, c.SA, c.W, c.SW, c.Y, (int)c.M, (int)c.N,
                   (int)c.K, group_m);
}
template <int MT, int NW>
static hipError_t launch_f4_stream(const Fp4Call& c, hipStream_t stream) {
  const long long nrb = (2 * c.N + 31) / 32, nmb = (c.M + 32 * MT - 1) / (32 * MT);
  if (nrb > 0x7fffffffLL || nmb > 65535) return hipErrorInvalidValue;
  return launch_op(fp4_stream_kernel<MT, NW>, dim3((unsigned)nrb, (unsigned)nmb), dim3(64 * NW),
                   stream, c.A, c.SA, c.W, c.SW, c.Y, (int)c.M, (int)c.N, (int)c.K);
}

static int fp4_variant(long long M, long long N) {
  auto tiles = [&](long long bm, long long bny) { return (M + bm - 1) / bm * ((N + bny - 1) / bny); };
  if (M <= 32) return 0;
  if (M <= 64) return 1;
  if (tiles(256, 128) >= 200) return 4;
  if (tiles(128, 64) >= 200 || M > 512) return 3;
  return 2;
}

hipError_t launch_forward_mxfp4(const Fp4Call& c, int variant, hipStream_t stream) {
  if (variant < 0) variant = fp4_variant(c.M, c.N);
  switch (variant) {
    case 0: return launch_f4_stream<1, 4>(c, stream);
    case 1: return launch_f4_stream<2, 4>(c, stream);
    case 2: return launch_f4_stream<4, 4>(c, stream);
    case 3: return launch_f4_tile<128, 128, 4, 2, 2>(c, stream);
    default: return launch_f4_tile<256, 256, 4, 2, 4>(c, stream);
  }
}

hipError_t launch_quantize_mxfp4(const uint16_t* X, uint8_t* Q, uint8_t* S, int rows, int K,
                                 hipStream_t stream) {
  const int groups = (K + 255) / 256;
  const long long nw = (long long)((rows + 31) / 32) * groups * 4;
  if (nw > 0x7ffffff0LL) return hipErrorInvalidValue;
  return launch_op(quantize_fp4_kernel, dim3((unsigned)((nw + 3) / 4)), dim3(256), stream, X, Q, S,
                   rows, K, groups, (int)nw);
}
hipError_t launch_dequantize_mxfp4(const uint8_t* Q, const uint8_t* S, uint16_t* X, int rows,
                                   int K, hipStream_t stream) {
  const int groups = (K + 255) / 256;
  const long long nw = (long long)((rows + 31) / 32) * groups * 4;
  if (nw > 0x7ffffff0LL) return hipErrorInvalidValue;
  return launch_op(dequantize_fp4_kernel, dim3((unsigned)((nw + 3) / 4)), dim3(256), stream, Q, S, X,
                   rows, K, groups, (int)nw);
}

}  // namespace swiglu
