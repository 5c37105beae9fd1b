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
// bytes of the four steps as the dword that the format wants.  Bound by memory:
// 8192 x 3584 to codes in 14.5 us (5.1 TB/s of bf16 in and codes out), back in
// 11.7; 128 x 896 in 2.6 and 2.5, which is a launch.
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
    const uint32_t codes = e2m1_codes(v[s], e8m0_scale(e));
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
  uint32_t c[4];  // a group is stored whole, so all four loads are in bounds
#pragma unroll
  for (int s = 0; s < 4; ++s)
    c[s] = *reinterpret_cast<const uint32_t*>(Q + ((((size_t)rg * 4 + s) * 2 + h) * 512 + 16 * i + 4 * q));
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int k = 256 * g + 64 * s + 32 * h;
    if (k >= K) break;
    const int e = (int)((scales >> (8 * s)) & 0xffu);
    const u32x4 v = e == 255 ? u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u}
                             : e2m1_values(c[s], e8m0_scale(e));
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(X + (size_t)row * K + k + 8 * q));
  }
}

// ============================================================================
// The product, LDS-tiled
// ============================================================================
// A tile is BM rows of A against BNW rows of W (Gate and Up rows alternate, so
// a pair is two adjacent registers of a lane), as D = W A^T on
// v_mfma_scale_f32_32x32x64_f8f6f4, which multiplies 4-bit sources at four
// times the bf16 rate and applies the block scales itself.  K runs in stored
// groups of 256 as two stages of 128 k each: 2 KB of every block of 32 rows,
// contiguous in HBM and copied as it is into a ring of two groups in LDS; a
// fragment is one 16-byte read a lane at 16 x lane, without bank conflicts.
// The scales of a group come with its first stage.
//
// At this rate a tile's products are over in about 20 us, so what a tile costs
// beside them shows: one workgroup stays on a CU and walks over tiles, the
// ring running on from one to the next (a tile's last stages already load the
// next one's first), and the output goes to memory straight from registers
// (two lane exchanges give each lane 8 columns of a row), so that LDS stays
// the ring's.  8192 x 18944 x 3584 in 511 to 542 us, by the power the card has left
// (4.1 to 4.4 PFLOP/s; 60 % of the cycles in the matrix pipes at 1.63 GHz; LDS moves
// all of its 128 bytes a clock while they run).
template <int BM, int BNW, int WGM, int WGN>
struct F4Tile {
  static constexpr int kWaves = WGM * WGN, kThreads = 64 * kWaves;
  static constexpr int BNY = BNW / 2;
  static constexpr int FA = BM / WGM / 32, FW = BNW / WGN / 32;  // blocks of 32 a wave
  static_assert(FA >= 1 && FW >= 1 && FA * WGM * 32 == BM && FW * WGN * 32 == BNW, "wave tile");
  static constexpr int NA = BM / 32, NW = BNW / 32, NB = NA + NW;  // blocks of 32 of the tile
  static constexpr int STAGE = NB * 2048, GROUP = 2 * STAGE;       // bytes
  static constexpr int A_LOADS = 2 * NA / kWaves, LOADS = 2 * NB / kWaves;  // 1 KB loads of a wave
  static_assert(2 * NA % kWaves == 0 && 2 * NB % kWaves == 0 && NA % 4 == 0 && NW % 4 == 0,
                "every wave loads as much, a load is of one tensor");
  static constexpr int SC_SLOT = NB * 256;  // scale bytes of a group
  static constexpr int SC_LOADS = (SC_SLOT / 1024 + kWaves - 1) / kWaves;
  static constexpr int SC_OFF = 2 * GROUP;
  static constexpr int JUNK = SC_OFF + 2 * SC_SLOT;  // for waves without scales to load
  static constexpr int LDS_BYTES = JUNK + 1024;
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
  static_assert((GROUP & (GROUP - 1)) == 0, "the ring's two halves differ in one address bit");
  // loads that may be in flight when the stage after this one has to have
  // landed: those of the two stages behind it, one of which has scales
  static constexpr int IN_FLIGHT = 2 * LOADS + SC_LOADS;
};

template <int BM, int BNW, int WGM, int WGN>
__global__ __launch_bounds__(64 * WGM * WGN) void fp4_tile_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ SA, const uint8_t* __restrict__ W,
    const uint8_t* __restrict__ SW, uint16_t* __restrict__ Y, int M, int N, int K, int group_m) {
  using C = F4Tile<BM, BNW, WGM, WGN>;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS_BYTES];
  const int lane = threadIdx.x & 63;
  const int wave_u = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wm = wave_u / WGN, wn = wave_u % WGN;
  const int ntm = (M + BM - 1) / BM, ntn = (N + C::BNY - 1) / C::BNY, ntiles = ntm * ntn;
  // workgroup b runs on XCD b % 8; each XCD owns a contiguous range of tiles,
  // which its workgroups take in turn
  const int wg = blockIdx.x, nwg = gridDim.x, x = wg % 8;
  const int stride = nwg / 8 + (x < nwg % 8 ? 1 : 0);
  const int lo = x * (ntiles / 8) + min(x, ntiles % 8);
  const int end = lo + ntiles / 8 + (x < ntiles % 8 ? 1 : 0);
  const int first = lo + wg / 8;
  if (first >= end) return;

  const int G = (K + 255) / 256;   // groups stored
  const int Gp = max(G, 2);        // groups run: a ring of them at least
  const int nra = (M + 31) / 32, nrw = (2 * N + 31) / 32;
  const i32x4 rsA = make_rsrc(A, (uint32_t)nra * (uint32_t)G * 4096u);
  const i32x4 rsW = make_rsrc(W, (uint32_t)nrw * (uint32_t)G * 4096u);
  const uint32_t lds0 = lds_addr(smem);

  // A tile's position: bands of group_m tile rows, column after column.
  struct Tile {
    int tm, tn;
    uint32_t a, w;  // byte offsets of its first blocks' codes (a 16th for scales)
  };
  auto locate = [&](int t) __attribute__((always_inline)) {
    Tile o{0, 0, kOutOfRange, kOutOfRange};  // past the last tile: zeros
    if (t < end) {
      const int band = t / (group_m * ntn), in = t % (group_m * ntn);
      const int high = min(ntm - band * group_m, group_m);
      o.tm = band * group_m + in % high;
      o.tn = in / high;
      o.a = (uint32_t)(o.tm * C::NA) * (uint32_t)G * 4096u;
      o.w = (uint32_t)(o.tn * C::NW) * (uint32_t)G * 4096u;
    }
    o.tm = __builtin_amdgcn_readfirstlane(o.tm);
    o.tn = __builtin_amdgcn_readfirstlane(o.tn);
    o.a = __builtin_amdgcn_readfirstlane(o.a);
    o.w = __builtin_amdgcn_readfirstlane(o.w);
    return o;
  };

  // This wave's loads of a stage: load q is 1 KB, half a stage of one block of
  // 32 rows, A's blocks before W's.  Blocks past a tensor lie past its buffer
  // and give zeros.
  uint32_t off[C::LOADS];
#pragma unroll
  for (int q = 0; q < C::LOADS; ++q) {
    const int c = q * C::kWaves + wave_u, blk = q < C::A_LOADS ? c >> 1 : (c >> 1) - C::NA;
    off[q] = (uint32_t)blk * (uint32_t)G * 4096u + (uint32_t)(c & 1) * 1024u + (uint32_t)lane * 16u;
  }
  // scales: load q is of four blocks of 32 rows, of one tensor
  uint32_t sc_off[C::SC_LOADS];
  bool sc_a[C::SC_LOADS], sc_own[C::SC_LOADS];
  i32x4 rsS[C::SC_LOADS];
  {
    const i32x4 rsSA = make_rsrc(SA, (uint32_t)nra * (uint32_t)G * 256u);
    const i32x4 rsSW = make_rsrc(SW, (uint32_t)nrw * (uint32_t)G * 256u);
#pragma unroll
    for (int q = 0; q < C::SC_LOADS; ++q) {
      const int c = q * C::kWaves + wave_u, blk = 4 * c + (lane >> 4);
      sc_a[q] = 4 * c < C::NA;
      sc_own[q] = c * 1024 < C::SC_SLOT;
      sc_off[q] = (uint32_t)(sc_a[q] ? blk : blk - C::NA) * (uint32_t)G * 256u + (uint32_t)(lane & 15) * 16u;
#pragma unroll
      for (int i = 0; i < 4; ++i) rsS[q][i] = sc_a[q] ? rsSA[i] : rsSW[i];
    }
  }
  // load q of stage HALF of group g of a tile into ring slot `slot`; groups
  // past K load zeros
  auto dma = [&](const Tile& o, int g, int slot, int half, int q) __attribute__((always_inline)) {
    const bool in = g < G;
    if (q < C::LOADS) {
      const uint32_t at = (q < C::A_LOADS ? o.a : o.w) + (uint32_t)g * 4096u + (uint32_t)half * 2048u;
      lds_dma16(lds0 + slot * C::GROUP + half * C::STAGE + (q * C::kWaves + wave_u) * 1024,
                off[q] + (in ? at : kOutOfRange), q < C::A_LOADS ? rsA : rsW);
    } else {
      const int s = q - C::LOADS;
      const uint32_t base = sc_a[s] ? o.a : o.w;
      const bool there = in && sc_own[s] && base != kOutOfRange;
      lds_dma16(lds0 + (sc_own[s] ? C::SC_OFF + slot * C::SC_SLOT + (s * C::kWaves + wave_u) * 1024
                                  : C::JUNK),
                sc_off[s] + (there ? base / 16u + (uint32_t)g * 256u : kOutOfRange), rsS[s]);
    }
  };

  u32x4 af[2][C::FA], wf[2][C::FW];              // fragments, by sub-step of 64 k
  uint32_t sa[C::FA], sw[C::FW], sa_n[C::FA], sw_n[C::FW];  // a group's scale dwords; the next's
  // where this wave's fragments are in the ring's current slot
  uint32_t fa = (uint32_t)(wm * C::FA * 2048 + lane * 16);
  uint32_t fw = (uint32_t)((C::NA + wn * C::FW) * 2048 + lane * 16);
  auto frag = [&](uint32_t ba, uint32_t bw, int half, int sub, int r) __attribute__((always_inline)) {
    const int at = half * C::STAGE + sub * 1024;
    if (r < C::FA)
      af[sub][r] = *reinterpret_cast<const u32x4*>(smem + ba + (at + r * 2048));
    else
      wf[sub][r - C::FA] = *reinterpret_cast<const u32x4*>(smem + bw + (at + (r - C::FA) * 2048));
  };
  // lane i + 32 h: the dword at [block][h][i]
  auto scales = [&](int slot) __attribute__((always_inline)) {
    const uint8_t* s = smem + C::SC_OFF + slot * C::SC_SLOT + lane * 4;
#pragma unroll
    for (int j = 0; j < C::FA; ++j)
      sa_n[j] = *reinterpret_cast<const uint32_t*>(s + (wm * C::FA + j) * 256);
#pragma unroll
    for (int i = 0; i < C::FW; ++i)
      sw_n[i] = *reinterpret_cast<const uint32_t*>(s + (C::NA + wn * C::FW + i) * 256);
  };
  auto take_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < C::FA; ++j) sa[j] = sa_n[j];
#pragma unroll
    for (int i = 0; i < C::FW; ++i) sw[i] = sw_n[i];
  };
  f32x16 acc[C::FW][C::FA];

  // Sub-step B (64 k) of a group.  The even ones read the other sub-step of
  // their stage; the odd ones wait for the next stage, and behind the barrier
  // (every wave has read this stage) read the next one's first fragments and
  // load the stage of the group after next in this one's place.
  constexpr int NMF = C::FW * C::FA, NFRAG = C::FW + C::FA;
  auto step = [&](auto b_c, const Tile& o, int g, int slot) __attribute__((always_inline)) {
    constexpr int B = decltype(b_c)::value, SUB = B & 1, HALF = B >> 1;
    constexpr int TL = C::LOADS + (HALF == 0 ? C::SC_LOADS : 0);
    if constexpr (SUB == 1) {
      wait_vmcnt<C::IN_FLIGHT>();
      __syncthreads();
      if constexpr (HALF == 1) scales(slot ^ 1);
    }
    const uint32_t na = HALF == 1 && SUB == 1 ? fa ^ C::GROUP : fa;
    const uint32_t nw = HALF == 1 && SUB == 1 ? fw ^ C::GROUP : fw;
    auto one = [&](auto q_c) __attribute__((always_inline)) {
      constexpr int Q = decltype(q_c)::value, i = Q / C::FA, j = Q % C::FA;
      acc[i][j] = mfma32_f4<B, B>(wf[SUB][i], af[SUB][j], acc[i][j], sw[i], sa[j]);
#pragma unroll
      for (int r = Q * NFRAG / NMF; r < (Q + 1) * NFRAG / NMF; ++r)
        frag(na, nw, SUB == 0 ? HALF : HALF ^ 1, SUB ^ 1, r);
      if constexpr (SUB == 1) {
#pragma unroll
        for (int q = Q * TL / NMF; q < (Q + 1) * TL / NMF; ++q) dma(o, g, slot, HALF, q);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    [&]<int... Q>(std::integer_sequence<int, Q...>) __attribute__((always_inline)) {
      (one(std::integral_constant<int, Q>{}), ...);
    }(std::make_integer_sequence<int, NMF>{});
  };

  // ---- the first tile's first two groups, and the fragments of its first stage -----
  Tile cur = locate(first), nxt = cur;
#pragma unroll
  for (int st = 0; st < 4; ++st) {
#pragma unroll
    for (int q = 0; q < C::LOADS + (st % 2 == 0 ? C::SC_LOADS : 0); ++q)
      dma(cur, st / 2, st / 2, st % 2, q);
  }
  wait_vmcnt<3 * C::LOADS + C::SC_LOADS>();
  __syncthreads();
  scales(0);
#pragma unroll
  for (int r = 0; r < NFRAG; ++r) frag(fa, fw, 0, 0, r);

  int slot = 0;
  for (int t = first; t < end; t += stride) {
    nxt = locate(t + stride);
#pragma unroll
    for (int i = 0; i < C::FW; ++i)
#pragma unroll
      for (int j = 0; j < C::FA; ++j) acc[i][j] = f32x16{};
    for (int g = 0; g < Gp; ++g) {
      take_scales();
      const bool over = g + 2 >= Gp;  // the group to load is the next tile's
      const Tile o{0, 0, over ? nxt.a : cur.a, over ? nxt.w : cur.w};
      const int lg = over ? g + 2 - Gp : g + 2;
      step(std::integral_constant<int, 0>{}, o, lg, slot);
      step(std::integral_constant<int, 1>{}, o, lg, slot);
      step(std::integral_constant<int, 2>{}, o, lg, slot);
      step(std::integral_constant<int, 3>{}, o, lg, slot);
      fa ^= C::GROUP;
      fw ^= C::GROUP;
      slot ^= 1;
    }
    // SiLU(Gate) Up of this tile.  Registers 4 q .. 4 q + 3 are W rows 8 q + 4 h
    // + 0 .. 3 (h = lane / 32), i.e. output columns 4 q + 2 h and + 1; the
    // exchanges leave columns 0 .. 7 of the block of 16 in the lower half of
    // the wave, 8 .. 15 in the upper one.
#pragma unroll
    for (int j = 0; j < C::FA; ++j) {
      const int row = cur.tm * BM + (wm * C::FA + j) * 32 + (lane & 31);
#pragma unroll
      for (int i = 0; i < C::FW; ++i) {
        const f32x16& d = acc[i][j];
        uint32_t p[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          p[q] = pack_bf16x2(silu(d[4 * q]) * d[4 * q + 1], silu(d[4 * q + 2]) * d[4 * q + 3]);
        swap_halves(p[0], p[2]);
        swap_halves(p[1], p[3]);
        const int col = cur.tn * C::BNY + (wn * C::FW + i) * 16 + 8 * (lane >> 5);
        if (row < M && col < N)
          *reinterpret_cast<u32x4*>(Y + (size_t)row * N + col) = u32x4{p[0], p[2], p[1], p[3]};
      }
    }
    cur = nxt;
  }
  // the zero loads issued past the last tile still write LDS
  wait_vmcnt<0>();
}

// ============================================================================
// The product for few rows: weight streaming
// ============================================================================
// A workgroup takes one block of 32 rows of W and MT blocks of 32 rows of A;
// its NW waves take every NW-th group of 256 k, all of a group's loads (4 KB of
// codes and 256 bytes of scales for each block) issued before its
// first product.  The waves' fp32 sums are added in LDS in wave order, then
// SiLU.  The weights are read once for every 32 MT rows.  Eight waves: four gave
// 16.0 instead of 15.2 us at 16 x 18944 x 3584, 7.3 instead of 5.9 at 50 x 4000 x
// 3584.
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
template <int BM, int BNW, int WGM, int WGN>
static hipError_t launch_f4_tile(const Fp4Call& c, hipStream_t stream) {
  using C = F4Tile<BM, BNW, WGM, WGN>;
  const long long ntm = (c.M + BM - 1) / BM, ntn = (c.N + C::BNY - 1) / C::BNY;
  if (ntm * ntn > 0x7fffffffLL) return hipErrorInvalidValue;
  const int group_m = (int)std::min(ntm, 4LL);
  const int per_cu = C::LDS_BYTES <= 80 * 1024 ? 2 : 1;
  // eight at least: each XCD's range of tiles needs a workgroup there
  const long long wgs = std::min<long long>(ntm * ntn, std::max<long long>((long long)c.cu_count * per_cu, 8));
  return launch_op(fp4_tile_kernel<BM, BNW, WGM, WGN>, dim3((unsigned)wgs), dim3(C::kThreads),
                   stream, c.A, c.SA, c.W, c.SW, c.Y, (int)c.M, (int)c.N, (int)c.K, group_m);
}
template <int MT, int NW>
static hipError_t launch_f4_stream(const Fp4Call& c, hipStream_t stream) {
  const long long nrb = (2 * c.N + 31) / 32, nmb = (c.M + 32 * MT - 1) / (32 * MT);
  if (nrb > 0x7fffffffLL || nmb > 65535) return hipErrorInvalidValue;
  return launch_op(fp4_stream_kernel<MT, NW>, dim3((unsigned)nrb, (unsigned)nmb), dim3(64 * NW),
                   stream, c.A, c.SA, c.W, c.SW, c.Y, (int)c.M, (int)c.N, (int)c.K);
}

// Few rows stream the weights, and so do calls too small to give a quarter of
// the CUs a small tile (us, variants 1 / 2: 50 x 4000 x 3584 5.9 / 9.8, 300 x 800 x
// 3584 6.5 / 9.7, 100 x 2400 x 3584 9.1 / 9.7, 2000 x 200 x 2048 8.7 / 7.2, 64 x 18944 x
// 3584 19.9 / 17.4).
// Otherwise the large tiles (one workgroup a CU)
// run 1.25 times as fast as the small ones (two a CU), but in whole rounds: of
// the time of one large tile, they take ceil(tiles / CUs), the small ones about
// 0.59 for every two a CU and half of that more for the end.  Measured (us,
// large / small): 8192 x 18944 x 3584 542 / 659 (18.5 rounds), 4620 x 1528 x 1504
// 18.7 / 22.3 (0.9), 1024 x 4864 x 896 11.9 / 10.3 (0.6), 2048 x 8960 x 1536 45.0 /
// 39.6 (2.2), 512 x 18944 x 3584 53.1 / 43.4 (1.2).
static int fp4_variant(long long M, long long N, int cu_count) {
  auto tiles = [&](long long bm, long long bny) { return (M + bm - 1) / bm * ((N + bny - 1) / bny); };
  const long long small = tiles(128, 64), large = tiles(256, 128), cus = std::max(cu_count, 1);
  if (M <= 32) return 0;
  if (small < (M <= 64 ? 200 : 64)) return 1;
  const double t_large = (double)((large + cus - 1) / cus);
  const double t_small = 0.59 * ((double)small / (2.0 * cus) + 0.5);
  return t_large <= t_small ? 3 : 2;
}

hipError_t launch_forward_mxfp4(const Fp4Call& c, int variant, hipStream_t stream) {
  if (variant < 0) variant = fp4_variant(c.M, c.N, c.cu_count);
  switch (variant) {
    case 0: return launch_f4_stream<1, 8>(c, stream);
    case 1: return launch_f4_stream<2, 8>(c, stream);
    case 2: return launch_f4_tile<128, 128, 2, 2>(c, stream);
    default: return launch_f4_tile<256, 256, 2, 4>(c, stream);
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
